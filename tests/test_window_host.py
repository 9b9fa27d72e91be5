"""Windowed calls and rotary positions on the CPU: their plain 64-bit forms
against torch, argument checks, the allocator's trimming (no GPU needed)."""
import ctypes

import numpy as np
import pytest

import window_reference as wr
import workloads as wl

torch = pytest.importorskip("torch")
pk = pytest.importorskip("paged_kv_cache_425_b200")


# ---------------------------------------------------------------- the plain forms
@pytest.mark.parametrize("window,sinks", [(1, 0), (7, 3), (64, 20), (1000, 0)])
def test_plain_window_matches_masked_attention(window, sinks):
    p = wr.Windowed(wl.rng_for(1), [50, 9, 0], [20, 9, 0], 6, 2, 16, wl.F16, window, sinks)
    out, _ = p.reference()
    for s, (L, n) in enumerate(zip(p.lens, p.chunk)):
        if n == 0:
            continue
        rows = slice(p.start[s], p.start[s + 1])
        q = torch.from_numpy(wr.to_f64(p.q[rows], p.dtype)).transpose(0, 1)
        k = torch.from_numpy(wr.to_f64(p.k[s], p.dtype)).transpose(0, 1).repeat_interleave(3, 0)
        v = torch.from_numpy(wr.to_f64(p.v[s], p.dtype)).transpose(0, 1).repeat_interleave(3, 0)
        mask = torch.zeros(n, L, dtype=torch.bool)
        for i in range(n):
            for j in range(L):
                at = L - n + i
                mask[i, j] = bool(j <= at and (j > at - window or j < sinks))
        ref = torch.nn.functional.scaled_dot_product_attention(q, k, v, attn_mask=mask, scale=p.scale)
        assert np.allclose(out[rows], ref.transpose(0, 1).numpy(), rtol=0, atol=1e-12)


def test_plain_rotation_matches_complex_numbers():
    rng = wl.rng_for(2)
    x = rng.standard_normal((5, 3, 32))
    pos = rng.integers(0, 1000, size=(2, 5))
    freq = np.array([1.0, 0.5, 0.25, 0.1, 0.01, 0.001, 0.3, 0.7], np.float32)
    axes = [0, 1, 0, 1, 1, 0, 0, 1]
    for inter in (False, True):
        y = wr.rotate(x, pos, freq, axes, inter)
        for i in range(8):
            a, b = (2 * i, 2 * i + 1) if inter else (i, i + 8)
            z = (x[..., a] + 1j * x[..., b]) * np.exp(1j * pos[axes[i]] * float(freq[i]))[:, None]
            assert np.allclose(y[..., a], z.real, atol=1e-11) and np.allclose(y[..., b], z.imag, atol=1e-11)
        assert np.array_equal(y[..., 16:], x[..., 16:])


# ---------------------------------------------------------------- workspace sizes
def test_workspace_sizes():
    size = pk.decode_window_workspace_size
    assert size(64, 32, 32, 128, 128, 100) == 0                   # one partition sees it all
    assert size(1, 32, 8, 128, 2048, 8192, 4) == 0                # few rows: one cluster each
    assert size(100, 32, 8, 128, 2048, 8192, 4) > 0
    assert size(64, 32, 32, 128, 1 << 20, 2 ** 31 - 1, 2 ** 31 - 1) > 0
    # the table bounds what a window can see
    assert size(100, 8, 8, 64, 400, 100000) == size(100, 8, 8, 64, 400, 6400) > 0
    assert size(1, 8, 8, 64, 4, 0) == 0 and size(1, 8, 8, 64, 4, 5, -1) == 0
    pre = pk.prefill_window_workspace_size
    assert pre(16, 8192, 512, 32, 8, 128, 1024, 4096) == 0        # enough work without a split
    assert pre(1, 512, 512, 32, 8, 128, 1024, 4096) == 0          # as items of half the rows
    assert pre(1, 256, 256, 32, 8, 128, 1024, 4096) > 0
    assert pre(1, 1, 512, 32, 8, 128, 1024, 4096) == pre(1, 1, 1, 32, 8, 128, 1024, 4096)
    assert pre(1, 5, 5, 6, 0, 64, 8, 5) == 0 and pre(1, 5, 5, 512, 1, 64, 8, 5) == 0
    with pytest.raises(ValueError):
        size(1, 8, 8, 64, 4, 2 ** 31)
    # head counts no call accepts: no plan, and no division by zero on the way
    for hq, hkv in ((4, 8), (0, 4), (300, 1), (7, 2), (-8, 2), (8, -2), (17, 1)):
        assert size(100, hq, hkv, 64, 1000, 9000) == 0
    for hq, hkv in ((4, 8), (0, 4), (300, 1), (7, 2), (-8, 2), (8, -2), (129, 1)):
        assert pre(1, 512, 512, hq, hkv, 64, 1000, 9000) == 0
    assert pre(1, 512, 512, 128, 1, 64, 1000, 9000) >= 0
    big = 2 ** 31 - 1
    assert size(100, 8, 8, 64, big, big, big) == 0 and pre(1, 9, 9, 8, 8, 64, big, big, big) == 0


# ---------------------------------------------------------------- refusals (before any launch)
P = ctypes.c_void_p(4096)  # aligned, never dereferenced: every call below is refused
ODD = ctypes.c_void_p(4096 + 8)


def decode_status(**kw):
    a = dict(out=P, q=P, k_new=P, v_new=P, kc=P, vc=P, tbl=P, lens=P, window=64, sinks=4, hkv=2,
             scale=0.1, S=3, hq=8, d=64, bs=16, maxb=64, nb=100, dtype=0, ws=None, wsb=0)
    a.update(kw)
    tail = (a["tbl"], a["lens"], a["window"], a["sinks"], a["hkv"], a["scale"], a["S"], a["hq"], a["d"],
            a["bs"], a["maxb"], a["nb"], a["dtype"], a["ws"], a["wsb"], None)
    plain = pk.pa_decode_window(a["out"], a["q"], a["kc"], a["vc"], *tail)
    app = pk.pa_decode_append_window(a["out"], a["q"], a["k_new"], a["v_new"], a["kc"], a["vc"], *tail)
    return plain, app


@pytest.mark.parametrize("change,status", [
    (dict(window=0), pk.PA_ERR_INVALID_ARG), (dict(window=-5), pk.PA_ERR_INVALID_ARG),
    (dict(sinks=-1), pk.PA_ERR_INVALID_ARG), (dict(q=ODD), pk.PA_ERR_INVALID_ARG),
    (dict(out=ODD), pk.PA_ERR_INVALID_ARG), (dict(kc=ODD), pk.PA_ERR_INVALID_ARG),
    (dict(q=None), pk.PA_ERR_INVALID_ARG), (dict(tbl=None), pk.PA_ERR_INVALID_ARG),
    (dict(hq=9), pk.PA_ERR_INVALID_ARG), (dict(hq=34), pk.PA_ERR_UNSUPPORTED),
    (dict(d=96), pk.PA_ERR_UNSUPPORTED), (dict(bs=32), pk.PA_ERR_UNSUPPORTED),
    (dict(dtype=2), pk.PA_ERR_UNSUPPORTED), (dict(maxb=(1 << 26) + 1), pk.PA_ERR_UNSUPPORTED),
    (dict(S=100, window=5000, maxb=1000), pk.PA_ERR_WORKSPACE),
    (dict(S=100, window=5000, maxb=1000, ws=P, wsb=100), pk.PA_ERR_WORKSPACE),
    (dict(S=100, window=5000, maxb=1000, ws=ODD, wsb=1 << 30), pk.PA_ERR_WORKSPACE),
])
def test_decode_window_refusals(change, status):
    assert decode_status(**change) == (status, status)


def test_decode_append_window_refuses_bad_new_rows():
    for kw in (dict(k_new=None), dict(v_new=ODD)):
        assert decode_status(q=P, S=100, window=5000, maxb=1000, **kw) == (pk.PA_ERR_WORKSPACE,
                                                                        pk.PA_ERR_INVALID_ARG)


def test_windowed_calls_with_nothing_to_do():
    assert decode_status(S=0, out=None, q=None) == (0, 0)
    assert prefill_status(S=0) == 0 and prefill_status(rows=0) == 0 and prefill_status(max_len=0) == 0


def prefill_status(**kw):
    a = dict(out=P, q=P, kc=P, vc=P, tbl=P, lens=P, start=P, max_len=100, window=64, sinks=4, hkv=2,
             scale=0.1, S=3, hq=8, rows=300, d=64, bs=16, maxb=64, nb=100, dtype=0, ws=None, wsb=0)
    a.update(kw)
    return pk.pa_prefill_window(a["out"], a["q"], a["kc"], a["vc"], a["tbl"], a["lens"], a["start"],
                                a["max_len"], a["window"], a["sinks"], a["hkv"], a["scale"], a["S"],
                                a["hq"], a["rows"], a["d"], a["bs"], a["maxb"], a["nb"], a["dtype"],
                                a["ws"], a["wsb"], None)


@pytest.mark.parametrize("change,status", [
    (dict(window=0), pk.PA_ERR_INVALID_ARG), (dict(sinks=-1), pk.PA_ERR_INVALID_ARG),
    (dict(scale=0.0), pk.PA_ERR_UNSUPPORTED), (dict(scale=-1.0), pk.PA_ERR_UNSUPPORTED),
    (dict(scale=float("nan")), pk.PA_ERR_UNSUPPORTED), (dict(scale=float("inf")), pk.PA_ERR_UNSUPPORTED),
    (dict(hq=2 * 129), pk.PA_ERR_UNSUPPORTED), (dict(hq=7), pk.PA_ERR_INVALID_ARG),
    (dict(q=ODD), pk.PA_ERR_INVALID_ARG), (dict(out=ODD), pk.PA_ERR_INVALID_ARG),
    (dict(start=None), pk.PA_ERR_INVALID_ARG), (dict(max_len=-1), pk.PA_ERR_INVALID_ARG),
    (dict(maxb=(1 << 26) + 1), pk.PA_ERR_UNSUPPORTED),
    (dict(S=100, max_len=1, rows=100, window=5000, maxb=1000), pk.PA_ERR_WORKSPACE),
    (dict(S=1, window=5000, maxb=1000), pk.PA_ERR_WORKSPACE),
])
def test_prefill_window_refusals(change, status):
    assert prefill_status(**change) == status


def rope_status(rope=None, **kw):
    a = dict(qo=P, q=P, k=P, v=P, kc=P, vc=P, slots=P, pos=P, qs=512, ks=128, vs=128, T=3, hq=8, hkv=2,
             d=64, bs=16, nb=10, dtype=0)
    a.update(kw)
    rope = rope or pk.Rope(np.ones(32))
    return pk.pa_rope_and_cache(a["qo"], a["q"], a["k"], a["v"], a["kc"], a["vc"], a["slots"], a["pos"],
                                rope._ref, a["qs"], a["ks"], a["vs"], a["T"], a["hq"], a["hkv"], a["d"],
                                a["bs"], a["nb"], a["dtype"], None)


@pytest.mark.parametrize("change,status", [
    (dict(q=None), pk.PA_ERR_INVALID_ARG), (dict(qo=ODD), pk.PA_ERR_INVALID_ARG),
    (dict(k=ODD), pk.PA_ERR_INVALID_ARG), (dict(ks=132), pk.PA_ERR_INVALID_ARG),
    (dict(vs=-8), pk.PA_ERR_INVALID_ARG), (dict(pos=None), pk.PA_ERR_INVALID_ARG),
    (dict(T=-1), pk.PA_ERR_INVALID_ARG), (dict(d=80), pk.PA_ERR_UNSUPPORTED),
    (dict(T=0, q=None), pk.PA_OK),
])
def test_rope_refusals(change, status):
    assert rope_status(**change) == status


def test_rope_plans_are_checked():
    assert rope_status(rope=pk.Rope(np.ones(64)), d=64) == pk.PA_ERR_INVALID_ARG  # 128 of 64 elements
    for args, status in [((np.ones(12),), pk.PA_ERR_UNSUPPORTED), ((np.ones(72),), pk.PA_ERR_UNSUPPORTED),
                         ((np.full(8, np.inf),), pk.PA_ERR_INVALID_ARG),
                         ((np.ones(8), [0] * 7 + [8]), pk.PA_ERR_UNSUPPORTED),
                         ((np.ones(8), [-1] + [0] * 7), pk.PA_ERR_INVALID_ARG)]:
        with pytest.raises(pk.PagedError) as e:
            pk.Rope(*args)
        assert e.value.status == status
    with pytest.raises(ValueError):
        pk.Rope(np.ones(8), [0] * 7)
    assert pk.Rope(np.ones(8), [0] * 8, num_axes=3).num_axes == 3


def test_rope_turns_wrap_exactly():
    """Position times the 64-bit fraction of a turn, against 80-bit arithmetic."""
    freq = np.array([1.0, 0.5, 1e-4, 7.25, -0.3, 3e-7, 100.0, 0.0], np.float32)
    r = pk.Rope(freq)
    turn = np.longdouble("6.28318530717958647692528676655900576839433879875021")
    for p in (0, 1, 17, 2 ** 31 - 1, -2 ** 31):
        for i, f in enumerate(freq):
            got = ((p * r._struct.turns[i]) % 2 ** 64) / 2.0 ** 64
            want = np.longdouble(p) * np.longdouble(f) / turn
            want = float(want - np.floor(want))
            d = abs(got - want)
            assert min(d, 1 - d) < 2.0 ** -26


# ---------------------------------------------------------------- trimming
def test_trim_drops_exactly_the_unseen_blocks():
    for window, sinks in [(1, 0), (16, 0), (17, 5), (40, 16), (33, 40), (500, 1)]:
        for L in (1, 16, 17, 64, 130):
            a = pk.BlockAllocator(64)
            a.add_seq(7, L)
            before = a.block_table(7)
            for at in (0, L // 2, L - 1, L):
                n = a.trim_window(7, at, window, sinks)
                table = a.block_table(7)
                # what any query from position `at` on can see
                vis = wr.seen(np.arange(at, at + 200), np.arange(len(table) * 16), window, sinks).any(0)
                for b in range(len(table)):
                    gone = not vis[16 * b:16 * b + 16].any()
                    assert (table[b] == -1) == gone, (window, sinks, L, at, b)
                    if not gone:
                        assert table[b] == before[b]
                assert a.stats()["used_blocks"] == (table >= 0).sum()
                assert n <= len(table)
            slot, pair = a.append_slot(7)
            assert pair == (-1, -1) and slot == a.block_table(7)[L // 16] * 16 + L % 16
            a.free_seq(7)
            assert a.stats()["free_blocks"] == 64


def test_trim_refusals():
    a = pk.BlockAllocator(8)
    a.add_seq(1, 40)
    for args in [(2, 0, 4, 0), (1, -1, 4, 0), (1, 41, 4, 0), (1, 40, 0, 0), (1, 40, 4, -1)]:
        with pytest.raises(pk.PagedError):
            a.trim_window(*args)
    assert (a.block_table(1) >= 0).all()
    assert a.trim_window(1, 40, 2 ** 31 - 1, 2 ** 31 - 1) == 0


def test_trim_with_forks_and_copy_on_write():
    a = pk.BlockAllocator(16)
    a.add_seq(0, 70)  # 5 blocks
    a.fork(0, 1)
    assert a.trim_window(0, 70, 10, 0) == 3
    assert a.stats()["used_blocks"] == 5  # the other branch still holds them
    a.fork(0, 2)                          # a trimmed parent: shares what is left
    assert list(a.block_table(2)[:3]) == [-1] * 3
    assert a.trim_window(1, 70, 10, 0) == 3 and a.trim_window(1, 70, 10, 0) == 0
    assert a.stats()["used_blocks"] == 2
    _, (src, dst) = a.append_slot(2)
    assert src >= 0 and dst >= 0
    tables, lens = a.build_tables([0, 1, 2], 6)
    assert (tables[:, :3] == -1).all() and list(lens) == [70, 70, 71]
    for s in (0, 1, 2):
        a.free_seq(s)
    st = a.stats()
    assert st["free_blocks"] == 16 and st["logical_blocks"] == 0


def test_trimmed_prefix_blocks_stay_findable():
    a = pk.BlockAllocator(8)
    a.enable_prefix_caching()
    tokens = np.arange(64)
    assert a.add_seq_tokens(0, tokens) == 0
    assert a.trim_window(0, 64, 16, 0) == 3
    assert a.add_seq_tokens(1, tokens) == 64  # all four again, three off the free list
    assert a.stats()["used_blocks"] == 4
    a.free_seq(0)
    a.free_seq(1)
    assert a.stats()["free_blocks"] == 8


def test_random_trims_keep_the_pool_consistent():
    rng = np.random.default_rng(3)
    a = pk.BlockAllocator(200)
    live, nxt = {}, 0
    for _ in range(3000):
        op = rng.integers(0, 5)
        if op == 0 or not live:
            n = int(rng.integers(0, 120))
            if a.stats()["free_blocks"] >= -(-n // 16):
                a.add_seq(nxt, n)
                live[nxt] = n
                nxt += 1
        else:
            s = int(rng.choice(list(live)))
            if op == 1:
                a.free_seq(s)
                del live[s]
            elif op == 2 and a.stats()["free_blocks"]:
                a.append_slot(s)
                live[s] += 1
            elif op == 3:
                a.trim_window(s, int(rng.integers(0, live[s] + 1)), int(rng.integers(1, 60)),
                              int(rng.integers(0, 40)))
            elif op == 4:
                a.fork(s, nxt)
                live[nxt] = live[s]
                nxt += 1
        count = np.zeros(200, int)
        for t in live:
            b = a.block_table(t)
            np.add.at(count, b[b >= 0], 1)
        assert [a.refcount(b) for b in range(200)] == list(count)
        st = a.stats()
        assert st["used_blocks"] == (count > 0).sum() and st["free_blocks"] == 200 - st["used_blocks"]


# ---------------------------------------------------------------- the binding's own checks
def binding_args(**kw):
    a = dict(out=torch.zeros(2, 4, 64, dtype=torch.float16), q=torch.zeros(2, 4, 64, dtype=torch.float16),
             kc=torch.zeros(8, 2, 16, 64, dtype=torch.float16), vc=torch.zeros(8, 2, 16, 64, dtype=torch.float16),
             tbl=torch.zeros(2, 4, dtype=torch.int32), lens=torch.ones(2, dtype=torch.int32), hkv=2)
    a.update(kw)
    return a["out"], a["q"], a["kc"], a["vc"], a["tbl"], a["lens"], a["hkv"], 0.1, 16


@pytest.mark.parametrize("change", [
    dict(q=torch.zeros(2, 4, 32, dtype=torch.float16)), dict(out=torch.zeros(2, 5, 64, dtype=torch.float16)),
    dict(lens=torch.ones(3, dtype=torch.int32)), dict(hkv=4),
    dict(vc=torch.zeros(8, 2, 16, 32, dtype=torch.float16)),
    dict(),  # host tensors
])
def test_binding_refuses_before_the_library(change):
    with pytest.raises(ValueError):
        pk.decode_window(*binding_args(**change))


def test_packed_arguments_match_the_structures():
    """The packed formats are the C structures: the same refusals through both."""
    def call(window, call=pk.WINDOW_DECODE, maxb=64):
        return pk.pa_window_call(pk._pack_window(4096, 4096, 0, 0, 4096, 4096, 4096, 4096, 4096, 0, 0, 0, 100,
                                                 call, window, 4, 2, 0, 8, 300, 100, 64, 16, maxb, 0, 0.1))
    assert call(64) == pk.PA_OK  # no sequences: nothing to do
    assert call(0) == pk.PA_ERR_INVALID_ARG and call(64, call=3) == pk.PA_ERR_INVALID_ARG
    assert call(64, maxb=(1 << 26) + 1) == pk.PA_ERR_UNSUPPORTED
    assert call(64, call=pk.WINDOW_PREFILL) == pk.PA_OK
    assert call(-1, call=pk.WINDOW_PREFILL) == pk.PA_ERR_INVALID_ARG
    rope = pk.Rope(np.ones(32))

    def rope_call(T, d=64, ks=128):
        return pk.pa_rope_call(pk._pack_rope(4096, 4096, 4096, 4096, 4096, 4096, 4096, 4096, rope._address, 0, 512,
                                             ks, 128, 10, T, 8, 2, d, 16, 0))
    assert rope_call(0) == pk.PA_OK and rope_call(-1) == pk.PA_ERR_INVALID_ARG
    assert rope_call(3, d=96) == pk.PA_ERR_UNSUPPORTED and rope_call(3, ks=129) == pk.PA_ERR_INVALID_ARG
    assert pk._lib.pa_window_call(None) == pk.PA_ERR_INVALID_ARG
    assert pk._lib.pa_rope_call(None) == pk.PA_ERR_INVALID_ARG
