"""Windowed attention on the GPU against its plain 64-bit form: decode, decode
with the new token's write, chunked prefill.  Wherever no query looks the pool
holds NaN and infinities, and table entries no query needs are -1."""
import numpy as np
import pytest

import workloads as wl
from window_reference import BS, Windowed

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import gpu_harness as gh  # noqa: E402

pk = pytest.importorskip("paged_kv_cache_425_b200")


def device(p):
    return dict(kc=gh.to_dev(p.key_cache, p.dtype), vc=gh.to_dev(p.value_cache, p.dtype),
                tbl=gh.ints(p.tables), lens=gh.ints(p.lens), q=gh.to_dev(p.q, p.dtype))


def scratch(n):
    # NaN bytes: nothing in a workspace has to start at zero
    return torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda") if n else None


def decode_ws(p):
    return scratch(pk.decode_window_workspace_size(len(p.lens), p.hq, p.hkv, p.d, p.tables.shape[1],
                                                   p.window, p.sinks))


def run_decode(p, stream=None):
    t = device(p)
    # one row per sequence, the empty ones too
    q = torch.zeros((len(p.lens), p.hq, p.d), dtype=t["q"].dtype, device="cuda")
    live = torch.from_numpy(p.chunk > 0).cuda()
    q[live] = t["q"]
    out = torch.full_like(q, float("nan"))
    pk.decode_window(out, q, t["kc"], t["vc"], t["tbl"], t["lens"], p.hkv, p.scale, p.window, p.sinks,
                     workspace=decode_ws(p), stream=stream)
    torch.cuda.synchronize()
    assert pk.get_error() == (0, 0)
    return out, live


def run_prefill(p, max_len=None, rows=None):
    t = device(p)
    rows = rows or t["q"].shape[0]
    q = torch.full((rows, p.hq, p.d), float("nan"), dtype=t["q"].dtype, device="cuda")
    q[:t["q"].shape[0]] = t["q"]
    out = torch.full_like(q, float("nan"))
    max_len = max_len or int(p.chunk.max())
    n = pk.prefill_window_workspace_size(len(p.lens), rows, max_len, p.hq, p.hkv, p.d,
                                         p.tables.shape[1], p.window, p.sinks)
    pk.prefill_window(out, q, t["kc"], t["vc"], t["tbl"], t["lens"], gh.ints(p.start), max_len, p.hkv,
                      p.scale, p.window, p.sinks, workspace=scratch(n))
    torch.cuda.synchronize()
    return out


def assert_close(got, p):
    ref, tol = p.reference()
    g = gh.to_f64(got)
    assert np.all(np.isfinite(g))
    worst = np.max(np.abs(g - ref) / tol) if g.size else 0.0
    assert worst <= 1.0, f"error {worst:.3f} of the tolerance"


LENS = [0, 1, 2, 15, 16, 17, 31, 33, 64, 100, 257, 700, 1025]
SHAPES = [(4, 4, 64, wl.F16), (8, 2, 128, wl.BF16), (7, 1, 128, wl.F16), (12, 1, 64, wl.BF16),
          (32, 2, 128, wl.BF16)]


# ---------------------------------------------------------------- decode
@pytest.mark.parametrize("hq,hkv,d,dtype", SHAPES)
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (5, 4), (16, 0), (17, 16), (100, 33),
                                          (512, 5), (2 ** 31 - 1, 0), (3, 2 ** 31 - 1)])
def test_decode_window(hq, hkv, d, dtype, window, sinks):
    rng = wl.rng_for(window % 1000 + sinks % 1000 + hq)
    chunk = np.minimum(LENS, 1)
    p = Windowed(rng, LENS, chunk, hq, hkv, d, dtype, window, sinks)
    out, live = run_decode(p)
    assert_close(out[live], p)
    assert not out[~live].any()  # empty contexts: zero rows


@pytest.mark.parametrize("hq,hkv,d,dtype", SHAPES)
def test_decode_window_every_alignment(hq, hkv, d, dtype):
    """Each place of the window's first token and of the sinks' last in a block."""
    for window in (15, 16, 18):
        lens = np.arange(1, 97)
        p = Windowed(wl.rng_for(window), lens, np.ones(96, int), hq, hkv, d, dtype, window, window - 9)
        out, live = run_decode(p)
        assert_close(out, p)


@pytest.mark.parametrize("hq,hkv,d,dtype", [(8, 1, 128, wl.BF16), (4, 4, 64, wl.F16), (16, 1, 128, wl.F16)])
@pytest.mark.parametrize("window", [1000, 6000, 20000])
def test_decode_window_of_many_partitions(hq, hkv, d, dtype, window):
    p = Windowed(wl.rng_for(window), [9000, 20001, 37], [1, 1, 1], hq, hkv, d, dtype, window, 21)
    out, _ = run_decode(p)
    assert_close(out, p)
    again, _ = run_decode(p)
    assert torch.equal(out, again)


def test_decode_window_wide_enough_equals_decode():
    rng = wl.rng_for(5)
    lens = [700, 1, 33]
    p = Windowed(rng, lens, [1, 1, 1], 8, 2, 128, wl.BF16, 5000, 0)
    out, _ = run_decode(p)
    ref = gh.run_decode(pk, p.q, p.key_cache, p.value_cache, p.tables, p.lens, p.hkv, p.scale, p.dtype)
    assert_close(ref, p)
    assert_close(out, p)


def test_decode_window_large_batch():
    """More (sequence, kv head) pairs than resident CTAs."""
    rng = wl.rng_for(8)
    lens = rng.integers(1, 900, size=300)
    p = Windowed(rng, lens, np.ones(300, int), 16, 4, 64, wl.F16, 300, 4)
    out, _ = run_decode(p)
    assert_close(out, p)


@pytest.mark.parametrize("hq,hkv,d,dtype", [(32, 32, 128, wl.BF16), (64, 32, 64, wl.F16), (90, 10, 128, wl.F16)])
@pytest.mark.parametrize("top,window,sinks", [(1, 5, 0), (60, 16, 1), (900, 40, 5), (96, 5000, 3)])
def test_decode_window_many_short_runs(hq, hkv, d, dtype, top, window, sinks):
    """A warp per run: thousands of (sequence, kv head) pairs of a few blocks,
    empty ones among them, and a last CTA that is not full."""
    rng = wl.rng_for(top + hq)
    S = 107 if hkv == 10 else 31
    lens = rng.integers(0, top + 1, size=S)
    lens[0] = top
    p = Windowed(rng, lens, np.minimum(lens, 1), hq, hkv, d, dtype, window, sinks)
    out, live = run_decode(p)
    assert_close(out[live], p)
    assert not out[~live].any()


def test_prefill_window_many_short_runs():
    """Chunks of up to 8 rows per kv head take the same shape."""
    rng = wl.rng_for(33)
    lens = rng.integers(1, 80, size=300)
    p = Windowed(rng, lens, np.minimum(lens, rng.integers(0, 4, size=300)), 8, 4, 64, wl.BF16, 20, 2)
    out = run_prefill(p, max_len=4)
    assert pk.get_error() == (0, 0)
    assert_close(out, p)
    # and longer ones over short contexts: three runs of rows per sequence and head
    lens = rng.integers(1, 49, size=31)
    p = Windowed(rng, lens, np.minimum(lens, rng.integers(0, 60, size=31)), 32, 32, 128, wl.F16, 900, 1)
    out = run_prefill(p, max_len=48)
    assert pk.get_error() == (0, 0)
    assert_close(out, p)


@pytest.mark.parametrize("hq,hkv,d,dtype", SHAPES)
def test_decode_append_window_equals_write_then_decode(hq, hkv, d, dtype):
    rng = wl.rng_for(60 + hq)
    lens = np.array([1, 16, 17, 32, 100, 511, 513, 0, 3000])
    p = Windowed(rng, lens, np.minimum(lens, 1), hq, hkv, d, dtype, 200, 6)
    t = device(p)
    S = len(lens)
    q = torch.zeros((S, hq, d), dtype=t["q"].dtype, device="cuda")
    q[torch.from_numpy(lens > 0).cuda()] = t["q"]
    k_new = gh.to_dev(wl.draw_values(rng, (S, hkv, d), dtype), dtype)
    v_new = gh.to_dev(wl.draw_values(rng, (S, hkv, d), dtype), dtype)
    slots = np.array([p.tables[s, (L - 1) // BS] * BS + (L - 1) % BS if L else -1
                      for s, L in enumerate(lens)], np.int64)
    kc1, vc1 = t["kc"].clone(), t["vc"].clone()
    out1 = torch.full_like(q, float("nan"))
    pk.reshape_and_cache(k_new, v_new, kc1, vc1, gh.ints(slots, torch.int64))
    pk.decode_window(out1, q, kc1, vc1, t["tbl"], t["lens"], hkv, p.scale, 200, 6, workspace=decode_ws(p))
    out2 = torch.full_like(q, float("nan"))
    pk.decode_append_window(out2, q, k_new, v_new, t["kc"], t["vc"], t["tbl"], t["lens"], hkv, p.scale,
                            200, 6, workspace=decode_ws(p))
    torch.cuda.synchronize()
    assert pk.get_error() == (0, 0)
    assert torch.equal(out1, out2)
    # the pool holds NaN: compare the bits
    assert torch.equal(kc1.view(torch.int16), t["kc"].view(torch.int16))
    assert torch.equal(vc1.view(torch.int16), t["vc"].view(torch.int16))
    for s, L in enumerate(lens):
        if L:
            p.k[s][L - 1] = gh.to_host_bits(k_new)[s]
            p.v[s][L - 1] = gh.to_host_bits(v_new)[s]
    assert_close(out2[torch.from_numpy(lens > 0).cuda()], p)


def test_decode_append_window_many_short_runs():
    rng = wl.rng_for(71)
    S, hq, hkv, d = 40, 32, 32, 64
    lens = rng.integers(0, 70, size=S)
    p = Windowed(rng, lens, np.minimum(lens, 1), hq, hkv, d, wl.F16, 30, 4)
    t = device(p)
    live = torch.from_numpy(lens > 0).cuda()
    q = torch.zeros((S, hq, d), dtype=t["q"].dtype, device="cuda")
    q[live] = t["q"]
    k_new, v_new = (gh.to_dev(wl.draw_values(rng, (S, hkv, d), wl.F16), wl.F16) for _ in range(2))
    slots = np.array([p.tables[s, (L - 1) // BS] * BS + (L - 1) % BS if L else -1
                      for s, L in enumerate(lens)], np.int64)
    kc, vc = t["kc"].clone(), t["vc"].clone()
    pk.reshape_and_cache(k_new, v_new, kc, vc, gh.ints(slots, torch.int64))
    out = torch.full_like(q, float("nan"))
    pk.decode_append_window(out, q, k_new, v_new, t["kc"], t["vc"], t["tbl"], t["lens"], hkv, p.scale, 30, 4)
    torch.cuda.synchronize()
    assert pk.get_error() == (0, 0)
    assert torch.equal(kc.view(torch.int16), t["kc"].view(torch.int16))
    assert torch.equal(vc.view(torch.int16), t["vc"].view(torch.int16))
    for s, L in enumerate(lens):
        if L:
            p.k[s][L - 1], p.v[s][L - 1] = gh.to_host_bits(k_new)[s], gh.to_host_bits(v_new)[s]
    assert_close(out[live], p)


def test_bad_block_ids_count_only_where_something_is_seen():
    p = Windowed(wl.rng_for(3), [500], [1], 8, 2, 64, wl.F16, 64, 4)
    good, _ = run_decode(p)
    p.tables[0, 5] = 1 << 20  # between the sinks and the window: not read
    out, _ = run_decode(p)
    assert torch.equal(good, out)
    p.tables[0, 500 // BS] = 1 << 20
    t = device(p)
    out = torch.full_like(t["q"], float("nan"))
    kc = t["kc"].clone()
    k_new = torch.zeros((1, 2, 64), dtype=torch.float16, device="cuda")
    pk.decode_append_window(out, t["q"], k_new, k_new, t["kc"], t["vc"], t["tbl"], t["lens"], 2, p.scale,
                            64, 4, workspace=decode_ws(p))
    torch.cuda.synchronize()
    assert pk.get_error() == (pk.PA_ERR_OUT_OF_RANGE, pk.DEVERR_BLOCK_ID)
    assert bool(torch.isfinite(out).all())
    assert torch.equal(kc.view(torch.int16), t["kc"].view(torch.int16))


# ---------------------------------------------------------------- prefill
@pytest.mark.parametrize("hq,hkv,d,dtype", SHAPES + [(10, 2, 64, wl.BF16)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (5, 4), (16, 0), (100, 33), (130, 128), (256, 5),
                                          (2 ** 31 - 1, 0), (3, 2 ** 31 - 1)])
def test_prefill_window(hq, hkv, d, dtype, window, sinks):
    rng = wl.rng_for(window % 999 + sinks % 999 + hq)
    lens = [1, 16, 40, 0, 130, 300, 700, 1000]
    chunk = [1, 3, 40, 0, 129, 17, 260, 1]
    p = Windowed(rng, lens, chunk, hq, hkv, d, dtype, window, sinks)
    out = run_prefill(p, max_len=300)
    assert pk.get_error() == (0, 0)
    assert_close(out, p)


@pytest.mark.parametrize("hq,hkv,d,dtype", SHAPES)
@pytest.mark.parametrize("window,sinks", [(1, 1), (17, 4), (400, 20), (5000, 0)])
def test_prefill_window_of_few_rows(hq, hkv, d, dtype, window, sinks):
    """Up to 16 query rows per kv head: the decode kernel, split over the keys."""
    n = 16 // (hq // hkv)
    rng = wl.rng_for(window + hq)
    chunk = np.array([n, 1, max(1, n - 1), 0, n])
    p = Windowed(rng, [2500, 700, 33, 8, n], chunk, hq, hkv, d, dtype, window, sinks)
    out = run_prefill(p)
    assert pk.get_error() == (0, 0)
    assert_close(out, p)


@pytest.mark.parametrize("hq,hkv,d,dtype,n", [(8, 2, 128, wl.BF16, 400), (4, 4, 64, wl.F16, 400),
                                              (32, 1, 128, wl.F16, 400), (32, 1, 128, wl.F16, 100),
                                              (6, 2, 64, wl.BF16, 333)])
@pytest.mark.parametrize("window", [1000, 2000, 20000])
def test_prefill_window_split_over_keys(hq, hkv, d, dtype, n, window):
    """Few work items: each one's keys go to several CTAs and are joined."""
    p = Windowed(wl.rng_for(window), [6000], [n], hq, hkv, d, dtype, window, 18)
    size = pk.prefill_window_workspace_size(1, n, n, hq, hkv, d, p.tables.shape[1], window, 18)
    assert size > 0 or window == 1000 or n * hq // hkv > 3200     # enough items of one query tile
    out = run_prefill(p)
    assert pk.get_error() == (0, 0)
    assert_close(out, p)
    assert torch.equal(out, run_prefill(p))


@pytest.mark.parametrize("hq,hkv,d,dtype,chunk", [(32, 8, 128, wl.BF16, 32), (32, 8, 128, wl.F16, 25),
                                                  (48, 16, 64, wl.BF16, 42), (8, 8, 128, wl.BF16, 128)])
@pytest.mark.parametrize("window,sinks", [(4000, 9), (1500, 0), (5100, 200)])
def test_prefill_window_of_one_query_tile(hq, hkv, d, dtype, chunk, window, sinks):
    """At most 128 rows per kv head over many keys: the key tiles are shared out."""
    p = Windowed(wl.rng_for(window + chunk), [5200, 130, 4444], [chunk, 1, chunk - 3], hq, hkv, d, dtype,
                 window, sinks)
    out = run_prefill(p)
    assert pk.get_error() == (0, 0)
    assert_close(out, p)
    assert torch.equal(out, run_prefill(p))


@pytest.mark.parametrize("hq,hkv,d,dtype,chunk,window", [
    (32, 8, 128, wl.BF16, 512, 1900), (24, 8, 64, wl.F16, 630, 1300), (32, 32, 128, wl.F16, 500, 700),
    (32, 1, 128, wl.BF16, 473, 2 ** 31 - 1)])
def test_prefill_window_items_of_one_query_tile(hq, hkv, d, dtype, chunk, window):
    """Chunks of several query tiles, too few for two of them per work item."""
    p = Windowed(wl.rng_for(chunk), [2100], [chunk], hq, hkv, d, dtype, window, 5)
    out = run_prefill(p)
    assert pk.get_error() == (0, 0)
    assert_close(out, p)
    assert torch.equal(out, run_prefill(p))


@pytest.mark.parametrize("group", [17, 43, 100, 128])
def test_prefill_window_wide_groups(group):
    """More than 16 query heads per kv head, odd ones among them."""
    p = Windowed(wl.rng_for(group), [500, 90, 33], [7, 1, 20], group, 1, 64, wl.BF16, 70, 3)
    out = run_prefill(p)
    assert pk.get_error() == (0, 0)
    assert_close(out, p)


def test_prefill_window_many_items():
    rng = wl.rng_for(12)
    lens = rng.integers(200, 1500, size=40)
    p = Windowed(rng, lens, np.minimum(lens, 150), 8, 4, 64, wl.BF16, 333, 7)
    out = run_prefill(p)
    assert pk.get_error() == (0, 0)
    assert_close(out, p)


def test_prefill_window_one_token_chunks_agree_with_decode():
    p = Windowed(wl.rng_for(2), [900, 40, 2000], [1, 1, 1], 8, 2, 128, wl.BF16, 500, 4)
    dec, _ = run_decode(p)
    assert torch.equal(dec, run_prefill(p))


@pytest.mark.parametrize("max_len", [4, 40])
def test_prefill_window_leaves_other_rows_alone(max_len):
    """Rows behind the last sequence, and those of a chunk longer than announced."""
    p = Windowed(wl.rng_for(4), [90, 80, 70], [max_len, max_len - 1, 1], 4, 1, 64, wl.F16, 30, 2)
    rows = int(p.start[-1])
    out = run_prefill(p, rows=rows + 50)
    assert pk.get_error() == (0, 0)
    assert_close(out[:rows], p)
    assert bool(torch.isnan(out[rows:]).all())
    out = run_prefill(p, max_len=max_len - 1, rows=rows + 50)  # sequence 0 is longer
    assert pk.get_error() == (pk.PA_ERR_OUT_OF_RANGE, pk.DEVERR_CONTEXT_LEN)
    assert bool(torch.isnan(out[:max_len]).all()) and bool(torch.isnan(out[rows:]).all())
    ref, tol = p.reference()
    assert np.all(np.abs(gh.to_f64(out[max_len:rows]) - ref[max_len:]) <= tol[max_len:])


# ---------------------------------------------------------------- streams and graphs
def test_windowed_calls_replay_from_a_graph_on_a_side_stream():
    p = Windowed(wl.rng_for(21), [3000, 77, 1200], [1, 1, 1], 8, 2, 128, wl.BF16, 900, 4)
    pf = Windowed(wl.rng_for(22), [3000, 77], [60, 20], 8, 2, 128, wl.BF16, 900, 4)
    want, want_pf = run_decode(p)[0], run_prefill(pf)
    t, u = device(p), device(pf)
    out, out_pf = torch.zeros_like(t["q"]), torch.zeros_like(u["q"])
    ws = decode_ws(p)
    n = pk.prefill_window_workspace_size(2, 80, 60, 8, 2, 128, pf.tables.shape[1], 900, 4)
    ws_pf, start = scratch(n), gh.ints(pf.start)

    def step():
        pk.decode_window(out, t["q"], t["kc"], t["vc"], t["tbl"], t["lens"], 2, p.scale, 900, 4, workspace=ws)
        pk.prefill_window(out_pf, u["q"], u["kc"], u["vc"], u["tbl"], u["lens"], start, 60, 2, pf.scale,
                          900, 4, workspace=ws_pf)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for _ in range(2):
        out.zero_()
        out_pf.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(out_pf, want_pf)
    # new contents, same graph
    t["q"].neg_()
    graph.replay()
    torch.cuda.synchronize()
    p.q ^= 0x8000
    assert_close(out, p)
