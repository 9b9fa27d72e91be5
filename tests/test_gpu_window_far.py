"""Windowed calls far out: caches whose elements pass 32-bit offsets, contexts
of hundreds of thousands of tokens."""
import numpy as np
import pytest

import workloads as wl
from window_reference import Windowed

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import gpu_harness as gh  # noqa: E402

pk = pytest.importorskip("paged_kv_cache_425_b200")


def test_blocks_beyond_32_bit_offsets():
    """The same problem in a small pool and at the far end of one of over 2^32
    elements: the same bits, in the outputs and in the rows written."""
    hq, hkv, d, window, sinks = 8, 2, 128, 300, 4
    far_blocks = 2 ** 32 // (hkv * 16 * d) + 4096
    shape = (far_blocks, hkv, 16, d)
    free, _ = torch.cuda.mem_get_info()
    if free < 3 * 2 * int(np.prod(shape)):
        pytest.skip("needs 26 GB of free device memory")
    p = Windowed(wl.rng_for(1), [500, 37, 900], [1, 1, 1], hq, hkv, d, wl.BF16, window, sinks)
    pf = Windowed(wl.rng_for(2), [700, 64], [90, 64], hq, hkv, d, wl.BF16, window, sinks)
    far_k, far_v = (torch.empty(shape, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    rng = wl.rng_for(3)
    k_new, v_new, q3 = (gh.to_dev(wl.draw_values(rng, (3, h, d), wl.BF16), wl.BF16) for h in (hkv, hkv, hq))
    rope = pk.Rope(10000.0 ** (-np.arange(64) / 64), interleaved=True)
    pos = gh.ints(np.array([[5, 70000, 2 ** 31 - 1]]))

    def run(shift, kc, vc):
        outs = []
        for prob in (p, pf):
            n = prob.num_blocks
            kc[shift:shift + n] = gh.to_dev(prob.key_cache, wl.BF16)
            vc[shift:shift + n] = gh.to_dev(prob.value_cache, wl.BF16)
            tbl = gh.ints(np.where(prob.tables >= 0, prob.tables + shift, -1))
            lens, q = gh.ints(prob.lens), gh.to_dev(prob.q, wl.BF16)
            out = torch.empty_like(q)
            if prob is p:
                pk.decode_append_window(out, q, k_new, v_new, kc, vc, tbl, lens, hkv, p.scale, window, sinks)
            else:
                m = pk.prefill_window_workspace_size(2, q.shape[0], 90, hq, hkv, d, tbl.shape[1], window, sinks)
                ws = torch.empty(max(m, 256), dtype=torch.uint8, device="cuda")
                pk.prefill_window(out, q, kc, vc, tbl, lens, gh.ints(prob.start), 90, hkv, prob.scale, window,
                                  sinks, workspace=ws)
            outs += [out, kc[shift:shift + n].clone(), vc[shift:shift + n].clone()]
        slots = torch.tensor([shift * 16 + 3, shift * 16 + 40, shift * 16 + 17], device="cuda")
        q_out = torch.empty_like(q3)
        pk.rope_and_cache(q_out, q3, k_new, v_new, kc, vc, slots, pos, rope)
        torch.cuda.synchronize()
        assert pk.get_error() == (0, 0)
        return outs + [q_out, kc[shift:shift + 4].clone(), vc[shift:shift + 4].clone()]

    near = run(0, *(torch.empty((2048, hkv, 16, d), dtype=torch.bfloat16, device="cuda") for _ in range(2)))
    far = run(far_blocks - 2048, far_k, far_v)
    for a, b in zip(near, far):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))


@pytest.mark.parametrize("window", [300, 70000, 500000])
def test_contexts_of_hundreds_of_thousands_of_tokens(window):
    L, S, hq, hkv, d, sinks = 600001, 2, 4, 1, 64, 40
    gen = torch.Generator(device="cuda").manual_seed(window)
    nblk = -(-L // 16)
    kc, vc = (torch.randn(S * nblk, hkv, 16, d, generator=gen, device="cuda").half() for _ in range(2))
    tbl = torch.randperm(S * nblk, generator=gen, device="cuda").int().view(S, nblk)
    lens = torch.tensor([L, L - 33], dtype=torch.int32, device="cuda")
    for n in (1, 3, 70):
        q = torch.randn(S * n, hq, d, generator=gen, device="cuda").half()
        out = torch.full_like(q, float("nan"))
        start = torch.arange(S + 1, dtype=torch.int32, device="cuda") * n
        if n == 1:
            m = pk.decode_window_workspace_size(S, hq, hkv, d, nblk, window, sinks)
            ws = torch.empty(m, dtype=torch.uint8, device="cuda") if m else None
            pk.decode_window(out, q, kc, vc, tbl, lens, hkv, 0.125, window, sinks, workspace=ws)
        else:
            m = pk.prefill_window_workspace_size(S, S * n, n, hq, hkv, d, nblk, window, sinks)
            ws = torch.empty(m, dtype=torch.uint8, device="cuda") if m else None
            pk.prefill_window(out, q, kc, vc, tbl, lens, start, n, hkv, 0.125, window, sinks, workspace=ws)
        assert pk.get_error() == (0, 0)
        for s in range(S):
            Ls = int(lens[s])
            first = Ls - n
            lo = max(0, first - window + 1)
            keys = torch.cat([torch.arange(min(sinks, lo)), torch.arange(lo, Ls)]).cuda()
            ids = tbl[s, keys // 16].long()
            K, V = kc[ids, 0, keys % 16].double(), vc[ids, 0, keys % 16].double()
            at = torch.arange(first, Ls, device="cuda")[:, None]
            hidden = (keys > at) | ((keys <= at - window) & (keys >= sinks))
            x = torch.einsum("rhd,nd->rhn", q[s * n:(s + 1) * n].double(), K) * 0.125
            w = torch.softmax(x.masked_fill(hidden[:, None], float("-inf")), -1)
            ref, mean = w @ V, w @ V.abs()
            # the weights' and the result's rounding as in window_reference; the f32
            # sums are of at most 256 terms per warp or thread and 1024 joined
            # parts, 2^-24 each: below 2^-13 once for the product, once for the sum
            tol = (2.0 ** -11 + 2.0 ** -12 + 2.0 ** -12) * mean + 2.0 ** -11 * ref.abs() + 1e-7
            assert bool(((out[s * n:(s + 1) * n].double() - ref).abs() <= tol).all())
