"""Windowed calls whose keys are split over several CTAs and joined through the
workspace, against the 64-bit form.  Each test asserts that there is a split, so
that a change of the launch plan cannot empty it."""
import numpy as np
import pytest

import window_shapes as ws
import workloads as wl
from test_gpu_window import assert_close, decode_ws, device, run_decode, run_prefill, scratch
from window_reference import BS, Windowed

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import gpu_harness as gh  # noqa: E402

pk = pytest.importorskip("paged_kv_cache_425_b200")


@pytest.mark.parametrize("heads", ws.HEADS, ids=str)
@pytest.mark.parametrize("shape", ws.SPLIT)
def test_decode_window_split(shape, heads):
    p = ws.decode_problem(shape, *heads, sinks=21)
    assert decode_ws(p) is not None
    out, _ = run_decode(p)
    assert_close(out, p)
    assert torch.equal(out, run_decode(p)[0])


@pytest.mark.parametrize("heads", [ws.HEADS[0], ws.HEADS[1], ws.HEADS[2]], ids=str)
@pytest.mark.parametrize("shape", ws.SPLIT)
def test_decode_append_window_split(shape, heads):
    """The new token's block lies behind the loads that a warp starts with."""
    p = ws.decode_problem(shape, *heads, sinks=4, seed=1)
    work = decode_ws(p)
    assert work is not None
    t, S = device(p), len(p.lens)
    rng = wl.rng_for(S + p.d)
    new = [wl.draw_values(rng, (S, p.hkv, p.d), p.dtype) for _ in range(2)]
    k_new, v_new = (gh.to_dev(x, p.dtype) for x in new)
    before = [x.view(torch.int16).clone() for x in (t["kc"], t["vc"])]
    out = torch.full_like(t["q"], float("nan"))
    pk.decode_append_window(out, t["q"], k_new, v_new, t["kc"], t["vc"], t["tbl"], t["lens"], p.hkv, p.scale,
                            p.window, p.sinks, workspace=work)
    torch.cuda.synchronize()
    assert pk.get_error() == (0, 0)
    for s, L in enumerate(p.lens):
        p.k[s][L - 1], p.v[s][L - 1] = new[0][s], new[1][s]
        b = int(p.tables[s, (L - 1) // BS])
        before[0][b, :, (L - 1) % BS] = k_new[s].view(torch.int16)
        before[1][b, :, (L - 1) % BS] = v_new[s].view(torch.int16)
    assert_close(out, p)
    assert torch.equal(before[0], t["kc"].view(torch.int16))
    assert torch.equal(before[1], t["vc"].view(torch.int16))


@pytest.mark.parametrize("hq,d,dtype,n", [(8, 128, wl.BF16, 2), (2, 64, wl.F16, 8), (10, 128, wl.F16, 1),
                                          (32, 64, wl.BF16, 1)])
@pytest.mark.parametrize("window", [2500, 4500, 9000])
def test_prefill_window_of_few_rows_split(hq, d, dtype, n, window):
    """Chunks of at most 8 rows per kv head, or of one token, in partitions."""
    rng = wl.rng_for(window + hq)
    lens = rng.integers(n, 70, size=80)
    lens[[1, 40]] = window + 100, window // 2
    chunk = rng.integers(1, n + 1, size=80)
    chunk[1] = n
    p = Windowed(rng, lens, chunk, hq, 2, d, dtype, window, 5)
    assert pk.prefill_window_workspace_size(80, int(chunk.sum()), n, hq, 2, d, p.tables.shape[1], window, 5) > 0
    out = run_prefill(p)
    assert pk.get_error() == (0, 0)
    assert_close(out, p)


@pytest.mark.parametrize("hq,hkv,d,dtype,n,window", [
    (8, 2, 128, wl.F16, 400, 2000), (4, 4, 64, wl.BF16, 400, 2000), (32, 8, 128, wl.BF16, 32, 4000),
    (48, 16, 64, wl.F16, 42, 4000), (32, 1, 128, wl.BF16, 100, 5000), (7, 1, 64, wl.F16, 200, 20000)])
def test_prefill_window_of_long_chunks_split(hq, hkv, d, dtype, n, window):
    p = Windowed(wl.rng_for(window + hq), [5300, 777], [n, min(n, 50)], hq, hkv, d, dtype, window, 18)
    rows = int(p.chunk.sum())
    assert pk.prefill_window_workspace_size(2, rows, n, hq, hkv, d, p.tables.shape[1], window, 18) > 0
    out = run_prefill(p)
    assert pk.get_error() == (0, 0)
    assert_close(out, p)


@pytest.mark.parametrize("hq,hkv,d,dtype,n,window", [
    (32, 8, 128, wl.BF16, 512, 700), (32, 32, 128, wl.F16, 500, 700), (24, 8, 64, wl.F16, 630, 600)])
def test_prefill_window_of_long_chunks_unsplit(hq, hkv, d, dtype, n, window):
    p = Windowed(wl.rng_for(n), [2100], [n], hq, hkv, d, dtype, window, 5)
    assert pk.prefill_window_workspace_size(1, n, n, hq, hkv, d, p.tables.shape[1], window, 5) == 0
    out = run_prefill(p)
    assert pk.get_error() == (0, 0)
    assert_close(out, p)


def test_two_streams_in_partitions_match_the_plain_form():
    """Overlapping calls with a workspace each."""
    jobs = []
    for seed in range(2):
        p = ws.decode_problem("partitions of 64 blocks", 4, 128, wl.BF16, sinks=4, seed=seed)
        jobs.append((p, device(p), decode_ws(p), torch.cuda.Stream()))
        assert jobs[-1][2] is not None
    outs = [torch.full_like(t["q"], float("nan")) for _, t, _, _ in jobs]
    torch.cuda.synchronize()
    for _ in range(4):
        for out, (p, t, work, stream) in zip(outs, jobs):
            pk.decode_window(out, t["q"], t["kc"], t["vc"], t["tbl"], t["lens"], p.hkv, p.scale, p.window,
                             p.sinks, workspace=work, stream=stream)
    torch.cuda.synchronize()
    assert pk.get_error() == (0, 0)
    for out, (p, _, _, _) in zip(outs, jobs):
        assert_close(out, p)
