"""Contexts of nearly 2^30 tokens: tables as wide as the windowed calls take,
with -1 between the sinks and the window."""
import numpy as np
import pytest

import workloads as wl
from test_gpu_window import assert_close
from window_reference import BS, Windowed

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import gpu_harness as gh  # noqa: E402

pk = pytest.importorskip("paged_kv_cache_425_b200")

WIDTH = 1 << 26


@pytest.mark.parametrize("hq,hkv,d,n", [(8, 2, 128, 1), (4, 4, 64, 3), (4, 2, 128, 150)])
def test_far_contexts_equal_near_ones(hq, hkv, d, n):
    """The blocks behind the sinks moved to the end of the table: the same bits."""
    free, _ = torch.cuda.mem_get_info()
    if free < 2 << 30:
        pytest.skip("needs 1 GB of free device memory")
    window, sinks, lens = 300, 20, [1003, 40]
    p = Windowed(wl.rng_for(n), lens, np.minimum(lens, n), hq, hkv, d, wl.BF16, window, sinks)
    rows, blocks = int(p.start[-1]), p.tables.shape[1]
    moved = WIDTH - blocks - 1
    q, start = gh.to_dev(p.q, p.dtype), gh.ints(p.start)
    k_new, v_new = (gh.to_dev(wl.draw_values(wl.rng_for(7), (2, hkv, d), p.dtype), p.dtype) for _ in range(2))
    far = torch.full((2, WIDTH), -1, dtype=torch.int32, device="cuda")
    near = torch.full((2, 128), -1, dtype=torch.int32, device="cuda")
    near[:, :blocks] = gh.ints(p.tables)
    far[1] = torch.nn.functional.pad(near[1], (0, WIDTH - 128), value=-1)
    far[0, :2] = near[0, :2]
    far[0, moved + 2:moved + blocks] = near[0, 2:blocks]

    def run(tbl, first):
        kc, vc = gh.to_dev(p.key_cache, p.dtype), gh.to_dev(p.value_cache, p.dtype)
        ln = gh.ints(np.array([first, lens[1]]))
        out = torch.full_like(q, float("nan"))
        if n == 1:
            size = pk.decode_window_workspace_size(2, hq, hkv, d, tbl.shape[1], window, sinks)
            assert size == 0
            pk.decode_window(out, q, kc, vc, tbl, ln, hkv, p.scale, window, sinks)
            more = torch.full_like(q, float("nan"))
            pk.decode_append_window(more, q, k_new, v_new, kc, vc, tbl, ln, hkv, p.scale, window, sinks)
            outs = [out, more, kc, vc]
        else:
            size = pk.prefill_window_workspace_size(2, rows, n, hq, hkv, d, tbl.shape[1], window, sinks)
            work = torch.empty(max(size, 256), dtype=torch.uint8, device="cuda")
            pk.prefill_window(out, q, kc, vc, tbl, ln, start, n, hkv, p.scale, window, sinks, workspace=work)
            outs = [out]
        torch.cuda.synchronize()
        assert pk.get_error() == (0, 0)
        return outs

    want, got = run(near, lens[0]), run(far, lens[0] + moved * BS)
    assert_close(want[0], p)
    for a, b in zip(want, got):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))
