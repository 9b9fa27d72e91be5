"""Seeded random shapes for the windowed calls: heads, lengths, windows, sinks,
types and batch sizes drawn over the ranges that reach every launch shape."""
import numpy as np
import pytest

import workloads as wl
from test_gpu_window import assert_close, run_decode, run_prefill
from window_reference import Windowed

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

pk = pytest.importorskip("paged_kv_cache_425_b200")


def log_int(rng, lo, hi):
    return int(round(np.exp(rng.uniform(np.log(lo), np.log(hi)))))


def draw(seed, most_tokens):
    rng = wl.rng_for(9000 + seed)
    hkv = int(rng.choice([1, 2, 3, 8]))
    group = int(rng.choice([1, 2, 4, 5, 8, 11, 16]))
    d, dtype = int(rng.choice([64, 128])), int(rng.choice([wl.F16, wl.BF16]))
    window, sinks = log_int(rng, 1, 5000), int(rng.choice([0, 1, 4, 17, 100]))
    top = log_int(rng, 1, 6000)
    seqs = max(1, min(log_int(rng, 1, 400), most_tokens // (min(window + sinks, top) * hkv)))
    lens = rng.integers(0 if rng.random() < 0.3 else max(1, top // 2), top + 1, size=seqs)
    return rng, lens, hkv * group, hkv, d, dtype, window, sinks


@pytest.mark.parametrize("seed", range(30))
def test_random_decode_window(seed):
    rng, lens, hq, hkv, d, dtype, window, sinks = draw(seed, 60000)
    p = Windowed(rng, lens, np.minimum(lens, 1), hq, hkv, d, dtype, window, sinks)
    out, live = run_decode(p)
    assert_close(out[live], p)
    assert not out[~live].any()


@pytest.mark.parametrize("seed", range(30, 70))
def test_random_prefill_window(seed):
    rng, lens, hq, hkv, d, dtype, window, sinks = draw(seed, 12000)
    lens = np.maximum(lens, 1)
    longest = log_int(rng, 1, 300)
    chunk = np.minimum(rng.integers(0, longest + 1, size=len(lens)), lens)
    chunk[0] = min(longest, lens[0])
    # at most 2e8 scores for the 64-bit form
    while (chunk * np.minimum(lens, window + sinks + longest)).sum() * hq > 2e8:
        chunk = -(-chunk // 2)
    p = Windowed(rng, lens, chunk, hq, hkv, d, dtype, window, sinks)
    out = run_prefill(p, max_len=int(chunk.max()) + int(rng.integers(0, 3)))
    assert pk.get_error() == (0, 0)
    assert_close(out, p)
