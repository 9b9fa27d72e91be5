"""Visible scores that are not finite: a score of -infinity has weight 0 (a row
with no other is zero), NaN or +infinity makes its row NaN, on every launch
shape of the windowed calls."""
import numpy as np
import pytest

import window_shapes as ws
from test_gpu_window import run_decode, run_prefill

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import gpu_harness as gh  # noqa: E402

pk = pytest.importorskip("paged_kv_cache_425_b200")


@pytest.mark.parametrize("heads", [ws.HEADS[1], ws.HEADS[3]], ids=str)
@pytest.mark.parametrize("kind", ws.KINDS)
@pytest.mark.parametrize("shape", ws.DECODE)
def test_decode_window(shape, kind, heads):
    p = ws.decode_problem(shape, *heads)
    ws.not_finite(p, kind)
    out, live = run_decode(p)
    assert bool(live.all())
    assert ws.worst(gh.to_f64(out), p) <= 1.0


@pytest.mark.parametrize("kind", ws.KINDS)
@pytest.mark.parametrize("shape", ws.PREFILL)
def test_prefill_window(shape, kind):
    """150 sinks: whole key tiles of -infinity in front of the window."""
    p = ws.prefill_problem(shape, 150 if kind in ("half", "all") else 1)
    ws.not_finite(p, kind)
    out = run_prefill(p)
    assert pk.get_error() == (0, 0)
    assert ws.worst(gh.to_f64(out), p) <= 1.0
