"""Rotary positions with the cache write, against their plain 64-bit form."""
import numpy as np
import pytest

import workloads as wl
from paged_inputs import to_f64
from window_reference import EPS, rotate

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import gpu_harness as gh  # noqa: E402

pk = pytest.importorskip("paged_kv_cache_425_b200")

FAR = [0, 1, -1, 7, 131071, 10 ** 6 + 3, 2 ** 30 + 1, 2 ** 31 - 1, -2 ** 31, -12345]


class Problem:
    """q, k, v as slices of one projection; every third token is padding."""

    def __init__(self, seed, T, hq, hkv, d, dtype, pairs, axes, interleaved, theta=10000.0):
        rng = wl.rng_for(seed)
        self.hq, self.hkv, self.d, self.dtype, self.T = hq, hkv, d, dtype, T
        self.x = wl.draw_values(rng, (T, hq + 2 * hkv, d), dtype)
        self.num_axes = max(axes) + 1
        self.axes, self.interleaved = np.asarray(axes, np.int32), interleaved
        self.freq = (theta ** (-np.arange(pairs) / pairs)).astype(np.float32)
        self.pos = rng.integers(0, 200000, size=(self.num_axes, T)).astype(np.int32)
        m = min(T, len(FAR))
        for a in range(self.num_axes):
            self.pos[a, :m] = np.roll(FAR, a)[:m]
        blocks = T // 16 + 3
        self.slots = rng.permutation(blocks * 16)[:T].astype(np.int64)
        self.slots[2::3] = -1
        self.kc = wl.draw_values(rng, (blocks, hkv, 16, d), dtype)
        self.vc = wl.draw_values(rng, (blocks, hkv, 16, d), dtype)

    def run(self, q_out=None, in_place=False):
        x = gh.to_dev(self.x, self.dtype)
        hq, hkv = self.hq, self.hkv
        q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
        if in_place:
            q = q_out = q.contiguous()
        elif q_out is None:
            q_out = torch.full((self.T, hq, self.d), float("nan"), dtype=x.dtype, device="cuda")
        kc, vc = gh.to_dev(self.kc, self.dtype), gh.to_dev(self.vc, self.dtype)
        rope = pk.Rope(self.freq, self.axes, interleaved=self.interleaved)
        pk.rope_and_cache(q_out, q, k, v, kc, vc, gh.ints(self.slots, torch.int64), gh.ints(self.pos), rope)
        torch.cuda.synchronize()
        return q_out, kc, vc

    def check(self, q_out, kc, vc):
        x = to_f64(self.x, self.dtype)
        turned = rotate(x, self.pos, self.freq, self.axes, self.interleaved)
        # one rounding (half a step of the result) of a sum of two products
        # whose factors carry at most 2^-21 (f32 angle of up to a half turn, its
        # cosine and sine, the products)
        reach = np.abs(x).max(-1, keepdims=True)
        tol = EPS[self.dtype] / 2 * np.abs(turned) + 2.0 ** -20 * reach + EPS[self.dtype] / 2 * 2.0 ** -13
        hq, hkv = self.hq, self.hkv
        assert np.all(np.abs(gh.to_f64(q_out) - turned[:, :hq]) <= tol[:, :hq])
        keep = self.slots >= 0
        b, o = self.slots[keep] // 16, self.slots[keep] % 16
        got = gh.to_f64(kc)[b, :, o]
        assert np.all(np.abs(got - turned[keep, hq:hq + hkv]) <= tol[keep, hq:hq + hkv])
        # v, and every cache row that no token went to, bit for bit
        want_v = self.vc.copy()
        want_v[b, :, o] = self.x[keep, hq + hkv:]
        assert np.array_equal(gh.to_host_bits(vc), want_v)
        rest = np.ones(self.kc.shape[0] * 16, bool)
        rest[self.slots[keep]] = False
        rest = rest.reshape(-1, 16)
        assert np.array_equal(gh.to_host_bits(kc).transpose(0, 2, 1, 3)[rest],
                              self.kc.transpose(0, 2, 1, 3)[rest])


CASES = [
    # T, hq, hkv, d, dtype, pairs, axes, interleaved
    (1, 4, 4, 64, wl.F16, 32, [0] * 32, False),
    (1, 32, 8, 128, wl.BF16, 64, [0] * 16 + [1] * 24 + [2] * 24, False),
    (37, 12, 1, 64, wl.BF16, 16, [0, 1] * 8, False),
    (64, 32, 8, 128, wl.F16, 64, [0, 1, 2, 3] * 16, True),
    (33, 7, 7, 128, wl.BF16, 8, [0] * 8, False),
    (50, 5, 1, 128, wl.F16, 40, [0] * 10 + [2] * 30, True),
    (300, 64, 16, 128, wl.BF16, 64, [7] * 64, False),
    (29, 16, 2, 64, wl.F16, 24, [0] * 24, True),
]


@pytest.mark.parametrize("T,hq,hkv,d,dtype,pairs,axes,interleaved", CASES)
def test_rope_and_cache(T, hq, hkv, d, dtype, pairs, axes, interleaved):
    p = Problem(T + hq, T, hq, hkv, d, dtype, pairs, axes, interleaved)
    got = p.run()
    assert pk.get_error() == (0, 0)
    p.check(*got)


def test_rope_in_place_and_bit_equal():
    p = Problem(1, 40, 8, 2, 128, wl.BF16, 64, [0] * 32 + [1] * 32, False)
    a, b = p.run(), p.run(in_place=True)
    p.check(*b)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_rope_without_query_heads_and_without_tokens():
    p = Problem(2, 20, 0, 3, 64, wl.F16, 32, [0] * 32, False)
    q_out, kc, vc = p.run()
    p.check(q_out, kc, vc)
    p = Problem(2, 0, 4, 3, 64, wl.F16, 32, [0] * 32, False)
    q_out, kc, vc = p.run()
    assert np.array_equal(gh.to_host_bits(kc), p.kc) and np.array_equal(gh.to_host_bits(vc), p.vc)


def test_rope_slot_beyond_the_pool_is_reported():
    p = Problem(3, 9, 4, 2, 128, wl.F16, 64, [0] * 64, True)
    p.slots[4] = p.kc.shape[0] * 16
    q_out, kc, vc = p.run()
    assert pk.get_error() == (pk.PA_ERR_OUT_OF_RANGE, pk.DEVERR_SLOT)
    p.slots[4] = -1
    p.check(q_out, kc, vc)


def test_rope_zero_position_and_pass_through_keep_the_bits():
    p = Problem(4, 12, 4, 2, 128, wl.BF16, 16, [0] * 16, False)
    p.pos[:] = 0
    q_out, kc, _ = p.run()
    assert np.array_equal(gh.to_host_bits(q_out), p.x[:, :4])
    p.pos[:] = 12345
    q_out, _, _ = p.run()
    assert np.array_equal(gh.to_host_bits(q_out)[..., 32:], p.x[:, :4, 32:])


def test_rope_undoes_itself():
    """Turning by p and then by -p gives the input back, up to two roundings."""
    p = Problem(5, 60, 4, 1, 64, wl.F16, 32, [0] * 32, False)
    p.pos[:] = np.where(p.pos == -2 ** 31, 5, p.pos)
    q1, _, _ = p.run()
    back = Problem(5, 60, 4, 1, 64, wl.F16, 32, [0] * 32, False)
    back.pos = -p.pos
    back.x[:, :4] = gh.to_host_bits(q1)
    q2, _, _ = back.run()
    x = to_f64(p.x, wl.F16)[:, :4]
    size = np.sqrt(x[..., :32] ** 2 + x[..., 32:] ** 2)
    tol = np.concatenate([size, size], -1) * (3 * EPS[wl.F16] / 2) + 2.0 ** -18
    assert np.all(np.abs(gh.to_f64(q2) - x) <= tol)
