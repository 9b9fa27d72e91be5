"""Plain 64-bit forms of the windowed attention and of the rotary positions,
and paged problems to run them on.  Nothing here calls the CUDA library."""
from __future__ import annotations

import numpy as np

import workloads as wl
from paged_inputs import to_f64

BS = 16
EPS = {wl.F16: 2.0 ** -10, wl.BF16: 2.0 ** -7}
NAN_BITS = {wl.F16: 0x7E00, wl.BF16: 0x7FC0}
INF_BITS = {wl.F16: 0x7C00, wl.BF16: 0x7F80}


def seen(pos, keys, window, sinks):
    """[rows][keys] mask: key j is seen from position p."""
    p, j = np.asarray(pos)[:, None], np.asarray(keys)[None]
    return (j <= p) & ((p - j < window) | (j < sinks))


def attend(q, k, v, mask, scale):
    """q [rows][G][d], k, v [n][d], mask [rows][n] -> (out, mean |v| under the
    weights), both [rows][G][d], in 64 bits; a row that sees nothing gives 0."""
    x = np.einsum("rgd,nd->rgn", q, k) * scale
    x = np.where(mask[:, None], x, -np.inf)
    m = x.max(-1, keepdims=True, initial=-np.inf)
    w = np.exp(x - np.where(np.isfinite(m), m, 0.0))
    den = w.sum(-1, keepdims=True)
    w = w / np.where(den > 0, den, 1.0)
    return np.einsum("rgn,nd->rgd", w, v), np.einsum("rgn,nd->rgd", w, np.abs(v))


class Windowed:
    """Sequences of lens[s] tokens whose last chunk[s] are queries.  The pool
    holds NaN and infinities wherever no query looks: in free blocks, behind
    the context, and in the unseen rows of blocks that are read.  Table entries
    of blocks without a seen token are -1."""

    def __init__(self, rng, lens, chunk, hq, hkv, d, dtype, window, sinks, max_blocks=None,
                 spare=3, scale=None):
        self.lens = np.asarray(lens, np.int32)
        self.chunk = np.asarray(chunk, np.int32)
        self.hq, self.hkv, self.d, self.dtype = hq, hkv, d, dtype
        self.window, self.sinks = window, sinks
        self.scale = 1.0 / np.sqrt(d) if scale is None else scale
        S = len(self.lens)
        lmax = max(int(self.lens.max()), 1)
        mb = max_blocks or -(-lmax // BS)
        self.start = np.concatenate([[0], np.cumsum(self.chunk)]).astype(np.int32)
        self.q = wl.draw_values(rng, (int(self.start[-1]), hq, d), dtype)
        self.k = [wl.draw_values(rng, (int(L), hkv, d), dtype) for L in self.lens]
        self.v = [wl.draw_values(rng, (int(L), hkv, d), dtype) for L in self.lens]
        self.any_seen = []
        for L, n in zip(self.lens, self.chunk):
            pos = np.arange(L - n, L)
            self.any_seen.append(seen(pos, np.arange(L), window, sinks).any(0) if n else
                                 np.zeros(L, bool))
        held = [[b for b in range(-(-int(L) // BS)) if a[b * BS:(b + 1) * BS].any()]
                for L, a in zip(self.lens, self.any_seen)]
        self.num_blocks = sum(map(len, held)) + spare
        ids = iter(rng.permutation(self.num_blocks).astype(np.int32))
        self.tables = np.full((S, mb), -1, np.int32)
        self.key_cache = np.full((self.num_blocks, hkv, BS, d), NAN_BITS[dtype], np.uint16)
        self.value_cache = np.full_like(self.key_cache, INF_BITS[dtype])
        for s in range(S):
            for b in held[s]:
                i = next(ids)
                self.tables[s, b] = i
                for t in range(b * BS, min((b + 1) * BS, int(self.lens[s]))):
                    if self.any_seen[s][t]:
                        self.key_cache[i, :, t % BS] = self.k[s][t]
                        self.value_cache[i, :, t % BS] = self.v[s][t]

    def reference(self):
        """(out, tolerance) [rows][Hq][d] in 64 bits.

        The kernels round each weight to the 16-bit type for the P V product
        (half a step, relative) while the sum of weights stays in f32, and round
        the result once (half a step of |out|).  With A = sum_j w_j |V_j| the
        first costs at most EPS / 2 * A; the exponentials (relative error below
        8e-5, once in the product and once in the sum) and the f32 sums of at
        most 128 products per logit cost less than 2^-12 * A more."""
        G = self.hq // self.hkv
        out = np.zeros((int(self.start[-1]), self.hq, self.d))
        mean_abs = np.zeros_like(out)
        for s, (L, n) in enumerate(zip(self.lens, self.chunk)):
            if n == 0 or L == 0:
                continue
            pos = np.arange(L - n, L)
            keys = np.nonzero(self.any_seen[s])[0]
            mask = seen(pos, keys, self.window, self.sinks)
            k, v = to_f64(self.k[s], self.dtype)[keys], to_f64(self.v[s], self.dtype)[keys]
            rows = slice(self.start[s], self.start[s + 1])
            q = to_f64(self.q[rows], self.dtype)
            for h in range(self.hkv):
                hs = slice(h * G, (h + 1) * G)
                out[rows, hs], mean_abs[rows, hs] = attend(q[:, hs], k[:, h], v[:, h], mask, self.scale)
        half = EPS[self.dtype] / 2
        return out, (half + 2.0 ** -12) * mean_abs + half * np.abs(out) + 1e-7


def rotate(x, positions, inv_freq, axes, interleaved):
    """x [T][heads][d] f64; positions [num_axes][T]; -> turned x.  The angle
    is reduced exactly: position and (float32) frequency are rationals with few
    bits, so their product modulo a turn is taken in extended precision."""
    pairs = len(inv_freq)
    ld = np.longdouble
    turn = ld("6.28318530717958647692528676655900576839433879875021")
    ang = np.stack([np.fmod(positions[a].astype(ld) * ld(np.float32(f)), turn)
                    for f, a in zip(inv_freq, axes)], 1)  # T, pairs
    c, s = np.cos(ang).astype(np.float64)[:, None], np.sin(ang).astype(np.float64)[:, None]
    i = np.arange(pairs)
    ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + pairs)
    y = x.copy()
    y[..., ia] = x[..., ia] * c - x[..., ib] * s
    y[..., ib] = x[..., ib] * c + x[..., ia] * s
    return y
