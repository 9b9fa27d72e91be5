"""Problems that reach every launch shape of the windowed calls, and visible
scores that are not finite.  Nothing here calls the CUDA library."""
from __future__ import annotations

import numpy as np

import workloads as wl
from window_reference import BS, INF_BITS, NAN_BITS, Windowed

# Decode: sequences, kv heads, window, blocks of the longest context beyond the
# window.  The shape follows from runs = sequences * kv heads and from the
# visible blocks of the longest context.
DECODE = {
    "cluster": (2, 2, 3000, 30),
    "one CTA of many warps": (40, 2, 400, 5),
    "one CTA": (90, 2, 400, 5),
    "a warp per run": (120, 8, 50, 2),
    "partitions of 32 blocks": (90, 2, 2500, 10),
    "partitions of 64 blocks": (90, 2, 4500, 10),
    "more than 8 partitions": (90, 2, 9000, 10),
}
SPLIT = [n for n in DECODE if "partitions" in n]
# query heads per kv head, head_dim, type
HEADS = [(1, 64, wl.F16), (4, 128, wl.BF16), (16, 128, wl.F16), (16, 64, wl.BF16), (1, 128, wl.BF16)]

# Chunks: lengths, chunk lengths, query heads, kv heads, head_dim, type, window
PREFILL = {
    "decode kernel, few runs": ([700, 40, 300], [2, 1, 2], 8, 2, 64, wl.F16, 250),
    "decode kernel, a warp per run": ([90] * 40, [4, 1, 3, 2] * 10, 64, 32, 128, wl.BF16, 60),
    "decode kernel, partitions": ([2900, 2600] + [40] * 88, [2, 1] * 45, 8, 2, 128, wl.BF16, 2500),
    "two query tiles": ([700, 300, 150, 160] * 10, [150] * 40, 8, 4, 64, wl.BF16, 333),
    "two query tiles, f16": ([700, 300, 150, 160] * 10, [150] * 40, 8, 4, 128, wl.F16, 333),
    "one query tile, ranges": ([2600, 90], [32, 20], 32, 8, 128, wl.BF16, 2300),
    "one query tile, f16 ranges": ([2600, 90], [42, 20], 48, 16, 64, wl.F16, 2300),
    "two query tiles, ranges": ([2600], [400], 4, 4, 64, wl.BF16, 2100),
    "wide group": ([500, 90], [7, 20], 43, 1, 128, wl.BF16, 300),
}


def decode_problem(name, group, d, dtype, sinks=1, seed=0):
    """The first sequences are as long as the shape needs, the others short,
    so that the 64-bit form stays quick."""
    seqs, hkv, window, beyond = DECODE[name]
    rng = wl.rng_for(window + group + d + seed)
    lens = rng.integers(1, 70, size=seqs)
    top = window + BS * beyond - 3
    lens[:3] = [top, top // 2, window + 1][:min(3, seqs)]
    lens[seqs // 2] = top - 5
    return Windowed(rng, lens, np.ones(seqs, int), group * hkv, hkv, d, dtype, window, sinks)


def prefill_problem(name, sinks, seed=0):
    lens, chunk, hq, hkv, d, dtype, window = PREFILL[name]
    rng = wl.rng_for(window + hq + seed)
    return Windowed(rng, lens, np.minimum(lens, chunk), hq, hkv, d, dtype, window, sinks)


DIM = 3  # the element of a key that is not finite
ONE = {wl.F16: 0x3C00, wl.BF16: 0x3F80}


def spoil(p, s, tokens, bits):
    """Set element DIM of the keys of sequence s's tokens, in the cache too."""
    for t in tokens:
        p.k[s][t][:, DIM] = bits
        b = p.tables[s, t // BS]
        if b >= 0 and p.any_seen[s][t]:
            p.key_cache[b, :, t % BS] = p.k[s][t]


def not_finite(p, kind):
    """Make visible scores of every second sequence -infinity ("first": the
    first seen token, "half": the first half of the seen ones, "all": every
    one), +infinity or NaN (one token), or its queries NaN."""
    q_one = ONE[p.dtype]
    p.q[..., DIM] = q_one if kind == "+inf" else q_one | 0x8000
    for s in range(0, len(p.lens), 2):
        seen = np.nonzero(p.any_seen[s])[0]
        if not len(seen):
            continue
        if kind == "nan query":
            p.q[p.start[s]:p.start[s + 1], ::2, 5] = NAN_BITS[p.dtype]
            continue
        tokens = {"first": seen[:1], "half": seen[:(len(seen) + 1) // 2], "all": seen,
                  "+inf": seen[:1], "nan": seen[:1]}[kind]
        spoil(p, s, tokens, NAN_BITS[p.dtype] if kind == "nan" else INF_BITS[p.dtype])


KINDS = ["first", "half", "all", "+inf", "nan", "nan query"]


def worst(got, p):
    """Largest error over the tolerance; NaN has to stand where the definition
    gives it, and nowhere else."""
    with np.errstate(invalid="ignore", over="ignore"):
        ref, tol = p.reference()
    assert np.array_equal(np.isnan(got), np.isnan(ref)), "NaN in the wrong rows"
    ok = ~np.isnan(ref)
    assert np.all(np.isfinite(got[ok]))
    return float(np.max(np.abs(got - ref)[ok] / tol[ok])) if ok.any() else 0.0
