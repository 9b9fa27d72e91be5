"""Calls of the windowed and rotary binding that are refused on the host, before
any address reaches the library, and the limits of those that are not (no GPU
needed)."""
from fractions import Fraction

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pk = pytest.importorskip("paged_kv_cache_425_b200")


@pytest.mark.parametrize("shape", [(3, 4, 64), (3, 4, 120), (3, 4, 256), (3, 512), (3, 4, 2, 64)])
def test_rope_refuses_a_q_out_of_another_head_dim(shape):
    """The kernel stores head_dim elements per head: a narrower q_out would be
    written past its end.  The check comes before the one of the device, so
    host tensors show it."""
    q, k = torch.zeros(3, 4, 128, dtype=torch.float16), torch.zeros(3, 2, 128, dtype=torch.float16)
    cache = torch.zeros(2, 2, 16, 128, dtype=torch.float16)
    rope = pk.Rope(np.ones(32))
    with pytest.raises(ValueError, match="q_out must be"):
        pk.rope_and_cache(torch.zeros(shape, dtype=torch.float16), q, k, k, cache, cache.clone(),
                          torch.zeros(3, dtype=torch.int64), torch.zeros(1, 3, dtype=torch.int32), rope)


def inverse_turn(bits):
    """1 / (2 pi) within 2^-bits: pi by Machin's formula in exact arithmetic."""
    def arctan_of_inverse(n):
        total, k, term = 0, 0, (1 << (bits + 16)) // n
        while term:
            total += (-1) ** k * (term // (2 * k + 1))
            term //= n * n
            k += 1
        return total
    pi = 4 * (4 * arctan_of_inverse(5) - arctan_of_inverse(239))
    return Fraction(1 << (bits + 16), 2 * pi)


def test_rope_angles_keep_their_bound():
    """Position times the stored step against exact arithmetic: at most
    2^-32 + |inv_freq| 2^-34 of a turn for every int32 position."""
    inv = inverse_turn(160)
    rng = np.random.default_rng(5)
    freq = np.concatenate([np.exp(rng.uniform(np.log(1e-9), np.log(128), size=46)) * rng.choice([-1, 1], size=46),
                           [128, -128, 127.99999, 1, -1, 2.0 ** -149, -2.0 ** -149, 0.0, -1e-30, 6.2831855]])
    freq = freq.astype(np.float32)
    rope = pk.Rope(np.concatenate([freq, np.zeros(-len(freq) % 8, np.float32)]))
    for f, step in zip(freq, rope._struct.turns):
        for p in (1, -1, 12345, 2 ** 31 - 1, -2 ** 31):
            d = (Fraction(p * step, 2 ** 64) - p * Fraction(float(f)) * inv) % 1
            assert min(d, 1 - d) <= Fraction(1, 2 ** 32) + abs(Fraction(float(f))) / 2 ** 34


@pytest.mark.parametrize("f", [128.00002, -129.0, 1e6, -1e12, 3e38])
def test_rope_refuses_frequencies_beyond_its_bound(f):
    """A step that cannot be held closely enough turned far tokens by anything."""
    with pytest.raises(pk.PagedError) as e:
        pk.Rope(np.array([1.0] * 7 + [f], np.float32))
    assert e.value.status == pk.PA_ERR_UNSUPPORTED


def test_decode_window_takes_tables_as_wide_as_documented():
    """2^26 blocks per sequence: the refusals that follow the width's check are
    reached (nothing is launched)."""
    import ctypes
    p = ctypes.c_void_p(4096)  # aligned, never dereferenced

    def call(width, window, ws=None):
        tail = (p, p, window, 4, 2, 0.1, 100, 8, 64, 16, width, 100, 0, ws, 0, None)
        return (pk.pa_decode_window(p, p, p, p, *tail), pk.pa_decode_append_window(p, p, None, p, p, p, *tail))
    assert call(1 << 26, 5000) == (pk.PA_ERR_WORKSPACE, pk.PA_ERR_INVALID_ARG)
    assert call((1 << 26) + 1, 5000) == (pk.PA_ERR_UNSUPPORTED,) * 2
    # more than 65535 partitions: the part of pa_decode_window that stays refused
    assert call(1 << 26, 2 ** 31 - 1)[0] == pk.PA_ERR_UNSUPPORTED


@pytest.mark.parametrize("args", [(64, 2 ** 32 + 16, 0), (64, 16, 2 ** 32), (2 ** 32 + 64, 16, 0), (64, 2 ** 63, 0)])
def test_trim_refuses_arguments_that_do_not_fit_32_bits(args):
    """Cut to 32 bits, a window of 2^32 + 16 would free blocks that are in sight."""
    a = pk.BlockAllocator(8)
    a.add_seq(1, 64)
    with pytest.raises(ValueError, match="32 bits"):
        a.trim_window(1, *args)
    assert (a.block_table(1) >= 0).all() and a.stats()["used_blocks"] == 4
