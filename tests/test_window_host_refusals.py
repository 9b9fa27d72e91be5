"""Calls of the windowed and rotary binding that are refused on the host, before
any address reaches the library (no GPU needed)."""
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
