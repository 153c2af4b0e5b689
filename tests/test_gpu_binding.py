"""What the native binding raises, and what it takes: errors of torch under their own types."""
import pytest
import torch

pytestmark = pytest.mark.gpu
CH = 64


@pytest.fixture(scope="module")
def L():
    from learned_sparse_kv_b200 import lsa
    return lsa


def test_memory_that_is_not_there_is_torchs_error(L):
    """Outputs of many terabytes: torch.OutOfMemoryError, a RuntimeError, as the other calls raise it; the next call works."""
    pool = L.q4_pool(1, 1, 576)
    ints = torch.zeros(1, dtype=torch.int32, device="cuda")
    wide = L.q4_pool(1, 1024, 4096)
    with pytest.raises(torch.OutOfMemoryError):
        L.read_q4(wide, torch.full((1 << 20,), -1, dtype=torch.int64, device="cuda"), out_dtype=torch.float32)
    with pytest.raises(torch.OutOfMemoryError):
        L.qk_norm_rope(torch.zeros(1, 1, 1024, device="cuda").expand(1 << 24, 1024, 1024), None, ints, ints.float())
    q = torch.zeros(1, 1, 576, device="cuda", dtype=torch.bfloat16)
    with pytest.raises(RuntimeError, match="out of memory"):
        L.sparse_decode_q4(q.expand(60000, 1 << 19, 576), pool, None, ints[None], None, None, ints, ints, 64, 512, 1.0)
    out, lse = L.sparse_decode_q4(q, pool, None, ints[None], None, None, ints, ints + 3, 64, 512, 1.0)
    assert bool((out == 0).all()) and torch.allclose(lse, torch.log(torch.tensor(3.0, device="cuda")))
