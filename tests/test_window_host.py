"""Windows that cannot run are refused with the library's error before anything is allocated (no GPU needed)."""
import pytest
import torch

from learned_sparse_kv_b200 import build as lbuild


@pytest.mark.parametrize("latent", [False, True])
def test_cold_4bit_pools_are_refused(latent):
    lbuild.build()
    from learned_sparse_kv_b200 import lsa
    from learned_sparse_kv_b200.decode import Shapes, Window
    dqk, dv = (576, 512) if latent else (128, 128)
    sh = Shapes(B=1, Hn=2, dn=64, Hl=2, dl=64, k=64, Hq=16, dqk=dqk, dv=dv, latent=latent, window=64, steps=1, scale=1.0)
    pool = torch.zeros(4, 1, 36 * dqk, dtype=torch.uint8)
    t = dict(q=torch.zeros(1, 1, 16, dqk), khat=torch.zeros(4, 64), kv=pool, k=pool, v=pool, li=torch.zeros(4, 64, 64))
    with pytest.raises(lsa.LSAError, match="4-bit"):
        Window(sh, t, 4, 4, cold=dict(host_pools=[pool], dev_pools=[pool], first_window_chunk=1))
