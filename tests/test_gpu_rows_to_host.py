"""Blocks of a row-scaled cache read back into pinned host memory, as the block moves write theirs."""
import pytest
import torch

from tests import _gpu
from tests import _ref64 as R
from tests.test_gpu_cache_ops import gen, rows_pool

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt,D,bs", [("bf16", 128, 16), ("f16", 64, 8)])
def test_read_back_to_pinned_memory(dt, D, bs):
    pa = _gpu.lib()
    NB, Hkv = 7, 3
    k, v, ks, vs = rows_pool(gen(D), NB, Hkv, bs, D)
    pool = [t.cuda() for t in (k, v, ks, vs)]
    ids = torch.tensor([5, 0, NB, 3])
    host = [torch.full((4, Hkv, bs, D), 3.0, dtype=R.DT[dt], pin_memory=True) for _ in range(2)]
    pa.gather_blocks_rows(*host, *pool, ids.cuda())
    torch.cuda.synchronize()
    assert pa.get_device_error() == pa.DEVERR_BLOCK_ID
    for dst, codes, s in ((host[0], k, ks), (host[1], v, vs)):
        want = (codes.float() * s[..., None]).to(R.DT[dt])
        assert torch.equal(dst[[0, 1, 3]], want[[5, 0, 3]]) and (dst[2] == 3).all()
    for bad in (torch.zeros(4, Hkv, bs, D, dtype=R.DT[dt]), host[0][:, :, :, ::2], host[0].float().pin_memory()):
        with pytest.raises((ValueError, TypeError)):
            pa.gather_blocks_rows(bad, host[1], *pool, ids.cuda())
        with pytest.raises((ValueError, TypeError)):
            pa.gather_blocks_rows(host[0], bad, *pool, ids.cuda())
    assert pa.get_device_error() == 0
