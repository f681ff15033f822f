"""MXFP4 operators on the GPU where memory, scales and logits are at their ends,
against the float64 oracle; bounds as derived in tests/test_gpu_mx4.py."""
import numpy as np
import pytest

from oracle import mx4_oracle as M
from tests import _gpu as G
from tests import test_gpu_mx4 as B

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------------------
# what lies behind a tensor
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("m,n,k", [(17, 129, 17440), (64, 130, 17440), (33, 257, 13344), (9, 4613, 17440)])
def test_linear_whatever_follows_the_scales(m, n, k):
    """n k / 32 bytes of scales end inside a dword: what else it holds is not the
    weight's, and the same call gives the same bits over it."""
    import torch
    import gemm_exl3_linear_amd as X
    rng = np.random.default_rng(m + n)
    codes, scales = B.rand_mx(rng, n, k, lo=112, hi=122)
    size = scales.size
    assert size % 4
    room = torch.zeros(size + 64, dtype=torch.uint8, device=G.dev())
    room[:size] = G.to_dev(scales).reshape(-1)
    w = X.Exl3Mx4(G.to_dev(codes), room[:size].view(n, k // 32))
    x = rng.standard_normal((m, k)).astype(np.float16)
    xd = G.to_dev(x)
    got = []
    for fill in (0, 255, 90):
        room[size:] = fill
        got.append(X.exl3_mx4_linear(xd, w, out_dtype=torch.float32))
    cols = np.unique(np.concatenate([np.arange(0, n, max(1, n // 200)), np.arange(n - 2, n)]))
    ref, mag = M.product(x, M.decode(codes[cols], scales[cols]))
    B.assert_within(got[0].cpu().numpy()[:, cols], ref, B.bound(ref, mag, k, True))
    assert torch.equal(got[0], got[1]) and torch.equal(got[0], got[2])
