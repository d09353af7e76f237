"""The adapter call on more than 65535 token tiles (of at most 240 tokens): what it
takes depends on the sizes that the header names, not on the tile width that the
schedule picks.  Bounds: test_gpu_lora.py's, on the tokens around every border (all
of them would take minutes in fp64)."""
import pytest
import torch

import test_gpu_lora
from ffn_testutil import layer

pytestmark = pytest.mark.gpu

T = 65535 * 240 + 1  # the last token is a tile of its own behind 65535 full ones


@pytest.fixture(scope="module")
def nm():
    import semi_structured_sparse_diag_b200 as nm
    nm.load()
    return nm


# mma.sync, and with 904 columns and rank 24 tcgen05 (28 GB of X); no requests at all
@pytest.mark.parametrize("K,r,indptr,ids", [(8, 8, [0, 100, 65534 * 240 - 3, T], [1, 0, 1]), (8, 8, [0], []),
                                            (904, 24, [0, 100, 65534 * 240 - 3, T], [1, -1, 0])])
def test_many_tokens(nm, K, r, indptr, ids):
    R, m, n = 8, 4, 2
    g = torch.Generator(device="cuda").manual_seed(K)
    X = torch.empty((T, K), dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    proj = layer(nm, R, K, m, seed=1)
    A, B, scale = test_gpu_lora._adapters(n, r, R, K, seed=2)
    Y = nm.sparse_gemm_lora(X, proj["packed"], R, m, A, B, scale, test_gpu_lora._i32(indptr), test_gpu_lora._i32(ids))
    torch.cuda.synchronize()
    nm.check_device_error()
    assert not bool(Y.isnan().any())
    for lo, hi in ((0, 500), (32768 * 240 - 300, 32768 * 240 + 300), (65533 * 240, T)):
        cut = [min(max(c, lo), hi) - lo for c in indptr]
        test_gpu_lora._check(X[lo:hi], proj, A, B, scale, test_gpu_lora._i32(cut), test_gpu_lora._i32(ids), Y[lo:hi])
