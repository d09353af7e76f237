"""Request lists of the adapter call that are wrong in ways that its blocks could
read differently.  The blocks of a cluster each work out their tile's slots and
meet at one barrier per slot and round of tokens, so they have to come to the same
plan whatever the list holds.  The outputs of such a call are unspecified: what is
checked is that it ends, reports the list, repeats itself where one tile holds
all tokens, and leaves the next call right."""
import pytest
import torch

import test_gpu_lora
from ffn_testutil import layer, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nm():
    import semi_structured_sparse_diag_b200 as nm
    nm.load()
    return nm


def _colliding(T, requests):
    # every second request starts on token 0, with another end and another adapter;
    # those between run backwards.  More requests than a block has threads.
    ends = [1 + (37 * i) % T for i in range(requests // 2 + 1)]
    return [0 if i % 2 == 0 else ends[i // 2] for i in range(requests + 1)]


# one tile and several; mma.sync and (1024 tokens and up, rank above 16) tcgen05
@pytest.mark.parametrize("T,R,K,m,r,n,requests", [(200, 264, 256, 4, 8, 5, 300), (240, 264, 520, 8, 40, 7, 700),
                                                  (900, 264, 256, 6, 16, 5, 300), (4096, 264, 904, 4, 24, 5, 250)])
def test_requests_that_start_on_one_token(nm, T, R, K, m, r, n, requests):
    X = randn(T, K, 1.0, seed=1)
    proj = layer(nm, R, K, m, seed=2)
    A, B, scale = test_gpu_lora._adapters(n, r, R, K, seed=3)
    args = (X, proj["packed"], R, m, A, B, scale)
    bad = test_gpu_lora._i32(_colliding(T, requests)), test_gpu_lora._i32([(3 * i) % n for i in range(requests)])
    outs = []
    for _ in range(3):
        outs.append(nm.sparse_gemm_lora(*args, *bad))
        with pytest.raises(nm.NMError, match="NM_ERR_DEVICE"):
            nm.check_device_error()
    if T <= 240:
        assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
    good = test_gpu_lora._i32([T * i // requests for i in range(requests + 1)]), bad[1]
    Y = nm.sparse_gemm_lora(*args, *good)
    torch.cuda.synchronize()
    nm.check_device_error()
    test_gpu_lora._check(X, proj, A, B, scale, *good, Y)
