"""The plain GEMMs captured into a graph and replayed on new tokens.

A stream-K launch hands partial sums on under flags that carry its sequence
number, and every replay of a captured launch carries the same one: the owner
of a tile clears the flags that it has seen, so that a replay waits for its own
sums.  Bound: fp32 sums (ffn_testutil.sum_bound, twice where a tile is split)
and one rounding to bf16.
"""
import pytest
import torch

from ffn_testutil import HALF_STEP, assert_within, layer, randn, sum_bound

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nm():
    import semi_structured_sparse_diag_b200 as nm
    nm.load()
    return nm


def test_sparse_gemm_replayed_with_other_tokens(nm):
    # the plain products' stream-K flags under replay: the sums are this replay's
    T, R, K, m = 16, 512, 4096, 4
    X = randn(T, K, 1.0, seed=1)
    proj = layer(nm, R, K, m, seed=2)
    nm.set_gemm_schedule(2, 0)
    try:
        nm.sparse_gemm(X, proj["packed"], R, m), nm.dense_gemm(X, proj["dense"])
        torch.cuda.synchronize()
        nm.set_poison(False)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = nm.sparse_gemm(X, proj["packed"], R, m), nm.dense_gemm(X, proj["dense"])
        for i in range(8):
            X.copy_(randn(T, K, 1.0, seed=30 + i))
            g.replay()
            torch.cuda.synchronize()
            nm.check_device_error()
            want = X.double() @ proj["w64"].T
            for Y in outs:
                assert_within(Y, want, HALF_STEP * want.abs() + 2 * sum_bound(X.double(), proj["w64"]) + 1e-30, "Y")
    finally:
        nm.set_gemm_schedule(0, 0)
