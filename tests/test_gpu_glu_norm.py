"""The gated product in the 2-norm.  G, U and H are each rounded once to bf16 (rms at
most 2^-8 / sqrt 3 of a value), so their errors stay below 2^-8 in the 2-norm by a
wide margin; an element's own bound (test_gpu_glu.py) allows for sums that are
large next to their result, and would not see partial sums kept in fewer bits
than fp32.  An fp32 sum's part is below 2^-12 here: (K + 32) 2^-23 of the sum of
magnitudes, at most sqrt(K) times the result's size in the norm."""
import pytest
import torch

from ffn_testutil import act64, layer, norm_error, randn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,R,K,m,act", [(16, 1000, 4096, 4, "silu"), (333, 520, 2050, 8, "gelu"), (700, 600, 1003, 6, "relu2"),
                                         (90, 300, 2010, 10, "silu")])
@pytest.mark.parametrize("policy", [0, 1, 2])
def test_norm(T, R, K, m, act, policy):
    import semi_structured_sparse_diag_b200 as nm
    X = randn(T, K, 1.0, seed=T)
    gate, up = layer(nm, R, K, m, seed=R), layer(nm, R, K, m, seed=R + 1)
    nm.set_gemm_schedule(policy, 0)
    try:
        H, G, U = nm.sparse_glu(X, gate["packed"], up["packed"], R, m, act=act, save=True)
    finally:
        nm.set_gemm_schedule(0, 0)
    torch.cuda.synchronize()
    nm.check_device_error()
    g, u = X.double() @ gate["w64"].T, X.double() @ up["w64"].T
    for got, want in ((G, g), (U, u), (H, act64(g, act) * u)):
        assert norm_error(got, want) < 2.0 ** -8
