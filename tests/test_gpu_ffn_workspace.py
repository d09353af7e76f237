"""Workspaces that a caller gives the feed-forward operators: a tensor whose bytes
are not one after another is refused, not written through."""
import pytest
import torch

import test_gpu_lora
from ffn_testutil import layer, randn

pytestmark = pytest.mark.gpu


def test_strided_workspaces_are_refused():
    import semi_structured_sparse_diag_b200 as nm
    T, K, R, m, r, n = 16, 64, 40, 8, 8, 2
    X, dH = randn(T, K, 1.0, seed=1), randn(T, R, 1.0, seed=2)
    side = layer(nm, R, K, m, seed=3)
    A, B, scale = test_gpu_lora._adapters(n, r, R, K, seed=4)
    indptr, ids = test_gpu_lora._i32([0, T]), test_gpu_lora._i32([1])
    lib = nm.load()
    for need, call in (
            (lib.nm_sparse_glu_workspace_bytes(T, K, m),
             lambda ws: nm.sparse_glu(X, side["packed"], side["packed"], R, m, ws=ws)),
            (lib.nm_sparse_glu_backward_workspace_bytes(T, R),
             lambda ws: nm.sparse_glu_backward(dH, X, dH, dH, side["dense"], side["dense"], ws=ws)),
            (lib.nm_sparse_gemm_lora_workspace_bytes(T, K, m, r, n, 1),
             lambda ws: nm.sparse_gemm_lora(X, side["packed"], R, m, A, B, scale, indptr, ids, ws=ws))):
        assert need > 0
        both = torch.full((need, 2), 7, dtype=torch.uint8, device="cuda")
        with pytest.raises(nm.NMError, match="contiguous"):
            call(both[:, 0])
        torch.cuda.synchronize()
        assert bool((both == 7).all())
        call(torch.empty(need, dtype=torch.uint8, device="cuda"))
        torch.cuda.synchronize()
        nm.check_device_error()
