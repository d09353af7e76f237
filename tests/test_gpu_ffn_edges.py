"""Calls of the feed-forward operators that their documentation allows and that the
other files leave out.  Bounds: test_gpu_glu.py's and test_gpu_lora.py's."""
import pytest
import torch

import test_gpu_glu
import test_gpu_lora
from ffn_testutil import layer, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nm():
    import semi_structured_sparse_diag_b200 as nm
    nm.load()
    return nm


def _sync_ok(nm):
    torch.cuda.synchronize()
    nm.check_device_error()


@pytest.mark.parametrize("m", [6, 8, 10])
def test_staged_patterns_replayed_on_other_inputs(nm, m):
    # the staging kernel, V and the product start before their predecessors end: what
    # each replay reads are the values written just before it, by kernels that read
    # and write the same arrays
    T, R, K, r, n = 50, 520, 1024, 16, 6
    X, next_x = randn(T, K, 1.0, seed=1), randn(T, K, 1.0, seed=2)
    proj = layer(nm, R, K, m, seed=3)
    A, B, scale = test_gpu_lora._adapters(n, r, R, K, seed=4)
    indptr, ids = test_gpu_lora._i32(list(range(T + 1))), test_gpu_lora._i32([i % n for i in range(T)])
    ws = torch.empty(nm.load().nm_sparse_gemm_lora_workspace_bytes(T, K, m, r, n, T), dtype=torch.uint8, device="cuda")

    def step():
        X.copy_(X.roll(1, 0) * 0.5 + next_x)
        ids.copy_((ids * 5 + 2) % (n + 1) - 1)
        A.copy_(A.flip(0))
        scale.mul_(-1)
        return nm.sparse_gemm_lora(X, proj["packed"], R, m, A, B, scale, indptr, ids, ws=ws)

    ids.clamp_(min=0)
    step()
    torch.cuda.synchronize()
    nm.set_poison(False)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        Y = step()
    for _ in range(6):
        ids.add_(1)
        Y.fill_(float("nan"))
        g.replay()
        _sync_ok(nm)
        test_gpu_lora._check(X, proj, A, B, scale, indptr, ids, Y)


@pytest.mark.parametrize("m", [4, 6, 8, 10])
@pytest.mark.parametrize("T", [1, 300])
def test_no_requests(nm, m, T):
    R, K = 264, 1003
    X = randn(T, K, 1.0, seed=1)
    proj = layer(nm, R, K, m, seed=2)
    A, B, scale = test_gpu_lora._adapters(2, 8, R, K, seed=3)
    Y = nm.sparse_gemm_lora(X, proj["packed"], R, m, A, B, scale, test_gpu_lora._i32([0]), test_gpu_lora._i32([]))
    _sync_ok(nm)
    test_gpu_lora._check(X, proj, A, B, scale, test_gpu_lora._i32([0]), test_gpu_lora._i32([]), Y)


def test_bit_patterns_and_given_outputs(nm):
    # bf16 as 16-bit patterns, outputs of the caller's with rows further apart
    T, R, K, m, r, n = 40, 264, 320, 6, 8, 3
    X, dH = randn(T, K, 1.0, seed=1), randn(T, R, 0.1, seed=2)
    gate, up = layer(nm, R, K, m, seed=3), layer(nm, R, K, m, seed=4)
    A, B, scale = test_gpu_lora._adapters(n, r, R, K, seed=5)
    req = test_gpu_lora._i32([0, 10, 40]), test_gpu_lora._i32([2, 0])
    out = [torch.full((T, 400), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    nm.sparse_glu(X.view(torch.int16), gate["packed"], up["packed"], R, m, H=out[0][:, :R].view(torch.int16))
    nm.sparse_gemm_lora(X.view(torch.uint16), gate["packed"], R, m, A.view(torch.int16), B.view(torch.uint16), scale, *req,
                        Y=out[1][:, :R])
    H, G, U = nm.sparse_glu(X, gate["packed"], up["packed"], R, m, save=True)
    a = nm.sparse_glu_backward(dH, X, G, U, gate["dense"], up["dense"])
    b = nm.sparse_glu_backward(dH.view(torch.int16), X.view(torch.int16), G, U.view(torch.uint16), gate["dense"].view(torch.int16),
                               up["dense"])
    _sync_ok(nm)
    assert torch.equal(out[0][:, :R], H)
    test_gpu_lora._check(X, gate, A, B, scale, *req, out[1][:, :R])
    assert all(bool((o[:, R:] == 7.0).all()) for o in out)
    assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_calls_at_once(nm):
    # backward passes and adapters of two streams side by side, each with its own workspace
    T, R, K = 300, 520, 640
    streams = [torch.cuda.Stream() for _ in range(2)]
    sets = [test_gpu_glu._backward_inputs(nm, T, R, K, m, seed=m) for m in (4, 8)]
    A, B, scale = test_gpu_lora._adapters(4, 16, R, K, seed=5)
    req = test_gpu_lora._i32([0, 10, 90, 300]), test_gpu_lora._i32([0, 3, 1])
    outs = []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        for (X, dH, G, U, gate, up), s, m in zip(sets, streams, (4, 8)):
            outs.append((nm.sparse_glu_backward(dH, X, G, U, gate["dense"], up["dense"], stream=s),
                         nm.sparse_gemm_lora(X, gate["packed"], R, m, A, B, scale, *req, stream=s)))
    for s in streams:
        torch.cuda.current_stream().wait_stream(s)
    _sync_ok(nm)
    for i, (grads, Y) in enumerate(outs):
        X, dH, G, U, gate, up = sets[i % 2]
        test_gpu_glu._check_backward(X, dH, G, U, gate, up, "silu", False, grads)
        test_gpu_lora._check(X, gate, A, B, scale, *req, Y)
