"""The feed-forward operators together, as a user runs them: a decode step of a
block captured into a graph, a training step of a gated layer, and the calls
that the binding refuses.  Bounds: the sub-steps' own (test_gpu_glu.py,
test_gpu_lora.py), each step checked on the inputs that it was given."""
import pytest
import torch

import test_gpu_glu
import test_gpu_lora
from ffn_testutil import HALF_STEP, act64, assert_within, keep_bits, layer, randn, sum_bound

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nm():
    import semi_structured_sparse_diag_b200 as nm
    nm.load()
    return nm


def _sync_ok(nm):
    torch.cuda.synchronize()
    nm.check_device_error()


@pytest.mark.parametrize("m", [4, 8])
def test_decode_block_captured(nm, m):
    # gate and up, then the down projection with the requests' adapters and, beside
    # it, the plain one: twelve requests of a token each, replayed on new tokens
    T, D, F, r, n = 12, 512, 768, 16, 4
    X = randn(T, D, 1.0, seed=1)
    gate, up, down = layer(nm, F, D, m, seed=2), layer(nm, F, D, m, seed=3), layer(nm, D, F, m, seed=4)
    A, B, scale = test_gpu_lora._adapters(n, r, D, F, seed=5)
    indptr, ids = test_gpu_lora._i32(list(range(T + 1))), test_gpu_lora._i32([i % (n + 1) - 1 for i in range(T)])

    def step():
        H = nm.sparse_glu(X, gate["packed"], up["packed"], F, m)
        return H, nm.sparse_gemm_lora(H, down["packed"], D, m, A, B, scale, indptr, ids), nm.sparse_gemm(H, down["packed"], D, m)

    step()
    torch.cuda.synchronize()
    nm.set_poison(False)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        H, Y, Z = step()
    for i in range(4):
        X.copy_(randn(T, D, 1.0, seed=10 + i))
        ids.copy_(ids.roll(1))
        for t in (H, Y, Z):
            t.fill_(float("nan"))
        g.replay()
        _sync_ok(nm)
        test_gpu_glu._check_glu(X, gate, up, "silu", H)
        test_gpu_lora._check(H, down, A, B, scale, indptr, ids, Y)
        z = H.double() @ down["w64"].T
        assert_within(Z, z, HALF_STEP * z.abs() + 2 * sum_bound(H.double(), down["w64"]) + 1e-30, "Z")


def test_training_step(nm):
    # prune by the Hessian score, forward, backward, a step on the latent weights:
    # the loss's change is what the gradients say
    T, D, F, m = 192, 320, 256, 8
    X, dH = randn(T, D, 1.0, seed=1), randn(T, F, 0.1, seed=2)
    W = [randn(F, D, 0.05, seed=3 + i) for i in range(2)]
    H64 = nm.hessian_diag(X)
    sides = []
    for w in W:
        mask, vals, _ = nm.score_prune_compress(H64, w, m - 2, m)
        dense = nm.sparse_densify(vals, mask, F, D, m - 2, m)
        sides.append(dict(mask=mask, dense=dense, w64=dense.double(), packed=nm.sparse_prepare_from_mask(vals, mask, F, D, m)))
    gate, up = sides
    H, G, U = nm.sparse_glu(X, gate["packed"], up["packed"], F, m, save=True)
    dX, dWg, dWu = nm.sparse_glu_backward(dH, X, G, U, gate["dense"], up["dense"], mask_gate=gate["mask"], mask_up=up["mask"], m=m)
    _sync_ok(nm)
    test_gpu_glu._check_glu(X, gate, up, "silu", (H, G, U))
    test_gpu_glu._check_backward(X, dH, G, U, gate, up, "silu", True, (dX, dWg, dWu))
    for got, side in ((dWg, gate), (dWu, up)):
        assert bool((got[~keep_bits(side["mask"], D)] == 0).all())

    def loss(wg, wu):
        x = X.double()
        return (dH.double() * act64(x @ wg.T, "silu") * (x @ wu.T)).sum()

    # along the gradients themselves: central differences in fp64 against |dW|^2;
    # dW is off by less than 2^-7 in the 2-norm (two roundings, and those of G and U)
    h = 1e-5
    g, u = dWg.double(), dWu.double()
    slope = float((loss(gate["w64"] + h * g, up["w64"] + h * u) - loss(gate["w64"] - h * g, up["w64"] - h * u)) / (2 * h))
    want = float(g.norm() ** 2 + u.norm() ** 2)
    assert abs(slope - want) <= 2.0 ** -6 * want


def test_one_row_of_any_stride(nm):
    # a single token: its row stride does not matter
    K, R, m = 1003, 520, 4
    x = torch.randn(1, K, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    assert x.stride(0) % 8 != 0
    gate, up = layer(nm, R, K, m, seed=2), layer(nm, R, K, m, seed=3)
    H, G, U = nm.sparse_glu(x, gate["packed"], up["packed"], R, m, save=True)
    _sync_ok(nm)
    test_gpu_glu._check_glu(x, gate, up, "silu", (H, G, U))


def test_binding_refusals(nm):
    T, K, R, m = 16, 64, 40, 4
    X, dH = randn(T, K, 1.0, seed=1), randn(T, R, 1.0, seed=2)
    side = layer(nm, R, K, m, seed=3)
    packed, W, mask = side["packed"], side["dense"], side["mask"]
    A, B, scale = test_gpu_lora._adapters(2, 8, R, K, seed=4)
    indptr, ids = test_gpu_lora._i32([0, T]), test_gpu_lora._i32([1])
    lora = lambda **kw: nm.sparse_gemm_lora(**{**dict(X=X, packed=packed, R=R, m=m, A=A, B=B, scale=scale, indptr=indptr, ids=ids), **kw})
    back = lambda **kw: nm.sparse_glu_backward(**{**dict(dH=dH, X=X, G=dH, U=dH, Wg=W, Wu=W), **kw})
    bad = [
        lambda: nm.sparse_glu(X, packed, packed, R, m, act="tanh"), lambda: nm.sparse_glu(X.float(), packed, packed, R, m),
        lambda: nm.sparse_glu(X[0], packed, packed, R, m), lambda: nm.sparse_glu(X.t(), packed, packed, R, m),
        lambda: nm.sparse_glu(X, packed, packed[:-1], R, m), lambda: nm.sparse_glu(X, packed, packed, R, 5),
        lambda: nm.sparse_glu(X, packed, packed, R, m, H=dH[:, :8]), lambda: nm.sparse_glu(X, packed, packed.cpu(), R, m),
        lambda: nm.sparse_glu(X[:0], packed, packed, R, m), lambda: nm.sparse_glu(X[:1].expand(T, K), packed, packed, R, m),
        lambda: nm.sparse_glu(X, packed, packed, R, 8, ws=torch.empty(16, dtype=torch.uint8, device="cuda")),
        lambda: back(dH=dH[:8]), lambda: back(Wg=W[:, :32]), lambda: back(G=dH.float()), lambda: back(act="silu2"),
        lambda: back(need_dx=False, need_dw=False), lambda: back(mask_gate=mask), lambda: back(mask_gate=mask, mask_up=mask),
        lambda: back(mask_gate=mask[:, :1], mask_up=mask, m=m), lambda: back(X=X.cpu()),
        lambda: back(ws=torch.empty(16, dtype=torch.uint8, device="cuda")),
        lambda: nm.sparse_densify(side["vals"], mask, R, K, 3, m), lambda: nm.sparse_densify(side["vals"], mask, R, K, 4, 4),
        lambda: lora(A=A[0]), lambda: lora(A=A[:, :4]), lambda: lora(B=B[:, :8]), lambda: lora(scale=scale.double()),
        lambda: lora(scale=scale[:1]), lambda: lora(indptr=indptr.long()), lambda: lora(indptr=indptr[:1]),
        lambda: lora(ids=ids.cpu()), lambda: lora(A=A[:1].expand(2, 8, K)), lambda: lora(Y=dH[:8]), lambda: lora(X=X[:0]),
        lambda: lora(ws=torch.empty(16, dtype=torch.uint8, device="cuda")),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(nm.NMError):
            call()
            pytest.fail(f"call {i} was not refused")
    _sync_ok(nm)
