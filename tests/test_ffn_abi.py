"""Host-side checks of the feed-forward and adapter calls (no GPU needed):
workspace sizes, and bad calls refused by the library and by the binding before
anything is launched."""
import pytest
import torch

import semi_structured_sparse_diag_b200 as nm

A = 0x10000    # fake but 16-byte aligned device addresses: refused before any use
MIS = 0x10002
BIG = 1 << 40


def test_workspace_sizes():
    lib = nm.load()
    up = lambda b: (b + 255) // 256 * 256
    # gated product: the staged activations only
    assert lib.nm_sparse_glu_workspace_bytes(2048, 4096, 4) == 0
    assert lib.nm_sparse_glu_workspace_bytes(2048, 4096, 8) == 2048 * 2048 * 2
    assert lib.nm_sparse_glu_workspace_bytes(7, 1003, 6) == 7 * 1344 * 2
    assert lib.nm_sparse_glu_workspace_bytes(0, 64, 4) == 0 and lib.nm_sparse_glu_workspace_bytes(4, 64, 5) == 0
    # its backward pass: dG and dU, rows padded to 8 columns
    assert lib.nm_sparse_glu_backward_workspace_bytes(300, 131) == 2 * up(300 * 136 * 2)
    assert lib.nm_sparse_glu_backward_workspace_bytes(0, 131) == 0
    # adapters: a tile's count and first slot, a slot's adapter, V; tiles of at
    # least 16 tokens, slots of at most 240 rows

    def lora(T, K, m, r, n, q):
        staged = {4: 0, 8: T * ((K + 7) // 8 * 4) * 2}[m]
        cap, tiles = min(q, n, 240), T // 16 + 2
        slots = min(q + tiles, tiles * cap)
        rows = min((q + 1) * 240 + T, (T + 240) * cap)
        return up(staged) + 2 * up(4 * tiles) + up(4 * slots) + up(rows * r * 2)
    for args in ((1, 4096, 4, 16, 8, 1), (128, 4096, 4, 16, 128, 128), (777, 2010, 8, 8, 5, 9), (8192, 4096, 4, 64, 16, 24),
                 (33, 64, 4, 8, 1, 0)):
        assert lib.nm_sparse_gemm_lora_workspace_bytes(*args) == lora(*args)
    for bad in ((0, 64, 4, 8, 1, 1), (4, 64, 5, 8, 1, 1), (4, 64, 4, 4, 1, 1), (4, 64, 4, 12, 1, 1), (4, 64, 4, 264, 1, 1),
                (4, 64, 4, 8, 0, 1), (4, 64, 4, 8, 1, -1)):
        assert lib.nm_sparse_gemm_lora_workspace_bytes(*bad) == 0


def glu(l, X=A, T=4, K=16, ldx=16, g=A, u=A, R=8, m=4, act=0, H=A, ldh=8, G=None, U=None, ldgu=0, ws=None, wsb=0):
    return l.nm_sparse_glu(X, T, K, ldx, g, u, R, m, act, H, ldh, G, U, ldgu, ws, wsb, None)


@pytest.mark.parametrize("kw,expect", [
    (dict(X=None), 1), (dict(g=None), 1), (dict(u=None), 1), (dict(H=None), 1), (dict(G=A), 1), (dict(U=A), 1),
    (dict(T=0), 2), (dict(K=0), 2), (dict(R=0), 2), (dict(ldx=8), 2), (dict(ldh=0), 2), (dict(G=A, U=A, ldgu=4), 2),
    (dict(T=1 << 31), 2), (dict(K=1 << 30, ldx=1 << 30), 2), (dict(R=1 << 31, ldh=1 << 31), 2),
    (dict(m=5), 4), (dict(m=12), 4), (dict(act=3), 4), (dict(act=-1), 4),
    (dict(X=MIS), 3), (dict(g=MIS), 3), (dict(u=MIS), 3), (dict(H=MIS), 3), (dict(ldx=20), 3), (dict(ldh=12), 3),
    (dict(G=MIS, U=A, ldgu=8), 3), (dict(G=A, U=A, ldgu=12), 3), (dict(ws=MIS, wsb=BIG), 3),
    (dict(m=8), 5), (dict(m=6, ws=A, wsb=8), 5),
])
def test_glu_refusals(kw, expect):
    assert glu(nm.load(), **kw) == expect


def backward(l, dH=A, lddh=8, X=A, T=4, K=16, ldx=16, G=A, U=A, ldgu=8, Wg=A, Wu=A, R=8, ldw=16, act=0, mg=None, mu=None,
             m=4, dX=A, lddx=16, dWg=A, dWu=A, lddw=16, ws=A, wsb=BIG):
    return l.nm_sparse_glu_backward(dH, lddh, X, T, K, ldx, G, U, ldgu, Wg, Wu, R, ldw, act, mg, mu, m, dX, lddx, dWg, dWu,
                                    lddw, ws, wsb, None)


@pytest.mark.parametrize("kw,expect", [
    (dict(dH=None), 1), (dict(G=None), 1), (dict(U=None), 1), (dict(ws=None), 1), (dict(X=None), 1), (dict(Wg=None), 1),
    (dict(Wu=None), 1), (dict(dWg=None), 1), (dict(dWu=None), 1), (dict(dX=None, dWg=None, dWu=None), 1), (dict(mg=A), 1),
    (dict(mu=A), 1),
    (dict(T=0), 2), (dict(K=0), 2), (dict(R=0), 2), (dict(lddh=4), 2), (dict(ldgu=4), 2), (dict(ldx=8), 2), (dict(ldw=8), 2),
    (dict(lddx=8), 2), (dict(lddw=8), 2), (dict(T=1 << 31), 2),
    (dict(act=3), 4), (dict(mg=A, mu=A, m=17), 4), (dict(mg=A, mu=A, m=1), 4),
    (dict(dH=MIS), 3), (dict(X=MIS), 3), (dict(Wg=MIS), 3), (dict(dX=MIS), 3), (dict(dWu=MIS), 3), (dict(ws=MIS), 3),
    (dict(lddh=12), 3), (dict(ldgu=12), 3), (dict(ldx=20), 3), (dict(ldw=20), 3), (dict(lddx=20), 3), (dict(lddw=20), 3),
    (dict(mg=MIS, mu=A), 3),
    (dict(wsb=100), 5),
])
def test_glu_backward_refusals(kw, expect):
    assert backward(nm.load(), **kw) == expect


def lora(l, X=A, T=4, K=16, ldx=16, packed=A, R=8, m=4, a=A, lda=16, sda=128, b=A, ldb=8, sdb=64, scale=A, n=2, r=8,
         indptr=A, ids=A, q=1, Y=A, ldy=8, ws=A, wsb=BIG):
    return l.nm_sparse_gemm_lora(X, T, K, ldx, packed, R, m, a, lda, sda, b, ldb, sdb, scale, n, r, indptr, ids, q, Y, ldy,
                                 ws, wsb, None)


@pytest.mark.parametrize("kw,expect", [
    (dict(X=None), 1), (dict(packed=None), 1), (dict(a=None), 1), (dict(b=None), 1), (dict(scale=None), 1),
    (dict(indptr=None), 1), (dict(ids=None), 1), (dict(Y=None), 1), (dict(ws=None), 1),
    (dict(T=0), 2), (dict(K=0), 2), (dict(R=0), 2), (dict(ldx=8), 2), (dict(ldy=4), 2), (dict(lda=8), 2), (dict(ldb=0), 2),
    (dict(sda=64), 2), (dict(sdb=32), 2), (dict(n=0), 2), (dict(q=-1), 2), (dict(q=1 << 24), 2), (dict(T=1 << 31), 2),
    (dict(m=5), 4), (dict(r=4), 4), (dict(r=12), 4), (dict(r=264), 4), (dict(r=0), 4),
    (dict(X=MIS), 3), (dict(packed=MIS), 3), (dict(a=MIS), 3), (dict(b=MIS), 3), (dict(Y=MIS), 3), (dict(ws=MIS), 3),
    (dict(scale=MIS), 3), (dict(indptr=MIS), 3), (dict(ids=MIS), 3), (dict(ldx=20), 3), (dict(ldy=12), 3), (dict(lda=20, sda=160), 3),
    (dict(ldb=12, sdb=96), 3), (dict(sda=132), 3), (dict(sdb=68), 3),
    (dict(wsb=100), 5),
])
def test_lora_refusals(kw, expect):
    assert lora(nm.load(), **kw) == expect


@pytest.mark.parametrize("call,expect", [
    (lambda l: l.nm_sparse_densify(None, A, 4, 16, 2, 4, A, 16, None), 1),
    (lambda l: l.nm_sparse_densify(A, None, 4, 16, 2, 4, A, 16, None), 1),
    (lambda l: l.nm_sparse_densify(A, A, 4, 16, 2, 4, None, 16, None), 1),
    (lambda l: l.nm_sparse_densify(A, A, 0, 16, 2, 4, A, 16, None), 2),
    (lambda l: l.nm_sparse_densify(A, A, 4, 16, 2, 4, A, 8, None), 2),
    (lambda l: l.nm_sparse_densify(A, A, 4, 16, 4, 4, A, 16, None), 4),
    (lambda l: l.nm_sparse_densify(A, A, 4, 16, 2, 17, A, 16, None), 4),
    (lambda l: l.nm_sparse_densify(A, A, 4, 16, 0, 4, A, 16, None), 4),
    (lambda l: l.nm_sparse_densify(A, A, 4, 16, 2, 4, MIS, 16, None), 3),
    (lambda l: l.nm_sparse_densify(A, A, 4, 16, 2, 4, A, 20, None), 3),
    (lambda l: l.nm_sparse_densify(A + 1, A, 4, 16, 2, 4, A, 16, None), 3),
    (lambda l: l.nm_sparse_densify(A, MIS, 4, 16, 2, 4, A, 16, None), 3),
])
def test_densify_refusals(call, expect):
    assert call(nm.load()) == expect


def test_binding_refuses_host_tensors():
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32)
    packed = torch.zeros(nm.load().nm_sparse_prepare_bytes(8, 16, 4), dtype=torch.uint8)
    for call in (lambda: nm.sparse_glu(bf(4, 16), packed, packed, 8, 4),
                 lambda: nm.sparse_glu_backward(bf(4, 8), bf(4, 16), bf(4, 8), bf(4, 8), bf(8, 16), bf(8, 16)),
                 lambda: nm.sparse_densify(bf(8, 8), torch.zeros((8, 1), dtype=torch.int32), 8, 16, 2, 4),
                 lambda: nm.sparse_gemm_lora(bf(4, 16), packed, 8, 4, bf(2, 8, 16), bf(2, 8, 8), torch.ones(2), i32(0, 4), i32(1))):
        with pytest.raises(nm.NMError, match="CUDA tensor"):
            call()
