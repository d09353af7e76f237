"""GPU parity of the gated feed-forward's first half with sparse projections and
of its backward pass, against plain fp64 formulas of the same bf16 inputs.

Bounds.  fp32 sums: ffn_testutil.sum_bound (call it E).  H = act(g) u is
rounded once: |dH| <= 2^-8 |H| + (slope) E_g |u| + |act(g)| E_u, with the slope
bounded by 1.13 (silu 1.1, gelu 1.13; squared relu 2 (|g| + E_g)) and 2^-18 of
|act(g) u| + |u| for the fp32 activation (e^x good to 2^-21 (1 + |x|), |x| < 8
wherever the result is not negligible).  Backward: dG and dU are rounded to
bf16 (2^-8 each) before products that sum in fp32, and the result is rounded
once: |d| <= 2^-8 |dX| + (2^-8 + 2^-16) (|dG| |Wg| + |dU| |Wu|) + E.  In the
2-norm the independent roundings (rms <= 2^-8 / sqrt 3) give at most
sqrt(2/3) 2^-8 < 2^-8.
"""
import pytest
import torch

from ffn_testutil import (HALF_STEP, act64, assert_within, keep_bits, layer, norm_error, randn, slope64,
                          sum_bound)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nm():
    import semi_structured_sparse_diag_b200 as nm
    nm.load()
    yield nm
    nm.set_gemm_schedule(0, 0)


@pytest.fixture
def schedule(nm):
    yield lambda policy, pairs=0: nm.set_gemm_schedule(policy, pairs)
    nm.set_gemm_schedule(0, 0)


def _sync_ok(nm):
    torch.cuda.synchronize()
    nm.check_device_error()


def _check_glu(X, gate, up, act, out):
    x = X.double()
    g, u = x @ gate["w64"].T, x @ up["w64"].T
    Eg, Eu = sum_bound(x, gate["w64"]), sum_bound(x, up["w64"])
    H, G, U = out if isinstance(out, tuple) else (out, None, None)
    a = act64(g, act)
    slope = 2 * (g.abs() + Eg) if act == "relu2" else 1.13
    bound = (slope * Eg * (u.abs() + Eu) + a.abs() * Eu) * (1 + HALF_STEP) + HALF_STEP * (a * u).abs() \
        + 2.0 ** -18 * ((a * u).abs() + u.abs()) + 1e-30
    assert_within(H, a * u, bound, "H")
    if G is not None:
        assert_within(G, g, HALF_STEP * g.abs() + 2 * Eg + 1e-30, "G")
        assert_within(U, u, HALF_STEP * u.abs() + 2 * Eu + 1e-30, "U")


# one token; odd and ragged T, R, K; every pattern; several tiles in both
# directions; tokens in the second half of a tile only just there
GLU_CASES = [
    (1, 1, 1, 4, "silu", False), (1, 300, 512, 4, "silu", True), (17, 131, 1003, 6, "gelu", False),
    (33, 520, 2056, 8, "relu2", True), (129, 256, 640, 10, "silu", False), (240, 260, 256, 4, "gelu", True),
    (241, 1000, 384, 4, "silu", True), (777, 700, 1030, 8, "silu", False), (16, 4096, 4096, 4, "silu", False),
    (1100, 515, 90, 10, "relu2", True),
    (2100, 11001, 64, 4, "silu", True),  # outputs too large for L2: streamed
]


@pytest.mark.parametrize("T,R,K,m,act,save", GLU_CASES)
def test_glu_vs_fp64(nm, T, R, K, m, act, save):
    X = randn(T, K, 1.0, seed=T + K)
    gate, up = layer(nm, R, K, m, seed=R), layer(nm, R, K, m, seed=R + 1)
    out = nm.sparse_glu(X, gate["packed"], up["packed"], R, m, act=act, save=save)
    _sync_ok(nm)
    _check_glu(X, gate, up, act, out)


# split tiles: whole tiles, stream-K over every pair and over a few
@pytest.mark.parametrize("T,R,K,m,pairs", [(1, 300, 4096, 4, 0), (16, 1000, 1024, 8, 0), (130, 256, 2048, 4, 0),
                                           (240, 515, 768, 6, 3), (500, 700, 512, 4, 5)])
def test_glu_stream_k(nm, schedule, T, R, K, m, pairs):
    X = randn(T, K, 1.0, seed=T)
    gate, up = layer(nm, R, K, m, seed=R), layer(nm, R, K, m, seed=R + 1)
    ws = torch.empty(nm.load().nm_sparse_glu_workspace_bytes(T, K, m), dtype=torch.uint8, device="cuda")
    schedule(2, pairs)
    outs = [nm.sparse_glu(X, gate["packed"], up["packed"], R, m, save=True, ws=ws) for _ in range(3)]
    schedule(1)
    whole = nm.sparse_glu(X, gate["packed"], up["packed"], R, m, save=True, ws=ws)
    _sync_ok(nm)
    for o in outs:
        _check_glu(X, gate, up, "silu", o)
        assert all(torch.equal(a, b) for a, b in zip(o, outs[0]))  # deterministic
    _check_glu(X, gate, up, "silu", whole)


def test_glu_strides_and_no_workspace(nm):
    # rows further apart than their width, outputs into a wider matrix, whose
    # other columns stay, and a 2:4 call without a workspace
    T, R, K, m = 70, 264, 320, 4
    X = randn(T, K, 1.0, seed=1, pad=24)
    gate, up = layer(nm, R, K, m, seed=2), layer(nm, R, K, m, seed=3)
    wide = torch.full((T, 400), 7.0, dtype=torch.bfloat16, device="cuda")
    lib = nm.load()
    st = lib.nm_sparse_glu(X.data_ptr(), T, K, X.stride(0), gate["packed"].data_ptr(), up["packed"].data_ptr(), R, m, 0,
                           wide.data_ptr(), 400, None, None, 0, None, 0, torch.cuda.current_stream().cuda_stream)
    assert st == 0
    _sync_ok(nm)
    _check_glu(X, gate, up, "silu", wide[:, :R])
    assert bool((wide[:, R:] == 7.0).all())


def test_glu_special_values(nm):
    # an infinity and a NaN in one token stay in that token
    T, R, K, m = 40, 256, 256, 4
    X = randn(T, K, 1.0, seed=5)
    X[3, 7], X[20, 0] = float("inf"), float("nan")
    gate, up = layer(nm, R, K, m, seed=6), layer(nm, R, K, m, seed=7)
    H = nm.sparse_glu(X, gate["packed"], up["packed"], R, m)
    _sync_ok(nm)
    rows = [t for t in range(T) if t not in (3, 20)]
    _check_glu(X[rows], gate, up, "silu", H[rows])
    # pruned weights take no part: only features with a kept gate or up weight at
    # the column see it
    for t, col in ((3, 7), (20, 0)):
        hit = (gate["w64"][:, col] != 0) | (up["w64"][:, col] != 0)
        assert torch.equal(~H[t].isfinite(), hit)
    assert bool((H[20].isfinite() | H[20].isnan()).all())


def test_glu_same_operand_twice_and_streams(nm):
    T, R, K, m = 64, 512, 512, 8
    X, X2 = randn(T, K, 1.0, seed=8), randn(T, K, 1.0, seed=9)
    one = layer(nm, R, K, m, seed=10)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a = nm.sparse_glu(X, one["packed"], one["packed"], R, m)          # two calls at once
    b = nm.sparse_glu(X2, one["packed"], one["packed"], R, m, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    _sync_ok(nm)
    _check_glu(X, one, one, "silu", a)
    _check_glu(X2, one, one, "silu", b)


@pytest.mark.parametrize("m", [4, 8])
def test_glu_replayed_graphs_share_a_workspace(nm, schedule, m):
    T, R, K = 16, 512, 2048
    X = randn(T, K, 1.0, seed=11)
    gate, up = layer(nm, R, K, m, seed=12), layer(nm, R, K, m, seed=13)
    ws = torch.empty(nm.load().nm_sparse_glu_workspace_bytes(T, K, m), dtype=torch.uint8, device="cuda")
    schedule(2)
    nm.sparse_glu(X, gate["packed"], up["packed"], R, m, ws=ws)
    torch.cuda.synchronize()
    graphs = []
    nm.set_poison(False)
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            H = nm.sparse_glu(X, gate["packed"], up["packed"], R, m, ws=ws)
        graphs.append((g, H))
    for i in range(6):
        X.copy_(randn(T, K, 1.0, seed=20 + i))
        g, H = graphs[i % 2]
        H.fill_(float("nan"))
        g.replay()
        _sync_ok(nm)
        _check_glu(X, gate, up, "silu", H)


def _backward_inputs(nm, T, R, K, m, seed):
    X, dH = randn(T, K, 1.0, seed=seed), randn(T, R, 0.1, seed=seed + 1)
    G, U = randn(T, R, 1.2, seed=seed + 2), randn(T, R, 1.2, seed=seed + 3)
    return X, dH, G, U, layer(nm, R, K, m, seed=seed + 4), layer(nm, R, K, m, seed=seed + 5)


def _check_backward(X, dH, G, U, gate, up, act, masked, grads):
    x, dh, g, u = X.double(), dH.double(), G.double(), U.double()
    dg, du = dh * u * slope64(g, act), dh * act64(g, act)
    op = HALF_STEP + 2.0 ** -16  # of |dG|, |dU|: the rounding to bf16, the fp32 formulas
    # and where the slope itself is a difference (near its zero) 2^-20 of |dH U|
    near = 2.0 ** -20 * dh.abs() * (u.abs() + 1)
    dX, dWg, dWu = grads
    if dX is not None:
        want = dg @ gate["w64"] + du @ up["w64"]
        mag = dg.abs() @ gate["w64"].abs() + du.abs() @ up["w64"].abs()
        E = (2 * g.shape[1] + 32) * 2.0 ** -23 * mag + near @ (gate["w64"].abs() + up["w64"].abs())
        assert_within(dX, want, (HALF_STEP * want.abs() + (op * mag + E) * (1 + HALF_STEP)) + 1e-30, "dX")
        if want.numel() >= 4096:
            assert norm_error(dX, want) < 2.0 ** -8
    for got, d, side, name in ((dWg, dg, gate, "dWg"), (dWu, du, up, "dWu")):
        if got is None:
            continue
        want, mag = d.T @ x, d.abs().T @ x.abs()
        E = (x.shape[0] + 32) * 2.0 ** -23 * mag + near.T @ x.abs()
        bound = HALF_STEP * want.abs() + (op * mag + E) * (1 + HALF_STEP) + 1e-30
        if masked:
            keep = keep_bits(side["mask"], x.shape[1])
            want, bound = want * keep, bound * keep
        assert_within(got, want, bound, name)
        if want.numel() >= 4096 and x.shape[0] >= 16:
            assert norm_error(got, want) < 2.0 ** -8


BACKWARD_CASES = [
    (1, 1, 1, 4, "silu", False), (1, 300, 512, 4, "gelu", True), (77, 131, 1003, 6, "gelu", True),
    (64, 256, 256, 4, "silu", False), (300, 520, 1030, 8, "relu2", True), (513, 260, 90, 10, "silu", True),
    (1000, 1000, 520, 4, "silu", False), (4096, 64, 64, 8, "gelu", False), (40, 3000, 300, 4, "silu", True),
]


@pytest.mark.parametrize("T,R,K,m,act,masked", BACKWARD_CASES)
def test_backward_vs_fp64(nm, T, R, K, m, act, masked):
    X, dH, G, U, gate, up = _backward_inputs(nm, T, R, K, m, seed=T + R)
    kw = dict(mask_gate=gate["mask"], mask_up=up["mask"], m=m) if masked else {}
    grads = nm.sparse_glu_backward(dH, X, G, U, gate["dense"], up["dense"], act=act, **kw)
    again = nm.sparse_glu_backward(dH, X, G, U, gate["dense"], up["dense"], act=act, **kw)
    _sync_ok(nm)
    _check_backward(X, dH, G, U, gate, up, act, masked, grads)
    assert all(torch.equal(a, b) for a, b in zip(grads, again))


def test_backward_parts(nm):
    X, dH, G, U, gate, up = _backward_inputs(nm, 100, 300, 200, 4, seed=3)
    full = nm.sparse_glu_backward(dH, X, G, U, gate["dense"], up["dense"])
    dX, none, _ = nm.sparse_glu_backward(dH, X, G, U, gate["dense"], up["dense"], need_dw=False)
    nodx, dWg, dWu = nm.sparse_glu_backward(dH, X, G, U, gate["dense"], up["dense"], need_dx=False)
    _sync_ok(nm)
    assert none is None and nodx is None
    assert torch.equal(dX, full[0]) and torch.equal(dWg, full[1]) and torch.equal(dWu, full[2])


# the derivative of sum(dH * H) along a direction: central differences of the
# fp64 formula (error ~ eps^2 = 1e-8 of the third derivative) against the
# gradients' inner product with it; along the gradient itself the inner product
# is its norm, so the relative error is at most the 2-norm's
@pytest.mark.parametrize("act", ["silu", "gelu", "relu2"])
def test_gradients_against_differences(nm, act):
    T, R, K, m = 96, 256, 192, 4
    X, dH = randn(T, K, 1.0, seed=1), randn(T, R, 0.1, seed=2)
    gate, up = layer(nm, R, K, m, seed=3), layer(nm, R, K, m, seed=4)
    _, G, U = nm.sparse_glu(X, gate["packed"], up["packed"], R, m, act=act, save=True)
    dX, dWg, dWu = nm.sparse_glu_backward(dH, X, G, U, gate["dense"], up["dense"], act=act)
    _sync_ok(nm)

    def loss(x, wg, wu):
        return (dH.double() * act64(x @ wg.T, act) * (x @ wu.T)).sum()

    at = [X.double(), gate["w64"], up["w64"]]
    for i, grad in enumerate((dX, dWg, dWu)):
        d = grad.double() / grad.double().norm()
        lo, hi = list(at), list(at)
        lo[i], hi[i] = at[i] - 1e-4 * d, at[i] + 1e-4 * d
        slope = float((loss(*hi) - loss(*lo)) / 2e-4)
        # G and U were rounded to bf16 too: two more roundings of the same size
        assert abs(float((grad.double() * d).sum()) - slope) <= 2.0 ** -7 * abs(slope)


def test_backward_captured(nm):
    X, dH, G, U, gate, up = _backward_inputs(nm, 200, 300, 264, 4, seed=30)
    ws = torch.empty(nm.load().nm_sparse_glu_backward_workspace_bytes(200, 300), dtype=torch.uint8, device="cuda")
    nm.sparse_glu_backward(dH, X, G, U, gate["dense"], up["dense"], ws=ws)
    torch.cuda.synchronize()
    nm.set_poison(False)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        grads = nm.sparse_glu_backward(dH, X, G, U, gate["dense"], up["dense"], ws=ws)
    for i in range(2):
        dH.copy_(randn(200, 300, 0.1, seed=40 + i))
        for t in grads:
            t.fill_(float("nan"))
        g.replay()
        _sync_ok(nm)
        _check_backward(X, dH, G, U, gate, up, "silu", False, grads)


@pytest.mark.parametrize("R,K,n,m", [(1, 1, 2, 4), (130, 1003, 4, 6), (64, 520, 6, 8), (33, 2010, 8, 10),
                                     (20, 77, 1, 3), (20, 200, 5, 16), (3, 40, 1, 2), (300, 4096, 2, 4)])
def test_densify(nm, R, K, n, m):
    W = randn(R, K, 0.02, seed=R + K)
    mask, vals, _ = nm.score_prune_compress(None, W, n, m)
    D = nm.sparse_densify(vals, mask, R, K, n, m)
    _sync_ok(nm)
    assert torch.equal(D, torch.where(keep_bits(mask, K), W, torch.zeros_like(W)))


def test_densify_reports_a_wrong_mask(nm):
    W = randn(8, 64, 0.02, seed=1)
    mask, vals, _ = nm.score_prune_compress(None, W, 2, 4)
    mask[3, 1] = -1
    nm.sparse_densify(vals, mask, 8, 64, 2, 4)
    with pytest.raises(nm.NMError, match="NM_ERR_DEVICE"):
        nm.check_device_error()


@pytest.mark.parametrize("act", ["silu", "gelu", "relu2"])
def test_backward_at_large_gates(nm, act):
    # gates where the sigmoid has reached 0 or 1 and g^2 leaves fp32: the slope is
    # the asymptote's (2 g for relu^2, whose gate stays below 1e18 here)
    T, R, K = 8, 64, 64
    big = 1e18 if act == "relu2" else 3e38
    G = torch.tensor([0.0, 1e4, -1e4, 1e9, -1e9, 1e12, big, -big]).to(torch.bfloat16).cuda()[:, None].expand(T, R).contiguous()
    U, dH = randn(T, R, 1.0, seed=1), randn(T, R, 1e-20, seed=2)
    W = torch.eye(R, K, dtype=torch.bfloat16, device="cuda")
    dX, _, _ = nm.sparse_glu_backward(dH, randn(T, K, 1.0, seed=3), G, U, W, torch.zeros_like(W), act=act)
    _sync_ok(nm)
    g = G.double()
    slope = 2 * g.clamp(min=0) if act == "relu2" else torch.where(g == 0, 0.5, (g > 0).double())
    want = dH.double() * U.double() * slope  # W is the identity: dX = dG
    assert_within(dX, want, (2 * HALF_STEP + 2.0 ** -15) * want.abs() + 1e-38, "dX")


def test_first_call_captured():
    # nothing has to run before a capture: in a process of its own
    import subprocess
    import sys
    code = """
import sys
sys.path[:0] = ["tests", "."]
import torch
import semi_structured_sparse_diag_b200 as nm
from ffn_testutil import layer, randn
X, dH = randn(40, 256, 1.0, 1), randn(40, 300, 1.0, 2)
side, A, B = layer(nm, 300, 256, 8, 3), randn(16, 256, 1.0, 4).view(2, 8, 256), randn(600, 8, 1.0, 5).view(2, 300, 8)
scale, indptr, ids = torch.ones(2, device="cuda"), torch.tensor([0, 20, 40], dtype=torch.int32, device="cuda"), torch.tensor([1, 0], dtype=torch.int32, device="cuda")
torch.cuda.synchronize()
def step():
    H, G, U = nm.sparse_glu(X, side["packed"], side["packed"], 300, 8, save=True)
    return (H, G, U, nm.sparse_gemm_lora(X, side["packed"], 300, 8, A, B, scale, indptr, ids),
            *nm.sparse_glu_backward(dH, X, G, U, side["dense"], side["dense"]))
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    outs = step()
g.replay()
torch.cuda.synchronize()
nm.check_device_error()
assert all(torch.equal(a, b) for a, b in zip(outs, step()))
print("same")
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=240)
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]


@pytest.mark.parametrize("T,m", [(65539, 6), (65536, 10), (262147, 6)])
def test_glu_of_many_tokens(nm, T, m):
    # past 65535 tokens, and past as many runs of the staging kernel's four
    R, K = 24, 22
    X = randn(T, K, 1.0, seed=T)
    gate, up = layer(nm, R, K, m, seed=1), layer(nm, R, K, m, seed=2)
    out = nm.sparse_glu(X, gate["packed"], up["packed"], R, m, act="silu")
    lifted = nm.lift_activations(X, m)
    _sync_ok(nm)
    _check_glu(X, gate, up, "silu", out)
    g = (K + m - 1) // m
    pairs = torch.nn.functional.pad(X, (0, g * m - K)).reshape(T, g, m // 2, 2)
    want = torch.stack((pairs[:, :, :-1], pairs[:, :, 1:]), 3).reshape(T, -1)
    assert torch.equal(lifted[:, :want.shape[1]], want)
