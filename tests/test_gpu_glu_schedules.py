"""The backward pass of the gated feed-forward under forced schedules and over many
tiles: whole and split tiles of dX, few pairs that each compute many tiles (the
accumulators and the stages are used over and over), a last round of dX that leaves
pairs to the tiles of dW, more than one band of the tile order, and dX in a launch
of its own.  Bounds: test_gpu_glu.py's."""
import pytest
import torch

import test_gpu_glu
from ffn_testutil import randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nm():
    import semi_structured_sparse_diag_b200 as nm
    nm.load()
    yield nm
    nm.set_gemm_schedule(0, 0)


@pytest.fixture
def schedule(nm):
    yield lambda policy, clusters=0: nm.set_gemm_schedule(policy, clusters)
    nm.set_gemm_schedule(0, 0)


@pytest.mark.parametrize("T,R,K,m,masked,policy,clusters", [
    (300, 520, 1030, 8, True, 1, 1),      # 40 tiles, all by one pair
    (700, 260, 1540, 4, False, 1, 3),     # 21 tiles of dX over three pairs, 28 of dW
    (515, 1100, 800, 6, True, 1, 5),      # dX: 12 tiles over 5 pairs, three pairs start on dW
    (40, 3000, 300, 4, True, 2, 2),       # a cluster for each tile of dX, then 48 tiles of dW
    (200, 1030, 700, 10, False, 2, 3),
    (200, 1030, 700, 10, False, 2, 1),    # fewer clusters than tiles: whole after all
    (40, 4200, 2000, 4, False, 0, 0),     # two bands of dW, several tiles a pair
    (2560, 320, 2304, 4, False, 0, 0),    # 90 tiles of dX: a second round with idle pairs
    (4864, 64, 4096, 4, False, 0, 0),     # 304 tiles of dX: a launch of their own, two bands
    (4864, 64, 4096, 4, True, 1, 7),
])
def test_backward_schedules(nm, schedule, T, R, K, m, masked, policy, clusters):
    X, dH, G, U, gate, up = test_gpu_glu._backward_inputs(nm, T, R, K, m, seed=T + R)
    kw = dict(mask_gate=gate["mask"], mask_up=up["mask"], m=m) if masked else {}
    schedule(policy, clusters)
    grads = nm.sparse_glu_backward(dH, X, G, U, gate["dense"], up["dense"], **kw)
    again = nm.sparse_glu_backward(dH, X, G, U, gate["dense"], up["dense"], **kw)
    torch.cuda.synchronize()
    nm.check_device_error()
    test_gpu_glu._check_backward(X, dH, G, U, gate, up, "silu", masked, grads)
    assert all(torch.equal(a, b) for a, b in zip(grads, again))


def test_the_schedule_decides_whether_dx_is_split(nm, schedule):
    # dX = sum_r dG[r] over 2^24, 2998 times 2^-6, -2^24 (dG = 2 dH U at g = 1 with a
    # squared-relu gate, U = 1; Wg = 1, Wu = 0).  A k-step adds 16 products of 2^-6 at
    # most, 1/4, to a whole tile's sum of 2^24, whose fp32 step is 2: all are lost,
    # and -2^24 leaves no more than that step.  A split of the 94 blocks (47 of Wg,
    # then 47 of Wu) over eight pairs, the cheapest, gives the second and the third
    # pair 12 blocks of 64 products each, 12 in their sums, which 2^24 + 12 + 12
    # keeps (multiples of 2); the fourth's -2^24 comes with 0 to 12 more.
    T, R, K = 4, 3000, 64
    dH = torch.full((T, R), 2.0 ** -7, device="cuda").to(torch.bfloat16)
    dH[:, 0], dH[:, -1] = 2.0 ** 23, -2.0 ** 23
    one = torch.ones((T, R), dtype=torch.bfloat16, device="cuda")
    W = torch.ones((R, K), dtype=torch.bfloat16, device="cuda")
    call = lambda: nm.sparse_glu_backward(dH, randn(T, K, 1.0, seed=1), one, one, W, torch.zeros_like(W), act="relu2", need_dw=False)[0]
    schedule(1)
    whole = call()
    schedule(2)
    split = call()
    torch.cuda.synchronize()
    nm.check_device_error()
    assert float(whole.abs().max()) <= 2
    assert 24 <= float(split.min()) and float(split.max()) <= 36
