"""GPU parity of a sparse projection with low-rank adapters, against plain fp64
formulas of the same bf16 inputs.

Bound: scale V is rounded to bf16 before its product (2^-8 of it, and 2^-22 for
the fp32 scaling), every sum runs in fp32 (sum_bound of ffn_testutil; the V
sum's error goes through B), Y is rounded once:
  |d| <= 2^-8 |Y| + ((2^-8 + 2^-20) |s V| + s E_V) |B| + E_Y.
"""
import pytest
import torch

from ffn_testutil import HALF_STEP, assert_within, layer, randn, sum_bound

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


def _adapters(n, r, R, K, seed, pad=0):
    A = randn(n * r, K, K ** -0.5, seed=seed, pad=pad)
    A = A.as_strided((n, r, K), (r * A.stride(0), A.stride(0), 1))
    B = randn(n * R, r, 0.2, seed=seed + 1, pad=pad)
    B = B.as_strided((n, R, r), (R * B.stride(0), B.stride(0), 1))
    scale = (torch.rand(n, generator=torch.Generator().manual_seed(seed)) * 2 - 0.5).cuda()
    return A, B, scale


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _check(X, proj, A, B, scale, indptr, ids, Y):
    x = X.double()
    want = x @ proj["w64"].T
    err = sum_bound(x, proj["w64"])
    for i, a in enumerate(ids.tolist()):
        lo, hi = indptr[i].item(), indptr[i + 1].item()
        if a < 0 or lo == hi:
            continue
        xr, s = x[lo:hi], scale[a].double()
        v = s * (xr @ A[a].double().T)
        b = B[a].double()
        want[lo:hi] += v @ b.T
        err[lo:hi] += ((HALF_STEP + 2.0 ** -20) * v.abs() + s.abs() * sum_bound(xr, A[a].double())) @ b.abs().T \
            + (b.shape[1] + 32) * 2.0 ** -23 * (v.abs() @ b.abs().T) \
            + (x.shape[1] + 32) * 2.0 ** -23 * (v.abs() @ b.abs().T)
    assert_within(Y, want, HALF_STEP * want.abs() + err * (1 + HALF_STEP) + 1e-30, "Y")


# (T, R, K, m, r, adapters, indptr, ids)
CASES = {
    "one token": (1, 300, 512, 4, 16, 3, [0, 1], [2]),
    "one of everything": (1, 1, 1, 4, 8, 1, [0, 1], [0]),
    "a token each, shared adapters": (40, 520, 1003, 6, 8, 5, list(range(41)), [(7 * i) % 6 - 1 for i in range(40)]),
    "a token each, its own adapter": (70, 260, 256, 4, 24, 70, list(range(71)), list(range(70))),
    "empty requests, gaps at both ends": (100, 515, 640, 8, 64, 4, [3, 3, 20, 20, 61, 90], [1, 3, 0, 3, 1]),
    "no adapter anywhere": (30, 256, 256, 4, 16, 2, [0, 10, 30], [-1, -1]),
    "rank 128, several tiles": (700, 1000, 384, 4, 128, 3, [0, 1, 239, 241, 500, 700], [0, 2, 0, 1, 2]),
    "rank 256": (50, 256, 90, 10, 256, 2, [0, 25, 50], [1, 0]),
    "rank 72, 8:10": (260, 600, 1030, 10, 72, 4, [0, 240, 260], [3, 2]),
    "one request over many tiles": (1100, 300, 200, 4, 32, 2, [0, 1100], [1]),
    "short requests of two adapters, rank 128": (230, 300, 333, 4, 128, 2, [min(230, 11 * i) for i in range(21)] + [230],
                                                 [i % 2 for i in range(21)]),
    "short requests, rank 40, several tiles": (900, 520, 1000, 8, 40, 7, list(range(0, 901, 10)), [(5 * i) % 8 - 1 for i in range(90)]),
    "prompts, rank 128, 8:10": (1500, 264, 515, 10, 128, 3, [7, 400, 400, 900, 1301, 1490], [2, 0, -1, 1, 2]),
    "prompts, rank 8": (2000, 300, 40, 4, 8, 2, [0, 1000, 1010, 2000], [1, 0, 1]),
    "prompts, rank 72, 6:8": (1030, 520, 1030, 8, 72, 5, [0, 100, 330, 331, 1030], [4, 2, 0, 4]),
    "streamed outputs": (3100, 11001, 64, 4, 16, 3, [0, 1200, 3099], [2, 0]),
    "long prompts, rank 128, 8:10": (1500, 264, 1003, 10, 128, 3, [7, 400, 400, 900, 1301, 1490], [2, 0, -1, 1, 2]),
    "long prompts, rank 8": (2000, 300, 1100, 4, 8, 2, [0, 1000, 1010, 2000], [1, 0, 1]),
    "streamed outputs of prompts": (3100, 11001, 904, 4, 16, 3, [0, 1200, 3099], [2, 0]),
    "prompts of five tokens and of a thousand": (1200, 260, 960, 4, 72, 9, [0, *range(100, 201, 5), 1200],
                                                 [i % 10 - 1 for i in range(22)]),
    "prompts of 24 tokens, rank 16": (1440, 300, 1003, 6, 16, 6, list(range(0, 1441, 24)), [(5 * i) % 7 - 1 for i in range(60)]),
    "many short requests over tiles": (600, 256, 128, 8, 8, 200, list(range(0, 601, 3)), [(3 * i) % 200 for i in range(200)]),
}


@pytest.mark.parametrize("name", CASES)
@pytest.mark.parametrize("policy", [0, 1, 2])
def test_lora_vs_fp64(nm, schedule, name, policy):
    T, R, K, m, r, n, indptr, ids = CASES[name]
    X = randn(T, K, 1.0, seed=T + K)
    proj = layer(nm, R, K, m, seed=R)
    A, B, scale = _adapters(n, r, R, K, seed=r, pad=8 if r == 24 else 0)
    schedule(policy)
    args = (X, proj["packed"], R, m, A, B, scale, _i32(indptr), _i32(ids))
    Y, again = nm.sparse_gemm_lora(*args), nm.sparse_gemm_lora(*args)
    _sync_ok(nm)
    _check(X, proj, A, B, scale, _i32(indptr), _i32(ids), Y)
    assert torch.equal(Y, again)


def test_lora_without_requests(nm):
    X = randn(33, 128, 1.0, seed=1)
    proj = layer(nm, 264, 128, 4, seed=2)
    A, B, scale = _adapters(2, 8, 264, 128, seed=3)
    Y = nm.sparse_gemm_lora(X, proj["packed"], 264, 4, A, B, scale, _i32([0]), _i32([]))
    _sync_ok(nm)
    _check(X, proj, A, B, scale, _i32([0]), _i32([]), Y)


def test_lora_replayed_with_other_requests(nm, schedule):
    # a captured decode step: other tokens, adapters and lengths at every replay
    T, R, K, m, r, n = 24, 512, 1024, 4, 16, 6
    X = randn(T, K, 1.0, seed=1)
    proj = layer(nm, R, K, m, seed=2)
    A, B, scale = _adapters(n, r, R, K, seed=3)
    indptr, ids = _i32(list(range(T + 1))), _i32([i % n for i in range(T)])
    ws = torch.empty(nm.load().nm_sparse_gemm_lora_workspace_bytes(T, K, m, r, n, T), dtype=torch.uint8, device="cuda")
    schedule(2)
    nm.sparse_gemm_lora(X, proj["packed"], R, m, A, B, scale, indptr, ids, ws=ws)
    torch.cuda.synchronize()
    nm.set_poison(False)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        Y = nm.sparse_gemm_lora(X, proj["packed"], R, m, A, B, scale, indptr, ids, ws=ws)
    for i in range(5):
        gen = torch.Generator().manual_seed(i)
        X.copy_(randn(T, K, 1.0, seed=50 + i))
        ids.copy_(torch.randint(-1, n, (T,), generator=gen, dtype=torch.int32))
        indptr.copy_(torch.randint(0, T + 1, (T + 1,), generator=gen, dtype=torch.int32).sort().values)
        Y.fill_(float("nan"))
        g.replay()
        _sync_ok(nm)
        _check(X, proj, A, B, scale, indptr, ids, Y)


def test_lora_reports_bad_requests(nm):
    # a list that is out of order, past the batch, or names no adapter: the error
    # word is set, nothing outside the arguments is touched, and the next call is right
    T, R, K, m, r, n = 64, 256, 256, 4, 8, 3
    X = randn(T, K, 1.0, seed=1)
    proj = layer(nm, R, K, m, seed=2)
    A, B, scale = _adapters(n, r, R, K, seed=3)
    for indptr, ids in (([0, 40, 20, 64], [0, 1, 2]), ([0, 20, 40, 65], [0, 1, 2]), ([-1, 20, 40, 64], [0, 1, 2]),
                        ([0, 20, 40, 64], [0, 3, 1]), ([0, 20, 40, 64], [0, -2, 1])):
        nm.sparse_gemm_lora(X, proj["packed"], R, m, A, B, scale, _i32(indptr), _i32(ids))
        with pytest.raises(nm.NMError, match="NM_ERR_DEVICE"):
            nm.check_device_error()
    good = _i32([0, 20, 40, 64]), _i32([0, 2, 1])
    Y = nm.sparse_gemm_lora(X, proj["packed"], R, m, A, B, scale, *good)
    _sync_ok(nm)
    _check(X, proj, A, B, scale, *good, Y)


def test_lora_other_stream(nm):
    T, R, K, m, r, n = 64, 300, 512, 8, 16, 4
    X = randn(T, K, 1.0, seed=1)
    proj = layer(nm, R, K, m, seed=2)
    A, B, scale = _adapters(n, r, R, K, seed=3)
    req = _i32([0, 10, 30, 64]), _i32([0, 3, 1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a = nm.sparse_gemm_lora(X, proj["packed"], R, m, A, B, scale, *req)
    b = nm.sparse_gemm_lora(X, proj["packed"], R, m, A, B, scale, *req, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    _sync_ok(nm)
    _check(X, proj, A, B, scale, *req, a)
    assert torch.equal(a, b)
