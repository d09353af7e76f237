"""Infinities and NaN in one adapter, token or scale stay with the tokens that they
belong to, although a tile multiplies every adapter among its tokens by all of them.
Bounds: test_gpu_lora.py's."""
import pytest
import torch

import test_gpu_lora
from ffn_testutil import layer, norm_error, randn

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


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


# (T, R, K, m, r, adapters, indptr, ids): tokens of their own adapter, shared ones,
# requests without one, tokens behind the last request; one tile and several, 256
# and 512 rows, both kernels of V
CASES = {
    "a token each, 2:4": (17, 300, 512, 4, 16, 5, list(range(18)), [(5 * i) % 6 - 1 for i in range(17)]),
    "a token each, 4:6": (40, 520, 1003, 6, 8, 5, list(range(41)), [(7 * i) % 6 - 1 for i in range(40)]),
    "a token each, 6:8": (33, 1000, 1030, 8, 24, 7, list(range(34)), [(5 * i) % 8 - 1 for i in range(33)]),
    "rank 72, 8:10": (260, 600, 1030, 10, 72, 4, [0, 100, 240, 255], [3, 1, 2]),
    "several tiles, 6:8": (700, 1000, 384, 8, 128, 3, [0, 1, 239, 241, 500, 690], [0, 2, -1, 1, 2]),
    "prompts, 2:4": (1500, 1100, 1003, 4, 40, 4, [7, 400, 400, 900, 1301, 1490], [2, 0, -1, 1, 3]),
    "prompts, 6:8": (1030, 520, 1030, 8, 72, 5, [0, 100, 330, 331, 1030], [4, 2, 0, 1]),
}


def _case(name):
    T, R, K, m, r, n, indptr, ids = CASES[name]
    return (T, R, K, m, r, n, randn(T, K, 1.0, seed=T + K), *test_gpu_lora._adapters(n, r, R, K, seed=r),
            test_gpu_lora._i32(indptr), test_gpu_lora._i32(ids))


def _copy(t):
    """The same values, rows as far apart."""
    return torch.empty(0, dtype=t.dtype, device=t.device).set_(t.untyped_storage().clone(), t.storage_offset(), t.shape, t.stride())


@pytest.mark.parametrize("name", CASES)
@pytest.mark.parametrize("policy", [0, 1, 2])
def test_b_of_one_adapter(nm, schedule, name, policy):
    T, R, K, m, r, n, X, A, B, scale, indptr, ids = _case(name)
    proj = layer(nm, R, K, m, seed=R)
    a = ids[ids >= 0].unique()
    B[a[0], 5, r - 1], B[a[0], 6] = INF, NAN
    B[a[-1], 5, 0], B[a[-1], R - 1, 2] = NAN, -INF   # two adapters at one feature
    B[a[1], 256:258, 1] = -INF                       # the tile's second 256 rows
    schedule(policy)
    Y = nm.sparse_gemm_lora(X, proj["packed"], R, m, A, B, scale, indptr, ids)
    again = nm.sparse_gemm_lora(X, proj["packed"], R, m, A, B, scale, indptr, ids)
    torch.cuda.synchronize()
    nm.check_device_error()
    test_gpu_lora._check(X, proj, A, B, scale, indptr, ids, Y)
    assert torch.equal(Y.view(torch.int16), again.view(torch.int16))


def test_b_all_nan_and_replayed(nm):
    # an adapter of NaN, then its finite self again, through one captured call
    T, R, K, m, r, n, X, A, B, scale, indptr, ids = _case("a token each, 6:8")
    proj = layer(nm, R, K, m, seed=R)
    good = B.clone()
    ws = torch.empty(nm.load().nm_sparse_gemm_lora_workspace_bytes(T, K, m, r, n, T), dtype=torch.uint8, device="cuda")
    nm.sparse_gemm_lora(X, proj["packed"], R, m, A, B, scale, indptr, ids, ws=ws)
    torch.cuda.synchronize()
    nm.set_poison(False)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        Y = nm.sparse_gemm_lora(X, proj["packed"], R, m, A, B, scale, indptr, ids, ws=ws)
    for bad in (3, None, 0):
        B.copy_(good)
        if bad is not None:
            B[bad] = NAN
        Y.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        nm.check_device_error()
        test_gpu_lora._check(X, proj, A, B, scale, indptr, ids, Y)


@pytest.mark.parametrize("name", CASES)
def test_x_a_and_scale(nm, name):
    # a token, an adapter's A and a scale: bit for bit the same for every other token
    T, R, K, m, r, n, X, A, B, scale, indptr, ids = _case(name)
    proj = layer(nm, R, K, m, seed=R)
    clean = nm.sparse_gemm_lora(X, proj["packed"], R, m, A, B, scale, indptr, ids)
    adapter = torch.full((T,), -1, device="cuda")
    for i, a in enumerate(ids.tolist()):
        adapter[int(indptr[i]):int(indptr[i + 1])] = a
    used = adapter[adapter >= 0].unique()
    for what in ("x", "a", "scale"):
        x, a, s = _copy(X), _copy(A), scale.clone()
        for value in (INF, NAN):
            if what == "x":
                hit = torch.arange(T, device="cuda") == int(indptr[1])
                x[hit, 3] = value
            else:
                hit = adapter == used[0]
                if what == "a":
                    a[used[0], r - 1, K - 1] = value
                else:
                    s[used[0]] = value
            Y = nm.sparse_gemm_lora(x, proj["packed"], R, m, a, B, s, indptr, ids)
            torch.cuda.synchronize()
            nm.check_device_error()
            assert torch.equal(Y[~hit], clean[~hit]), f"{what} {value}"
            assert not bool(Y[hit].isfinite().all()), f"{what} {value}"


@pytest.mark.parametrize("name", CASES)
def test_norm(nm, name):
    # roundings are independent, so in the 2-norm (rms of one to bf16: 2^-8 / sqrt 3)
    # that of Y and that of V, whose share of Y is the smaller one, stay below 2^-8;
    # partial sums kept in fewer bits than fp32 would not
    T, R, K, m, r, n, X, A, B, scale, indptr, ids = _case(name)
    proj = layer(nm, R, K, m, seed=R)
    Y = nm.sparse_gemm_lora(X, proj["packed"], R, m, A, B, scale, indptr, ids)
    torch.cuda.synchronize()
    want = X.double() @ proj["w64"].T
    for i, a in enumerate(ids.tolist()):
        lo, hi = int(indptr[i]), int(indptr[i + 1])
        if a >= 0 and lo < hi:
            want[lo:hi] += scale[a].double() * (X[lo:hi].double() @ A[a].double().T) @ B[a].double().T
    assert norm_error(Y, want) < 2.0 ** -8
