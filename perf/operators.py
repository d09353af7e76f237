"""Cases, plain forms and calls of the pruned layer's feed-forward and adapter operators.

Three operators of a transformer whose projections are (m-2):m sparse:

``glu``           the gated feed-forward's first half, H = act(X Wg^T) * (X Wu^T), with both
                  projections sparse; a training step also keeps G = X Wg^T and U = X Wu^T
``glu_backward``  its gradients from dH and the kept G and U: dX, dWg, dWu (straight through to
                  every weight, or kept to the mask)
``lora``          a shared sparse projection with the low-rank adapters of many requests at once,
                  Y[t] = X[t] W^T + scale[a] (X[t] A[a]^T) B[a]^T with a = the adapter of t's request
"""
import math

import torch

own = False

LARGEST = 8192 * 11008 * 4096  # tokens x out x in features of the largest listed call


def listed():
    return [
        # one sequence being decoded: a single token through the 7B-shaped gate and up projections
        dict(name="glu decode 1", op="glu", T=1, R=11008, K=4096, m=4, act="silu", save=False),
        # sixteen sequences decoded together, 6:8 weights
        dict(name="glu decode 16 6of8", op="glu", T=16, R=11008, K=4096, m=8, act="silu", save=False),
        # a short prompt through a narrow layer of odd sizes, 4:6 weights and a gelu gate
        dict(name="glu ragged 333 4of6", op="glu", T=333, R=1390, K=1003, m=6, act="gelu", save=False),
        # the forward pass of a training step, with what the backward pass needs
        dict(name="glu train 8192", op="glu", T=8192, R=11008, K=4096, m=4, act="silu", save=True),
        # a few tokens of a small layer while its masked weights are tuned
        dict(name="glu backward 77 4of6", op="glu_backward", T=77, R=1390, K=1003, m=6, act="gelu", masked=True),
        # a layer of 6:8 weights tuned under a fixed mask, squared-relu gate
        dict(name="glu backward 2048 6of8", op="glu_backward", T=2048, R=4096, K=4096, m=8, act="relu2", masked=True),
        # the backward pass of a training step, straight through to the latent weights
        dict(name="glu backward 8192", op="glu_backward", T=8192, R=11008, K=4096, m=4, act="silu", masked=False),
        # one request with its adapter: a single token through the down projection
        dict(name="lora decode 1", op="lora", T=1, R=4096, K=11008, m=4, r=16, adapters=8, requests=1),
        # 64 requests decoded together that share eight adapters
        dict(name="lora decode 64 shared", op="lora", T=64, R=4096, K=4096, m=4, r=32, adapters=8, requests=64),
        # 128 requests decoded together, about as many adapters as requests
        dict(name="lora decode 128 own", op="lora", T=128, R=11008, K=4096, m=4, r=16, adapters=128, requests=128),
        # a mixed batch of odd sizes: requests of every length, 6:8 weights, the smallest rank
        dict(name="lora ragged 777 6of8", op="lora", T=777, R=1390, K=2010, m=8, r=8, adapters=5, requests=9),
        # prompts of 24 requests in one ragged batch
        dict(name="lora prompts 8192", op="lora", T=8192, R=11008, K=4096, m=4, r=64, adapters=16, requests=24),
    ]


def draw(rng):
    def size(lo, hi):
        return min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))

    while True:
        op = rng.choice(("glu", "glu_backward", "lora"))
        c = dict(op=op, T=size(1, 8192), R=size(256, 11008), K=size(256, 11008), m=rng.choice((4, 4, 6, 8, 10)))
        if rng.random() < 0.5:  # feature sizes are often round
            c["R"], c["K"] = c["R"] // 64 * 64, c["K"] // 64 * 64
        if c["T"] * c["R"] * c["K"] > LARGEST // 2:
            continue
        if op == "lora":
            c |= dict(r=rng.choice((8, 16, 24, 32, 64, 128)), adapters=size(1, 128))
            c["requests"] = min(c["T"], size(1, 128))
        else:
            c["act"] = rng.choice(("silu", "gelu", "relu2"))
            c["save" if op == "glu" else "masked"] = rng.random() < 0.5
        return c


def _matrix(g, rows, cols, std):
    """bf16 [rows x cols] with its rows on 16 bytes, as the framework takes it."""
    ld = (cols + 7) // 8 * 8
    t = torch.empty((rows, ld), dtype=torch.float32, device="cuda").normal_(0, std, generator=g)
    return t.to(torch.bfloat16)[:, :cols]


def _layer(g, R, K, m):
    """A pruned projection: the masked weights, the kept values and the mask words of the m-2
    largest magnitudes in each group of m, ties to the lower column."""
    groups = (K + m - 1) // m
    w = torch.zeros((R, groups * m), dtype=torch.bfloat16, device="cuda")
    w[:, :K] = _matrix(g, R, K, 0.02)
    s = w.abs().view(R, groups, m)
    lower = torch.ones((m, m), dtype=torch.bool, device="cuda").tril(-1)
    ahead = (s[..., None, :] > s[..., :, None]) | ((s[..., None, :] == s[..., :, None]) & lower)
    keep = (ahead.sum(-1, dtype=torch.int8) < m - 2).view(R, groups * m)
    del s, ahead
    words = (groups * m + 31) // 32
    bits = torch.nn.functional.pad(keep, (0, words * 32 - groups * m)).view(R, words, 32).to(torch.int32)
    mask = (bits << torch.arange(32, dtype=torch.int32, device="cuda")).sum(-1, dtype=torch.int32)
    vals = w[keep].view(R, groups * (m - 2))
    dense = torch.zeros((R, (K + 7) // 8 * 8), dtype=torch.bfloat16, device="cuda")
    dense[:, :K] = (w * keep)[:, :K]
    return dict(w=dense[:, :K], keep=keep[:, :K].contiguous(), mask=mask, vals=vals)


def _pack(layer, R, K, m):
    import semi_structured_sparse_diag_b200 as nm

    return nm.sparse_prepare_from_mask(layer["vals"], layer["mask"], R, K, m)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    T, R, K, m = case["T"], case["R"], case["K"], case["m"]
    s = dict(case, x=_matrix(g, T, K, 1.0))
    if case["op"] == "lora":
        n, r = case["adapters"], case["r"]
        s["layer"] = _layer(g, R, K, m)
        s["a"] = torch.empty((n, r, (K + 7) // 8 * 8), dtype=torch.float32, device="cuda").normal_(
            0, K ** -0.5, generator=g).to(torch.bfloat16)[:, :, :K]
        s["b"] = torch.empty((n, R, r), dtype=torch.float32, device="cuda").normal_(0, 0.05, generator=g).to(torch.bfloat16)
        s["scale"] = torch.empty(n, dtype=torch.float32, device="cuda").uniform_(0.5, 2.0, generator=g)
        if case["requests"] == T:  # decoding: one token each
            cuts = torch.arange(T + 1, device="cuda")
        else:  # prompts of every length, none too, and a few rows behind the last one
            end = T - T // 64
            cuts = torch.randint(0, end + 1, (case["requests"] + 1,), device="cuda", generator=g).sort().values
            cuts[0], cuts[-1] = 0, end
        s["indptr"] = cuts.to(torch.int32)
        ids = torch.randint(0, n, (case["requests"],), device="cuda", generator=g)
        bare = torch.rand((case["requests"],), device="cuda", generator=g) < 0.1  # requests without an adapter
        if case["requests"] > 1:
            ids = torch.where(bare, -1, ids)
        s["ids"] = ids.to(torch.int32)
        if own:
            s["packed"] = _pack(s["layer"], R, K, m)
        return s
    s["gate"], s["up"] = _layer(g, R, K, m), _layer(g, R, K, m)
    if case["op"] == "glu":
        if own:
            s["packed_gate"], s["packed_up"] = _pack(s["gate"], R, K, m), _pack(s["up"], R, K, m)
        return s
    s["dh"] = _matrix(g, T, R, 0.1)
    s["g"], s["u"] = _matrix(g, T, R, 1.2), _matrix(g, T, R, 1.2)
    return s


def _act(g, act):
    if act == "silu":
        return g / (1 + torch.exp(-g))
    if act == "gelu":  # the tanh form
        return 0.5 * g * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g * g * g)))
    return g.clamp(min=0) ** 2


def _act_slope(g, act):
    if act == "silu":
        p = 1 / (1 + torch.exp(-g))
        return p * (1 + g * (1 - p))
    if act == "gelu":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (g + 0.044715 * g * g * g))
        return 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 3 * 0.044715 * g * g)
    return 2 * g.clamp(min=0)


def run(s):
    T, R, K, m = s["T"], s["R"], s["K"], s["m"]
    if own:
        import semi_structured_sparse_diag_b200 as nm

        if s["op"] == "glu":
            return nm.sparse_glu(s["x"], s["packed_gate"], s["packed_up"], R, m, act=s["act"], save=s["save"])
        if s["op"] == "glu_backward":
            masks = dict(mask_gate=s["gate"]["mask"], mask_up=s["up"]["mask"], m=m) if s["masked"] else {}
            return nm.sparse_glu_backward(s["dh"], s["x"], s["g"], s["u"], s["gate"]["w"], s["up"]["w"], act=s["act"], **masks)
        return nm.sparse_gemm_lora(s["x"], s["packed"], R, m, s["a"], s["b"], s["scale"], s["indptr"], s["ids"])
    x, half = s["x"].float(), torch.bfloat16
    if s["op"] == "glu":
        g, u = x @ s["gate"]["w"].float().T, x @ s["up"]["w"].float().T
        h = (_act(g, s["act"]) * u).to(half)
        return (h, g.to(half), u.to(half)) if s["save"] else h
    if s["op"] == "glu_backward":
        dh, g, u = s["dh"].float(), s["g"].float(), s["u"].float()
        dg, du = dh * u * _act_slope(g, s["act"]), dh * _act(g, s["act"])
        dx = dg @ s["gate"]["w"].float() + du @ s["up"]["w"].float()
        dwg, dwu = dg.T @ x, du.T @ x
        if s["masked"]:
            dwg, dwu = dwg * s["gate"]["keep"], dwu * s["up"]["keep"]
        return dx.to(half), dwg.to(half), dwu.to(half)
    # every token times every adapter, and the products of the others' adapters set to zero
    n, r = s["adapters"], s["r"]
    at = torch.searchsorted(s["indptr"][1:].contiguous(), torch.arange(T, dtype=torch.int32, device="cuda"), right=True)
    ids = torch.cat((s["ids"], s["ids"].new_full((1,), -1)))[at]
    v = (x @ s["a"].float().reshape(n * r, K).T).view(T, n, r) * s["scale"][:, None]
    v = torch.where((ids[:, None] == torch.arange(n, device="cuda"))[..., None], v, 0.0).reshape(T, n * r)
    y = x @ s["layer"]["w"].float().T + v @ s["b"].float().transpose(0, 1).reshape(R, n * r).T
    return y.to(half)


def exact(case, seed):
    s = prepare(case, seed)
    x = s["x"].double()
    if case["op"] == "lora":
        y = torch.nn.functional.linear(x, s["layer"]["w"].double())
        cuts = s["indptr"].tolist()
        for i, a in enumerate(s["ids"].tolist()):
            if a >= 0 and cuts[i + 1] > cuts[i]:
                rows = slice(cuts[i], cuts[i + 1])
                y[rows] += s["scale"][a].double() * ((x[rows] @ s["a"][a].double().T) @ s["b"][a].double().T)
        return y
    wg, wu = s["gate"]["w"].double(), s["up"]["w"].double()
    if case["op"] == "glu":
        g, u = torch.nn.functional.linear(x, wg), torch.nn.functional.linear(x, wu)
        h = _exact_act(g, case["act"]) * u
        return (h, g, u) if case["save"] else h
    g, u = s["g"].double().requires_grad_(), s["u"].double().requires_grad_()
    (_exact_act(g, case["act"]) * u).backward(s["dh"].double())
    dwg, dwu = torch.einsum("tr,tk->rk", g.grad, x), torch.einsum("tr,tk->rk", u.grad, x)
    if case["masked"]:
        dwg, dwu = dwg.masked_fill(~s["gate"]["keep"], 0), dwu.masked_fill(~s["up"]["keep"], 0)
    return torch.addmm(u.grad @ wu, g.grad, wg), dwg, dwu


def _exact_act(g, act):
    if act == "silu":
        return torch.nn.functional.silu(g)
    if act == "gelu":
        return torch.nn.functional.gelu(g, approximate="tanh")
    return torch.nn.functional.relu(g).square()


def work(case):
    T, R, K, m = case["T"], case["R"], case["K"], case["m"]
    groups = (K + m - 1) // m
    kept = R * groups * (m - 2)  # weights that take part
    layer = kept * 2 + R * groups * (m // 2 - 1) / 2  # their values and window index pairs
    if case["op"] == "glu":
        return {"bytes": 2 * T * K + 2 * layer + 2 * T * R * (3 if case["save"] else 1), "flops": 4 * T * kept}
    if case["op"] == "glu_backward":
        grad = kept if case["masked"] else R * K
        return {"bytes": 2 * (3 * T * R + T * K + 2 * R * K) + 2 * (T * K + 2 * R * K), "flops": 4 * T * (kept + grad)}
    r, n = case["r"], min(case["adapters"], case["requests"])
    return {"bytes": 2 * T * K + layer + 2 * T * R + 2 * n * r * (K + R), "flops": 2 * T * kept + 2 * T * r * (K + R)}
