"""Shared by the tests of the feed-forward operators: pruned layers made from the
oracle's masks, and bounds of fp32 sums."""
from __future__ import annotations

import numpy as np
import torch

import datagen
import oracle
from nm_testutil import to_dev

HALF_STEP = 2.0 ** -8  # of bf16: a rounding is off by at most eps / 2 of the value


def layer(nm, R, K, m, seed, n_outliers=0):
    """A pruned projection: dict with the masked weights (fp64 and bf16, on the
    device), the kept values, the mask and the packed operand."""
    W = datagen.make_weight(R, K, 0.02, seed=seed)
    mask, vals, _ = nm.score_prune_compress(None, to_dev(W, (K + 7) // 8 * 8), m - 2, m)
    dense = nm.sparse_densify(vals, mask, R, K, m - 2, m)
    packed = nm.sparse_prepare_from_mask(vals, mask, R, K, m)
    return dict(W=W, mask=mask, vals=vals, dense=dense, packed=packed, w64=dense.double())


def keep_bits(mask, K):
    """bool [R x K] of the mask words."""
    bits = (mask[:, :, None].to(torch.int64) >> torch.arange(32, device=mask.device)) & 1
    return bits.reshape(mask.shape[0], -1)[:, :K].bool()


def randn(rows, cols, std, seed, pad=None):
    """bf16 [rows x cols] on the device with rows on 16 bytes; the columns that
    only pad the rows hold NaN."""
    ld = (cols + 7) // 8 * 8 + (pad or 0)
    g = torch.Generator().manual_seed(seed)
    t = torch.full((rows, ld), float("nan"), dtype=torch.float32)
    t[:, :cols] = torch.randn((rows, cols), generator=g) * std
    return t.to(torch.bfloat16).cuda()[:, :cols]


def sum_bound(a64, b64):
    """Bound of |fp32 sum - exact| of a @ b.T: each of the K additions of exact
    bf16 products is off by at most 2^-23 of the sum of magnitudes (one step,
    for an adder that truncates), and so are the joins of partial sums."""
    return (a64.shape[1] + 32) * 2.0 ** -23 * (a64.abs() @ b64.abs().T)


def act64(g, act):
    if act == "silu":
        return g * torch.sigmoid(g)
    if act == "gelu":
        return 0.5 * g * (1 + torch.tanh(np.sqrt(2 / np.pi) * (g + 0.044715 * g ** 3)))
    return g.clamp(min=0) ** 2


def slope64(g, act):
    if act == "silu":
        s = torch.sigmoid(g)
        return s * (1 + g * (1 - s))
    if act == "gelu":
        c = np.sqrt(2 / np.pi)
        t = torch.tanh(c * (g + 0.044715 * g ** 3))
        return 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 3 * 0.044715 * g * g)
    return 2 * g.clamp(min=0)


def assert_within(got, want, bound, what):
    """|got - want| <= bound for every element; NaN and infinities in the same places."""
    got = got.double()
    assert torch.equal(got.isnan(), want.isnan()), f"{what}: NaN in other places"
    fine = want.isfinite()
    assert torch.equal(got[~fine & ~want.isnan()], want[~fine & ~want.isnan()]), f"{what}: infinities differ"
    over = (got - want).abs()[fine] - bound[fine]
    assert bool((over <= 0).all()), f"{what}: {int((over > 0).sum())} of {over.numel()} beyond the bound, by {float(over.max())}"


def norm_error(got, want):
    return float((got.double() - want).norm() / want.norm())
