"""ffn_moe_route against the formula in 64 bits: indices equal, weights within
the fp32 roundings (a score at most 17 x 2^-24, the sum of the chosen the same
plus 5, a division and the scale: below 48 x 2^-24)."""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

W_TOL = 48 * 2.0 ** -24


@pytest.fixture(scope="module")
def env():
    import torch
    from transformer_ffn_rmsnorm_gb300 import ffn
    return torch, ffn


def reference(logits, k, bias=None, groups=1, topk_groups=1, scale=1.0, sigmoid=False, renorm=False):
    """float64 [rows, experts] logits -> (idx, weights), token by token."""
    rows, experts = logits.shape
    idx, w = np.full((rows, k), -1, np.int32), np.zeros((rows, k))
    for t in range(rows):
        l = np.minimum(np.where(np.isnan(logits[t]), -np.inf, logits[t]), np.finfo(np.float32).max.astype(np.float64))
        ok = l > -np.inf
        if not ok.any():
            continue
        with np.errstate(over="ignore"):
            s = 1 / (1 + np.exp(-l)) if sigmoid else np.exp(l - l.max()) / np.exp(l - l.max()).sum()
        full = s if bias is None else s + bias
        order = np.where(ok, l if bias is None else full, -np.inf)
        if groups > 1:
            per = experts // groups
            score = []
            for g in range(groups):
                v = sorted((full[e] for e in range(g * per, (g + 1) * per) if ok[e]), reverse=True)
                score.append(sum(v[:2]) if v else -np.inf)
            kept = [g for g in sorted(range(groups), key=lambda g: (-score[g], g))[:topk_groups] if score[g] > -np.inf]
            order = np.where(np.isin(np.arange(experts) // per, kept), order, -np.inf)
        best = [e for e in sorted(range(experts), key=lambda e: (-order[e], e))[:k] if order[e] > -np.inf]
        v = s[best]
        idx[t, :len(best)] = best
        w[t, :len(best)] = scale * (v / max(v.sum(), 2.0 ** -100) if renorm else v)
    return idx, w


def run(env, logits, k, bias=None, **kw):
    torch, ffn = env
    sigmoid, renorm = kw.pop("sigmoid", False), kw.pop("renorm", False)
    flags = (ffn.FFN_ROUTE_SIGMOID if sigmoid else 0) | (ffn.FFN_ROUTE_RENORM if renorm else 0)
    idx, w = ffn.ffn_moe_route(logits, k, bias=bias, flags=flags, **kw)
    ri, rw = reference(logits.double().cpu().numpy(), k, None if bias is None else bias.double().cpu().numpy(),
                       sigmoid=sigmoid, renorm=renorm, **kw)
    assert np.array_equal(idx.cpu().numpy(), ri)
    got = w.double().cpu().numpy()
    assert np.all(np.isfinite(got))
    assert np.all(np.abs(got - rw) <= W_TOL * np.abs(rw) + 1e-37)
    return idx, w


@pytest.mark.parametrize("experts,k", [(1, 1), (2, 2), (8, 2), (31, 31), (33, 5), (60, 4), (64, 6), (128, 8), (160, 6),
                                       (256, 8), (300, 32), (512, 10), (1000, 32), (1024, 8)])
@pytest.mark.parametrize("sigmoid,renorm,with_bias", [(False, False, False), (False, True, False), (False, True, True),
                                                      (True, True, True), (True, False, False)])
def test_plain(env, experts, k, sigmoid, renorm, with_bias):
    torch, _ = env
    gen = torch.Generator(device="cuda").manual_seed(experts * 37 + k)
    logits = 1.5 * torch.randn(67, experts, generator=gen, device="cuda")
    bias = 0.1 * torch.randn(experts, generator=gen, device="cuda") if with_bias else None
    run(env, logits, k, bias, sigmoid=sigmoid, renorm=renorm, scale=2.5)


@pytest.mark.parametrize("groups,per,topk_groups,k", [(8, 32, 4, 8), (4, 12, 1, 6), (8, 20, 3, 6), (32, 1, 5, 5),
                                                      (32, 32, 7, 32), (3, 5, 2, 4), (2, 512, 1, 8), (5, 2, 5, 10)])
@pytest.mark.parametrize("sigmoid,with_bias", [(True, True), (False, False), (False, True)])
def test_groups(env, groups, per, topk_groups, k, sigmoid, with_bias):
    torch, _ = env
    gen = torch.Generator(device="cuda").manual_seed(groups * per + k)
    logits = 1.2 * torch.randn(90, groups * per, generator=gen, device="cuda")
    logits[3] = -float("inf")
    logits[4, : per * (groups - 1)] = -float("inf")     # one group has eligible experts
    logits[5, ::2] = -float("inf")
    bias = 0.05 * torch.randn(groups * per, generator=gen, device="cuda") if with_bias else None
    run(env, logits, k, bias, groups=groups, topk_groups=topk_groups, sigmoid=sigmoid, renorm=True)


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("with_bias", [False, True])
def test_ties_go_to_the_lower_index(env, dtype, with_bias):
    """16-bit logits from few values: most of them are equal to others; equal
    biases keep the ties, and the groups' scores tie as well."""
    torch, _ = env
    gen = torch.Generator(device="cuda").manual_seed(2)
    logits = (torch.randint(-3, 4, (200, 128), generator=gen, device="cuda") * 0.5).to(getattr(torch, dtype))
    bias = torch.full((128,), 0.25, device="cuda") if with_bias else None
    run(env, logits, 8, bias, sigmoid=True)
    run(env, logits, 8, bias, renorm=True)
    run(env, logits, 8, bias, groups=8, topk_groups=3, sigmoid=True, renorm=True)


@pytest.mark.parametrize("sigmoid", [True, False])
def test_close_scores_are_decided_exactly(env, sigmoid):
    """Scores that differ by less than the fp32 arithmetic resolves: logits one
    to three units in the last place apart, an (almost) constant bias, and
    sigmoids that saturate at 1 in fp32 but not in fp64 (logits 17 to 30)."""
    torch, _ = env
    gen = torch.Generator(device="cuda").manual_seed(4)
    base = torch.full((300, 96), 0.7, device="cuda")
    ulp = 2.0 ** -24
    logits = base + ulp * torch.randint(0, 4, base.shape, generator=gen, device="cuda")
    bias = torch.full((96,), 0.125, device="cuda")
    run(env, logits, 8, bias, sigmoid=sigmoid)
    bias2 = bias + 2.0 ** -27 * torch.randint(0, 3, (96,), generator=gen, device="cuda")
    run(env, logits, 8, bias2, sigmoid=sigmoid, renorm=True)
    run(env, logits, 6, bias2, sigmoid=sigmoid, groups=8, topk_groups=2, renorm=True)
    wide = 17 + 13 * torch.rand(64, 96, generator=gen, device="cuda")
    run(env, wide, 8, bias, sigmoid=sigmoid)
    run(env, wide, 8, None, sigmoid=sigmoid, groups=4, topk_groups=2)


def test_masked_not_finite_and_extreme(env):
    torch, _ = env
    inf, nan = float("inf"), float("nan")
    logits = torch.randn(12, 40, device="cuda", generator=torch.Generator(device="cuda").manual_seed(6))
    logits[0] = -inf
    logits[1, 3:] = -inf                       # three eligible experts for k = 6
    logits[2, ::3] = nan
    logits[3, 7] = inf
    logits[4, [5, 9]] = inf
    logits[5] = nan
    logits[6] = 3.0e38
    logits[7] *= 1e30
    logits[8] = -200 - logits[8].abs()         # sigmoids vanish in fp32
    logits[9] = torch.finfo(torch.float32).min
    logits[10, :39] = torch.finfo(torch.float32).min
    bias = 0.1 * torch.randn(40, device="cuda", generator=torch.Generator(device="cuda").manual_seed(7))
    for kw in ({}, {"renorm": True}, {"sigmoid": True}, {"groups": 4, "topk_groups": 2, "renorm": True}):
        run(env, logits, 6, None, **kw)
        run(env, logits, 6, bias, **kw)
    # a large bias decides alone
    big = torch.zeros(40, device="cuda")
    big[[30, 4]] = 1e6
    idx, _ = run(env, logits[6:7], 2, big, sigmoid=True)
    assert idx.tolist() == [[4, 30]]


@pytest.mark.parametrize("rows", [0, 1, 3, 4, 5, 4097])
def test_rows_and_a_captured_call(env, rows):
    torch, ffn = env
    gen = torch.Generator(device="cuda").manual_seed(rows)
    logits = torch.randn(rows + 2, 64, generator=gen, device="cuda")
    idx, w = torch.full((rows + 2, 6), 77, dtype=torch.int32, device="cuda"), torch.full((rows + 2, 6), 7.0, device="cuda")
    ffn.ffn_moe_route(logits[:rows], 6, idx=idx[:rows], weights=w[:rows])
    assert bool((idx[rows:] == 77).all()) and bool((w[rows:] == 7).all())
    if rows == 0:
        return
    ri, _ = reference(logits[:rows].double().cpu().numpy(), 6)
    assert np.array_equal(idx[:rows].cpu().numpy(), ri)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ffn.ffn_moe_route(logits, 6, idx=idx, weights=w)
    logits.copy_(logits.flip(0).clone())
    graph.replay()
    ri, _ = reference(logits.double().cpu().numpy(), 6)
    assert np.array_equal(idx.cpu().numpy(), ri)
