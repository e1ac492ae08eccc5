"""The operators around a routed (mixture-of-experts) feed-forward layer, as they are measured.

A pre-norm layer with routed experts, r = x + res, n = RMSNorm(r) * g, logits = n W_r^T, runs

  norm   ffn_add_rmsnorm / ffn_add_rmsnorm_e4m3   the residual's addition with the norm, n in 16 bits, or in
                                                  8 (e4m3) with a scale for each row or for each 128 columns
  route  ffn_moe_route                            scores, a bias for balance, groups, top-k, weights
  moe    ffn_moe_forward                          the chosen experts' SwiGLU blocks and their weighted sum
  q4     ffn_moe_forward_q4                       the same with 4-bit weights and a scale for each 32 of them

`run` computes each in its plain form (elementary torch operations in 32 bits, the router's scores in 64 where
the order of close values decides) or, with `own`, by the library's entry point.
"""

import math

import numpy as np
import torch

own = False

_TORCH = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-6
E4M3_MAX = 448.0
SMALLEST_AMAX = 2.0 ** -100     # of a row or group whose values are all (nearly) zero
SMALLEST_SUM = 2.0 ** -100      # of a token's chosen scores


def _route(name, rows, experts, k, groups, topk_groups, sigmoid, bias, renorm, scale, masked, dtype):
    return {"name": name, "op": "route", "rows": rows, "experts": experts, "k": k, "groups": groups,
            "topk_groups": topk_groups, "sigmoid": sigmoid, "bias": bias, "renorm": renorm, "scale": scale,
            "masked": masked, "dtype": dtype}


def _norm(name, rows, d, quant, group, dtype):
    return {"name": name, "op": "norm", "rows": rows, "d": d, "quant": quant, "group": group, "dtype": dtype}


def _moe(name, op, rows, d, ffn_, experts, k, residual, prepared, dtype):
    return {"name": name, "op": op, "rows": rows, "d": d, "ffn": ffn_, "experts": experts, "k": k,
            "residual": residual, "prepared": prepared, "dtype": dtype}


def listed():
    return [
        # one token of one sequence: launch latency and little else
        _route("route_1x64_k6", 1, 64, 6, 1, 1, False, False, False, 1.0, 0, "f32"),
        # a ragged prompt, experts in groups of which half are kept, a bias for balance; padding rows masked
        _route("route_4097x256_k8_g8", 4097, 256, 8, 8, 4, True, True, True, 2.5, 5, "f32"),
        # a large prefill batch, 16-bit logits (many equal ones)
        _route("route_16384x128_k8_bf16", 16384, 128, 8, 1, 1, False, False, True, 1.0, 0, "bf16"),
        # one token between two layers
        _norm("norm_1x4096_bf16", 1, 4096, False, 0, "bf16"),
        # a ragged prompt, 8-bit activations with a scale for each 128 columns
        _norm("norm_4099x5120_e4m3_g128_bf16", 4099, 5120, True, 128, "bf16"),
        # a large prefill batch, 8-bit activations with a scale for each token
        _norm("norm_16384x4096_e4m3_row_f16", 16384, 4096, True, 0, "f16"),
        # one token: six of 64 small experts are read, a stream of weights
        _moe("moe_1x2048x1408_64e6_bf16", "moe", 1, 2048, 1408, 64, 6, True, False, "bf16"),
        # a prompt over 64 small experts, weights prepared once as fp16; unequal loads, ragged tiles
        _moe("moe_4096x2048x1408_64e6_prep", "moe", 4096, 2048, 1408, 64, 6, True, True, "bf16"),
        # an odd-length prompt over 8 large experts: matrix products above all
        _moe("moe_2731x4096x14336_8e2_f16", "moe", 2731, 4096, 14336, 8, 2, False, False, "f16"),
        # one token, 4-bit experts
        _moe("q4_1x5120x2176_32e4", "q4", 1, 5120, 2176, 32, 4, True, False, "bf16"),
        # a decode batch of 16 sequences over 8 large 4-bit experts: every expert is read
        _moe("q4_16x4096x14336_8e2", "q4", 16, 4096, 14336, 8, 2, False, False, "bf16"),
        # a short prompt over 64 small 4-bit experts
        _moe("q4_777x2048x1408_64e6", "q4", 777, 2048, 1408, 64, 6, True, False, "bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "norm", "moe", "q4"])
    if op == "route":
        groups = rng.choice([1, 1, 4, 8])
        experts = groups * rng.choice([8, 12, 20, 32]) if groups > 1 else rng.choice([8, 40, 60, 64, 128, 160, 256])
        topk_groups = rng.randint(1, groups)
        k = rng.randint(1, min(8, topk_groups * (experts // groups)))
        return {"op": op, "rows": _log(rng, 1, 16384), "experts": experts, "k": k, "groups": groups,
                "topk_groups": topk_groups, "sigmoid": rng.random() < 0.5, "bias": rng.random() < 0.5,
                "renorm": rng.random() < 0.6, "scale": rng.choice([1.0, 2.5]), "masked": rng.choice([0, 0, 1]),
                "dtype": rng.choice(["f32", "f32", "bf16", "f16"])}
    if op == "norm":
        rows = _log(rng, 1, 16384)
        d = 8 * _log(rng, 32, 1024)
        quant = rng.random() < 0.6
        return {"op": op, "rows": min(rows, 67108864 // d), "d": d, "quant": quant,
                "group": rng.choice([0, 32, 64, 128]) if quant else 0, "dtype": rng.choice(["bf16", "bf16", "f16", "f32"])}
    step = 32 if op == "q4" else 8
    while True:
        d, ffn_ = step * _log(rng, 512 // step, 5120 // step), step * _log(rng, 512 // step, 14336 // step)
        experts = rng.choice([8, 16, 24, 32, 64, 96])
        if experts * 3 * d * ffn_ <= 1.4e9:
            break
    k = rng.choice([1, 2, 4, 6, 8])
    rows = _log(rng, 1, 4096)
    while 6.0 * rows * k * d * ffn_ > 1.9e12:
        rows = rows // 2 + 1
    prepared = op == "moe" and rng.random() < 0.4
    return {"op": op, "rows": rows, "d": d, "ffn": ffn_, "experts": experts, "k": k, "residual": rng.random() < 0.5,
            "prepared": prepared, "dtype": "bf16" if op == "q4" else rng.choice(["bf16", "f16"])}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(1000003 * int(seed) + 17)
    return g


def _activations(gen, rows, d, scale=1.0):
    """Hidden states: unit rows with a few columns that stand out, as a trained model's have."""
    col = 1.0 + 7.0 * (torch.rand(d, generator=gen, device="cuda") < 0.01).float()
    return torch.randn(rows, d, generator=gen, device="cuda") * col * scale


def _router_logits(gen, rows, experts):
    """Scores of unequally liked experts."""
    liked = 0.5 * torch.randn(experts, generator=gen, device="cuda")
    return 1.2 * torch.randn(rows, experts, generator=gen, device="cuda") + liked


def _q4_layout(q, s):
    """[out, in] codes (-8..7) and [out, in/32] scales in the device layout: byte 16 t + 4 b + e of a 64-byte group is
    canonical byte 4 t + e of the group's block b; the last group of a row is filled up with zeros."""
    out, inn = q.shape
    blocks, ngrp = inn // 32, -(-inn // 128)
    u = (q + 8).to(torch.uint8).view(out, blocks, 32)
    byte = u[:, :, :16] | (u[:, :, 16:] << 4)
    full = torch.zeros(out, 4 * ngrp, 16, dtype=torch.uint8, device=q.device)
    full[:, :blocks] = byte
    qs = full.view(out, ngrp, 4, 4, 4).permute(0, 1, 3, 2, 4).reshape(out, 64 * ngrp)
    sc = torch.zeros(out, 4 * ngrp, dtype=torch.float16, device=q.device)
    sc[:, :blocks] = s
    return qs.contiguous(), sc.contiguous()


def _q4_weight(gen, experts, out, inn):
    """Normal weights of variance 1/in, quantised by blocks of 32 to 4 bits with fp16 scales."""
    ngrp = -(-inn // 128)
    qs = torch.empty(experts, out, 64 * ngrp, dtype=torch.uint8, device="cuda")
    sc = torch.empty(experts, out, 4 * ngrp, dtype=torch.float16, device="cuda")
    for e in range(experts):
        w = torch.randn(out, inn // 32, 32, generator=gen, device="cuda") / math.sqrt(inn)
        s = (w.abs().amax(-1) / 7.5).half()
        q = torch.clamp(torch.round(w / s.float()[..., None]), -8, 7).to(torch.int8).view(out, inn)
        qs[e], sc[e] = _q4_layout(q, s)
    return qs, sc


def prepare(case, seed):
    gen = _gen(seed)
    dt = _TORCH[case["dtype"]]
    st = {"case": dict(case)}
    if own:
        from transformer_ffn_rmsnorm_gb300 import ffn
        st["ffn"] = ffn
    rows = case["rows"]
    if case["op"] == "route":
        l = _router_logits(gen, rows, case["experts"])
        if case["masked"]:
            l[max(0, rows - case["masked"]):] = -math.inf     # padding rows: nothing may be chosen
        st["logits"] = l.to(dt)
        st["bias"] = 0.05 * torch.randn(case["experts"], generator=gen, device="cuda") if case["bias"] else None
        st["idx"] = torch.empty(rows, case["k"], dtype=torch.int32, device="cuda")
        st["w"] = torch.empty(rows, case["k"], dtype=torch.float32, device="cuda")
        return st
    if case["op"] == "norm":
        d = case["d"]
        st["x"] = _activations(gen, rows, d, 0.3).to(dt)
        st["res"] = _activations(gen, rows, d).to(dt)
        st["g"] = (1.0 + 0.1 * torch.randn(d, generator=gen, device="cuda")).to(dt)
        st["r"] = torch.empty_like(st["x"])
        if case["quant"]:
            st["q"] = torch.empty(rows, d, dtype=torch.float8_e4m3fn, device="cuda")
            st["scales"] = torch.empty(rows, -(-d // case["group"]) if case["group"] else 1, device="cuda")
        else:
            st["n"] = torch.empty_like(st["x"])
        return st
    d, f, experts, k = case["d"], case["ffn"], case["experts"], case["k"]
    st["x"] = _activations(gen, rows, d).to(dt)
    st["res"] = _activations(gen, rows, d).to(dt) if case["residual"] else None
    l = _router_logits(gen, rows, experts)
    top = torch.topk(l, k, dim=1)
    st["idx"] = top.indices.to(torch.int32)
    st["w"] = torch.softmax(top.values, dim=1).contiguous()
    if case["op"] == "q4":
        st["gate"], st["up"] = _q4_weight(gen, experts, f, d), _q4_weight(gen, experts, f, d)
        st["down"] = _q4_weight(gen, experts, d, f)
    else:
        def weight(o, i):
            w = torch.empty(experts, o, i, dtype=dt, device="cuda")
            for e in range(experts):
                w[e] = torch.randn(o, i, generator=gen, device="cuda") / math.sqrt(i)
            return w
        st["gate"], st["up"], st["down"] = weight(f, d), weight(f, d), weight(d, f)
    st["y"] = torch.empty_like(st["x"])
    if own:
        flags = 0
        if case["op"] == "q4":
            need = ffn.ffn_moe_q4_workspace_bytes(rows, d, f, experts, k)
        else:
            if case["prepared"]:                    # laid out once, where the weights are loaded
                flags = ffn.FFN_PREPARED_WEIGHTS
                for name in ("gate", "up", "down"):
                    st[name] = ffn.ffn_prepare_weights(st[name])
            need = ffn.ffn_moe_workspace_bytes(rows, d, f, experts, k, dt, flags)
        st["flags"], st["ws"] = flags, ffn.workspace(need, "cuda")
    return st


# ------------------------------------------------------------------ plain forms
def _plain_route(st):
    c = st["case"]
    l = st["logits"].double()
    l = torch.where(torch.isnan(l), -math.inf, l).clamp(max=3.4028234663852886e38)
    live = l > -math.inf
    top = l.max(dim=1, keepdim=True).values
    top = torch.where(top > -math.inf, top, 0.0)
    if c["sigmoid"]:
        s = 1.0 / (1.0 + torch.exp(-l))
    else:
        e = torch.exp(l - top)
        s = e / e.sum(dim=1, keepdim=True).clamp(min=1e-300)
    order = s + st["bias"].double() if st["bias"] is not None else l     # scores rise with the logits
    order = torch.where(live, order, -math.inf)
    if c["groups"] > 1:
        two = (s + st["bias"].double()) if st["bias"] is not None else s
        two = torch.where(live, two, -math.inf).view(len(l), c["groups"], -1)
        two = two.sort(dim=2, descending=True).values[:, :, :2]
        none = two[:, :, 0] == -math.inf
        group = torch.where(none, -math.inf, torch.where(two > -math.inf, two, 0.0).sum(dim=2))
        kept = group.sort(dim=1, descending=True, stable=True).indices[:, :c["topk_groups"]]
        keep = torch.zeros_like(group, dtype=torch.bool).scatter_(1, kept, True)
        keep = keep[:, :, None].expand(-1, -1, c["experts"] // c["groups"]).reshape(len(l), -1)
        order = torch.where(keep, order, -math.inf)
    best = order.sort(dim=1, descending=True, stable=True)
    idx, some = best.indices[:, :c["k"]], best.values[:, :c["k"]] > -math.inf
    w = torch.where(some, s.gather(1, idx), 0.0)
    if c["renorm"]:
        w = w / w.sum(dim=1, keepdim=True).clamp(min=SMALLEST_SUM)
    return {"idx": torch.where(some, idx, -1).to(torch.int32), "w": (w * c["scale"]).float()}


def _plain_norm(st):
    c = st["case"]
    r = (st["x"].float() + st["res"].float()).to(st["x"].dtype)
    f = r.float()
    n = f * torch.rsqrt((f * f).mean(dim=1, keepdim=True) + EPS) * st["g"].float()
    if not c["quant"]:
        return {"r": r, "n": n.to(r.dtype)}
    rows, d = n.shape
    group = c["group"] or d
    ngrp = -(-d // group)
    full = n if ngrp * group == d else torch.cat([n, n.new_zeros(rows, ngrp * group - d)], dim=1)
    full = full.view(rows, ngrp, group)
    amax = full.abs().amax(dim=2).clamp(min=SMALLEST_AMAX)
    q = (full * (E4M3_MAX / amax)[:, :, None]).view(rows, -1)[:, :d]
    return {"r": r, "q": q.to(torch.float8_e4m3fn), "scales": amax / E4M3_MAX}


def _q4_values(qs, sc, inn):
    """The 32-bit weights of experts' matrices in the device layout."""
    lead = qs.shape[:-1]
    byte = qs.view(*lead, -1, 4, 4, 4).transpose(-3, -2).reshape(*lead, -1, 16)
    u = torch.cat([byte & 15, byte >> 4], dim=-1).float() - 8.0
    return (u * sc.float()[..., None]).view(*lead, -1)[..., :inn]


def _plain_moe(st):
    c = st["case"]
    rows, k = st["idx"].shape
    x, w = st["x"].float(), st["w"]
    idx = st["idx"].long()

    def weights(which, pick, inn):
        if c["op"] == "q4":
            return _q4_values(st[which][0][pick], st[which][1][pick], inn)
        return st[which][pick].float()

    def silu(z):
        return z / (1.0 + torch.exp(-z))

    d, f = c["d"], c["ffn"]
    y = st["res"].float() if st["res"] is not None else torch.zeros_like(x)
    if rows * k <= c["experts"]:                     # few tokens: their experts' weights, one product each
        pick = idx.reshape(-1)
        xs = x.repeat_interleave(k, dim=0)[:, :, None]
        h = silu(torch.bmm(weights("gate", pick, d), xs)) * torch.bmm(weights("up", pick, d), xs)
        o = torch.bmm(weights("down", pick, f), h)[:, :, 0]
        y = y + (o.view(rows, k, d) * w[:, :, None]).sum(dim=1)
    else:                                            # each expert's tokens together
        y = y.clone()
        for e in range(c["experts"]):
            at, slot = torch.nonzero(idx == e, as_tuple=True)
            xs = x[at]
            h = silu(xs @ weights("gate", e, d).T) * (xs @ weights("up", e, d).T)
            y.index_add_(0, at, (h @ weights("down", e, f).T) * w[at, slot][:, None])
    return y.to(st["x"].dtype)


def run(state):
    c = state["case"]
    op = c["op"]
    if not own:
        return _plain_route(state) if op == "route" else _plain_norm(state) if op == "norm" else _plain_moe(state)
    ffn = state["ffn"]
    if op == "route":
        flags = (ffn.FFN_ROUTE_SIGMOID if c["sigmoid"] else 0) | (ffn.FFN_ROUTE_RENORM if c["renorm"] else 0)
        idx, w = ffn.ffn_moe_route(state["logits"], c["k"], bias=state["bias"], groups=c["groups"],
                                   topk_groups=c["topk_groups"], scale=c["scale"], flags=flags, idx=state["idx"],
                                   weights=state["w"])
        return {"idx": idx, "w": w}
    if op == "norm":
        if c["quant"]:
            r, q, scales = ffn.ffn_add_rmsnorm_e4m3(state["x"], state["g"], EPS, res=state["res"], group=c["group"],
                                                    r_out=state["r"], out=state["q"], scales=state["scales"])
            return {"r": r, "q": q, "scales": scales}
        r, n = ffn.ffn_add_rmsnorm(state["x"], state["g"], EPS, res=state["res"], r_out=state["r"], out=state["n"])
        return {"r": r, "n": n}
    if op == "q4":
        return ffn.ffn_moe_forward_q4(state["x"], state["idx"], state["w"], state["gate"], state["up"], state["down"],
                                      ffn=c["ffn"], res=state["res"], out=state["y"], ws=state["ws"])
    return ffn.ffn_moe_forward(state["x"], state["idx"], state["w"], state["gate"], state["up"], state["down"],
                               res=state["res"], flags=state["flags"], out=state["y"], ws=state["ws"])


# ------------------------------------------------------------------ work and exact values
def work(case):
    es = 4 if case["dtype"] == "f32" else 2
    rows = case["rows"]
    if case["op"] == "route":
        return {"bytes": rows * (case["experts"] * es + case["k"] * 8) + (4 * case["experts"] if case["bias"] else 0),
                "flops": rows * case["experts"] * 4.0}
    if case["op"] == "norm":
        d = case["d"]
        out = rows * d + 4 * rows * (-(-d // case["group"]) if case["group"] else 1) if case["quant"] else rows * d * es
        return {"bytes": 3 * rows * d * es + d * es + out, "flops": 5.0 * rows * d}
    d, f, experts, k = case["d"], case["ffn"], case["experts"], case["k"]
    read = experts * (1.0 - (1.0 - k / experts) ** rows)      # experts that some token chooses, at equal odds
    if case["op"] == "q4":
        per = 2 * f * (-(-d // 128)) * 72 + d * (-(-f // 128)) * 72
    else:
        per = 3 * d * f * es
    return {"bytes": read * per + rows * d * es * (3 if case["residual"] else 2) + rows * k * 8,
            "flops": 6.0 * rows * k * d * f}


def _exact_route(st):
    c = st["case"]
    l = st["logits"].double().cpu().numpy()
    b = st["bias"].double().cpu().numpy() if st["bias"] is not None else None
    rows, experts = l.shape
    k, per = c["k"], experts // c["groups"]
    idx = np.full((rows, k), -1, dtype=np.int32)
    w = np.zeros((rows, k))
    for t in range(rows):
        z = l[t]
        ok = np.isfinite(z)
        if not ok.any():
            continue
        if c["sigmoid"]:
            s = 1.0 / (1.0 + np.exp(-z))
        else:
            s = np.exp(z - z[ok].max())
            s = s / s.sum()
        score = s + b if b is not None else s
        score = np.where(ok, score, -np.inf)
        key = score if b is not None else np.where(ok, z, -np.inf)
        if c["groups"] > 1:
            g = np.sort(score.reshape(-1, per), axis=1)[:, ::-1]
            total = g[:, 0] + (np.where(np.isinf(g[:, 1]), 0.0, g[:, 1]) if per > 1 else 0.0)
            kept = np.argsort(-total, kind="stable")[:c["topk_groups"]]
            inside = np.isin(np.arange(experts) // per, kept)
            key = np.where(inside, key, -np.inf)
        best = np.argsort(-key, kind="stable")[:k]
        best = best[key[best] > -np.inf]
        idx[t, :len(best)] = best
        v = s[best]
        w[t, :len(best)] = c["scale"] * (v / max(v.sum(), SMALLEST_SUM) if c["renorm"] else v)
    return {"idx": torch.from_numpy(idx), "w": torch.from_numpy(w)}


def _exact_norm(st):
    c = st["case"]
    r = st["x"].double() + st["res"].double()
    stored = r.to(st["x"].dtype).double()
    n = stored / torch.sqrt(torch.sum(stored ** 2, dim=1, keepdim=True) / c["d"] + EPS) * st["g"].double()
    if not c["quant"]:
        return {"r": r, "n": n}
    group = c["group"] or c["d"]
    parts = [n[:, i:i + group] for i in range(0, c["d"], group)]
    scale = [torch.clamp(p.abs().max(dim=1, keepdim=True).values, min=SMALLEST_AMAX) / E4M3_MAX for p in parts]
    return {"r": r, "q": torch.cat([p / s for p, s in zip(parts, scale)], dim=1), "scales": torch.cat(scale, dim=1)}


def _exact_q4(qs, sc, inn):
    """One matrix' weights by the layout's definition, weight by weight."""
    i = torch.arange(inn, device=qs.device)
    j = i % 32                                                   # weight inside its block
    byte = j % 16                                                # canonical byte
    at = 64 * (i // 128) + 16 * (byte // 4) + 4 * ((i // 32) % 4) + byte % 4
    u = (qs[:, at].to(torch.int64) >> (4 * (j // 16))) & 15
    return (u - 8).double() * sc.double()[:, i // 32]


def _exact_moe(st):
    c = st["case"]
    idx = st["idx"].long()
    x = st["x"].double()
    y = st["res"].double() if st["res"] is not None else torch.zeros_like(x)
    for e in torch.unique(idx).tolist():
        if c["op"] == "q4":
            wg, wu, wd = (_exact_q4(st[n][0][e], st[n][1][e], i) for n, i in (("gate", c["d"]), ("up", c["d"]),
                                                                               ("down", c["ffn"])))
        else:
            wg, wu, wd = (st[n][e].double() for n in ("gate", "up", "down"))
        share = torch.where(idx == e, st["w"].double(), 0.0).sum(dim=1)
        at = torch.nonzero((idx == e).any(dim=1))[:, 0]
        g, u = x[at] @ wg.T, x[at] @ wu.T
        y[at] = y[at] + share[at, None] * ((g * torch.sigmoid(g) * u) @ wd.T)
    return y


def exact(case, seed):
    if case["op"] in ("moe", "q4") and 6.0 * case["rows"] * case["k"] * case["d"] * case["ffn"] > 4e12:
        return None                                              # over 20 seconds in 64 bits
    global own
    was, own = own, False                                        # the weights as they were made
    try:
        st = prepare(case, seed)
    finally:
        own = was
    return _exact_route(st) if case["op"] == "route" else _exact_norm(st) if case["op"] == "norm" else _exact_moe(st)
