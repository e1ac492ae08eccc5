"""The documented gradient of the routed 8-bit layer is the layer's gradient: the examples, run as they stand on a plain
64-bit implementation of the entry points that rounds nothing, against autograd and against differences (CPU)."""

import pytest
import torch

from readme_blocks import block


class Plain:
    """The entry points that the examples call, in 64 bits and without any quantisation."""

    FFN_ROUTE_RENORM = 2

    @staticmethod
    def ffn_quantize_e4m3(x, block_rows=1, transpose=False):
        return (x.transpose(-1, -2) if transpose else x), None

    @staticmethod
    def ffn_add_rmsnorm_e4m3(x, g, eps, res, group):
        r = x + res
        return r, r / torch.sqrt((r * r).mean(dim=1, keepdim=True) + eps) * g, None

    @staticmethod
    def ffn_moe_route(logits, k, flags):
        p, idx = torch.softmax(logits, dim=1).topk(k, dim=1)
        return idx.int(), p / p.sum(dim=1, keepdim=True)

    @staticmethod
    def ffn_moe_sort(x, idx, experts, x_scales=None):
        flat = idx.flatten().long()
        order = torch.argsort(flat, stable=True)
        pos = torch.empty_like(order)
        pos[order] = torch.arange(len(order))
        offsets = torch.cat([torch.zeros(1, dtype=torch.long), torch.bincount(flat, minlength=experts).cumsum(0)])
        return x[order // idx.shape[1]], None, pos.view(idx.shape), offsets

    @staticmethod
    def ffn_linear_e4m3(x, _, w, offsets, res=None, dtype=None):
        at = offsets.tolist()
        y = torch.cat([x[at[e]:at[e + 1]] @ w[0][e].T for e in range(len(w[0]))])
        return y if res is None else res + y

    @classmethod
    def ffn_gateup_e4m3(cls, x, s, w_gate, w_up, offsets):
        gate, up = (cls.ffn_linear_e4m3(x, s, w, offsets) for w in (w_gate, w_up))
        return gate * torch.sigmoid(gate) * up, None

    @staticmethod
    def ffn_moe_unsort(ys, pos, weights=None, res=None):
        rows = ys[pos]
        y = (rows if weights is None else rows * weights[:, :, None]).sum(dim=1)
        return y if res is None else y + res

    @staticmethod
    def ffn_moe_unsort_backward(dy, ys, pos, weights):
        dys = torch.zeros_like(ys)
        dys[pos.flatten()] = (weights[:, :, None] * dy[:, None]).flatten(0, 1)
        return dys, (ys[pos] * dy[:, None]).sum(dim=2)


@pytest.fixture()
def names():
    gen = torch.Generator().manual_seed(3)
    rows, d, f, experts = 11, 12, 20, 10

    def rnd(*shape):
        return torch.randn(*shape, generator=gen, dtype=torch.float64)
    return {"torch": torch, "ffn": Plain, "experts": experts, "x": rnd(rows, d), "stream": rnd(rows, d),
            "g": 1 + 0.1 * rnd(d), "logits": rnd(rows, experts), "dstream": rnd(rows, d),
            "w_gate": rnd(experts, f, d), "w_up": rnd(experts, f, d), "w_down": rnd(experts, d, f)}


def layer(n, w, names):
    """The sum over a token's experts, from the norm's output and the router's weights: the formula, token by token."""
    out = []
    for t in range(len(n)):
        y = 0
        for j, e in enumerate(names["idx"][t].tolist()):
            gate, up = names["w_gate"][e] @ n[t], names["w_up"][e] @ n[t]
            y = y + w[t, j] * (names["w_down"][e] @ (gate * torch.sigmoid(gate) * up))
        out.append(y)
    return torch.stack(out)


def test_example_is_the_layers_gradient(names):
    dstream = names["dstream"]
    exec(block("ffn.ffn_gateup_e4m3(xs"), names)      # rebinds stream, w
    exec(block("ffn.ffn_moe_unsort_backward("), names)
    n, w = names["n"].clone().requires_grad_(), names["w"].clone().requires_grad_()
    y = layer(n, w, names)
    assert torch.allclose(names["r"] + y, names["stream"], rtol=1e-11, atol=1e-11)
    dn, dw = torch.autograd.grad(y, (n, w), dstream)
    assert torch.allclose(names["dn"], dn, rtol=1e-10, atol=1e-10)
    assert torch.allclose(names["dw"], dw, rtol=1e-10, atol=1e-10)
    for at, grad, of in ((names["n"], names["dn"], "n"), (names["w"], names["dw"], "w")):
        step = 1e-6 * torch.randn(at.shape, generator=torch.Generator().manual_seed(4), dtype=torch.float64)
        ends = [layer(at + s * step, names["w"], names) if of == "n" else layer(names["n"], at + s * step, names)
                for s in (1, -1)]
        left, right = ((ends[0] - ends[1]) * dstream).sum() / 2, (grad * step).sum()
        assert abs(left - right) <= 1e-6 * abs(right), of
