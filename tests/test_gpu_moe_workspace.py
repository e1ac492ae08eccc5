"""One workspace, sized for the largest batch, for batches of every smaller size:
a server's last, partial batches.  The split count of the down product and the
choice of kernels change on the way."""

import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    import torch
    from transformer_ffn_rmsnorm_gb300 import ffn
    return torch, ffn


ROWS = [600, 512, 456, 455, 400, 257, 128, 97, 96, 95, 64, 33, 16, 7, 1]


@pytest.mark.parametrize("kind", ["bfloat16", "float16", "prepared"])
def test_one_workspace(env, kind):
    import test_gpu_moe as m
    torch, ffn = env
    dt = torch.float16 if kind == "float16" else torch.bfloat16
    flags = ffn.FFN_PREPARED_WEIGHTS if kind == "prepared" else 0
    d, f, experts, k = 256, 4096, 4, 2
    x, idx, w, wg, wu, wd, res = m.make(torch, ROWS[0], d, f, experts, k, dt)
    mats = [ffn.ffn_prepare_weights(t) for t in (wg, wu, wd)] if flags else [wg, wu, wd]
    for top in (600, 97):
        ws = ffn.workspace(ffn.ffn_moe_workspace_bytes(top, d, f, experts, k, dt, flags), "cuda")
        for r in [r for r in ROWS if r <= top]:
            y = ffn.ffn_moe_forward(x[:r], idx[:r], w[:r], *mats, res=res[:r], flags=flags, ws=ws)
            m.check(torch, y, *m.reference(torch, x[:r], idx[:r], w[:r], wg, wu, wd, res[:r], bool(flags)))
    ffn.ffn_device_status()


def test_one_workspace_q4(env):
    import test_gpu_moe_q4 as m
    torch, ffn = env
    d, f, experts, k = 256, 4096, 4, 2
    x, idx, w, packed, values, res = m.make(torch, ROWS[0], d, f, experts, k)
    for top in (600, 456):
        ws = ffn.workspace(ffn.ffn_moe_q4_workspace_bytes(top, d, f, experts, k), "cuda")
        for r in [r for r in ROWS if r <= top]:
            y = ffn.ffn_moe_forward_q4(x[:r], idx[:r], w[:r], *packed, ffn=f, res=res[:r], ws=ws)
            m.check(torch, y, *m.reference(torch, x[:r], idx[:r], w[:r], values, res[:r]))
    ffn.ffn_device_status()
