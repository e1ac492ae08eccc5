"""The end of a kernel on CTA pairs after one of the CTAs has given up: all loads of both have landed."""

import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("even,odd", [(1, 1), (4, 4), (0, 1), (1, 0), (0, 4), (4, 0), (2, 3), (3, 2), (4, 8), (8, 4),
                                      (5, 8), (8, 6), (63, 64), (64, 60), (61, 64), (64, 64)])
def test_loads_of_both_land_before_the_pair_ends(even, odd):
    """The even CTA has issued more loads, or the odd one, or both equally many; every wait ends by the loads alone."""
    import torch
    from transformer_ffn_rmsnorm_gb300 import ffn
    ffn.ffn_device_status()
    gen = torch.Generator(device="cuda").manual_seed(even * 100 + odd)
    for _ in range(20):
        src = torch.randint(0, 255, (8192 * max(even, odd),), generator=gen, device="cuda", dtype=torch.uint8)
        assert ffn.ffn_selftest_pair_end(src, even, odd).tolist() == [0, 0]
    ffn.ffn_device_status()
