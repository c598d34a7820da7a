"""Sampling by dspark_verify_tree: logits with Gumbel noise, in float32."""
import numpy as np
import pytest
import torch

from confidence_driven_speculative_gb300 import binding

pytestmark = pytest.mark.gpu

V, B = 64, 65536


def draws(base, dtype):
    """The tokens of B roots alone, whose row is ``base`` + noise."""
    gen = torch.Generator(device="cuda").manual_seed(0)
    u = torch.rand((B, V), generator=gen, device="cuda").clamp_(1e-7, 1 - 1e-7)
    z = (base - torch.log(-torch.log(u))).to(dtype)
    i32 = dict(dtype=torch.int32, device="cuda")
    h = binding.TreeBuffers(B=B, rows=B, q_max=1, V=V)
    h.bind(z, torch.arange(B + 1, **i32), torch.zeros(B, **i32), torch.zeros(B, **i32))
    binding.dspark_verify_tree(h.tree)
    torch.cuda.synchronize()
    assert (h.num_emitted == 1).all()
    return h.out_tokens.cpu().numpy().reshape(-1)


def test_draws_follow_the_softmax(cuda_lib):
    """Each token's share within five standard deviations."""
    base = torch.linspace(-3, 3, V, device="cuda") + 20
    p = torch.softmax(base.double(), 0).cpu().numpy()
    share = np.bincount(draws(base, torch.float32), minlength=V) / B
    assert (np.abs(share - p) <= 5 * np.sqrt(p * (1 - p) / B)).all()


def test_noise_rounded_to_bfloat16_leans_to_low_ids(cuda_lib):
    """V equal logits: the tokens' mean is (V - 1) / 2, and its standard deviation sqrt((V^2 - 1) / 12 / B).  At 20
    bfloat16 has steps of 1/8: two of the largest are then equal in some 6 of 100 rows, and the lower id wins."""
    base, five = torch.full((V,), 20.0, device="cuda"), 5 * np.sqrt((V * V - 1) / 12 / B)
    assert abs(draws(base, torch.float32).mean() - (V - 1) / 2) <= five
    assert draws(base, torch.bfloat16).mean() < (V - 1) / 2 - five
