"""Clipped bf16 gradients: the exact product with the factor, rounded once, to the bit."""
import pytest
import torch

import load_balancing_amd as mx

pytestmark = pytest.mark.gpu


def once(exact):
    """fp64 values rounded once to bf16, ties to even; below 2^-126 its steps are 2^-133."""
    _, e = torch.frexp(exact)
    step = torch.ldexp(torch.ones_like(exact), (e - 8).clamp(min=-133))
    return (torch.round(exact / step) * step).bfloat16()


def near_tie(g):
    """A factor of 24 bits below 1 whose product with the odd integer g (8 bits) is no tie
    of bf16, but one once it is rounded to 24 bits: 2 k + 1 halves of a bf16 step, and up to
    g / 2 of the product's last bit beside them, of 2^8 that fp32 drops."""
    out = []
    for k in range(128, 256):
        tie = (2 * k + 1) << 23
        f = (2 * tie + g) // (2 * g)
        if 1 << 23 <= f < 1 << 24 and f * g != tie:
            out.append(f * 2.0 ** -24)
    return out


FACTORS = [f for g in (129, 151, 171, 201, 223, 255) for f in near_tie(g)[::29]]


def clipped(g, f, in_place):
    """g scaled by f: a limit of f on a norm that is given as 1."""
    out = g.clone() if in_place else torch.full_like(g, 5.0)
    table = mx.moonep_grad_table([out]) if in_place else mx.moonep_grad_table([g], [out])
    norm = torch.empty(1, device="cuda")
    mx.moonep_grad_clip(table, f, norm, None, torch.ones(1, device="cuda", dtype=torch.float64))
    assert norm.item() == 1.0
    return out


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("scale", [2.0 ** -7, 2.0 ** 100, 2.0 ** -133])
def test_one_rounding(gpu_ready, scale, in_place):
    """Every significand of bf16 and both signs; the last five values are not part of a
    whole vector.  With the smallest scale results are subnormal, too."""
    g = torch.arange(128, 256, device="cuda").float() * scale
    g = torch.cat([g, -g, -g[-5:]]).bfloat16()
    for f in FACTORS:
        want = once(g.double() * f)  # 8 bits by 24: exact in fp64
        assert torch.equal(clipped(g, f, in_place), want), f


def test_a_norm_beyond_fp32(gpu_ready):
    """Finite gradients whose norm is not finite in fp32 are clipped; the norm says infinity."""
    g = torch.full((1000,), 3.0e38, device="cuda")
    h = g[:10].bfloat16()
    total = ((g.double() ** 2).sum() + (h.double() ** 2).sum()).sqrt().item()
    f = torch.tensor(1.0e30 / total).float().item()
    out = [torch.zeros_like(g), torch.zeros_like(h)]
    norm, work = torch.empty(1, device="cuda"), torch.empty(mx.GRAD_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")
    mx.moonep_grad_clip(mx.moonep_grad_table([g, h], out), 1.0e30, norm, work)
    assert norm.item() == float("inf")
    # the sum of squares in another order may give the factor's neighbour
    assert ((out[0].double() - g.double() * f).abs() <= 2.0 ** -22 * g.double() * f).all()
    assert ((out[1].double() - h.double() * f).abs() <= (2.0 ** -8 + 2.0 ** -22) * h.double() * f).all()
