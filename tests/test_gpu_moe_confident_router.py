"""The router's gradient where one expert has nearly all of a token: its own part is
the sum of the others' small ones, not what rounding leaves of a difference.

Bounds, with E = 2^-24: an exponent is a rounded difference (E times it), an
exponential is good to 2 ulp, sums of up to 1024 terms by 32 lanes to 64 E, and the
few products, quotients and sums besides to 64 E; relative to the terms of
  dz_j = g_j (d_j - sum_i g_i d_i + dg_m rest), d_j = dg_j - dg_m,
m the choice of largest logit and rest the probability that no choice has."""
import pytest
import torch

import newton_schulz_07_gb300 as ns

pytestmark = pytest.mark.gpu

E = 2.0 ** -24
U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def _reference(z, dg, chosen, renormalize):
    """(gradient in 64 bits, size of its terms), from terms without cancellation."""
    d, dg, at = z.double(), dg.double(), chosen.long()
    picked = torch.zeros_like(d, dtype=torch.bool).scatter_(1, at, True)
    p = torch.softmax(torch.where(picked, d, torch.full_like(d, -torch.inf)) if renormalize else d, 1)
    rest = torch.where(picked, torch.zeros_like(p), p).sum(1, keepdim=True)
    g = p.gather(1, at)
    each = (g[:, None, :] * (dg[:, :, None] - dg[:, None, :])).sum(2) + rest * dg
    dz = (-p * (g * dg).sum(1, keepdim=True)).scatter(1, at, g * each)
    m = d.gather(1, at).argmax(1, keepdim=True)
    off = (dg - dg.gather(1, m)).abs()
    term = g * (off + (g * off).sum(1, keepdim=True) + dg.gather(1, m).abs() * rest)
    size = (p * (g * dg).abs().sum(1, keepdim=True)).scatter(1, at, term)
    return dz, size


@pytest.mark.parametrize("tokens,experts,k", [(300, 40, 1), (300, 40, 2), (70, 40, 8), (501, 200, 13), (100, 1000, 32), (33, 2, 2)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("renormalize", [True, False])
def test_gradient_of_a_confident_token(tokens, experts, k, dtype, renormalize):
    g = torch.Generator().manual_seed(tokens + k)
    z = torch.randn((tokens, experts), generator=g)
    lead = torch.randint(0, experts, (tokens, 1), generator=g)
    z.scatter_add_(1, lead, torch.rand((tokens, 1), generator=g) * 60)
    z, dg = z.to(dtype).cuda(), torch.randn((tokens, k), generator=g).cuda()
    chosen = ns.muon_route(z, k, renormalize=renormalize)[1]
    got = ns.muon_route_grad(dg, z, chosen, renormalize=renormalize).double()
    ref, size = _reference(z, dg, chosen, renormalize)
    spread = (z.double().amax(1, keepdim=True) - z.double().amin(1, keepdim=True)).clamp(max=80.0)
    off = (200 + 2 * spread) * E * size
    # (A product of 1e-37 leaves 2^-24 of itself below the smallest number.)
    assert torch.all((got - ref).abs() <= off + U[dtype] * (ref.abs() + off) + 1e-37)
