"""8-bit storage of blocks near the smallest numbers, whose scales are a few steps
of 2^-149 or would be 0.

Bounds: a scale below the normal numbers is the quotient by 448 rounded up, so less
than 2^-149 above it; a code is off by half a step, 2^-4 of its value or 2^-10, and
the quotient before it by 2^-24."""
import pytest
import torch

import newton_schulz_07_gb300 as ns

pytestmark = pytest.mark.gpu

STEP = 2.0 ** -149


def _rows(tops, dim, seed):
    """fp32 rows of the given largest magnitudes, in whole steps, zeros among them."""
    g = torch.Generator().manual_seed(seed)
    t = torch.tensor(tops, dtype=torch.float64)[:, None]
    x = ((torch.rand((len(tops), dim), generator=g, dtype=torch.float64) * 2 - 1) * t / STEP).round() * STEP
    x[:, ::7] = 0.0
    x[:, 1::128] = t
    return x.float()


def _check(x, q, scales, wide):
    """Rows x in 64 bits against codes and scales; `wide` the scales of each value."""
    assert torch.isfinite(q.float()).all() and torch.isfinite(scales).all()
    x, q, wide = x.double().cpu(), q.double().cpu(), wide.double().cpu()
    off = torch.maximum(2.0 ** -4 * x.abs(), 2.0 ** -10 * wide) * (1 + 2.0 ** -20)
    assert torch.all((q * wide - x).abs() <= off)


TOPS = [STEP, 2 * STEP, 100 * STEP, 224 * STEP, 225 * STEP, 447 * STEP, 627 * STEP, 672 * STEP, 1000 * STEP, 6000 * STEP, 1e-41, 1e-39,
        5e-36, 1e-34]


@pytest.mark.parametrize("dim", [128, 130, 264, 129])
def test_rows(dim):
    x = _rows(TOPS, dim, 1).cuda()
    q, scales = ns.muon_quantize8(x)
    assert not q.float()[:, ::7].any()
    _check(x, q, scales, scales.repeat_interleave(128, 1)[:, :dim])
    top = torch.nn.functional.pad(x.double(), (0, -dim % 128)).unflatten(1, (-1, 128)).abs().amax(2)
    # (A block of zeros, here the one column of the first row behind 128, has a scale of 1.)
    s, want = scales.double(), torch.where(top > 0, top / 448.0, torch.ones_like(top))
    low = want < 2.0 ** -126
    assert torch.all((s >= want) & (s < want + STEP) | ~low)
    assert torch.all((s - want).abs() <= 2.0 ** -23 * want + STEP * low.double())


def test_blocks_of_a_matrix_and_their_product():
    for top in (STEP, 200 * STEP, 3e-43, 1e-42):
        W = torch.randn((1, 200, 272), generator=torch.Generator().manual_seed(2)).cuda()
        W[0, :128, 128:256] = _rows([top] * 128, 128, 3).cuda()
        q, scales = ns.muon_quantize8(W, square=True)
        wide = scales.repeat_interleave(128, 1)[:, :200].repeat_interleave(128, 2)[:, :, :272]
        _check(W[0, :128, 128:256], q[0, :128, 128:256], scales, wide[0, :128, 128:256])
        x, xs = ns.muon_quantize8(torch.randn((5, 272), device="cuda"))
        y = ns.muon_experts8(x, xs, q, scales, torch.tensor([0, 5], dtype=torch.int32, device="cuda"))
        assert torch.isfinite(y.float()).all()


@pytest.mark.parametrize("dim", [300, 20000])
def test_norm_in_8_bits(dim):
    # eps is all of the mean, so r = 1 and the results are the rows themselves; short
    # rows have the scale rounded to nearest, with codes of the exact quotient.
    x = _rows(TOPS, dim, 4).cuda()
    q, scales, _, rstd = ns.muon_rms_norm8(x, torch.ones(dim, device="cuda"), eps=1.0)
    assert torch.all(rstd == 1) and torch.isfinite(q.float()).all() and torch.isfinite(scales).all()
    got = q.double() * scales.double().repeat_interleave(128, 1)[:, :dim]
    size = torch.nn.functional.pad(x.double(), (0, -dim % 128)).unflatten(1, (-1, 128)).abs().amax(2).repeat_interleave(128, 1)[:, :dim]
    off = torch.maximum(2.0 ** -4 * x.double().abs(), 2.0 ** -10 * (size / 448.0 + STEP)) + 448 * STEP
    assert torch.all((got - x.double()).abs() <= off * (1 + 2.0 ** -20))
