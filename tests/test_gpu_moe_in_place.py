"""What the norm returns as its sum where its result is written over its input."""
import pytest
import torch

import newton_schulz_07_gb300 as ns

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_no_sum_is_left_where_y_is_written_over_x(dtype):
    g = torch.Generator(device="cuda").manual_seed(1)
    x, more = (torch.randn((6, 264), generator=g, device="cuda").to(dtype) for _ in range(2))
    w = torch.rand(264, generator=g, device="cuda")
    y, s, rstd = ns.muon_rms_norm(x, w)
    assert s is x
    for view in (lambda t: t, lambda t: t.view(2, 3, 264).view(6, 264)):
        a = x.clone()
        got = ns.muon_rms_norm(a, w, out=view(a))
        assert got[1] is None and torch.equal(got[0], y) and torch.equal(a, y) and torch.equal(got[2], rstd)
    with pytest.raises(TypeError):
        ns.muon_rms_norm_grad(y, got[1], w, rstd)
    # With a residual the sum is kept, wherever y goes.
    y, s, rstd = ns.muon_rms_norm(x, w, residual=more)
    for i in range(2):
        a, b = x.clone(), more.clone()
        got = ns.muon_rms_norm(a, w, residual=b, out=(a, b)[i])
        assert torch.equal(got[0], y) and torch.equal(got[1], s)
    assert ns.muon_rms_norm(x[:0], w, out=x[:0])[1].shape == (0, 264)
