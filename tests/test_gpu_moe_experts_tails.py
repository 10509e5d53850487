"""dW of experts whose rows end anywhere in an MMA's 16, beside experts of NaN."""
import pytest
import torch

import newton_schulz_07_gb300 as ns
from test_gpu_moe_experts import _inputs, _near

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("out,dim", [(64, 72), (136, 264), (520, 512)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_every_tail_beside_nan(out, dim, dtype):
    # Every second expert is NaN, those between have every number of rows from 1 to
    # 80 and some of several stages; a row of a neighbour in any sum would show, in
    # each of the repetitions.
    counts = []
    for n in [*range(1, 81), 127, 128, 129, 191, 200, 321, 399]:
        counts += [n, 1 + n % 23]
    x, W, dy, offsets = _inputs(counts, out, dim, 1)
    at = offsets.tolist()
    for e in range(1, len(counts), 2):
        x[at[e]:at[e + 1]] = float("nan")
        dy[at[e]:at[e + 1]] = float("nan")
    first = None
    for _ in range(20):
        dW = ns.muon_experts_grad(dy, x, W, offsets, dW=torch.empty_like(W, dtype=dtype), need_dx=False)[1]
        if first is None:
            first = dW
            for e in range(0, len(counts), 2):
                q = slice(at[e], at[e + 1])
                _near(dW[e], dy[q].t(), x[q], counts[e])
            assert torch.isnan(dW[1::2]).all()
        assert torch.equal(dW[::2], first[::2])


def test_tails_added_to_what_is_there():
    counts = [5, 40, 0, 77, 16, 129, 1]
    x, W, dy, offsets = _inputs(counts, 136, 264, 2, before=3, after=20)
    x[:3], dy[-20:] = float("nan"), float("inf")
    alone = ns.muon_experts_grad(dy, x, W, offsets, need_dx=False)[1]
    start = torch.randn(alone.shape, device="cuda")
    got = ns.muon_experts_grad(dy, x, W, offsets, dW=start.clone(), accumulate=True, need_dx=False)[1]
    assert torch.isfinite(alone).all() and torch.equal(got, start + alone)


def test_added_right_behind_the_kernel_that_wrote_it():
    # dW is written by ordinary stores of the kernel just before, and read back by
    # ordinary loads of the one just behind.
    counts = [33, 5, 0, 200]
    x, W, dy, offsets = _inputs(counts, 264, 520, 5)
    alone = ns.muon_experts_grad(dy, x, W, offsets, need_dx=False)[1]
    dW = torch.empty_like(alone)
    same = []
    for i in range(50):
        dW.fill_(i)
        ns.muon_experts_grad(dy, x, W, offsets, dW=dW, accumulate=True, need_dx=False)
        same.append((dW == alone + i).all())
        ns.muon_experts_grad(dy, x, W, offsets, dW=dW, need_dx=False)
        same.append((dW == alone).all())
    assert torch.stack(same).all()


def test_the_rows_gradient_needs_no_rows():
    x, W, dy, offsets = _inputs([33, 5, 0, 200], 264, 520, 6)
    ref = ns.muon_experts_grad(dy, x, W, offsets, need_dW=False)[0]
    assert torch.equal(ns.muon_experts_grad(dy, None, W, offsets, need_dW=False)[0], ref)
    with pytest.raises(TypeError):
        ns.muon_experts_grad(dy, None, W, offsets)
