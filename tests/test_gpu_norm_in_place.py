"""Norms whose outputs go over their inputs.  exl3_rms_norm_i8 writes h over x or the residual while the
blocks of the other outputs would still read it: few rows, two to four outputs, again and again, with
the bits of a call into tensors of its own."""
import pytest
import torch

from trellis_decode_gemv_gb300 import binding as B

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,n", [(1, 1152), (1, 16384), (3, 4096), (16, 2048), (16, 8192), (5, 32768)])
@pytest.mark.parametrize("outs", [2, 3, 4])
@pytest.mark.parametrize("over", ["x", "residual"])
def test_sum_over_an_input(rows, n, outs, over):
    g = torch.Generator(device="cuda").manual_seed(rows + n + outs)
    w = (1 + 0.2 * torch.randn(n, generator=g, device="cuda")).half()
    signs = [torch.where(torch.randn(n, generator=g, device="cuda") < 0, -1.0, 1.0).half() for _ in range(outs - 1)] + [None]
    calls = []
    for _ in range(100):
        x, r = (torch.randn((rows, n), generator=g, device="cuda").half() for _ in range(2))
        want = B.exl3_rms_norm_i8(x, w, 1e-5, signs, residual=r)
        calls.append((x, r, want))
    torch.cuda.synchronize()
    got = [B.exl3_rms_norm_i8(x, w, 1e-5, signs, residual=r, h=x if over == "x" else r) for x, r, _ in calls]
    for (x, r, want), mine in zip(calls, got):
        assert mine[2] is (x if over == "x" else r)
        assert all(torch.equal(a, b) for a, b in zip(want, mine))


def test_outputs_between_the_rows_of_an_input_and_over_it():
    """What may share memory does: y in the gap behind an input's first row, y and h over inputs of one row of any stride; two
    outputs in one place, and one over an input of another stride, are refused and leave everything as it was."""
    g = torch.Generator(device="cuda").manual_seed(2)
    n, rows = 256, 3
    wide = torch.randn((rows, 4 * n), generator=g, device="cuda").half()
    r = torch.randn((rows, n), generator=g, device="cuda").half()
    w = (1 + 0.2 * torch.randn(n, generator=g, device="cuda")).half()
    x = wide[:, :n]
    want, sums = B.exl3_rms_norm(x, w, 1e-5, residual=r)
    gap = wide[0, n:].view(rows, n)
    y, h = B.exl3_rms_norm(x, w, 1e-5, residual=r, out=gap)
    assert torch.equal(gap, want) and torch.equal(h, sums)
    one, res = wide[:1, :n].clone(), r[:1].clone()
    B.exl3_rms_norm(one, w, 1e-5, residual=res, out=one, h=res)
    assert torch.equal(one, want[:1]) and torch.equal(res, sums[:1])
    before = [t.clone() for t in (wide, r, w)]
    full = wide.view(-1)[:rows * n].view(rows, n)      # x's first bytes, of another stride
    both = torch.empty_like(r)
    for out, total in ((both, both), (r, r), (full, None), (None, full)):
        with pytest.raises(B.Exl3Error):
            B.exl3_rms_norm(x, w, 1e-5, residual=r, out=out, h=total)
    for a, b in zip(before, (wide, r, w)):
        assert torch.equal(a, b)
