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
