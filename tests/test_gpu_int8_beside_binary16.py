"""Int8 and binary16 calls of one layer in turn on one workspace: either leaves zero what the
other needs zero, so every result is that of a call on a fresh workspace.

Allowed: as at changing batches, 2^-9 of the largest output (sums of split layers are added in
any order, in binary32, then rounded to binary16)."""
import pytest
import torch

from trellis_decode_gemv_gb300 import binding as B
from trellis_decode_gemv_gb300 import synth
from tests.gpu_helpers import upload

pytestmark = pytest.mark.gpu

K = 3


@pytest.fixture
def prefill_of_choice():
    yield
    B.exl3_set_prefill(B.PREFILL_AUTO)


def calls(m, n):
    w = upload({k: v for k, v in synth.layer_inputs(m, n, K, 1, config=95, index=n // 128).items() if k != "x"})

    def half(x, ws):
        if ws is None:
            ws = torch.zeros(B.exl3_gemm_workspace_bytes(m, n, x.shape[0]), dtype=torch.uint8, device="cuda")
        return B.exl3_gemm(w["codes"], K, B.CB_1MAD, m, n, w["s_in"], w["s_out"], w["scales"], x, workspace=ws)

    def int8(x, ws):
        return B.exl3_gemm_int8act(w["codes"], K, B.CB_1MAD, m, n, w["s_in"], w["s_out"], w["scales"], x, workspace=ws)

    def quantized(x, ws):
        q, s = B.exl3_quantize_act(B.exl3_rht_in(x, w["s_in"]))
        return B.exl3_gemm_i8(w["codes"], K, B.CB_1MAD, m, n, w["s_out"], w["scales"], q, s, workspace=ws)
    return dict(half=half, int8=int8, quantized=quantized)


def in_turn(m, n, nbytes, sequence):
    ws = torch.zeros(nbytes, dtype=torch.uint8, device="cuda")
    call = calls(m, n)
    for i, (name, M) in enumerate(sequence):
        x = torch.randn((M, n), generator=torch.Generator(device="cuda").manual_seed(i), device="cuda").half()
        y, want = call[name](x, ws), call[name](x, None)
        assert float((y.float() - want.float()).abs().max()) <= 2.0 ** -9 * float(want.abs().max()), (i, name, M)


# Layers that prefills split along n: 2048 columns in two, 4096 in up to four.
@pytest.mark.parametrize("m,n", [(128, 2048), (640, 4096), (128, 512)])
@pytest.mark.parametrize("prefill", [B.PREFILL_FUSED, B.PREFILL_DECODE_ONCE])
@pytest.mark.parametrize("most", [33, 300])
def test_int8_rows_between_prefills(m, n, prefill, most, prefill_of_choice):
    B.exl3_set_prefill(prefill)
    sequence = [("int8", 32), ("half", most), ("quantized", 16), ("half", 33), ("int8", 4), ("half", most), ("half", 7), ("quantized", 32),
                ("half", most), ("half", 1), ("int8", 1), ("half", 33), ("half", 32), ("int8", 31), ("half", most)]
    in_turn(m, n, max(B.exl3_gemm_workspace_bytes(m, n, most), B.exl3_gemm_i8_workspace_bytes(m, n, 32)), sequence)


@pytest.mark.parametrize("m,n", [(128, 2048), (1024, 384), (640, 128)])
@pytest.mark.parametrize("most", [32, 20, 5])
def test_int8_and_binary16_steps(m, n, most):
    """No prefill: the size that either kind needs at the largest batch of all."""
    sequence = [(name, M) for M in (most, 1, most - 1, 3, most, 2, 4) for name in ("half", "int8", "quantized")]
    in_turn(m, n, max(B.exl3_gemm_workspace_bytes(m, n, most), B.exl3_gemm_i8_workspace_bytes(m, n, most)), sequence)
