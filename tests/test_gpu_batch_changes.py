"""One layer and one workspace at changing batches: a call leaves zero what another
batch needs zero, so every result is that of a call on a fresh workspace.

Allowed: the row sums of a layer that is split between blocks are added in any order, in
binary32 (a few 2^-24 of their largest term, about the largest output), then rounded to
binary16 (2^-11): 2^-9 of the largest output covers either call's roundings."""
import pytest
import torch

from trellis_decode_gemv_gb300 import binding as B
from trellis_decode_gemv_gb300 import synth
from tests.gpu_helpers import upload

pytestmark = pytest.mark.gpu

BATCHES = [3, 7, 1, 32, 2, 16, 5, 31, 4]
PREFILLS = [108, 3, 7, 300, 33, 160, 9, 32, 257, 64, 1, 300, 12]


def layer(m, n, K=3):
    w = upload({k: v for k, v in synth.layer_inputs(m, n, K, 1, config=93, index=m // 128).items() if k != "x"})
    return w, K


@pytest.fixture
def fewer_paths():
    yield
    B.exl3_set_path(B.PATH_AUTO)
    B.exl3_set_prefill(B.PREFILL_AUTO)


@pytest.mark.parametrize("m,n", [(128, 512), (640, 128), (1024, 384)])
@pytest.mark.parametrize("path,prefill", [(B.PATH_AUTO, B.PREFILL_FUSED), (B.PATH_AUTO, B.PREFILL_DECODE_ONCE), (B.PATH_SHUFFLE, B.PREFILL_AUTO),
                                          (B.PATH_TENSOR, B.PREFILL_AUTO)])
def test_linear_at_changing_batches(m, n, path, prefill, fewer_paths):
    w, K = layer(m, n)
    B.exl3_set_path(path)
    B.exl3_set_prefill(prefill)
    make = lambda M: B.Exl3Linear(w["codes"], K, B.CB_1MAD, m, n, w["s_in"], w["s_out"], w["scales"], max_batch=M)  # noqa: E731
    for most, batches in ((32, BATCHES), (300, PREFILLS)):
        one = make(most)
        for i, M in enumerate(batches):
            x = torch.randn((M, n), generator=torch.Generator(device="cuda").manual_seed(i), device="cuda").half()
            y, want = one(x), make(M)(x)
            # sums of split layers are added in any order: equal up to that
            scale = float(want.abs().max())
            assert float((y.float() - want.float()).abs().max()) <= 2.0 ** -9 * scale, (M, i)


@pytest.mark.parametrize("m,n", [(128, 512), (1024, 384)])
def test_int8_layer_at_changing_batches(m, n):
    w, K = layer(m, n)
    ws = torch.zeros(B.exl3_gemm_i8_workspace_bytes(m, n, 32), dtype=torch.uint8, device="cuda")
    for i, M in enumerate(BATCHES):
        x = torch.randn((M, n), generator=torch.Generator(device="cuda").manual_seed(i), device="cuda").half()
        q, s = B.exl3_quantize_act(B.exl3_rht_in(x, w["s_in"]))
        for call in (lambda t: B.exl3_gemm_i8(w["codes"], K, B.CB_1MAD, m, n, w["s_out"], w["scales"], q, s, workspace=t),
                     lambda t: B.exl3_gemm_int8act(w["codes"], K, B.CB_1MAD, m, n, w["s_in"], w["s_out"], w["scales"], x, workspace=t)):
            y, want = call(ws), call(None)
            assert float((y.float() - want.float()).abs().max()) <= 2.0 ** -9 * float(want.abs().max()), (M, i)
