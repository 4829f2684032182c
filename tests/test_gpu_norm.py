"""exl3_rms_norm and exl3_rms_norm_i8 on the GPU against float64.

The error allowed: one rounding to binary16 (2^-11 of the value, or half a
subnormal step, 2^-25), and what binary32 adds before it: the sum of squares over a
row (chains of at most 64 terms, 10 levels of joining), the quotient, the root and two
products, in all under 100 roundings of 2^-24, half of them under the root: 2^-18.
The transform adds 10 roundings of 2^-24 of sum |y| / sqrt(128) of the block at most.
"""
import numpy as np
import pytest
import torch

from oracle import block_oracle as BO
from oracle import exl3_oracle as O
from trellis_decode_gemv_gb300 import binding as B
from trellis_decode_gemv_gb300 import synth
from tests.gpu_helpers import assert_layer_close, upload

pytestmark = pytest.mark.gpu


def cuda(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def make(rng, rows, n, spread=0.5):
    x = rng.standard_normal((rows, n)).astype(np.float16)
    r = (rng.standard_normal((rows, n)) * np.exp(spread * rng.standard_normal(n))).astype(np.float16)
    w = (1 + 0.2 * rng.standard_normal(n)).astype(np.float16)
    return x, r, w


def close16(got, ref, more=0.0):
    got = got.double().cpu().numpy()
    allowed = np.abs(ref) * (2.0 ** -11 + 2.0 ** -18) + 2.0 ** -25 + more
    assert np.isfinite(got).all()
    off = np.abs(got - ref)
    assert (off <= allowed).all(), f"{(off / allowed).max():.3f} times what is allowed"


def check_i8(q, qscale, y, signs):
    """y [rows, n] float64 before the rotation, one output after the other."""
    q, qscale = q.double().cpu().numpy(), qscale.double().cpu().numpy()
    for o, s in enumerate(signs):
        z = BO.rotate(y, s).reshape(*y.shape[:-1], -1, 128)
        room = np.abs(y).reshape(z.shape).sum(-1, keepdims=True) / 128 ** 0.5 * 10 * 2.0 ** -24 if s is not None else 0
        off = room + np.abs(z) * 2.0 ** -18 + np.abs(y).reshape(z.shape).max(-1, keepdims=True) * 2.0 ** -18 * 12
        scale = np.abs(z).max(-1) / 127
        got = qscale[o].reshape(scale.shape)
        assert (np.abs(got - scale) <= off.max(-1) / 127 + scale * 2.0 ** -23).all()
        v = q[o].reshape(z.shape) * got[..., None]
        assert (np.abs(v - z) <= got[..., None] * (0.5 + 2.0 ** -16) + off).all()


@pytest.mark.parametrize("rows,n", [(1, 8), (1, 4096), (3, 40), (5, 256), (4, 264), (2, 512), (7, 1000), (9, 1024), (1, 1032), (6, 2048),
                                    (200, 1040), (160, 8192), (2, 16384), (155, 16384), (3, 32768), (200, 32760), (1000, 64)])
@pytest.mark.parametrize("residual", [True, False])
def test_norm(rows, n, residual):
    x, r, w = make(np.random.default_rng(rows + n), rows, n)
    y, h = B.exl3_rms_norm(cuda(x), cuda(w), 1e-5, residual=cuda(r) if residual else None)
    ref, h_ref = BO.rms_norm(x, w, 1e-5, r if residual else None)
    close16(y, ref)
    if residual:
        close16(h, h_ref)
    else:
        assert torch.equal(h.cpu(), torch.from_numpy(x))


@pytest.mark.parametrize("rows,n", [(1, 128), (5, 256), (3, 384), (2, 1024), (16, 4096), (200, 1152), (1, 16384), (170, 8320), (2, 32768)])
@pytest.mark.parametrize("residual", [True, False])
def test_norm_i8(rows, n, residual):
    rng = np.random.default_rng(rows + n)
    x, r, w = make(rng, rows, n)
    signs = [np.where(rng.random(n) < 0.5, -1, 1).astype(np.float16), None, np.where(rng.random(n) < 0.5, -1, 1).astype(np.float16)]
    q, s, h = B.exl3_rms_norm_i8(cuda(x), cuda(w), 1e-5, [None if t is None else cuda(t) for t in signs], residual=cuda(r) if residual else None)
    ref, h_ref = BO.rms_norm(x, w, 1e-5, r if residual else None)
    assert q.shape == (3, rows, n) and s.shape == (3, rows, n // 128)
    check_i8(q, s, ref, signs)
    if residual:
        close16(h, h_ref)


def test_slices_and_outputs_in_place():
    """x and residual as slices of wider tensors; h in place of the residual, y in place of x."""
    rng = np.random.default_rng(1)
    x, r, w = make(rng, 9, 1032)
    wide = torch.zeros((9, 1104), dtype=torch.float16, device="cuda")
    wide[:, 16:1048] = cuda(x)
    res = torch.full((9, 2064), 3.0, dtype=torch.float16, device="cuda")
    res[:, :1032] = cuda(r)
    y, h = B.exl3_rms_norm(wide[:, 16:1048], cuda(w), 1e-6, residual=res[:, :1032])
    ref, h_ref = BO.rms_norm(x, w, 1e-6, r)
    close16(y, ref)
    close16(h, h_ref)
    a, b = cuda(x), cuda(r)
    y2, h2 = B.exl3_rms_norm(a, cuda(w), 1e-6, residual=b, out=a, h=b)
    assert y2 is a and h2 is b and torch.equal(a, y) and torch.equal(b, h)
    one, _ = B.exl3_rms_norm(cuda(x[0]), cuda(w), 1e-6, residual=cuda(r[0]))
    assert one.shape == (1032,) and torch.equal(one, y[0])


def test_rows_that_are_not_finite_stay_alone_and_zeros():
    rng = np.random.default_rng(2)
    x, r, w = make(rng, 6, 2048)
    x[1], r[1] = 0, 0
    x[2, 5], x[3, 700], x[4, 9] = np.nan, np.inf, 65504
    r[4, 9] = 65504                                    # the sum is past binary16: infinite in h, finite in y
    s = np.where(rng.random(2048) < 0.5, -1, 1).astype(np.float16)
    y, h = B.exl3_rms_norm(cuda(x), cuda(w), 1e-5, residual=cuda(r))
    assert torch.isnan(y[2]).all() and torch.isnan(y[3, 700]) and (y[1] == 0).all() and (h[1] == 0).all() and torch.isinf(h[4, 9])
    keep = [0, 1, 4, 5]
    ref, h_ref = BO.rms_norm(x[keep], w, 1e-5, r[keep])
    close16(y[keep], ref)
    assert torch.isfinite(h[[0, 1, 5]]).all()
    q, scale, _ = B.exl3_rms_norm_i8(cuda(x), cuda(w), 1e-5, [cuda(s), None], residual=cuda(r))
    assert torch.isnan(scale[:, 2]).all() and (q[:, 2] == 0).all() and torch.isnan(scale[:, 3, 700 // 128]).all()
    assert (q[:, 3, 640:768] == 0).all() and (scale[:, 1] == 0).all() and (q[:, 1] == 0).all()
    check_i8(q[:, keep], scale[:, keep], ref, [s, None])


def test_eps_and_tiny_values():
    x = np.full((2, 128), 6e-8, np.float16)            # the smallest subnormal
    w = np.ones(128, np.float16)
    for eps in (1e-5, 1e-12, 0.0):
        y, _ = B.exl3_rms_norm(cuda(x), cuda(w), eps)
        close16(y, BO.rms_norm(x, w, eps)[0])


def test_no_rows():
    y, h = B.exl3_rms_norm(torch.empty((0, 256), dtype=torch.float16, device="cuda"), torch.ones(256, device="cuda").half(), 1e-5,
                           residual=torch.empty((0, 256), dtype=torch.float16, device="cuda"))
    assert y.shape == (0, 256) and h.shape == (0, 256)


def test_captured_and_on_another_stream():
    rng = np.random.default_rng(3)
    x, r, w = (cuda(t) for t in make(rng, 5, 4096))
    s = torch.ones(4096, device="cuda").half()
    want = B.exl3_rms_norm(x, w, 1e-5, residual=r) + B.exl3_rms_norm_i8(x, w, 1e-5, [s], residual=r)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = B.exl3_rms_norm(x, w, 1e-5, residual=r) + B.exl3_rms_norm_i8(x, w, 1e-5, [s], residual=r)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = B.exl3_rms_norm(x, w, 1e-5, residual=r) + B.exl3_rms_norm_i8(x, w, 1e-5, [s], residual=r)
    x.copy_(x.flip(0))
    graph.replay()
    want = B.exl3_rms_norm(x, w, 1e-5, residual=r) + B.exl3_rms_norm_i8(x, w, 1e-5, [s], residual=r)
    assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("rows", [1, 7])
def test_norm_before_int8_projections(rows):
    """The norm's int8 outputs through the int8 projections that read them."""
    m, n, K, cb = 256, 512, 3, B.CB_1MAD
    rng = np.random.default_rng(rows)
    x, r, w = make(rng, rows, n)
    hosts = [synth.layer_inputs(m, n, K, rows, config=91, index=i) for i in range(2)]
    devs = [upload({k: v for k, v in t.items() if k != "x"}) for t in hosts]
    q, scale, _ = B.exl3_rms_norm_i8(cuda(x), cuda(w), 1e-5, [d["s_in"] for d in devs], residual=cuda(r))
    for i, (host, dev) in enumerate(zip(hosts, devs)):
        y = B.exl3_gemm_i8(dev["codes"], K, cb, m, n, dev["s_out"], dev["scales"], q[i], scale[i])
        values = (q[i].double().cpu().numpy().reshape(rows, -1, 128) * scale[i].double().cpu().numpy()[..., None]).reshape(rows, n)
        # the layer without its input side, on the values that q and scale stand for
        ref = O.layer_forward(host["codes"], K, cb, m, n, None, host["s_out"], host["scales"], values)
        assert_layer_close(y, ref, f"projection {i}")
