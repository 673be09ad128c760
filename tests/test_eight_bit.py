"""The 8-bit operators on the CPU: their oracle's pins, the binding's refusals
and the C ABI's argument errors.  No test here needs a GPU."""

import ctypes
from fractions import Fraction

import numpy as np
import pytest
import torch

import oracle
from factored_weight_norm_b200 import build as build_mod
from factored_weight_norm_b200 import dora as D

# ------------------------------------------------------------ oracle's pins


def _nearest_even(q: Fraction) -> int:
    low = q.numerator // q.denominator
    rest = q - low
    if rest != Fraction(1, 2):
        return low + (rest > Fraction(1, 2))
    return low + (low & 1)


@pytest.mark.parametrize("width", [None, 4, 128])
def test_encode_is_the_rational_rounding(width):
    rng = np.random.default_rng(3)
    v = rng.standard_normal((6, 11)).astype(np.float32)
    v[1] = torch.from_numpy(v[1]).to(torch.bfloat16).float().numpy()
    v[2] = np.arange(11) / 2.0 * 127.0 / 8.0     # halves: 127 v / max is k + 1/2 for some
    v[3] = np.array([1.0, 0.5, 0.25, -0.5, 2.0, 1.0, -1.0, 0.125, 4.0, -2.0, 1.5])  # power-of-two tops: exact ties
    v[4] = 0.0
    codes, scale = oracle.encode(v, width)
    w = 11 if width is None else width
    for i in range(v.shape[0]):
        for j in range(v.shape[1]):
            part = [Fraction(float(x)) for x in v[i, j // w * w:(j // w + 1) * w]]
            top = max(abs(x) for x in part)
            want = _nearest_even(127 * Fraction(float(v[i, j])) / top) if top else 0
            assert codes[i, j] == want
            assert scale[i, j // w] == float(top) / 127.0
    assert np.all(np.abs(oracle.decode(codes, scale, width) - v) <= scale.max() / 2 * (1 + 1e-12))


def test_encode_of_tiny_and_non_finite_rows():
    v = np.array([[1e-31, -1e-31], [np.inf, 1.0], [np.nan, 1.0], [2.0 ** -100, 0.0]])
    codes, scale = oracle.encode(v)
    assert scale[0, 0] == 0 and not codes[0].any()
    assert np.isnan(scale[1, 0]) and np.isnan(scale[2, 0]) and not codes[1:3].any()
    assert codes[3, 0] == 127


def test_linear_and_backward_against_loops_and_autograd():
    rng = np.random.default_rng(4)
    T, K, N, r, s = 3, 5, 4, 2, -0.75
    xq, wq = rng.integers(-128, 128, (T, K)), rng.integers(-128, 128, (N, K))
    xs, ws, m, n, b = (rng.uniform(0.5, 2, k) for k in (T, N, N, N, N))
    x, A, B = rng.standard_normal((T, K)), rng.standard_normal((r, K)), rng.standard_normal((N, r))
    y = oracle.linear_i8(xq, xs, wq, ws, x, A, B, m, n, s, b)
    for t in range(T):
        for o in range(N):
            base = sum(int(xq[t, k]) * int(wq[o, k]) for k in range(K)) * xs[t] * ws[o]
            low = sum(sum(x[t, k] * A[j, k] for k in range(K)) * B[o, j] for j in range(r))
            assert abs(y[t, o] - (b[o] + m[o] / n[o] * (base + s * low))) < 1e-12 * max(1.0, abs(y[t, o]))
    plain = oracle.linear_i8(xq, xs, wq, ws, None, None, None, None, None, s, None)
    assert np.allclose(plain, (xq @ wq.T) * np.outer(xs, ws), rtol=1e-13)

    base, lora, dy = (rng.standard_normal((T, N)) for _ in range(3))
    tb, tl, tm = (torch.from_numpy(a.copy()).requires_grad_() for a in (base, lora, m))
    (torch.from_numpy(dy) * (tm / torch.from_numpy(n)) * (tb + s * tl)).sum().backward()
    got = oracle.compose_backward_kept(dy, base + s * lora, m, n, s)
    for a, want in zip(got, (tb.grad, tl.grad, tm.grad)):
        assert np.allclose(a, want.numpy(), rtol=1e-12, atol=1e-14)


def test_rms_factor_against_a_loop():
    h = np.random.default_rng(5).standard_normal((3, 7))
    f = oracle.rms_factor(h, 1e-3)
    for i in range(3):
        assert abs(f[i, 0] - (sum(v * v for v in h[i]) / 7 + 1e-3) ** -0.5) < 1e-14


# ------------------------------------------------------- binding's refusals
T, N, K, R = 4, 256, 32, 8
BF, F32 = torch.bfloat16, torch.float32


def _z(*shape, dtype=BF):
    return torch.zeros(*shape, dtype=dtype)


def _linear(**over):
    a = dict(x_q=_z(T, K, dtype=torch.int8), x_scale=_z(T, dtype=F32), W_q=_z(N, K, dtype=torch.int8),
             w_scale=_z(N, dtype=F32), x=_z(T, K), A=_z(R, K), B=_z(N, R), m=_z(N, dtype=F32), n=_z(N, dtype=F32),
             s=0.5, bias=None, y=None)
    return {**a, **over}


@pytest.mark.parametrize("over, exc", [
    (dict(x_q=_z(T, K)), TypeError),
    (dict(W_q=_z(N, K + 16, dtype=torch.int8)), ValueError),
    (dict(x_scale=_z(T + 1, dtype=F32)), ValueError),
    (dict(w_scale=_z(N)), TypeError),
    (dict(x=None), ValueError),
    (dict(B=None), ValueError),
    (dict(x=None, A=None), ValueError),
    (dict(m=None), ValueError),
    (dict(x=_z(T, K, dtype=F32)), TypeError),
    (dict(A=_z(R, K + 8)), ValueError),
    (dict(B=_z(N, R + 8)), ValueError),
    (dict(bias=_z(N, dtype=F32)), TypeError),
    (dict(y=_z(T, N, dtype=F32)), TypeError),
    (dict(y=_z(T, N - 8)), ValueError),
    (dict(x_q=_z(T, dtype=torch.int8)), ValueError),
    (dict(), ValueError),  # consistent, but on the host
])
def test_linear_i8_mismatches_raise(over, exc):
    with pytest.raises(exc):
        D.dora_linear_i8_fwd(**_linear(**over))


@pytest.mark.parametrize("call, exc", [
    (lambda: D.dora_quantize_rows_i8(_z(T)), ValueError),
    (lambda: D.dora_quantize_rows_i8(_z(T, N, dtype=torch.float16)), TypeError),
    (lambda: D.dora_quantize_rows_i8(_z(T, N), residual=_z(T, N, dtype=F32)), TypeError),
    (lambda: D.dora_quantize_rows_i8(_z(T, N), h=_z(T, N)), ValueError),
    (lambda: D.dora_quantize_rows_i8(_z(T, N), q=_z(T, N)), TypeError),
    (lambda: D.dora_quantize_rows_i8(_z(T, N), scale=_z(T, 1, dtype=F32)), ValueError),
    (lambda: D.dora_quantize_rows_i8(_z(T, N)), ValueError),
    (lambda: D.dora_rms_norm_i8(_z(T, N), _z(N, dtype=F32)), TypeError),
    (lambda: D.dora_rms_norm_i8(_z(T, N), _z(N - 8)), ValueError),
    (lambda: D.dora_rms_norm_i8(_z(T, N), _z(N), y=_z(T, N, dtype=F32)), TypeError),
    (lambda: D.dora_rms_norm_i8(_z(T, N), _z(N), residual=_z(T + 1, N)), ValueError),
    (lambda: D.dora_rms_norm_i8(_z(T, N), _z(N)), ValueError),
    (lambda: D.dora_dequantize_i8(_z(T, N), _z(T, dtype=F32)), TypeError),
    (lambda: D.dora_dequantize_i8(_z(T, N, dtype=torch.int8), _z(T, 3, dtype=F32)), ValueError),
    (lambda: D.dora_dequantize_i8(_z(T, N, dtype=torch.int8), _z(T, dtype=F32), dtype=torch.float16), TypeError),
    (lambda: D.dora_dequantize_i8(_z(T, N, dtype=torch.int8), _z(T, dtype=F32), out=_z(T, 8)), ValueError),
    (lambda: D.dora_dequantize_i8(_z(T, N, dtype=torch.int8), _z(T, dtype=F32)), ValueError),
])
def test_rows_i8_mismatches_raise(call, exc):
    with pytest.raises(exc):
        call()


def _fwd(**over):
    a = dict(base_out=_z(T, N), lora_out=_z(T, N), m=_z(N, dtype=F32), n=_z(N, dtype=F32), s=0.5)
    return {**a, **over}


def _bwd(**over):
    a = dict(dy=_z(T, N), z8=_z(T, N, dtype=torch.int8), z_scale=_z(T, N // 128, dtype=F32), m=_z(N, dtype=F32),
             n=_z(N, dtype=F32), s=0.5)
    return {**a, **over}


@pytest.mark.parametrize("fn, over, exc", [
    ("f", dict(lora_out=_z(T, N, dtype=F32)), TypeError),
    ("f", dict(y=_z(T, N + 8)), ValueError),
    ("f", dict(z8=_z(T, N)), TypeError),
    ("f", dict(z_scale=_z(T, dtype=F32)), ValueError),
    ("f", dict(bias=_z(N, dtype=F32)), TypeError),
    ("f", dict(m=_z(N)), TypeError),
    ("f", dict(), ValueError),
    ("b", dict(z8=_z(T, N)), TypeError),
    ("b", dict(z8=_z(T + 1, N, dtype=torch.int8)), ValueError),
    ("b", dict(z_scale=_z(T, N, dtype=F32)), ValueError),
    ("b", dict(z_scale=_z(T, N // 128)), TypeError),
    ("b", dict(d_base=_z(T, N, dtype=F32)), TypeError),
    ("b", dict(d_m=_z(N)), TypeError),
    ("b", dict(n=_z(N - 8, dtype=F32)), ValueError),
    ("b", dict(), ValueError),
])
def test_checkpoint_mismatches_raise(fn, over, exc):
    with pytest.raises(exc):
        D.dora_compose_fwd_ckpt8(**_fwd(**over)) if fn == "f" else D.dora_compose_bwd_ckpt8(**_bwd(**over))


def test_fused_linear_checkpoint_mismatches_raise():
    a = dict(x=_z(T, K), W=_z(N, K), A=_z(R, K), B=_z(N, R), m=_z(N, dtype=F32), n=_z(N, dtype=F32), s=0.5)
    for over, exc in ((dict(z8=_z(T, N)), TypeError), (dict(z_scale=_z(T, 1, dtype=F32)), ValueError),
                      (dict(x=_z(T, K, dtype=F32)), TypeError), (dict(B=_z(N, R + 8)), ValueError), ({}, ValueError)):
        with pytest.raises(exc):
            D.dora_fused_linear_fwd_ckpt8(**{**a, **over})


# ---------------------------------------------------- C ABI argument errors
FAKE = ctypes.c_void_p(0x10000)  # aligned, never dereferenced
ODD = ctypes.c_void_p(0x10002)


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    return D.lib()


def _call(fn, names, good, **over):
    a = {**dict(zip(names, good)), **over}
    return fn(*[a[k] for k in names])


ROWS = ("x", "residual", "rows", "cols", "dt", "h", "q", "scale", "stream")
ROWS_OK = (FAKE, FAKE, 4, 64, D.DORA_BF16, FAKE, FAKE, FAKE, None)
NORM = ("x", "residual", "weight", "eps", "tokens", "d", "dt", "h", "y", "q", "scale", "stream")
NORM_OK = (FAKE, FAKE, FAKE, 1e-6, 4, 64, D.DORA_BF16, FAKE, FAKE, FAKE, FAKE, None)
LIN = ("x_q", "x_scale", "W_q", "w_scale", "x", "A", "B", "bias", "m", "n", "s", "tokens", "d_in", "d_out", "r", "dt",
       "y", "workspace", "bytes", "stream")
LIN_OK = (FAKE,) * 10 + (0.5, 4, 64, 64, 16, D.DORA_BF16, FAKE, FAKE, 1 << 20, None)
FWD = ("base", "lora", "bias", "m", "n", "s", "tokens", "d_out", "dt", "y", "z8", "z_scale", "stream")
FWD_OK = (FAKE,) * 5 + (0.5, 4, 64, D.DORA_BF16, FAKE, FAKE, FAKE, None)
BWD = ("dy", "z8", "z_scale", "m", "n", "s", "tokens", "d_out", "dt", "d_base", "d_lora", "d_m", "workspace", "bytes",
       "stream")
BWD_OK = (FAKE,) * 5 + (0.5, 4, 64, D.DORA_BF16, FAKE, FAKE, FAKE, FAKE, 1 << 20, None)
FUSED = ("x", "W", "A", "B", "bias", "m", "n", "s", "tokens", "d_in", "d_out", "r", "dt", "y", "z8", "z_scale",
         "workspace", "bytes", "stream")
FUSED_OK = (FAKE,) * 7 + (0.5, 4, 64, 64, 16, D.DORA_BF16, FAKE, FAKE, FAKE, FAKE, 1 << 20, None)
INV, UNS, WS, OK = D.DORA_ERR_INVALID_ARG, D.DORA_ERR_UNSUPPORTED, D.DORA_ERR_WORKSPACE, D.DORA_OK


@pytest.mark.parametrize("name, names, good, cases", [
    ("dora_quantize_rows_i8", ROWS, ROWS_OK, [
        (dict(x=None), INV), (dict(q=None), INV), (dict(scale=None), INV), (dict(h=None), INV), (dict(rows=-1), INV),
        (dict(cols=-8), INV), (dict(cols=60), UNS), (dict(cols=0), UNS), (dict(dt=7), UNS), (dict(x=ODD), UNS),
        (dict(residual=ODD), UNS), (dict(h=ODD), UNS), (dict(q=ODD), UNS), (dict(scale=ODD), UNS),
        (dict(dt=D.DORA_F32, x=ODD), UNS), (dict(rows=1 << 31), UNS), (dict(rows=0), OK)]),
    ("dora_rms_norm_i8", NORM, NORM_OK, [
        (dict(weight=None), INV), (dict(eps=-1.0), INV), (dict(eps=float("nan")), INV), (dict(h=None), INV),
        (dict(weight=ODD), UNS), (dict(y=ODD), UNS), (dict(d=12), UNS), (dict(tokens=0), OK)]),
    ("dora_dequantize_i8", ("q", "scale", "rows", "cols", "block", "dt", "out", "stream"),
     (FAKE, FAKE, 4, 64, 0, D.DORA_BF16, FAKE, None), [
        (dict(q=None), INV), (dict(scale=None), INV), (dict(out=None), INV), (dict(rows=-1), INV),
        (dict(block=64), UNS), (dict(dt=5), UNS), (dict(out=ctypes.c_void_p(0x10001)), UNS), (dict(scale=ODD), UNS),
        (dict(rows=0), OK), (dict(cols=0), OK)]),
    ("dora_linear_i8_fwd", LIN, LIN_OK, [
        (dict(x_q=None), INV), (dict(x_scale=None), INV), (dict(W_q=None), INV), (dict(w_scale=None), INV),
        (dict(y=None), INV), (dict(x=None), INV), (dict(A=None), INV), (dict(B=None), INV), (dict(m=None), INV),
        (dict(n=None), INV), (dict(tokens=-1), INV), (dict(r=-8), INV), (dict(dt=D.DORA_F32), UNS),
        (dict(d_in=72), UNS), (dict(d_in=0), UNS), (dict(d_out=60), UNS), (dict(r=12), UNS), (dict(d_in=131072), UNS),
        (dict(x_q=ODD), UNS), (dict(W_q=ODD), UNS), (dict(y=ODD), UNS), (dict(x=ODD), UNS), (dict(B=ODD), UNS),
        (dict(x_scale=ODD), UNS), (dict(m=ODD), UNS), (dict(bias=ctypes.c_void_p(0x10001)), UNS),
        (dict(workspace=None), WS), (dict(bytes=255), WS), (dict(workspace=ODD), UNS),
        (dict(tokens=0), OK), (dict(d_out=0), OK)]),
    ("dora_compose_fwd_ckpt8", FWD, FWD_OK, [
        (dict(base=None), INV), (dict(z8=None), INV), (dict(z_scale=None), INV), (dict(tokens=-1), INV),
        (dict(d_out=60), UNS), (dict(dt=9), UNS), (dict(z8=ODD), UNS), (dict(bias=ODD), UNS), (dict(z_scale=ODD), UNS),
        (dict(dt=D.DORA_F32, y=ODD), UNS), (dict(tokens=0), OK), (dict(d_out=0), OK)]),
    ("dora_compose_bwd_ckpt8", BWD, BWD_OK, [
        (dict(d_m=None), INV), (dict(z8=None), INV), (dict(dy=None), INV), (dict(d_out=-8), INV),
        (dict(d_out=60), UNS), (dict(z8=ODD), UNS), (dict(d_base=ODD), UNS), (dict(z_scale=ODD), UNS),
        (dict(workspace=None), WS), (dict(bytes=100), WS), (dict(workspace=ODD), UNS), (dict(d_out=0), OK)]),
    ("dora_fused_linear_fwd_ckpt8", FUSED, FUSED_OK, [
        (dict(z8=None), INV), (dict(z_scale=None), INV), (dict(x=None), INV), (dict(z8=ODD), UNS),
        (dict(z_scale=ODD), UNS), (dict(d_in=60), UNS), (dict(workspace=None), WS), (dict(tokens=0), OK)]),
], ids=lambda v: v if isinstance(v, str) else "")
def test_argument_errors(lib, name, names, good, cases):
    for over, status in cases:
        assert _call(getattr(lib, name), names, good, **over) == status, (name, over)


def test_workspaces_have_no_token_by_channel_term(lib):
    assert lib.dora_linear_i8_fwd_workspace_size(8192, 384) == 8192 * 384 * 2
    assert lib.dora_linear_i8_fwd_workspace_size(8192, 0) == 256
    ws = lib.dora_compose_bwd_ckpt8_workspace_size(8192, 8192)
    assert 0 < ws < 8192 * 8192 / 16 and lib.dora_compose_bwd_ckpt8_workspace_size(65536, 8192) == ws
    assert lib.dora_compose_bwd_ckpt8_workspace_size(-1, 8) == 0


def test_rows_written_in_place_are_not_read_through_the_non_coherent_path():
    # h may be x or residual: in the kernels that write it only the weight, which
    # nothing writes, may be read as memory that stays as it is
    import os
    import re

    with open(os.path.join(build_mod.CSRC, "quant8.cuh")) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    rows = text[text.index("struct RowsI8Args"):text.index("void __launch_bounds__(256) dequant_i8_kernel")]
    reads = re.findall(r"(?:IO|VecIO<T, VEC>)::(?:raw|load)\([^\n]*|__ldg\([^\n]*|ld_stream\w*\([^\n]*|ld\.global\.nc", rows)
    assert not reads, reads
    assert "ld.global.nc" not in text[text.index("ld_row(const T* p)"):text.index("struct RowsI8Args")]
