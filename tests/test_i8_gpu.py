"""The 8-bit rows (quantiser, norm, reader) and the int8 linear against fp64.

Codes are integers defined by the rounding of an exact quotient, so they are
compared for equality: with bf16 rows every value (and every product with a
bf16 weight) is exact in fp32, with fp32 rows the product is rounded to fp32
once on both sides.  Tolerances, with u = 2^-8 (half a bf16 step) and
e = 2^-24 (half an fp32 step), both relative to the value:
  * a plain row's scale is one fp32 division: equal to the rounded quotient;
  * the norm's factor: a sum of d squares is off by at most d e of itself, so
    its root by d e / 2, and four more operations round: (d / 2 + 4) e;
  * a bf16 output adds u of its value;
  * the linear: P is an fp32 sum of d_in terms rounded to bf16, the adapter's
    product a sum of r more, the epilogue at most eight roundings.
"""

import numpy as np
import pytest
import torch

import oracle
from factored_weight_norm_b200 import dora as D
from tests import parity as P

pytestmark = pytest.mark.gpu
DEV = "cuda"
U, E = 2.0 ** -8, 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32


def _gen(seed):
    return torch.Generator(device="cpu").manual_seed(seed)


def _rows(rows, cols, dtype, seed):
    g = _gen(seed)
    x = torch.randn(rows, cols, generator=g) * torch.exp(0.5 * torch.randn(cols, generator=g))
    return x.to(dtype).to(DEV)


def _host(t):
    return t.detach().cpu().numpy() if t.dtype != BF else P.f64(t)


def _assert_within(got, ref, tol, what):
    err = np.abs(P.f64(got) - ref)
    assert np.all(err <= tol), f"{what}: {np.max(err - tol)} over its bound at {np.argwhere(err > tol)[0]}"


# every thread layout: one, two and four vectors a thread, few and many rows,
# scalar fp32 rows, and rows longer than the registers of one CTA
ROWS = [(1, 8, BF), (3, 264, BF), (1, 8192, BF), (400, 2048, BF), (301, 4096, BF), (300, 8192, BF), (297, 16384, BF),
        (2, 32768, BF), (2, 33000, BF), (1, 1, F32), (5, 33, F32), (2, 4099, F32), (300, 4099, F32), (300, 6000, F32),
        (299, 1024, F32), (1, 8192, F32), (2, 33001, F32), (2, 40000, F32),
        (2500, 4096, BF), (1300, 8192, BF), (1250, 8200, BF), (2400, 4104, F32), (700, 16384, BF), (1200, 8196, F32)]


@pytest.mark.parametrize("rows, cols, dtype", ROWS, ids=lambda v: str(v).replace("torch.", ""))
@pytest.mark.parametrize("residual", [False, True])
def test_quantize_rows(rows, cols, dtype, residual):
    x = _rows(rows, cols, dtype, 1)
    res = _rows(rows, cols, dtype, 2) if residual else None
    q, scale, h = D.dora_quantize_rows_i8(x, residual=res)
    torch.cuda.synchronize()
    want_h = x if res is None else (x.float() + res.float()).to(dtype)
    assert (h is None) if res is None else torch.equal(h, want_h)
    codes, sc = oracle.encode(P.f64(want_h))
    assert np.array_equal(q.cpu().numpy(), codes)
    assert np.array_equal(scale.cpu().numpy(), sc[:, 0].astype(np.float32))


def _norm_reference(h, w, eps, dtype):
    v = P.f64(h) * P.f64(w) if dtype == BF else (h.cpu().numpy() * w.cpu().numpy()).astype(np.float64)
    codes, sc = oracle.encode(v)
    f = oracle.rms_factor(P.f64(h), eps)
    return codes, sc * f, v * f


@pytest.mark.parametrize("rows, cols, dtype", ROWS, ids=lambda v: str(v).replace("torch.", ""))
@pytest.mark.parametrize("residual", [False, True])
def test_rms_norm(rows, cols, dtype, residual):
    eps = 1e-5
    x = _rows(rows, cols, dtype, 3)
    res = _rows(rows, cols, dtype, 4) if residual else None
    w = (1 + 0.2 * torch.randn(cols, generator=_gen(5))).to(dtype).to(DEV)
    q, scale, h, y = D.dora_rms_norm_i8(x, w, eps, residual=res, want_y=True)
    q2, scale2, _, y2 = D.dora_rms_norm_i8(x, w, eps, residual=res)
    torch.cuda.synchronize()
    want_h = x if res is None else (x.float() + res.float()).to(dtype)
    assert (h is None) if res is None else torch.equal(h, want_h)
    assert y2 is None and torch.equal(q, q2) and torch.equal(scale, scale2)
    codes, sc, v = _norm_reference(want_h, w, eps, dtype)
    assert np.array_equal(q.cpu().numpy(), codes)
    rel = (cols / 2 + 5) * E
    _assert_within(scale, sc[:, 0], rel * sc[:, 0], "scale")
    _assert_within(y, v, (rel + E + (U if dtype == BF else 0)) * np.abs(v) * (1 + U), "y")


@pytest.mark.parametrize("dtype", [BF, F32])
def test_rms_norm_updates_the_residual_stream_in_place(dtype):
    x, res = _rows(64, 1024, dtype, 6), _rows(64, 1024, dtype, 7)
    w = torch.ones(1024, dtype=dtype, device=DEV)
    q, scale, h, _ = D.dora_rms_norm_i8(x, w, residual=res)
    for keep in ("residual", "x"):
        a, b = x.clone(), res.clone()
        out = b if keep == "residual" else a
        q2, scale2, h2, _ = D.dora_rms_norm_i8(a, w, residual=b, h=out)
        torch.cuda.synchronize()
        assert h2 is out and torch.equal(out, h) and torch.equal(q2, q) and torch.equal(scale2, scale)
    long_x, long_r = _rows(2, 40000, dtype, 8), _rows(2, 40000, dtype, 9)
    q, scale, h = D.dora_quantize_rows_i8(long_x, residual=long_r)
    q2, scale2, _ = D.dora_quantize_rows_i8(long_x, residual=long_r, h=long_r)
    torch.cuda.synchronize()
    assert torch.equal(long_r, h) and torch.equal(q2, q) and torch.equal(scale2, scale)


@pytest.mark.parametrize("dtype, cols", [(BF, 512), (F32, 512), (F32, 513), (BF, 40000)])
def test_rows_at_the_format_s_edges(dtype, cols):
    x = torch.randn(12, cols, generator=_gen(10))
    x[0] = 0.0
    x[1, 3] = float("inf")
    x[2, 5] = float("nan")
    x[3] = 1e-31
    x[4] = torch.finfo(dtype).max
    x[5] = torch.arange(cols) % 255 / 254.0  # power-of-two tops: exact halves
    x[6] = torch.where(torch.arange(cols) % 2 == 0, 1.0, 0.5)
    x[7] = 2.0 ** -100
    x[8] = -127.0
    x[9, 1:] = 0.0
    x[10] = 2.0 ** -126
    x[11] = (torch.arange(cols) % 8 + 0.5) * (127.0 if dtype == F32 else 128.0) / 128.0
    x = x.to(dtype).to(DEV)
    q, scale, _ = D.dora_quantize_rows_i8(x)
    v = D.dora_dequantize_i8(q, scale, dtype=F32)
    torch.cuda.synchronize()
    codes, sc = oracle.encode(P.f64(x))
    assert np.array_equal(q.cpu().numpy(), codes)
    assert np.array_equal(scale.cpu().numpy(), sc[:, 0].astype(np.float32), equal_nan=True)
    assert torch.isnan(v[1]).all() and torch.isnan(v[2]).all() and not v[0].any() and not v[3].any()
    # a norm whose squares leave fp32's range must not come back as numbers
    q, scale, _, y = D.dora_rms_norm_i8(x, torch.ones(cols, dtype=dtype, device=DEV), want_y=True)
    torch.cuda.synchronize()
    assert torch.isnan(scale[[1, 2, 4]]).all() and scale[0] == 0 and not y[0].any()
    assert torch.isfinite(scale[[0, 3, 5, 6, 7, 8, 9, 10, 11]]).all()


@pytest.mark.parametrize("rows, cols, block", [(1, 1, 0), (3, 130, 128), (70, 128, 128), (5, 4099, 128),
                                                (333, 2056, 128), (9, 1000, 0), (1, 8192, 0), (0, 16, 0), (2, 0, 128)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_dequantize(rows, cols, block, dtype):
    g = _gen(11)
    q = torch.randint(-128, 128, (rows, cols), generator=g, dtype=torch.int8).to(DEV)
    scale = torch.rand((rows,) if block == 0 else (rows, -(-cols // 128)), generator=g).to(DEV)
    out = D.dora_dequantize_i8(q, scale, dtype=dtype)
    into = torch.empty_like(out)
    assert D.dora_dequantize_i8(q, scale, out=into) is into
    torch.cuda.synchronize()
    wide = scale[:, None].expand(rows, cols) if block == 0 else scale.repeat_interleave(128, dim=1)[:, :cols]
    want = (q.float() * wide).to(dtype)
    assert torch.equal(out, want) and torch.equal(into, want)


# ------------------------------------------------------------------- linear
def _module(T, d_in, d_out, r, s=0.5, bias=True, mag=True, seed=20, full=False):
    g = _gen(seed)
    rn = lambda *k: torch.randn(*k, generator=g)  # noqa: E731
    W = (0.02 * rn(d_out, d_in)).to(BF).to(DEV)
    x = rn(T, d_in).to(BF).to(DEV)
    if full:
        xq = torch.randint(-128, 128, (T, d_in), generator=g, dtype=torch.int8).to(DEV)
        wq = torch.randint(-128, 128, (d_out, d_in), generator=g, dtype=torch.int8).to(DEV)
        xs, ws = torch.rand(T, generator=g).to(DEV), torch.rand(d_out, generator=g).to(DEV)
    else:
        xq, xs, _ = D.dora_quantize_rows_i8(x)
        wq, ws, _ = D.dora_quantize_rows_i8(W)
    k = dict(x_q=xq, x_scale=xs, W_q=wq, w_scale=ws, s=s)
    if r:
        k.update(x=x, A=((2 * torch.rand(r, d_in, generator=g) - 1) / d_in ** 0.5).to(BF).to(DEV),
                 B=(0.02 * rn(d_out, r)).to(BF).to(DEV))
    if mag:
        k.update(m=(1 + 0.1 * rn(d_out)).to(DEV), n=(1 + 0.1 * torch.rand(d_out, generator=g)).to(DEV))
    if bias:
        k.update(bias=(0.3 * rn(d_out)).to(BF).to(DEV))
    return k


def _check_linear(k, y, rows=slice(None), cols=slice(None)):
    f = lambda n, i=slice(None): None if k.get(n) is None else P.f64(k[n])[i]  # noqa: E731
    ref = oracle.linear_i8(f("x_q", rows), f("x_scale", rows), f("W_q", cols), f("w_scale", cols), f("x", rows),
                           f("A"), f("B", cols), f("m", cols), f("n", cols), k["s"], f("bias", cols))
    g = np.abs(f("m", cols) / f("n", cols)) if k.get("m") is not None else np.ones(ref.shape[1])
    base = np.abs(f("x_q", rows) @ f("W_q", cols).T) * np.outer(f("x_scale", rows), f("w_scale", cols))
    low = low_err = 0.0
    if k.get("A") is not None:
        s, x, A, B = abs(k["s"]), np.abs(f("x", rows)), np.abs(f("A")), np.abs(f("B", cols))
        Pm = s * np.abs(f("x", rows) @ f("A").T)          # |P|
        p_err = x.shape[1] * E * s * (x @ A.T) + U * Pm   # its fp32 sum, then bf16
        low = Pm @ B.T
        low_err = p_err @ B.T * (1 + U) + A.shape[0] * E * low
    b = 0.0 if k.get("bias") is None else np.abs(f("bias", cols))[None, :]
    tol = g * (low_err + 8 * E * (base + low)) + 8 * E * b
    _assert_within(np.asarray(P.f64(y))[rows][:, cols], ref, tol + U * (np.abs(ref) + tol), "y")


LINEAR = [(1, 16, 8, 8), (1, 8192, 264, 384), (2, 144, 136, 0), (7, 1040, 1000, 48), (16, 528, 520, 64),
          (17, 4112, 256, 16), (33, 2048, 4096, 384), (64, 272, 392, 72), (65, 512, 128, 8), (128, 1024, 2056, 0),
          (129, 400, 264, 40), (200, 2064, 1000, 128), (256, 256, 2048, 64), (300, 640, 512, 384), (513, 1024, 776, 8),
          (1030, 528, 264, 24),
          (5, 16, 24, 512), (300, 32, 264, 1000),  # more rank than input columns
          (2560, 64, 3840, 8),                     # several waves of 128-wide tiles
          (2500, 64, 5000, 24)]                    # several waves of 256-wide ones


@pytest.mark.parametrize("T, d_in, d_out, r", LINEAR)
@pytest.mark.parametrize("bias, mag", [(True, True), (False, False)])
def test_linear_i8(T, d_in, d_out, r, bias, mag):
    k = _module(T, d_in, d_out, r, bias=bias, mag=mag)
    y = D.dora_linear_i8_fwd(**k)
    y2 = D.dora_linear_i8_fwd(**k)
    torch.cuda.synchronize()
    assert D.dora_device_status() == D.DORA_OK
    assert torch.equal(y, y2)
    _check_linear(k, y)


@pytest.mark.parametrize("T, d_in, d_out, r", [(1, 528, 264, 8), (19, 2064, 136, 0), (140, 4096, 264, 16), (520, 656, 520, 8)])
@pytest.mark.parametrize("s", [-1.75, 0.0])
def test_linear_i8_all_codes_and_scales(T, d_in, d_out, r, s):
    # every code from -128 to 127, negative and zero s
    k = _module(T, d_in, d_out, r, s=s, full=True)
    y = D.dora_linear_i8_fwd(**k)
    torch.cuda.synchronize()
    _check_linear(k, y)


@pytest.mark.parametrize("T", [1, 40, 300])
def test_linear_i8_reaches_the_end_of_int32(T):
    # 131056 products of two lowest codes: 2^14 * 131056 = 2^31 - 2^18
    d_in = 131056
    k = dict(x_q=torch.full((T, d_in), -128, dtype=torch.int8, device=DEV), x_scale=torch.ones(T, device=DEV),
             W_q=torch.full((8, d_in), -128, dtype=torch.int8, device=DEV), w_scale=torch.ones(8, device=DEV))
    k["W_q"][1] = 127
    y = D.dora_linear_i8_fwd(**k)
    torch.cuda.synchronize()
    want = torch.full((T, 8), float(2 ** 14 * d_in), device=DEV)
    want[:, 1] = float(-128 * 127 * d_in)
    assert torch.equal(y, want.to(BF))


def test_linear_i8_zero_scales_and_nan_rows():
    k = _module(5, 256, 264, 16, bias=True)
    k["x_scale"] = k["x_scale"].clone()
    k["x_scale"][1] = 0.0
    k["x_scale"][3] = float("nan")
    y = D.dora_linear_i8_fwd(**k)
    torch.cuda.synchronize()
    assert torch.isnan(y[3]).all() and torch.isfinite(y[[0, 1, 2, 4]]).all()


def test_linear_i8_no_tokens_no_channels_and_a_rank_of_zero():
    k = _module(0, 64, 256, 0)
    assert D.dora_linear_i8_fwd(**k).shape == (0, 256)
    k = _module(3, 64, 8, 0, bias=False, mag=False)
    k.update(W_q=k["W_q"][:0].contiguous(), w_scale=k["w_scale"][:0].contiguous())
    assert D.dora_linear_i8_fwd(**k).shape == (3, 0)
    k = _module(3, 64, 16, 0)
    y = D.dora_linear_i8_fwd(**k)
    empty = dict(x=torch.zeros(3, 64, dtype=BF, device=DEV), A=torch.zeros(0, 64, dtype=BF, device=DEV),
                 B=torch.zeros(16, 0, dtype=BF, device=DEV))
    assert torch.equal(D.dora_linear_i8_fwd(**{**k, **empty}), y)


@pytest.mark.parametrize("T", [1, 33, 300])
def test_linear_i8_writes_only_its_rows_and_allocates_nothing(T):
    k = _module(T, 512, 520, 64)
    d_out = 520
    buf = torch.full((T + 2, d_out), 7.0, dtype=BF, device=DEV)
    y = buf[1:1 + T]
    ws = torch.empty(D.dora_linear_i8_fwd_workspace_size(T, 64) + 256, dtype=torch.uint8, device=DEV).fill_(123)
    work = ws[: D.dora_linear_i8_fwd_workspace_size(T, 64)]
    ref = D.dora_linear_i8_fwd(**k)
    torch.cuda.synchronize()
    free0, _ = torch.cuda.mem_get_info()
    D.dora_linear_i8_fwd(**k, y=y, workspace=work)
    torch.cuda.synchronize()
    assert torch.cuda.mem_get_info()[0] == free0
    assert torch.equal(y, ref) and (buf[0] == 7).all() and (buf[-1] == 7).all()
    assert (ws[work.numel():] == 123).all()
    with pytest.raises(RuntimeError):
        D.dora_linear_i8_fwd(**k, workspace=work[:16])


def test_serving_chain_captured_and_replayed():
    # norm -> gate-like projection -> quantised rows -> projection back, as a layer runs it
    T, d, f, r = 3, 512, 1048, 32
    up, down = _module(T, d, f, r, seed=31), _module(T, 1056, d, r, seed=32)
    h0 = _rows(T, d, BF, 33)
    stream = h0.clone()
    x = _rows(T, d, BF, 34)
    w = (1 + 0.1 * torch.randn(d, generator=_gen(35))).to(BF).to(DEV)
    pad = torch.zeros(T, 1056, dtype=BF, device=DEV)
    out = torch.empty(T, d, dtype=BF, device=DEV)
    bufs = dict(q=torch.empty(T, d, dtype=torch.int8, device=DEV), scale=torch.empty(T, device=DEV),
                y=torch.empty(T, d, dtype=BF, device=DEV))
    mid = torch.empty(T, f, dtype=BF, device=DEV)
    q2, s2 = torch.empty(T, 1056, dtype=torch.int8, device=DEV), torch.empty(T, device=DEV)
    ws1 = torch.empty(D.dora_linear_i8_fwd_workspace_size(T, r), dtype=torch.uint8, device=DEV)
    ws2 = torch.empty_like(ws1)

    def layer():
        D.dora_rms_norm_i8(x, w, residual=stream, h=stream, **bufs)
        D.dora_linear_i8_fwd(**{**up, "x_q": bufs["q"], "x_scale": bufs["scale"], "x": bufs["y"]}, y=mid, workspace=ws1)
        pad[:, :f].copy_(mid)
        D.dora_quantize_rows_i8(pad, q=q2, scale=s2)
        D.dora_linear_i8_fwd(**{**down, "x_q": q2, "x_scale": s2, "x": pad}, y=out, workspace=ws2)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer()
    for seed in (36, 37):
        stream.copy_(_rows(T, d, BF, seed))
        x.copy_(_rows(T, d, BF, seed + 10))
        keep = stream.clone()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (stream, mid, out)]
        stream.copy_(keep)
        layer()
        torch.cuda.synchronize()
        for a, b in zip(got, (stream, mid, out)):
            assert torch.equal(a, b)
        _check_linear({**up, "x_q": bufs["q"], "x_scale": bufs["scale"], "x": bufs["y"]}, mid)
        _check_linear({**down, "x_q": q2, "x_scale": s2, "x": pad}, out)
        codes, sc, _ = _norm_reference((x.float() + keep.float()).to(BF), w, 1e-6, BF)
        assert np.array_equal(bufs["q"].cpu().numpy(), codes)
    assert D.dora_device_status() == D.DORA_OK


def test_two_streams_at_once():
    a, b = _module(4, 2048, 1024, 64, seed=41), _module(300, 1024, 776, 16, seed=42)
    ra, rb = D.dora_linear_i8_fwd(**a), D.dora_linear_i8_fwd(**b)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = []
    for _ in range(4):
        for st, k, ref in zip(streams, (a, b), (ra, rb)):
            with torch.cuda.stream(st):
                outs.append((D.dora_linear_i8_fwd(**k), ref))
    torch.cuda.synchronize()
    assert all(torch.equal(y, ref) for y, ref in outs)
    assert D.dora_device_status() == D.DORA_OK


def test_linear_i8_headline_sampled():
    # 8192 tokens through the 8192 x 8192 module at rank 384
    k = _module(8192, 8192, 8192, 384, seed=51)
    y = D.dora_linear_i8_fwd(**k)
    torch.cuda.synchronize()
    assert D.dora_device_status() == D.DORA_OK
    _check_linear(k, y, rows=np.array([0, 127, 128, 255, 256, 4099, 8191]), cols=np.array([0, 127, 128, 300, 8191]))


def test_a_given_stream_owns_what_the_call_makes():
    # memory freed behind long work on the current stream must not become the
    # output of a call on another one, nor that call's workspace go back early
    k = _module(40, 2048, 1024, 64, seed=61)
    ref = D.dora_linear_i8_fwd(**k)
    x = _rows(40, 2048, BF, 62)
    q0, s0, _ = D.dora_quantize_rows_i8(x)
    v0 = D.dora_dequantize_i8(q0, s0)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    busy = torch.randn(4096, 4096, device=DEV)
    for _ in range(5):
        for n in (ref.numel(), q0.numel() // 2, 40 * 64, 256):
            t = torch.zeros(n, dtype=BF, device=DEV)
            for _ in range(4):
                busy = busy @ busy * 1e-3
            t.add_(busy.flatten()[: n].to(BF))  # late on the current stream
            del t
        y = D.dora_linear_i8_fwd(**k, stream=side)
        q, sc, _ = D.dora_quantize_rows_i8(x, stream=side)
        v = D.dora_dequantize_i8(q, sc, stream=side)
        side.synchronize()
        torch.cuda.synchronize()
        assert torch.equal(y, ref) and torch.equal(q, q0) and torch.equal(sc, s0) and torch.equal(v, v0)


def test_linear_i8_of_millions_of_tokens():
    # more token tiles than one grid dimension but the first holds
    T = 8_400_003
    k = _module(T, 16, 8, 8, seed=63)
    y = D.dora_linear_i8_fwd(**k)
    torch.cuda.synchronize()
    assert D.dora_device_status() == D.DORA_OK
    rows = np.array([0, 1, 127, 255, 4_000_000, 8_388_607, 8_388_608, T - 1])
    small = {n: (k[n] if n not in ("x_q", "x_scale", "x") else k[n][torch.as_tensor(rows, device=DEV)]) for n in k}
    _check_linear(small, y[torch.as_tensor(rows, device=DEV)])


@pytest.mark.parametrize("r", [0, 64])
def test_captured_behind_anything_and_before_anything(r):
    # the calls start under the launch before them: that launch may be nothing
    # (the graph's first node), a copy, a memset, another library's kernel, the
    # join of two streams, or a long kernel whose output the call reads
    T, d = 96, 1024
    k = _module(T, d, 520, r, seed=71)
    w = torch.ones(d, dtype=BF, device=DEV)
    src, x, res = _rows(T, d, BF, 72), _rows(T, d, BF, 73), _rows(T, d, BF, 74)
    q, sc, y = torch.empty(T, d, dtype=torch.int8, device=DEV), torch.empty(T, device=DEV), torch.empty_like(x)
    out, val = torch.empty(T, 520, dtype=BF, device=DEV), torch.empty_like(x)
    ws = torch.empty(max(256, D.dora_linear_i8_fwd_workspace_size(T, r)), dtype=torch.uint8, device=DEV)
    late = torch.randn(2048, 2048, device=DEV)
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    lin = {**k, "x_q": q, "x_scale": sc, **({"x": y} if r else {})}

    def chain(where):
        main = torch.cuda.current_stream()
        if where == "copy":
            x.copy_(src)
        elif where == "memset":
            res.zero_()
        elif where == "kernel":
            torch.mul(src, 0.5, out=x)
        elif where == "join":
            for st, (dst, f) in zip(side, ((x, 2.0), (res, 0.25))):
                st.wait_stream(main)
                with torch.cuda.stream(st):
                    torch.mul(src, f, out=dst)
            for st in side:
                main.wait_stream(st)
        elif where == "late":
            m = late
            for _ in range(6):
                m = (m @ late) * 1e-2
            x.copy_(src + m[:T, :d].to(BF) * 0)
        D.dora_rms_norm_i8(x, w, residual=res, h=res, q=q, scale=sc, y=y)
        D.dora_linear_i8_fwd(**lin, y=out, workspace=ws)
        D.dora_dequantize_i8(q, sc, out=val)
        if where != "first":
            torch.add(val, y, out=x)  # overwrites what the chain has read
            D.dora_quantize_rows_i8(x, q=q, scale=sc)
            D.dora_linear_i8_fwd(**lin, y=out, workspace=ws)

    for where in ("first", "copy", "memset", "kernel", "join", "late"):
        chain(where)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            chain(where)
        for _ in range(3):
            res.copy_(_rows(T, d, BF, 75))
            x.copy_(_rows(T, d, BF, 76))
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            got = [t.clone() for t in (res, x, q, sc, y, out, val)]
            res.copy_(_rows(T, d, BF, 75))
            x.copy_(_rows(T, d, BF, 76))
            chain(where)
            torch.cuda.synchronize()
            for a, b in zip(got, (res, x, q, sc, y, out, val)):
                assert torch.equal(a, b), where
        _check_linear(lin, out)
    assert D.dora_device_status() == D.DORA_OK


def test_back_to_back_calls_see_each_other_s_results():
    # dependent launches in one stream, outputs overwritten while the next call waits
    T, d = 2048, 2048
    x = _rows(T, d, BF, 81)
    acc = torch.zeros_like(x)
    ref = torch.zeros_like(x)
    for i in range(6):
        q, sc, h = D.dora_quantize_rows_i8(x, residual=acc, h=acc)
        v = D.dora_dequantize_i8(q, sc)
        acc.sub_(v)  # what the codes lost
    torch.cuda.synchronize()
    for i in range(6):
        ref = (x.float() + ref.float()).to(BF)
        codes, sc64 = oracle.encode(P.f64(ref))
        val = (torch.from_numpy(codes).float() * torch.from_numpy(sc64.astype(np.float32))).to(BF).to(DEV)
        ref = ref - val
    assert torch.equal(acc, ref)


def test_offsets_past_32_bits():
    # rows and products with more than 2^31 elements: the last ones against fp64
    T, d = 262160, 8192
    x = torch.zeros(T, d, dtype=BF, device=DEV)
    x[-3:] = _rows(3, d, BF, 91)
    w = torch.ones(d, dtype=BF, device=DEV)
    q, sc, _, y = D.dora_rms_norm_i8(x, w, 1e-5, want_y=True)
    torch.cuda.synchronize()
    # three rows by themselves would take more threads a row and add the squares in
    # another order, so the norm's factor is held to fp64, not to a small call's bits:
    # d non-negative terms in fp32 add at most d E to the sum, half of that to its
    # root, and the mean, eps, root, reciprocal and product 5 E (as test_rms_norm)
    codes, ref_sc, v = _norm_reference(x[-3:], w, 1e-5, BF)
    rel = (d / 2 + 5) * E
    assert np.array_equal(q[-3:].cpu().numpy(), codes)
    _assert_within(sc[-3:], ref_sc[:, 0], rel * ref_sc[:, 0], "scale")
    _assert_within(y[-3:], v, (rel + E + U) * np.abs(v) * (1 + U), "y")
    assert not q[:5].any() and not sc[:5].any()
    del x, q, y
    k = _module(70001, 16, 32768, 8, seed=92)
    y = D.dora_linear_i8_fwd(**k)
    torch.cuda.synchronize()
    rows = torch.tensor([0, 65535, 65536, 70000], device=DEV)
    part = {n: (v[rows] if n in ("x_q", "x_scale", "x") else v) for n, v in k.items()}
    _check_linear(part, y[rows], cols=np.array([0, 127, 128, 20000, 32767]))
    assert D.dora_device_status() == D.DORA_OK


@pytest.mark.parametrize("rows, cols, dtype", [(300, 4099, F32), (3, 33001, F32), (7, 129, F32), (2, 40000, F32),
                                               (3, 40000, BF), (400, 2048, BF), (2, 20008, BF)],
                         ids=lambda v: str(v).replace("torch.", ""))
@pytest.mark.parametrize("where", ["x", "residual", "both"])
@pytest.mark.parametrize("norm", [False, True])
def test_rows_in_place_in_every_layout(rows, cols, dtype, where, norm):
    # h over x, over residual, and over one tensor that is both: in registers, in
    # two passes, by vectors and by single values, at row bases off 128 bytes
    x = _rows(rows, cols, dtype, 101)
    res = x if where == "both" else _rows(rows, cols, dtype, 102)
    w = (1 + 0.2 * torch.randn(cols, generator=_gen(103))).to(dtype).to(DEV)

    def call(a, b, h):
        if norm:
            return D.dora_rms_norm_i8(a, w, residual=b, h=h, want_y=True)
        return D.dora_quantize_rows_i8(a, residual=b, h=h)

    ref = call(x, res, None)
    want_h = (x.float() + res.float()).to(dtype)
    a = x.clone()
    b = a if where == "both" else res.clone()
    got = call(a, b, b if where == "residual" else a)
    torch.cuda.synchronize()
    assert torch.equal(ref[2], want_h)
    assert all(torch.equal(p, q) for p, q in zip(ref, got))
    v = P.f64(want_h)
    if norm:
        v = v * P.f64(w) if dtype == BF else (want_h.cpu().numpy() * w.cpu().numpy()).astype(np.float64)
    assert np.array_equal(got[0].cpu().numpy(), oracle.encode(v)[0])


@pytest.mark.parametrize("dtype, cols", [(BF, 264), (F32, 1024), (F32, 4099), (BF, 40000), (F32, 33001)])
@pytest.mark.parametrize("eps", [0.0, 1e-45, 1e-30])
def test_rms_norm_of_rows_near_zero(dtype, cols, eps):
    # the factor 1 / sqrt(mean + eps) where the squares leave fp32's normal range:
    # a zero row gives zeros, a row whose mean square is too small for fp32 gives
    # NaN and not infinities, and the smallest that is not keeps its values
    x = torch.zeros(6, cols)
    x[1] = 2.0 ** -80 * (1 + torch.arange(cols) % 3)  # squares below the smallest subnormal
    x[2] = 2.0 ** -73                                  # squares of one subnormal step's size
    x[3] = 2.0 ** -62 * (1 + torch.arange(cols) % 5)   # mean square above 2^-124
    x[4] = torch.randn(cols, generator=_gen(111))
    x[5, 0] = 2.0 ** -20                               # one value in a row of zeros
    x = x.to(dtype).to(DEV)
    w = (1 + 0.2 * torch.rand(cols, generator=_gen(112))).to(dtype).to(DEV)
    eps32 = float(np.float32(eps))
    q, scale, _, y = D.dora_rms_norm_i8(x, w, eps, want_y=True)
    v = D.dora_dequantize_i8(q, scale, dtype=F32)
    torch.cuda.synchronize()
    assert scale[0] == 0 and not y[0].any() and not v[0].any()
    with np.errstate(divide="ignore", invalid="ignore"):  # the zero row's own factor
        codes, sc, want = _norm_reference(x, w, eps32, dtype)
    kept = [3, 4, 5] if eps < 1e-40 else [1, 2, 3, 4, 5]
    for i in (1, 2):
        if i not in kept:
            assert torch.isnan(scale[i]) and torch.isnan(y[i]).all() and torch.isnan(v[i]).all()
    rel = (cols / 2 + 6) * E  # as above; each square's own rounding may be 2^-150, 2^-24 of 2^-126
    assert np.array_equal(q[kept].cpu().numpy(), codes[kept])
    _assert_within(scale[kept], sc[kept, 0], rel * sc[kept, 0], "scale")
    _assert_within(y[kept], want[kept], (rel + E + (U if dtype == BF else 0)) * np.abs(want[kept]) * (1 + U), "y")


@pytest.mark.parametrize("d_in, d_out", [(528, 264), (4112, 1000)])
@pytest.mark.parametrize("bias, mag", [(True, True), (False, False)])
def test_without_an_adapter_a_token_does_not_depend_on_its_batch(d_in, d_out, bias, mag):
    # every token tile of the slices, and the pair product on both sides of their
    # border: the int32 sums are exact and the epilogues the same operations
    k = _module(300, d_in, d_out, 0, bias=bias, mag=mag, seed=121)
    y = D.dora_linear_i8_fwd(**k)
    for T in (1, 3, 16, 17, 32, 33, 64, 65, 127, 128, 129, 256, 257):
        part = {**k, "x_q": k["x_q"][:T], "x_scale": k["x_scale"][:T]}
        assert torch.equal(D.dora_linear_i8_fwd(**part), y[:T]), T
    torch.cuda.synchronize()
    assert D.dora_device_status() == D.DORA_OK
    _check_linear(k, y)


@pytest.mark.parametrize("T", [2, 40, 200])
def test_serving_a_module_with_the_norm_of_its_codes(T):
    # the weight's codes, n from the weight that they stand for, a norm's codes, the product
    d_in, d_out, r, s = 1024, 520, 32, 0.5
    g = _gen(131)
    rn = lambda *k: torch.randn(*k, generator=g)  # noqa: E731
    W = (0.02 * rn(d_out, d_in)).to(BF).to(DEV)
    A = ((2 * torch.rand(r, d_in, generator=g) - 1) / d_in ** 0.5).to(BF).to(DEV)
    B = (0.05 * rn(d_out, r)).to(BF).to(DEV)
    m = (0.6 + 0.1 * torch.rand(d_out, generator=g)).to(DEV)
    W_q, w_scale, _ = D.dora_quantize_rows_i8(W)
    n = D.dora_factored_norm(D.dora_dequantize_i8(W_q, w_scale), A, B, s)
    x = _rows(T, d_in, BF, 132)
    q, scale, _, y = D.dora_rms_norm_i8(x, torch.ones(d_in, dtype=BF, device=DEV), 1e-6, want_y=True)
    k = dict(x_q=q, x_scale=scale, W_q=W_q, w_scale=w_scale, x=y, A=A, B=B, m=m, n=n, s=s)
    out = D.dora_linear_i8_fwd(**k)
    torch.cuda.synchronize()
    _check_linear(k, out)
    # n is the norm of codes * scale + s B A: its rounding to bf16 moves the weight by
    # U of itself at most, and with it the norm; the norm's own tolerance comes on top
    kept = oracle.decode(W_q.cpu().numpy(), w_scale.cpu().numpy())
    exact = oracle.row_norm(kept, P.f64(A), P.f64(B), s)
    slack = U * np.linalg.norm(kept, axis=1) + P.NORM_RTOL_BF16 * exact
    assert np.all(np.abs(P.f64(n) - exact) <= slack)


@pytest.mark.parametrize("captured", [False, True])
def test_buffers_rewritten_under_dependent_launches(captured):
    # every call starts under the one before it, which has just rewritten what it
    # reads: the same small buffers over and over, so that the lines which an SM
    # read last time would still be in its cache
    T, d, N, turns = 160, 512, 136, 60
    xs = [_rows(T, d, BF, 140 + i) * 2.0 ** (i % 5) for i in range(4)]
    w = torch.ones(d, dtype=BF, device=DEV)
    k = _module(T, d, N, 0, seed=139)
    x, q, sc = torch.empty_like(xs[0]), torch.empty(T, d, dtype=torch.int8, device=DEV), torch.empty(T, device=DEV)
    val, out = torch.empty_like(x), torch.empty(T, N, dtype=BF, device=DEV)
    small = torch.empty(64, N, dtype=BF, device=DEV)
    want = []
    for t in xs:
        a, b, _, _ = D.dora_rms_norm_i8(t, w)
        torch.cuda.synchronize()
        lin = {**k, "x_q": a, "x_scale": b}
        part = {**k, "x_q": a[:64].clone(), "x_scale": b[:64].clone()}
        want.append([D.dora_dequantize_i8(a, b), D.dora_linear_i8_fwd(**lin), D.dora_linear_i8_fwd(**part)])
        torch.cuda.synchronize()
    got = [[torch.empty_like(t) for t in want[0]] for _ in range(turns)]

    def chain():
        for i in range(turns):
            x.copy_(xs[i % 4])
            D.dora_rms_norm_i8(x, w, q=q, scale=sc)
            D.dora_dequantize_i8(q, sc, out=val)
            D.dora_linear_i8_fwd(**{**k, "x_q": q, "x_scale": sc}, y=out)
            D.dora_linear_i8_fwd(**{**k, "x_q": q[:64], "x_scale": sc[:64]}, y=small)
            D.dora_quantize_rows_i8(val, q=q, scale=sc)  # rewritten at once
            for dst, src in zip(got[i], (val, out, small)):
                dst.copy_(src)

    if captured:
        chain()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            chain()
        for row in got:
            for t in row:
                t.fill_(7.0)
        graph.replay()
    else:
        chain()
    torch.cuda.synchronize()
    assert D.dora_device_status() == D.DORA_OK
    for i, row in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(row, want[i % 4])), i
