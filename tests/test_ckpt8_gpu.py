"""The 8-bit checkpoints: the forwards that write them, the backward that reads
them, against fp64.

y is the plain forward's, bit for bit.  z is an fp32 value formed by rounded
operations that the test repeats, so the codes are compared for equality; the
fused forward's z comes from a tensor-core sum, so its codes may differ from
the exact z's by that sum's error, and its kept values are held to half a scale
plus that error.  Tolerances with u = 2^-8, e = 2^-24 relative to the value:
bf16 outputs u, fp32 sums of k terms k e of the terms' magnitudes.
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


def _acts(T, d, dtype, bias, seed=1):
    g = _gen(seed)
    rn = lambda *k: torch.randn(*k, generator=g)  # noqa: E731
    base, lora = (rn(T, d) * torch.exp(0.5 * rn(d))).to(dtype), (0.2 * rn(T, d)).to(dtype)
    m = (1.5 + 0.1 * rn(d)).float()
    n = (m / (1 + 5e-4 * rn(d))).float()
    b = (0.3 * rn(d)).to(dtype) if bias else None
    dy = rn(T, d).to(dtype)
    return tuple(None if t is None else t.to(DEV) for t in (base, lora, m, n, b, dy))


def _z32(base, lora, bias, s):
    """z by rounded fp32 operations."""
    base, lora = base.float().cpu().numpy(), lora.float().cpu().numpy()
    inner = base if bias is None else base - bias.float().cpu().numpy()
    return inner + np.float32(s) * lora


SHAPES = [(1, 8, BF), (3, 120, BF), (5, 128, BF), (1, 8192, BF), (70, 1000, BF), (257, 2056, BF), (1100, 264, BF),
          (2, 27648, BF), (1, 1, F32), (4, 127, F32), (33, 129, F32), (257, 4099, F32), (40, 1000, F32),
          (1030, 260, F32), (1, 4096, F32)]
IDS = lambda v: str(v).replace("torch.", "")  # noqa: E731


@pytest.mark.parametrize("T, d, dtype", SHAPES, ids=IDS)
@pytest.mark.parametrize("bias, s", [(False, 0.5), (True, -0.35)])
def test_forward(T, d, dtype, bias, s):
    base, lora, m, n, b, _ = _acts(T, d, dtype, bias)
    y, z8, zs = D.dora_compose_fwd_ckpt8(base, lora, m, n, s, bias=b)
    plain = D.dora_compose_fwd(base, lora, m, n, s, bias=b)
    torch.cuda.synchronize()
    assert torch.equal(y, plain)
    codes, sc = oracle.encode(_z32(base, lora, b, s), 128)
    assert np.array_equal(z8.cpu().numpy(), codes)
    assert np.array_equal(zs.cpu().numpy(), sc.astype(np.float32))


@pytest.mark.parametrize("T, d, dtype", SHAPES, ids=IDS)
@pytest.mark.parametrize("s", [0.5, -1.7])
def test_backward(T, d, dtype, s):
    base, lora, m, n, _, dy = _acts(T, d, dtype, False, seed=2)
    _, z8, zs = D.dora_compose_fwd_ckpt8(base, lora, m, n, s)
    got = D.dora_compose_bwd_ckpt8(dy, z8, zs, m, n, s)
    again = D.dora_compose_bwd_ckpt8(dy, z8, zs, m, n, s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    z = oracle.decode(z8.cpu().numpy(), zs.cpu().numpy(), 128)
    rb, rl, rm = oracle.compose_backward_kept(P.f64(dy), z, P.f64(m), P.f64(n), np.float32(s))
    last = U if dtype == BF else E
    for g, r, name in ((got[0], rb, "d_base"), (got[1], rl, "d_lora")):
        assert np.all(np.abs(P.f64(g) - r) <= (last + 4 * E) * np.abs(r) * (1 + U)), name
    terms = np.sum(np.abs(P.f64(dy) * z), axis=0) / np.abs(P.f64(n))
    assert np.all(np.abs(P.f64(got[2]) - rm) <= (T + 4) * E * terms), "d_m"
    # and the checkpoint's own error: half a scale of each z at most
    exact = np.sum(P.f64(dy) * (P.f64(base) + s * P.f64(lora)), axis=0) / P.f64(n)
    half = np.sum(np.abs(P.f64(dy)) * 0.5 * zs.cpu().double().numpy()[:, np.arange(d) // 128], axis=0) / np.abs(P.f64(n))
    assert np.all(np.abs(P.f64(got[2]) - exact) <= half * (1 + 1e-5) + (T + 8) * E * terms), "d_m against plain z"


def test_backward_is_the_gradient_by_differences():
    # the forward is linear in base, lora and m: a difference quotient is exact up to fp64 rounding of the oracle
    T, d, s = 6, 40, 0.75
    base, lora, m, n, _, dy = _acts(T, d, F32, False, seed=3)
    _, z8, zs = D.dora_compose_fwd_ckpt8(base, lora, m, n, s)
    d_base, d_lora, d_m = D.dora_compose_bwd_ckpt8(dy, z8, zs, m, n, s)
    torch.cuda.synchronize()
    f = lambda b, l, mm: float(np.sum(P.f64(dy) * oracle.compose_forward(b, l, mm, P.f64(n), s)))  # noqa: E731
    b64, l64, m64 = P.f64(base), P.f64(lora), P.f64(m)
    half = 0.5 * zs.cpu().double().numpy()[:, np.arange(d) // 128]
    for i in (0, 17, 39):
        step = np.zeros_like(m64)
        step[i] = 1e-3
        diff = (f(b64, l64, m64 + step) - f(b64, l64, m64 - step)) / 2e-3
        slack = float(np.sum(np.abs(P.f64(dy))[:, i] * half[:, i]) / n[i].item())
        assert abs(diff - d_m[i].item()) <= slack * 1.001 + 1e-6 * abs(diff) + 1e-9
        bump = np.zeros_like(b64)
        bump[2, i] = 1e-3
        for which, grad in ((0, d_base), (1, d_lora)):
            hi, lo = ((b64 + bump, l64, m64), (b64 - bump, l64, m64)) if which == 0 else \
                ((b64, l64 + bump, m64), (b64, l64 - bump, m64))
            diff = (f(*hi) - f(*lo)) / 2e-3
            assert abs(diff - grad[2, i].item()) <= 1e-6 * abs(diff) + 1e-9


@pytest.mark.parametrize("dtype, d", [(BF, 264), (F32, 264), (F32, 263)])
def test_blocks_at_the_format_s_edges(dtype, d):
    base, lora, m, n, _, dy = _acts(9, d, dtype, False, seed=4)
    base[0, :128] = 0
    lora[0, :128] = 0
    base[1, 130] = float("inf")
    base[2, 7] = float("nan")
    base[3, :] = 1e-31
    lora[3, :] = 0
    y, z8, zs = D.dora_compose_fwd_ckpt8(base, lora, m, n, 0.5)
    d_base, d_lora, d_m = D.dora_compose_bwd_ckpt8(dy, z8, zs, m, n, 0.5)
    torch.cuda.synchronize()
    codes, sc = oracle.encode(_z32(base, lora, None, 0.5), 128)
    assert np.array_equal(z8.cpu().numpy(), codes)
    assert np.array_equal(zs.cpu().numpy(), sc.astype(np.float32), equal_nan=True)
    assert torch.isnan(d_m[:256]).all() and torch.isfinite(d_m[256:]).all()
    assert torch.isfinite(d_base).all() and torch.isfinite(d_lora).all()


@pytest.mark.parametrize("d", [0, 8, 264])
def test_no_tokens(d):
    e = torch.empty(0, d, dtype=BF, device=DEV)
    v = torch.ones(d, device=DEV)
    y, z8, zs = D.dora_compose_fwd_ckpt8(e, e, v, v, 0.5)
    assert y.shape == z8.shape == (0, d) and zs.shape == (0, -(-d // 128))
    d_m = torch.full((d,), 3.0, device=DEV)
    D.dora_compose_bwd_ckpt8(e, z8, zs, v, v, 0.5, d_m=d_m)
    torch.cuda.synchronize()
    assert not d_m.any()


def test_outputs_stay_inside_their_rows():
    T, d = 37, 520
    base, lora, m, n, _, dy = _acts(T, d, BF, False, seed=5)
    z8 = torch.full((T + 2, d), 77, dtype=torch.int8, device=DEV)
    zs = torch.full((T + 2, 5), 7.0, device=DEV)
    outs = [torch.full((T + 2, d), 7.0, dtype=BF, device=DEV) for _ in range(3)]
    D.dora_compose_fwd_ckpt8(base, lora, m, n, 0.5, y=outs[0][1:-1], z8=z8[1:-1], z_scale=zs[1:-1])
    D.dora_compose_bwd_ckpt8(dy, z8[1:-1], zs[1:-1], m, n, 0.5, d_base=outs[1][1:-1], d_lora=outs[2][1:-1])
    torch.cuda.synchronize()
    for t, v in ((z8, 77), (zs, 7.0), *((o, 7.0) for o in outs)):
        assert (t[0] == v).all() and (t[-1] == v).all()


FUSED = [(128, 64, 256, 16), (300, 520, 1000, 48), (257, 1024, 512, 384), (64, 4104, 264, 512), (1, 64, 8, 8),
         (130, 136, 2056, 40), (96, 128, 120, 0), (200, 256, 128, 8), (520, 264, 392, 24),
         (140, 8, 136, 256),                        # more rank than input columns
         (2560, 64, 3840, 8), (2500, 64, 5000, 24)]  # several waves of 128- and of 256-wide tiles


@pytest.mark.parametrize("T, d_in, d_out, r", FUSED)
@pytest.mark.parametrize("bias", [False, True])
def test_fused_forward(T, d_in, d_out, r, bias):
    g, s = _gen(6), 0.5
    rn = lambda *k: torch.randn(*k, generator=g)  # noqa: E731
    x, W = rn(T, d_in).to(BF).to(DEV), (0.02 * rn(d_out, d_in)).to(BF).to(DEV)
    A = ((2 * torch.rand(r, d_in, generator=g) - 1) / d_in ** 0.5).to(BF).to(DEV)
    B = (0.02 * rn(d_out, r)).to(BF).to(DEV)
    m = (1 + 0.1 * rn(d_out)).to(DEV)
    n = (1 + 0.1 * torch.rand(d_out, generator=g)).to(DEV)
    b = (0.3 * rn(d_out)).to(BF).to(DEV) if bias else None
    y, z8, zs = D.dora_fused_linear_fwd_ckpt8(x, W, A, B, m, n, s, bias=b)
    plain = D.dora_fused_linear_fwd(x, W, A, B, m, n, s, bias=b)
    torch.cuda.synchronize()
    assert D.dora_device_status() == D.DORA_OK
    P.assert_act_close(y, P.f64(plain), "y against the plain fused forward")
    X, Wd, Ad, Bd = P.f64(x), P.f64(W), P.f64(A), P.f64(B)
    Pm = s * (X @ Ad.T)
    z = X @ Wd.T + Pm @ Bd.T
    low = np.abs(Pm) @ np.abs(Bd).T
    terms = np.abs(X) @ np.abs(Wd).T + low
    # P in two bf16 halves: an fp32 sum, then twice a rounding to 8 bits
    p_err = d_in * E * s * (np.abs(X) @ np.abs(Ad).T) + U * U * np.abs(Pm)
    err = p_err @ np.abs(Bd).T + (d_in + r) * E * terms
    zv = oracle.decode(z8.cpu().numpy(), zs.cpu().numpy(), 128)
    half = 0.5 * zs.cpu().double().numpy()[:, np.arange(d_out) // 128]
    assert np.all(np.abs(zv - z) <= err + half * (1 + 4 * E) + 4 * E * np.abs(z)), "kept z"
    top = np.stack([np.max(np.abs(z[:, j:j + 128]), axis=1) for j in range(0, d_out, 128)], axis=1)
    top_err = np.stack([np.max(err[:, j:j + 128], axis=1) for j in range(0, d_out, 128)], axis=1)
    assert np.all(np.abs(127 * zs.cpu().double().numpy() - top) <= top_err + 4 * E * top), "scales"
    gm = P.f64(m) / P.f64(n)
    ref = gm * z + (0.0 if b is None else P.f64(b))
    tol = np.abs(gm) * (err + 8 * E * np.abs(z)) + 8 * E * np.abs(ref)
    assert np.all(np.abs(P.f64(y) - ref) <= tol + U * (np.abs(ref) + tol)), "y"


def test_training_step_captured_and_replayed():
    # fused forward with the checkpoint, then the backward that reads it, as one graph
    T, d_in, d_out, r, s = 320, 256, 520, 16, 0.5
    g = _gen(7)
    x = torch.randn(T, d_in, generator=g).to(BF).to(DEV)
    W = (0.05 * torch.randn(d_out, d_in, generator=g)).to(BF).to(DEV)
    A = (0.05 * torch.randn(r, d_in, generator=g)).to(BF).to(DEV)
    B = (0.05 * torch.randn(d_out, r, generator=g)).to(BF).to(DEV)
    m = (1 + 0.1 * torch.rand(d_out, generator=g)).to(DEV)
    n = D.dora_factored_norm(W, A, B, s)
    dy = torch.randn(T, d_out, generator=g).to(BF).to(DEV)
    y, d_base, d_lora = (torch.empty(T, d_out, dtype=BF, device=DEV) for _ in range(3))
    z8, zs = torch.empty(T, d_out, dtype=torch.int8, device=DEV), torch.empty(T, 5, device=DEV)
    d_m = torch.empty(d_out, device=DEV)
    ws_f = torch.empty(D.dora_fused_linear_fwd_ckpt8_workspace_size(T, r), dtype=torch.uint8, device=DEV)
    ws_b = torch.empty(D.dora_compose_bwd_ckpt8_workspace_size(T, d_out), dtype=torch.uint8, device=DEV)

    def step():
        D.dora_fused_linear_fwd_ckpt8(x, W, A, B, m, n, s, y=y, z8=z8, z_scale=zs, workspace=ws_f)
        D.dora_compose_bwd_ckpt8(dy, z8, zs, m, n, s, d_base, d_lora, d_m, ws_b)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (8, 9):
        x.copy_(torch.randn(T, d_in, generator=_gen(seed)).to(BF))
        dy.copy_(torch.randn(T, d_out, generator=_gen(seed + 10)).to(BF))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (y, z8, zs, d_base, d_lora, d_m)]
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, (y, z8, zs, d_base, d_lora, d_m)))
        # d_m against the plain pair on the exact z: the checkpoint's half scales and P's rounding
        X = P.f64(x)
        Pm = s * (X @ P.f64(A).T)
        z = X @ P.f64(W).T + Pm @ P.f64(B).T
        err = U * U * np.abs(Pm) @ np.abs(P.f64(B)).T + 2 * (d_in + r) * E * (
            np.abs(X) @ np.abs(P.f64(W)).T + s * np.abs(X) @ np.abs(P.f64(A)).T @ np.abs(P.f64(B)).T)
        half = 0.5 * zs.cpu().double().numpy()[:, np.arange(d_out) // 128]
        exact = np.sum(P.f64(dy) * z, axis=0) / P.f64(n)
        slack = np.sum(np.abs(P.f64(dy)) * (half * 1.00001 + err + (T + 4) * E * np.abs(z)), axis=0) / P.f64(n)
        assert np.all(np.abs(P.f64(d_m) - exact) <= slack)
    assert D.dora_device_status() == D.DORA_OK


def test_offsets_past_32_bits():
    # 2^31 + elements of codes and activations: the last rows against fp64
    T, d = 262160, 8192
    base = torch.zeros(T, d, dtype=BF, device=DEV)
    lora = torch.zeros(T, d, dtype=BF, device=DEV)
    tail, tl, m, n, _, tdy = _acts(16, d, BF, False, seed=11)
    base[-16:], lora[-16:] = tail, tl
    y, z8, zs = D.dora_compose_fwd_ckpt8(base, lora, m, n, 0.5)
    codes, sc = oracle.encode(_z32(tail, tl, None, 0.5), 128)
    assert torch.equal(y[-16:], D.dora_compose_fwd(tail, tl, m, n, 0.5))
    del y, base
    assert np.array_equal(z8[-16:].cpu().numpy(), codes) and not z8[:16].any()
    assert np.array_equal(zs[-16:].cpu().numpy(), sc.astype(np.float32))
    lora[-16:] = tdy
    d_base, d_lora, d_m = D.dora_compose_bwd_ckpt8(lora, z8, zs, m, n, 0.5)
    small = D.dora_compose_bwd_ckpt8(tdy, z8[-16:], zs[-16:], m, n, 0.5)
    torch.cuda.synchronize()
    assert torch.equal(d_base[-16:], small[0]) and torch.equal(d_lora[-16:], small[1])
    terms = np.sum(np.abs(P.f64(tdy) * oracle.decode(codes, sc, 128)), axis=0) / P.f64(n)
    assert np.all(np.abs(P.f64(d_m) - P.f64(small[2])) <= 40 * E * terms)
    v = D.dora_dequantize_i8(z8, zs)
    torch.cuda.synchronize()
    assert torch.equal(v[-16:], D.dora_dequantize_i8(z8[-16:].clone(), zs[-16:].clone()))


def test_fused_scales_hold_fp32_over_a_long_k():
    # the scales of z at K = 8192: an fp32 sum of chunks of at most 1024 terms.
    # Within a chunk the tensor core's additions (of 16 products) drop bits, at
    # most 2^-23 of the running sum each: 64 of them
    T, K, N, r = 130, 8192, 384, 64
    g = _gen(12)
    x = torch.randn(T, K, generator=g).to(BF).to(DEV)
    W = (0.015 * torch.randn(N, K, generator=g)).to(BF).to(DEV)
    A = ((2 * torch.rand(r, K, generator=g) - 1) / K ** 0.5).to(BF).to(DEV)
    B = (0.02 * torch.randn(N, r, generator=g)).to(BF).to(DEV)
    one = torch.ones(N, device=DEV)
    _, _, zs = D.dora_fused_linear_fwd_ckpt8(x, W, A, B, one, one, 0.5)
    torch.cuda.synchronize()
    z = P.f64(x) @ P.f64(W).T + 0.5 * (P.f64(x) @ P.f64(A).T) @ P.f64(B).T
    top = np.stack([np.max(np.abs(z[:, j:j + 128]), axis=1) for j in range(0, N, 128)], axis=1)
    rel = np.linalg.norm(127 * zs.cpu().double().numpy() - top) / np.linalg.norm(top)
    assert rel <= 64 * 2.0 ** -23, rel


def test_a_given_stream_runs_the_training_pair():
    base, lora, m, n, _, dy = _acts(70, 1000, BF, False, seed=13)
    ref = D.dora_compose_fwd_ckpt8(base, lora, m, n, 0.5)
    back = D.dora_compose_bwd_ckpt8(dy, ref[1], ref[2], m, n, 0.5)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        got = D.dora_compose_fwd_ckpt8(base, lora, m, n, 0.5, stream=side)
        gb = D.dora_compose_bwd_ckpt8(dy, got[1], got[2], m, n, 0.5, stream=side)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((*got, *gb), (*ref, *back)))


def test_fused_offsets_past_32_bits():
    T, d_in, d_out, r = 70001, 16, 32768, 8
    g = _gen(14)
    x = torch.randn(T, d_in, generator=g).to(BF).to(DEV)
    W = (0.1 * torch.randn(d_out, d_in, generator=g)).to(BF).to(DEV)
    A = (0.1 * torch.randn(r, d_in, generator=g)).to(BF).to(DEV)
    B = (0.1 * torch.randn(d_out, r, generator=g)).to(BF).to(DEV)
    one = torch.ones(d_out, device=DEV)
    y, z8, zs = D.dora_fused_linear_fwd_ckpt8(x, W, A, B, one, one, 0.5)
    rows = torch.tensor([0, 65535, 65536, 70000], device=DEV)
    ys, z8s, zss = D.dora_fused_linear_fwd_ckpt8(x[rows], W, A, B, one, one, 0.5)
    torch.cuda.synchronize()
    assert D.dora_device_status() == D.DORA_OK
    # the small call sums P over another split of K, so its rounding may differ in the last bits
    z = P.f64(x[rows]) @ P.f64(W).T + 0.5 * (P.f64(x[rows]) @ P.f64(A).T) @ P.f64(B).T
    for yy, cc, ss in ((y[rows], z8[rows], zs[rows]), (ys, z8s, zss)):
        half = 0.5 * ss.cpu().double().numpy()[:, np.arange(d_out) // 128]
        assert np.all(np.abs(oracle.decode(cc.cpu().numpy(), ss.cpu().numpy(), 128) - z) <= half + 64 * E * (1 + np.abs(z)))
        assert np.all(np.abs(P.f64(yy) - z) <= U * np.abs(z) + 64 * E * (1 + np.abs(z)))


def test_fused_forward_over_millions_of_input_columns():
    # a K of 125,000 steps in 20,834 chunks: their product passes 32 bits.  Operands
    # of -1, 0 and 1 make every partial sum an integer below 2^24, exact in any
    # order and under any rounding, and P (below 2^16) exact in two bf16 halves
    T, K, N, r = 3, 16_000_000, 16, 8
    g = torch.Generator(device=DEV).manual_seed(15)
    tri = lambda *k: torch.randint(-1, 2, k, generator=g, device=DEV, dtype=torch.int8).to(BF)  # noqa: E731
    x, W, A, B = tri(T, K), tri(N, K), tri(r, K), tri(N, r)
    one = torch.ones(N, device=DEV)
    y, z8, zs = D.dora_fused_linear_fwd_ckpt8(x, W, A, B, one, one, 1.0)
    torch.cuda.synchronize()
    assert D.dora_device_status() == D.DORA_OK
    xd = x.double()
    Pm = torch.cat([xd @ A[j:j + 1].double().T for j in range(r)], dim=1)
    z = torch.cat([xd @ W[j:j + 1].double().T for j in range(N)], dim=1) + Pm @ B.double().T
    assert Pm.abs().max() < 2 ** 16 and z.abs().max() < 2 ** 24  # of the inputs, not of the kernel
    codes, sc = oracle.encode(P.f64(z), 128)
    assert np.array_equal(zs.cpu().numpy(), sc.astype(np.float32))
    assert np.array_equal(z8.cpu().numpy(), codes)
    assert torch.equal(y, z.to(BF))


def _scale_bias(T, K, N, r, adapter):
    """Mean relative error of the scales of z for positive operands: the tensor
    core's truncation always goes down, rounding to nearest goes both ways.  With
    ``adapter`` the base weight is zero and B picks one rank a channel, so z is P."""
    g = torch.Generator(device=DEV).manual_seed(16)
    x = torch.rand(T, K, generator=g, device=DEV).to(BF)
    one = torch.ones(N, device=DEV)
    if adapter:
        W = torch.zeros(N, K, dtype=BF, device=DEV)
        A = torch.rand(r, K, generator=g, device=DEV).to(BF)
        B = torch.zeros(N, r, dtype=BF, device=DEV)
        B[torch.arange(N), torch.arange(N) % r] = 1
        z = (x.double() @ A.double().T).repeat(1, -(-N // r))[:, :N]
    else:
        W = torch.rand(N, K, generator=g, device=DEV).to(BF)
        A, B = torch.zeros(r, K, dtype=BF, device=DEV), torch.zeros(N, r, dtype=BF, device=DEV)
        z = x.double() @ W.double().T
    _, _, zs = D.dora_fused_linear_fwd_ckpt8(x, W, A, B, one, one, 1.0)
    top = torch.stack([z[:, j:j + 128].abs().amax(dim=1) for j in range(0, N, 128)], dim=1)
    torch.cuda.synchronize()
    assert D.dora_device_status() == D.DORA_OK
    return ((127 * zs.double() - top) / top).mean().item()


# A chunk is at most 768 of K: 48 additions of 16 products, and addition i of a
# growing sum drops less than 2^-23 of i / 48 of it, 24.5 * 2^-23 in all.  The 11
# chunks of K = 8192 are added with rounding (each 2^-24 of what is there so far,
# 6 * 2^-24 in all), and the scale takes two more roundings.
CHUNK_BIAS = 24.5 * 2.0 ** -23 + 6 * E + 2 * E


def test_scales_of_a_long_k_are_not_low():
    # one sum over 4096 of K would be 5e-6 low, over all 8192 1e-5
    bias = _scale_bias(256, 8192, 384, 0, False)
    assert abs(bias) <= CHUNK_BIAS, bias


@pytest.mark.parametrize("T, N, r", [(512, 8192, 384),   # P beside the product, K in one piece
                                     (6400, 256, 384),   # many tokens, K in one piece
                                     (140, 384, 128),    # K in eighths
                                     (40, 264, 72), (20, 264, 8), (7, 128, 8)])  # narrower token tiles
def test_scales_of_an_adapter_s_long_k_are_not_low(T, N, r):
    # z is P alone.  Its low half rounds by at most 2^-16 of P either way: over the
    # T rows and r / 128 distinct stretches that leaves six times 2^-16 over the
    # root of their number
    bias = _scale_bias(T, 8192, N, r, True)
    assert abs(bias) <= CHUNK_BIAS + 2 * E + 6 * U * U / (T * max(1, r // 128)) ** 0.5, bias


@pytest.mark.parametrize("T, N", [(9, 264), (300, 264), (300, 1000)])
@pytest.mark.parametrize("bias", [False, True])
def test_fused_rows_that_are_zero_or_not_finite(T, N, bias):
    # positive weights, so that an infinite input makes every channel +inf and not a difference of infinities
    K, r = 136, 24
    g = _gen(17)
    rand = lambda *k: (0.1 + torch.rand(*k, generator=g)).to(BF).to(DEV)  # noqa: E731
    x, W, A, B = rand(T, K), rand(N, K), rand(r, K), rand(N, r)
    x[0] = 0
    x[1, 5] = float("inf")
    x[2, 100] = float("nan")
    x[3] = 2.0 ** -122            # a stretch below 2^-100
    x[4, 7] = -float("inf")
    # P rounds to infinity in bf16 alone: 255.75 / 256 of 2^128 (B takes it back)
    x[5] = 0
    x[5, 0], x[5, 1] = 255 * 2.0 ** 120, 2.0 ** 118
    A[:, 0], A[:, 1] = 1.0, 3.0
    W[:, 0], W[:, 1] = 2.0 ** -20, 2.0 ** -20
    B *= 2.0 ** -12
    m = (1 + 0.1 * torch.rand(N, generator=g)).to(DEV)
    b = rand(N) if bias else None
    y, z8, zs = D.dora_fused_linear_fwd_ckpt8(x, W, A, B, m, torch.ones(N, device=DEV), 1.0, bias=b)
    dy = rand(T, N)
    d_base, d_lora, d_m = D.dora_compose_bwd_ckpt8(dy, z8, zs, m, torch.ones(N, device=DEV), 1.0)
    torch.cuda.synchronize()
    assert D.dora_device_status() == D.DORA_OK
    assert torch.equal(y[0], torch.zeros(N, dtype=BF, device=DEV) if b is None else b)
    plain = D.dora_fused_linear_fwd(x, W, A, B, m, torch.ones(N, device=DEV), 1.0, bias=b)
    assert torch.equal(y[[1, 2, 4]].nan_to_num(7.0), plain[[1, 2, 4]].nan_to_num(7.0))
    assert not z8[[0, 3]].any() and not zs[[0, 3]].any()
    assert (y[1] == float("inf")).all() and torch.isnan(y[2]).all() and (y[4] == -float("inf")).all()
    assert torch.isnan(zs[[1, 2, 4]]).all() and not z8[[1, 2, 4]].any()
    rest = torch.tensor([i for i in range(T) if i not in (1, 2, 4)], device=DEV)
    z = P.f64(x[rest]) @ P.f64(W).T + (P.f64(x[rest]) @ P.f64(A).T) @ P.f64(B).T
    want = P.f64(m) * z + (0.0 if b is None else P.f64(b))
    # positive sums of K + r terms in fp32, P in two halves, one bf16 rounding
    rel = (2 * K + r + 16) * E + U * U
    assert np.all(np.abs(P.f64(y[rest]) - want) <= (rel + U) * np.abs(want) * (1 + U))
    assert torch.isfinite(zs[rest]).all() and torch.isnan(d_m).all()
    assert torch.isfinite(d_base).all() and torch.isfinite(d_lora).all()


def test_two_graphs_share_a_workspace():
    # two captured backwards of different shapes and one eager call take turns on one workspace
    shapes = [(700, 520, BF), (260, 1100, F32)]
    size = max(D.dora_compose_bwd_ckpt8_workspace_size(T, d) for T, d, _ in shapes)
    ws = torch.randint(0, 256, (size,), dtype=torch.uint8, device=DEV)
    runs = []
    for i, (T, d, dtype) in enumerate(shapes):
        base, lora, m, n, _, dy = _acts(T, d, dtype, False, seed=20 + i)
        _, z8, zs = D.dora_compose_fwd_ckpt8(base, lora, m, n, 0.5)
        ref = D.dora_compose_bwd_ckpt8(dy, z8, zs, m, n, 0.5)
        out = [torch.empty_like(t) for t in ref]
        call = lambda a=(dy, z8, zs, m, n, 0.5), o=out: D.dora_compose_bwd_ckpt8(*a, *o, workspace=ws)  # noqa: E731
        call()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        runs.append((graph, call, out, ref))
    for turn in range(6):
        for graph, call, out, ref in runs if turn % 2 else runs[::-1]:
            for t in out:
                t.fill_(7.0)
            call() if turn == 3 else graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, ref)), turn


@pytest.mark.parametrize("dtype, d", [(BF, 520), (F32, 263)])
def test_a_checkpoint_rewritten_under_dependent_launches(dtype, d):
    # forward and backward over the same small buffers, magnitudes changed in place between them
    T, turns = 200, 60
    sets = [_acts(T, d, dtype, False, seed=40 + i) for i in range(4)]
    fresh = []
    for base, lora, m, n, _, dy in sets:
        y, z8, zs = D.dora_compose_fwd_ckpt8(base, lora, m, n, 0.5)
        fresh.append((y, z8, zs, *D.dora_compose_bwd_ckpt8(dy, z8, zs, m, n, 0.5)))
        torch.cuda.synchronize()
    cur = [torch.empty_like(t) for t in (sets[0][0], sets[0][1], sets[0][2], sets[0][3], sets[0][5])]
    out = [torch.empty_like(t) for t in fresh[0]]
    ws = torch.empty(D.dora_compose_bwd_ckpt8_workspace_size(T, d), dtype=torch.uint8, device=DEV)
    got = [[torch.empty_like(t) for t in fresh[0]] for _ in range(turns)]
    for i in range(turns):
        base, lora, m, n, _, dy = sets[i % 4]
        for dst, src in zip(cur, (base, lora, m, n, dy)):
            dst.copy_(src)
        D.dora_compose_fwd_ckpt8(*cur[:4], 0.5, *out[:3])
        D.dora_compose_bwd_ckpt8(cur[4], out[1], out[2], cur[2], cur[3], 0.5, *out[3:], workspace=ws)
        for dst, src in zip(got[i], out):
            dst.copy_(src)
    torch.cuda.synchronize()
    for i, row in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(row, fresh[i % 4])), i
