"""The operators of w4a4_ops.h against their formulas in 64 bits: the 4-bit layer for single tokens, layer
normalisation, 8-bit checkpoints and the gated feed-forward block.

Tolerances are sums of first-order rounding bounds, with u = 2^-24 for fp32 steps and 2^-8 (8 significant
bits) for a rounding to bf16: a sum of n terms in any order is off by at most n u times the sum of its
terms' magnitudes, a rounding by its unit times the value. Codes, scales and what they stand for are
exact."""
import ctypes
import math

import numpy as np
import pytest
import torch

import w4a4_quantized_gemm_smooth_amd as w4

U32, U16 = 2.0 ** -24, 2.0 ** -8
gpu = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu(request):
    if request.node.get_closest_marker("gpu"):
        if not torch.cuda.is_available():
            pytest.skip("no GPU visible")
        print(f"[{request.node.name}]", flush=True)
    w4.lib()


def _rand(seed, shape, std=1.0, dtype=torch.bfloat16):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(dtype).cuda()


def _empty(nbytes):
    return torch.full((max(nbytes, 16),), 0xA5, dtype=torch.uint8, device="cuda")   # never zeros


def _wide(t, extra, fill):
    """t as a column slice of a matrix of `extra` more columns holding `fill`."""
    w = torch.full((t.shape[0], t.shape[1] + extra), fill, dtype=t.dtype, device=t.device)
    w[:, : t.shape[1]] = t
    return w[:, : t.shape[1]]


def _within(got, want, tol, what):
    d = (got.double() - want).abs()
    bad = ~(d <= tol)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} outside, worst {float((d / tol).nan_to_num(0).max()):.3g} "
                           f"times the bound, first at {torch.nonzero(bad)[0].tolist()}")


# ------------------------------------------------------------------------------------------ matvec
E2M1 = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64)


def _matvec_case(M, N, K, rank, fmt, bias, seed):
    g = torch.Generator().manual_seed(seed)
    c = dict(M=M, N=N, K=K, rank=rank, fmt=fmt)
    c["x"] = (torch.randn((M, K), generator=g) * torch.where(torch.rand(K, generator=g) < 0.02, 30.0, 1.0)).bfloat16().cuda()
    c["inv"] = (torch.rand(K, generator=g) + 0.5).cuda()
    c["codes"] = torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8).cuda()
    if fmt == "int4_g64":
        c["scales"] = (torch.rand((N, K // 64), generator=g) * 0.02).bfloat16().cuda()
    else:
        c["scales"] = torch.randint(115, 125, (N, K // 32), generator=g, dtype=torch.uint8).cuda()
    rp, n_pad = -(-rank // 16) * 16, -(-N // 256) * 256
    c["l1t"] = c["l2t"] = None
    if rank:
        c["l1t"] = torch.zeros((rp, K), dtype=torch.bfloat16, device="cuda")
        c["l2t"] = torch.zeros((n_pad, rp), dtype=torch.bfloat16, device="cuda")
        c["l1t"][:rank] = (torch.randn((rank, K), generator=g) * 0.05).bfloat16()
        c["l2t"][:N, :rank] = (torch.randn((N, rank), generator=g) * 0.05).bfloat16()
    c["bias"] = torch.randn(N, generator=g).bfloat16().cuda() if bias else None
    sz = w4.matvec_sizes(M, N, K, rank, fmt)
    c["wv"], c["ws"] = _empty(sz["wv"]), _empty(sz["ws"])
    w4.matvec_weights(c["codes"], c["scales"], N, K, fmt, c["wv"])
    return c


def _matvec(c, x=None, y=None, ws=None, stream=None):
    x = c["x"] if x is None else x
    y = torch.full((x.shape[0], c["N"]), -7.0, dtype=torch.bfloat16, device="cuda") if y is None else y
    w4.matvec(x, c["inv"], c["l1t"], c["wv"], c["l2t"], c["bias"], y, c["N"], c["K"], c["rank"], c["fmt"],
              c["ws"] if ws is None else ws, stream)
    return y


def _matvec_weights64(c):
    q, s = c["codes"].cpu(), c["scales"].cpu()
    q = torch.stack((q & 15, q >> 4), -1).view(c["N"], -1)
    if c["fmt"] == "int4_g64":
        return ((q ^ 8).double() - 8) * s.double().repeat_interleave(64, 1)
    return E2M1[q.long()] * torch.ldexp(torch.ones((), dtype=torch.float64), s.int() - 127).repeat_interleave(32, 1)


def _matvec_reference(c, x=None):
    """The formula, and the bound: x^ carries 2^-16 from its two bf16 parts (each 2^-8 of its own) and 2^-24 from its product; a
    group's sum starts from 24 times its activations' sum and adds codes of up to 31 (INT4)."""
    x = (c["x"] if x is None else x).cpu().double() * c["inv"].cpu().double()
    w = _matvec_weights64(c)
    y, mag, K = x @ w.T, x.abs() @ w.abs().T, c["K"]
    tol = (2 * 2.0 ** -16 + (K + 64) * U32) * mag
    if c["fmt"] == "int4_g64":
        s = c["scales"].cpu().double().repeat_interleave(64, 1)
        tol = tol + 2 * (64 * U32) * (55 * x.abs()) @ s.T
    if c["rank"]:
        l1, l2 = c["l1t"].cpu().double(), c["l2t"].cpu().double()[: c["N"]]
        y = y + (x @ l1.T) @ l2.T
        tol = tol + (4 * 2.0 ** -16 + (K + c["rank"] + 64) * U32) * (x.abs() @ l1.abs().T) @ l2.abs().T
    if c["bias"] is not None:
        y = y + c["bias"].cpu().double()
    return y, tol + 2 * U16 * y.abs() + 2 * U32 * mag


@gpu
@pytest.mark.parametrize("fmt", ["int4_g64", "mxfp4_b32"])
@pytest.mark.parametrize("M,N,K,rank,bias", [
    (1, 1, 64, 0, False), (1, 17, 64, 1, True), (2, 128, 128, 16, False), (7, 129, 192, 20, True), (8, 300, 1088, 48, True),
    (9, 64, 320, 0, True), (16, 255, 2048, 128, True), (13, 640, 8256, 33, False), (1, 9216, 1024, 32, False),
    (16, 20000, 64, 16, True), (5, 40, 12288, 20, True),
    (16, 100, 960, 33, True), (12, 77, 512, 64, False), (3, 150, 1024, 128, True), (8, 1000, 1024, 17, True), (10, 500, 448, 0, False),
    (8, 333, 2048, 32, True), (1, 700, 1984, 20, False), (5, 260, 1152, 48, True)])
def test_matvec(fmt, M, N, K, rank, bias):
    c = _matvec_case(M, N, K, rank, fmt, bias, seed=M + N + K)
    y, tol = _matvec_reference(c)
    _within(_matvec(c).cpu(), y, tol, "y")


@gpu
@pytest.mark.parametrize("fmt", ["int4_g64", "mxfp4_b32"])
def test_matvec_of_every_code(fmt):
    """Unit vectors select single weights: every code of every position of a pair of groups comes back
    exactly (the activations and scales are powers of two)."""
    K, N = 128, 16
    c = _matvec_case(16, N, K, 0, fmt, False, seed=3)
    c["inv"].fill_(1.0)
    q = (torch.arange(N)[:, None] + torch.arange(K)[None, :]) % 16
    c["codes"].copy_((q[:, 0::2] | q[:, 1::2] << 4).to(torch.uint8))
    if fmt == "int4_g64":
        c["scales"].copy_(torch.tensor([[0.5, 2.0]]).expand(N, 2))
    else:
        c["scales"].copy_(torch.tensor([[126, 128, 120, 130]], dtype=torch.uint8).expand(N, 4))
    w4.matvec_weights(c["codes"], c["scales"], N, K, fmt, c["wv"])
    w = _matvec_weights64(c)
    for k0 in range(0, K, 16):
        x = torch.zeros((16, K), dtype=torch.bfloat16, device="cuda")
        x[torch.arange(16), k0 + torch.arange(16)] = 1.0
        assert torch.equal(_matvec(c, x).cpu().double(), w[:, k0: k0 + 16].T), f"codes at k {k0}"


@gpu
def test_matvec_strides_rows_and_workspace():
    """Strided x and y, the same rows in any batch, and a workspace full of NaN."""
    c = _matvec_case(12, 200, 448, 20, "int4_g64", True, seed=8)
    y = _matvec(c)
    wide = torch.full((12, 333), 5.0, dtype=torch.bfloat16, device="cuda")
    c["ws"].fill_(0xFF)
    _matvec(c, _wide(c["x"], 72, float("nan")), wide[:, 7:207])
    assert torch.equal(wide[:, 7:207], y) and (wide[:, :7] == 5).all() and (wide[:, 207:] == 5).all()
    ref, tol = _matvec_reference(c)
    for m in (0, 5, 11):
        _within(_matvec(c, c["x"][m: m + 1]).cpu(), ref[m: m + 1], tol[m: m + 1], f"row {m} alone")


@gpu
def test_matvec_non_finite_rows_stay_apart():
    for M in (6, 14):
        c = _matvec_case(M, 100, 256, 16, "int4_g64", False, seed=M)
        y = _matvec(c)
        x = c["x"].clone()
        x[1, 3], x[4, 200] = float("inf"), float("nan")
        z = _matvec(c, x)
        keep = [m for m in range(M) if m not in (1, 4)]
        assert torch.equal(z[keep], y[keep])
        assert not torch.isfinite(z[[1, 4]]).any()


@gpu
def test_matvec_of_a_prepared_layer():
    """The layer object's own form for single tokens: the weight-only product of what it prepared."""
    rng = np.random.default_rng(5)
    w_bits = (torch.from_numpy(rng.standard_normal((384, 256)).astype(np.float32)) * 0.02).bfloat16().view(torch.int16).numpy().view(np.uint16)
    inv = rng.uniform(0.5, 2.0, 256).astype(np.float32)
    lam = (1.0 / inv).astype(np.float32)
    x = _rand(6, (3, 256))
    for fmt in ("int4_g64", "mxfp4_b32"):
        prep = w4.prepare_weights(w_bits, lam, 24, fmt)
        layer = w4.W4A4Linear(prep, inv)
        y = layer.tokens(x)
        c = dict(M=3, N=384, K=256, rank=24, fmt=fmt, x=x, inv=torch.from_numpy(inv), bias=None,
                 codes=torch.from_numpy(w4.codes_to_canonical(prep["wq"], 384, 256, fmt)),
                 l1t=torch.from_numpy(prep["l1t"].view(np.int16)).view(torch.bfloat16).view(32, 256),
                 l2t=torch.from_numpy(prep["l2t"].view(np.int16)).view(torch.bfloat16).view(512, 32))
        s = torch.from_numpy(w4.scales_to_canonical(prep["wscale"], 384, 256, fmt).view(np.int16 if fmt == "int4_g64" else np.uint8))
        c["scales"] = s.view(torch.bfloat16) if fmt == "int4_g64" else s
        ref, tol = _matvec_reference(c)
        _within(y.cpu(), ref, tol, fmt)
        w = torch.from_numpy(w_bits.view(np.int16).copy()).view(torch.bfloat16).double()
        full = x.cpu().double() @ w.T
        assert (y.cpu().double() - full).norm() < 0.2 * full.norm()   # 4-bit weights: near the layer itself
    with pytest.raises(ValueError):
        layer.tokens(_rand(1, (17, 256)))


# -------------------------------------------------------------------------------------------- norm
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _norm_case(M, K, dt, pt, seed, offset=0.0):
    c = dict(M=M, K=K, x=(_rand(seed, (M, K), 1.0, torch.float32) * torch.linspace(0.1, 3, M, device="cuda")[:, None] + offset).to(DT[dt]),
             dy=_rand(seed + 1, (M, K), 0.1, DT[dt]))
    c["gamma"] = None if pt is None else (_rand(seed + 2, (K,), 0.3, torch.float32) + 1).to(DT[pt])
    c["beta"] = None if pt is None else _rand(seed + 3, (K,), 0.3, DT[pt])
    return c


def _norm_forward(c, x=None, eps=1e-5):
    x = c["x"] if x is None else x
    M, K = x.shape
    y = torch.full((M, K), -7.0, dtype=x.dtype, device="cuda")
    mean, rstd = torch.full((M,), -7.0, device="cuda"), torch.full((M,), -7.0, device="cuda")
    w4.layer_norm(x, c["gamma"], c["beta"], eps, y, mean, rstd)
    return y, mean, rstd


def _norm_backward(c, mean, rstd, dy=None, x=None):
    x, dy = c["x"] if x is None else x, c["dy"] if dy is None else dy
    M, K = x.shape
    dx = torch.full((M, K), -7.0, dtype=x.dtype, device="cuda")
    grads = c["gamma"] is not None
    dg, db = (torch.full((K,), -7.0, device="cuda") for _ in range(2)) if grads else (None, None)
    ws = _empty(w4.layer_norm_backward_bytes(M, K)).fill_(0xFF) if grads else None
    w4.layer_norm_backward(dy, x, c["gamma"], mean, rstd, dx, dg, db, ws)
    return dx, dg, db


def _check_norm_forward(c, y, mean, rstd, eps=1e-5):
    x, K = c["x"].cpu().double(), c["K"]
    g = 1.0 if c["gamma"] is None else c["gamma"].cpu().double()
    b = 0.0 if c["beta"] is None else c["beta"].cpu().double()
    mu = x.mean(1, keepdim=True)
    var = (x - mu).square().mean(1, keepdim=True)
    rs = 1 / torch.sqrt(var + eps)
    n = 160   # additions on the longest path of a row's sum, with a reserve
    emu = n * U32 * x.abs().mean(1, keepdim=True) + 2 * U32 * mu.abs()
    # the squares are taken around the computed mean: its error enters by its own square
    ers = rs * (n * U32 + 0.5 * emu.square() * rs.square()) + 4 * U32 * rs
    _within(mean.cpu()[:, None], mu, emu + 1e-30, "mean")
    _within(rstd.cpu()[:, None], rs, ers, "rstd")
    h = (x - mu) * rs
    tol = (emu * rs + (x - mu).abs() * ers + 4 * U32 * h.abs() + 2 * U32 * x.abs() * rs) * abs(g) + 2 * U32 * (abs(h * g) + abs(b))
    want = h * g + b
    if c["x"].dtype == torch.bfloat16:
        tol = tol + U16 * (want.abs() + tol)
    _within(y.cpu(), want, tol + 1e-30, "y")


def _check_norm_backward(c, mean, rstd, dx, dg, db):
    x, dy, K, M = c["x"].cpu().double(), c["dy"].cpu().double(), c["K"], c["M"]
    g = 1.0 if c["gamma"] is None else c["gamma"].cpu().double()
    mu, rs = mean.cpu().double()[:, None], rstd.cpu().double()[:, None]
    h, d = (x - mu) * rs, dy * g
    eh = 3 * U32 * (h.abs() + x.abs() * rs)
    m1, m2 = d.mean(1, keepdim=True), (d * h).mean(1, keepdim=True)
    n = 160
    e1 = n * U32 * d.abs().mean(1, keepdim=True)
    e2 = n * U32 * (d * h).abs().mean(1, keepdim=True) + (d.abs() * eh).mean(1, keepdim=True)
    want = rs * (d - m1 - h * m2)
    tol = rs * (4 * U32 * (d.abs() + m1.abs() + (h * m2).abs()) + e1 + h.abs() * e2 + eh * m2.abs())
    if c["x"].dtype == torch.bfloat16:
        tol = tol + U16 * (want.abs() + tol)
    _within(dx.cpu(), want, tol + 1e-30, "dx")
    if dg is not None:
        _within(dg.cpu(), (dy * h).sum(0), (M + 8) * U32 * (dy * h).abs().sum(0) + (dy.abs() * eh).sum(0) + 1e-30, "dgamma")
        _within(db.cpu(), dy.sum(0), (M + 8) * U32 * dy.abs().sum(0) + 1e-30, "dbeta")


@gpu
@pytest.mark.parametrize("dt,pt", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("f32", "bf16"), ("bf16", None), ("f32", None)])
@pytest.mark.parametrize("M,K", [(1, 1), (3, 2), (5, 7), (2, 64), (33, 255), (17, 512), (5, 513), (70, 1531), (9, 2048), (300, 2056),
                                 (6, 4097), (3, 8192), (5, 12289), (2, 16384), (4, 16391), (1030, 24)])
def test_layer_norm(dt, pt, M, K):
    c = _norm_case(M, K, dt, pt, seed=M * 31 + K)
    y, mean, rstd = _norm_forward(c)
    _check_norm_forward(c, y, mean, rstd)
    _check_norm_backward(c, mean, rstd, *_norm_backward(c, mean, rstd))


@gpu
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_layer_norm_large_offset(dt):
    """A common offset far above the spread: the squares around the mean keep their digits."""
    c = _norm_case(40, 1000, dt, "f32", seed=4, offset=300.0)
    y, mean, rstd = _norm_forward(c)
    _check_norm_forward(c, y, mean, rstd)


@gpu
def test_layer_norm_constant_rows_and_eps():
    """Rows without spread: y = beta and rstd = 1/sqrt(eps); with eps = 0, no finite value."""
    c = _norm_case(4, 100, "f32", "f32", seed=2)
    c["x"].fill_(2.5)
    y, mean, rstd = _norm_forward(c)
    assert torch.equal(y, c["beta"].expand(4, 100)) and (mean == 2.5).all()
    assert (rstd.double() * math.sqrt(1e-5) - 1).abs().max() < 1e-6
    y, _, rstd = _norm_forward(c, eps=0.0)
    assert torch.isinf(rstd).all() and torch.isnan(y).all()


@gpu
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("K", [96, 1000, 5000, 17001])
def test_layer_norm_strides_and_repeat(dt, K):
    """Row strides that break every alignment give the contiguous result, nothing is written beside the
    rows, and a second call the same bits."""
    c = _norm_case(9, K, dt, "bf16", seed=K)
    y, mean, rstd = _norm_forward(c)
    dx, dg, db = _norm_backward(c, mean, rstd)
    for extra in (1, 3):
        xs, dys = _wide(c["x"], extra, float("nan")), _wide(c["dy"], extra, float("nan"))
        y2, mean2, rstd2 = _norm_forward(c, xs)
        assert torch.equal(y, y2) and torch.equal(mean, mean2) and torch.equal(rstd, rstd2)
        out = torch.full((9, K + extra), 3.0, dtype=DT[dt], device="cuda")
        w4.layer_norm(xs, c["gamma"], c["beta"], 1e-5, out[:, extra:], mean2, rstd2)
        assert torch.equal(out[:, extra:], y) and (out[:, :extra] == 3).all()
        for a, b in zip((dx, dg, db), _norm_backward(c, mean, rstd, dys, xs)):
            assert torch.equal(a, b)


@gpu
def test_layer_norm_one_gradient_alone():
    c = _norm_case(50, 300, "bf16", "bf16", seed=12)
    _, mean, rstd = _norm_forward(c)
    dx, dg, db = _norm_backward(c, mean, rstd)
    ws = _empty(w4.layer_norm_backward_bytes(50, 300))
    dx2, g2 = torch.empty_like(dx), torch.empty_like(dg)
    w4.layer_norm_backward(c["dy"], c["x"], c["gamma"], mean, rstd, dx2, g2, None, ws)
    assert torch.equal(g2, dg) and torch.equal(dx2, dx)
    w4.layer_norm_backward(c["dy"], c["x"], c["gamma"], mean, rstd, dx2, None, g2, ws)
    assert torch.equal(g2, db)
    w4.layer_norm_backward(c["dy"], c["x"], c["gamma"], mean, rstd, dx2, None, None, None)
    assert torch.equal(dx2, dx)


@gpu
def test_layer_norm_non_finite_rows_stay_apart():
    c = _norm_case(20, 700, "bf16", "bf16", seed=1)
    y, mean, rstd = _norm_forward(c)
    dx, _, _ = _norm_backward(c, mean, rstd)
    x = c["x"].clone()
    x[3, 5], x[7, 600] = float("nan"), float("-inf")
    keep = [m for m in range(20) if m not in (3, 7)]
    y2, mean2, rstd2 = _norm_forward(c, x)
    assert torch.equal(y2[keep], y[keep]) and torch.isnan(y2[[3, 7]]).all()
    dx2, dg, db = _norm_backward(c, mean2, rstd2, x=x)
    assert torch.equal(dx2[keep], dx[keep]) and torch.isnan(dx2[[3, 7]]).all() and torch.isnan(dg).all()
    assert torch.isfinite(db).all()


# -------------------------------------------------------------------------------------- checkpoint
def _pack64(x):
    """Codes [blocks, K, 32], scale bytes [blocks, K] and values, by the definition."""
    M, K = x.shape
    nb = -(-M // 32)
    p = torch.zeros((nb * 32, K), dtype=torch.float64)
    p[:M] = x.cpu().double()
    p = p.view(nb, 32, K)
    bad = ~torch.isfinite(p).all(1)
    a = torch.where(bad, torch.zeros(()).double(), p.abs().amax(1))
    e = torch.full_like(a, -127)
    for _ in range(260):   # smallest e with 127 2^e >= a
        e = torch.where(127 * torch.pow(2.0, e) < a, e + 1, e)
    step = torch.pow(2.0, e)[:, None]
    most = torch.where(e == 122, 63.0, 127.0)[:, None]   # 64 2^122 would be no bf16 number
    q = torch.where(bad[:, None], torch.zeros(()).double(), torch.minimum(torch.maximum(torch.round(p / step), -most), most))
    back = torch.where(bad[:, None], torch.full((), float("nan")).double(), q * step)
    byte = torch.where(bad, torch.full((), 255.0).double(), e + 127)
    return q.transpose(1, 2).to(torch.int8), byte.to(torch.uint8), back.reshape(nb * 32, K)[:M]


def _pack(x):
    sz = w4.checkpoint_sizes(*x.shape)
    nb = -(-x.shape[0] // 32)
    codes = torch.full((nb, x.shape[1], 32), 99, dtype=torch.int8, device="cuda")
    scales = torch.full((nb, x.shape[1]), 99, dtype=torch.uint8, device="cuda")
    assert codes.numel() == sz["codes"] and scales.numel() == sz["scales"]
    w4.checkpoint_pack(x, codes, scales)
    return codes, scales


def _same(a, b):
    return torch.equal(torch.isnan(a), torch.isnan(b)) and torch.equal(a.nan_to_num(0), b.nan_to_num(0))


@gpu
@pytest.mark.parametrize("M,K", [(1, 8), (31, 16), (32, 1024), (33, 1032), (100, 3000), (65, 264)])
def test_checkpoint_codes(M, K):
    x = _rand(M + K, (M, K)) * torch.exp2(torch.randint(-20, 20, (K,)).float()).bfloat16().cuda()
    x[:, K // 2] = 0.0
    q, e, back = _pack64(x)
    for xin in (x, _wide(x, 8, float("nan"))):
        codes, scales = _pack(xin)
        assert torch.equal(codes.cpu(), q) and torch.equal(scales.cpu(), e)
        out = torch.full((M, K + 8), 4.0, dtype=torch.bfloat16, device="cuda")
        w4.checkpoint_unpack(codes, scales, out[:, :K])
        assert torch.equal(out[:, :K].cpu().double(), back) and (out[:, K:] == 4).all()
    assert (back - x.cpu().double()).abs().max() <= (torch.pow(2.0, e.double() - 128)).max()


@gpu
def test_checkpoint_of_every_bf16_value():
    """Every bf16 pattern as a block's largest magnitude, with smaller ones beside it (ties, subnormals,
    the largest number), and blocks with Inf or NaN."""
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16)
    x = torch.zeros((32, 65536), dtype=torch.bfloat16)
    top = bits.view(torch.bfloat16)
    for r in range(32):
        x[r] = (top.double() * ((32 - r) / 32.0)).bfloat16() if r else top
    q, e, back = _pack64(x)
    codes, scales = _pack(x.cuda())
    assert torch.equal(scales.cpu(), e) and torch.equal(codes.cpu(), q)
    out = torch.empty((32, 65536), dtype=torch.bfloat16, device="cuda")
    w4.checkpoint_unpack(codes, scales, out)
    assert _same(out.cpu().double(), back)


@gpu
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("M,N,K", [(1, 8, 8), (31, 8, 64), (33, 264, 40), (64, 256, 256), (97, 40, 520), (300, 520, 264), (2049, 16, 1000),
                                   (1500, 128, 136), (1000, 136, 8), (5000, 32, 72), (2100, 64, 520),
                                   (700, 72, 200), (1000, 200, 72), (300, 2600, 2000)])
def test_checkpoint_weight_grad(M, N, K, out):
    x, dy = _rand(M, (M, K)), _rand(N, (M, N), 0.1)
    codes, scales = _pack(x)
    back = _pack64(x)[2]
    want, mag = dy.cpu().double().T @ back, dy.cpu().double().abs().T @ back.abs()
    tol = (M + 16) * U32 * mag
    if out == "bf16":
        tol = tol + U16 * (want.abs() + tol)
    for dyin in (dy, _wide(dy, 8, float("nan"))):
        dw = torch.full((N, K), -7.0, dtype=DT[out], device="cuda")
        ws = _empty(w4.checkpoint_weight_grad_bytes(M, N, K)).fill_(0xFF)
        w4.checkpoint_weight_grad(dyin, codes, scales, K, dw, ws)
        _within(dw.cpu(), want, tol + 1e-30, "dw")


@gpu
def test_checkpoint_weight_grad_is_exact_in_whole_numbers():
    """Small whole numbers: every product and sum is exact, so any misplaced element shows."""
    g = torch.Generator().manual_seed(1)
    for M, N, K in ((70, 24, 88), (515, 264, 520), (1025, 32, 256)):
        x = torch.randint(-127, 128, (M, K), generator=g).double()
        dy = torch.randint(-3, 4, (M, N), generator=g).double()
        x[0::32] = 127.0   # every block's scale is 1
        codes, scales = _pack(x.bfloat16().cuda())
        dw = torch.empty((N, K), device="cuda")
        w4.checkpoint_weight_grad(dy.bfloat16().cuda(), codes, scales, K, dw, _empty(w4.checkpoint_weight_grad_bytes(M, N, K)))
        assert torch.equal(dw.cpu().double(), dy.T @ x), (M, N, K)


@gpu
def test_checkpoint_weight_grad_marks_bad_blocks():
    x, dy = _rand(3, (96, 64)), _rand(4, (96, 32))
    x[40, 7], x[3, 20] = float("inf"), float("nan")
    codes, scales = _pack(x)
    dw = torch.empty((32, 64), device="cuda")
    w4.checkpoint_weight_grad(dy, codes, scales, 64, dw, _empty(w4.checkpoint_weight_grad_bytes(96, 32, 64)))
    bad = torch.zeros(64, dtype=torch.bool, device="cuda")
    bad[[7, 20]] = True
    assert torch.isnan(dw[:, bad]).all() and torch.isfinite(dw[:, ~bad]).all()


# ------------------------------------------------------------------------------------------- gated
def _act64(g, act):
    if act == "silu":
        p = torch.special.expit(g)
        return g * p, p + g * p * torch.special.expit(-g)
    p = torch.special.ndtr(g)
    return g * p, p + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)


def _gated64(x, wg, wu, act):
    """H and its bound from fp32 sums of K products; |act'| <= 1.13, |act''| <= 0.8."""
    K = x.shape[1]
    g, u = x @ wg.T, x @ wu.T
    eg, eu = ((K + 8) * U32 * (x.abs() @ w.abs().T) for w in (wg, wu))
    a, s = _act64(g, act)
    # the activation itself in fp32: a few units of it, and of its exponent's argument
    ea = 1.13 * eg + (16 + 2 * g.abs().clamp(max=100)) * U32 * (a.abs() + g.abs().clamp(max=1))
    es = 0.8 * eg + (32 + 4 * g.abs().clamp(max=100)) * U32
    return dict(g=g, u=u, a=a, s=s, eg=eg, eu=eu, ea=ea, es=es, h=a * u, eh=ea * u.abs() + a.abs() * eu + 2 * U32 * (a * u).abs())


def _gated_inputs(M, K, F, seed, scale=1.0):
    return _rand(seed, (M, K)), _rand(seed + 1, (F, K), scale / math.sqrt(K)), _rand(seed + 2, (F, K), 1 / math.sqrt(K)), _rand(seed + 3, (M, F), 0.1)


def _gated_backward(x, wg, wu, dh, act):
    M, K, F = *x.shape, wg.shape[0]
    dx = torch.full((M, K), -7.0, dtype=torch.bfloat16, device="cuda")
    dwg, dwu = (torch.full((F, K), -7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    w4.gated_backward(dh, x, wg, wu, act, dx, dwg, dwu, _empty(w4.gated_backward_bytes(M, K, F)).fill_(0xFF))
    return dx, dwg, dwu


GATED = [(1, 8, 8), (1, 512, 200), (2, 72, 40), (16, 1032, 264), (17, 40, 136), (33, 200, 72), (48, 136, 520), (49, 64, 64), (255, 64, 128), (300, 520, 392), (64, 2048, 1000),
         (513, 96, 24), (2000, 256, 256), (1100, 2056, 1032), (1500, 1000, 2600)]


@gpu
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("M,K,F", GATED)
def test_gated_forward(M, K, F, act):
    x, wg, wu, _ = _gated_inputs(M, K, F, M + K + F, scale=2.0)
    r = _gated64(x.cpu().double(), wg.cpu().double(), wu.cpu().double(), act)
    h = torch.full((M, F), -7.0, dtype=torch.bfloat16, device="cuda")
    ws = _empty(w4.gated_forward_bytes(M, K, F)).fill_(0xFF)
    w4.gated_forward(x, wg, wu, act, h, ws)
    _within(h.cpu(), r["h"], r["eh"] + U16 * (r["h"].abs() + r["eh"]) + 1e-30, "h")
    wide = torch.full((M, F + 16), 3.0, dtype=torch.bfloat16, device="cuda")
    w4.gated_forward(_wide(x, 8, float("nan")), _wide(wg, 24, float("nan")), _wide(wu, 24, float("nan")), act, wide[:, 8: 8 + F], ws)
    assert torch.equal(wide[:, 8: 8 + F], h) and (wide[:, :8] == 3).all() and (wide[:, 8 + F:] == 3).all()


@gpu
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("M,K,F", GATED)
def test_gated_backward(M, K, F, act):
    x, wg, wu, dh = _gated_inputs(M, K, F, M + K + F, scale=2.0)
    x6, wg6, wu6, dh6 = (t.cpu().double() for t in (x, wg, wu, dh))
    r = _gated64(x6, wg6, wu6, act)
    dg, du = dh6 * r["u"] * r["s"], dh6 * r["a"]
    edg = dh6.abs() * (r["eu"] * r["s"].abs() + r["u"].abs() * r["es"]) + 4 * U32 * dg.abs()
    edu = dh6.abs() * r["ea"] + 2 * U32 * du.abs()
    edg, edu = edg + U16 * (dg.abs() + edg), edu + U16 * (du.abs() + edu)   # dG, dU are operands in bf16
    want = dict(dx=dg @ wg6 + du @ wu6, dwg=dg.T @ x6, dwu=du.T @ x6)
    tol = dict(dx=edg @ wg6.abs() + edu @ wu6.abs() + (2 * F + 16) * U32 * (dg.abs() @ wg6.abs() + du.abs() @ wu6.abs()),
               dwg=edg.T @ x6.abs() + (M + 16) * U32 * (dg.abs().T @ x6.abs()),
               dwu=edu.T @ x6.abs() + (M + 16) * U32 * (du.abs().T @ x6.abs()))
    got = dict(zip(("dx", "dwg", "dwu"), _gated_backward(x, wg, wu, dh, act)))
    for k in want:
        _within(got[k].cpu(), want[k], tol[k] + U16 * (want[k].abs() + tol[k]) + 1e-30, k)
        # and far inside the worst case as a whole: two roundings to bf16 (2^-8 each at most)
        assert (got[k].cpu().double() - want[k]).norm() <= 2 * U16 * want[k].norm() + 1e-30, k
    strided = _gated_backward(_wide(x, 8, float("nan")), _wide(wg, 16, float("nan")), _wide(wu, 16, float("nan")),
                              _wide(dh, 8, float("nan")), act)
    for k, s in zip(("dx", "dwg", "dwu"), strided):
        assert torch.equal(s, got[k]), k


@gpu
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("M,K,F", [(227, 2240, 2312), (40, 4096, 136), (1000, 4096, 264), (33, 1024, 8)])
def test_gated_long_contraction_in_parts(M, K, F, act):
    """Few blocks of outputs over a long contraction: its parts are added before the activation."""
    assert w4.gated_forward_bytes(M, K, F) >= 2 * 2 * M * F * 4
    test_gated_forward(M, K, F, act)
    test_gated_backward(M, K, F, act)


@gpu
def test_gated_saturated_and_non_finite():
    """Gates far outside the exponential's range, and rows with Inf or NaN that stay apart."""
    for M in (9, 40):
        x, wg, wu, dh = _gated_inputs(M, 64, 48, M, scale=2000.0)
        for act in ("silu", "gelu"):
            h = torch.empty((M, 48), dtype=torch.bfloat16, device="cuda")
            w4.gated_forward(x, wg, wu, act, h, None if not w4.gated_forward_bytes(M, 64, 48) else _empty(w4.gated_forward_bytes(M, 64, 48)))
            g = _gated_backward(x, wg, wu, dh, act)
            assert torch.isfinite(h).all() and all(torch.isfinite(t).all() for t in g)
            bad = x.clone()
            bad[2, 5], bad[4, 63] = float("inf"), float("nan")
            h2 = torch.empty_like(h)
            w4.gated_forward(bad, wg, wu, act, h2, None if not w4.gated_forward_bytes(M, 64, 48) else _empty(w4.gated_forward_bytes(M, 64, 48)))
            keep = [m for m in range(M) if m not in (2, 4)]
            assert torch.equal(h2[keep], h[keep]) and torch.isnan(h2[4]).all()


@gpu
@pytest.mark.parametrize("op", ["norm", "gated"])
def test_gradients_against_differences(op):
    """The kernels' gradients along a direction against central differences of the forward formula in 64
    bits (step 1e-5: its own error is far below the gradients' rounding to bf16)."""
    t = 1e-5
    if op == "norm":
        c = _norm_case(12, 130, "f32", "f32", seed=21)
        _, mean, rstd = _norm_forward(c)
        grads = _norm_backward(c, mean, rstd)
        at = [c["x"].cpu().double(), c["gamma"].cpu().double(), c["beta"].cpu().double()]
        dy = c["dy"].cpu().double()
        f = lambda x, g, b: (dy * ((x - x.mean(1, keepdim=True)) / torch.sqrt(x.var(1, unbiased=False, keepdim=True) + 1e-5) * g + b)).sum()  # noqa: E731
        rel = 2e-5
    else:
        x, wg, wu, dh = _gated_inputs(40, 72, 56, 33)
        grads = _gated_backward(x, wg, wu, dh, "silu")
        at, dy = [v.cpu().double() for v in (x, wg, wu)], dh.cpu().double()
        f = lambda x, g, u: (dy * _act64(x @ g.T, "silu")[0] * (x @ u.T)).sum()  # noqa: E731
        rel = 4 * U16
    for i, (a, g) in enumerate(zip(at, grads)):
        gen = torch.Generator().manual_seed(i)
        v = torch.randn(a.shape, generator=gen, dtype=torch.float64)
        hi, lo = list(at), list(at)
        hi[i], lo[i] = a + t * v, a - t * v
        want = float((f(*hi) - f(*lo)) / (2 * t))
        got = float((g.cpu().double() * v).sum())
        scale = float(g.cpu().double().norm() * v.norm()) / math.sqrt(v.numel())
        assert abs(got - want) <= rel * 4 * scale + 1e-6 * abs(want), (i, got, want)


# ------------------------------------------------------------------- offsets beyond 32 bits
def _big(M, K, seed):
    """[M, K] bf16 of more than 2^31 elements: one random stretch of 4096 rows after another, shifted."""
    base = _rand(seed, (4096, K))
    x = torch.empty((M, K), dtype=torch.bfloat16, device="cuda")
    for i in range(0, M, 4096):
        n = min(4096, M - i)
        x[i: i + n] = torch.roll(base, i // 4096, 0)[:n]
    return x


@gpu
def test_layer_norm_beyond_32_bits():
    M, K = 1_050_001, 2050
    c = dict(M=M, K=K, x=_big(M, K, 1), gamma=_rand(2, (K,)), beta=_rand(3, (K,)))
    y, mean, rstd = _norm_forward(c)
    dx = torch.empty_like(y)
    w4.layer_norm_backward(c["x"], c["x"], c["gamma"], mean, rstd, dx, None, None, None)
    rows = torch.tensor([0, 1, 524_287, 1_047_000, M - 2, M - 1])
    s = dict(c, M=len(rows), x=c["x"][rows.cuda()], dy=c["x"][rows.cuda()])
    _check_norm_forward(s, y[rows.cuda()], mean[rows.cuda()], rstd[rows.cuda()])
    _check_norm_backward(s, mean[rows.cuda()], rstd[rows.cuda()], dx[rows.cuda()], None, None)


@gpu
def test_checkpoint_beyond_32_bits():
    M, K = 1_060_000, 2056
    x = _big(M, K, 4)
    codes, scales = _pack(x)
    back = torch.empty_like(x)
    w4.checkpoint_unpack(codes, scales, back)
    for r in (0, 512_000, M - 64):
        q, e, want = _pack64(x[r: r + 64])
        b = r // 32
        assert torch.equal(codes[b: b + 2].cpu(), q) and torch.equal(scales[b: b + 2].cpu(), e)
        assert torch.equal(back[r: r + 64].cpu().double(), want)
    del back
    # one token of the last block and one of the first reach the gradient: whole numbers, exact
    dy = torch.zeros((M, 264), dtype=torch.bfloat16, device="cuda")
    dy[M - 1, 5], dy[3, 7] = 1.0, 2.0
    for n in (264, 8):
        dw = torch.empty((n, K), device="cuda")
        w4.checkpoint_weight_grad(dy[:, :n], codes, scales, K, dw, _empty(w4.checkpoint_weight_grad_bytes(M, n, K)))
        want = torch.zeros((n, K), dtype=torch.float64)
        want[5], want[7] = _pack64(x[M - 32:])[2][31], 2 * _pack64(x[:32])[2][3]
        assert torch.equal(dw.cpu().double(), want), n


@gpu
def test_gated_beyond_32_bits():
    M, K, F = 66_001, 64, 32_776
    x, wg, wu = _rand(1, (M, K)), _rand(2, (F, K), 0.125), _rand(3, (F, K), 0.125)
    h = torch.full((M, F), float("nan"), dtype=torch.bfloat16, device="cuda")
    w4.gated_forward(x, wg, wu, "silu", h, _empty(w4.gated_forward_bytes(M, K, F)))
    rows = torch.tensor([0, 40_000, 65_535, 65_536, M - 1])
    r = _gated64(x[rows.cuda()].cpu().double(), wg.cpu().double(), wu.cpu().double(), "silu")
    _within(h[rows.cuda()].cpu(), r["h"], r["eh"] + U16 * (r["h"].abs() + r["eh"]) + 1e-30, "h")
    assert not torch.isnan(h).any()   # every element is written


# ----------------------------------------------------------------------------- streams and graphs
def _all_ops():
    """Calls of every operator on fixed inputs, as (call, outputs)."""
    c = _matvec_case(3, 300, 448, 20, "int4_g64", True, seed=5)
    y = torch.empty((3, 300), dtype=torch.bfloat16, device="cuda")
    n = _norm_case(100, 1000, "bf16", "bf16", seed=6)
    ny, mean, rstd = torch.empty_like(n["x"]), torch.empty(100, device="cuda"), torch.empty(100, device="cuda")
    dx, dg, db = torch.empty_like(n["x"]), torch.empty(1000, device="cuda"), torch.empty(1000, device="cuda")
    nws = _empty(w4.layer_norm_backward_bytes(100, 1000))
    x, dy = _rand(7, (100, 264)), _rand(8, (100, 72))
    codes, scales = _pack(x)
    back, dw = torch.empty_like(x), torch.empty((72, 264), device="cuda")
    cws = _empty(w4.checkpoint_weight_grad_bytes(100, 72, 264))
    gx, wg, wu, dh = _gated_inputs(100, 264, 136, 9)
    h, gdx, dwg, dwu = torch.empty_like(dh), torch.empty_like(gx), torch.empty_like(wg), torch.empty_like(wu)
    ht, fws = torch.empty((1, 136), dtype=torch.bfloat16, device="cuda"), _empty(max(w4.gated_forward_bytes(m, 264, 136) for m in (1, 100)))
    gws = _empty(w4.gated_backward_bytes(100, 264, 136))

    def call(stream=None):
        _matvec(c, y=y, stream=stream)
        w4.layer_norm(n["x"], n["gamma"], n["beta"], 1e-5, ny, mean, rstd, stream)
        w4.layer_norm_backward(n["dy"], n["x"], n["gamma"], mean, rstd, dx, dg, db, nws, stream)
        w4.checkpoint_pack(x, codes, scales, stream)
        w4.checkpoint_unpack(codes, scales, back, stream)
        w4.checkpoint_weight_grad(dy, codes, scales, 264, dw, cws, stream)
        w4.gated_forward(gx, wg, wu, "silu", h, fws, stream)
        w4.gated_forward(gx[:1], wg, wu, "silu", ht, fws, stream)
        w4.gated_backward(dh, gx, wg, wu, "silu", gdx, dwg, dwu, gws, stream)
    return call, [y, ny, mean, rstd, dx, dg, db, codes, scales, back, dw, h, ht, gdx, dwg, dwu]


@gpu
def test_ops_on_another_stream_and_in_a_graph():
    """The same bits on a given stream and from several replays of a captured graph, with eager calls and
    overwritten outputs between them."""
    call, outs = _all_ops()
    call()
    torch.cuda.synchronize()
    want = [o.clone() for o in outs]

    def check(what):
        torch.cuda.synchronize()
        for i, (o, w) in enumerate(zip(outs, want)):
            assert torch.equal(o, w), f"{what}: output {i}"
            o.zero_()
        torch.cuda.synchronize()

    check("again")
    s = torch.cuda.Stream()
    call(s)
    s.synchronize()
    check("stream")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for i in range(3):
        graph.replay()
        check(f"replay {i}")
        call()
        check(f"eager {i}")


# ---------------------------------------------------------------------------------------- refusals
def _status(name, *args):
    return getattr(w4.lib(), name)(*args)


P = ctypes.c_void_p(1 << 20)   # an aligned address that no refused call touches
ODD = ctypes.c_void_p((1 << 20) + 1)


def test_refusals_of_the_c_calls():
    """Every call answers a bad argument with a status before it does anything (no GPU needed)."""
    mv = lambda **k: [k.get(n, d) for n, d in (("X", P), ("M", 1), ("K", 128), ("ldx", 128), ("inv", P), ("l1t", P), ("wv", P), ("l2t", P),  # noqa: E731
                      ("bias", None), ("Y", P), ("ldy", 64), ("N", 64), ("rank", 16), ("fmt", 0), ("ws", P), ("st", None))]
    for bad in (dict(M=0), dict(M=17), dict(K=100), dict(K=0), dict(N=0), dict(rank=-1), dict(rank=65), dict(ldx=120), dict(ldx=129),
                dict(ldy=63), dict(X=None), dict(inv=None), dict(wv=None), dict(Y=None), dict(ws=None), dict(l1t=None), dict(l2t=None),
                dict(X=ODD), dict(Y=ODD), dict(wv=ODD), dict(bias=ODD), dict(ldx=(1 << 26) + 8)):
        assert _status("w4a4_matvec", *mv(**bad)) == 1, bad
    assert _status("w4a4_matvec", *mv(fmt=2)) == 2 and _status("w4a4_matvec", *mv(fmt=9)) == 2
    assert _status("w4a4_matvec_weights", P, P, 64, 128, 2, P, None) == 2
    assert _status("w4a4_matvec_weights", None, P, 64, 128, 0, P, None) == 1
    assert _status("w4a4_matvec_weights", P, P, 64, 96, 0, P, None) == 1
    s = ctypes.c_size_t()
    assert _status("w4a4_matvec_sizes", 17, 64, 128, 16, 0, ctypes.byref(s), ctypes.byref(s)) == 1
    assert _status("w4a4_matvec_sizes", 1, 64, 128, 16, 0, None, ctypes.byref(s)) == 1

    ln = lambda **k: [k.get(n, d) for n, d in (("X", P), ("M", 2), ("K", 5), ("ldx", 5), ("dt", 0), ("g", None), ("b", None), ("pt", 0),  # noqa: E731
                      ("eps", 1e-5), ("Y", P), ("ldy", 5), ("mean", P), ("rstd", P), ("st", None))]
    for bad in (dict(M=0), dict(K=0), dict(ldx=4), dict(ldy=4), dict(X=None), dict(Y=None), dict(mean=None), dict(rstd=None),
                dict(X=ODD), dict(Y=ODD), dict(g=ODD), dict(b=ODD), dict(eps=-1.0), dict(eps=float("nan")), dict(K=(1 << 26) + 1),
                dict(M=(1 << 30) + 1)):
        assert _status("w4a4_layer_norm", *ln(**bad)) == 1, bad
    assert _status("w4a4_layer_norm", *ln(dt=2)) == 2 and _status("w4a4_layer_norm", *ln(pt=-1)) == 2
    lb = lambda **k: [k.get(n, d) for n, d in (("dY", P), ("lddy", 5), ("X", P), ("ldx", 5), ("dt", 0), ("g", None), ("pt", 0), ("mean", P),  # noqa: E731
                      ("rstd", P), ("M", 2), ("K", 5), ("dX", P), ("lddx", 5), ("dg", P), ("db", None), ("ws", P), ("st", None))]
    for bad in (dict(M=0), dict(K=0), dict(lddy=4), dict(ldx=4), dict(lddx=4), dict(dY=None), dict(X=None), dict(dX=None),
                dict(mean=None), dict(rstd=None), dict(ws=None), dict(dg=ODD), dict(ws=ODD), dict(dX=ODD)):
        assert _status("w4a4_layer_norm_backward", *lb(**bad)) == 1, bad
    assert _status("w4a4_layer_norm_backward", *lb(dt=7)) == 2
    assert w4.layer_norm_backward_bytes(0, 5) == 0 and w4.layer_norm_backward_bytes(3, 5) == 3 * 2 * 5 * 4

    for args in ((P, 0, 8, 8, P, P), (P, 1, 12, 16, P, P), (P, 1, 0, 8, P, P), (P, 1, 16, 8, P, P), (P, 1, 8, 12, P, P), (None, 1, 8, 8, P, P),
                 (P, 1, 8, 8, None, P), (P, 1, 8, 8, P, None), (ODD, 1, 8, 8, P, P), (P, 1, 8, 8, ODD, P), (P, 1, 8, 8, P, ODD)):
        assert _status("w4a4_checkpoint_pack", *args, None) == 1, args
        x, m, k, ld, c, e = args
        assert _status("w4a4_checkpoint_unpack", c, e, m, k, x, ld, None) == 1, args
    assert _status("w4a4_checkpoint_sizes", 1, 12, ctypes.byref(s), ctypes.byref(s)) == 1
    wg = lambda **k: [k.get(n, d) for n, d in (("dY", P), ("ld", 16), ("c", P), ("s", P), ("M", 5), ("N", 16), ("K", 8), ("dW", P), ("dt", 1),  # noqa: E731
                      ("ws", P), ("st", None))]
    for bad in (dict(M=0), dict(N=0), dict(N=12), dict(K=12), dict(ld=8), dict(ld=20), dict(dY=None), dict(c=None), dict(s=None), dict(dW=None),
                dict(ws=None), dict(dY=ODD), dict(dW=ODD), dict(ld=(1 << 21) + 8)):
        assert _status("w4a4_checkpoint_weight_grad", *wg(**bad)) == 1, bad
    assert _status("w4a4_checkpoint_weight_grad", *wg(dt=3)) == 2
    assert w4.checkpoint_weight_grad_bytes(5, 12, 8) == 0

    gf = lambda **k: [k.get(n, d) for n, d in (("X", P), ("M", 4), ("K", 16), ("ldx", 16), ("wg", P), ("wu", P), ("ldw", 16), ("F", 24),  # noqa: E731
                      ("act", 0), ("H", P), ("ldh", 24), ("ws", P), ("st", None))]
    for bad in (dict(M=0), dict(K=12), dict(F=20), dict(F=0), dict(ldx=8), dict(ldw=20), dict(ldh=16), dict(X=None), dict(wg=None),
                dict(wu=None), dict(H=None), dict(X=ODD), dict(H=ODD), dict(ldx=(1 << 21) + 8)):
        assert _status("w4a4_gated_forward", *gf(**bad)) == 1, bad
    assert _status("w4a4_gated_forward", *gf(act=2)) == 2
    gb = lambda **k: [k.get(n, d) for n, d in (("dH", P), ("lddh", 24), ("X", P), ("M", 4), ("K", 16), ("ldx", 16), ("wg", P), ("wu", P),  # noqa: E731
                      ("ldw", 16), ("F", 24), ("act", 0), ("dX", P), ("dwg", P), ("dwu", P), ("ws", P), ("st", None))]
    for bad in (dict(M=0), dict(K=12), dict(F=20), dict(lddh=16), dict(ldx=8), dict(ldw=8), dict(dH=None), dict(dX=None), dict(dwg=None),
                dict(dwu=None), dict(ws=None), dict(dX=ODD), dict(dwu=ODD), dict(ws=ODD)):
        assert _status("w4a4_gated_backward", *gb(**bad)) == 1, bad
    assert _status("w4a4_gated_backward", *gb(act=-1)) == 2
    assert w4.gated_backward_bytes(0, 8, 8) == 0


def test_ops_header_is_exported():
    import os
    import re
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "w4a4_ops.h")
    names = set(re.findall(r"^(?:w4a4_status_t|size_t) (w4a4_[a-z0-9_]+)\(", open(path).read(), re.M))
    assert len(names) == 15 and all(hasattr(w4.lib(), n) for n in names), sorted(names)


@gpu
def test_refusals_of_the_python_calls():
    x = _rand(1, (4, 64))
    y, m = torch.empty_like(x), torch.empty(4, device="cuda")
    for args, error in (((x.cpu(), None, None, 1e-5, y, m, m), ValueError), ((x.half(), None, None, 1e-5, y, m, m), ValueError),
                        ((x, None, None, 1e-5, y.float(), m, m), ValueError), ((x, None, None, 1e-5, y[:3], m, m), ValueError),
                        ((x, m, None, 1e-5, y, m, m), ValueError), ((x.T, None, None, 1e-5, y.T, m, m), ValueError),
                        ((x, None, None, 1e-5, y, m.double(), m), ValueError), ((x[0], None, None, 1e-5, y, m, m), ValueError),
                        ((x, None, None, -1.0, y, m, m), w4.W4A4Error), ((3, None, None, 1e-5, y, m, m), ValueError)):
        with pytest.raises(error):
            w4.layer_norm(*args)
    with pytest.raises(ValueError):
        w4.layer_norm_backward(x, x, None, m, m, y, torch.empty(64, device="cuda"), None, torch.empty(8, dtype=torch.uint8, device="cuda"))
    wg = _rand(2, (32, 64))
    h = torch.empty((4, 32), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        w4.gated_forward(x, wg, wg, "tanh", h)
    with pytest.raises(ValueError):
        w4.gated_forward(x, wg, wg[:16], "silu", h)
    with pytest.raises(ValueError):
        w4.gated_backward(h, x, wg, wg, "silu", y, torch.empty_like(wg), torch.empty_like(wg), torch.empty(16, dtype=torch.uint8, device="cuda"))
    codes, scales = _pack(x)
    with pytest.raises(ValueError):
        w4.checkpoint_unpack(codes, scales.flatten()[:-1], y)
    with pytest.raises(w4.W4A4Error):
        w4.checkpoint_sizes(4, 12)
    with pytest.raises(ValueError):
        w4.checkpoint_weight_grad(x, codes, scales, 64, torch.empty((64, 64), dtype=torch.float64, device="cuda"), y)
    c = _matvec_case(2, 64, 64, 16, "int4_g64", False, seed=1)
    with pytest.raises(ValueError):
        _matvec(dict(c, ws=c["ws"][:16]))
    with pytest.raises(w4.W4A4Error):
        _matvec(dict(c, fmt="w8a8"))
    with pytest.raises(w4.W4A4Error):
        _matvec(c, _rand(1, (17, 64)))
