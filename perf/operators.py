"""Measured cases of the training and single-token operators, with their plain forms.

    matvec      Y = X̂·deq(Q)ᵀ + (X̂·L1)·L2 (+ bias) for 1 to 16 rows, X̂ = X·diag(1/λ) kept in 16 bits or more:
                the layer's 4-bit weights with 16-bit activations
    norm        layer normalisation and its gradients
    checkpoint  activations kept in 8 bits (one power of two per channel and 32 tokens), what they
                stand for, and the weight gradient dYᵀ·X taken from them
    gated       H = act(X·Wgᵀ) ⊙ (X·Wuᵀ) and its gradients

``run`` is one call as a program makes it: with ``own`` true through this repository's package, with
``own`` false from elementary torch operations in 32 bits. ``exact`` gives the same outputs from the
definitions in 64 bits.
"""
import math

import torch

own = False

INT4, MXFP4 = "int4_g64", "mxfp4_b32"
BLOCK = 32           # tokens that share a checkpoint's scale
EPS = 1e-5
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # one token through the attention's input projection, the layer of the default benchmark
        dict(name="matvec token qkv", op="matvec", M=1, N=9216, K=3072, rank=32, fmt=INT4, bias=False),
        # the smallest call, where the launches are what it costs: one token, a small odd layer
        dict(name="matvec token small", op="matvec", M=1, N=635, K=256, rank=20, fmt=MXFP4, bias=True),
        # a batch of 13 sequences, one token each, through the second MLP layer with a merged LoRA
        dict(name="matvec batch mlp", op="matvec", M=13, N=3072, K=12288, rank=48, fmt=INT4, bias=True),
        # the norm in front of a block's projections at 4608 tokens
        dict(name="norm forward", op="norm", M=4608, K=3072, dtype="bf16", direction="forward", affine=True),
        # a large training batch's gradients
        dict(name="norm backward", op="norm", M=16384, K=4096, dtype="bf16", direction="backward", affine=True),
        # both directions on a 32-bit residual stream of an odd width
        dict(name="norm step odd", op="norm", M=777, K=1531, dtype="f32", direction="step", affine=True),
        # the hidden activations of an MLP kept in 8 bits, and read back
        dict(name="checkpoint kept", op="checkpoint", M=4608, N=0, K=12288, out="bf16"),
        # the gradient of a whole projection weight from them
        dict(name="checkpoint weight", op="checkpoint", M=4608, N=4096, K=12288, out="f32"),
        # the gradient of a low-rank factor, ragged token count
        dict(name="checkpoint factor", op="checkpoint", M=4607, N=32, K=4096, out="f32"),
        # one token through a gated feed-forward block
        dict(name="gated token", op="gated", M=1, K=4096, F=12288, act="silu", direction="forward"),
        # a prompt or a training batch
        dict(name="gated forward", op="gated", M=4608, K=4096, F=12288, act="gelu", direction="forward"),
        # the gradients, odd sizes
        dict(name="gated backward", op="gated", M=2041, K=2056, F=5624, act="silu", direction="backward"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _multiple(rng, lo, hi, of):
    return max(lo, min(hi, _log(rng, lo, hi) // of * of))


def draw(rng):
    most = max(work(c)["flops"] for c in listed())
    while True:
        op = rng.choice(["matvec", "norm", "checkpoint", "gated"])
        if op == "matvec":
            case = dict(op=op, M=rng.randint(1, 16), N=_log(rng, 64, 12288), K=_multiple(rng, 64, 12288, 64),
                        rank=rng.choice([0, 16, 20, 32, 48, 64]), fmt=rng.choice([INT4, MXFP4]), bias=rng.random() < 0.5)
        elif op == "norm":
            case = dict(op=op, M=_log(rng, 1, 16384), K=_log(rng, 40, 16384) if rng.random() < 0.5 else _multiple(rng, 64, 16384, 64),
                        dtype=rng.choice(["bf16", "f32"]), direction=rng.choice(["forward", "backward", "step"]),
                        affine=rng.random() < 0.8)
            if case["M"] * case["K"] > 4608 * 12288:
                continue
        elif op == "checkpoint":
            case = dict(op=op, M=_log(rng, 1, 16384), N=rng.choice([0, _multiple(rng, 8, 128, 8), _multiple(rng, 64, 12288, 8)]),
                        K=_multiple(rng, 64, 12288, 8), out=rng.choice(["bf16", "f32"]))
            if case["M"] * case["K"] > 4608 * 12288 or case["M"] * case["N"] > 4608 * 12288:
                continue
        else:
            case = dict(op=op, M=_log(rng, 1, 4608), K=_multiple(rng, 64, 4096, 8), F=_multiple(rng, 64, 12288, 8),
                        act=rng.choice(["silu", "gelu"]), direction=rng.choice(["forward", "backward"]))
        if work(case)["flops"] <= most:
            return case


def work(case):
    M, K = case["M"], case["K"]
    if case["op"] == "matvec":
        N, r = case["N"], case["rank"]
        scales = N * K // 64 * 2 if case["fmt"] == INT4 else N * K // 32
        return {"bytes": N * K // 2 + scales + 2 * r * (N + K) + 2 * M * (N + K) + 4 * K + (2 * N if case["bias"] else 0),
                "flops": 2 * M * N * K + 2 * M * r * (N + K)}
    if case["op"] == "norm":
        e = 2 if case["dtype"] == "bf16" else 4
        p = K * e if case["affine"] else 0
        forward = {"bytes": 2 * M * K * e + 8 * M + 2 * p, "flops": 8 * M * K}
        backward = {"bytes": 3 * M * K * e + 8 * M + p + (8 * K if case["affine"] else 0), "flops": 14 * M * K}
        if case["direction"] == "step":   # x, the statistics and gamma are one input to both
            return {"bytes": 4 * M * K * e + 8 * M + 2 * p + (8 * K if case["affine"] else 0), "flops": 22 * M * K}
        return forward if case["direction"] == "forward" else backward
    if case["op"] == "checkpoint":
        N, kept = case["N"], M * K + -(-M // BLOCK) * K
        if N == 0:
            return {"bytes": 4 * M * K + 2 * kept, "flops": 4 * M * K}
        return {"bytes": kept + 2 * M * N + N * K * (4 if case["out"] == "f32" else 2), "flops": 2 * M * N * K}
    F = case["F"]
    if case["direction"] == "forward":
        return {"bytes": 2 * (M * K + 2 * F * K + M * F), "flops": 4 * M * K * F}
    # both projections again, the input's gradient, the two weights' gradients
    return {"bytes": 2 * (2 * M * K + 4 * F * K + M * F), "flops": 12 * M * K * F}


# ----------------------------------------------------------------------------------------- inputs
def _normal(g, shape, std=1.0, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def _activations(g, M, K, scale=30.0, dtype=torch.bfloat16):
    """Standard normal with 1% outlier channels, a given factor larger."""
    x = torch.randn((M, K), generator=g, device="cuda")
    x[:, torch.randperm(K, generator=g, device="cuda")[: K // 100]] *= scale
    return x.to(dtype)


def _pad(a, rows, cols):
    out = torch.zeros((rows, cols), dtype=a.dtype, device=a.device)
    out[: a.shape[0], : a.shape[1]] = a
    return out


def _two(e, dtype=torch.float32):
    """2^e for whole e in the type's normal range, exactly."""
    if dtype == torch.float64:
        return ((e.long() + 1023) << 52).view(torch.float64)
    return ((e.int() + 127).clamp(min=1) << 23).view(torch.float32)


def _block_maxima(x):
    M, K = x.shape
    return _pad(x, -(-M // BLOCK) * BLOCK, K).float().abs().view(-1, BLOCK, K).amax(1)


def _block_exponents(x):
    """Smallest e with 127·2^e ≥ the block's largest magnitude, from −127 up: [blocks, K]."""
    f, p = torch.frexp(_block_maxima(x))
    e = torch.where(f * 128 <= 127, p - 7, p - 6).clamp(min=-127)
    return torch.where(f == 0, torch.full_like(e, -127), e)


def _codes(x, e):
    """Whole numbers in −127 .. 127, [M, K] (kept in 32 bits)."""
    s = e.repeat_interleave(BLOCK, 0)[: x.shape[0]]
    return torch.round(x.float() * _two(-s)).clamp(-127, 127)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    M, K = case["M"], case["K"]
    s = dict(case)
    if case["op"] == "matvec":
        N, r, int4 = case["N"], case["rank"], case["fmt"] == INT4
        s["x"] = _activations(g, M, K)
        s["inv"] = torch.rand(K, generator=g, device="cuda") + 0.5
        s["codes"] = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
        if int4:
            s["scales"] = ((torch.rand((N, K // 64), generator=g, device="cuda") + 0.5) * 0.01).bfloat16()
        else:
            s["scales"] = torch.randint(118, 122, (N, K // 32), generator=g, device="cuda", dtype=torch.uint8)
        rp = -(-r // 16) * 16
        s["l1t"] = _pad(_normal(g, (r, K), 0.05), rp, K) if r else None
        s["l2t"] = _pad(_normal(g, (N, r), 0.05), -(-N // 256) * 256, rp) if r else None
        s["bias"] = _normal(g, (N,)) if case["bias"] else None
        if own:
            import w4a4_quantized_gemm_smooth_amd as w4
            sizes = w4.matvec_sizes(M, N, K, r, case["fmt"])
            s["wv"] = torch.empty(sizes["wv"], dtype=torch.uint8, device="cuda")
            s["ws"] = torch.empty(sizes["ws"], dtype=torch.uint8, device="cuda")
            w4.matvec_weights(s["codes"], s["scales"], N, K, case["fmt"], s["wv"])
            s["y"] = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    elif case["op"] == "norm":
        dtype = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        s["x"] = _activations(g, M, K, 10.0, dtype)
        s["gamma"] = _normal(g, (K,), 0.2, dtype) + 1 if case["affine"] else None
        s["beta"] = _normal(g, (K,), 0.2, dtype) if case["affine"] else None
        s["dy"] = _normal(g, (M, K), 0.01, dtype)
        s["mean"] = s["x"].float().mean(1)
        s["rstd"] = torch.rsqrt((s["x"].float() - s["mean"][:, None]).square().mean(1) + EPS)
        if own:
            import w4a4_quantized_gemm_smooth_amd as w4
            s["y"], s["dx"] = torch.empty_like(s["x"]), torch.empty_like(s["x"])
            s["mean_out"], s["rstd_out"] = torch.empty_like(s["mean"]), torch.empty_like(s["rstd"])
            f32 = lambda: torch.empty(K, device="cuda") if case["affine"] else None  # noqa: E731
            s["dgamma"], s["dbeta"] = f32(), f32()
            s["ws"] = torch.empty(w4.layer_norm_backward_bytes(M, K), dtype=torch.uint8, device="cuda")
    elif case["op"] == "checkpoint":
        N = case["N"]
        x = _activations(g, M, K)
        if N == 0:
            s["x"] = x
        else:
            e = _block_exponents(x)
            c = _pad(_codes(x, e).to(torch.int8), -(-M // BLOCK) * BLOCK, K)
            s["codes"] = c.view(-1, BLOCK, K).transpose(1, 2).contiguous()   # [blocks, K, 32 tokens]
            s["scales"] = (e + 127).to(torch.uint8)                          # [blocks, K]
            s["dy"] = _normal(g, (M, N), 0.01)
        if own:
            import w4a4_quantized_gemm_smooth_amd as w4
            if N == 0:
                sizes = w4.checkpoint_sizes(M, K)
                s["codes"] = torch.empty(sizes["codes"], dtype=torch.int8, device="cuda")
                s["scales"] = torch.empty(sizes["scales"], dtype=torch.uint8, device="cuda")
                s["back"] = torch.empty_like(x)
            else:
                s["dw"] = torch.empty((N, K), dtype=torch.float32 if case["out"] == "f32" else torch.bfloat16, device="cuda")
                s["ws"] = torch.empty(w4.checkpoint_weight_grad_bytes(M, N, K), dtype=torch.uint8, device="cuda")
    else:
        F = case["F"]
        s["x"] = _activations(g, M, K)
        s["wg"] = _normal(g, (F, K), 0.02)
        s["wu"] = _normal(g, (F, K), 0.02)
        if case["direction"] == "backward":
            s["dh"] = _normal(g, (M, F), 0.01)
        if own:
            import w4a4_quantized_gemm_smooth_amd as w4
            if case["direction"] == "forward":
                s["h"] = torch.empty((M, F), dtype=torch.bfloat16, device="cuda")
                s["ws"] = torch.empty(w4.gated_forward_bytes(M, K, F), dtype=torch.uint8, device="cuda")
            else:
                s["dx"], s["dwg"], s["dwu"] = (torch.empty_like(s[k]) for k in ("x", "wg", "wu"))
                s["ws"] = torch.empty(w4.gated_backward_bytes(M, K, F), dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------------------------------- plain forms
def _decode(codes, scales, fmt, dtype):
    """The weights that packed 4-bit codes (even columns in the low nibbles) and their scales stand for."""
    q = torch.stack((codes & 15, codes >> 4), -1).view(codes.shape[0], -1)
    if fmt == INT4:
        return (((q ^ 8).to(dtype) - 8).view(q.shape[0], -1, 64) * scales.to(dtype)[:, :, None]).view(q.shape)
    values = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=dtype, device=codes.device)
    return (values[q.long()].view(q.shape[0], -1, 32) * _two(scales.int() - 127, dtype)[:, :, None]).view(q.shape)


def _act(g, kind):
    """act(g) and its derivative."""
    if kind == "silu":
        p = 1 / (1 + torch.exp(-g))
        return g * p, p * (1 + g * (1 - p))
    p = 0.5 * (1 + torch.erf(g * math.sqrt(0.5)))
    return g * p, p + g * torch.exp(-0.5 * g * g) * (1 / math.sqrt(2 * math.pi))


def _plain_matvec(s):
    x = s["x"].float() * s["inv"]
    y = x @ _decode(s["codes"], s["scales"], s["fmt"], torch.float32).T
    if s["rank"]:
        y = y + (x @ s["l1t"].float().T) @ s["l2t"][: s["N"]].float().T
    if s["bias"] is not None:
        y = y + s["bias"].float()
    return y.bfloat16()


def _plain_norm(s):
    x, out = s["x"].float(), {}
    gamma = s["gamma"].float() if s["affine"] else 1.0
    mean, rstd = s["mean"], s["rstd"]
    if s["direction"] != "backward":
        mean = x.mean(1)
        rstd = torch.rsqrt((x - mean[:, None]).square().mean(1) + EPS)
        y = (x - mean[:, None]) * rstd[:, None] * gamma
        out = dict(y=(y + s["beta"].float() if s["affine"] else y).to(s["x"].dtype), mean=mean, rstd=rstd)
    if s["direction"] != "forward":
        dy = s["dy"].float()
        h = (x - mean[:, None]) * rstd[:, None]
        d = dy * gamma
        dx = rstd[:, None] * (d - d.mean(1, keepdim=True) - h * (d * h).mean(1, keepdim=True))
        out["dx"] = dx.to(s["x"].dtype)
        if s["affine"]:
            out.update(dgamma=(dy * h).sum(0), dbeta=dy.sum(0))
    return out


def _plain_checkpoint(s):
    M, K = s["M"], s["K"]
    if s["N"] == 0:
        e = _block_exponents(s["x"])
        return (_codes(s["x"], e) * _two(e.repeat_interleave(BLOCK, 0)[:M])).bfloat16()
    x = (s["codes"].float() * _two(s["scales"].int() - 127)[:, :, None]).transpose(1, 2).reshape(-1, K)[:M]
    return (s["dy"].float().T @ x).to(torch.float32 if s["out"] == "f32" else torch.bfloat16)


def _plain_gated(s):
    x, wg, wu = s["x"].float(), s["wg"].float(), s["wu"].float()
    g, u = x @ wg.T, x @ wu.T
    a, slope = _act(g, s["act"])
    if s["direction"] == "forward":
        return (a * u).bfloat16()
    dh = s["dh"].float()
    dg, du = dh * u * slope, dh * a
    return dict(dx=(dg @ wg + du @ wu).bfloat16(), dwg=(dg.T @ x).bfloat16(), dwu=(du.T @ x).bfloat16())


# -------------------------------------------------------------------------------- this repository's
def _own(s):
    import w4a4_quantized_gemm_smooth_amd as w4
    if s["op"] == "matvec":
        w4.matvec(s["x"], s["inv"], s["l1t"], s["wv"], s["l2t"], s["bias"], s["y"], s["N"], s["K"], s["rank"], s["fmt"], s["ws"])
        return s["y"]
    if s["op"] == "norm":
        out, mean, rstd = {}, s["mean"], s["rstd"]
        if s["direction"] != "backward":
            mean, rstd = s["mean_out"], s["rstd_out"]
            w4.layer_norm(s["x"], s["gamma"], s["beta"], EPS, s["y"], mean, rstd)
            out = dict(y=s["y"], mean=mean, rstd=rstd)
        if s["direction"] != "forward":
            w4.layer_norm_backward(s["dy"], s["x"], s["gamma"], mean, rstd, s["dx"], s["dgamma"], s["dbeta"], s["ws"])
            out["dx"] = s["dx"]
            if s["affine"]:
                out.update(dgamma=s["dgamma"], dbeta=s["dbeta"])
        return out
    if s["op"] == "checkpoint":
        if s["N"] == 0:
            w4.checkpoint_pack(s["x"], s["codes"], s["scales"])
            w4.checkpoint_unpack(s["codes"], s["scales"], s["back"])
            return s["back"]
        w4.checkpoint_weight_grad(s["dy"], s["codes"], s["scales"], s["K"], s["dw"], s["ws"])
        return s["dw"]
    if s["direction"] == "forward":
        w4.gated_forward(s["x"], s["wg"], s["wu"], s["act"], s["h"], s["ws"])
        return s["h"]
    w4.gated_backward(s["dh"], s["x"], s["wg"], s["wu"], s["act"], s["dx"], s["dwg"], s["dwu"], s["ws"])
    return dict(dx=s["dx"], dwg=s["dwg"], dwu=s["dwu"])


def run(state):
    if own:
        return _own(state)
    return {"matvec": _plain_matvec, "norm": _plain_norm, "checkpoint": _plain_checkpoint, "gated": _plain_gated}[state["op"]](state)


# ---------------------------------------------------------------------------------------- 64 bits
def _exact_norm(s):
    """The normalised rows from centred sums; the gradient as the transposed Jacobian applied to dY·γ:
    J = rstd·(I − 1·1ᵀ/K − h·hᵀ/K)."""
    x, K, out = s["x"].double(), s["K"], {}
    if s["direction"] == "backward":
        mean, rstd = s["mean"].double(), s["rstd"].double()
    else:
        mean = x.sum(1) / K
        rstd = 1 / torch.sqrt((x - mean[:, None]).pow(2).sum(1) / K + EPS)
    h = (x - mean[:, None]) * rstd[:, None]
    one = torch.ones(K, dtype=torch.float64, device=x.device)
    gamma = s["gamma"].double() if s["affine"] else one
    if s["direction"] != "backward":
        out = dict(y=h * gamma + (s["beta"].double() if s["affine"] else 0), mean=mean, rstd=rstd)
    if s["direction"] != "forward":
        dy = s["dy"].double()
        out["dx"] = rstd[:, None] * (dy * gamma - ((dy @ gamma)[:, None] + h * ((dy * h) @ gamma)[:, None]) / K)
        if s["affine"]:
            out.update(dgamma=torch.einsum("mk,mk->k", dy, h), dbeta=torch.einsum("mk->k", dy))
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "matvec":
        w = _decode(s["codes"], s["scales"], s["fmt"], torch.float64)
        if s["rank"]:
            w = w + s["l2t"][: s["N"]].double() @ s["l1t"].double()
        y = (w @ (s["x"].double() * s["inv"].double()).T).T
        return y + s["bias"].double() if s["bias"] is not None else y
    if case["op"] == "norm":
        return _exact_norm(s)
    if case["op"] == "checkpoint":
        if s["N"] == 0:
            x = _pad(s["x"], -(-s["M"] // BLOCK) * BLOCK, s["K"]).double().view(-1, BLOCK, s["K"])
            top = x.abs().amax(1, keepdim=True)
            step = _two(torch.ceil(torch.log2(top / 127)).clamp(min=-127.0), torch.float64)
            return (torch.round(x / step) * step).view(-1, s["K"])[: s["M"]]
        x = s["codes"].double() * _two(s["scales"].int() - 127, torch.float64)[:, :, None]
        dy = _pad(s["dy"], x.shape[0] * BLOCK, s["N"]).double()
        return dy.T @ x.transpose(1, 2).reshape(-1, s["K"])
    x, both = s["x"].double(), torch.cat((s["wg"], s["wu"])).double()
    g, u = (x @ both.T).chunk(2, 1)
    if case["act"] == "silu":
        p = torch.special.expit(g)
        slope = p + g * p * torch.special.expit(-g)
    else:
        p = torch.special.ndtr(g)
        slope = p + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    if case["direction"] == "forward":
        return g * p * u
    d = torch.cat((s["dh"].double() * u * slope, s["dh"].double() * g * p), 1)
    dw = (x.T @ d).T
    return dict(dx=d @ both, dwg=dw[: s["F"]], dwu=dw[s["F"]:])
