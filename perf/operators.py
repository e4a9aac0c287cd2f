"""Cases of the layer operators around the quantised matrix products: the
residual addition with RMS norm and its MXFP8 output, its backward, the MX row
quantiser and the dense MXFP4-weight product.

Formats (OCP Microscaling v1.0): blocks of 32 consecutive elements of a row
share an E8M0 scale 2^X, X = floor(log2 amax) - emax clamped to [-127, 127]
(emax 8 for E4M3 elements, 2 for E2M1), stored as the byte X + 127; elements
are x / 2^X rounded to nearest even, saturating.  E2M1 codes are packed two per
byte, the even element in the low nibble.

``run`` is either the operators' plain form (elementary torch operations) or,
with ``own`` set, the calls a program makes of the library.  What is held in
8 bits comes back as torch's 8-bit floating types, which are the values the
bytes stand for; 4-bit codes are measured through the product that reads them.
"""
import math

import torch

if not hasattr(torch, "float8_e8m0fnu"):
    raise ImportError("torch with the 8-bit floating types is needed")

own = False

BF16, F32 = torch.bfloat16, torch.float32
EPS = 1e-6


# ------------------------------------------------------------------- cases
def listed():
    return [
        # a decoding step of one sequence: the norm in front of a layer's projections
        dict(name="norm_decode", op="norm", T=1, H=2048, res="bf16", train=False),
        # the learner's batch (16384 tokens, hidden 2048), everything the backward needs saved
        dict(name="norm_learner", op="norm", T=16384, H=2048, res="bf16", train=True),
        # scoring a ragged batch with the residual stream kept in 32 bits
        dict(name="norm_f32_ragged", op="norm", T=4097, H=4096, res="f32", train=False),
        # backward of a micro-batch
        dict(name="norm_bwd_micro", op="norm_bwd", T=61, H=2048, res="bf16"),
        # backward at the learner's batch
        dict(name="norm_bwd_learner", op="norm_bwd", T=16384, H=2048, res="bf16"),
        # backward of a wider layer with a 32-bit residual stream
        dict(name="norm_bwd_f32_wide", op="norm_bwd", T=8191, H=5120, res="f32"),
        # a short batch of attention outputs in front of the output projection
        dict(name="quant_short", op="quant", T=37, H=768, pad=0),
        # the learner's attention outputs, a column slice of a wider buffer
        dict(name="quant_learner", op="quant", T=16384, H=4096, pad=1024),
        # a decoding step: one token's query projection on the norm's 8-bit output
        dict(name="linear_decode", op="linear", T=1, K=2048, N=4096, fmt="fp8", x="codes"),
        # 48 sequences decoding into a vocabulary: quantisation and product
        dict(name="linear_vocab", op="linear", T=48, K=2048, N=65536, fmt="fp4", x="bf16"),
        # the query projection at the learner's batch: quantisation and product
        dict(name="linear_learner", op="linear", T=16384, K=2048, N=4096, fmt="fp4", x="bf16"),
        # a ragged batch through an output projection, 8-bit activations
        dict(name="linear_ragged", op="linear", T=5001, K=4096, N=2048, fmt="fp8", x="codes"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "quant", "linear", "linear"])
    if op != "linear":
        H = 32 * _log(rng, 8, 256)
        T = _log(rng, 1, min(16384, 16384 * 2048 // H))
        if op == "norm":
            return dict(op=op, T=T, H=H, res=rng.choice(["bf16", "f32"]), train=rng.random() < 0.5)
        if op == "norm_bwd":
            return dict(op=op, T=T, H=H, res=rng.choice(["bf16", "f32"]))
        return dict(op=op, T=T, H=H, pad=8 * rng.randrange(0, 65))
    K = 128 * _log(rng, 2, 64)
    N = 8 * _log(rng, 32, min(8192, 65536 * 2048 // K // 8))
    T = _log(rng, 1, max(1, min(16384, 16384 * 2048 * 4096 // (K * N))))
    return dict(op=op, T=T, K=K, N=N, fmt=rng.choice(["fp4", "fp8"]), x=rng.choice(["codes", "bf16"]))


def work(case):
    T = case["T"]
    if case["op"] == "linear":
        K, N = case["K"], case["N"]
        codes = K + K // 32 if case["fmt"] == "fp8" else K // 2 + K // 32
        x = 2 * K if case["x"] == "bf16" else codes
        return {"bytes": T * x + N * (K // 2 + K // 32) + 2 * T * N, "flops": 2 * T * K * N}
    H = case["H"]
    if case["op"] == "quant":
        return {"bytes": T * (2 * H + H + H // 32), "flops": 3 * T * H}
    r = 2 if case["res"] == "bf16" else 4
    if case["op"] == "norm":
        # x, residual, sum, codes, scales; the training form also y and rstd
        return {"bytes": T * (2 * H + 2 * r * H + H + H // 32 + (2 * H + 4 if case["train"] else 0)) + 2 * H,
                "flops": 7 * T * H}
    # dy, sum, the stream's gradient in and out, rstd; gamma and its gradient
    return {"bytes": T * (2 * H + 3 * r * H + 4) + 2 * H + 4 * H, "flops": 11 * T * H}


# ------------------------------------------------------------------ inputs
def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=F32)


def prepare(case, seed):
    g = _generator(seed)
    T, dev = case["T"], "cuda"
    empty = lambda dtype, *shape: torch.empty(*shape, dtype=dtype, device=dev)  # noqa: E731
    s = dict(case)
    if case["op"] == "linear":
        K, N = case["K"], case["N"]
        # activations with a few large channels, weights of the usual 0.02
        x = (_normal(g, T, K) * torch.exp(0.5 * _normal(g, K))).to(BF16)
        w = (0.02 * _normal(g, N, K)).to(BF16)
        wc, ws = _encode(w, "fp4")
        s["wq"] = dict(codes=wc, scales=ws)
        width = K if case["fmt"] == "fp8" else K // 2
        s["xq"] = dict(codes=empty(torch.uint8, T, width), scales=empty(torch.uint8, T, K // 32))
        if case["x"] == "codes":
            s["xq"]["codes"], s["xq"]["scales"] = _encode(x, case["fmt"])
        else:
            s["x"] = x
        s["y"] = empty(BF16, T, N)
        return s
    H = case["H"]
    if case["op"] == "quant":
        wide = (_normal(g, T, H + case["pad"]) * torch.exp(0.5 * _normal(g, H + case["pad"]))).to(BF16)
        s["x"] = wide[:, :H]
        s["out"] = dict(codes=empty(torch.uint8, T, H), scales=empty(torch.uint8, T, H // 32))
        return s
    rt = BF16 if case["res"] == "bf16" else F32
    # a residual stream a few times larger than a layer's output, with a few large channels
    channel = torch.exp(0.7 * _normal(g, H))
    stream = 3.0 * _normal(g, T, H) * channel
    s["gamma"] = (1.0 + 0.2 * _normal(g, H)).to(BF16)
    if case["op"] == "norm":
        s["x"], s["residual"] = _normal(g, T, H).to(BF16), stream.to(rt)
        s["out"] = dict(sum=empty(rt, T, H), codes=empty(torch.uint8, T, H), scales=empty(torch.uint8, T, H // 32))
        if case["train"]:
            s["out"].update(y=empty(BF16, T, H), rstd=empty(F32, T))
        return s
    s["sum"] = stream.to(rt)
    s["rstd"] = 1.0 / torch.sqrt(s["sum"].double().square().mean(1) + EPS).to(F32)
    s["dy"] = (0.01 * _normal(g, T, H)).to(BF16)
    s["dsum"] = (0.01 * _normal(g, T, H)).to(rt)
    s["out"] = dict(dres=empty(rt, T, H), dgamma=empty(F32, H))
    return s


# -------------------------------------------------------------- plain form
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _encode(x, fmt):
    """MX codes and scale bytes of the rows of x (bf16)."""
    R, K = x.shape
    v = x.to(F32).reshape(R, K // 32, 32)
    field = (v.abs().amax(2).view(torch.int32) >> 23) & 0xFF          # amax = 1.m 2^(field - 127)
    byte = torch.clamp(field - (8 if fmt == "fp8" else 2), min=0)
    q = v * ((254 - byte) << 23).view(F32)[..., None]                 # 2^-X, in its bits
    scales = byte.to(torch.uint8)
    if fmt == "fp8":
        codes = q.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
        return codes.reshape(R, K), scales
    a = q.abs()
    c = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    c = (c + 8 * torch.signbit(q).to(torch.uint8)).reshape(R, K // 2, 2)
    return c[..., 0] + 16 * c[..., 1], scales


def _decode(codes, scales, fmt):
    """The 32-bit values of MX rows."""
    R = codes.shape[0]
    if fmt == "fp8":
        v = codes.view(torch.float8_e4m3fn).to(F32)
    else:
        table = torch.tensor(E2M1 + tuple(-m for m in E2M1), dtype=F32, device=codes.device)
        v = torch.stack((table[(codes & 15).long()], table[(codes >> 4).long()]), -1)
    return (v.reshape(R, -1, 32) * scales.view(torch.float8_e8m0fnu).to(F32)[..., None]).reshape(R, -1)


def _values(codes, scales):
    return {"codes": codes.view(torch.float8_e4m3fn), "scales": scales.view(torch.float8_e8m0fnu)}


def _plain(s):
    op = s["op"]
    if op == "quant":
        return _values(*_encode(s["x"], "fp8"))
    if op == "linear":
        xc, xs = _encode(s["x"], s["fmt"]) if s["x"] != "codes" else (s["xq"]["codes"], s["xq"]["scales"])
        y = _decode(xc, xs, s["fmt"]) @ _decode(s["wq"]["codes"], s["wq"]["scales"], "fp4").t()
        return {"y": y.to(BF16)}
    gamma = s["gamma"].to(F32)
    if op == "norm":
        total = (s["x"].to(F32) + s["residual"].to(F32)).to(s["residual"].dtype)
        v = total.to(F32)
        rstd = 1.0 / torch.sqrt(v.square().mean(1) + EPS)
        y = (v * rstd[:, None] * gamma).to(BF16)
        out = {"sum": total, **_values(*_encode(y, "fp8"))}
        return {**out, "y": y, "rstd": rstd} if s["train"] else out
    v, dy = s["sum"].to(F32), s["dy"].to(F32)
    n = v * s["rstd"][:, None]
    dn = dy * gamma
    dres = s["rstd"][:, None] * (dn - n * (dn * n).mean(1, keepdim=True)) + s["dsum"].to(F32)
    return {"dres": dres.to(s["sum"].dtype), "dgamma": (dy * n).sum(0)}


# ------------------------------------------------------- the library's calls
def _own(s):
    from precision_rl_amd import binding as b

    op = s["op"]
    if op == "quant":
        q = b.w4a4_mx_quantize_rows(s["x"], b.MX_FP8, out=s["out"])
        return _values(q["codes"], q["scales"])
    if op == "linear":
        xq = s["xq"]
        if not isinstance(s["x"], str):
            xq = b.w4a4_mx_quantize_rows(s["x"], b.MX_FP8 if s["fmt"] == "fp8" else b.MX_FP4, out=xq)
        return {"y": b.w4a4_mx_linear_fwd(xq, s["wq"], s["T"], s["K"], s["N"], y=s["y"])}
    if op == "norm":
        r = b.w4a4_add_rmsnorm_fwd(s["x"], s["gamma"], EPS, residual=s["residual"], fmt=b.MX_FP8,
                                   y=s["train"], save=s["train"], out=s["out"])
        out = {"sum": r["sum"], **_values(r["codes"], r["scales"])}
        return {**out, "y": r["y"], "rstd": r["rstd"]} if s["train"] else out
    r = b.w4a4_add_rmsnorm_bwd(s["dy"], s["sum"], s["gamma"], s["rstd"], dsum=s["dsum"], out=s["out"])
    return {"dres": r["dres"], "dgamma": r["dgamma"]}


def run(state):
    return _own(state) if own else _plain(state)


# --------------------------------------------------- the definition in 64 bits
def _power(e):
    """2^e in 64 bits, for e above -1023."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _grid(a, low, bits):
    """|a| (64 bits) rounded to nearest even with `bits` fraction bits, exponents from `low` up."""
    _, e = torch.frexp(a)
    step = _power(torch.clamp(e - 1, min=low) - bits)
    return torch.round(a / step) * step


def _exact_block(x, fmt):
    """Element values (without the scale) and scales of the rows of x, in 64 bits."""
    v = x.double().reshape(x.shape[0], -1, 32)
    top = v.abs().amax(2)
    _, e = torch.frexp(top)
    X = torch.where(top > 0, (e - 1 - (8 if fmt == "fp8" else 2)).clamp(-127, 127), torch.full_like(e, -127))
    scale = _power(X)
    a = v.abs() / scale[..., None]
    m = _grid(a, -6, 3).clamp(max=448.0) if fmt == "fp8" else _grid(a, 0, 1).clamp(max=6.0)
    return torch.copysign(m, v).reshape(x.shape), scale


def _exact_bf16(v):
    return torch.copysign(_grid(v.abs(), -126, 7), v)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quant":
        codes, scales = _exact_block(s["x"], "fp8")
        return {"codes": codes, "scales": scales}
    if op == "linear":
        full = lambda m, c: (m.reshape(m.shape[0], -1, 32) * c[..., None]).reshape(m.shape)  # noqa: E731
        w64 = _decode(s["wq"]["codes"], s["wq"]["scales"], "fp4").double()
        if case["x"] == "bf16":
            x64 = full(*_exact_block(s["x"], case["fmt"]))
        else:
            x64 = _decode(s["xq"]["codes"], s["xq"]["scales"], case["fmt"]).double()
        return {"y": x64 @ w64.t()}
    gamma = s["gamma"].double()
    if op == "norm":
        total = s["x"].double() + s["residual"].double()
        total = _exact_bf16(total) if case["res"] == "bf16" else total.to(F32).double()
        rstd = (total.square().mean(1) + EPS).rsqrt()
        y = _exact_bf16(total * rstd[:, None] * gamma)
        codes, scales = _exact_block(y, "fp8")
        out = {"sum": total, "codes": codes, "scales": scales}
        return {**out, "y": y, "rstd": rstd} if case["train"] else out
    v, dy, r = s["sum"].double(), s["dy"].double(), s["rstd"].double()[:, None]
    inner = (dy * gamma * v).mean(1, keepdim=True)
    dres = r * gamma * dy - r.pow(3) * v * inner + s["dsum"].double()
    return {"dres": dres, "dgamma": (dy * v * r).sum(0)}
