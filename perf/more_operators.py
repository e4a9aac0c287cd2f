"""Cases of the operators around the experts' products: tokens sorted by expert
and back with the router's weights applied, both with their gradients, and the
SwiGLU whose input is kept in 8 bits for its backward pass.

Dispatch.  Slot j of token t goes to expert e = topk_idx[t, j].  The rows of one
expert are consecutive, in ascending order of t * k + j, and each expert's group
is padded to a multiple of `align` with rows of zeros.  An id outside [0, E) is
a slot that is not dispatched: the expert is another rank's.

    permute     xp[row_map[t, j]] = x[t]              its gradient  dx[t] = sum_j dxp[row_map[t, j]]
    unpermute   y[t] = sum_j w[t, j] o[row_map[t, j]] its gradient  do[row_map[t, j]] = w[t, j] dy[t]
                                                                    dw[t, j] = <dy[t], o[row_map[t, j]]>

SwiGLU of h = (gate, up): a = gate s up with s = sigmoid(gate); the checkpoint of
h is MXFP8 (OCP Microscaling v1.0: blocks of 32 elements share the scale 2^X,
X = floor(log2 amax) - 8, stored as the byte X + 127; elements E4M3, rounded to
nearest even, saturating).  The backward pass computes from the checkpoint's
values: dgate = da up s (1 + gate (1 - s)), dup = da gate s, and a once more.

``run`` is either the operators' plain form (elementary torch operations) or,
with ``own`` set, the calls a program makes of the library.  What is held in
8 bits comes back as torch's 8-bit floating types.  Rows behind the last one in
use are the state's own zeros on both sides.
"""
import math

import torch

if not hasattr(torch, "float8_e8m0fnu"):
    raise ImportError("torch with the 8-bit floating types is needed")

own = False

BF16, F32, F64, I32 = torch.bfloat16, torch.float32, torch.float64, torch.int32
TYPES = {"bf16": BF16, "f32": F32}
MOST = 131072 * 2048 * 2          # bytes of the largest listed case's expert rows


# ------------------------------------------------------------------- cases
def _moe(name, op, T, H=2048, E=128, k=8, ep=1, align=1, dtype="bf16"):
    return dict(name=name, op=op, T=T, H=H, E=E, k=k, ep=ep, align=align, dtype=dtype)


def _ffn(name, op, T, width, spare=0, ckpt=True, fmt="none"):
    return dict(name=name, op=op, T=T, I=width, spare=spare, ckpt=ckpt, fmt=fmt)


def listed():
    return [
        # one token of a decoding step to its eight experts
        _moe("dispatch_decode", "permute", 1),
        # the learner's batch (16384 tokens, hidden 2048, 128 experts, top 8)
        _moe("dispatch_learner", "permute", 16384),
        # gradient of a micro-batch's dispatch
        _moe("dispatch_grad_micro", "permute_grad", 61),
        # gradient in 32 bits on one of four ranks, a ragged batch and groups of 128 rows
        _moe("dispatch_grad_ragged", "permute_grad", 4097, H=4096, ep=4, E=32, align=128, dtype="f32"),
        # 48 sequences decoding
        _moe("combine_decode", "unpermute", 48),
        # the learner's batch back to token order
        _moe("combine_learner", "unpermute", 16384),
        # a micro-batch's gradients, groups of 16 rows
        _moe("combine_grad_micro", "unpermute_grad", 61, align=16),
        # the learner's gradients, the router weights' among them
        _moe("combine_grad_learner", "unpermute_grad", 16384),
        # a decoding token's eight expert rows, with codes for the next product
        _ffn("swiglu_decode", "swiglu", 8, 768, ckpt=False, fmt="fp8"),
        # the learner's expert rows, with the checkpoint for the backward pass
        _ffn("swiglu_learner", "swiglu", 131072, 768),
        # backward of a ragged batch of a dense layer
        _ffn("swiglu_grad_ragged", "swiglu_grad", 5001, 2048),
        # backward of the learner's expert rows from the checkpoint
        _ffn("swiglu_grad_learner", "swiglu_grad", 131072, 768),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(["permute", "permute_grad", "unpermute", "unpermute_grad", "swiglu", "swiglu_grad"])
    if op.startswith("swiglu"):
        width = 32 * _log(rng, 2, 256)
        T = _log(rng, 1, min(131072, 131072 * 768 // width))
        spare = rng.choice([0, 0, _log(rng, 1, 512)])
        if op == "swiglu":
            return dict(op=op, T=T, I=width, spare=spare, ckpt=rng.random() < 0.7, fmt=rng.choice(["none", "fp8"]))
        return dict(op=op, T=T, I=width, spare=spare, ckpt=rng.random() < 0.7, fmt="none")
    dtype = rng.choice(["bf16", "bf16", "f32"])
    H = 8 * _log(rng, 8, 1024)
    k = rng.randint(1, 8)
    E = _log(rng, k, 512)
    align = rng.choice([1, 1, 16, 32, 64, 128])
    row = H * (2 if dtype == "bf16" else 4)
    if E * (align - 1) * row > MOST // 2:
        align = 1
    T = _log(rng, 1, min(16384, max(1, (MOST // row - E * (align - 1)) // k)))
    return dict(op=op, T=T, H=H, E=E, k=k, ep=rng.choice([1, 1, 4]), align=align, dtype=dtype)


def work(case):
    T = case["T"]
    if case["op"].startswith("swiglu"):
        I = case["I"]  # noqa: E741
        kept = 2 * I + 2 * I // 32 if case["ckpt"] else 4 * I
        if case["op"] == "swiglu":
            out = 2 * I + (kept if case["ckpt"] else 0) + (I + I // 32 if case["fmt"] == "fp8" else 0)
            return {"bytes": T * (4 * I + out), "flops": 6 * T * I}
        return {"bytes": T * (2 * I + kept + 4 * I + 2 * I), "flops": 14 * T * I}
    k, ep = case["k"], case["ep"]
    row = case["H"] * (2 if case["dtype"] == "bf16" else 4)
    n = -(-T * k // ep)                                       # slots that this rank's experts take
    tokens = T * (1 - (1 - 1 / ep) ** k) if ep > 1 else T     # tokens with one of them
    if case["op"] == "permute":
        return {"bytes": tokens * row + n * row + 8 * T * k + 4 * n + 4 * (case["E"] + 1), "flops": T * k}
    if case["op"] == "permute_grad":
        return {"bytes": n * row + T * row + 4 * T * k, "flops": n * case["H"]}
    if case["op"] == "unpermute":
        return {"bytes": n * row + T * row + 8 * T * k, "flops": 2 * n * case["H"]}
    return {"bytes": 2 * n * row + tokens * row + 12 * T * k, "flops": 3 * n * case["H"]}


# ------------------------------------------------------------------ inputs
def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=F32)


def _capacity(case):
    return case["T"] * case["k"] + case["E"] * (case["align"] - 1)


def prepare(case, seed):
    g, dev = _generator(seed), "cuda"
    zeros = lambda dtype, *shape: torch.zeros(*shape, dtype=dtype, device=dev)  # noqa: E731
    s, T = dict(case), case["T"]
    if case["op"].startswith("swiglu"):
        I, R = case["I"], T + case["spare"]  # noqa: E741
        # pre-activations with a few large channels
        h = (_normal(g, R, 2 * I) * torch.exp(0.5 * _normal(g, 2 * I))).to(BF16)
        s["rows"] = torch.tensor([T], dtype=I32, device=dev) if case["spare"] else None
        if case["op"] == "swiglu":
            s["h"] = h
            s["out"] = dict(a=zeros(BF16, R, I))
            if case["ckpt"]:
                s["out"].update(h_codes=zeros(torch.uint8, R, 2 * I), h_scales=zeros(torch.uint8, R, 2 * I // 32))
            if case["fmt"] == "fp8":
                s["out"].update(codes=zeros(torch.uint8, R, I), scales=zeros(torch.uint8, R, I // 32))
            return s
        s["h"] = dict(zip(("h_codes", "h_scales"), _encode(h))) if case["ckpt"] else h
        s["da"] = (0.01 * _normal(g, R, I)).to(BF16)
        s["out"] = dict(dh=zeros(BF16, R, 2 * I), a=zeros(BF16, R, I))
        return s
    H, E, k, ep, dt = case["H"], case["E"], case["k"], case["ep"], TYPES[case["dtype"]]
    # a router over the experts of all ranks, some of them more popular; this rank's are the first E
    score = _normal(g, T, E * ep) + 0.7 * _normal(g, E * ep)
    top, idx = torch.topk(score, k, dim=1)
    s["topk_w"] = torch.softmax(top, 1)
    s["topk_idx"] = torch.where(idx < E, idx, torch.full_like(idx, -1)).to(I32)
    cap = _capacity(case)
    if case["op"] == "permute":
        s["x"] = _normal(g, T, H).to(dt)
        s["out"] = dict(xp=zeros(dt, cap, H), offsets=zeros(I32, E + 1), row_map=zeros(I32, T, k),
                        src_row=zeros(I32, cap))
        return s
    s["maps"] = _maps(s)
    if case["op"] == "permute_grad":
        s["dxp"] = (0.01 * _normal(g, cap, H)).to(dt)
        s["dx"] = zeros(dt, T, H)
        return s
    s["o"] = (0.3 * _normal(g, cap, H)).to(dt)
    if case["op"] == "unpermute":
        s["y"] = zeros(dt, T, H)
        return s
    s["dy"] = (0.01 * _normal(g, T, H)).to(dt)
    s["out"] = dict(do=zeros(dt, cap, H), dtopk_w=zeros(F32, T, k))
    return s


# -------------------------------------------------------------- plain form
def _maps(s):
    """offsets, row_map and src_row of the dispatch."""
    idx, E, align, k = s["topk_idx"], s["E"], s["align"], s["k"]
    cap, n, dev = _capacity(s), idx.numel(), idx.device
    key = idx.reshape(-1).long()
    key = torch.where((key >= 0) & (key < E), key, torch.full_like(key, E))
    order = torch.argsort(key, stable=True)
    count = torch.zeros(E + 1, dtype=torch.long, device=dev).index_add_(0, key, torch.ones_like(key))
    padded = (count[:E] + align - 1) // align * align
    offsets = torch.cat((padded.new_zeros(1), padded.cumsum(0)))
    start = torch.cat((count.new_zeros(1), count.cumsum(0)))            # without the padding
    by = key[order]
    row = offsets[by] + torch.arange(n, device=dev) - start[by]
    live = by < E
    row_map = torch.empty(n, dtype=torch.long, device=dev)
    row_map[order] = torch.where(live, row, torch.full_like(row, -1))
    src = torch.where(torch.arange(cap + 1, device=dev) < offsets[E], -1, 0)
    src[torch.where(live, row, torch.full_like(row, cap))] = torch.div(order, k, rounding_mode="floor")
    return dict(offsets=offsets.to(I32), row_map=row_map.reshape(idx.shape).to(I32), src_row=src[:cap].to(I32))


def _encode(x):
    """MXFP8 codes and scale bytes of the rows of x (bf16)."""
    R, K = x.shape
    v = x.to(F32).reshape(R, K // 32, 32)
    field = (v.abs().amax(2).view(I32) >> 23) & 0xFF                    # amax = 1.m 2^(field - 127)
    byte = torch.clamp(field - 8, min=0)
    q = (v * ((254 - byte) << 23).view(F32)[..., None]).clamp(-448.0, 448.0)
    return q.to(torch.float8_e4m3fn).view(torch.uint8).reshape(R, K), byte.to(torch.uint8)


def _decode(codes, scales):
    v = codes.view(torch.float8_e4m3fn).to(F32)
    return (v.reshape(v.shape[0], -1, 32) * scales.view(torch.float8_e8m0fnu).to(F32)[..., None]).reshape(v.shape)


def _values(codes, scales):
    return codes.view(torch.float8_e4m3fn), scales.view(torch.float8_e8m0fnu)


def _gathered(s, rows):
    """The rows of each token's slots in 32 bits [T, k, H], zeros for slots that are not dispatched."""
    at = s["maps"]["row_map"]
    v = rows[at.clamp(min=0).long()].to(F32)
    return torch.where((at >= 0)[..., None], v, 0.0) if s["ep"] > 1 else v


def _all_rows(s, v):
    """v [T, ...] with the spare rows' zeros behind it."""
    return torch.cat((v, v.new_zeros(s["spare"], *v.shape[1:]))) if s["spare"] else v


def _plain(s):
    op, T = s["op"], s["T"]
    if op == "permute":
        m = _maps(s)
        cap = _capacity(s)
        xp = torch.zeros(cap + 1, s["H"], dtype=s["x"].dtype, device=s["x"].device)
        to = torch.where(m["row_map"] >= 0, m["row_map"], cap).long()
        xp[to] = s["x"][:, None, :].expand(T, s["k"], s["H"])
        xp[cap] = 0
        return {"xp": xp[:cap], **m}
    if op == "permute_grad":
        return {"dx": _gathered(s, s["dxp"]).sum(1).to(s["dxp"].dtype)}
    if op == "unpermute":
        return {"y": (_gathered(s, s["o"]) * s["topk_w"][..., None]).sum(1).to(s["o"].dtype)}
    if op == "unpermute_grad":
        at, cap, dy = s["maps"]["row_map"], s["o"].shape[0], s["dy"].to(F32)
        dw = (_gathered(s, s["o"]) * dy[:, None, :]).sum(2)
        do = torch.zeros(cap + 1, s["H"], dtype=s["o"].dtype, device=dy.device)
        do[torch.where(at >= 0, at, cap).long()] = (s["topk_w"][..., None] * dy[:, None, :]).to(s["o"].dtype)
        do[cap] = 0
        return {"do": do[:cap], "dtopk_w": dw}
    I = s["I"]  # noqa: E741
    if op == "swiglu":
        h = s["h"][:T]
        v = h.to(F32)
        a = (v[:, :I] * torch.sigmoid(v[:, :I]) * v[:, I:]).to(BF16)
        out = {"a": _all_rows(s, a)}
        if s["ckpt"]:
            out["h_codes"], out["h_scales"] = _values(*(_all_rows(s, t) for t in _encode(h)))
        if s["fmt"] == "fp8":
            out["codes"], out["scales"] = _values(*(_all_rows(s, t) for t in _encode(a)))
        return out
    kept = s["h"]
    v = _decode(kept["h_codes"][:T], kept["h_scales"][:T]) if s["ckpt"] else kept[:T].to(F32)
    gate, up, da = v[:, :I], v[:, I:], s["da"][:T].to(F32)
    sg = torch.sigmoid(gate)
    dh = torch.cat((da * up * sg * (1.0 + gate * (1.0 - sg)), da * gate * sg), 1).to(BF16)
    return {"dh": _all_rows(s, dh), "a": _all_rows(s, (gate * sg * up).to(BF16))}


# ------------------------------------------------------- the library's calls
def _own(s):
    from precision_rl_amd import binding as b

    op = s["op"]
    if op == "permute":
        r = b.w4a4_permute_fwd(s["x"], s["topk_idx"], s["E"], s["align"], out=s["out"])
        return {n: r[n] for n in ("xp", "offsets", "row_map", "src_row")}
    if op == "permute_grad":
        return {"dx": b.w4a4_permute_bwd(s["dxp"], s["maps"], dx=s["dx"])}
    if op == "unpermute":
        return {"y": b.w4a4_unpermute_fwd(s["o"], s["maps"], s["topk_w"], y=s["y"])}
    if op == "unpermute_grad":
        r = b.w4a4_unpermute_bwd(s["dy"], s["o"], s["maps"], s["topk_w"], out=s["out"])
        return {"do": r["do"], "dtopk_w": r["dtopk_w"]}
    if op == "swiglu":
        r = b.w4a4_swiglu_fwd(s["h"], fmt=b.MX_FP8 if s["fmt"] == "fp8" else None, checkpoint=s["ckpt"],
                              rows=s["rows"], out=s["out"])
        out = {"a": r["a"]}
        if s["ckpt"]:
            out["h_codes"], out["h_scales"] = _values(r["h_codes"], r["h_scales"])
        if s["fmt"] == "fp8":
            out["codes"], out["scales"] = _values(r["codes"], r["scales"])
        return out
    r = b.w4a4_swiglu_bwd(s["da"], s["h"], a=True, rows=s["rows"], out=s["out"])
    return {"dh": r["dh"], "a": r["a"]}


def run(state):
    return _own(state) if own else _plain(state)


# --------------------------------------------------- the definition in 64 bits
def _power(e):
    """2^e in 64 bits, for e above -1023."""
    return ((e.long() + 1023) << 52).view(F64)


def _round_to(a, low, bits):
    """|a| (64 bits) rounded to nearest even with `bits` fraction bits, exponents from `low` up."""
    _, e = torch.frexp(a)
    step = _power(torch.clamp(e - 1, min=low) - bits)
    return torch.round(a / step) * step


def _exact_block(v):
    """Element values (without the scale) and scales of the MXFP8 rows of v, in 64 bits."""
    w = v.reshape(v.shape[0], -1, 32)
    top = w.abs().amax(2)
    _, e = torch.frexp(top)
    X = torch.where(top > 0, (e - 9).clamp(-127, 127), torch.full_like(e, -127))
    scale = _power(X)
    m = _round_to(w.abs() / scale[..., None], -6, 3).clamp(max=448.0)
    return torch.copysign(m, w).reshape(v.shape), scale


def _exact_swiglu(s):
    T, I = s["T"], s["I"]  # noqa: E741
    behind = lambda v: torch.cat((v, v.new_zeros(s["spare"], v.shape[1])))  # noqa: E731
    # zero bytes of a scale stand for 2^-127
    scales = lambda v: torch.cat((v, torch.full_like(v[:1], 2.0 ** -127).expand(s["spare"], -1)))  # noqa: E731
    if s["op"] == "swiglu":
        h = s["h"][:T].double()
        a = h[:, :I] / (1.0 + torch.exp(-h[:, :I])) * h[:, I:]
        out = {"a": behind(a)}
        if s["ckpt"]:
            c, x = _exact_block(h)
            out["h_codes"], out["h_scales"] = behind(c), scales(x)
        if s["fmt"] == "fp8":
            c, x = _exact_block(torch.copysign(_round_to(a.abs(), -126, 7), a))
            out["codes"], out["scales"] = behind(c), scales(x)
        return out
    if s["ckpt"]:
        c = s["h"]["h_codes"][:T].view(torch.float8_e4m3fn).double().reshape(T, -1, 32)
        h = (c * _power(s["h"]["h_scales"][:T].long() - 127)[..., None]).reshape(T, 2 * I)
    else:
        h = s["h"][:T].double()
    gate, up, da = h[:, :I], h[:, I:], s["da"][:T].double()
    sig = 1.0 / (1.0 + torch.exp(-gate))
    silu = gate * sig
    return {"dh": behind(torch.cat((da * up * (sig + silu * (1.0 - sig)), da * silu), 1)), "a": behind(silu * up)}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op.startswith("swiglu"):
        return _exact_swiglu(s)
    if op == "permute":
        # expert by expert: its slots in flat order, then the padding
        idx, x, k, align = s["topk_idx"].cpu().reshape(-1), s["x"].double(), case["k"], case["align"]
        xp = torch.zeros(_capacity(case), case["H"], dtype=F64, device=x.device)
        at = 0
        for e in range(case["E"]):
            tokens = torch.nonzero(idx == e)[:, 0] // k
            xp[at:at + len(tokens)] = x[tokens.to(x.device)]
            at += -(-len(tokens) // align) * align
        return {"xp": xp, "offsets": None, "row_map": None, "src_row": None}
    at = s["maps"]["row_map"].long()
    rows = s["dxp"] if op == "permute_grad" else s["o"]
    total, dw = torch.zeros(case["T"], case["H"], dtype=F64, device=rows.device), []
    do = torch.zeros(*rows.shape, dtype=F64, device=rows.device) if op == "unpermute_grad" else None
    for j in range(case["k"]):
        here = at[:, j] >= 0
        r = at[here, j]
        if op == "unpermute_grad":
            dy = s["dy"][here].double()
            do[r] = s["topk_w"][here, j].double()[:, None] * dy
            dw.append(torch.zeros(case["T"], dtype=F64, device=rows.device))
            dw[-1][here] = (dy * rows[r].double()).sum(1)
        else:
            w = s["topk_w"][here, j].double()[:, None] if op == "unpermute" else 1.0
            total[here] += w * rows[r].double()
    if op == "unpermute_grad":
        return {"do": do, "dtopk_w": torch.stack(dw, 1)}
    return {"dx" if op == "permute_grad" else "y": total}
