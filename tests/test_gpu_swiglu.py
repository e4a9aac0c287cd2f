"""GPU parity of the SwiGLU with its MX output and 8-bit checkpoint, and of its
backward pass, with the float64 oracle.

Codes and scale bytes are compared byte for byte with the row quantiser's, on
the same bf16 values.  Bounds of the rest, with u = 2^-24 and results rounded
once to bf16 (at most half a step, 2^-8 of the value):
  e^-g    the argument's two roundings move the exponent by at most 2 u |g|
          (relative to the power), the hardware's exp2 adds 2 u
  s       that, the addition (u) and the hardware's reciprocal (2 u): relative
          e_s = (2 |g| + 5) u; where 1 + e^-g passes the format's range or its
          reciprocal the normal numbers, s is off by less than 2^-126 instead
  a, dup  two more products: (e_s + 2 u)
  dgate   f = 1 + g (1 - s) is off by |g| (s e_s + u) from s and 1 - s, and u
          (|g (1 - s)| + |f|) from its own product and sum; three products more
"""
import numpy as np
import pytest

from oracle import dispatch, mxfp4
from gpu_util import bf16_host, print_case, u8

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

U = 2.0 ** -24
STEP = torch.finfo(torch.bfloat16).eps / 2
TINY = 2.0 ** -126


@pytest.fixture(scope="module")
def b():
    from precision_rl_amd import binding
    return binding


def _dev(v):
    return torch.from_numpy(np.asarray(v, dtype=np.float32)).to(torch.bfloat16).cuda()


def _inputs(T, I, seed, spread=1.0):  # noqa: E741
    rng = np.random.default_rng(seed)
    h = rng.standard_normal((T, 2 * I)) * np.exp(spread * rng.standard_normal(2 * I))
    return _dev(h), _dev(0.1 * rng.standard_normal((T, I)))


def _check_a(a, h64):
    gate, up = np.split(h64, 2, axis=1)
    ref = dispatch.swiglu(h64)
    rel = (2 * np.abs(gate) + 7) * U * 1.01
    slack = TINY * (1 + np.abs(gate * up))
    assert np.all(np.abs(bf16_host(a) - ref) <= (STEP + rel) * np.abs(ref) * (1 + STEP) + slack)


def _check_dh(dh, da64, h64):
    gate, up = np.split(h64, 2, axis=1)
    s = dispatch.sigmoid(gate)
    dg, du = np.split(dispatch.swiglu_bwd(da64, h64), 2, axis=1)
    es = (2 * np.abs(gate) + 5) * U * 1.01
    f = 1 + gate * (1 - s)
    off = np.abs(da64 * up * s) * (np.abs(f) * (es + 4 * U) + np.abs(gate) * (s * es + 2 * U)) * 1.01
    slack = TINY * (1 + np.abs(da64 * up) * (1 + np.abs(gate)) + np.abs(da64 * gate))
    got_g, got_u = np.split(bf16_host(dh), 2, axis=1)
    assert np.all(np.abs(got_g - dg) <= STEP * np.abs(dg) + off * (1 + STEP) + slack)
    assert np.all(np.abs(got_u - du) <= (STEP + (es + 3 * U) * (1 + STEP)) * np.abs(du) + slack)


def _values(b, codes, scales):
    """The checkpoint's values in float64."""
    v = codes.view(torch.float8_e4m3fn).float().double().cpu().numpy()
    return mxfp4.mx8_values(v, u8(scales))


# one block, one row, rows that share a workgroup, rows longer than one, odd
# numbers of blocks, several workgroups with a row across their border
SHAPES = [(1, 32), (8, 768), (1, 4096), (3, 96), (61, 768), (17, 4128), (2, 8192), (700, 160), (1, 65536), (5001, 64)]


@pytest.mark.parametrize("T,I", SHAPES)
@pytest.mark.parametrize("fmt,checkpoint", [(None, True), ("fp8", False), ("fp4", True), ("fp8", True)])
def test_forward(b, T, I, fmt, checkpoint):  # noqa: E741
    h, _ = _inputs(T, I, T + I)
    f = {"fp8": b.MX_FP8, "fp4": b.MX_FP4, None: None}[fmt]
    print_case("swiglu_fwd", T=T, I=I, fmt=fmt, checkpoint=checkpoint)
    r = b.w4a4_swiglu_fwd(h, fmt=f, checkpoint=checkpoint)
    _check_a(r["a"], bf16_host(h))
    if fmt:
        q = b.w4a4_mx_quantize_rows(r["a"], f)
        assert torch.equal(r["codes"], q["codes"]) and torch.equal(r["scales"], q["scales"])
        alone = b.w4a4_swiglu_fwd(h, fmt=f, a=False)
        assert torch.equal(alone["codes"], r["codes"]) and "a" not in alone
    if checkpoint:
        q = b.w4a4_mx_quantize_rows(h, b.MX_FP8)
        assert torch.equal(r["h_codes"], q["codes"]) and torch.equal(r["h_scales"], q["scales"])
        alone = b.w4a4_swiglu_fwd(h, a=False, checkpoint=True)
        assert torch.equal(alone["h_codes"], r["h_codes"]) and torch.equal(alone["h_scales"], r["h_scales"])


@pytest.mark.parametrize("T,I", SHAPES)
@pytest.mark.parametrize("checkpoint", [True, False])
def test_backward(b, T, I, checkpoint):  # noqa: E741
    h, da = _inputs(T, I, T + I + 1)
    print_case("swiglu_bwd", T=T, I=I, checkpoint=checkpoint)
    kept = b.w4a4_swiglu_fwd(h, a=False, checkpoint=True) if checkpoint else h
    h64 = _values(b, kept["h_codes"], kept["h_scales"]) if checkpoint else bf16_host(h)
    r = b.w4a4_swiglu_bwd(da, kept, a=True)
    _check_a(r["a"], h64)
    _check_dh(r["dh"], bf16_host(da), h64)
    assert torch.equal(b.w4a4_swiglu_bwd(da, kept)["dh"], r["dh"])
    assert torch.equal(b.w4a4_swiglu_bwd(None, kept, a=True, dh=False)["a"], r["a"])


@pytest.mark.parametrize("I", [8, 24, 136, 1000])
def test_rows_of_eight_without_blocks(b, I):  # noqa: E741
    h, da = _inputs(9, I, I)
    print_case("swiglu_rows_of_eight", I=I)
    r = b.w4a4_swiglu_fwd(h)
    _check_a(r["a"], bf16_host(h))
    g = b.w4a4_swiglu_bwd(da, h, a=True)
    assert torch.equal(g["a"], r["a"])
    _check_dh(g["dh"], bf16_host(da), bf16_host(h))


@pytest.mark.parametrize("live", [0, 1, 33, 64, 100, -5])
def test_rows_behind_the_count_are_left(b, live):
    """T is a capacity: rows from min(T, count) on keep what they hold, and are not read."""
    T, I = 64, 288  # noqa: E741
    n = max(0, min(T, live))
    h, da = _inputs(T, I, live + 9)
    h[n:] = float("nan")
    print_case("swiglu_rows", T=T, I=I, live=live)
    count = torch.tensor([live], dtype=torch.int32, device="cuda")
    full = lambda v, *s, dtype=torch.uint8: torch.full(s, v, dtype=dtype, device="cuda")  # noqa: E731
    bf = torch.bfloat16
    out = dict(a=full(7.0, T, I, dtype=bf), codes=full(7, T, I), scales=full(7, T, I // 32), h_codes=full(7, T, 2 * I),
               h_scales=full(7, T, 2 * I // 32))
    r = b.w4a4_swiglu_fwd(h, fmt=b.MX_FP8, checkpoint=True, rows=count, out=out)
    ref = b.w4a4_swiglu_fwd(h[:n], fmt=b.MX_FP8, checkpoint=True)
    assert all(torch.equal(r[m][:n], ref[m]) and bool((r[m][n:] == 7).all()) for m in ref)
    out = dict(dh=full(7.0, T, 2 * I, dtype=bf), a=full(7.0, T, I, dtype=bf))
    for kept, some in ((dict(h_codes=r["h_codes"], h_scales=r["h_scales"]),
                        dict(h_codes=r["h_codes"][:n], h_scales=r["h_scales"][:n])), (h, h[:n])):
        g, gref = b.w4a4_swiglu_bwd(da, kept, a=True, rows=count, out=out), b.w4a4_swiglu_bwd(da[:n], some, a=True)
        assert all(torch.equal(g[m][:n], gref[m]) and bool((g[m][n:] == 7).all()) for m in gref)


def test_slices_and_in_place(b):
    T, I = 45, 160  # noqa: E741
    wide, da = _inputs(T, I + 16, 3)
    h = wide[:, 16:16 + 2 * I]
    da = da[:, :I].contiguous()
    print_case("swiglu_slices", T=T, I=I)
    r, d = b.w4a4_swiglu_fwd(h, checkpoint=True), b.w4a4_swiglu_fwd(h.contiguous(), checkpoint=True)
    assert all(torch.equal(r[m], d[m]) for m in d)
    g, gd = b.w4a4_swiglu_bwd(da, h, a=True), b.w4a4_swiglu_bwd(da, h.contiguous(), a=True)
    assert all(torch.equal(g[m], gd[m]) for m in gd)
    dense, over = h.contiguous(), da.clone()
    p = b.w4a4_swiglu_bwd(over, dense, a=True, out=dict(dh=dense, a=over))   # dh over h, a over da
    assert p["dh"] is dense and torch.equal(dense, gd["dh"]) and torch.equal(over, gd["a"])


def test_special_values(b):
    """Gates so large that the exponential overflows or vanishes, zeros of both
    signs; infinities and NaN as the formulas have them, in the checkpoint all
    over their block and nowhere else."""
    I = 64  # noqa: E741
    h = torch.ones(4, 2 * I, dtype=torch.bfloat16, device="cuda")
    gates = [-3.0e38, -1000.0, -100.0, -88.0, -0.0, 0.0, 88.0, 1000.0, 3.0e38]
    h[0, :9] = torch.tensor(gates, dtype=torch.bfloat16)
    h[1, 40] = float("nan")
    h[2, I + 3] = float("inf")
    h[3, :9] = torch.tensor(gates, dtype=torch.bfloat16)
    h[3, I:I + 9] = -0.0
    print_case("swiglu_special", I=I)
    r = b.w4a4_swiglu_fwd(h, checkpoint=True)
    a = r["a"].float().cpu()
    assert torch.isfinite(a[0]).all() and torch.isnan(a[1, 40]) and torch.isinf(a[2, 3])
    assert a[0, 4] == 0 and torch.signbit(a[0, 4])
    _check_a(r["a"][:1], bf16_host(h[:1]))
    kept = {m: r[m] for m in ("h_codes", "h_scales")}
    assert u8(r["h_scales"])[1, 1] == 255 and u8(r["h_scales"])[2, 2] == 255
    da = torch.ones(4, I, dtype=torch.bfloat16, device="cuda")
    g = b.w4a4_swiglu_bwd(da, kept, a=True)
    nan = torch.isnan(g["a"].cpu())
    want = torch.zeros(4, I, dtype=torch.bool)
    want[1, 32:] = True
    want[2, :32] = True
    assert torch.equal(nan, want)
    dh = torch.isnan(g["dh"].cpu())
    assert torch.equal(dh[:, :I], want)                       # dgate reads gate and up
    want[2] = False
    assert torch.equal(dh[:, I:], want)                       # dup reads gate alone
    g = b.w4a4_swiglu_bwd(da[:1], h[:1], a=True)
    _check_dh(g["dh"], bf16_host(da[:1]), bf16_host(h[:1]))


def test_factors_whose_product_passes_the_range(b):
    """da up and da gate beyond 2^128 where the sigmoid is 0 or the result moderate."""
    I = 32  # noqa: E741
    h = torch.zeros(1, 2 * I, dtype=torch.bfloat16, device="cuda")
    h[0, :4] = torch.tensor([-1000.0, -1.0e30, -2.0, 2.0])
    h[0, I:I + 4] = torch.tensor([1.0e30, 1.0e30, 1.0e30, 1.0e-30])
    da = torch.zeros(1, I, dtype=torch.bfloat16, device="cuda")
    da[0, :4] = torch.tensor([1.0e30, 1.0e30, 1.0e-20, 1.0e30])
    print_case("swiglu_range", I=I)
    dh = b.w4a4_swiglu_bwd(da, h)["dh"]
    assert bool(torch.isfinite(dh).all()) and not dh[0, :2].any() and not dh[0, I:I + 2].any()
    _check_dh(dh[:, [2, 3, I + 2, I + 3]], bf16_host(da[:, 2:4]), bf16_host(h[:, [2, 3, I + 2, I + 3]]))


def test_smallest_scales(b):
    """Blocks near the bottom of the format: scale bytes 0 and 1, subnormal bf16."""
    I = 32  # noqa: E741
    h = torch.zeros(6, 2 * I, dtype=torch.bfloat16, device="cuda")
    bits = h.view(torch.int16)
    for r, top in enumerate((1, 0x7F, 0x80, 0x47F, 0x480, 0x500)):
        bits[r, I:] = (torch.arange(32, device="cuda") * top // 31).to(torch.int16)
    h[:, :I] = 1.0
    print_case("swiglu_smallest", I=I)
    r = b.w4a4_swiglu_fwd(h, checkpoint=True)
    v = _values(b, r["h_codes"], r["h_scales"])
    assert set(u8(r["h_scales"])[:, 1]) >= {0, 1}
    g = b.w4a4_swiglu_bwd(torch.ones(6, I, dtype=torch.bfloat16, device="cuda"), r, a=True)
    s = dispatch.sigmoid(1.0)
    dg = bf16_host(g["dh"])[:, :I]
    ref = v[:, I:] * s * (1 + 1 - s)
    assert np.all(np.abs(dg - ref) <= STEP * np.abs(ref) + 20 * U * np.abs(ref) + 2.0 ** -133)


def test_empty_batch(b):
    e = torch.empty(0, 128, dtype=torch.bfloat16, device="cuda")
    print_case("swiglu_empty")
    r = b.w4a4_swiglu_fwd(e, fmt=b.MX_FP8, checkpoint=True)
    assert r["a"].shape == (0, 64) and r["h_codes"].shape == (0, 128)
    assert b.w4a4_swiglu_bwd(e[:, :64].contiguous(), r, a=True)["dh"].shape == (0, 128)


def test_gradient_against_differences(b):
    """Against central differences of the float64 formula at the checkpoint's
    values: the GPU gradient, off by at most 2^-7 of the sum of magnitudes."""
    T, I = 13, 96  # noqa: E741
    h, da = _inputs(T, I, 21, spread=0.3)
    print_case("swiglu_differences", T=T, I=I)
    kept = b.w4a4_swiglu_fwd(h, checkpoint=True)
    v = _values(b, kept["h_codes"], kept["h_scales"])
    d64, dh = bf16_host(da), bf16_host(b.w4a4_swiglu_bwd(da, kept)["dh"])
    rng = np.random.default_rng(2)
    for _ in range(4):
        w, eps = rng.standard_normal(v.shape), 1e-5
        diff = np.sum(d64 * (dispatch.swiglu(v + eps * w) - dispatch.swiglu(v - eps * w))) / (2 * eps)
        assert abs(np.sum(dh * w) - diff) <= 2.0 ** -7 * np.sum(np.abs(dh * w))


def test_rows_beyond_4_gib(b):
    T, I = 300_000, 4096  # noqa: E741
    print_case("swiglu_large", T=T, I=I)
    g = torch.Generator(device="cuda").manual_seed(3)
    h = torch.randn(T, 2 * I, generator=g, device="cuda", dtype=torch.bfloat16)
    da = torch.randn(T, I, generator=g, device="cuda", dtype=torch.bfloat16)
    r = b.w4a4_swiglu_fwd(h, checkpoint=True)
    d = b.w4a4_swiglu_bwd(da, r)["dh"]
    for rows in (slice(0, 3), slice(131071, 131074), slice(T - 3, T)):
        ref = b.w4a4_swiglu_fwd(h[rows].clone(), checkpoint=True)
        assert all(torch.equal(r[m][rows], ref[m]) for m in ref)
        assert torch.equal(d[rows], b.w4a4_swiglu_bwd(da[rows].clone(), ref)["dh"])


def test_captured_graph_and_other_stream(b):
    T, I = 300, 224  # noqa: E741
    h, da = _inputs(T, I, 30)
    print_case("swiglu_graph", T=T, I=I)

    def step(h, da):
        r = b.w4a4_swiglu_fwd(h, fmt=b.MX_FP8, checkpoint=True)
        return r, b.w4a4_swiglu_bwd(da, r, a=True, out=dict(a=torch.empty_like(da)))

    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        step(h, da)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r, g = step(h, da)
    for n in range(3):
        nh, nda = _inputs(T, I, 31 + n)
        h.copy_(nh)
        da.copy_(nda)
        graph.replay()
        with torch.cuda.stream(stream):
            stream.wait_stream(torch.cuda.default_stream())
            er, eg = step(nh, nda)
        torch.cuda.synchronize()
        assert all(torch.equal(r[m], er[m]) for m in er) and all(torch.equal(g[m], eg[m]) for m in eg)


def test_dense_layer(b):
    """Norm, gate and up projection, SwiGLU with codes and checkpoint, down
    projection; backward from the checkpoint: the composition's bytes are those
    of the single calls, and the gradients come near the bf16 checkpoint's."""
    T, H, I = 96, 512, 768  # noqa: E741
    rng = np.random.default_rng(40)
    x, gamma = _dev(rng.standard_normal((T, H))), _dev(np.ones(H))
    wgu, wd = _dev(0.05 * rng.standard_normal((2 * I, H))), _dev(0.05 * rng.standard_normal((H, I)))
    dy = _dev(0.1 * rng.standard_normal((T, H)))
    print_case("dense_layer", T=T, H=H, I=I)
    guq, dq = b.w4a4_mx_quantize_rows(wgu, b.MX_FP4), b.w4a4_mx_quantize_rows(wd, b.MX_FP4)
    n = b.w4a4_add_rmsnorm_fwd(x, gamma, fmt=b.MX_FP8, save=True,
                               out=dict(offsets=torch.empty(2, dtype=torch.int32, device="cuda")))
    h = b.w4a4_mx_linear_fwd(n, guq, T, H, 2 * I)
    s = b.w4a4_swiglu_fwd(h, fmt=b.MX_FP8, checkpoint=True)
    y = b.w4a4_mx_linear_fwd(s, dq, T, I, H)
    assert torch.equal(y, b.w4a4_mx_linear_fwd(b.w4a4_mx_quantize_rows(s["a"], b.MX_FP8), dq, T, I, H))

    def backward(kept):
        a = b.w4a4_swiglu_bwd(None, kept, a=True, dh=False)["a"]
        down = b.w4a4_linear_bwd(dy, a, wd, n, T, I, H)
        dh = b.w4a4_swiglu_bwd(down["dx"], kept)["dh"]
        up = b.w4a4_linear_bwd(dh, n["y"], wgu, n, T, H, 2 * I)
        g = b.w4a4_add_rmsnorm_bwd(up["dx"], x, gamma, n["rstd"])
        return dict(dx=g["dres"], dgamma=g["dgamma"], dgu=up["dw"], dd=down["dw"])

    exact, kept = backward(h), backward({m: s[m] for m in ("h_codes", "h_scales")})
    for m in exact:
        assert float((kept[m].double() - exact[m].double()).norm() / exact[m].double().norm()) < 0.06, m


def test_refusals(b):
    h, da = _inputs(4, 64, 50)
    kept = b.w4a4_swiglu_fwd(h, checkpoint=True)
    for call in (lambda: b.w4a4_swiglu_fwd(h.float()), lambda: b.w4a4_swiglu_fwd(h[0]), lambda: b.w4a4_swiglu_fwd(h.cpu()),
                 lambda: b.w4a4_swiglu_fwd(h[:, :127]), lambda: b.w4a4_swiglu_fwd(h[:, :80], checkpoint=True),
                 lambda: b.w4a4_swiglu_fwd(h, a=False), lambda: b.w4a4_swiglu_fwd(h, fmt=7),
                 lambda: b.w4a4_swiglu_fwd(h, rows=torch.tensor([3], device="cuda")),
                 lambda: b.w4a4_swiglu_fwd(h, out=dict(a=da.float())), lambda: b.w4a4_swiglu_bwd(da, h.float()),
                 lambda: b.w4a4_swiglu_bwd(da[:3], h), lambda: b.w4a4_swiglu_bwd(None, h),
                 lambda: b.w4a4_swiglu_bwd(da, h, dh=False), lambda: b.w4a4_swiglu_bwd(da.float(), kept),
                 lambda: b.w4a4_swiglu_bwd(da, dict(kept, h_scales=kept["h_scales"][:3])),
                 lambda: b.w4a4_swiglu_bwd(da, h, out=dict(dh=kept["a"]))):
        with pytest.raises(b.W4A4Error):
            call()
