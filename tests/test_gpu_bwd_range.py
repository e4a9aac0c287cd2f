"""The SwiGLU backward inside the expert backwards where da up or da gate alone
passes the range and the sigmoid makes the result 0: as by itself
(w4a4_swiglu_bwd), no NaN."""
import pytest

from gpu_util import print_case

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

T, H, I, E, k, ALIGN = 128, 256, 256, 1, 1, 128  # noqa: E741


@pytest.fixture(scope="module")
def b():
    from precision_rl_amd import binding
    return binding


@pytest.fixture(scope="module")
def layer(b):
    """One token whose gradient of a is 2^100 in two features, with gates of -960 and -2^100 and up projections
    of 2^100 there, each in a block of 32 of its own; the products pass 2^128, the sigmoids are 0."""
    z = lambda *shape: torch.zeros(*shape, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    w1 = torch.randn(E, 2 * I, H, generator=g, device="cuda").bfloat16()
    cap = b.rows_capacity(T, k, E, ALIGN)
    w2, dy, h = z(E, H, I), z(T, H), z(cap, 2 * I)
    dy[5, 0] = 2.0 ** 67
    for col, gate in ((3, -960.0), (40, -2.0 ** 100)):
        w2[0, 0, col] = 2.0 ** 33
        h[5, col], h[5, I + col] = gate, 2.0 ** 100
    ids = torch.zeros(T, k, dtype=torch.int32, device="cuda")
    p = torch.ones(T, k, device="cuda")
    xq = b.w4a4_quantize_permute(x, ids, E, ALIGN)
    kept = b.w4a4_swiglu_fwd(h, checkpoint=True)
    da = z(cap, I)
    da[5, 3] = da[5, 40] = 2.0 ** 100
    assert bool(torch.isfinite(kept["a"]).all()) and not b.w4a4_swiglu_bwd(da, h)["dh"].any()
    assert not b.w4a4_swiglu_bwd(da, kept)["dh"].any()
    return dict(args=(dy, x, w1, w2), h=h, a=kept["a"], kept=kept, p=p, xq=xq)


@pytest.mark.parametrize("call", ["bf16", "checkpoint", "mxfp8"])
def test_factors_whose_product_passes_the_range(b, layer, call):
    L, sizes = layer, (T, H, I, E, k, ALIGN)
    print_case("expert_bwd_range", call=call)
    if call == "checkpoint":
        g = b.w4a4_expert_bwd_ckpt(*L["args"], L["kept"], L["p"], L["xq"], *sizes)
    else:
        bwd = b.w4a4_expert_bwd if call == "bf16" else b.w4a4_mx8_expert_bwd
        g = bwd(*L["args"], L["h"], L["a"], L["p"], L["xq"], *sizes)
    # dh is 0 everywhere, so are dx and dw1; a is 0 in the token's row, so is dw2
    for m in ("dx", "dw1", "dw2"):
        assert bool(torch.isfinite(g[m]).all()) and not g[m].any(), m


def test_a_factor_at_the_end_of_the_range(b):
    """up of the type's largest value where s (1 + gate (1 - s)) is 1.0998, its most: 0 for a da of 0, and no
    infinity where the result has none (a quarter of it: 9.3e37 +- 2^-8 of itself and FP32 roundings)."""
    I, top = 32, torch.finfo(torch.bfloat16).max  # noqa: E741
    h, da = torch.zeros(1, 2 * I, device="cuda"), torch.zeros(1, I, device="cuda")
    h[0, :6], h[0, I:I + 6] = 2.40625, torch.tensor([top, -top, top, -top, top, 1.0])
    da[0, :6] = torch.tensor([0.0, 0.0, 0.25, 0.25, 1.0, top])
    print_case("swiglu_range_end")
    h, da = h.bfloat16(), da.bfloat16()
    got = b.w4a4_swiglu_bwd(da, h)["dh"][0, :6].double().cpu()
    g = h[0, 0].double().cpu()
    s = 1.0 / (1.0 + torch.exp(-g))
    want = 0.25 * top * s * (1.0 + g * (1.0 - s))
    assert got[0] == 0 and got[1] == 0 and torch.isinf(got[4]) and torch.isinf(got[5])
    assert abs(got[2] - want) <= (2.0 ** -8 + 2.0 ** -20) * want and got[3] == -got[2]


@pytest.mark.parametrize("call", ["bf16", "checkpoint", "mxfp8"])
def test_no_gradient_of_a_factor_at_the_end_of_the_range(b, layer, call):
    """The same row in the expert backwards, where no gradient reaches it: dx and dw1 are 0 (dw2 takes a, which is
    infinite there)."""
    L, sizes = layer, (T, H, I, E, k, ALIGN)
    print_case("expert_bwd_range_end", call=call)
    h = torch.zeros_like(L["h"])
    h[5, :32], h[5, I:I + 32] = 2.40625, torch.finfo(h.dtype).max   # 448 2^119 in the checkpoint, its largest value
    kept = b.w4a4_swiglu_fwd(h, checkpoint=True)
    args = (torch.zeros_like(L["args"][0]), *L["args"][1:])
    if call == "checkpoint":
        g = b.w4a4_expert_bwd_ckpt(*args, kept, L["p"], L["xq"], *sizes)
    else:
        bwd = b.w4a4_expert_bwd if call == "bf16" else b.w4a4_mx8_expert_bwd
        g = bwd(*args, h, torch.zeros_like(L["a"]), L["p"], L["xq"], *sizes)
    for m in ("dx", "dw1"):
        assert bool(torch.isfinite(g[m]).all()) and not g[m].any(), m
