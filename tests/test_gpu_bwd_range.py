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
