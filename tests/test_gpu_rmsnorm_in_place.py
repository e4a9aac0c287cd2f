"""The pre-norm's outputs over those of its inputs that its description allows:
the bits of the same call into tensors of their own."""
import numpy as np
import pytest

from gpu_util import print_case

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

# few rows, several launches' worth of teams, every number of lanes and threads a row
SHAPES = [(1, 96), (100, 512), (61, 2048), (300, 1536), (700, 1024), (2100, 2048), (600, 4096), (2060, 8192)]


@pytest.fixture(scope="module")
def b():
    from precision_rl_amd import binding
    return binding


def _rows(rng, T, H, dtype=None):
    return torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32)).to(dtype or torch.bfloat16).cuda()


@pytest.mark.parametrize("T,H", SHAPES)
def test_forward_over_its_inputs(b, T, H):
    rng = np.random.default_rng(T + H)
    x, r, g = _rows(rng, T, H), _rows(rng, T, H), torch.ones(H, device="cuda")
    print_case("norm_forward_over_inputs", T=T, H=H)
    ref = b.w4a4_add_rmsnorm_fwd(x, g, 1e-6, residual=r, fmt=b.MX_FP8, save=True)
    for y_over, sum_over in (("x", None), ("r", None), ("x", "r"), ("r", "x"), (None, "x")):
        t = dict(x=x.clone(), r=r.clone())
        out = dict(y=t.get(y_over), sum=t.get(sum_over))
        got = b.w4a4_add_rmsnorm_fwd(t["x"], g, 1e-6, residual=t["r"], fmt=b.MX_FP8, save=True,
                                     out={n: v for n, v in out.items() if v is not None})
        for n in ref:
            assert torch.equal(got[n], ref[n]), (n, y_over, sum_over)


def test_one_row_over_a_strided_x(b):
    """Through the C call, whose one row has a pitch that nothing reads."""
    H = 2048
    x, g = _rows(np.random.default_rng(4), 1, H), torch.ones(H, device="cuda")
    print_case("norm_one_strided_row")
    want = b.w4a4_add_rmsnorm_fwd(x, g, 1e-6)["y"]
    stream = torch.cuda.current_stream().cuda_stream
    status = b.load().w4a4_add_rmsnorm_fwd(1, H, 1e-6, x.data_ptr(), 2 * H, None, 0, g.data_ptr(), 1, b.MX_NONE, None,
                                           x.data_ptr(), None, None, None, None, stream)
    assert status == 0 and torch.equal(x, want)


@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("res", ["bf16", "f32"])
def test_backward_over_its_inputs(b, T, H, res):
    rng = np.random.default_rng(T + H)
    rt = torch.bfloat16 if res == "bf16" else torch.float32
    ins = dict(dy=_rows(rng, T, H), s=_rows(rng, T, H, rt), ds=_rows(rng, T, H, rt))
    g, rstd = torch.ones(H, device="cuda"), torch.rand(T, device="cuda") + 0.5
    print_case("norm_backward_over_inputs", T=T, H=H, res=res)
    ref = b.w4a4_add_rmsnorm_bwd(ins["dy"], ins["s"], g, rstd, dsum=ins["ds"],
                                 out=dict(dx=torch.empty(T, H, dtype=torch.bfloat16, device="cuda")))
    pairs = [(None, "dy"), ("s", "dy"), ("ds", "dy")]   # (dres over, dx over)
    if res == "bf16":
        pairs += [("dy", "s"), ("dy", "ds"), ("s", "ds"), ("ds", "s"), ("ds", "dres")]
    for dres, dx in pairs:
        t = {n: v.clone() for n, v in ins.items()}
        t["dres"] = t[dres] if dres else torch.empty_like(t["s"])
        got = b.w4a4_add_rmsnorm_bwd(t["dy"], t["s"], g, rstd, dsum=t["ds"], out=dict(dres=t["dres"], dx=t[dx]))
        for n in ref:
            assert torch.equal(got[n], ref[n]), (n, dres, dx)
