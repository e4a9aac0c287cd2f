"""Single roundings of the pre-norm, at every number of lanes that takes a row.

With u = 2^-24 (half a step of FP32, relative):
  rstd  is computed in FP64 from squares summed in FP64 (error below
        (H + 4) 2^-53 <= 2^-39 of it) and rounded once: within (1 + 2^-15) u.
        Sums in FP32 would lose several u on most rows.
  y     is the bf16 nearest to the exact value: rounded to FP32 in between, 1
        value of 2^17 would move to the other side.  The 64-bit value's own
        error, below 2^-50 of it, decides a rounding with chance 2^-41.
"""
import numpy as np
import pytest

from oracle import rmsnorm

torch = pytest.importorskip("torch")

U = 2.0 ** -24
EPS = 2.0 ** -20
# 16 lanes x 1 and 2 chunks of 8, 64 x 1 and 2, 256 x 1 (few rows), 64 x 4 (more), 256 x 2 and 4; 2 to 4 million values
SHAPES = [(16000, 128), (8000, 256), (8000, 512), (4000, 1024), (2000, 2048), (2100, 2048), (1000, 4096), (500, 8192)]


def _rows(T, H, res, seed):
    rng = np.random.default_rng(seed)
    x = torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32)).to(torch.bfloat16)
    r = torch.from_numpy((3 * rng.standard_normal((T, H)) * np.exp(rng.standard_normal(H))).astype(np.float32)).to(res)
    g = torch.from_numpy((1 + 0.3 * rng.standard_normal(H)).astype(np.float32)).to(res)
    return x, r, g


def _nearest_bf16(y):
    _, e = np.frexp(y)
    step = np.ldexp(1.0, np.maximum(e - 1, -126) - 7)
    return np.rint(y / step) * step


def _check(s, g, y, rstd):
    """s, g, y, rstd in 64 bits."""
    y64, r64 = rmsnorm.forward(s, g, EPS)
    assert np.all(np.abs(rstd - r64) <= (1 + 2.0 ** -15) * U * r64), "rstd"
    assert np.array_equal(y, _nearest_bf16(y64)), "y"


@pytest.mark.cpu
@pytest.mark.parametrize("T,H", [(2000, 128), (500, 2048)])
def test_check_sees_fp32_sums_and_double_rounding(T, H):
    x, r, g = _rows(T, H, torch.float32, 7)
    s, gamma = (x.double() + r.double()).float().double().numpy(), g.double().numpy()
    y64, r64 = rmsnorm.forward(s, gamma, EPS)
    rstd = r64.astype(np.float32).astype(np.float64)
    _check(s, gamma, _nearest_bf16(y64), rstd)
    with pytest.raises(AssertionError, match="rstd"):   # squares summed in FP32, eight lanes' worth
        part = np.cumsum(np.square(s.astype(np.float32)).reshape(T, 8, -1), axis=2, dtype=np.float32)[:, :, -1]
        _check(s, gamma, _nearest_bf16(y64), 1 / np.sqrt(part.sum(1, dtype=np.float32).astype(np.float64) / H + EPS))
    if T * H >= 2 ** 20:
        with pytest.raises(AssertionError, match="y"):  # FP32 in between, some 8 values
            _check(s, gamma, _nearest_bf16(y64.astype(np.float32).astype(np.float64)), rstd)


@pytest.mark.gpu
@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("res", ["bf16", "f32"])
def test_norm_rounds_once_at_every_row_width(T, H, res):
    from gpu_util import print_case
    from precision_rl_amd import binding as b
    x, r, g = (t.cuda() for t in _rows(T, H, torch.bfloat16 if res == "bf16" else torch.float32, H))
    print_case("norm_rounds_once_widths", T=T, H=H, res=res)
    out = b.w4a4_add_rmsnorm_fwd(x, g, EPS, residual=r, save=True)
    host = lambda t: t.double().cpu().numpy()  # noqa: E731
    _check(host(out["sum"]), host(g), host(out["y"]), host(out["rstd"]))


@pytest.mark.gpu
@pytest.mark.parametrize("H", [4104, 8192])
@pytest.mark.parametrize("res", ["bf16", "f32"])
def test_wide_rows_have_the_same_bits_in_small_and_large_batches(H, res):
    """Across the row counts at which the backward's workgroups change: 512 (dgamma from the rows
    themselves), 2048 (256 threads a workgroup instead of 512)."""
    from gpu_util import print_case
    from precision_rl_amd import binding as b
    T = 2500
    x, r, g = (t.cuda() for t in _rows(T, H, torch.bfloat16 if res == "bf16" else torch.float32, 3))
    dy = _rows(T, H, torch.bfloat16, 4)[1].cuda()
    print_case("wide_rows_small_large", H=H, res=res)
    full = b.w4a4_add_rmsnorm_fwd(x, g, EPS, residual=r, save=True)
    back = b.w4a4_add_rmsnorm_bwd(dy, full["sum"], g, full["rstd"], dsum=r)
    for n in (1, 2, 511, 512, 513, 2047, 2048, 2049):
        some = b.w4a4_add_rmsnorm_fwd(x[:n], g, EPS, residual=r[:n], save=True)
        for name in ("sum", "y", "rstd"):
            assert torch.equal(some[name], full[name][:n]), (name, n)
        for dgamma in (True, False):
            part = b.w4a4_add_rmsnorm_bwd(dy[:n], some["sum"], g, some["rstd"], dsum=r[:n], dgamma=dgamma)
            assert torch.equal(part["dres"], back["dres"][:n]), (n, dgamma)
