"""Tensors of the pre-norm and dense MX calls that may not share an address:
a write of one row would fall on another row that is still read, or on another
output. Refused on the host, before any launch."""
import ctypes
import os

import pytest

pytestmark = pytest.mark.cpu

INVALID = -1
FP4, FP8, NONE, BF16, F32 = 0, 1, -1, 0, 1


@pytest.fixture(scope="module")
def lib():
    from precision_rl_amd import build, binding
    if not os.path.exists(build.LIB):
        build.build()
    return binding.load()


@pytest.fixture(scope="module")
def at():
    """Distinct 16-byte aligned addresses by name."""
    buf = ctypes.create_string_buffer(1 << 16)
    base = ctypes.addressof(buf) + (-ctypes.addressof(buf)) % 16
    places = {}

    def place(name):
        return ctypes.c_void_p(base + 2048 * places.setdefault(name, len(places)))

    place.keep = buf
    return place


def _refused(lib, status, *names):
    error = lib.w4a4_last_error().decode()
    return status == INVALID and "share" in error and all(n in error for n in names)


@pytest.mark.parametrize("one,other,how", [
    ("y", "residual", dict(rdt=F32)),      # y's row t lies over half a row of the float tensor
    ("y", "sum", dict(rdt=F32)), ("y", "sum", dict(rdt=BF16)),
    ("y", "x", dict(stride=128)),          # a dense y over a slice
    ("y", "gamma", {}), ("sum", "gamma", {}), ("codes", "x", {}), ("codes", "residual", {}), ("codes", "y", {}),
    ("codes", "sum", {}), ("scales", "codes", {}), ("scales", "x", {}), ("rstd", "gamma", {}), ("rstd", "y", {})])
def test_norm_forward(lib, at, one, other, how):
    p = {n: at(n) for n in ("x", "residual", "gamma", "sum", "y", "codes", "scales", "rstd")}
    p[one] = p[other]
    status = lib.w4a4_add_rmsnorm_fwd(4, 64, 1e-6, p["x"], how.get("stride", 64), p["residual"], how.get("rdt", BF16),
                                      p["gamma"], BF16, FP8, p["sum"], p["y"], p["codes"], p["scales"], p["rstd"],
                                      None, None)
    assert _refused(lib, status, one, other)


@pytest.mark.parametrize("one,other,rdt", [
    ("dx", "sum", F32), ("dx", "dsum", F32), ("dx", "dres", F32), ("dx", "gamma", BF16), ("dres", "gamma", BF16),
    ("dx", "rstd", BF16), ("dres", "rstd", BF16),
    ("dgamma", "gamma", BF16), ("dgamma", "rstd", BF16), ("dgamma", "dy", BF16), ("dgamma", "sum", F32),
    ("dgamma", "dres", F32), ("dgamma", "dsum", F32), ("dgamma", "dx", BF16)])
def test_norm_backward(lib, at, one, other, rdt):
    p = {n: at(n) for n in ("dy", "sum", "gamma", "rstd", "dsum", "dres", "dx", "dgamma")}
    p[one] = p[other]
    status = lib.w4a4_add_rmsnorm_bwd(4, 64, p["dy"], p["sum"], rdt, p["gamma"], BF16, p["rstd"], p["dsum"], p["dres"],
                                      p["dx"], p["dgamma"], None, 0, None)
    assert _refused(lib, status, one, other)


@pytest.mark.parametrize("one,other", [("codes", "x"), ("scales", "x"), ("scales", "codes")])
def test_quantize_rows(lib, at, one, other):
    p = {n: at(n) for n in ("x", "codes", "scales")}
    p[one] = p[other]
    assert _refused(lib, lib.w4a4_mx_quantize_rows(4, 64, FP8, p["x"], 64, p["codes"], p["scales"], None, None),
                    one, other)


@pytest.mark.parametrize("other", ["x_codes", "x_scales", "w_codes", "w_scales"])
def test_linear(lib, at, other):
    p = {n: at(n) for n in ("x_codes", "x_scales", "w_codes", "w_scales")}
    assert _refused(lib, lib.w4a4_mx_linear_fwd(4, 128, 64, FP8, p["x_codes"], p["x_scales"], p["w_codes"],
                                                p["w_scales"], p[other], 64, None), "y", other)
