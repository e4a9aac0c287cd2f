"""Refusals of the pre-norm and dense MX calls: host-side checks before any
launch, through the C ABI and the binding."""
import ctypes
import os

import pytest

pytestmark = pytest.mark.cpu
torch = pytest.importorskip("torch")

INVALID, UNSUPPORTED, WORKSPACE = -1, -2, -3
FP4, FP8, NONE, BF16, F32 = 0, 1, -1, 0, 1


@pytest.fixture(scope="module")
def lib():
    from precision_rl_amd import build, binding
    if not os.path.exists(build.LIB):
        build.build()
    return binding.load()


@pytest.fixture(scope="module")
def p():
    buf = ctypes.create_string_buffer(4096)
    ptr = ctypes.c_void_p(ctypes.addressof(buf) + (-ctypes.addressof(buf)) % 16)
    ptr.keep = buf
    return ptr


def _off(p, n=2):
    return ctypes.c_void_p(p.value + n)


def test_quantize_rows_refusals(lib, p):
    def q(T=4, K=64, fmt=FP8, x=p, stride=64, codes=p, scales=p, offsets=None):
        return lib.w4a4_mx_quantize_rows(T, K, fmt, x, stride, codes, scales, offsets, None)

    assert q(T=-1) == INVALID
    assert q(K=0) == INVALID
    assert q(K=48) == INVALID                      # blocks of 32
    assert q(fmt=NONE) == INVALID and q(fmt=2) == INVALID
    assert q(stride=56) == INVALID                 # shorter than the row
    assert q(stride=68) == INVALID                 # rows off the 16-byte grid
    assert q(x=None) == INVALID and q(codes=None) == INVALID and q(scales=None) == INVALID
    assert q(x=_off(p)) == INVALID and q(codes=_off(p)) == INVALID
    assert q(offsets=_off(p)) == INVALID
    assert q(T=1 << 31) == UNSUPPORTED
    assert "int32" in lib.w4a4_last_error().decode()
    assert q(T=0, x=None, codes=None, scales=None) == 0   # nothing to do, nothing launched


def test_norm_refusals(lib, p):
    def f(T=4, H=64, eps=1e-6, x=p, stride=64, res=None, rdt=BF16, gamma=p, gdt=BF16, fmt=FP8, total=None, y=None,
          codes=p, scales=p, rstd=None, offsets=None):
        return lib.w4a4_add_rmsnorm_fwd(T, H, eps, x, stride, res, rdt, gamma, gdt, fmt, total, y, codes, scales,
                                        rstd, offsets, None)

    assert f(T=-1) == INVALID and f(H=0) == INVALID
    assert f(H=72) == INVALID                      # codes need whole blocks of 32
    assert f(H=68, fmt=NONE, codes=None, scales=None) == INVALID   # and any row multiples of 8
    assert f(H=8224, stride=8224) == UNSUPPORTED
    for eps in (0.0, -1.0, float("inf"), float("nan")):
        assert f(eps=eps) == INVALID
    assert f(rdt=2) == INVALID and f(gdt=-1) == INVALID and f(fmt=3) == INVALID
    assert f(stride=32) == INVALID
    assert f(fmt=NONE) == INVALID                  # codes without a format
    assert f(codes=None) == INVALID and f(x=None) == INVALID and f(gamma=None) == INVALID
    assert f(res=_off(p)) == INVALID and f(total=_off(p)) == INVALID and f(y=_off(p)) == INVALID
    assert f(rstd=_off(p)) == INVALID
    assert f(total=p, rdt=F32) == INVALID          # a float sum over a bf16 x
    assert f(total=p, stride=128) == INVALID       # a dense sum over a slice
    assert f(T=1 << 31) == UNSUPPORTED
    assert f(T=0, x=None, gamma=None, codes=None, scales=None) == 0

    def b(T=4, H=64, dy=p, total=p, rdt=BF16, gamma=p, gdt=BF16, rstd=p, dsum=None, dres=p, dx=None, dgamma=p, ws=p,
          wsb=1 << 20):
        return lib.w4a4_add_rmsnorm_bwd(T, H, dy, total, rdt, gamma, gdt, rstd, dsum, dres, dx, dgamma, ws, wsb, None)

    assert b(T=-1) == INVALID and b(H=20) == INVALID and b(H=8200) == UNSUPPORTED
    assert b(dy=None) == INVALID and b(total=None) == INVALID and b(rstd=None) == INVALID and b(dres=None) == INVALID
    assert b(rdt=5) == INVALID and b(gdt=5) == INVALID
    assert b(rdt=F32) == INVALID                   # dres over a bf16 dy
    assert b(dsum=_off(p)) == INVALID and b(dx=_off(p)) == INVALID and b(dgamma=_off(p)) == INVALID
    assert b(T=600, ws=None) == WORKSPACE and b(T=600, wsb=16) == WORKSPACE
    assert b(T=0, dy=None, total=None, gamma=None, rstd=None, dres=None, dgamma=None, ws=None, wsb=0) == 0


def test_norm_workspace_size(lib):
    size = lambda T, H: lib.w4a4_workspace_size(6, T, H, 0, 1, 1, 1)  # noqa: E731
    assert size(1, 64) == 0 and size(600, 64) >= 64 * 4      # none for few rows
    assert size(16384, 2048) > size(600, 2048)
    assert size(-1, 64) == 0 and size(4, 0) == 0 and size(4, 16384) == 0


def test_linear_refusals(lib, p):
    def f(T=4, K=128, N=64, fmt=FP8, x=p, xs=p, w=p, ws=p, y=p, stride=64):
        return lib.w4a4_mx_linear_fwd(T, K, N, fmt, x, xs, w, ws, y, stride, None)

    assert f(T=-1) == INVALID and f(K=0) == INVALID and f(N=0) == INVALID
    assert f(K=100) == INVALID
    assert f(K=96) == UNSUPPORTED                  # whole blocks, but not whole stages
    assert f(N=20) == UNSUPPORTED
    assert "128" in lib.w4a4_last_error().decode()
    assert f(K=65536 + 128) == UNSUPPORTED
    assert f(N=(1 << 30) + 8, stride=(1 << 30) + 8) == UNSUPPORTED
    assert f(fmt=NONE) == INVALID
    assert f(stride=56) == INVALID and f(stride=68) == INVALID
    assert f(x=None) == INVALID and f(xs=None) == INVALID and f(w=None) == INVALID and f(ws=None) == INVALID
    assert f(y=None) == INVALID and f(y=_off(p)) == INVALID and f(w=_off(p)) == INVALID and f(xs=_off(p)) == INVALID
    assert f(T=1 << 31) == UNSUPPORTED
    assert f(T=0, x=None, xs=None, w=None, ws=None, y=None) == 0


def test_binding_refuses_host_tensors_and_wrong_types():
    from precision_rl_amd import binding as b
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    for call in (lambda: b.w4a4_mx_quantize_rows(x, b.MX_FP8),
                 lambda: b.w4a4_add_rmsnorm_fwd(x, torch.ones(64, dtype=torch.bfloat16)),
                 lambda: b.w4a4_add_rmsnorm_bwd(x, x, x[0], torch.ones(2)),
                 lambda: b.w4a4_mx_linear_fwd(dict(codes=x, scales=x), dict(codes=x, scales=x), 2, 64, 2)):
        with pytest.raises(b.W4A4Error):
            call()
