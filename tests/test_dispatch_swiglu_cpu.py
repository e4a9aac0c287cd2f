"""Arguments that the dispatch and SwiGLU calls refuse, with the documented
status and before any launch (the host-side checks alone: no GPU here)."""
import ctypes
import os

import pytest

pytestmark = pytest.mark.cpu

INVALID, UNSUPPORTED, WORKSPACE = -1, -2, -3
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

    def place(name, shift=0):
        return ctypes.c_void_p(base + 2048 * places.setdefault(name, len(places)) + shift)

    place.keep = buf
    return place


PERMUTE = ("T", "H", "k", "E", "align", "dtype", "x", "stride", "idx", "xp", "offsets", "row_map", "src_row", "ws", "wsb")
GATHER = ("T", "H", "k", "rows", "dtype", "src", "row_map", "out", "stride")
UNPERMUTE = ("T", "H", "k", "rows", "dtype", "src", "row_map", "w", "out", "stride")
UNPERMUTE_BWD = ("T", "H", "k", "E", "rows", "dtype", "dy", "stride", "o", "row_map", "w", "offsets", "src_row", "do", "dw")
SWIGLU = ("T", "I", "h", "stride", "rows", "fmt", "a", "codes", "scales", "hc", "hs")
SWIGLU_BWD = ("T", "I", "da", "h", "stride", "hc", "hs", "rows", "dh", "a")


def _status(lib, at, name, order, base, change):
    v = dict(base, **change)
    for n, p in list(v.items()):
        if isinstance(p, str):                    # another tensor's address, or "name+2": shifted by two bytes
            where, _, shift = p.partition("+")
            v[n] = at(where, int(shift or 0))
    return getattr(lib, name)(*[v[n] for n in order], None)


def _base(order, **sizes):
    return {n: sizes.get(n, n) for n in order}


@pytest.mark.parametrize("change,status,says", [
    (dict(T=-1), INVALID, "T=-1"), (dict(H=12), INVALID, "multiple of 8"), (dict(H=0), INVALID, "row length 0"),
    (dict(k=0), INVALID, "k=0"), (dict(E=0), INVALID, "E=0"), (dict(E=-1), INVALID, "E=-1"),
    (dict(align=3), INVALID, "row_align"), (dict(dtype=2), INVALID, "element type"),
    (dict(stride=56), INVALID, "x_stride"), (dict(stride=68), INVALID, "x_stride"),
    (dict(k=9), UNSUPPORTED, "k <= 8"), (dict(E=1025), UNSUPPORTED, "E <= 1024"),
    (dict(H=65544, stride=65544), UNSUPPORTED, "65536"), (dict(T=1 << 31), UNSUPPORTED, "int32"),
    (dict(T=1 << 28, k=8), UNSUPPORTED, "int32"), (dict(T=(1 << 28) - 1, k=8, E=1024, align=128), UNSUPPORTED, "int32"),
    (dict(x=None), INVALID, "x is NULL"), (dict(idx=None), INVALID, "topk_idx"), (dict(offsets=None), INVALID, "offsets"),
    (dict(row_map=None), INVALID, "row_map"), (dict(src_row=None), INVALID, "src_row"),
    (dict(x="x+2"), INVALID, "x is not 16"), (dict(xp="xp+8"), INVALID, "xp is not 16"),
    (dict(idx="idx+2"), INVALID, "4-byte"), (dict(T=1 << 20, ws=None, wsb=0), WORKSPACE, "workspace"),
    (dict(T=1 << 20, wsb=64), WORKSPACE, "workspace"), (dict(T=1 << 20, ws="ws+4"), INVALID, "workspace"),
    (dict(xp="x"), INVALID, "share"), (dict(row_map="idx"), INVALID, "share"), (dict(src_row="row_map"), INVALID, "share"),
    (dict(offsets="idx"), INVALID, "share"), (dict(T=1 << 20, ws="idx"), INVALID, "share")])
def test_permute(lib, at, change, status, says):
    base = _base(PERMUTE, T=4, H=64, k=2, E=8, align=1, dtype=BF16, stride=64, wsb=1 << 24)
    assert _status(lib, at, "w4a4_permute_fwd", PERMUTE, base, change) == status
    assert says in lib.w4a4_last_error().decode()


COMMON = [(dict(T=-1), INVALID, "T=-1"), (dict(H=12), INVALID, "multiple of 8"), (dict(k=0), INVALID, "k=0"),
          (dict(dtype=-1), INVALID, "element type"), (dict(stride=60), INVALID, "_stride"),
          (dict(rows=-1), INVALID, "rows=-1"), (dict(rows=1 << 31), INVALID, "rows="), (dict(k=9), UNSUPPORTED, "k <= 8"),
          (dict(H=65544, stride=65544), UNSUPPORTED, "65536"), (dict(T=1 << 31), UNSUPPORTED, "int32"),
          (dict(row_map=None), INVALID, "row_map"), (dict(row_map="row_map+2"), INVALID, "4-byte")]


@pytest.mark.parametrize("change,status,says", COMMON + [
    (dict(src=None), INVALID, "dxp is NULL"), (dict(out=None), INVALID, "dx is NULL"),
    (dict(src="src+4"), INVALID, "dxp is not 16"), (dict(out="out+8"), INVALID, "dx is not 16"),
    (dict(out="src"), INVALID, "share"), (dict(out="row_map"), INVALID, "share")])
def test_permute_gradient(lib, at, change, status, says):
    base = _base(GATHER, T=4, H=64, k=2, rows=8, dtype=BF16, stride=64)
    assert _status(lib, at, "w4a4_permute_bwd", GATHER, base, change) == status
    assert says in lib.w4a4_last_error().decode()


@pytest.mark.parametrize("change,status,says", COMMON + [
    (dict(src=None), INVALID, "o is NULL"), (dict(w=None), INVALID, "topk_w"), (dict(w="w+2"), INVALID, "4-byte"),
    (dict(out="src"), INVALID, "share"), (dict(out="w"), INVALID, "share")])
def test_unpermute(lib, at, change, status, says):
    base = _base(UNPERMUTE, T=4, H=64, k=2, rows=8, dtype=BF16, stride=64)
    assert _status(lib, at, "w4a4_unpermute_fwd", UNPERMUTE, base, change) == status
    assert says in lib.w4a4_last_error().decode()


@pytest.mark.parametrize("change,status,says", COMMON + [
    (dict(dy=None), INVALID, "dy is NULL"), (dict(o=None), INVALID, "o is NULL"), (dict(w=None), INVALID, "topk_w"),
    (dict(do=None, dw=None), INVALID, "neither"), (dict(E=0), INVALID, "E=0"), (dict(E=1025), UNSUPPORTED, "E <= 1024"),
    (dict(offsets=None), INVALID, "expert_offsets"), (dict(src_row=None), INVALID, "src_row"),
    (dict(do="o"), INVALID, "share"), (dict(do="dy"), INVALID, "share"), (dict(dw="w"), INVALID, "share"),
    (dict(do="src_row"), INVALID, "share"), (dict(dw="do"), INVALID, "share"), (dict(dw="dw+2"), INVALID, "4-byte")])
def test_unpermute_gradient(lib, at, change, status, says):
    base = _base(UNPERMUTE_BWD, T=4, H=64, k=2, E=8, rows=16, dtype=BF16, stride=64)
    assert _status(lib, at, "w4a4_unpermute_bwd", UNPERMUTE_BWD, base, change) == status
    assert says in lib.w4a4_last_error().decode()


@pytest.mark.parametrize("change,status,says", [
    (dict(T=-1), INVALID, "T=-1"), (dict(I=48), INVALID, "multiple of 32"), (dict(I=0), INVALID, "row length 0"),
    (dict(I=12, fmt=NONE, codes=None, scales=None, hc=None, hs=None), INVALID, "multiple of 8"),
    (dict(fmt=2), INVALID, "format"), (dict(fmt=NONE), INVALID, "need a format"), (dict(stride=120), INVALID, "h_stride"),
    (dict(I=65568, stride=1 << 18), UNSUPPORTED, "65536"), (dict(T=1 << 31), UNSUPPORTED, "int32"),
    (dict(h=None), INVALID, "h is NULL"), (dict(h="h+2"), INVALID, "h is not 16"), (dict(hs=None), INVALID, "both"),
    (dict(hc=None), INVALID, "both"), (dict(codes=None), INVALID, "codes is NULL"), (dict(scales=None), INVALID, "scales"),
    (dict(rows="rows+2"), INVALID, "4-byte"),
    (dict(a=None, fmt=NONE, codes=None, scales=None, hc=None, hs=None), INVALID, "none of"),
    (dict(a="h"), INVALID, "share"), (dict(hc="h"), INVALID, "share"), (dict(codes="a"), INVALID, "share"),
    (dict(hs="scales"), INVALID, "share"), (dict(a="rows"), INVALID, "share")])
def test_swiglu(lib, at, change, status, says):
    base = _base(SWIGLU, T=4, I=64, stride=128, fmt=FP8)
    assert _status(lib, at, "w4a4_swiglu_fwd", SWIGLU, base, change) == status
    assert says in lib.w4a4_last_error().decode()


@pytest.mark.parametrize("change,status,says", [
    (dict(T=-1), INVALID, "T=-1"), (dict(I=48), INVALID, "multiple of 32"),
    (dict(I=12, h="h", hc=None, hs=None), INVALID, "multiple of 8"), (dict(h="h"), INVALID, "either"),
    (dict(hc=None, hs=None), INVALID, "either"), (dict(hc=None, h="h"), INVALID, "both"), (dict(hs=None), INVALID, "both"),
    (dict(h="h", hc=None, hs=None, stride=64), INVALID, "h_stride"), (dict(dh=None, a=None), INVALID, "neither"),
    (dict(da=None), INVALID, "da is NULL"), (dict(I=65568), UNSUPPORTED, "65536"),
    (dict(dh="hc"), INVALID, "share"), (dict(dh="da"), INVALID, "share"), (dict(dh="a"), INVALID, "share"),
    (dict(a="hs"), INVALID, "share"), (dict(h="h", hc=None, hs=None, dh="h", stride=136), INVALID, "share"),
    (dict(h="h", hc=None, hs=None, a="h"), INVALID, "share"), (dict(hc="hc+8"), INVALID, "h_codes is not 16")])
def test_swiglu_gradient(lib, at, change, status, says):
    base = _base(SWIGLU_BWD, T=4, I=64, h=None, stride=128)
    assert _status(lib, at, "w4a4_swiglu_bwd", SWIGLU_BWD, base, change) == status
    assert says in lib.w4a4_last_error().decode()


def test_empty_batches_take_null_tensors(lib, at):
    assert lib.w4a4_permute_bwd(0, 64, 2, 0, BF16, None, None, None, 64, None) == 0
    assert lib.w4a4_unpermute_fwd(0, 64, 2, 0, BF16, None, None, None, None, 64, None) == 0
    assert lib.w4a4_unpermute_bwd(0, 64, 2, 8, 0, BF16, None, 64, None, None, None, None, None, None, None, None) == 0
    assert lib.w4a4_swiglu_fwd(0, 64, None, 128, None, FP8, None, None, None, None, None, None) == 0
    assert lib.w4a4_swiglu_bwd(0, 64, None, None, 128, None, None, None, None, None, None) == 0


def test_workspace_sizes(lib):
    size = lambda T, k, E: lib.w4a4_workspace_size(8, T, 0, 0, E, k, 1)  # noqa: E731
    assert size(1, 8, 128) == 0 and size(0, 8, 128) == 0
    assert size(16384, 8, 128) >= 4 * 128 * (16384 * 8 // 1024 + 1)
    assert size(16384, 9, 128) == size(16384, 8, 1025) == size(-1, 8, 128) == size(16384, 0, 128) == 0


CKPT = ("T", "H", "I", "E", "k", "align", "dy", "x", "w1", "w2", "hc", "hs", "p", "offsets", "row_map", "src_row", "dx",
        "dw1", "dw2", "ws", "wsb")


@pytest.mark.parametrize("change,status,says", [
    (dict(T=-1), INVALID, "T=-1"), (dict(H=250), INVALID, "multiples of 32"), (dict(H=288), UNSUPPORTED, "256"),
    (dict(I=96), UNSUPPORTED, "128"), (dict(k=9, E=16), UNSUPPORTED, "k <= 8"), (dict(align=2), INVALID, "row_align"),
    (dict(hc=None), INVALID, "h_codes"), (dict(hs=None), INVALID, "h_scales"), (dict(hc="hc+8"), INVALID, "h_codes"),
    (dict(dw2=None), INVALID, "dw2"), (dict(ws=None), WORKSPACE, "workspace"), (dict(wsb=1 << 10), WORKSPACE, "workspace"),
    (dict(ws="ws+4"), INVALID, "workspace")])
def test_expert_backward_from_a_checkpoint(lib, at, change, status, says):
    base = _base(CKPT, T=4, H=256, I=128, E=8, k=2, align=1, wsb=1 << 30)
    assert _status(lib, at, "w4a4_expert_bwd_ckpt", CKPT, base, change) == status
    assert says in lib.w4a4_last_error().decode()


def test_expert_backward_workspace_holds_a_beside_the_others(lib):
    size = lambda kind: lib.w4a4_workspace_size(kind, 64, 256, 128, 8, 2, 16)  # noqa: E731
    assert size(9) == size(2) + -(-(64 * 2 + 8 * 15) * 128 * 2 // 256) * 256


FWD = ("T", "H", "I", "E", "k", "align", "xc", "xs", "xo", "offsets", "row_map", "src_row", "p", "w1c", "w1s", "w1o", "w2c",
       "w2s", "w2o", "y", "hc", "hs", "o", "ws", "wsb")


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("change,status,says", [
    (dict(T=-1), INVALID, "T=-1"), (dict(H=288), UNSUPPORTED, "256"), (dict(I=96), UNSUPPORTED, "128"),
    (dict(hc=None), INVALID, "h_codes"), (dict(hs=None), INVALID, "h_scales"), (dict(hs="hs+8"), INVALID, "h_scales"),
    (dict(o="o+8"), INVALID, "o is not"), (dict(y=None), INVALID, "y"), (dict(ws=None), WORKSPACE, "workspace"),
    (dict(wsb=1 << 10), WORKSPACE, "workspace")])
def test_expert_forward_that_keeps_a_checkpoint(lib, at, mx, change, status, says):
    order = tuple(n for n in FWD if not mx or n not in ("xo", "w1o", "w2o"))
    base = _base(order, T=4, H=256, I=128, E=8, k=2, align=1, wsb=1 << 30)
    name = "w4a4_mx_grouped_expert_fwd_ckpt" if mx else "w4a4_grouped_expert_fwd_ckpt"
    assert _status(lib, at, name, order, base, change) == status
    assert says in lib.w4a4_last_error().decode()
