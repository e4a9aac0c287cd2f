"""Grids of the dispatch beyond what one launch holds (2^32 threads), with the
workgroups of pad rows in the second one; the library's own count of launches
tells that there were two."""
import pytest

from gpu_util import print_case

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

MOST = (2 ** 32 - 1) // 256 // 8 * 8       # workgroups of 256 threads that a launch takes
PART = 1 << 24                             # entries compared at a time


@pytest.fixture(scope="module")
def b():
    from precision_rl_amd import binding
    return binding


def _launches(b, kernel, call):
    b.w4a4_profiler_enable(True)
    try:
        out = call()
        return out, b.w4a4_profiler_report()[kernel]["count"]
    finally:
        b.w4a4_profiler_enable(False)


def _reversed_maps(T, k, pads):
    """One group: entry i in row T k - 1 - i, `pads` pad rows behind, then one row that is not in use."""
    n = T * k
    src = torch.zeros(n + pads + 1, dtype=torch.int32, device="cuda")
    src[n:] = -1
    row = torch.arange(n - 1, -1, -1, dtype=torch.int32, device="cuda").view(T, k)
    return dict(row_map=row, src_row=src, offsets=torch.tensor([0, n + pads], dtype=torch.int32, device="cuda"))


def _check_do(do, dy, w, k, n, pads):
    for i0 in range(0, n, PART):
        i1 = min(n, i0 + PART)
        want = (w.view(-1)[i0:i1, None] * dy[i0 // k:-(-i1 // k)].float().repeat_interleave(k, 0)[:i1 - i0]).to(do.dtype)
        assert torch.equal(do[n - i1:n - i0].flip(0), want), i0
    assert not do[n:n + pads].any() and bool((do[n + pads:] == 7).all())


def test_unpermute_gradients_by_entries(b):
    """2^28 + 40 entries of 16 lanes: both gradients, whole.  dp: 8 products of a chunk, one chunk, 6 joins."""
    T, k, H, pads = (1 << 25) + 5, 8, 8, 24
    n = T * k
    assert MOST < -(-n // 16) < MOST + 16
    print_case("unpermute_bwd_entries_launches", T=T, k=k, H=H)
    g = torch.Generator(device="cuda").manual_seed(1)
    perm = _reversed_maps(T, k, pads)
    rows = n + pads + 1
    o = torch.randn(rows, H, generator=g, device="cuda", dtype=torch.bfloat16)
    dy = torch.randn(T, H, generator=g, device="cuda", dtype=torch.bfloat16)
    w = torch.rand(T, k, generator=g, device="cuda")
    out = dict(do=torch.full((rows, H), 7.0, dtype=torch.bfloat16, device="cuda"))
    r, launches = _launches(b, "unpermute_bwd", lambda: b.w4a4_unpermute_bwd(dy, o, perm, w, out=out))
    assert launches == 2
    _check_do(r["do"], dy, w, k, n, pads)
    for i0 in range(0, n, PART):
        i1 = min(n, i0 + PART)
        v = o[n - i1:n - i0].flip(0).double() * dy[i0 // k:-(-i1 // k)].double().repeat_interleave(k, 0)[:i1 - i0]
        off = (r["dtopk_w"].view(-1)[i0:i1].double() - v.sum(1)).abs()
        assert bool((off <= 15 * 2.0 ** -24 * (1 + 2.0 ** -10) * v.abs().sum(1)).all()), i0


def test_unpermute_gradient_by_tokens(b):
    """2^24 + 5 tokens of a workgroup: the rows' gradient alone."""
    T, k, H, pads = (1 << 24) + 5, 1, 8, 24
    assert T > MOST
    print_case("unpermute_bwd_scatter_launches", T=T, k=k, H=H)
    g = torch.Generator(device="cuda").manual_seed(2)
    perm = _reversed_maps(T, k, pads)
    dy = torch.randn(T, H, generator=g, device="cuda")
    w = torch.rand(T, k, generator=g, device="cuda")
    out = dict(do=torch.full((T + pads + 1, H), 7.0, device="cuda"))
    r, launches = _launches(b, "unpermute_bwd",
                            lambda: b.w4a4_unpermute_bwd(dy, None, perm, w, dtopk_w=False, out=out))
    assert launches == 2
    _check_do(r["do"], dy, w, k, T, pads)


def test_permute_of_narrow_rows(b):
    """2^28 + 5 tokens of 16 lanes to three experts in turn, groups of 128: maps and rows whole."""
    T, H, E, align = (1 << 28) + 5, 8, 3, 128
    assert MOST < -(-T // 16) < MOST + 16
    print_case("permute_narrow_launches", T=T, H=H, E=E, align=align)
    g = torch.Generator(device="cuda").manual_seed(3)
    bits = torch.randint(-2 ** 15, 2 ** 15, (T, H), generator=g, device="cuda", dtype=torch.int16)
    each = torch.arange(T, dtype=torch.int32, device="cuda")
    ids = (each % E).view(T, 1)
    cap = b.rows_capacity(T, 1, E, align)
    out = dict(xp=torch.full((cap, H), 7, dtype=torch.int16, device="cuda").view(torch.bfloat16),
               src_row=torch.full((cap,), -7, dtype=torch.int32, device="cuda"))
    r, launches = _launches(b, "permute_rows",
                            lambda: b.w4a4_permute_fwd(bits.view(torch.bfloat16), ids, E, align, out=out))
    assert launches == 2
    xp, start = r["xp"].view(torch.int16), 0
    for e in range(E):
        count = -(-(T - e) // E)
        end, stop = start + count, start + -(-count // align) * align
        assert r["offsets"][e].item() == start and r["offsets"][e + 1].item() == stop and end < stop
        assert torch.equal(xp[start:end], bits[e::E]) and torch.equal(r["src_row"][start:end], each[e::E])
        assert torch.equal(r["row_map"][e::E, 0], torch.arange(start, end, dtype=torch.int32, device="cuda"))
        assert not xp[end:stop].any() and bool((r["src_row"][end:stop] == -1).all())
        start = stop
    assert bool((xp[start:] == 7).all()) and bool((r["src_row"][start:] == -7).all())
