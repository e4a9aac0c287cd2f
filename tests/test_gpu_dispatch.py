"""GPU parity of the token dispatch (rows sorted by expert and back, the
router's weights applied, both gradients) with the float64 oracle.

The maps and copied rows are compared bit for bit.  Bounds of the rest, with u
= 2^-24 and results rounded once to their type (a half step: 2^-8 in bf16, u in
float32, relative to the value):
  dx, y   at most 8 roundings of FP32, each at most u of the partial sums, which
          the magnitudes' sum bounds: 8 u sum|.|, times the final rounding.
  do      one product: u, and the rounding.
  dp      a lane adds a 16-byte chunk's products one by one and then its chunks (16
          lanes up to 64 chunks, 32 below 128, else 64), at most 6 steps join the
          lanes: (products a chunk + chunks a lane + 6) u sum|dy o|.
"""
import numpy as np
import pytest

from oracle import dispatch
from gpu_util import bf16_host, print_case

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

U = 2.0 ** -24
TINY = 2.0 ** -126
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def b():
    from precision_rl_amd import binding
    return binding


def _step(dtype):
    return torch.finfo(dtype).eps / 2


def _dev(v, dtype):
    return torch.from_numpy(np.asarray(v, dtype=np.float32)).to(dtype).cuda()


def _f64(t):
    return t.detach().double().cpu().numpy()


def _ids(T, k, E, how, rng):
    """Routings: distinct experts, any ids (experts named twice), some not dispatched, none dispatched, one expert."""
    if how == "distinct":
        return np.argsort(rng.random((T, E)), axis=1)[:, :k].astype(np.int32)
    if how == "any":
        return rng.integers(0, E, (T, k)).astype(np.int32)
    if how == "partial":      # ids of other ranks on both sides, whole tokens without a slot
        idx = rng.integers(-E, 3 * E, (T, k)).astype(np.int32)
        idx[::5] = -1
        idx[1::7] = np.iinfo(np.int32).max
        idx[2::11] = np.iinfo(np.int32).min
        return idx
    return np.full((T, k), -1 if how == "none" else E - 1, dtype=np.int32)


def _case(T, k, E, align, how, seed):
    rng = np.random.default_rng(seed)
    idx = _ids(T, k, E, how, rng)
    off, row, src = dispatch.maps(idx, E, align)
    return rng, idx, off, row, src, T * k + E * (align - 1)


def _perm(off, row, src, cap, k):
    pad = np.concatenate((src, np.full(cap - len(src), -7)))
    return {n: torch.from_numpy(np.asarray(v, dtype=np.int32)).cuda()
            for n, v in (("offsets", off), ("row_map", row), ("src_row", pad))}


# one token; batches of one launch with a token or eight a workgroup (border at
# 256 tokens) and of three (2048 tokens with 8 slots, 5792 with one), chunks of
# 1024 entries and their borders; one expert, a thousand; every alignment; rows
# of one chunk, of the two teams, and beyond a chunk a lane
CASES = [(1, 8, 2048, 128, 1, "distinct"), (1, 1, 8, 1, 1, "any"), (128, 8, 64, 16, 1, "distinct"),
         (129, 8, 1032, 16, 16, "any"), (61, 8, 2048, 128, 128, "distinct"), (341, 3, 264, 7, 32, "partial"),
         (342, 3, 512, 7, 64, "partial"), (1024, 1, 72, 1024, 1, "any"), (1025, 1, 72, 1024, 16, "any"),
         (500, 5, 1024, 33, 1, "partial"), (40, 2, 4104, 5, 16, "none"), (700, 4, 256, 3, 16, "one"),
         (3001, 8, 40, 128, 32, "partial"), (2, 6, 8200, 3, 1, "any"), (4096, 8, 16, 1000, 1, "any"),
         (4099, 8, 16, 1024, 16, "partial"), (16400, 2, 8, 1, 128, "any"), (33001, 1, 24, 300, 1, "partial"),
         (6500, 7, 520, 12, 64, "one"), (256, 4, 80, 11, 16, "any"), (257, 4, 80, 11, 16, "any"),
         (2048, 8, 72, 500, 32, "partial"), (2049, 8, 72, 500, 32, "partial"), (5792, 1, 8, 5, 16, "any")]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,k,H,E,align,how", CASES)
def test_permute(b, T, k, H, E, align, how, dtype):
    rng, idx, off, row, src, cap = _case(T, k, E, align, how, T + H)
    print_case("permute", T=T, k=k, H=H, E=E, align=align, how=how, dtype=dtype)
    x = _dev(rng.standard_normal((T, H)), TYPES[dtype])
    out = dict(xp=torch.full((cap, H), 7.0, dtype=TYPES[dtype], device="cuda"),
               src_row=torch.full((cap,), -7, dtype=torch.int32, device="cuda"))
    r = b.w4a4_permute_fwd(x, torch.from_numpy(idx).cuda(), E, align, out=out)
    n = off[-1]
    assert np.array_equal(r["offsets"].cpu().numpy(), off)
    assert np.array_equal(r["row_map"].cpu().numpy(), row)
    assert np.array_equal(r["src_row"].cpu().numpy(), np.concatenate((src, np.full(cap - n, -7))))
    assert np.array_equal(_f64(r["xp"]), np.concatenate((dispatch.permute(_f64(x), row, n), np.full((cap - n, H), 7.0))))
    maps = b.w4a4_permute_fwd(None, torch.from_numpy(idx).cuda(), E, align)
    assert all(torch.equal(maps[m], r[m]) for m in ("offsets", "row_map")) and "xp" not in maps
    assert torch.equal(maps["src_row"][:n], r["src_row"][:n])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,k,H,E,align,how", CASES)
def test_permute_gradient_and_unpermute(b, T, k, H, E, align, how, dtype):
    rng, idx, off, row, src, cap = _case(T, k, E, align, how, T + H + 1)
    print_case("gather", T=T, k=k, H=H, E=E, align=align, how=how, dtype=dtype)
    perm, dt = _perm(off, row, src, cap, k), TYPES[dtype]
    o = _dev(rng.standard_normal((cap, H)), dt)
    w = torch.from_numpy(rng.standard_normal((T, k)).astype(np.float32)).cuda()
    for got, (ref, mag) in ((b.w4a4_permute_bwd(o, perm), dispatch.gather_sum(_f64(o), row)),
                            (b.w4a4_unpermute_fwd(o, perm, w), dispatch.gather_sum(_f64(o), row, _f64(w)))):
        bound = (8 * U * mag) * (1 + _step(dt)) + _step(dt) * np.abs(ref) + TINY
        assert got.dtype == dt and np.all(np.abs(_f64(got) - ref) <= bound)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,k,H,E,align,how", CASES)
def test_unpermute_gradient(b, T, k, H, E, align, how, dtype):
    rng, idx, off, row, src, cap = _case(T, k, E, align, how, T + H + 2)
    print_case("unpermute_bwd", T=T, k=k, H=H, E=E, align=align, how=how, dtype=dtype)
    perm, dt = _perm(off, row, src, cap, k), TYPES[dtype]
    o, dy = _dev(rng.standard_normal((cap, H)), dt), _dev(rng.standard_normal((T, H)), dt)
    w = torch.from_numpy(rng.standard_normal((T, k)).astype(np.float32)).cuda()
    out = dict(do=torch.full((cap, H), 7.0, dtype=dt, device="cuda"),
               dtopk_w=torch.full((T, k), 7.0, device="cuda"))
    r = b.w4a4_unpermute_bwd(dy, o, perm, w, out=out)
    do, dp, mag = dispatch.unpermute_bwd(_f64(dy), _f64(o), row, _f64(w))
    n = off[-1]
    do[n:] = 7.0                                    # rows behind the last group
    got = _f64(r["do"])
    assert np.array_equal(got[n:], do[n:]) and not np.any(got[:n][src < 0])
    assert np.all(np.abs(got - do) <= (_step(dt) + U) * (1 + U) * np.abs(do) + TINY)
    chunks = H * o.element_size() // 16
    steps = 16 // o.element_size() + -(-chunks // (16 if chunks <= 64 else 32 if chunks < 128 else 64)) + 6
    assert np.all(np.abs(_f64(r["dtopk_w"]) - dp) <= steps * U * (1 + 2.0 ** -10) * mag)
    alone = b.w4a4_unpermute_bwd(dy, o, perm, w, do=False)
    assert torch.equal(alone["dtopk_w"], r["dtopk_w"]) and "do" not in alone
    alone = b.w4a4_unpermute_bwd(dy, None, perm, w, dtopk_w=False)
    assert torch.equal(alone["do"][:n], r["do"][:n]) and "dtopk_w" not in alone


def test_gradients_against_differences(b):
    """Everything is linear in x, o and w, so the difference of two calls is the
    gradient's product up to the calls' own roundings: in float32, 2 results of
    magnitude below 64 sums of 8 roundings each over T H terms, far below 1e-5
    of the sum of magnitudes."""
    T, k, H, E = 37, 4, 136, 6
    rng, idx, off, row, src, cap = _case(T, k, E, 16, "partial", 5)
    print_case("dispatch_differences", T=T, k=k, H=H, E=E)
    f32 = torch.float32
    x, v, dy = (_dev(rng.standard_normal((T, H)), f32) for _ in range(3))
    perm = b.w4a4_permute_fwd(x, torch.from_numpy(idx).cuda(), E, 16)
    n = off[-1]
    o, vo, g = (_dev(rng.standard_normal((cap, H)), f32) for _ in range(3))
    w, vw = (_dev(rng.standard_normal((T, k)), f32) for _ in range(2))
    dot = lambda a, c: float((a.double() * c.double()).sum())  # noqa: E731
    size = lambda a, c: float((a.double() * c.double()).abs().sum())  # noqa: E731

    xp2 = b.w4a4_permute_fwd(x + v, torch.from_numpy(idx).cuda(), E, 16)["xp"]
    dx = b.w4a4_permute_bwd(g, perm)
    d = (xp2 - perm["xp"])[:n]
    assert abs(dot(g[:n], d) - dot(dx, v)) <= 1e-5 * size(g[:n], d)
    y = b.w4a4_unpermute_fwd(o, perm, w)
    r = b.w4a4_unpermute_bwd(dy, o, perm, w)
    d = b.w4a4_unpermute_fwd(o + vo, perm, w) - y
    assert abs(dot(dy, d) - dot(r["do"][:n], vo[:n])) <= 1e-5 * size(dy, d)
    d = b.w4a4_unpermute_fwd(o, perm, w + vw) - y
    assert abs(dot(dy, d) - dot(r["dtopk_w"], vw)) <= 1e-5 * size(dy, d)


def test_column_slices(b):
    T, k, H, E = 83, 3, 264, 5
    rng, idx, off, row, src, cap = _case(T, k, E, 1, "any", 6)
    print_case("dispatch_slices", T=T, k=k, H=H, E=E)
    ids = torch.from_numpy(idx).cuda()
    wide = _dev(rng.standard_normal((T, H + 24)), torch.bfloat16)
    x = wide[:, 8:8 + H]
    perm, dense = b.w4a4_permute_fwd(x, ids, E), b.w4a4_permute_fwd(x.contiguous(), ids, E)
    assert torch.equal(perm["xp"], dense["xp"])
    w = torch.from_numpy(rng.random((T, k)).astype(np.float32)).cuda()
    o = _dev(rng.standard_normal((cap, H)), torch.bfloat16)
    for call, ref in ((lambda y: b.w4a4_permute_bwd(o, perm, dx=y), b.w4a4_permute_bwd(o, perm)),
                      (lambda y: b.w4a4_unpermute_fwd(o, perm, w, y=y), b.w4a4_unpermute_fwd(o, perm, w))):
        whole = torch.full((T, H + 24), 7.0, dtype=torch.bfloat16, device="cuda")
        call(whole[:, 8:8 + H])
        assert torch.equal(whole[:, 8:8 + H], ref) and bool((whole[:, :8] == 7).all() & (whole[:, 8 + H:] == 7).all())
    r, d = b.w4a4_unpermute_bwd(x, o, perm, w), b.w4a4_unpermute_bwd(x.contiguous(), o, perm, w)
    assert torch.equal(r["do"], d["do"]) and torch.equal(r["dtopk_w"], d["dtopk_w"])


def test_special_values(b):
    """An infinity or a NaN reaches the tokens and weights of its own row alone,
    also at a weight of zero; a slot that is not dispatched has none."""
    T, k, H, E = 6, 2, 72, 3
    idx = np.array([[0, 1], [1, 2], [2, -1], [-1, -1], [0, 2], [3, 0]], dtype=np.int32)
    off, row, src = dispatch.maps(idx, E, 1)
    perm = _perm(off, row, src, T * k, k)
    print_case("dispatch_special", T=T, k=k, H=H, E=E)
    o = torch.ones(T * k, H, dtype=torch.bfloat16, device="cuda")
    o[row[1, 0], 5] = float("nan")
    o[row[4, 1], 7] = float("inf")
    o[off[-1]:] = float("nan")                     # rows behind the last group are not read
    w = torch.full((T, k), 0.5, device="cuda")
    w[4, 1] = 0.0
    w[3] = float("nan")                            # weights of slots that are not dispatched are not looked at
    w[2, 1] = float("inf")
    y = b.w4a4_unpermute_fwd(o, perm, w).float().cpu()
    assert torch.isnan(y[1, 5]) and torch.isnan(y[4, 7])      # 0 times infinity
    y[1, 5] = y[4, 7] = 0.0
    want = torch.tensor([1.0, 1.0, 0.5, 0.0, 0.5, 0.5])[:, None].expand(T, H).clone()
    want[1, 5] = want[4, 7] = 0.0
    assert torch.equal(y, want)
    r = b.w4a4_unpermute_bwd(torch.ones(T, H, dtype=torch.bfloat16, device="cuda"), o, perm, w)
    dp = r["dtopk_w"].cpu()
    assert torch.isnan(dp[1, 0]) and torch.isinf(dp[4, 1])
    dp[1, 0] = dp[4, 1] = H
    assert torch.equal(dp, torch.tensor(np.where(row >= 0, float(H), 0.0), dtype=torch.float32))


def test_row_indices_outside_the_buffer_are_not_dispatched(b):
    """A map made for more rows than the buffer holds: the slots beyond it count as not dispatched."""
    T, k, H = 9, 2, 40
    row = np.arange(T * k).reshape(T, k)
    rows = 11
    perm = _perm(np.array([0, rows]), row, np.zeros(rows, dtype=np.int64), rows, k)
    print_case("dispatch_short_buffer", T=T, k=k, H=H, rows=rows)
    rng = np.random.default_rng(8)
    o, dy = _dev(rng.standard_normal((rows, H)), torch.float32), _dev(rng.standard_normal((T, H)), torch.float32)
    w = torch.ones(T, k, device="cuda")
    inside = np.where(row < rows, row, -1)
    assert np.allclose(_f64(b.w4a4_unpermute_fwd(o, perm, w)), dispatch.gather_sum(_f64(o), inside)[0], rtol=1e-6)
    r = b.w4a4_unpermute_bwd(dy, o, perm, w)
    do, dp, _ = dispatch.unpermute_bwd(_f64(dy), _f64(o), inside, np.ones((T, k)))
    assert np.allclose(_f64(r["do"]), do, rtol=1e-6) and not np.any(_f64(r["dtopk_w"])[inside < 0])


def test_a_token_does_not_depend_on_its_batch(b):
    """Also across the two ways to make the maps (one launch, three)."""
    T, k, H, E = 4000, 8, 1032, 64
    rng, idx, off, row, src, cap = _case(T, k, E, 1, "distinct", 9)
    print_case("dispatch_batches", T=T, k=k, H=H, E=E)
    ids, x = torch.from_numpy(idx).cuda(), _dev(rng.standard_normal((T, H)), torch.bfloat16)
    w = torch.from_numpy(rng.random((T, k)).astype(np.float32)).cuda()
    whole = b.w4a4_permute_fwd(x, ids, E)
    y, r = b.w4a4_unpermute_fwd(whole["xp"], whole, w), b.w4a4_unpermute_bwd(x, whole["xp"], whole, w)
    for t0, n in ((0, 1), (17, 100), (3990, 10)):
        part = b.w4a4_permute_fwd(x[t0:t0 + n], ids[t0:t0 + n], E)
        assert torch.equal(y[t0:t0 + n], b.w4a4_unpermute_fwd(part["xp"], part, w[t0:t0 + n]))
        p = b.w4a4_unpermute_bwd(x[t0:t0 + n], part["xp"], part, w[t0:t0 + n])
        assert torch.equal(r["dtopk_w"][t0:t0 + n], p["dtopk_w"])


def test_empty_batch(b):
    e = torch.empty
    print_case("dispatch_empty")
    x, ids, w = e(0, 64, dtype=torch.bfloat16, device="cuda"), e(0, 2, dtype=torch.int32, device="cuda"), e(0, 2, device="cuda")
    r = b.w4a4_permute_fwd(x, ids, 8, 16, out=dict(offsets=torch.full((9,), 5, dtype=torch.int32, device="cuda")))
    assert not r["offsets"].any() and r["xp"].shape == (120, 64)
    assert b.w4a4_permute_bwd(r["xp"], r).shape == (0, 64) and b.w4a4_unpermute_fwd(r["xp"], r, w).shape == (0, 64)
    assert b.w4a4_unpermute_bwd(x, r["xp"], r, w)["dtopk_w"].shape == (0, 2)


def test_rows_beyond_4_gib(b):
    """1.4 M expert rows of 4 KB (5.7 GB): rows and tokens at both ends."""
    T, k, H, E = 175_000, 8, 2048, 128
    print_case("dispatch_large", T=T, k=k, H=H, E=E)
    g = torch.Generator(device="cuda").manual_seed(3)
    ids = torch.rand(T, E, generator=g, device="cuda").topk(k, 1).indices.to(torch.int32)
    x = torch.randn(T, H, generator=g, device="cuda", dtype=torch.bfloat16)
    w = torch.rand(T, k, generator=g, device="cuda")
    r = b.w4a4_permute_fwd(x, ids, E)
    assert int(r["offsets"][-1]) == T * k
    assert torch.equal(r["src_row"].long()[r["row_map"].long()], torch.arange(T, device="cuda")[:, None].expand(T, k))
    for rows in (slice(0, 64), slice(T * k - 64, T * k), slice((1 << 20) - 32, (1 << 20) + 32)):
        assert torch.equal(r["xp"][rows], x[r["src_row"][rows].long()])
    y, grad = b.w4a4_unpermute_fwd(r["xp"], r, w), b.w4a4_unpermute_bwd(x, r["xp"], r, w)
    for ts in (slice(0, 8), slice(T - 8, T)):
        ref = (w[ts].double().sum(1)[:, None] * x[ts].double())
        assert bool(((y[ts].double() - ref).abs() <= (2.0 ** -8 + 16 * U) * ref.abs() + TINY).all())
        dp = x[ts].double().square().sum(1)
        assert bool(((grad["dtopk_w"][ts].double() - dp[:, None]).abs() <= 18 * U * 1.01 * dp[:, None]).all())
        assert torch.equal(grad["do"][r["row_map"][ts].long()], (w[ts][..., None] * x[ts][:, None, :].float()).bfloat16())


def test_more_entries_than_a_launch_holds(b):
    """2^26 + 40 entries of a wave each are more than 2^32 threads: two launches of
    the gradient, rows of both against the same tokens alone."""
    T, k, H = (1 << 23) + 5, 8, 8
    print_case("unpermute_bwd_launches", T=T, k=k, H=H)
    n = T * k
    g = torch.Generator(device="cuda").manual_seed(4)
    perm = dict(row_map=(n - 1 - torch.arange(n, dtype=torch.int32, device="cuda")).view(T, k),
                offsets=torch.tensor([0, n], dtype=torch.int32, device="cuda"),
                src_row=torch.zeros(n, dtype=torch.int32, device="cuda"))
    o = torch.randn(n, H, generator=g, device="cuda").bfloat16()
    dy, w = torch.randn(T, H, generator=g, device="cuda").bfloat16(), torch.rand(T, k, generator=g, device="cuda")
    r = b.w4a4_unpermute_bwd(dy, o, perm, w)
    y = b.w4a4_unpermute_fwd(o, perm, w)
    for t0 in (0, (1 << 23) - 8, T - 4):
        m = min(16, T - t0)
        rows = perm["row_map"][t0:t0 + m].long()
        small = dict(row_map=torch.arange(m * k, dtype=torch.int32, device="cuda").view(m, k),
                     offsets=torch.tensor([0, m * k], dtype=torch.int32, device="cuda"),
                     src_row=torch.zeros(m * k, dtype=torch.int32, device="cuda"))
        os = o[rows.view(-1)].contiguous()
        alone = b.w4a4_unpermute_bwd(dy[t0:t0 + m], os, small, w[t0:t0 + m])
        assert torch.equal(r["dtopk_w"][t0:t0 + m], alone["dtopk_w"])
        assert torch.equal(r["do"][rows.view(-1)], alone["do"])
        assert torch.equal(y[t0:t0 + m], b.w4a4_unpermute_fwd(os, small, w[t0:t0 + m]))


def test_more_chunks_than_a_launch_holds(b):
    """2^18 + 5 rows of 65536 in float32 are more than 2^32 chunks, a lane each: two
    launches of the combination (69 GB)."""
    T, k, H, rows = (1 << 18) + 5, 2, 65536, 5
    print_case("gather_launches", T=T, k=k, H=H)
    g = torch.Generator(device="cuda").manual_seed(5)
    perm = dict(row_map=torch.randint(-1, rows, (T, k), generator=g, device="cuda", dtype=torch.int32))
    o, w = torch.randn(rows, H, generator=g, device="cuda"), torch.rand(T, k, generator=g, device="cuda")
    y = b.w4a4_unpermute_fwd(o, perm, w)
    for t0 in (0, (1 << 18) - 4, T - 3):
        m = min(8, T - t0)
        part = dict(row_map=perm["row_map"][t0:t0 + m].contiguous())
        assert torch.equal(y[t0:t0 + m], b.w4a4_unpermute_fwd(o, part, w[t0:t0 + m].contiguous()))
    ref, mag = dispatch.gather_sum(_f64(o), perm["row_map"][-3:].cpu().numpy(), _f64(w[-3:]))
    assert np.all(np.abs(_f64(y[-3:]) - ref) <= 9 * U * mag + TINY)


def test_more_tokens_than_a_launch_holds(b):
    """2^24 + 5 tokens with a workgroup each are more than 2^32 threads: two launches of the copy (70 GB)."""
    T, H, E = (1 << 24) + 5, 1032, 3
    print_case("permute_launches", T=T, H=H, E=E)
    x = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(6)
    ids = torch.randint(0, E, (T, 1), generator=g, device="cuda", dtype=torch.int32)
    some = [0, 1, (1 << 24) - 9, (1 << 24) - 8, (1 << 24) - 1, 1 << 24, T - 1]
    for t in some:
        x[t] = torch.randn(H, generator=g, device="cuda").bfloat16()
    r = b.w4a4_permute_fwd(x, ids, E)
    count = torch.bincount(ids.view(-1), minlength=E)
    assert torch.equal(r["offsets"].long(), torch.cat((count.new_zeros(1), count.cumsum(0))))
    order = torch.argsort(ids.view(-1), stable=True)
    assert torch.equal(r["src_row"].long(), order)
    for t in some:
        assert torch.equal(r["xp"][int(r["row_map"][t, 0])], x[t])


@pytest.mark.parametrize("dtype,T,H,align", [("bf16", 8200, 2056, 16), ("f32", 5000, 2048, 1)])
def test_gradients_of_many_wide_rows(b, dtype, T, H, align):
    """Beyond 256 MiB of rows the two gradients come in passes of their own: the bits of
    each alone and of the same tokens in a small batch; pads zero, rows behind them left."""
    k, E, dt = 8, 24, TYPES[dtype]
    print_case("unpermute_bwd_apart", T=T, H=H, align=align, dtype=dtype)
    g = torch.Generator(device="cuda").manual_seed(12)
    ids = torch.randint(-2, E, (T, k), generator=g, device="cuda", dtype=torch.int32)
    x = torch.randn(T, H, generator=g, device="cuda").to(dt)
    w = torch.randn(T, k, generator=g, device="cuda")
    perm = b.w4a4_permute_fwd(x, ids, E, align)
    o = torch.randn(perm["xp"].shape, generator=g, device="cuda").to(dt)
    out = dict(do=torch.full_like(o, 7.0), dtopk_w=torch.full((T, k), 7.0, device="cuda"))
    r = b.w4a4_unpermute_bwd(x, o, perm, w, out=out)
    n = int(perm["offsets"][-1])
    assert bool((r["do"][n:] == 7).all())
    src, row = perm["src_row"][:n], perm["row_map"].long()
    assert not r["do"][:n][src < 0].any()
    live = row >= 0
    assert torch.equal(r["do"][row[live]], (w[..., None] * x[:, None, :].float())[live].to(dt))
    assert not r["dtopk_w"][~live].any()
    for t0 in (0, 4000, T - 60):
        part = b.w4a4_permute_fwd(x[t0:t0 + 60], ids[t0:t0 + 60].contiguous(), E)
        op = torch.zeros_like(part["xp"])
        op[part["row_map"].long()[live[t0:t0 + 60]]] = o[row[t0:t0 + 60][live[t0:t0 + 60]]]
        p = b.w4a4_unpermute_bwd(x[t0:t0 + 60], op, part, w[t0:t0 + 60].contiguous())
        assert torch.equal(p["dtopk_w"], r["dtopk_w"][t0:t0 + 60])


@pytest.mark.parametrize("dtype,T,H,k,align", [("bf16", 2100, 2056, 8, 16), ("f32", 2100, 1032, 8, 1),
                                               ("bf16", 8100, 520, 8, 32), ("bf16", 6000, 2808, 2, 1),
                                               ("f32", 2700, 1032, 7, 128)])
def test_many_rows_that_share_lines(b, dtype, T, H, k, align):
    """From 64 MiB of rows that 64 bytes do not divide each is written by the lines of its place: to buffers that
    start inside a line, from a column slice; rows behind the last group and beside the buffers are left."""
    E, dt = 19, TYPES[dtype]
    print_case("dispatch_lines", T=T, H=H, k=k, align=align, dtype=dtype)
    g = torch.Generator(device="cuda").manual_seed(T + H)
    ids = torch.randint(-1, E, (T, k), generator=g, device="cuda", dtype=torch.int32)
    x = torch.randn(T, H + 16, generator=g, device="cuda").to(dt)[:, 8:8 + H]
    w = torch.randn(T, k, generator=g, device="cuda")
    cap, skip = b.rows_capacity(T, k, E, align), 16 // x.element_size()
    flat = torch.full((2, cap * H + 2 * skip), 7.0, dtype=dt, device="cuda")
    xp, do = (flat[i, skip:-skip].view(cap, H) for i in range(2))
    perm = b.w4a4_permute_fwd(x, ids, E, align, out=dict(xp=xp))
    b.w4a4_unpermute_bwd(x, None, perm, w, dtopk_w=False, out=dict(do=do))
    n, row, live = int(perm["offsets"][-1]), perm["row_map"].long(), perm["row_map"] >= 0
    assert torch.equal(live, ids >= 0) and torch.equal(perm["src_row"].long()[row[live]], live.nonzero()[:, 0])
    assert torch.equal(xp[row[live]], x[live.nonzero()[:, 0]])
    assert torch.equal(do[row[live]], (w[..., None] * x[:, None, :].float())[live].to(dt))
    pad = perm["src_row"][:n] < 0
    assert int(pad.sum()) == n - int(live.sum())
    for out in (xp, do):
        assert not out[:n][pad].any() and bool((out[n:] == 7).all())
    assert bool((flat[:, :skip] == 7).all()) and bool((flat[:, -skip:] == 7).all())


@pytest.mark.parametrize("T,H,k,E", [(1, 8200, 1, 1), (9, 65536, 2, 3), (300, 4104, 2, 2), (5, 1032, 8, 600)])
def test_wide_pads_of_few_experts(b, T, H, k, E):
    """Pad rows that several workgroups clear for an expert."""
    print_case("dispatch_pads", T=T, H=H, k=k, E=E)
    g = torch.Generator(device="cuda").manual_seed(T + H)
    ids = torch.randint(0, E, (T, k), generator=g, device="cuda", dtype=torch.int32)
    x = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    w = torch.randn(T, k, generator=g, device="cuda")
    cap = b.rows_capacity(T, k, E, 128)
    full = lambda: torch.full((cap, H), 7.0, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    perm = b.w4a4_permute_fwd(x, ids, E, 128, out=dict(xp=full()))
    r = b.w4a4_unpermute_bwd(x, perm["xp"], perm, w, out=dict(do=full()))
    alone = b.w4a4_unpermute_bwd(x, None, perm, w, dtopk_w=False, out=dict(do=full()))
    n = int(perm["offsets"][-1])
    pad = perm["src_row"][:n] < 0
    assert int(pad.sum()) == n - T * k
    for out in (perm["xp"], r["do"], alone["do"]):
        assert not out[:n][pad].any() and bool((out[n:] == 7).all()) and bool((out[:n][~pad] != 7).any())
    assert torch.equal(r["do"], alone["do"])


def test_two_graphs_share_a_workspace(b):
    """Two captured calls on one workspace, replayed in turn with eager work between: each replay ranks anew."""
    T, k, H, E = 6100, 8, 64, 40
    print_case("dispatch_two_graphs", T=T, k=k, H=H, E=E)
    ws = torch.full((b.workspace_size(b.WS_PERMUTE, T, 0, 0, E, k),), 255, dtype=torch.uint8, device="cuda")
    assert ws.numel() > 0
    inputs, graphs = [], []
    for n in range(2):
        rng = np.random.default_rng(70 + n)
        x, ids = _dev(rng.standard_normal((T, H)), torch.bfloat16), torch.from_numpy(_ids(T, k, E, "any", rng)).cuda()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = b.w4a4_permute_fwd(x, ids, E, 32, workspace=ws)
        inputs.append((x, ids))
        graphs.append((graph, got))
    for _ in range(3):
        for (x, ids), (graph, got) in zip(inputs, graphs):
            graph.replay()
            torch.cuda.synchronize()
            want = b.w4a4_permute_fwd(x, ids, E, 32)
            n = int(want["offsets"][-1])
            assert torch.equal(got["offsets"], want["offsets"]) and torch.equal(got["row_map"], want["row_map"])
            assert torch.equal(got["src_row"][:n], want["src_row"][:n]) and torch.equal(got["xp"][:n], want["xp"][:n])
            ids.copy_(torch.roll(ids, 1, 0))


def test_streams_and_captured_graph(b):
    """A training step's four calls in one captured graph with a workspace of its
    own, replayed with new inputs between eager calls on another stream."""
    T, k, H, E = 700, 4, 520, 9
    rng, idx, off, row, src, cap = _case(T, k, E, 16, "partial", 10)
    print_case("dispatch_graph", T=T, k=k, H=H, E=E)
    static = dict(x=_dev(rng.standard_normal((T, H)), torch.bfloat16), ids=torch.from_numpy(idx).cuda(),
                  w=torch.from_numpy(rng.random((T, k)).astype(np.float32)).cuda())

    def step(s, buf):
        p = b.w4a4_permute_fwd(s["x"], s["ids"], E, 16, out=buf["perm"], workspace=buf["ws"])
        y = b.w4a4_unpermute_fwd(p["xp"], p, s["w"], y=buf["y"])
        g = b.w4a4_unpermute_bwd(y, p["xp"], p, s["w"], out=buf["grad"])
        return p, y, g, b.w4a4_permute_bwd(g["do"], p, dx=buf["dx"])

    def buffers():
        z = lambda dtype, *shape: torch.zeros(*shape, dtype=dtype, device="cuda")  # noqa: E731
        bf, i32 = torch.bfloat16, torch.int32
        return dict(perm=dict(xp=z(bf, cap, H), offsets=z(i32, E + 1), row_map=z(i32, T, k), src_row=z(i32, cap)),
                    ws=z(torch.uint8, b.workspace_size(b.WS_PERMUTE, T, 0, 0, E, k)), y=z(bf, T, H), dx=z(bf, T, H),
                    grad=dict(do=z(bf, cap, H), dtopk_w=z(torch.float32, T, k)))

    buf, other = buffers(), buffers()
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        step(static, buf)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p, y, g, dx = step(static, buf)
    for n in range(3):
        new = dict(x=_dev(rng.standard_normal((T, H)), torch.bfloat16),
                   ids=torch.from_numpy(_ids(T, k, E, ("partial", "any", "none")[n], rng)).cuda(),
                   w=torch.from_numpy(rng.random((T, k)).astype(np.float32)).cuda())
        for name, v in new.items():
            static[name].copy_(v)
        graph.replay()
        with torch.cuda.stream(stream):
            stream.wait_stream(torch.cuda.default_stream())
            ep, ey, eg, edx = step(new, other)
        torch.cuda.synchronize()
        rows = int(ep["offsets"][-1])
        assert torch.equal(p["offsets"], ep["offsets"]) and torch.equal(p["row_map"], ep["row_map"])
        assert torch.equal(p["xp"][:rows], ep["xp"][:rows]) and torch.equal(y, ey) and torch.equal(dx, edx)
        assert torch.equal(g["do"][:rows], eg["do"][:rows]) and torch.equal(g["dtopk_w"], eg["dtopk_w"])


def test_around_the_expert_calls(b):
    """Dispatch, the library's expert calls on the dispatched rows as tokens of
    their own (k = 1), and the way back give the bits of the calls that do all in
    one, forward and backward; and the gradient of the router's weights."""
    from precision_rl_amd import synth
    from gpu_util import bf16_dev
    T, H, E, k, I = 200, 512, 12, 3, 256  # noqa: E741
    d = synth.make_inputs(T, H, E, k, I, backward=True, n_empty=2, routing="zipf", seed=12)
    print_case("dispatch_chain", T=T, H=H, E=E, k=k, I=I)
    x, w1, w2, dy = (bf16_dev(d[n], torch) for n in ("x", "w1", "w2", "dy"))
    ids, p = torch.from_numpy(d["topk_idx"]).cuda(), torch.from_numpy(d["topk_w"]).cuda()
    w1q, w2q = b.quantize_weights(w1), b.quantize_weights(w2)
    xq = b.w4a4_quantize_permute(x, ids, E)
    f = b.w4a4_grouped_expert_fwd(xq, p, w1q, w2q, T, H, I, E, k, save=True)
    g = b.w4a4_expert_bwd(dy, x, w1, w2, f["h"], f["a"], p, xq, T, H, I, E, k)

    perm = b.w4a4_permute_fwd(x, ids, E)
    assert all(torch.equal(perm[m], xq[m]) for m in ("offsets", "row_map", "src_row"))
    R = T * k
    rows = b.w4a4_quantize_permute(perm["xp"], None, 1)
    assert torch.equal(rows["codes"], xq["codes"]) and torch.equal(rows["outer"], xq["outer"])
    each = torch.arange(R, dtype=torch.int32, device="cuda")
    rq = dict(rows, offsets=perm["offsets"], row_map=each[:, None].contiguous(), src_row=each)
    one = torch.ones(R, 1, device="cuda")
    fr = b.w4a4_grouped_expert_fwd(rq, one, w1q, w2q, R, H, I, E, 1, save=True)
    y = b.w4a4_unpermute_fwd(fr["y"], perm, p)
    assert torch.equal(y, f["y"]) and torch.equal(fr["h"], f["h"])
    back = b.w4a4_unpermute_bwd(dy, fr["y"], perm, p)
    gr = b.w4a4_expert_bwd(back["do"], perm["xp"], w1, w2, fr["h"], fr["a"], one, rq, R, H, I, E, 1)
    assert torch.equal(b.w4a4_permute_bwd(gr["dx"], perm), g["dx"])
    assert torch.equal(gr["dw1"], g["dw1"]) and torch.equal(gr["dw2"], g["dw2"])
    _, dp, mag = dispatch.unpermute_bwd(bf16_host(dy), bf16_host(fr["y"]), perm["row_map"].cpu().numpy(), _f64(p))
    assert np.all(np.abs(_f64(back["dtopk_w"]) - dp) <= 18 * U * 1.01 * mag)


def test_experts_of_two_ranks(b):
    """Each rank dispatches the slots of its own experts (the others' ids fall
    outside its range), runs its experts and combines: the ranks' sums are the
    whole layer's, and each slot's weight gradient comes from one rank."""
    from precision_rl_amd import synth
    from gpu_util import bf16_dev
    T, H, E, k, I, ranks = 150, 256, 8, 4, 128, 2  # noqa: E741
    d = synth.make_inputs(T, H, E, k, I, backward=True, seed=31)
    print_case("dispatch_ranks", T=T, H=H, E=E, k=k, I=I, ranks=ranks)
    x, w1, w2, dy = (bf16_dev(d[n], torch) for n in ("x", "w1", "w2", "dy"))
    ids, p = torch.from_numpy(d["topk_idx"]).cuda(), torch.from_numpy(d["topk_w"]).cuda()
    w1q, w2q = b.quantize_weights(w1), b.quantize_weights(w2)
    whole = b.w4a4_grouped_expert_fwd_ckpt(b.w4a4_quantize_permute(x, ids, E), p, w1q, w2q, T, H, I, E, k, save_o=True)
    perm = b.w4a4_permute_fwd(x, ids, E)
    dp = b.w4a4_unpermute_bwd(dy, whole["o"], perm, p, do=False)["dtopk_w"]
    ref, mag = dispatch.gather_sum(bf16_host(whole["o"]), perm["row_map"].cpu().numpy(), _f64(p))
    own, R = E // ranks, T * k
    each, one = torch.arange(R, dtype=torch.int32, device="cuda"), torch.ones(R, 1, device="cuda")
    y, dp_sum = torch.zeros(T, H, device="cuda"), torch.zeros(T, k, device="cuda")
    for r in range(ranks):
        mine = b.w4a4_permute_fwd(x, ids - r * own, own, out=dict(xp=torch.zeros(R, H, dtype=torch.bfloat16, device="cuda")))
        assert int(mine["offsets"][-1]) == int(((ids >= r * own) & (ids < (r + 1) * own)).sum())
        q = b.w4a4_quantize_permute(mine["xp"], None, 1)
        part = lambda w: {n: v[r * own:(r + 1) * own] for n, v in w.items()}  # noqa: E731
        o = b.w4a4_grouped_expert_fwd(dict(q, offsets=mine["offsets"], row_map=each[:, None].contiguous(), src_row=each),
                                      one, part(w1q), part(w2q), R, H, I, own, 1)["y"]
        y += b.w4a4_unpermute_fwd(o.float(), mine, p)
        dp_sum += b.w4a4_unpermute_bwd(dy, o, mine, p, do=False)["dtopk_w"]
    assert np.all(np.abs(_f64(y) - ref) <= 10 * U * mag + TINY)
    assert torch.equal(dp_sum, dp)


def test_calls_of_two_threads(b):
    """Two host threads on a stream each, batches of the one- and three-launch forms."""
    import threading
    print_case("dispatch_threads")
    shapes, got, want, errors = [(200, 8, 512, 32), (4100, 8, 264, 128)], {}, {}, []
    inputs = []
    for n, (T, k, H, E) in enumerate(shapes):
        rng = np.random.default_rng(60 + n)
        inputs.append((_dev(rng.standard_normal((T, H)), torch.bfloat16),
                       torch.from_numpy(_ids(T, k, E, "distinct", rng)).cuda(),
                       torch.from_numpy(rng.random((T, k)).astype(np.float32)).cuda(), E))

    def step(n):
        x, ids, w, E = inputs[n]
        p = b.w4a4_permute_fwd(x, ids, E)
        y = b.w4a4_unpermute_fwd(p["xp"], p, w)
        return p["row_map"], y, b.w4a4_unpermute_bwd(x, p["xp"], p, w)["dtopk_w"]

    for n in range(2):
        want[n] = step(n)
    torch.cuda.synchronize()

    def run(n):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(20):
                    got[n] = step(n)
                torch.cuda.current_stream().synchronize()
        except Exception as e:   # shown by the main thread
            errors.append(e)

    threads = [threading.Thread(target=run, args=(n,)) for n in range(2)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not errors, errors
    for n in range(2):
        assert all(torch.equal(a, c) for a, c in zip(got[n], want[n]))


def test_refusals(b):
    T, k, H, E = 8, 2, 64, 4
    x, ids = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda"), torch.zeros(T, k, dtype=torch.int32, device="cuda")
    w = torch.zeros(T, k, device="cuda")
    perm = b.w4a4_permute_fwd(x, ids, E)
    err = pytest.raises(b.W4A4Error)
    for call in (lambda: b.w4a4_permute_fwd(x.half(), ids, E), lambda: b.w4a4_permute_fwd(x, ids.long(), E),
                 lambda: b.w4a4_permute_fwd(x[:4], ids, E), lambda: b.w4a4_permute_fwd(x.cpu(), ids, E),
                 lambda: b.w4a4_permute_fwd(x, ids.cpu(), E), lambda: b.w4a4_permute_fwd(x, ids, 0),
                 lambda: b.w4a4_permute_fwd(x, ids, E, 3), lambda: b.w4a4_permute_fwd(x.t(), ids, E),
                 lambda: b.w4a4_permute_fwd(x, ids, E, out=dict(xp=x)), lambda: b.w4a4_permute_fwd(x[:, :60], ids, E),
                 lambda: b.w4a4_permute_fwd(x.repeat(8000, 1), ids.repeat(8000, 1), E,
                                            workspace=torch.empty(16, dtype=torch.uint8, device="cuda")),
                 lambda: b.w4a4_permute_bwd(perm["xp"].half(), perm), lambda: b.w4a4_permute_bwd(perm["xp"], perm, dx=x[:4]),
                 lambda: b.w4a4_unpermute_fwd(perm["xp"], perm, w.double()),
                 lambda: b.w4a4_unpermute_fwd(perm["xp"], perm, w[:4]),
                 lambda: b.w4a4_unpermute_fwd(perm["xp"], perm, w, y=x.float()),
                 lambda: b.w4a4_unpermute_bwd(x, None, perm, w), lambda: b.w4a4_unpermute_bwd(x, perm["xp"].float(), perm, w),
                 lambda: b.w4a4_unpermute_bwd(x, perm["xp"], perm, w, do=False, dtopk_w=False),
                 lambda: b.w4a4_unpermute_bwd(x, perm["xp"], perm, w, out=dict(do=perm["xp"]))):
        with err:
            call()
