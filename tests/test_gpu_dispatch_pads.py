"""Pad rows of the combination's gradient in buffers that hold no more rows than
there are slots: with slots that are not dispatched the groups may be padded
all the same.  Copies and zeros are compared bit for bit, rows behind those in
use stay as they were."""
import pytest

from gpu_util import print_case

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def b():
    from precision_rl_amd import binding
    return binding


def _cut(perm, rows):
    """The maps beside buffers of `rows` rows."""
    return dict(perm, src_row=perm["src_row"][:rows].contiguous())


# rows of a chunk, of several lanes, of a wave and beyond; one pass and (2048 in bf16, 8300
# tokens) two; rows that share cache lines, from 64 MiB of them written by their lines; one
# expert, experts of which most get nothing
@pytest.mark.parametrize("dtype,T,k,H,E,ep,align", [
    ("bf16", 1000, 8, 256, 32, 4, 128), ("f32", 1000, 8, 64, 32, 4, 128), ("bf16", 61, 8, 2048, 8, 4, 16),
    ("f32", 300, 4, 1032, 1, 3, 64), ("bf16", 5, 8, 8, 2, 6, 16), ("bf16", 8300, 8, 2048, 32, 4, 128),
    ("bf16", 8300, 8, 520, 32, 4, 32), ("f32", 2700, 7, 1032, 19, 4, 128), ("bf16", 40, 8, 8200, 300, 40, 16)])
def test_pads_of_a_buffer_cut_to_the_rows_in_use(b, dtype, T, k, H, E, ep, align):
    dt = TYPES[dtype]
    print_case("unpermute_bwd_cut", dtype=dtype, T=T, k=k, H=H, E=E, ep=ep, align=align)
    g = torch.Generator(device="cuda").manual_seed(T + H)
    # experts of `ep` ranks, this one's first; the first token has a slot here
    ids = torch.randint(0, E * ep, (T, k), generator=g, device="cuda", dtype=torch.int32)
    ids[0, 0] = 0
    dy, w = torch.randn(T, H, generator=g, device="cuda").to(dt), torch.randn(T, k, generator=g, device="cuda")
    perm = b.w4a4_permute_fwd(None, ids, E, align)
    n = int(perm["offsets"][-1])
    assert n < T * k
    row = perm["row_map"].long()
    want = torch.zeros(n, H, dtype=dt, device="cuda")
    want[row[row >= 0]] = (w[..., None] * dy[:, None, :].float())[row >= 0].to(dt)
    pads = int((perm["src_row"][:n] < 0).sum())
    assert pads == n - int((row >= 0).sum()) and pads > 0
    # cut to the rows in use, inside the last group's padding (or its slots), at the slots' number
    for rows in (n, n - 3, T * k):
        part, used = _cut(perm, rows), min(n, rows)
        o = torch.randn(rows, H, generator=g, device="cuda").to(dt)
        out = lambda: dict(do=torch.full((rows, H), 7.0, dtype=dt, device="cuda"))  # noqa: E731
        both = b.w4a4_unpermute_bwd(dy, o, part, w, out=out())
        alone = b.w4a4_unpermute_bwd(dy, None, part, w, dtopk_w=False, out=out())
        for r in (both, alone):
            assert torch.equal(r["do"][:used], want[:used]) and bool((r["do"][used:] == 7).all()), rows
        whole = b.w4a4_unpermute_bwd(dy, o, part, w, do=False)
        assert torch.equal(whole["dtopk_w"], both["dtopk_w"])


def test_every_row_is_padding_but_one(b):
    """Groups of one slot and 127 pads, in a buffer cut between two groups."""
    T, k, H, E = 300, 8, 72, 4
    print_case("unpermute_bwd_cut_single", T=T, k=k, H=H, E=E)
    ids = torch.full((T, k), -1, dtype=torch.int32, device="cuda")
    for e in range(E):
        ids[17 * e, e] = e
    perm = b.w4a4_permute_fwd(None, ids, E, 128)
    dy, w = torch.ones(T, H, device="cuda"), torch.full((T, k), 2.0, device="cuda")
    for rows in (128, 129, 256, 384, 511, 512):
        do = torch.full((rows, H), 7.0, device="cuda")
        b.w4a4_unpermute_bwd(dy, None, _cut(perm, rows), w, dtopk_w=False, out=dict(do=do))
        want = torch.zeros(rows, H, device="cuda")
        want[::128] = 2.0
        assert torch.equal(do, want), rows


def test_unpadded_groups_have_no_pads(b):
    """The last row of a group is a slot's where nothing is padded; short and full buffers."""
    T, k, H, E = 200, 4, 136, 7
    print_case("unpermute_bwd_unpadded", T=T, k=k, H=H, E=E)
    g = torch.Generator(device="cuda").manual_seed(2)
    ids = torch.randint(-2, E, (T, k), generator=g, device="cuda", dtype=torch.int32)
    dy, w = torch.randn(T, H, generator=g, device="cuda"), torch.randn(T, k, generator=g, device="cuda")
    perm = b.w4a4_permute_fwd(None, ids, E)
    n, row = int(perm["offsets"][-1]), perm["row_map"].long()
    want = torch.full((T * k, H), 7.0, device="cuda")
    want[row[row >= 0]] = (w[..., None] * dy[:, None, :])[row >= 0]
    for rows in (n - 1, n, T * k):
        do = torch.full((rows, H), 7.0, device="cuda")
        b.w4a4_unpermute_bwd(dy, None, _cut(perm, rows), w, dtopk_w=False, out=dict(do=do))
        assert torch.equal(do, want[:rows]), rows
