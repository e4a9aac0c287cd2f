"""Both gradients of the combination of many wide rows, which come in one pass or
two by the share of the slots that are dispatched: the same bits as each by
itself, on both sides of the border (five eighths of the slots in use)."""
import pytest

from gpu_util import print_case

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

T, K, E = 8300, 8, 24


@pytest.fixture(scope="module")
def b():
    from precision_rl_amd import binding
    return binding


@pytest.mark.parametrize("dtype,H", [(torch.bfloat16, 2048), (torch.float32, 1032)])
@pytest.mark.parametrize("align", [1, 32])
@pytest.mark.parametrize("live", [0, 1, T * K // 4, T * K // 8 * 5 - 1, T * K // 8 * 5, T * K])
def test_gradients_by_the_share_of_slots(b, dtype, H, align, live):
    print_case("unpermute_bwd_share", dtype=dtype, H=H, align=align, live=live)
    g = torch.Generator(device="cuda").manual_seed(live + H)
    ids = torch.randint(0, E, (T, K), generator=g, device="cuda", dtype=torch.int32)
    ids.view(-1)[torch.randperm(T * K, generator=g, device="cuda")[live:]] = -1
    dy = torch.randn(T, H, generator=g, device="cuda").to(dtype)
    w = torch.randn(T, K, generator=g, device="cuda")
    perm = b.w4a4_permute_fwd(None, ids, E, align)
    n, cap = int(perm["offsets"][-1]), b.rows_capacity(T, K, E, align)
    o = torch.randn(cap, H, generator=g, device="cuda").to(dtype)
    out = lambda: dict(do=torch.full((cap, H), 7.0, dtype=dtype, device="cuda"),  # noqa: E731
                       dtopk_w=torch.full((T, K), 7.0, device="cuda"))
    both = b.w4a4_unpermute_bwd(dy, o, perm, w, out=out())
    row = perm["row_map"].long()
    assert int((row >= 0).sum()) == live
    want = torch.full((cap, H), 7.0, dtype=dtype, device="cuda")
    want[:n] = 0
    want[row[row >= 0]] = (w[..., None] * dy[:, None, :].float())[row >= 0].to(dtype)
    assert torch.equal(both["do"], want)
    assert torch.equal(both["dtopk_w"], b.w4a4_unpermute_bwd(dy, o, perm, w, do=False, out=out())["dtopk_w"])
    assert not both["dtopk_w"][row < 0].any() and bool((both["dtopk_w"][row >= 0] != 7).all())
    assert torch.equal(b.w4a4_unpermute_bwd(dy, None, perm, w, dtopk_w=False, out=out())["do"], want)
