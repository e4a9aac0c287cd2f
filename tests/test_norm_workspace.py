"""The pre-norm backward's workspace as its caller gives it: anything but enough
dense bytes on the rows' device is refused, none is replaced."""
import pytest

torch = pytest.importorskip("torch")

NEED = 4096


def _bad(device):
    return {"too small": torch.empty(NEED - 1, dtype=torch.uint8, device=device),
            "empty": torch.empty(0, dtype=torch.uint8, device=device),
            "other type": torch.empty(NEED, dtype=torch.float32, device=device),
            "strided": torch.empty(2 * NEED, dtype=torch.uint8, device=device)[::2]}


@pytest.mark.cpu
def test_workspace_check():
    from precision_rl_amd import binding as b
    host = -1   # the device index of host tensors
    for name, ws in _bad("cpu").items():
        with pytest.raises(b.W4A4Error, match="workspace"):
            b._check_workspace(ws, NEED, host)
            print("not refused:", name)
    good = torch.empty(NEED, dtype=torch.uint8)
    b._check_workspace(good, NEED, host)
    b._check_workspace(good.view(64, -1), NEED, host)
    b._check_workspace(good, 0, host)
    with pytest.raises(b.W4A4Error, match="workspace"):
        b._check_workspace(good, NEED, 0)   # a host tensor for rows on a GPU


@pytest.mark.gpu
@pytest.mark.parametrize("T", [5, 700])
def test_norm_backward_refuses_workspaces(T):
    from precision_rl_amd import binding as b
    H = 256
    x = torch.ones(T, H, dtype=torch.bfloat16, device="cuda")
    g, r = torch.ones(H, device="cuda"), torch.ones(T, device="cuda")
    need = b.workspace_size(b.WS_RMSNORM_BACKWARD, T, H, 0, 1, 1)
    bad = {"host": torch.empty(max(need, 1), dtype=torch.uint8),
           "other type": torch.empty(max(need, 1), dtype=torch.float32, device="cuda"),
           "strided": torch.empty(2 * max(need, 2), dtype=torch.uint8, device="cuda")[::2]}
    if need:
        bad["too small"] = torch.empty(need - 1, dtype=torch.uint8, device="cuda")
    for name, ws in bad.items():
        with pytest.raises(b.W4A4Error, match="workspace"):
            b.w4a4_add_rmsnorm_bwd(x, x, g, r, workspace=ws)
            print("not refused:", name)
    want = b.w4a4_add_rmsnorm_bwd(x, x, g, r)
    got = b.w4a4_add_rmsnorm_bwd(x, x, g, r, workspace=torch.empty(need, dtype=torch.uint8, device="cuda"))
    assert torch.equal(got["dres"], want["dres"]) and torch.equal(got["dgamma"], want["dgamma"])
