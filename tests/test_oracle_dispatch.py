"""Pins of the oracle's dispatch and SwiGLU: the maps by hand, every gradient
against central differences in float64."""
import numpy as np
import pytest

from oracle import dispatch, moe

pytestmark = pytest.mark.cpu


def test_maps_by_hand():
    # expert 0: (0, 1); expert 1: (0, 0), (2, 0), (2, 1); expert 2: none; ids 7 and -1 are not dispatched
    idx = np.array([[1, 0], [7, -1], [1, 1]])
    off, row, src = dispatch.maps(idx, 3, 1)
    assert off.tolist() == [0, 1, 4, 4] and row.tolist() == [[1, 0], [-1, -1], [2, 3]] and src.tolist() == [0, 0, 2, 2]
    off, row, src = dispatch.maps(idx, 3, 16)
    assert off.tolist() == [0, 16, 32, 32] and row.tolist() == [[16, 0], [-1, -1], [17, 18]]
    assert src.tolist() == [0] + [-1] * 15 + [0, 2, 2] + [-1] * 13


@pytest.mark.parametrize("align", [1, 32])
def test_maps_are_the_routing_of_distinct_experts(align):
    rng = np.random.default_rng(3)
    idx = np.argsort(rng.random((57, 9)), axis=1)[:, :4]
    off, row, src = dispatch.maps(idx, 9, align)
    r = moe.route(idx, 9, align)
    for mine, theirs in zip((off, row, src), r if isinstance(r, tuple) else (r["offsets"], r["row_map"], r["src_row"])):
        assert np.array_equal(mine, theirs[:len(mine)])


def _difference(f, v, d, eps=1e-5):
    return (f(v + eps * d) - f(v - eps * d)) / (2 * eps)


def test_gradients_against_differences():
    """Central differences of step 1e-5: truncation below 1e-9 of values of
    order 1 (third derivatives of order 1), cancellation below 1e-10."""
    rng = np.random.default_rng(4)
    T, k, H = 11, 3, 24
    idx = rng.integers(-1, 5, (T, k))
    off, row, src = dispatch.maps(idx, 5, 16)
    x, o, w = rng.standard_normal((T, H)), rng.standard_normal((off[-1], H)), rng.random((T, k))
    dy, dxp = rng.standard_normal((T, H)), rng.standard_normal((off[-1], H))
    v = rng.standard_normal((T, H))
    assert np.isclose(_difference(lambda x: np.sum(dxp * dispatch.permute(x, row, off[-1])), x, v),
                      np.sum(dispatch.gather_sum(dxp, row)[0] * v), rtol=1e-8, atol=1e-8)
    do, dp, _ = dispatch.unpermute_bwd(dy, o, row, w)
    v = rng.standard_normal(o.shape)
    assert np.isclose(_difference(lambda o: np.sum(dy * dispatch.gather_sum(o, row, w)[0]), o, v), np.sum(do * v),
                      rtol=1e-8, atol=1e-8)
    v = rng.standard_normal(w.shape)
    assert np.isclose(_difference(lambda w: np.sum(dy * dispatch.gather_sum(o, row, w)[0]), w, v), np.sum(dp * v),
                      rtol=1e-8, atol=1e-8)
    h, da = 2 * rng.standard_normal((7, 2 * H)), rng.standard_normal((7, H))
    v = rng.standard_normal(h.shape)
    assert np.isclose(_difference(lambda h: np.sum(da * dispatch.swiglu(h)), h, v),
                      np.sum(dispatch.swiglu_bwd(da, h) * v), rtol=1e-7, atol=1e-7)


def test_swiglu_is_the_expert_forwards():
    h = np.random.default_rng(5).standard_normal((6, 64))
    assert np.allclose(dispatch.swiglu(h), moe.swiglu(h, 32), rtol=1e-15, atol=0)
