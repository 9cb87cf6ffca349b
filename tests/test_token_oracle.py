"""The fp64 definitions of the operators on tokens, against results worked out by hand."""
import numpy as np
import pytest

from oracle import token_oracle as to

INF = float("inf")
LN = np.log


def test_order_and_top():
    z = [1.0, -INF, 3.0, 1.0, np.nan, 3.0]
    assert list(to.order(z)) == [2, 5, 0, 3]
    ids, values, lse = to.top_row([LN(2.0), LN(1.0), LN(5.0)], 2)
    assert list(ids) == [2, 0] and np.allclose(values, [LN(5.0), LN(2.0)]) and np.isclose(lse, LN(8.0))
    ids, values, lse = to.top_row([-INF, 0.0], 2)
    assert list(ids) == [1, -1] and values[1] == -INF and lse == 0.0


# weights 8, 4, 2, 1, 1 (of 16) at ids 3, 0, 4, 1, 2
ROW = LN(np.array([4.0, 1.0, 1.0, 8.0, 2.0]))


@pytest.mark.parametrize("u,settings,token,share", [
    # by id: 4, 5, 6, 14, 16
    (0.0, {}, 0, 4 / 16), (0.24, {}, 0, 4 / 16), (0.26, {}, 1, 1 / 16), (0.33, {}, 2, 1 / 16),
    (0.5, {}, 3, 8 / 16), (0.9, {}, 4, 2 / 16), (1.0, {}, 4, 2 / 16), (np.nan, {}, 0, 4 / 16),
    # the three first of the order: 4, 12, 14
    (0.27, dict(top_k=3), 0, 4 / 14), (0.3, dict(top_k=3), 3, 8 / 14), (0.9, dict(top_k=3), 4, 2 / 14),
    # the shortest prefix with 12.8 of 16 (8, 4 and 2), and with 11.9 of 14 (8 and 4)
    (0.9, dict(top_p=0.8), 4, 2 / 14), (0.9, dict(top_k=3, top_p=0.85), 3, 8 / 12),
    (0.1, dict(top_p=0.0), 3, 1.0), (0.99, dict(top_p=0.7), 3, 8 / 12),
    # weights of at least a quarter of the largest
    (0.9, dict(min_p=0.25), 4, 2 / 14), (0.99, dict(min_p=0.3), 3, 8 / 12),
    # squares of the weights: 16, 1, 1, 64, 4 of 86
    (0.19, dict(temperature=0.5), 1, 1 / 86), (0.5, dict(temperature=0.0), 3, 1.0),
])
def test_sample(u, settings, token, share):
    t, lp, _ = to.sample_row(ROW, u, **settings)
    assert t == token and np.isclose(lp, LN(share))


def test_sample_of_nothing():
    assert to.sample_row([-INF, np.nan], 0.5)[:2] == (-1, -INF)


def test_embed_and_its_gradient():
    out = to.embed([[1.0, 2.0], [3.0, 4.0]], np.array([1, -1, 0, 2]), 0.5)
    assert out.tolist() == [[1.5, 2.0], [0, 0], [0.5, 1.0], [0, 0]]
    g, mag = to.embed_backward(np.array([1, 1, -1, 0, 5]), [[1.0], [-3.0], [9.0], [2.0], [9.0]], 3, 2.0,
                               [[1.0], [1.0], [1.0]])
    assert g.tolist() == [[5.0], [-3.0], [1.0]] and mag.tolist() == [[4.0], [8.0], [0.0]]


def _loss(ids, logits, **kw):
    """A head whose logits are log 1, log 2, log 5 of 8, one hidden value of 1."""
    W = LN(np.array([[1.0], [2.0], [5.0]]))
    return to.distill_loss(np.ones((1, 1)), W, np.array([ids]), np.array([logits]), **kw)


def test_distillation():
    # q = 1/4 and 3/4 on tokens 1 and 2, p = 1/4 and 5/8
    o = _loss([2, 1], [LN(3.0), 0.0])
    assert np.isclose(o["loss"][0], 0.75 * LN(0.75 / 0.625))
    assert np.isclose(o["d_hidden"][0, 0], 0.125 * LN(1.0) + 0.0 * LN(2.0) - 0.125 * LN(5.0))
    assert np.allclose(o["d_lm_head"], [[0.125], [0.0], [-0.125]])
    # the teacher's own log-sum-exp: q = 1/8 and 3/8, Q = 1/2
    o = _loss([2, 1], [LN(3.0), 0.0], lse=[LN(8.0)])
    assert np.isclose(o["loss"][0], 0.375 * LN(0.375 / 0.625) + 0.125 * LN(0.125 / 0.25))
    assert np.allclose(o["d_lm_head"], [[0.0625], [0.0], [0.3125 - 0.375]])
    # half the temperature
    o = _loss([2, 1], [LN(3.0), 0.0], t_scale=2.0)
    assert np.isclose(o["loss"][0], 0.9 * LN(0.9 / 0.625) + 0.1 * LN(0.1 / 0.25))


@pytest.mark.parametrize("ids,logits,rows,dropped", [
    ([2, 1, -1], [0.0, 0.0, 0.0], 1, 0), ([2, 1, 1], [0.0, 0.0, -INF], 1, 0),
    ([2, 1, 3], [0.0, 0.0, -INF], 1, 0), ([2, 1, 3], [0.0, 0.0, 0.0], 0, 1),
    ([2, 1, 1], [0.0, 0.0, 0.0], 0, 1), ([-1, 3, 2 ** 31 - 1], [0.0, -INF, -INF], 0, 0)])
def test_which_rows_of_lists_count(ids, logits, rows, dropped):
    o = _loss(ids, logits)
    assert (o["n_rows"], o["dropped"]) == (rows, dropped)
    if rows:
        assert np.isclose(o["loss"][0], 0.5 * LN(0.5 / 0.625) + 0.5 * LN(0.5 / 0.25))
