"""The training operators' oracle against differences and closed forms."""
import numpy as np
import pytest

from oracle import train_oracle as to


def _difference(f, a, eps=1e-5):
    g = np.zeros_like(a)
    for i in np.ndindex(*a.shape):
        keep = a[i]
        a[i] = keep + eps
        up = f()
        a[i] = keep - eps
        g[i] = (up - f()) / (2 * eps)
        a[i] = keep
    return g


@pytest.mark.parametrize("form", ["full", "bias", "d2t"])
@pytest.mark.parametrize("reduction", ["mean", "sum"])
@pytest.mark.parametrize("markov", [True, False])
def test_loss_gradients_match_differences(form, reduction, markov):
    rng = np.random.default_rng(7)
    T, H, V, r = 5, 4, 9, 3
    d2t = np.array([0, 2, 3, 7, 8]) if form == "d2t" else None
    Vh = V if d2t is None else len(d2t)
    bias = np.where(np.arange(V) % 3 == 1, -1e9, 0.3) if form == "bias" else None
    h, W = rng.normal(size=(T, H)), rng.normal(size=(Vh, H))
    w1 = rng.normal(size=(V, r)) if markov else None
    w2 = rng.normal(size=(r, Vh)) if markov else None
    args = dict(labels=[2, 3, -1, 4, 8], prev=[1, 0, 5, 1, 1] if markov else None, w1=w1, w2=w2,
                lm_bias=bias, d2t=d2t, weights=np.array([1.0, 0.5, 3.0, 2.0, 0.0]),
                reduction=reduction, loss_scale=1.7, V=V)
    o = to.head_loss(h, W, **args)
    assert o["n_rows"] == {"full": 4, "bias": 3, "d2t": 3}[form]
    total = lambda: to.head_loss(h, W, **args)["total"]   # noqa: E731
    pairs = [("d_hidden", h), ("d_lm_head", W)]
    if markov:
        pairs += [("d_markov_w1", w1), ("d_markov_w2", w2)]
    for name, a in pairs:
        np.testing.assert_allclose(o[name], _difference(total, a), atol=2e-8)


def test_loss_of_equal_logits_is_the_log_of_the_emittable_rows():
    bias = np.array([0.0, -1e9, 0.0, 0.0, -1e9])
    o = to.head_loss(np.zeros((3, 2)), np.ones((5, 2)), [0, 1, 3], lm_bias=bias)
    np.testing.assert_allclose(o["loss"], [np.log(3), 0, np.log(3)])
    assert o["n_rows"] == 2 and not o["d_lm_head"][[1, 4]].any()


def test_loss_without_rows_is_zero():
    o = to.head_loss(np.ones((2, 2)), np.ones((3, 2)), [-1, 5])
    assert o["total"] == 0 and o["n_rows"] == 0 and not o["d_hidden"].any()


@pytest.mark.parametrize("y", [True, False])
@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("span", [0, 1, 3])
def test_norm_gradients_match_differences(y, post, span):
    if not y and (post or span):
        pytest.skip("w_post and gate act on y")
    rng = np.random.default_rng(3)
    T, H = 5, 6
    x, w_pre = rng.normal(size=(T, H)), rng.normal(size=H)
    yy = rng.normal(size=(T, H)) if y else None
    w_post = rng.normal(size=H) if post else None
    gate = rng.normal(size=((T + span - 1) // span, H)) if span else None
    dh, up = rng.normal(size=(T, H)), rng.normal(size=(T, H))
    kw = dict(gate=gate, w_post=w_post, eps=1e-3, scale=0.7, offset=1.0, span=max(1, span))

    def total():
        xo, h = to.block_norm(x, yy, w_pre, **kw)
        return (xo * up).sum() + (h * dh).sum()

    o = to.block_norm_backward(x, yy, w_pre, dh, up, **kw)
    for name, a in (("d_x", x), ("d_y", yy), ("d_gate", gate), ("d_w_post", w_post),
                    ("d_w_pre", w_pre)):
        if a is not None:
            np.testing.assert_allclose(o[name], _difference(total, a), atol=2e-8)


def test_clip():
    norm, out = to.clip_grads([np.array([3.0]), np.array([0.0, 4.0])], 2.5)
    assert norm == 5.0
    np.testing.assert_allclose(out[0], [1.5], rtol=1e-6)
    norm, out = to.clip_grads([np.array([3.0])], 10.0)
    assert out[0][0] == 3.0
    _, out = to.clip_grads([np.array([np.inf, 1.0])], 1.0)
    assert out[0][1] == 1.0
