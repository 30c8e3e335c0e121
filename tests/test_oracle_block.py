"""The float64 oracle of the feed-forward block's operators: values against torch's own
functions, gradients against central differences of the oracle's forward functions (CPU).

A central difference with step h is off by h^2 / 6 of the third derivative and by 2^-53 / h of
the sums; h = 1e-5 and values of order 1 to 100 leave less than 1e-6 of them."""

import numpy as np
import pytest
import torch

from oracle import block as O

H = 1e-5


def differences(f, x):
    """d f(x) / d x for a scalar f, element by element."""
    out = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        up, down = x.copy(), x.copy()
        up[i] += H
        down[i] -= H
        out[i] = (f(up) - f(down)) / (2 * H)
    return out


def agree(a, b):
    return np.all(np.abs(a - b) <= 1e-6 * (1.0 + np.abs(b).max()))


@pytest.mark.parametrize("act", ["relu", "silu", "gelu_tanh"])
def test_activations(act):
    v = np.linspace(-40.0, 40.0, 2001) + 0.003
    t = torch.from_numpy(v)
    want = {"relu": torch.relu(t), "silu": torch.nn.functional.silu(t),
            "gelu_tanh": torch.nn.functional.gelu(t, approximate="tanh")}[act].numpy()
    val, slope = O.activation(v, act)
    assert np.allclose(val, want, rtol=1e-12, atol=1e-14)
    diff = (O.activation(v + H, act)[0] - O.activation(v - H, act)[0]) / (2 * H)
    assert np.abs(slope - diff).max() < 1e-6


@pytest.mark.parametrize("act", ["relu", "silu", "gelu_tanh"])
def test_gated_gradient(act):
    rng = np.random.default_rng(1)
    w, x, dy = rng.normal(size=(6, 5)), rng.normal(size=(4, 5)), rng.normal(size=(4, 3))
    _, pre, _ = O.gated(w, x, 1.0, 1.0, None, act)
    dpre = O.gated_backward(dy, pre, act)
    loss = lambda w, x, c: (dy * O.gated(w, x, 1.0, 1.0, c, act)[0]).sum()  # noqa: E731
    assert agree(dpre, differences(lambda c: loss(w, x, c), np.zeros((4, 6))))
    assert agree(dpre @ w, differences(lambda v: loss(w, v, None), x))
    assert agree(dpre.T @ x, differences(lambda v: loss(v, x, None), w))


def test_gated_scales_and_addend():
    rng = np.random.default_rng(2)
    w, x, c = rng.normal(size=(4, 3)), rng.normal(size=(2, 3)), rng.normal(size=(2, 4))
    y, _, _ = O.gated(w, x, 0.5, 2.0, c, "silu")
    g, u = 0.5 * x @ w[:2].T + c[:, :2], 2.0 * x @ w[2:].T + c[:, 2:]
    assert np.allclose(y, torch.nn.functional.silu(torch.from_numpy(g)).numpy() * u)


OFFSETS, IDS = np.array([1, 3, 3, 6, 7, 9]), np.array([1, 0, 0, -1, 1])  # rows 0 and 9: in no group


def test_lora_gradient():
    rng = np.random.default_rng(3)
    x, a, b = rng.normal(size=(10, 4)), rng.normal(size=(3, 2, 4)), rng.normal(size=(3, 5, 2))
    scale, base, dy = np.array([0.5, 2.0, 1.0]), rng.normal(size=(10, 5)), rng.normal(size=(10, 5))
    out, z, _, _, written = O.lora(x, a, b, OFFSETS, IDS, scale, base, 5)
    assert list(written) == [False] + [True] * 8 + [False]
    assert np.array_equal(out[[0, 6, 9]], base[[0, 6, 9]])
    assert np.allclose(out[7], base[7] + 2.0 * b[1] @ (a[1] @ x[7]))
    loss = lambda x, a, b: (dy * O.lora(x, a, b, OFFSETS, IDS, scale, base, 5)[0]).sum()  # noqa: E731
    dx, da, db, *_ = O.lora_backward(dy, x, z, a, b, OFFSETS, IDS, scale, None)
    assert agree(dx, differences(lambda v: loss(v, a, b), x))
    assert agree(da, differences(lambda v: loss(x, v, b), a)) and not da[2].any()
    assert agree(db, differences(lambda v: loss(x, a, v), b)) and not db[2].any()


@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("gates", [0, 1, 3, 6])
def test_norm_gradient(post, gates):
    rng = np.random.default_rng([4, post, gates])
    r, o, dy, dr = (rng.normal(size=(6, 5)) for _ in range(4))
    w, wo, gate = rng.normal(size=5), rng.normal(size=5) if post else None, rng.normal(size=(gates, 5)) if gates else None

    def loss(r, o, w, wo, gate):
        y, res = O.norm(r, w, o, wo, gate, 0.7, 1e-3, lambda v: v)
        return (dy * y).sum() + (dr * res).sum()

    res = O.norm(r, w, o, wo, gate, 0.7, 1e-3, lambda v: v)[1]
    g = O.norm_backward(dy, dr, res, w, o, wo, gate, 0.7, 1e-3)
    assert agree(g["residual"], differences(lambda v: loss(v, o, w, wo, gate), r))
    assert agree(g["block"], differences(lambda v: loss(r, v, w, wo, gate), o))
    assert agree(g["weight"], differences(lambda v: loss(r, o, v, wo, gate), w))
    if post:
        assert agree(g["block_weight"], differences(lambda v: loss(r, o, w, v, gate), wo))
    if gates:
        assert agree(g["gate"], differences(lambda v: loss(r, o, w, wo, v), gate))


def test_plain_norm():
    rng = np.random.default_rng(5)
    x, w, dy = rng.normal(size=(3, 4)), rng.normal(size=4), rng.normal(size=(3, 4))
    y, res = O.norm(x, w, None, None, None, 0.5, 1e-6, lambda v: v)
    t = torch.from_numpy(x)
    assert np.array_equal(res, x) and np.allclose(y, (torch.nn.functional.rms_norm(t, (4,), torch.from_numpy(w), 1e-6)).numpy())
    g = O.norm_backward(dy, None, x, w, None, None, None, 0.5, 1e-6)
    loss = lambda x, w: (dy * O.norm(x, w, None, None, None, 0.5, 1e-6, lambda v: v)[0]).sum()  # noqa: E731
    assert agree(g["residual"], differences(lambda v: loss(v, w), x))
    assert agree(g["weight"], differences(lambda v: loss(x, v), w))
