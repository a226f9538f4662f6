"""CPU checks of the gated delta rule's and layer norm's oracles: central
differences of their own forwards, closed forms and identities."""
import numpy as np
import pytest

from oracle import gdelta as og


def inputs(B=2, T=5, H=4, G=2, K=3, V=2, seed=0, h0=True):
    r = np.random.default_rng(seed)
    x = dict(q=r.standard_normal((B, T, G, K)), k=r.standard_normal((B, T, G, K)), v=r.standard_normal((B, T, H, V)),
             a_raw=r.standard_normal((B, T, H)), b_raw=r.standard_normal((B, T, H)), a_log=r.uniform(-1, 1, H),
             dt_bias=r.uniform(-2, 0, H))
    x["h0"] = r.standard_normal((B, H, V, K)) if h0 else None
    return x


@pytest.mark.parametrize("h0", [True, False])
def test_gradients_are_central_differences(h0):
    x = inputs(h0=h0)
    dy = np.random.default_rng(9).standard_normal(x["v"].shape)
    g = og.backward(dy, **x)
    for name in g:
        num, step = np.empty_like(x[name]), 1e-6
        flat, out = x[name].reshape(-1), num.reshape(-1)
        for i in range(flat.size):
            keep = flat[i]
            flat[i] = keep + step
            up = (og.forward(**x)[0] * dy).sum()
            flat[i] = keep - step
            out[i] = ((up - (og.forward(**x)[0] * dy).sum())) / (2 * step)
            flat[i] = keep
        # step^2 truncation and 2^-53 / step cancellation are both below 1e-9 of values of order 1
        assert np.abs(num - g[name]).max() < 1e-7, name


def test_full_write_strength_without_decay_stores_the_value():
    """beta -> 1, alpha -> 1, one key twice: the state answers the last value, whatever was stored before."""
    x = inputs(B=1, T=2, H=1, G=1, K=4, V=3)
    x["k"][:, 1] = x["k"][:, 0]
    x["q"] = x["k"].copy()
    x["b_raw"][:] = 50.0
    x["a_raw"][:] = -800.0
    y, _ = og.forward(**x, scale=1.0, eps=1e-30)
    assert np.abs(y[:, 1] - x["v"][:, 1]).max() < 1e-12


def test_no_write_is_decay_alone():
    x = inputs()
    x["b_raw"][:] = -700.0
    _, last = og.forward(**x)
    g = -np.exp(x["a_log"]) * np.logaddexp(0, x["a_raw"] + x["dt_bias"])
    assert np.abs(last - np.exp(g.sum(1))[..., None, None] * x["h0"]).max() < 1e-12


def test_a_split_sequence_carries_its_state():
    x = inputs(T=7)
    y, last = og.forward(**x)
    seq = ("q", "k", "v", "a_raw", "b_raw")
    a, mid = og.forward(**{n: t[:, :3] if n in seq else t for n, t in x.items()})
    b, end = og.forward(**dict({n: t[:, 3:] if n in seq else t for n, t in x.items()}, h0=mid))
    assert np.abs(np.concatenate([a, b], 1) - y).max() < 1e-13 and np.abs(end - last).max() < 1e-13


def test_layernorm_gradients_are_central_differences():
    r = np.random.default_rng(3)
    x, w, b, dy = r.standard_normal((3, 5)), r.standard_normal(5), r.standard_normal(5), r.standard_normal((3, 5))
    dx, dw, db = og.layernorm_backward(dy, x, w)
    for a, g in ((x, dx), (w, dw), (b, db)):
        flat = a.reshape(-1)
        for i in range(flat.size):
            keep = flat[i]
            flat[i] = keep + 1e-6
            up = (og.layernorm_forward(x, w, b)[0] * dy).sum()
            flat[i] = keep - 1e-6
            down = (og.layernorm_forward(x, w, b)[0] * dy).sum()
            flat[i] = keep
            assert abs((up - down) / 2e-6 - g.reshape(-1)[i]) < 1e-7


def test_layernorm_constant_row():
    y, mean, rstd = og.layernorm_forward(np.full((1, 8), 3.0), np.ones(8), np.full(8, 0.25), eps=1e-4)
    assert np.all(y == 0.25) and mean[0] == 3.0 and abs(rstd[0] - 100.0) < 1e-9
