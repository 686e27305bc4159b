"""Pins of the oracle's adapters, token logprobs and losses: independent formulations, closed forms and central
differences."""
import numpy as np
import pytest
from scipy.special import log_softmax as scipy_log_softmax

from oracle import adapters as A
from oracle import scores as O


def test_adapters_equal_the_merged_weights():
    rng = np.random.default_rng(0)
    R, H, S, V_s, n, rank = 7, 24, 3, 20, 3, 8
    hidden = rng.normal(size=(R, H))
    w = [rng.normal(size=(V_s, H)) for _ in range(S)]
    a, b = rng.normal(size=(n, rank, H)), [rng.normal(size=(n, V_s, rank)) for _ in range(S)]
    scale = rng.uniform(0.5, 2, n)
    ids = np.array([0, 2, -1, 1, 5, 0, 2])
    out = A.adapters_add([hidden @ x.T for x in w], hidden, a, b, ids, scale)
    for r, i in enumerate(ids):
        for s in range(S):
            merged = w[s] + (scale[i] * b[s][i] @ a[i] if 0 <= i < n else 0.0)
            assert np.allclose(out[s][r], merged @ hidden[r], rtol=1e-12, atol=1e-12)


@pytest.mark.parametrize("T", [1.0, 0.7])
def test_logprobs_and_entropy_equal_scipy(T):
    rng = np.random.default_rng(1)
    l = rng.normal(size=(5, 40)) * 4
    l[1, 3:20] = -np.inf
    tokens = np.array([3, 25, 0, -1, 40])
    want = scipy_log_softmax(l / T, axis=1)
    lp, ent = O.token_logprobs(l, tokens, T)
    p = np.exp(want)
    h = -np.where(p > 0, p * np.where(p > 0, want, 0), 0).sum(1)
    for r in range(3):
        assert abs(lp[r] - want[r, tokens[r]]) < 1e-12 and abs(ent[r] - h[r]) < 1e-12
    assert (lp[3:] == 0).all() and (ent[3:] == 0).all()       # tokens outside the vocabulary


def test_uniform_row_and_invalid_rows():
    l = np.zeros((5, 16))
    l[1, 2], l[2, 2], l[3] = np.nan, np.inf, -np.inf
    l[4] = np.finfo(np.float32).min
    lp, ent = O.token_logprobs(l, np.zeros(5, int))
    assert lp[0] == pytest.approx(-np.log(16)) and ent[0] == pytest.approx(np.log(16))
    assert np.isnan(lp[1:4]).all() and np.isnan(ent[1:4]).all()
    assert lp[4] == pytest.approx(-np.log(16))


def _difference(f, l, j, step=1e-5):
    up, down = l.copy(), l.copy()
    up[j] += step
    down[j] -= step
    return (f(up) - f(down)) / (2 * step)


def test_gradient_of_logprob_and_entropy_against_differences():
    rng = np.random.default_rng(2)
    R, V, T = 4, 9, 0.8
    l = rng.normal(size=(R, V)) * 2
    l[0, 4] = -np.inf
    tokens = np.array([0, 8, -1, 3])
    dl, de = rng.normal(size=R), rng.normal(size=R)

    def f(x):
        lp, ent = O.token_logprobs(x, tokens, T)
        return float((dl * lp + de * ent).sum())
    g = O.token_logprobs_grad(l, tokens, dl, de, T)
    for j in np.ndindex(R, V):
        if np.isfinite(l[j]):
            assert abs(g[j] - _difference(f, l, j)) < 1e-8
    assert g[0, 4] == 0 and (g[2] == 0).all()


@pytest.mark.parametrize("kl_coef,ent_coef", [(0.0, 0.0), (0.1, 0.0), (0.05, 0.02)])
def test_policy_gradient_against_differences(kl_coef, ent_coef):
    rng = np.random.default_rng(3)
    R, V, T = 8, 7, 1.3
    l = rng.normal(size=(R, V)) * 2
    tokens = rng.integers(0, V, R)
    tokens[6] = -1
    lp, _ = O.token_logprobs(l, np.maximum(tokens, 0), T)
    delta = np.array([0.0, 0.5, -0.5, 0.5, -0.5, 0.05, 0.0, 0.1])   # ratio inside, above and below the borders
    adv = np.array([1.0, 1.0, 1.0, -1.0, -1.0, 0.7, 1.0, 1.0])
    w = np.array([1, 1, 1, 1, 0.5, 1, 1, 0.0])
    kw = dict(T=T, weights=w, ref=lp + 0.3 * rng.normal(size=R), lo=0.2, hi=0.28, kl_coef=kl_coef, ent_coef=ent_coef)
    res = O.policy_loss(l, tokens, lp - delta, adv, **kw)
    f = lambda x: O.policy_loss(x, tokens, lp - delta, adv, **kw)["loss"].sum()  # noqa: E731
    for j in np.ndindex(R, V):
        assert abs(res["grad"][j] - _difference(f, l, j)) < 1e-8
    assert (res["grad"][6:] == 0).all() and (res["loss"][6:] == 0).all()


def test_policy_closed_forms():
    l = np.log(np.array([[0.5, 0.25, 0.25]]))
    one = lambda **kw: O.policy_loss(l, np.array([0]), **kw)  # noqa: E731
    assert one(old=[np.log(0.5)], adv=[2.0])["loss"][0] == pytest.approx(-2.0)                 # ratio 1
    r = one(old=[np.log(0.25)], adv=[2.0])                                                     # ratio 2: clipped to 1.2
    assert r["loss"][0] == pytest.approx(-2.4) and (r["grad"] == 0).all()
    r = one(old=[np.log(0.25)], adv=[-2.0])                                                    # ratio 2, A < 0: not clipped
    assert r["loss"][0] == pytest.approx(4.0) and r["grad"][0, 0] == pytest.approx(4.0 * 0.5)
    r = one(old=[np.log(0.5)], adv=[0.0], ref=[np.log(0.25)], kl_coef=1.0)
    assert r["kl"][0] == pytest.approx(0.5 - np.log(0.5) - 1)                                   # exp(d) - d - 1, d = log 0.5
    assert one(old=[np.log(0.5)], adv=[0.0], ent_coef=1.0)["loss"][0] == pytest.approx(-1.5 * np.log(2))


def test_preference_closed_forms_and_differences():
    rng = np.random.default_rng(4)
    lp, ref = rng.normal(size=12), rng.normal(size=12)
    at = np.array([1, 3, 3, 7, 10])                     # an empty rejected sequence; rows 0, 10, 11 in none
    w = np.array([1.0, 0.5])
    loss, rewards, d = O.preference_loss(lp, ref, at, 0.3, 0.1, w)
    s = [0.3 * (lp - ref)[i:j].sum() for i, j in zip(at[:-1], at[1:])]
    assert np.allclose(rewards.ravel(), s) and rewards[0, 1] == 0
    sig = lambda h: 1 / (1 + np.exp(-h))  # noqa: E731
    for q in range(2):
        h = s[2 * q] - s[2 * q + 1]
        assert loss[q] == pytest.approx(w[q] * (-0.9 * np.log(sig(h)) - 0.1 * np.log(sig(-h))))
    for r in range(12):
        diff = _difference(lambda x: O.preference_loss(x, ref, at, 0.3, 0.1, w)[0].sum(), lp, r)
        assert abs(d[r] - diff) < 1e-9
    assert (d[[0, 10, 11]] == 0).all()
    assert O.preference_loss(lp, lp, at, 0.3)[0] == pytest.approx([np.log(2)] * 2)
    loss, rewards, d = O.preference_loss(lp, ref, at, 0.3, weights=[0.0, 1.0])
    assert loss[0] == 0 and (rewards[0] == 0).all() and (d[1:3] == 0).all()
