"""Rows with one token far above the rest, as a trained model's are: logprobs, entropies and gradients keep the digits
of what the rest leaves (GPU).

Bounds, by arithmetic.  The row's own token enters z in 64 bits; r, the rest relative to it, in float32: a term's
exponential is off by 2^-22 (ex2.approx) and 2^-24 (its mean error, taken out), its exponent of 2 by half a step, 2^-20
below 32 (terms 2^-32 below the largest count for nothing), times ln 2; the temperature's log2(e) / T by 2^-24, that is
by 2^-24 of each distance from the token; and z has at most V / (16 x 128 x 1) + 16 additions in a thread's chain, 2^-24
each.  A term that stands far above the rest and is not the token's is off by 2^-22 + 2^-24 and by half a step of an
exponent below 8, 2^-22 ln 2; what an addition to it loses is at most what is added.  In 64 bits there remain, beside
numbers of size 1 (z = 1 + r and what its logarithm is taken from): the oracle's exponential, sum and logarithm, and the
kernel's exponent, exponential, sum, logarithm and difference, 8 half-steps of 2^-53; for the entropy twice as many.
"""
import numpy as np
import pytest
import torch

import vocab_sharded_logits_b200 as vsl
from oracle import scores as O

pytestmark = pytest.mark.gpu
STEP = 2.0 ** -24


def _rest_error(V, dist):
    return 2.0 ** -22 + 2 * STEP + 2.0 ** -20 * np.log(2) + dist * STEP + (V / 2048 + 16) * STEP


def _rows(V, height, seed, at):
    """16 rows of N(0, 2), one token of each `height` and a little above what the row begins with."""
    rng = np.random.default_rng([V, seed])
    l = (rng.normal(size=(16, V)) * 2).astype(np.float32)
    top = np.array([int(V * f) for f in np.linspace(*at, 16)]).clip(0, V - 1)
    l[np.arange(16), top] = (l.max(1) + height + rng.random(16)).astype(np.float32)
    return l, top.astype(np.int32)


def _slices(l, S, dev):
    return [torch.from_numpy(np.ascontiguousarray(x)).to(dev) for x in np.split(l, S, axis=1)]


def _np(x):
    return x.float().cpu().numpy().astype(np.float64)


SIZES = [(1024, 2), (20000, 4), (151936, 4)]
AT = [(0.0, 0.02), (0.3, 0.9999)]       # the token is among the first logits read, or far from them


@pytest.mark.parametrize("height", [3.0, 10.0, 18.0, 28.0, 80.0, 900.0])
@pytest.mark.parametrize("at", AT)
@pytest.mark.parametrize("V,S", SIZES)
def test_the_token_on_top(cuda_device, V, S, at, height):
    l, top = _rows(V, height, 1, at)
    logp = O.log_softmax(l)
    lp, ent = O.token_logprobs(l, top)
    p, dist = np.exp(logp), (logp[np.arange(16), top][:, None] - logp)
    p[np.arange(16), top] = 0.0
    rest, near = p.sum(1), np.where(p > 2.0 ** -60, dist, 0.0).max(1)
    eps = _rest_error(V, near)
    bound = rest * eps + STEP * np.abs(lp) + 2.0 ** -50
    slices, tok = _slices(l, S, cuda_device), torch.from_numpy(top).to(cuda_device)
    fwd = vsl.token_logprobs(slices, tok, entropy=True)
    one = torch.ones(16, device=cuda_device)
    pol = vsl.policy_loss(slices, tok, 0 * one, one, entropy_coef=0.01)
    # the entropy's terms p_j (dist_j + 1): each as p_j is, and its exponent's size beside it
    size = (p * (2 * dist + 34)).sum(1)
    for got in (fwd, pol):
        off = np.abs(_np(got.logprob) - lp)
        assert (off <= bound).all(), (off / bound).max()
        off = np.abs(_np(got.entropy) - ent)
        assert (off <= size * eps + STEP * ent + 2.0 ** -49).all(), (off / (size * eps + STEP * ent)).max()
    assert torch.equal(vsl.token_logprobs(slices, tok).logprob, fwd.logprob)


@pytest.mark.parametrize("height", [10.0, 17.0, 27.0, 36.0])
@pytest.mark.parametrize("at", AT)
@pytest.mark.parametrize("V,S", SIZES)
def test_another_token_on_top(cuda_device, V, S, at, height):
    """The row's token stands 1 below the top one: the top one's exponential is what its logprob rests on."""
    l, top = _rows(V, height, 2, at)
    tok = (top + V // 2 + 3) % V
    l[np.arange(16), tok] = l[np.arange(16), top] - 1.0
    logp = O.log_softmax(l)
    lp, ent = O.token_logprobs(l, tok)
    p = np.exp(logp)
    rows = np.arange(16)
    dist = np.abs(logp[rows, tok][:, None] - logp)
    p[rows, tok] = p[rows, top] = 0.0
    rest = p.sum(1)
    of_top = 2.0 ** -22 + 2 * STEP + 2.0 ** -22 * np.log(2) + 2 * STEP
    eps = _rest_error(V, np.where(p > 2.0 ** -60, dist, 0.0).max(1))
    bound = of_top + rest * (1 + eps) + STEP * np.abs(lp)
    slices, t = _slices(l, S, cuda_device), torch.from_numpy(tok).to(cuda_device)
    one = torch.ones(16, device=cuda_device)
    fwd = vsl.token_logprobs(slices, t, entropy=True)
    pol = vsl.policy_loss(slices, t, _dev(lp, cuda_device), one, entropy_coef=0.01)
    size = (p * (2 * dist + 34)).sum(1)
    for got in (fwd, pol):
        off = np.abs(_np(got.logprob) - lp)
        assert (off <= bound).all(), (off / bound).max()
        # log z and the top term's share of the mean, two nearly equal numbers below 8 ln 2 in size: two roundings
        # of the sum of e y beside the exponential's own error, which moves both
        off = np.abs(_np(got.entropy) - ent)
        assert (off <= 3 * of_top + 8 * STEP + size * (1 + eps) + STEP * ent).all(), off.max()
    # p of the top one in the gradient: as its exponential, z in 32 bits, and the coefficient
    g = np.concatenate([_np(x) for x in vsl.token_logprobs_grad(slices, t, fwd, one)], 1)
    want = O.token_logprobs_grad(l, tok, np.ones(16))
    off = np.abs(g - want)[rows, top]
    assert (off <= 2 * of_top + rest * (1 + eps) + 4 * STEP).all(), off.max()


def _dev(x, dev):
    return torch.from_numpy(np.asarray(x, np.float32)).to(dev)


def test_the_tokens_own_term_alone(cuda_device):
    """Nothing beside the token above -inf, or far below it: probability 1, entropy 0; and the token itself impossible."""
    V = 6000
    l = np.full((8, V), -np.inf, np.float32)
    t = np.array([0, V - 1, 77, 4097, 5, 6, 7, 8], np.int32)
    l[np.arange(8), t] = [0.0, -300.0, 5e6, np.finfo(np.float32).min, 2e9, 1.0, np.inf, np.nan]
    l[4] = np.where(np.isfinite(l[4]), l[4], -1e30)
    l[5, 9] = -5000.0
    slices, tok = _slices(l, 2, cuda_device), torch.from_numpy(t).to(cuda_device)
    one = torch.ones(8, device=cuda_device)
    fwd = vsl.token_logprobs(slices, tok, entropy=True)
    pol = vsl.policy_loss(slices, tok, 0 * one, one, entropy_coef=0.1)
    grad = np.concatenate([_np(x) for x in vsl.token_logprobs_grad(slices, tok, fwd, one, one)], 1)
    for got in (fwd, pol):
        assert (_np(got.logprob)[:6] == 0).all() and (_np(got.entropy)[:6] == 0).all()
        assert np.isnan(_np(got.logprob)[6:]).all() and np.isnan(_np(got.entropy)[6:]).all()
    # 1 - p_token: the exponential's, z's and the coefficient's roundings
    assert (np.abs(grad[:6]) <= 2.0 ** -22 + 2.0 ** -21).all() and np.isnan(grad[6:]).all()


@pytest.mark.parametrize("height", [3.0, 10.0, 18.0, 28.0])
@pytest.mark.parametrize("ent_coef", [0.0, 0.02])
@pytest.mark.parametrize("V,S", SIZES)
def test_the_gradient_at_a_token_on_top(cuda_device, V, S, ent_coef, height):
    """(g (1 - p) - h p (log p + H)) / T at the token.  The policy loss has the row's sums in 64 bits: 1 - p is what the
    rest leaves, not a difference of two numbers near 1.  The logprobs' gradient gets z and the entropy in 32 and takes
    the difference: p's exponential (2^-22 and its mean error), its exponent below 1/2 and the steps of z, the
    coefficients, their product and the difference."""
    l, top = _rows(V, height, 3, (0.3, 0.9999))
    rows = np.arange(16)
    logp = O.log_softmax(l)
    lp, ent = O.token_logprobs(l, top)
    p, dist = np.exp(logp), logp[rows, top][:, None] - logp
    p[rows, top] = 0.0
    rest, near = p.sum(1), np.where(p > 2.0 ** -60, dist, 0.0).max(1)
    eps, size = _rest_error(V, near), (p * (2 * dist + 34)).sum(1)
    slices, tok = _slices(l, S, cuda_device), torch.from_numpy(top).to(cuda_device)
    old = np.zeros(16, np.float32)
    want = O.policy_loss(l, top, old, -np.ones(16), ent_coef=np.float64(np.float32(ent_coef)))
    one = torch.ones(16, device=cuda_device)
    pol = vsl.policy_loss(slices, tok, 0 * one, -one, entropy_coef=ent_coef)
    got = np.concatenate([_np(x) for x in pol.grad], 1)[rows, top]
    exact = want["grad"][rows, top]
    # ratio exp(log p - old) moves with log p, by rest * eps; 1 - p, log p and H by the same and by size * eps
    bound = 2 * rest * eps + ent_coef * (rest + size) * eps + STEP * np.abs(exact) + 2.0 ** -48
    assert (np.abs(got - exact) <= bound).all(), (np.abs(got - exact) / bound).max()
    fwd = vsl.token_logprobs(slices, tok, entropy=True)
    h = np.full(16, ent_coef, np.float32)
    grad = vsl.token_logprobs_grad(slices, tok, fwd, one, _dev(h, cuda_device) if ent_coef else None)
    exact = O.token_logprobs_grad(l, top, np.ones(16), h.astype(np.float64))[rows, top]
    off = np.abs(np.concatenate([_np(x) for x in grad], 1)[rows, top] - exact)
    bound = (1 + 2 * ent_coef) * (2.0 ** -22 + 6 * STEP) + rest * eps + ent_coef * ((rest + size) * eps + STEP * ent)
    assert (off <= bound).all(), (off / bound).max()


@pytest.mark.parametrize("low", [-23.0, -25.0, -27.0, -100.0, -600.0, -2000.0])
@pytest.mark.parametrize("V,S", SIZES)
def test_rows_far_below_zero(cuda_device, V, S, low):
    """The top one at `low`, the row's token 1 below it, the others far down: as near 0 as far from it, the top one's
    exponential is what the logprob rests on."""
    rng = np.random.default_rng([V, int(-low)])
    l = (rng.normal(size=(16, V)) * 2 + low - 30).astype(np.float32)
    rows, top = np.arange(16), np.arange(16) * (V // 16) + 5
    tok = ((top + V // 2 + 3) % V).astype(np.int32)
    l[rows, top] = (low + np.arange(16) / 37.0).astype(np.float32)
    l[rows, tok] = l[rows, top] - np.float32(1.0)
    logp = O.log_softmax(l)
    lp, ent = O.token_logprobs(l, tok)
    p = np.exp(logp)
    p[rows, tok] = p[rows, top] = 0.0
    rest = p.sum(1)
    of_top = 2.0 ** -22 + 2 * STEP + 2.0 ** -22 * np.log(2) + 2 * STEP
    bound = of_top + 2 * rest + STEP * np.abs(lp)
    slices, t = _slices(l, S, cuda_device), torch.from_numpy(tok).to(cuda_device)
    one = torch.ones(16, device=cuda_device)
    fwd = vsl.token_logprobs(slices, t, entropy=True)
    pol = vsl.policy_loss(slices, t, _dev(lp, cuda_device), one, entropy_coef=0.01)
    for got in (fwd, pol):
        off = np.abs(_np(got.logprob) - lp)
        assert (off <= bound).all(), (off / bound).max()
        off = np.abs(_np(got.entropy) - ent)
        assert (off <= 3 * of_top + 8 * STEP + 80 * rest + STEP * ent).all(), off.max()
