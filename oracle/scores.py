"""Oracle of the logprobs of given tokens, their gradient, and the policy and preference losses: float64.

Test infrastructure only: shares no code with the CUDA path.  Rows whose token lies outside the vocabulary (or, in
the losses, whose weight is 0) do not count: zeros.  A row with a NaN or +inf logit, or with none above -inf: NaN.
"""
import numpy as np


def log_softmax(l, T=1.0):
    """[R, V] log-probabilities of logits l at temperature T; -inf where l is -inf, NaN for an invalid row."""
    x = np.asarray(l, np.float64) / T
    with np.errstate(all="ignore"):
        top = x.max(1, keepdims=True)
        shifted = x - top  # before the sum's logarithm: it would be lost beside a large top
        out = shifted - np.log(np.exp(shifted).sum(1, keepdims=True))
    bad = np.isnan(x).any(1) | (x == np.inf).any(1) | (x == -np.inf).all(1)
    out[bad] = np.nan
    return out


def _plogp(logp):
    with np.errstate(all="ignore"):
        return np.where(logp == -np.inf, 0.0, np.exp(logp) * logp)


def counts(tokens, V, weights=None):
    tokens = np.asarray(tokens)
    on = (tokens >= 0) & (tokens < V)
    return on if weights is None else on & (np.asarray(weights) != 0)


def token_logprobs(l, tokens, T=1.0):
    """(logprob, entropy) of each row's token."""
    logp = log_softmax(l, T)
    on = counts(tokens, logp.shape[1])
    t = np.where(on, tokens, 0)
    lp = np.where(on, logp[np.arange(len(t)), t], 0.0)
    ent = np.where(on, -_plogp(logp).sum(1), 0.0)
    return lp, ent


def token_logprobs_grad(l, tokens, d_logprob, d_entropy=None, T=1.0, on=None):
    """[R, V] gradient of sum(d_logprob * logprob + d_entropy * entropy)."""
    logp = log_softmax(l, T)
    R, V = logp.shape
    on = counts(tokens, V) if on is None else on
    d_logprob = np.asarray(d_logprob, np.float64)
    d_entropy = np.zeros(R) if d_entropy is None else np.asarray(d_entropy, np.float64)
    on = on & ((d_logprob != 0) | (d_entropy != 0))
    with np.errstate(all="ignore"):
        p = np.exp(logp)
        ent = -_plogp(logp).sum(1)
        g = -p * d_logprob[:, None]
        shift = np.where(logp == -np.inf, 0.0, logp + ent[:, None])
        g = np.where((d_entropy != 0)[:, None], g - d_entropy[:, None] * p * shift, g)
        t = np.where(on, tokens, 0)
        g[np.arange(R), t] += d_logprob
        g /= T
    return np.where(on[:, None], g, 0.0)


def policy_rows(lp, ent, tokens, V, old, adv, weights=None, ref=None, lo=0.2, hi=0.2, kl_coef=0.0, ent_coef=0.0):
    """Per row (loss, kl, dloss/dlogprob, dloss/dentropy) from its logprob and entropy."""
    R = len(lp)
    w = np.ones(R) if weights is None else np.asarray(weights, np.float64)
    on = counts(tokens, V, weights)
    old, adv = np.asarray(old, np.float64), np.asarray(adv, np.float64)
    with np.errstate(all="ignore"):
        ratio = np.exp(lp - old)
        free, clip = ratio * adv, np.clip(ratio, 1 - lo, 1 + hi) * adv
        loss = -np.minimum(free, clip)
        g = np.where(np.isnan(free), np.nan, np.where(free <= clip, -adv * ratio, 0.0))
        kl = np.zeros(R)
        if ref is not None:
            d = np.asarray(ref, np.float64) - lp
            kl = np.where(d > 700, np.inf, np.expm1(d) - d)  # not inf - inf
            if kl_coef:
                loss = loss + kl_coef * kl
                g = g - kl_coef * np.expm1(d)
        if ent_coef:
            loss = loss - ent_coef * ent
        loss = w * loss
    zero = lambda x: np.where(on, x, 0.0)  # noqa: E731
    return zero(loss), zero(kl), zero(w * g), zero(-w * ent_coef * np.ones(R))


def policy_loss(l, tokens, old, adv, T=1.0, weights=None, ref=None, **coef):
    """dict of loss, logprob, kl, entropy [R] and grad [R, V] (the gradient of loss.sum())."""
    V = np.asarray(l).shape[1]
    on = counts(tokens, V, weights)
    lp, ent = token_logprobs(l, tokens, T)
    loss, kl, d_lp, d_ent = policy_rows(lp, ent, tokens, V, old, adv, weights, ref, **coef)
    grad = token_logprobs_grad(l, tokens, d_lp, d_ent, T, on)
    return dict(loss=loss, logprob=np.where(on, lp, 0.0), kl=kl, entropy=np.where(on, ent, 0.0), grad=grad, d_lp=d_lp,
                d_ent=d_ent)


def _log_sigmoid(h):
    return -np.logaddexp(0.0, -h)


def preference_loss(logprob, ref, offsets, beta, smoothing=0.0, weights=None):
    """(loss [pairs], rewards [pairs, 2], d_logprob [R])."""
    lp = np.asarray(logprob, np.float64)
    ref = np.zeros_like(lp) if ref is None else np.asarray(ref, np.float64)
    at = np.clip(np.asarray(offsets, np.int64), 0, len(lp))
    pairs = (len(at) - 1) // 2
    loss, rewards, d = np.zeros(pairs), np.zeros((pairs, 2)), np.zeros(len(lp))
    for q in range(pairs):
        w = 1.0 if weights is None else float(weights[q])
        if w == 0.0:
            continue
        rows = [slice(at[2 * q + i], at[2 * q + i + 1]) for i in range(2)]
        rewards[q] = [beta * (lp[r] - ref[r]).sum() for r in rows]
        h = rewards[q, 0] - rewards[q, 1]
        loss[q] = w * (-(1 - smoothing) * _log_sigmoid(h) - smoothing * _log_sigmoid(-h))
        dh = w * (smoothing * np.exp(_log_sigmoid(h)) - (1 - smoothing) * np.exp(_log_sigmoid(-h)))
        d[rows[0]], d[rows[1]] = beta * dh, -beta * dh
    return loss, rewards, d
