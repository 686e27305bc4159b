"""How far a float32 softmax pass may be off the float64 oracle, by arithmetic.

z = sum exp((l - m) / T) over V terms, at least 128 partial sums: a float32 sum of n terms is off by at most n
half-steps (2^-24) of its value, so V / 128 additions and up to 64 merges; a term's exponential by 2^-22 (ex2.approx)
plus the roundings of l - m and of the exponent, 2 x 2^-24 |l - m| / T, whose mean over p is at most ln V; and each of
up to V / 2048 rescalings (a new maximum at every 16 logits of a partial sum) and 32 merges by one more exponential.
"""
import numpy as np

HALF = {"fp32": 2.0 ** -24, "bf16": 2.0 ** -8}   # half a step, relative


def eps_z(V):
    return (V / 128 + 64) * 2.0 ** -24 + (V / 2048 + 32) * 2.0 ** -22 + np.log(max(V, 2)) * 2.0 ** -23


def mean_shift(logp):
    """E_p[(m - l) / T] of each row."""
    with np.errstate(all="ignore"):
        top = logp.max(1, keepdims=True)
        p = np.exp(logp)
        return np.where(p > 0, p * (top - logp), 0.0).sum(1)


def logprob_bound(logp, lp):
    return eps_z(logp.shape[1]) + HALF["fp32"] * np.abs(lp) + 1e-12


def entropy_bound(logp, ent):
    e = eps_z(logp.shape[1])
    return e * (1 + 2 * mean_shift(logp)) + HALF["fp32"] * np.abs(ent) + 1e-12


def grad_bound(logp, tokens, T, d_lp, d_ent, err_lp, err_ent, grad, kind):
    """Elementwise bound of G = (g 1[t] - p (g + h (log p + H))) / T.  err_lp / err_ent: how far the derivatives
    g and h may themselves be off."""
    V = logp.shape[1]
    g, h = np.abs(d_lp)[:, None], np.abs(d_ent)[:, None]
    with np.errstate(all="ignore"):
        p = np.exp(logp)
        log_z = -logp.max(1, keepdims=True)
        far = np.where(p > 0, logp.max(1, keepdims=True) - logp, 0.0)     # |l - m| / T
        ent = -np.where(p > 0, p * logp, 0.0).sum(1)[:, None]
        size = p * (g + h * (far + log_z + ent))                          # alpha's and gamma's parts, no cancellation
        # a term's exponential, z (twice: in p and in H), alpha, gamma and their sum
        rel = 2.0 ** -22 + far * 2.0 ** -23 + 2 * eps_z(V) + 6 * 2.0 ** -24
        err = size * rel + p * (err_lp[:, None] + err_ent[:, None] * (far + log_z + ent))
        err = err + p * h * entropy_bound(logp, ent[:, 0])[:, None]
    at = np.where((tokens >= 0) & (tokens < V), tokens, 0)
    err[np.arange(len(at)), at] += np.abs(d_lp) * 2.0 ** -23 + err_lp
    return err / T + np.abs(grad) * HALF[kind] + np.where(kind == "bf16", 2.0 ** -133, 2.0 ** -126) * (1 + size / T)
