"""Parity of the token logprobs, their gradient, the policy loss and the preference loss with the float64 oracle (GPU).
Tolerances: ``score_bounds``, derived from the arithmetic."""
import numpy as np
import pytest
import torch

import vocab_sharded_logits_b200 as vsl
from oracle import scores as O
import score_bounds as B

pytestmark = pytest.mark.gpu
FMIN = float(np.finfo(np.float32).min)

# rows, slices, ids per slice: one id group to several slices, odd sizes, more rows than CTAs, a long row
SHAPES = [(1, 1, 4), (3, 1, 8), (5, 3, 20), (4, 2, 512), (7, 16, 4), (33, 5, 1004), (300, 1, 260), (2, 4, 37984),
          (3, 1, 151936), (1, 8, 32768),
          (1500, 3, 100), (500, 2, 6000), (160, 1, 12000), (40, 4, 20000)]   # one to eight CTAs per row, several rows each


def _rng(*k):
    return np.random.default_rng(list(k))


def _logits(R, V, rng, masked=True):
    l = (rng.normal(size=(R, V)) * 2).astype(np.float32)
    if masked and V >= 8:
        l[rng.random((R, V)) < 0.1] = -np.inf
        l[:, 0] = 1.0                                   # no row is empty
        if R > 2:
            l[1] += 300.0                               # far from 0
            l[2, 1:] = np.where(rng.random(V - 1) < 0.5, FMIN, l[2, 1:])
    return l


def _slices(l, S, dev):
    return [torch.from_numpy(np.ascontiguousarray(x)).to(dev) for x in np.split(l, S, axis=1)]


def _tokens(l, rng):
    """A token of each row with a finite logit; every 5th row's lies outside the vocabulary."""
    R, V = l.shape
    t = np.array([rng.choice(np.flatnonzero(np.isfinite(l[r]) & (l[r] > FMIN))) for r in range(R)], np.int32)
    t[4::5] = np.where(np.arange(len(t[4::5])) % 2, V, -1)
    return t


def _dev(x, dev, dtype=torch.float32):
    return None if x is None else torch.from_numpy(np.array(x)).to(dev, dtype)


def _cat(slices):
    return torch.cat([x.float() for x in slices], 1).cpu().numpy().astype(np.float64)


def _close(got, want, bound, what):
    got = got.cpu().numpy().astype(np.float64) if isinstance(got, torch.Tensor) else got
    bad = ~(np.abs(got - want) <= bound) & ~(np.isnan(got) & np.isnan(want)) & ~(got == want)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, first at {np.argwhere(bad)[0]}: " \
        f"{got[bad][0]} against {want[bad][0]} (bound {np.broadcast_to(bound, got.shape)[bad][0]})"


def _check_logprobs(l, tokens, S, T, rng, dev):
    R, V = l.shape
    V_s, T64 = V // S, np.float64(np.float32(T))
    slices = _slices(l, S, dev)
    tok = _dev(tokens, dev, torch.int32)
    fwd = vsl.token_logprobs(slices, tok, temperature=T, entropy=True)
    logp = O.log_softmax(l, T64)
    lp, ent = O.token_logprobs(l, tokens, T64)
    _close(fwd.logprob, lp, B.logprob_bound(logp, lp), "logprob")
    _close(fwd.entropy, ent, B.entropy_bound(logp, ent), "entropy")
    alone = vsl.token_logprobs(slices, tok, temperature=T)
    assert alone.entropy is None and torch.equal(alone.row_stats, fwd.row_stats)
    assert torch.equal(alone.logprob, fwd.logprob)
    dl, de = rng.normal(size=R).astype(np.float32), rng.normal(size=R).astype(np.float32)
    dl[R // 2] = 0.0
    on = O.counts(tokens, V)
    for d_ent in (None, de):
        want = O.token_logprobs_grad(l, tokens, dl, d_ent, T64)
        h = np.where(on, 0.0 if d_ent is None else d_ent, 0.0)
        for kind, dtype in (("fp32", torch.float32), ("bf16", torch.bfloat16)):
            got = vsl.token_logprobs_grad(slices, tok, fwd, _dev(dl, dev), _dev(d_ent, dev), grad_dtype=dtype)
            assert all(x.dtype == dtype and x.shape == (R, V_s) for x in got)
            zero = np.zeros(R)
            bound = B.grad_bound(logp, tokens, T, np.where(on, dl, 0.0), h, zero, zero, want, kind)
            _close(_cat(got), want, bound, f"gradient {kind}")
    in_place = [x.clone() for x in slices]
    first = vsl.token_logprobs_grad(slices, tok, fwd, _dev(dl, dev), _dev(de, dev))
    vsl.token_logprobs_grad(in_place, tok, fwd, _dev(dl, dev), _dev(de, dev), grad=in_place)
    assert all(torch.equal(x, y) for x, y in zip(first, in_place))


@pytest.mark.parametrize("T", [1.0, 0.37])
@pytest.mark.parametrize("R,S,V_s", SHAPES)
def test_logprobs_and_gradient(cuda_device, R, S, V_s, T):
    rng = _rng(R, S, V_s)
    l = _logits(R, S * V_s, rng)
    _check_logprobs(l, _tokens(l, rng), S, T, rng, cuda_device)


def _extreme_rows(V, rng):
    """Rows whose logits are far from what a row begins with, from 0 or from one another."""
    l = rng.normal(size=(12, V)).astype(np.float32)
    l[1] += 5e6
    l[2, : V // 2] = -1e4                            # a mask of a large finite value, first
    l[3, -1] = 200.0                                 # far above all that came before
    l[4] = FMIN                                      # nothing but the lowest value
    l[5, : V // 3] = FMIN
    l[6] *= np.float32(1e30)
    l[7] -= 300.0
    l[8] = -1e9
    l[8, [5, V // 2, V - 1]] = [1.0, 2.0, 3.0]
    l[9] = -np.inf
    l[9, V - 2] = -70.0                              # one finite logit
    l[10, : V - 4] = -np.inf
    l[11] = 3e38
    l[11, 7] = -3e38
    return l


def _extreme_tokens(l):
    return np.array([int(np.argmax(x)) if i % 2 else int(np.flatnonzero(np.isfinite(x))[0]) for i, x in enumerate(l)], np.int32)


@pytest.mark.parametrize("V,S,T", [(8, 1, 1.0), (2000, 2, 1.0), (20000, 2, 1.0), (20000, 1, 0.5), (151936, 4, 1.0),
                                   (2000, 2, 1e-6), (2000, 2, 1e6)])
def test_extreme_rows(cuda_device, V, S, T):
    rng = _rng(V, S, 3)
    l = _extreme_rows(V, rng)
    tokens = _extreme_tokens(l)
    T64 = np.float64(np.float32(T))
    lp, _ = O.token_logprobs(l, tokens, T64)
    keep = np.abs(lp) < 1e30                         # a token at -1e35 of the rest has no ratio to speak of
    tokens[~keep] = -1
    _check_logprobs(l, tokens, S, T, rng, cuda_device)
    lp, _ = O.token_logprobs(l, tokens, T64)
    old = np.asarray(lp - 0.05, np.float32)
    far = np.abs(lp) > 1e3                           # float32 old logprobs cannot name a ratio near 1 there
    tokens[far] = -1
    adv, w = rng.normal(size=12).astype(np.float32), np.ones(12, np.float32)
    _check_policy(l, tokens, S, T, old, old.copy(), adv, w, 0.0, 0.0, cuda_device)
    _check_policy(l, tokens, S, T, old, old.copy(), adv, w, 0.1, 0.03, cuda_device)


def _policy_case(R, V, rng, l, tokens, T):
    lp, _ = O.token_logprobs(l, tokens, T)
    delta = rng.normal(size=R) * 0.3
    for border in (np.log(0.8), np.log(1.28)):
        delta = np.where(np.abs(delta - border) < 1e-2, delta + 3e-2, delta)
    f = lambda x: np.asarray(x, np.float32)  # noqa: E731
    w = f(rng.uniform(0.1, 1, R))
    w[3::7] = 0.0
    old, ref, adv = f(lp - delta), f(lp + rng.normal(size=R) * 0.3), f(rng.normal(size=R))
    old[3::7] = np.nan                                   # a row that does not count is not looked at
    return old, ref, adv, w


def _check_policy(l, tokens, S, T, old, ref, adv, w, kl_coef, ent_coef, dev):
    R, V = l.shape
    T64 = np.float64(np.float32(T))
    f64 = lambda x: np.float64(np.float32(x))  # noqa: E731
    want = O.policy_loss(l, tokens, old, adv, T=T64, weights=w, ref=ref, lo=f64(0.2), hi=f64(0.28), kl_coef=f64(kl_coef),
                         ent_coef=f64(ent_coef))
    slices, tok = _slices(l, S, dev), _dev(tokens, dev, torch.int32)
    rows = [_dev(x, dev) for x in (old, adv, w, ref)]
    kw = dict(weights=rows[2], ref_logprob=rows[3], clip_low=0.2, clip_high=0.28, kl_coef=kl_coef,
              entropy_coef=ent_coef, temperature=T)
    logp = O.log_softmax(l, T64)
    on = O.counts(tokens, V, w)
    err = np.where(on, B.logprob_bound(logp, want["logprob"]), 0.0)   # of the logprob inside the kernel
    err_h = np.where(on, B.entropy_bound(logp, 0 * adv), 0.0)
    ratio = np.where(on, np.exp(want["logprob"] - np.where(on, old, 0)), 0.0)
    d = np.where(on, ref - want["logprob"], 0.0)
    err_g = np.where(on, np.abs(w) * (np.abs(adv) * ratio + kl_coef * np.exp(d)) * err * 1.01, 0.0)
    err_loss = np.abs(w) * ((np.abs(adv) * ratio + kl_coef * np.abs(np.expm1(d))) * err * 1.01 + ent_coef * err_h)
    for kind, dtype in (("fp32", torch.float32), ("bf16", torch.bfloat16)):
        got = vsl.policy_loss(slices, tok, rows[0], rows[1], grad_dtype=dtype, **kw)
        _close(got.loss, want["loss"], err_loss + 2.0 ** -24 * np.abs(want["loss"]), "loss")
        _close(got.logprob, want["logprob"], err + 2.0 ** -24 * np.abs(want["logprob"]), "logprob")
        _close(got.entropy, want["entropy"], err_h + 2.0 ** -24 * want["entropy"], "entropy")
        _close(got.kl, want["kl"], np.abs(np.expm1(d)) * err * 1.01 + err ** 2 + 2.0 ** -24 * want["kl"], "kl")
        bound = B.grad_bound(logp, tokens, T, want["d_lp"], want["d_ent"], err_g, np.zeros(R), want["grad"], kind)
        _close(_cat(got.grad), want["grad"], bound, f"gradient {kind}")
    # in place, and without a gradient: the same numbers
    over = [x.clone() for x in slices]
    same = vsl.policy_loss(over, tok, rows[0], rows[1], grad=over, **kw)
    plain = vsl.policy_loss(slices, tok, rows[0], rows[1], **kw)
    none = vsl.policy_loss(slices, tok, rows[0], rows[1], grad=False, **kw)
    assert none.grad is None and torch.equal(none.loss, plain.loss) and torch.equal(same.loss, plain.loss)
    assert all(torch.equal(x, y) for x, y in zip(plain.grad, over))


@pytest.mark.parametrize("kl_coef,ent_coef,T", [(0.0, 0.0, 1.0), (0.05, 0.0, 0.8), (0.1, 0.03, 1.3)])
@pytest.mark.parametrize("R,S,V_s", SHAPES)
def test_policy_loss(cuda_device, R, S, V_s, kl_coef, ent_coef, T):
    rng = _rng(R, S, V_s, 1)
    l = _logits(R, S * V_s, rng)
    tokens = _tokens(l, rng)
    old, ref, adv, w = _policy_case(R, S * V_s, rng, l, tokens, np.float64(np.float32(T)))
    _check_policy(l, tokens, S, T, old, ref, adv, w, kl_coef, ent_coef, cuda_device)


def test_policy_gradient_against_differences(cuda_device):
    """The loss's change along a direction u: (f(l + s u) - f(l - s u)) / 2s.  The difference's own error: the third
    derivative, at most a few times the terms' size here (s^2), and the losses' float32 roundings over 2s."""
    rng = _rng(11)
    R, V, s = 6, 24, 2.0 ** -7
    l = rng.normal(size=(R, V)).astype(np.float32)
    tokens = rng.integers(0, V, R).astype(np.int32)
    lp, _ = O.token_logprobs(l, tokens)
    f = lambda x: _dev(np.asarray(x, np.float32), cuda_device)  # noqa: E731
    old, adv, ref = f(lp + 0.05), f(rng.normal(size=R)), f(lp + 0.2)
    u = np.round(rng.normal(size=(R, V)) * 16) / 16
    run = lambda x: vsl.policy_loss(_slices(x.astype(np.float32), 2, cuda_device),  # noqa: E731
                                    _dev(tokens, cuda_device, torch.int32), old, adv, ref_logprob=ref, kl_coef=0.1,
                                    entropy_coef=0.05)
    up, down, at = run(l + s * u), run(l - s * u), run(l)
    for r in range(R):
        slope = (float(up.loss[r]) - float(down.loss[r])) / (2 * s)
        want = float((_cat(at.grad)[r] * u[r]).sum())
        size = float(np.abs(u[r]).max()) ** 3 * (1 + abs(float(adv[r])))
        # l +- s u is rounded to float32: 2^-24 |l| |u'| in the argument; the losses to 2^-24 and z by eps_z
        assert abs(slope - want) <= 4 * size * s * s + (2 * B.eps_z(V) + 2.0 ** -22) * (1 + abs(float(adv[r])) + abs(slope)) / s


def test_rows_that_are_invalid_leave_the_others_alone(cuda_device):
    rng = _rng(5)
    R, V = 6, 1200
    l = _logits(R, V, rng, masked=False)
    tokens = np.full(R, 7, np.int32)
    l[1, 900], l[2, 3], l[3], l[4, 7] = np.nan, np.inf, -np.inf, -np.inf
    slices, tok = _slices(l, 3, cuda_device), _dev(tokens, cuda_device, torch.int32)
    one = torch.ones(R, device=cuda_device)
    fwd = vsl.token_logprobs(slices, tok, entropy=True)
    pol = vsl.policy_loss(slices, tok, -one, one)
    grad = _cat(vsl.token_logprobs_grad(slices, tok, fwd, one, one))
    bad = np.array([False, True, True, True, False, False])
    assert np.array_equal(np.isnan(fwd.logprob.cpu().numpy()), bad)
    assert np.array_equal(np.isnan(fwd.entropy.cpu().numpy()), bad)
    assert np.array_equal(np.isnan(pol.loss.cpu().numpy()), bad)
    assert float(fwd.logprob[4]) == -np.inf                      # the token has probability 0
    assert float(pol.loss[4]) == 0.0                             # ratio 0
    assert np.isnan(grad[bad]).all() and np.isfinite(grad[~bad]).all()
    pg = _cat(pol.grad)
    assert np.isnan(pg[bad]).all() and np.isfinite(pg[~bad]).all()
    # the same rows, weighted 0 or without a token: zeros
    w = torch.from_numpy((~bad).astype(np.float32)).to(cuda_device)
    pol = vsl.policy_loss(slices, tok, -one, one, weights=w)
    assert np.isfinite(_cat(pol.grad)).all() and (_cat(pol.grad)[bad] == 0).all() and bool((pol.loss[1:4] == 0).all())
    tok2 = torch.where(w > 0, tok, -1)
    fwd = vsl.token_logprobs(slices, tok2, entropy=True)
    assert bool((fwd.logprob[1:4] == 0).all()) and bool((fwd.entropy[1:4] == 0).all())
    assert (_cat(vsl.token_logprobs_grad(slices, tok2, fwd, one, one))[bad] == 0).all()


def test_infinite_kl_matters_only_with_a_coefficient(cuda_device):
    l = np.zeros((2, 8), np.float32)
    l[:, 3] = -np.inf
    tok = torch.full((2,), 3, dtype=torch.int32, device=cuda_device)
    one = torch.ones(2, device=cuda_device)
    s = _slices(l, 1, cuda_device)
    free = vsl.policy_loss(s, tok, -one, one, ref_logprob=-one)
    assert bool(torch.isinf(free.kl).all()) and bool((free.loss == 0).all()) and np.isfinite(_cat(free.grad)).all()
    held = vsl.policy_loss(s, tok, -one, one, ref_logprob=-one, kl_coef=0.1)
    assert bool((held.loss == np.inf).all())


@pytest.mark.parametrize("lens", [[1, 1], [5, 0, 3, 4], [0, 0], [200, 1000, 1, 129, 64, 63]])
@pytest.mark.parametrize("smoothing", [0.0, 0.1])
def test_preference_loss(cuda_device, lens, smoothing):
    rng = _rng(len(lens), sum(lens))
    at = np.concatenate([[2], 2 + np.cumsum(lens)]).astype(np.int32)
    R, pairs = int(at[-1]) + 3, len(lens) // 2
    lp, ref = rng.normal(size=R).astype(np.float32) - 3, rng.normal(size=R).astype(np.float32) - 3
    w = rng.uniform(0.5, 2, pairs).astype(np.float32)
    if pairs > 1:
        w[1] = 0.0
        lp[at[2]:at[4]] = np.nan                          # a pair of weight 0 is not read
    beta, e = np.float64(np.float32(0.3)), np.float64(np.float32(smoothing))
    dev = lambda x: torch.from_numpy(x).to(cuda_device)  # noqa: E731
    for r, weights in ((ref, w), (None, w), (ref, None)):
        if weights is None:
            lp = np.nan_to_num(lp)
        loss, rewards, d = O.preference_loss(lp, r, at, beta, e, weights)
        got = vsl.preference_loss(dev(lp), None if r is None else dev(r), dev(at), 0.3, smoothing,
                                  None if weights is None else dev(weights))
        # 64-bit sums of up to 1000 terms of size < 10 (2^-53 each), an output rounding to 32 bits
        _close(got.loss, loss, 2.0 ** -24 * np.abs(loss) + 1e-9, "loss")
        _close(got.rewards, rewards, 2.0 ** -24 * np.abs(rewards) + 1e-9, "rewards")
        _close(got.d_logprob, d, 2.0 ** -24 * np.abs(d) + 1e-9, "d_logprob")


def test_preference_offsets_outside_the_rows_stay_inside(cuda_device):
    lp = torch.randn(8, device=cuda_device)
    at = torch.tensor([-5, 4, 1 << 20], dtype=torch.int32, device=cuda_device)
    got = vsl.preference_loss(lp, None, at, 0.5)
    want = vsl.preference_loss(lp, None, torch.tensor([0, 4, 8], dtype=torch.int32, device=cuda_device), 0.5)
    assert torch.equal(got.loss, want.loss) and torch.equal(got.d_logprob, want.d_logprob)


def test_extreme_preference_margins(cuda_device):
    at = torch.tensor([0, 1, 2], dtype=torch.int32, device=cuda_device)
    for m in (-2000.0, -30.0, 30.0, 2000.0):
        lp = torch.tensor([m, 0.0], device=cuda_device)
        got = vsl.preference_loss(lp, None, at, 1.0)
        loss, _, d = O.preference_loss(lp.cpu().numpy(), None, [0, 1, 2], 1.0)
        _close(got.loss, loss, 2.0 ** -23 * loss, "loss")
        _close(got.d_logprob, d, 2.0 ** -23 * np.abs(d) + 1e-37, "d_logprob")


def test_bitwise_repeatable_and_poison_overwritten(cuda_device):
    rng = _rng(9)
    R, S, V_s = 37, 3, 5004
    l = _logits(R, S * V_s, rng)
    slices = _slices(l, S, cuda_device)
    tok = _dev(_tokens(l, rng), cuda_device, torch.int32)
    one = torch.ones(R, device=cuda_device)
    res = []
    for fill in (float("nan"), 3.0):
        grad = [torch.full((R, V_s), fill, device=cuda_device) for _ in range(S)]
        out = vsl.policy_loss(slices, tok, -9 * one, one, entropy_coef=0.01, grad=grad)
        fwd = vsl.token_logprobs(slices, tok, entropy=True)
        g2 = vsl.token_logprobs_grad(slices, tok, fwd, one, one, grad=[torch.full_like(x, fill) for x in grad])
        res.append([out.loss, out.entropy, fwd.logprob, fwd.entropy, *grad, *g2])
    for x, y in zip(*res):
        assert bool(torch.isfinite(x).all()) and torch.equal(x, y)


def test_graph_capture_and_another_stream(cuda_device):
    """Captured on a side stream and replayed on new values; then run on a stream that is not the current one."""
    rng = _rng(12)
    R, S, V_s = 9, 2, 2000
    slices = _slices(_logits(R, S * V_s, rng), S, cuda_device)
    tok = _dev(_tokens(_logits(R, S * V_s, rng, masked=False), rng), cuda_device, torch.int32)
    one = torch.ones(R, device=cuda_device)
    at = torch.tensor([0, 4, R], dtype=torch.int32, device=cuda_device)

    def step(stream=None):
        p = vsl.policy_loss(slices, tok, -9 * one, one, entropy_coef=0.01, stream=stream)
        f = vsl.token_logprobs(slices, tok, stream=stream)
        d = vsl.preference_loss(f.logprob, None, at, 0.1, stream=stream)
        g = vsl.token_logprobs_grad(slices, tok, f, d.d_logprob, stream=stream)
        return [p.loss, *p.grad, f.logprob, d.loss, *g]
    step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        captured = step()
    new = _slices(_logits(R, S * V_s, _rng(13)), S, cuda_device)
    for x, y in zip(slices, new):
        x.copy_(y)
    graph.replay()
    torch.cuda.synchronize()
    for x, y in zip(captured, step()):
        assert torch.equal(x, y)
    want = step()
    side.wait_stream(torch.cuda.current_stream())
    got = step(stream=side)
    torch.cuda.synchronize()
    for x, y in zip(got, want):
        assert torch.equal(x, y)


@pytest.mark.parametrize("smoothing", [0.0, 1.0])
def test_a_term_without_weight_may_be_infinite(cuda_device, smoothing):
    """A token of probability 0 makes one of the two terms infinite; left out, it does not matter."""
    at = torch.tensor([0, 1, 2], dtype=torch.int32, device=cuda_device)
    lp = torch.tensor([-np.inf, -1.0] if smoothing else [-1.0, -np.inf], device=cuda_device)
    got = vsl.preference_loss(lp, None, at, 0.5, smoothing)
    assert got.loss.item() == 0.0 and bool((got.d_logprob == 0).all())


def test_an_output_filled_again_holds_no_older_entropy(cuda_device):
    rng = _rng(21)
    old, new = (_slices(_logits(5, 2000, rng), 2, cuda_device) for _ in range(2))
    tok = _dev(_tokens(_logits(5, 2000, rng, masked=False), rng), cuda_device, torch.int32)
    out = vsl.token_logprobs(old, tok, entropy=True)
    before = out.entropy.clone()
    assert vsl.token_logprobs(new, tok, out=out) is out and not torch.equal(out.entropy, before)
    assert torch.equal(out.entropy, vsl.token_logprobs(new, tok, entropy=True).entropy)


def test_two_streams_at_once(cuda_device):
    """Losses of different batches overlapping on two streams, again and again: each as when run alone."""
    rng = _rng(22)
    sizes = [(150, 2, 20000), (40, 4, 37984)]
    batches = []
    for R, S, V_s in sizes:
        l = _logits(R, S * V_s, rng)
        batches.append((_slices(l, S, cuda_device), _dev(_tokens(l, rng), cuda_device, torch.int32),
                        torch.ones(R, device=cuda_device)))

    def step(batch, stream=None):
        s, tok, one = batch
        p = vsl.policy_loss(s, tok, -9 * one, one, entropy_coef=0.01, stream=stream)
        f = vsl.token_logprobs(s, tok, entropy=True, stream=stream)
        g = vsl.token_logprobs_grad(s, tok, f, one, one, stream=stream)
        return [p.loss, *p.grad, f.logprob, f.entropy, *g]
    want = [step(b) for b in batches]
    streams = [torch.cuda.Stream() for _ in batches]
    torch.cuda.synchronize()
    for _ in range(4):
        got = []
        for b, stream in zip(batches, streams):
            with torch.cuda.stream(stream):
                got.append(step(b))
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for w, g in zip(want, got) for x, y in zip(w, g))
