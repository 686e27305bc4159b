"""Corners of the scoring calls: outputs that are partly there, the C call with outputs left out, what a row's parts
share, and sharper bounds than the general ones (GPU)."""
import ctypes

import numpy as np
import pytest
import torch

import vocab_sharded_logits_b200 as vsl
from oracle import scores as O

pytestmark = pytest.mark.gpu


def _slices(l, S, dev):
    return [torch.from_numpy(np.ascontiguousarray(x)).to(dev) for x in np.split(l, S, axis=1)]


def _np(x):
    return x.float().cpu().numpy().astype(np.float64)


def test_an_output_to_fill_gets_what_it_lacks(cuda_device):
    g = torch.Generator(device=cuda_device)
    g.manual_seed(3)
    slices = [torch.randn(5, 400, generator=g, device=cuda_device) for _ in range(2)]
    tok = torch.arange(5, dtype=torch.int32, device=cuda_device)
    want = vsl.token_logprobs(slices, tok)
    mine = torch.empty(5, device=cuda_device)
    for logprob in (mine, None):
        out = vsl.TokenLogprobs(logprob, None, None, 1.0)
        assert vsl.token_logprobs(slices, tok, out=out) is out and (logprob is None or out.logprob is mine)
        assert torch.equal(out.logprob, want.logprob) and torch.equal(out.row_stats, want.row_stats)
        assert out.entropy is None


# ------------------------------------------------------------------ what the parts of a row share

CUTS = [(1, 1, 8), (3, 2, 1004), (60, 5, 2000), (60, 3, 17004), (60, 4, 37984), (160, 1, 12000), (400, 3, 17004),
        (700, 2, 600), (60, 1, 262144), (200, 8, 18992)]


@pytest.mark.parametrize("R,S,V_s", CUTS)
def test_every_logit_counts_once(cuda_device, R, S, V_s):
    """Equal logits of 0: every exponential is 1 but for its own error (2^-22, and the mean error taken out of it), whole
    numbers add up exactly, and a unit of four left out or read twice moves the logprob by 4 / V."""
    V = S * V_s
    slices = [torch.zeros(R, V_s, device=cuda_device) for _ in range(S)]
    tok = torch.arange(R, dtype=torch.int32, device=cuda_device) * 7 % V
    one = torch.ones(R, device=cuda_device)
    bound = (2.0 ** -22 + 2.0 ** -24) + 2.0 ** -24 * np.log(V)
    assert 4 / V > 4 * bound
    for lp in (vsl.token_logprobs(slices, tok, entropy=True).logprob, vsl.token_logprobs(slices, tok).logprob,
               vsl.policy_loss(slices, tok, -one, one, entropy_coef=0.1).logprob):
        assert (np.abs(_np(lp) + np.log(V)) <= bound).all()


@pytest.mark.parametrize("R,S,V_s", [(1, 2, 1004), (60, 3, 17004), (60, 4, 37984), (160, 1, 12000), (400, 3, 17004),
                                     (30, 1, 262144), (200, 8, 18992)])
def test_mass_at_the_edges_of_parts_and_slices(cuda_device, R, S, V_s):
    """Rows whose mass is one unit of four at either side of where a row could be cut: between slices, between the parts
    of 1 to 8 CTAs, between the batches of 128 to 512 threads.  Left out or read twice the unit moves the logprob by
    log 2 or more; the bound is of four exponentials and of V at 2^-43."""
    V, units, per_slice = S * V_s, S * V_s // 4, V_s // 4
    edges = {per_slice * s for s in range(1, S)}
    for c in (1, 2, 4, 8):
        part = -(-units // c)
        edges |= {part * k for k in range(1, c)}
        for threads in (128, 256, 512):
            edges |= {part * (c - 1) + threads * k for k in (1, 3, 4, 5)} | {threads * 4}
    at = sorted({u + d for u in edges for d in (-1, 0) if 0 <= u + d < units} | {0, units - 1})
    at = np.resize(np.array(at), R) if R < len(at) else np.array(at)[np.arange(R) % len(at)]
    l = np.full((R, V), -30.0, np.float32)
    for r in range(R):
        l[r, 4 * at[r]:4 * at[r] + 4] = [0.0, 1.0, 0.5, -1.0]
    tok = ((4 * at + V // 2) % V).astype(np.int32)                 # elsewhere
    lp, ent = O.token_logprobs(l, tok)
    slices, t = _slices(l, S, cuda_device), torch.from_numpy(tok).to(cuda_device)
    one = torch.ones(R, device=cuda_device)
    # 2^-22 of an exponential, its exponent below 2 (2^-24), 8 additions, c over a distance of 32
    bound = 2.0 ** -22 + 2.0 ** -24 * (2 + 8 + 32) + 2.0 ** -24 * np.abs(lp)
    for got in (vsl.token_logprobs(slices, t), vsl.policy_loss(slices, t, -30 * one, one)):
        assert (np.abs(_np(got.logprob) - lp) <= bound).all()
    grad = vsl.policy_loss(slices, t, torch.from_numpy(lp.astype(np.float32)).to(cuda_device), one).grad
    want = O.policy_loss(l, tok, lp.astype(np.float32), np.ones(R))["grad"]
    # ratio 1 (the logprob's error and old's rounding in it); p: the same errors again, and z's and the coefficient's
    off = np.abs(np.concatenate([_np(x) for x in grad], 1) - want)
    assert (off <= 3 * bound.max() * np.abs(want) + 2.0 ** -23).all()


# ------------------------------------------------------------------ sharper bounds

def _chain(V, R):
    """Additions one after another in a thread at the fewest threads a row can have (one CTA of 128, or of 256 above 2,048
    units), then of the batch, the warp and the CTAs."""
    return V / 16 / (128 if V <= 8192 else 256) + 16


@pytest.mark.parametrize("R,S,V_s", [(64, 2, 512), (64, 5, 2000), (600, 3, 4000), (64, 4, 37984), (160, 4, 37984),
                                     (64, 1, 262144)])
@pytest.mark.parametrize("T", [1.0, 0.7])
def test_logprobs_within_the_fast_forms_own_roundings(cuda_device, R, S, V_s, T):
    """z: an exponential within 2^-22 and its mean error; its exponent's half step, 2^-24 |y| for |y| the distance from
    the first logits' largest, at most the row's spread, over p; the additions; c over the distance from the mean."""
    V = S * V_s
    rng = np.random.default_rng([R, V])
    l = (rng.normal(size=(R, V)) * 2).astype(np.float32)
    l[rng.random((R, V)) < 0.1] = -np.inf
    l[:, 0] = 0.0
    tok = np.argsort(l, 1)[np.arange(R), -1 - rng.integers(0, V // 2, R)].astype(np.int32)
    T64 = np.float64(np.float32(T))
    logp = O.log_softmax(l, T64)
    lp, ent = O.token_logprobs(l, tok, T64)
    p, far = np.exp(logp), np.where(np.isfinite(logp), logp.max(1, keepdims=True) - logp, 0.0)
    spread = (p * far).sum(1)
    mean = lp + ent                                                # distance of x_t from the mean of x
    eps = 2.0 ** -22 + 2.0 ** -24 + 2.0 ** -24 * (spread + 2) + _chain(V, R) * 2.0 ** -24
    bound = eps + 2.0 ** -24 * np.abs(mean) + 2.0 ** -24 * np.abs(lp)
    slices, t = _slices(l, S, cuda_device), torch.from_numpy(tok).to(cuda_device)
    fwd = vsl.token_logprobs(slices, t, temperature=T, entropy=True)
    one = torch.ones(R, device=cuda_device)
    pol = vsl.policy_loss(slices, t, -9 * one, one, temperature=T, entropy_coef=0.01)
    for got in (fwd, pol):
        off = np.abs(_np(got.logprob) - lp)
        assert (off <= bound).all(), (off / bound).max()
        # entropy: log z as above, and the mean of x: each e y by the same, sizes spread + 2
        off = np.abs(_np(got.entropy) - ent)
        assert (off <= eps * (2 * spread + 5) + 2.0 ** -24 * ent).all(), (off / eps).max()


def test_logprobs_have_no_error_in_the_mean(cuda_device):
    """ex2.approx is off by -5.2e-8 in the mean, which z, a sum of many, would keep: over 8,192 rows the logprobs' error
    has the mean that c's rounding gives it and no other.  c = fl(log2 e) = (1 + d) log2 e is the temperature 1 / (1 + d):
    log p_t moves by d (x_t - sum p x) = d (log p_t + H), 3e-8 here.  A row's error beside it: the output's rounding,
    uniform in +-half a step of a number between 8 and 16 (2^-21 / sqrt 3 = 2.8e-7), and z's, of which 2^-22 is the most;
    over sqrt 8,192 five standard deviations of the two together are 2.1e-8."""
    R, V = 8192, 4096
    g = torch.Generator(device=cuda_device)
    g.manual_seed(17)
    x = torch.randn(R, V, generator=g, device=cuda_device) * 1.5
    tok = x.topk(V // 2).indices[:, -1].int()                       # near the median: logprobs of -9.4 or so
    logp = torch.log_softmax(x.double(), 1)
    want = logp.gather(1, tok.long()[:, None])[:, 0]
    d = float(np.float32(np.log2(np.e))) / np.log2(np.e) - 1
    shift = d * float((want - (logp.exp() * logp).sum(1)).mean())
    assert bool((want < -8).all()) and bool((want > -16).all())
    one = torch.ones(R, device=cuda_device)
    for lp in (vsl.token_logprobs([x], tok).logprob, vsl.policy_loss([x], tok, -9 * one, one, grad=False).logprob):
        assert abs(float((lp.double() - want).mean()) - shift) <= 2.1e-8


# ------------------------------------------------------------------ the C call with outputs left out

def _policy_c(slices, tok, old, adv, ref, kl_coef, kind, grad, with_kl, with_lp):
    R, V_s = slices[0].shape
    vp = ctypes.c_void_p
    at = (vp * len(slices))(*[x.data_ptr() for x in slices])
    loss = torch.full((R,), float("nan"), device=slices[0].device)
    lp, kl = torch.full_like(loss, float("nan")), torch.full_like(loss, float("nan"))
    i = vsl._PolicyInputs(tok.data_ptr(), old.data_ptr(), adv.data_ptr(), ref.data_ptr(), None, 0.2, 0.28, kl_coef, 0.0, 1.0)
    o = vsl._PolicyOutputs()
    o.loss, o.logprob, o.kl, o.entropy = loss.data_ptr(), lp.data_ptr() if with_lp else None, kl.data_ptr() if with_kl else None, None
    o.grad_type = kind
    if grad is not None:
        o.grad_slices = (vp * len(grad))(*[x.data_ptr() for x in grad])
    stream = vp(torch.cuda.current_stream().cuda_stream)
    assert vsl.lib.vsl_policy_loss(at, R, len(slices), V_s, ctypes.byref(i), ctypes.byref(o), stream) == 0
    return loss, lp, kl


# CTAs of 128, 256 and 512 threads, the row kept in registers between its passes or read again
FORMS = [(4, 2, 1000), (1500, 1, 8000), (16, 2, 10000), (40, 4, 37984), (100, 1, 12000), (300, 3, 17004), (2, 1, 4)]


@pytest.mark.parametrize("R,S,V_s", FORMS)
def test_policy_loss_without_entropy(cuda_device, R, S, V_s):
    """The form without the entropy's sums: the same numbers, bit for bit, as the one with them."""
    g = torch.Generator(device=cuda_device)
    g.manual_seed(R + V_s)
    slices = [torch.randn(R, V_s, generator=g, device=cuda_device) * 2 for _ in range(S)]
    tok = torch.randint(0, S * V_s, (R,), generator=g, device=cuda_device, dtype=torch.int32)
    tok[R // 2] = -1
    if R > 2:
        slices[0][1, 1], slices[0][0, 2] = float("nan"), -float("inf")
    lp = vsl.token_logprobs(slices, tok).logprob
    old, ref = lp - 0.1, lp + 0.2
    adv = torch.randn(R, generator=g, device=cuda_device)
    same = lambda x, y: torch.equal(x.view(torch.uint8), y.view(torch.uint8))  # noqa: E731
    for kind, dtype in ((0, torch.float32), (1, torch.bfloat16)):
        for kl_coef in (0.0, 0.05):
            want = vsl.policy_loss(slices, tok, old, adv, ref_logprob=ref, clip_high=0.28, kl_coef=kl_coef, grad_dtype=dtype)
            grad = [torch.full_like(x, 3.0, dtype=dtype) for x in slices]
            loss, lp_out, kl = _policy_c(slices, tok, old, adv, ref, kl_coef, kind, grad, True, True)
            assert same(loss, want.loss) and same(lp_out, want.logprob) and same(kl, want.kl)
            assert all(same(x, y) for x, y in zip(grad, want.grad))
            loss, lp_out, kl = _policy_c(slices, tok, old, adv, ref, kl_coef, kind, None, False, False)
            assert same(loss, want.loss) and bool(torch.isnan(lp_out).all()) and bool(torch.isnan(kl).all())
