"""Parity of the low-rank adapters with the float64 oracle (GPU); the bound is ``oracle.adapters.adapters_add_bound``."""
import numpy as np
import pytest
import torch

import vocab_sharded_logits_b200 as vsl
from oracle import adapters as A

pytestmark = pytest.mark.gpu


def _inputs(R, H, S, V_s, n, rank, seed, dev, ids=None):
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g, device=dev)  # noqa: E731
    hidden = rand(R, H).bfloat16()
    logits = [rand(R, V_s) for _ in range(S)]
    a = (rand(n, rank, H) / H ** 0.5).bfloat16()
    b = [(rand(n, V_s, rank) * 0.3).bfloat16() for _ in range(S)]
    scale = 0.5 + torch.rand(n, generator=g, device=dev)
    if ids is None:
        ids = np.random.default_rng(seed).integers(-1, n + 1, R)      # -1 and n: no adapter
    return hidden, logits, a, b, scale, torch.as_tensor(ids, dtype=torch.int32, device=dev)


def _np(x):
    return x.float().cpu().numpy().astype(np.float64)


def _check(out, logits, hidden, a, b, ids, scale):
    args = ([_np(x) for x in logits], _np(hidden), _np(a), [_np(x) for x in b], ids.cpu().numpy(),
            None if scale is None else _np(scale))
    want, bound = A.adapters_add(*args), A.adapters_add_bound(*args)
    for o, w, e in zip(out, want, bound):
        off = np.abs(_np(o) - w)
        assert (off <= e).all(), (off / e).max()


@pytest.mark.parametrize("R,H,S,V_s,n,rank", [
    (1, 8, 1, 4, 1, 8),            # the smallest call
    (1, 4096, 2, 1000, 3, 16),     # one row
    (5, 136, 3, 132, 2, 24),       # ragged H, ids, rank
    (16, 64, 1, 128, 4, 16),       # whole groups
    (17, 512, 2, 1004, 20, 40),    # a group of one row; rank not a multiple of 16
    (33, 264, 4, 260, 3, 64),
    (70, 320, 1, 388, 70, 8),      # nearly every row its own adapter
    (130, 128, 2, 516, 5, 48),
    (20, 64, 2, 144, 3, 256),      # the largest rank
    (1000, 64, 1, 64, 7, 16),      # many rows, few ids
    (600, 64, 16, 132, 9, 32),     # three tiles of rows, blocks over many slices
    (300, 1040, 2, 1000, 40, 64),  # H shared by a cluster, ragged units
    (280, 72, 3, 20, 4, 56),       # slices of less than a block
    (100, 72, 2, 388, 2, 128),     # ranks above 64, several units an adapter
    (300, 64, 1, 260, 1, 200),
])
def test_parity(cuda_device, R, H, S, V_s, n, rank):
    hidden, logits, a, b, scale, ids = _inputs(R, H, S, V_s, n, rank, R + rank, cuda_device)
    for s in (scale, None):
        out = vsl.adapters_add(logits, hidden, a, b, ids, scale=s)
        _check(out, logits, hidden, a, b, ids, s)
    # in place, with the tile statistics: the same logits; the statistics are those of the statistics kernel
    want = vsl.adapters_add(logits, hidden, a, b, ids, scale=scale)
    over = [x.clone() for x in logits]
    got, stats = vsl.adapters_add(over, hidden, a, b, ids, scale=scale, out=over, tile_stats=True)
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    ref = vsl.tile_stats(want)
    assert torch.equal(stats[..., :4], ref[..., :4]) and torch.equal(stats[..., 5:], ref[..., 5:])
    # sums of at most 128 exponentials, each within 2^-22 + 2^-23 |l - c| (below 16 here), in two orders
    assert bool(((stats[..., 4] - ref[..., 4]).abs() <= ref[..., 4] * 2 * (2.0 ** -22 + 2.0 ** -19 + 2.0 ** -17)).all())
    over = [x.clone() for x in logits]
    vsl.adapters_add(over, hidden, a, b, ids, scale=scale, out=over)
    assert all(torch.equal(x, y) for x, y in zip(over, want))


@pytest.mark.parametrize("rank", [8, 16, 24, 32, 40, 64, 72, 128, 200, 256])
@pytest.mark.parametrize("per", [1, 2, 3])
def test_units_of_few_rows(cuda_device, rank, per):
    """Every adapter with one, two or three rows: multiply-adds up to two, products above."""
    R = 6 * per
    ids = np.arange(R) // per
    hidden, logits, a, b, scale, ids = _inputs(R, 72, 2, 300, 6, rank, rank + per, cuda_device, ids)
    out, stats = vsl.adapters_add(logits, hidden, a, b, ids, scale=scale, tile_stats=True)
    _check(out, logits, hidden, a, b, ids, scale)
    ref = vsl.tile_stats(out)
    assert torch.equal(stats[..., :4], ref[..., :4]) and torch.equal(stats[..., 5:], ref[..., 5:])
    assert bool(((stats[..., 4] - ref[..., 4]).abs() <= ref[..., 4] * 2 * (2.0 ** -22 + 2.0 ** -19 + 2.0 ** -17)).all())


@pytest.mark.parametrize("pattern", ["alone", "three"])
def test_statistics_of_unusual_logits(cuda_device, pattern):
    """-inf, +inf, NaN and zeros in the base logits: the records are those of the statistics kernel on the result."""
    R = 8
    ids = {"alone": np.arange(R), "three": np.arange(R) // 3}[pattern]
    hidden, logits, a, b, scale, ids = _inputs(R, 64, 2, 388, 8, 16, 6, cuda_device, ids)
    a[0], b[0][1], b[1][1] = 0.0, 0.0, 0.0
    for x in logits:
        x[0, 3:40], x[1, 128:256], x[2, 7], x[3, 200], x[4, 384:] = 0.0, -np.inf, np.inf, np.nan, -np.inf
        x[5] = -np.inf
    out, stats = vsl.adapters_add(logits, hidden, a, b, ids, scale=scale, tile_stats=True)
    ref = vsl.tile_stats(out)
    quarter_nan = torch.cat([torch.nn.functional.pad(x, (0, -388 % 128)).view(R, -1, 4, 32).isnan().any(3) for x in out], 1)
    same = (stats[..., :4] == ref[..., :4]) | quarter_nan         # a quarter that holds a NaN has no maximum to agree on
    assert bool(same.all())
    assert torch.equal(stats[..., 5:], ref[..., 5:])
    s, r = stats[..., 4], ref[..., 4]
    bad = ~torch.isfinite(r)
    assert torch.equal(bad, ~torch.isfinite(s)) and torch.equal(r.isnan(), s.isnan())
    assert bool(((s - r).abs() <= r * 2 * (2.0 ** -22 + 2.0 ** -19 + 2.0 ** -17))[~bad].all())


@pytest.mark.parametrize("pattern", ["one", "none", "runs", "distinct", "alternate"])
def test_patterns_of_ids(cuda_device, pattern):
    R, n = 96, 96
    ids = {"one": np.full(R, 5), "none": np.full(R, -1), "runs": np.arange(R) // 8, "distinct": np.arange(R)[::-1].copy(),
           "alternate": np.arange(R) % 2 * 3}[pattern]
    hidden, logits, a, b, scale, ids = _inputs(R, 256, 2, 516, n, 16, 3, cuda_device, ids)
    out = vsl.adapters_add(logits, hidden, a, b, ids, scale=scale)
    _check(out, logits, hidden, a, b, ids, scale)
    if pattern == "none":
        assert all(torch.equal(x, y) for x, y in zip(out, logits))


def test_rows_without_an_adapter_keep_their_bits(cuda_device):
    R, n = 50, 4
    ids = np.where(np.arange(R) % 3 == 0, [-1, n, 2 ** 31 - 1, -2 ** 31] * 12 + [-1, -1], np.arange(R) % n)
    hidden, logits, a, b, scale, ids = _inputs(R, 128, 2, 260, n, 16, 4, cuda_device, ids)
    for x in logits:
        x[0, 5], x[3, 7], x[6, 1] = float("nan"), float("inf"), float("-inf")
    out = vsl.adapters_add(logits, hidden, a, b, ids, scale=scale)
    for x, y in zip(out, logits):
        assert torch.equal(x[::3].view(torch.int32), y[::3].view(torch.int32))


def test_integer_inputs_are_exact(cuda_device):
    """Small integers: every product and sum is exact, so any order of summation gives the same numbers."""
    g = torch.Generator(device=cuda_device)
    g.manual_seed(1)
    R, H, V_s, n, rank = 40, 512, 300, 6, 24
    r = lambda *s: torch.randint(-3, 4, s, generator=g, device=cuda_device)  # noqa: E731
    hidden, a, b = r(R, H).bfloat16(), r(n, rank, H).bfloat16(), [r(n, V_s, rank).bfloat16() for _ in range(2)]
    logits = [r(R, V_s).float() for _ in range(2)]
    ids = torch.randint(-1, n, (R,), generator=g, device=cuda_device, dtype=torch.int32)
    out = vsl.adapters_add(logits, hidden, a, b, ids)
    want = A.adapters_add([_np(x) for x in logits], _np(hidden), _np(a), [_np(x) for x in b], ids.cpu().numpy())
    for o, w in zip(out, want):
        assert np.array_equal(_np(o), w)


def test_another_rows_infinities_do_not_spread(cuda_device):
    """Row groups hold several adapters: NaN and inf in one row's hidden states, logits or adapter reach that row only."""
    R, n = 16, 4
    ids = np.arange(R) % n
    hidden, logits, a, b, scale, ids = _inputs(R, 128, 1, 260, n, 16, 5, cuda_device, ids)
    clean = vsl.adapters_add(logits, hidden, a, b, ids, scale=scale)[0]
    hidden[5, 3] = float("nan")
    a[2, 1, 7] = float("inf")
    b[0][3, 11] = float("nan")
    b[0][3, 12] = float("inf")
    got = vsl.adapters_add(logits, hidden, a, b, ids, scale=scale)[0]
    touched = np.zeros((R, 260), bool)
    touched[5] = True
    touched[2::4] = True
    touched[3::4, 11:13] = True
    same = (got.view(torch.int32) == clean.view(torch.int32)).cpu().numpy()
    assert same[~touched].all()
    g = got.cpu().numpy()
    assert np.isnan(g[5]).all() and not np.isfinite(g[2::4]).any() and np.isnan(g[3::4, 11]).all()


def test_large_and_small_terms_keep_24_bits(cuda_device):
    """u of 1 + 2^-20 against B of 1 and a logit of -1: rounding u to fewer bits would lose the difference."""
    hidden = torch.zeros(1, 16, device=cuda_device).bfloat16()
    hidden[0, 0], hidden[0, 1] = 1.0, 2.0 ** -20
    a = torch.ones(1, 8, 16, device=cuda_device).bfloat16()
    b = [torch.zeros(1, 4, 8, device=cuda_device).bfloat16()]
    b[0][0, :, 0] = 1.0
    logits = [torch.full((1, 4), -1.0, device=cuda_device)]
    out = vsl.adapters_add(logits, hidden, a, b, torch.zeros(1, dtype=torch.int32, device=cuda_device))[0]
    assert bool((out == 2.0 ** -20).all())


def test_repeatable_streams_graphs_and_workspaces(cuda_device):
    """Bitwise repeatable; two captured graphs with a workspace each, replayed at once; a stream that is not current."""
    cases = [_inputs(40, 512, 2, 2000, 8, 16, seed, cuda_device) for seed in (1, 2)]
    want = [vsl.adapters_add(l, h, a, b, i, scale=s) for h, l, a, b, s, i in cases]
    again = [vsl.adapters_add(l, h, a, b, i, scale=s) for h, l, a, b, s, i in cases]
    graphs, outs, streams = [], [], [torch.cuda.Stream(), torch.cuda.Stream()]
    spaces = [torch.empty(vsl.adapters_workspace_bytes(40, 8, 16), dtype=torch.uint8, device=cuda_device) for _ in cases]
    torch.cuda.synchronize()
    for (h, l, a, b, s, i), ws, stream in zip(cases, spaces, streams):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            outs.append(vsl.adapters_add(l, h, a, b, i, scale=s, workspace=ws))
        graphs.append(graph)
    for _ in range(20):
        for graph, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    h, l, a, b, s, i = cases[0]
    streams[0].wait_stream(torch.cuda.current_stream())
    side = vsl.adapters_add(l, h, a, b, i, scale=s, stream=streams[0])
    torch.cuda.synchronize()
    for k in range(2):
        for x, y, z in zip(want[k], again[k], outs[k]):
            assert torch.equal(x, y) and torch.equal(x, z)
    assert all(torch.equal(x, y) for x, y in zip(side, want[0]))
    small = torch.empty(16, dtype=torch.uint8, device=cuda_device)
    with pytest.raises(vsl.VslError):
        vsl.adapters_add(l, h, a, b, i, workspace=small)


def test_from_projection_to_gradient(cuda_device):
    """The operators as they are used together: projection, adapters, sampling with the statistics, scoring under
    the policy and under the base model, the policy loss and its gradient, then a preference loss of the same rows."""
    from oracle import scores as O
    import score_bounds as B
    R, H, S, V_s, n, rank = 24, 256, 2, 520, 3, 16
    hidden, _, a, b, scale, ids = _inputs(R, H, S, V_s, n, rank, 8, cuda_device, np.arange(24) % 4 - 1)
    g = torch.Generator(device=cuda_device)
    g.manual_seed(2)
    w = [(torch.randn(V_s, H, generator=g, device=cuda_device) * 0.1).bfloat16() for _ in range(S)]
    base = vsl.logits_local(hidden, w)
    logits, stats = vsl.adapters_add(base, hidden, a, b, ids, scale=scale, tile_stats=True)
    params = vsl.make_row_params(np.ones(R), np.full(R, 40), np.ones(R), np.arange(R), np.zeros(R), cuda_device)
    drawn = vsl.sample(logits, params, 7, 5, tile_stats=stats)
    plain = vsl.sample(logits, params, 7, 5)
    assert torch.equal(drawn.token_ids, plain.token_ids)
    policy = vsl.token_logprobs(logits, drawn.token_ids, entropy=True)
    V = S * V_s
    l64 = np.concatenate([_np(x) for x in logits], 1)
    tokens = drawn.token_ids.cpu().numpy()
    logp = O.log_softmax(l64)
    lp, _ = O.token_logprobs(l64, tokens)
    assert (np.abs(_np(policy.logprob) - lp) <= B.logprob_bound(logp, lp)).all()
    assert (np.abs(_np(drawn.token_logprob) - lp) <= 1e-4).all()      # the sampler's own tolerance
    ref = vsl.token_logprobs(base, drawn.token_ids)
    none = (ids < 0).cpu().numpy()
    assert torch.equal(ref.logprob[torch.from_numpy(none)], policy.logprob[torch.from_numpy(none)])
    adv = torch.randn(R, generator=g, device=cuda_device)
    old = policy.logprob.clone()
    out = vsl.policy_loss(logits, drawn.token_ids, old, adv, weights=torch.full((R,), 1 / R, device=cuda_device),
                          ref_logprob=ref.logprob, kl_coef=0.1)
    f = lambda t: _np(t)  # noqa: E731
    want = O.policy_loss(l64, tokens, f(old), f(adv), weights=np.full(R, np.float32(1 / R)), ref=f(ref.logprob),
                         lo=np.float64(np.float32(0.2)), hi=np.float64(np.float32(0.2)), kl_coef=np.float64(np.float32(0.1)))
    err = B.logprob_bound(logp, 0 * lp)
    d = f(ref.logprob) - want["logprob"]
    err_g = 1 / R * (np.abs(f(adv)) + 0.1 * np.exp(d)) * err * 1.01
    bound = B.grad_bound(logp, tokens, 1.0, want["d_lp"], want["d_ent"], err_g, 0 * err, want["grad"], "fp32")
    got = np.concatenate([_np(x) for x in out.grad], 1)
    assert (np.abs(got - want["grad"]) <= bound).all()
    at = torch.arange(0, 25, 6, dtype=torch.int32, device=cuda_device)
    pref = vsl.preference_loss(policy.logprob, ref.logprob, at, 0.1)
    grad = vsl.token_logprobs_grad(logits, drawn.token_ids, policy, pref.d_logprob)
    _, _, dl = O.preference_loss(f(policy.logprob), f(ref.logprob), at.cpu().numpy(), np.float64(np.float32(0.1)))
    want_g = O.token_logprobs_grad(l64, tokens, dl)
    bound = B.grad_bound(logp, tokens, 1.0, dl, 0 * dl, np.abs(dl) * 2.0 ** -23, 0 * dl, want_g, "fp32")
    assert (np.abs(np.concatenate([_np(x) for x in grad], 1) - want_g) <= bound).all()
    assert V == l64.shape[1] and vsl.device_error() == (0, 0)


@pytest.mark.parametrize("rank", [8, 16, 32, 64])
def test_small_terms_survive_a_cancelled_logit(cuda_device, rank):
    """u = 1 + 2^-10 + 2^-20, B = 1 + 2^-7: the product has 28 bits, and the base logit takes the first away."""
    R, H, V_s = 20, 8, 260
    hidden = torch.zeros(R, H)
    hidden[:, 0], hidden[:, 1], hidden[:, 2] = 1.0, 2.0 ** -10, 2.0 ** -20
    a, b = torch.zeros(1, rank, H), torch.zeros(1, V_s, rank)
    a[0, 0, :3], b[0, :, 0] = 1.0, 1 + 2.0 ** -7
    bf16 = lambda x: x.to(cuda_device, torch.bfloat16)  # noqa: E731
    logits = torch.full((R, V_s), -(1 + 2.0 ** -7), device=cuda_device)
    ids = torch.zeros(R, dtype=torch.int32, device=cuda_device)
    out, = vsl.adapters_add([logits], bf16(hidden), bf16(a), [bf16(b)], ids)
    assert bool((out == 2.0 ** -10 + 2.0 ** -17 + 2.0 ** -20 + 2.0 ** -27).all())


@pytest.mark.parametrize("rank", [8, 16, 32, 64, 128])
@pytest.mark.parametrize("per", [1, 2, 3])
@pytest.mark.parametrize("V_s", [132, 260, 388])
def test_statistics_of_a_slice_that_ends_in_an_infinity(cuda_device, V_s, per, rank):
    """The last id's product overflows to +inf; what is behind it in its block belongs to no id."""
    R = 6 * per
    hidden, logits, a, b, scale, ids = _inputs(R, 64, 2, V_s, 6, rank, rank + per, cuda_device, np.arange(R) // per)
    hidden[:, 0] = 2.0 ** 126
    a[:, :, 0] = 0.0
    a[:, 0] = 0.0
    a[:, 0, 0] = 1.0                                      # u = 2^126 in the first rank alone
    for x in b:
        x[:, :, 0] = 0.0
        x[:, V_s - 1, 0] = 8.0
    out, stats = vsl.adapters_add(logits, hidden, a, b, ids, tile_stats=True)
    assert all(bool((x[:, -1] == float("inf")).all()) and bool(torch.isfinite(x[:, :-1]).all()) for x in out)
    ref = vsl.tile_stats(out)
    assert torch.equal(stats[..., :4], ref[..., :4]) and torch.equal(stats[..., 5:], ref[..., 5:])
    s, r = stats[..., 4], ref[..., 4]
    bad = ~torch.isfinite(r)
    assert bool((s[bad] == r[bad]).all())                 # +inf, no NaN
    assert bool(((s - r).abs() <= r * 2 * (2.0 ** -22 + 2.0 ** -19 + 2.0 ** -17))[~bad].all())


@pytest.mark.parametrize("rank", [72, 128, 200, 256])
def test_small_terms_survive_a_cancelled_logit_above_rank_64(cuda_device, rank):
    """The same, with the ranks that count at both ends of the sum."""
    R, H, V_s = 20, 8, 260
    hidden = torch.zeros(R, H)
    hidden[:, 0], hidden[:, 1], hidden[:, 2] = 1.0, 2.0 ** -10, 2.0 ** -20
    for k in (0, rank // 2, rank - 1):
        a, b = torch.zeros(1, rank, H), torch.zeros(1, V_s, rank)
        a[0, k, :3], b[0, :, k] = 1.0, 1 + 2.0 ** -7
        bf16 = lambda x: x.to(cuda_device, torch.bfloat16)  # noqa: E731
        logits = torch.full((R, V_s), -(1 + 2.0 ** -7), device=cuda_device)
        ids = torch.zeros(R, dtype=torch.int32, device=cuda_device)
        out, = vsl.adapters_add([logits], bf16(hidden), bf16(a), [bf16(b)], ids)
        assert bool((out == 2.0 ** -10 + 2.0 ** -17 + 2.0 ** -20 + 2.0 ** -27).all())


@pytest.mark.parametrize("rank", [8, 16, 32, 64, 128])
@pytest.mark.parametrize("per", [1, 2, 3, 20])
def test_a_finite_product_at_the_end_of_the_range(cuda_device, rank, per):
    """u = +-(2^128 - 2^118), finite in float32 and above the largest bf16: its terms are finite too.  B = 2^-120 gives
    +-255.75 exactly, B = 0 nothing, however many rows share the adapter."""
    R, H, V_s = 2 * per, 16, 260
    hidden = torch.zeros(R, H)
    hidden[:, :10] = 2.0 ** torch.arange(127.0, 117.0, -1.0)
    hidden[per:] *= -1
    a, b = torch.zeros(2, rank, H), torch.zeros(2, V_s, rank)
    a[:, rank - 1], b[:, ::2, rank - 1] = 1.0, 2.0 ** -120
    bf16 = lambda x: x.to(cuda_device, torch.bfloat16)  # noqa: E731
    logits = torch.ones(R, V_s, device=cuda_device)
    ids = (torch.arange(R, device=cuda_device) // per).int()
    out, = vsl.adapters_add([logits], bf16(hidden), bf16(a), [bf16(b)], ids)
    assert bool((out[:, 1::2] == 1).all())
    assert bool((out[:per, ::2] == 256.75).all()) and bool((out[per:, ::2] == -254.75).all())


def _unit_sums(a, b, ids, hidden, logits):
    """The formula in float64 (products of these bf16 values are exact in it): infinities and NaNs as they come."""
    out = [_np(x) for x in logits]
    with np.errstate(all="ignore"):
        for r, i in enumerate(ids):
            u = (_np(a[i]) * _np(hidden[r])).sum(1)
            for x, y in zip(out, b):
                x[r] += (_np(y[i]) * u).sum(1)
    return out


@pytest.mark.parametrize("rank", [8, 16, 24, 40, 64, 72, 200])
@pytest.mark.parametrize("per", [1, 2, 3, 20])
def test_infinite_factors_of_a_rows_own(cuda_device, rank, per):
    """An infinity in a row's own factors gives what the formula gives, +inf, -inf or NaN, however many rows share the
    adapter and whatever the rank is padded to."""
    R, H, V_s = 5 * per, 16, 260
    g = torch.Generator(device=cuda_device)
    g.manual_seed(rank + per)
    hidden, logits, a, b, scale, ids = _inputs(R, H, 2, V_s, 5, rank, 3, cuda_device, np.arange(R) // per)
    inf = float("inf")
    b[0][0, 3, rank - 1], b[0][0, 5, 0], b[1][0, V_s - 1, 2], b[1][0, 7, :2] = inf, -inf, inf, torch.tensor([inf, -inf])
    hidden[per:2 * per, 0] = inf                 # u infinite: of one sign in every rank, then of both
    a[1, :, 0] = a[1, :, 0].abs() + 1
    b[0][1] = b[0][1].abs() + 1
    hidden[2 * per:3 * per, 2] = -inf
    a[3] = 0.0                                   # u = 1 exactly: its small terms are 0
    a[3, :, 1], hidden[3 * per:4 * per, 1] = 1.0, 1.0
    b[0][3, 11], b[1][3, 12, rank // 2] = inf, -inf
    hidden[4 * per:, 3], b[0][4, 9, 1] = inf, inf
    got = vsl.adapters_add(logits, hidden, a, b, ids)
    want = _unit_sums(a, b, ids.cpu().numpy(), hidden, logits)
    for x, y in zip(got, want):
        x = _np(x)
        assert np.array_equal(np.isnan(x), np.isnan(y))
        assert np.array_equal(np.isposinf(x), np.isposinf(y)) and np.array_equal(np.isneginf(x), np.isneginf(y))
