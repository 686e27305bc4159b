"""Cases of the operators beside the projection and the sampler: per-row low-rank adapters on the
logits slices, logprobs of given tokens with their gradient, and the two losses made of them.

Every operator works on the vocab-sliced layout: S fp32 slices of [R, V_s], row r the
concatenation of its slices.  ``run`` computes a case with elementary torch operations, or, where
``own`` is true, with the calls of ``vocab_sharded_logits_b200``.
"""
import math

import torch

own = False

DEV = "cuda"

# ----------------------------------------------------------------------------- the cases


def listed():
    return [
        # adapters_add -- serving.  One request decoding one token: latency counts.
        dict(name="adapters 1 row", op="adapters", R=1, per=1, S=4, V_s=37984, H=4096, n=8, rank=16, none=False,
             stats=False),
        # 64 requests decoding, each with an adapter of its own: every adapter's vocabulary factor is read.
        dict(name="adapters 64 requests", op="adapters", R=64, per=1, S=4, V_s=37984, H=4096, n=64, rank=16,
             none=False, stats=False),
        # speculative verification: 128 requests x 4 rows, a quarter of them on the base model; the sampler
        # that follows reads the tile statistics.
        dict(name="adapters spec, statistics", op="adapters", R=512, per=4, S=4, V_s=37984, H=4096, n=24, rank=32,
             none=True, stats=True),
        # a large batch (256 requests x 8 rows) over a few adapters of high rank.
        dict(name="adapters large batch", op="adapters", R=2048, per=8, S=8, V_s=18992, H=5120, n=8, rank=64,
             none=False, stats=False),
        # token_logprobs -- scoring an odd number of prompt positions over an odd-sized vocabulary.
        dict(name="logprobs odd sizes", op="logprobs", R=77, S=3, V_s=17004, T=1.0, ent=True, grad="none"),
        # scoring a reference policy: 64 rows of the wide vocabulary, logprobs alone.
        dict(name="logprobs wide", op="logprobs", R=64, S=8, V_s=31040, T=1.0, ent=False, grad="none"),
        # the backward pass of a loss of logprobs and entropies over a spec-sized batch.
        dict(name="logprobs and gradient", op="logprobs", R=512, S=4, V_s=37984, T=0.8, ent=True, grad="fp32"),
        # policy_loss -- the smallest batch and vocabulary: latency.
        dict(name="policy tiny", op="policy", R=4, S=2, V_s=512, T=1.0, kl=0.05, ent=0.0, grad="fp32"),
        # an ordinary update: bf16 gradient for the next product, temperature, entropy bonus.
        dict(name="policy 512 rows, bf16", op="policy", R=512, S=4, V_s=37984, T=0.8, kl=0.02, ent=0.01, grad="bf16"),
        # the largest batch.
        dict(name="policy 2048 rows", op="policy", R=2048, S=8, V_s=18992, T=1.0, kl=0.05, ent=0.0, grad="fp32"),
        # preference_loss between the logprobs and their gradient: a few short ragged pairs.
        dict(name="preference 4 pairs", op="preference", pairs=4, length=9, S=4, V_s=3000, T=1.0, grad="fp32"),
        # 16 pairs of longer answers over the largest vocabulary, bf16 gradient.
        dict(name="preference 16 pairs", op="preference", pairs=16, length=32, S=8, V_s=32768, T=1.0, grad="bf16"),
    ]


def _log_int(rng, lo, hi, step=1):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step))


def draw(rng):
    op = rng.choice(["adapters", "adapters", "logprobs", "policy", "policy", "preference"])
    S = rng.choice([1, 2, 3, 4, 5, 8])
    V_s = _log_int(rng, 512, 262144 // S, 4)
    most = 120_000_000 // (S * V_s)  # rows: at most some 0.5 GB of logits
    T = rng.choice([1.0, 1.0, 0.7, 1.3])
    grad = rng.choice(["fp32", "bf16"])
    if op == "adapters":
        per = rng.choice([1, 1, 2, 4, 8])
        R = per * _log_int(rng, 1, max(1, min(1024, most) // per))
        rank = rng.choice([8, 16, 16, 24, 32, 48, 64])
        n = _log_int(rng, 1, max(1, min(64, 1024 // rank)))
        return dict(op=op, R=R, per=per, S=S, V_s=V_s, H=_log_int(rng, 64, 5120, 8), n=n, rank=rank,
                    none=rng.random() < 0.4, stats=rng.random() < 0.3)
    if op == "preference":
        length = _log_int(rng, 2, 64)
        return dict(op=op, pairs=_log_int(rng, 1, max(1, min(256, most // (2 * length)))), length=length, S=S, V_s=V_s,
                    T=T, grad=grad)
    R = _log_int(rng, 1, min(1024, most))
    if op == "logprobs":
        return dict(op=op, R=R, S=S, V_s=V_s, T=T, ent=rng.random() < 0.5, grad=rng.choice(["none", "fp32", "bf16"]))
    return dict(op=op, R=R, S=S, V_s=V_s, T=T, kl=rng.choice([0.0, 0.05]), ent=rng.choice([0.0, 0.01]), grad=grad)


# ----------------------------------------------------------------------------- inputs


def _adapter_of_request(case):
    """The adapter of each request (-1: the base model), before they are shuffled."""
    requests = case["R"] // case["per"]
    ids = torch.arange(requests) % case["n"]
    if case["none"]:
        ids[::4] = -1
    return ids


def _prepare_adapters(case, g):
    R, S, V_s, H, n, rank = (case[k] for k in ("R", "S", "V_s", "H", "n", "rank"))
    rand = lambda *shape: torch.randn(*shape, generator=g, device=DEV)  # noqa: E731
    hidden = rand(R, H).bfloat16()
    logits = [rand(R, V_s) * (0.02 * math.sqrt(H)) for _ in range(S)]  # the spread of hidden . W for std(W) = 0.02
    a = (rand(n, rank, H) / math.sqrt(H)).bfloat16()
    b = [(rand(n, V_s, rank) * 0.1).bfloat16() for _ in range(S)]
    scale = 0.5 + torch.rand(n, generator=g, device=DEV)
    ids = _adapter_of_request(case).to(DEV)
    ids = ids[torch.randperm(ids.numel(), generator=g, device=DEV)].repeat_interleave(case["per"])
    return dict(case=case, hidden=hidden, logits=logits, a=a, b=b, scale=scale, ids=ids.to(torch.int32))


def _prepare_rows(case, R, g):
    """Logits of the projection's spread, and tokens drawn from them as the sampler would draw them."""
    S, V_s, T = case["S"], case["V_s"], case["T"]
    full = torch.randn(R, S * V_s, generator=g, device=DEV) * 1.28
    tokens = torch.multinomial(torch.softmax(full / T, 1), 1, generator=g)[:, 0]
    full64 = full.double().div_(T)
    lp = full64.gather(1, tokens[:, None])[:, 0] - torch.logsumexp(full64, 1)
    logits = [full[:, s * V_s:(s + 1) * V_s].contiguous() for s in range(S)]
    return dict(case=case, logits=logits, tokens=tokens.to(torch.int32)), lp


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    if case["op"] == "adapters":
        return _prepare_adapters(case, g)
    noise = lambda k, sd: torch.randn(k, generator=g, device=DEV, dtype=torch.float64) * sd  # noqa: E731
    if case["op"] == "preference":
        # ragged answers; each starts with a prompt token, which does not count (-1)
        lens = torch.randint(max(1, case["length"] // 2), case["length"] + 1, (2 * case["pairs"],), generator=g,
                             device=DEV)
        offsets = torch.zeros(2 * case["pairs"] + 1, dtype=torch.int32, device=DEV)
        offsets[1:] = lens.cumsum(0)
        R = 2 * case["pairs"] * case["length"]  # rows behind the last sequence are padding
        st, lp = _prepare_rows(case, R, g)
        st["tokens"][offsets[:-1].long()] = -1
        st["tokens"][int(offsets[-1]):] = -1
        st["offsets"] = offsets
        st["ref"] = torch.where(st["tokens"] >= 0, lp + noise(R, 0.3), 0.0).float()
        return st
    R = case["R"]
    st, lp = _prepare_rows(case, R, g)
    if case["op"] == "logprobs":
        st["d_logprob"], st["d_entropy"] = noise(R, 1.0).float(), noise(R, 0.1).float()
        return st
    # policy: the behaviour policy a few updates old; no ratio within 1e-3 of a clipping border
    delta = noise(R, 0.2)
    for border in (math.log(1 - 0.2), math.log(1 + 0.28)):
        delta = torch.where((delta - border).abs() < 1e-3, delta + 3e-3, delta)
    st["old"], st["ref"], st["adv"] = (lp - delta).float(), (lp + noise(R, 0.3)).float(), noise(R, 1.0).float()
    on = max(1, R - R // 10)  # the batch is padded: the last tenth of the rows do not count
    st["weights"] = torch.zeros(R, device=DEV)
    st["weights"][:on] = 1.0 / on
    return st


# ----------------------------------------------------------------------------- one pass


def _tile_statistics(slices):
    """Per block of 128 ids: the four 32-id maxima, sum of exp(l - block maximum), the smallest logit, the smallest
    nonzero |l|, 0."""
    R, V_s = slices[0].shape
    x = torch.stack(slices, 1)
    pad = -V_s % 128
    low = torch.nn.functional.pad(x, (0, pad), value=-math.inf).view(R, -1, 4, 32)
    high = torch.nn.functional.pad(x, (0, pad), value=math.inf).view(R, -1, 128)
    quarters = low.amax(3)
    top = quarters.amax(2)
    total = torch.exp(low.reshape(R, -1, 128) - top[..., None]).sum(2)
    least = torch.where(high == 0, math.inf, high.abs()).amin(2)
    return torch.cat([quarters, torch.stack([total, high.amin(2), least, torch.zeros_like(top)], 2)], 2)


def _plain_adapters(st):
    case = st["case"]
    n, rank = case["n"], case["rank"]
    mine = (st["ids"][:, None] == torch.arange(n, device=DEV)) * st["scale"]  # [R, n]: a row's scale at its adapter
    u = st["hidden"].float() @ st["a"].float().reshape(n * rank, -1).T
    u = (u.view(-1, n, rank) * mine[:, :, None]).reshape(-1, n * rank)
    return [x + u @ b.float().transpose(1, 2).reshape(n * rank, -1) for x, b in zip(st["logits"], st["b"])]


def _plain_rows(st):
    """Softmax statistics of every row: x - max, exp of it, its sum, and the token's logprob and the entropy."""
    x = torch.cat(st["logits"], 1) / st["case"]["T"]
    x = x - x.amax(1, keepdim=True)
    e = torch.exp(x)
    z = e.sum(1, dtype=torch.float64)
    on = (st["tokens"] >= 0) & (st["tokens"] < x.shape[1])
    t = st["tokens"].long().clamp(0, x.shape[1] - 1)
    lp = torch.where(on, x.gather(1, t[:, None])[:, 0] - torch.log(z), 0.0)
    h = torch.where(on, torch.log(z) - (e * x).sum(1, dtype=torch.float64) / z, 0.0)
    return dict(x=x, e=e, z=z, on=on, t=t, lp=lp, h=h)


def _plain_gradient(st, rows, d_lp, d_h, kind):
    """The gradient of a function of the rows' logprobs and entropies (its derivatives by them: d_lp, d_h)."""
    d_lp, d_h = torch.where(rows["on"], d_lp, 0.0), torch.where(rows["on"], d_h, 0.0)
    p = rows["e"] / rows["z"][:, None].float()
    shift = (rows["h"] - torch.log(rows["z"]))[:, None].float()
    grad = -p * (d_lp[:, None].float() + d_h[:, None].float() * (rows["x"] + shift))
    grad.scatter_add_(1, rows["t"][:, None], d_lp[:, None].float())
    grad = grad / st["case"]["T"]
    return list((grad.bfloat16() if kind == "bf16" else grad).split(st["case"]["V_s"], 1))


def _plain_policy(st):
    case, rows, w, adv = st["case"], _plain_rows(st), st["weights"].double(), st["adv"].double()
    ratio = torch.exp(rows["lp"] - st["old"])
    clipped = ratio.clamp(1 - 0.2, 1 + 0.28)
    d = st["ref"] - rows["lp"]
    on = rows["on"] & (w != 0)
    kl = torch.where(on, torch.exp(d) - d - 1, 0.0)
    inside = (ratio * adv <= clipped * adv).double()
    loss = torch.where(on, w * (-torch.minimum(ratio * adv, clipped * adv) + case["kl"] * kl - case["ent"] * rows["h"]), 0.0)
    d_lp = torch.where(on, w * (-adv * ratio * inside + case["kl"] * (1 - torch.exp(d))), 0.0)
    out = dict(loss=loss, logprob=torch.where(on, rows["lp"], 0.0), kl=kl, entropy=torch.where(on, rows["h"], 0.0))
    out = {k: v.float() for k, v in out.items()}
    return dict(out, grad=_plain_gradient(st, rows, d_lp, -w * case["ent"], case["grad"]))


def _plain_preference(st):
    rows = _plain_rows(st)
    margin = rows["lp"].float().double() - st["ref"].double()
    offsets = st["offsets"].long()
    total = torch.nn.functional.pad(margin.cumsum(0), (1, 0))
    s = BETA * (total[offsets[1:]] - total[offsets[:-1]]).view(-1, 2)
    h = s[:, 0] - s[:, 1]
    loss = (1 - SMOOTHING) * torch.log1p(torch.exp(-h)) + SMOOTHING * torch.log1p(torch.exp(h))
    d_h = BETA * (SMOOTHING - 1 / (1 + torch.exp(h)))
    of_row = torch.bucketize(torch.arange(margin.numel(), device=DEV), offsets, right=True) - 1  # its sequence
    pair = (of_row // 2).clamp(max=h.numel() - 1)
    d_lp = torch.where(of_row < 2 * h.numel(), d_h[pair] * (1.0 - 2.0 * (of_row % 2)), 0.0)
    d_lp = torch.where(rows["on"], d_lp, 0.0)
    return dict(logprob=rows["lp"].float(), loss=loss.float(), rewards=s.float(),
                grad=_plain_gradient(st, rows, d_lp, torch.zeros_like(d_lp), st["case"]["grad"]))


BETA, SMOOTHING = 0.1, 0.05


def _own(st):
    import vocab_sharded_logits_b200 as vsl
    case = st["case"]
    if case["op"] == "adapters":
        out = vsl.adapters_add(st["logits"], st["hidden"], st["a"], st["b"], st["ids"], scale=st["scale"],
                               tile_stats=case["stats"])
        return dict(logits=out[0], stats=out[1]) if case["stats"] else dict(logits=out)
    kind = torch.bfloat16 if case["grad"] == "bf16" else torch.float32
    if case["op"] == "logprobs":
        fwd = vsl.token_logprobs(st["logits"], st["tokens"], temperature=case["T"], entropy=case["ent"])
        out = dict(logprob=fwd.logprob)
        if case["ent"]:
            out["entropy"] = fwd.entropy
        if case["grad"] != "none":
            out["grad"] = vsl.token_logprobs_grad(st["logits"], st["tokens"], fwd, st["d_logprob"],
                                                  d_entropy=st["d_entropy"] if case["ent"] else None, grad_dtype=kind)
        return out
    if case["op"] == "policy":
        r = vsl.policy_loss(st["logits"], st["tokens"], st["old"], st["adv"], weights=st["weights"],
                            ref_logprob=st["ref"], clip_low=0.2, clip_high=0.28, kl_coef=case["kl"],
                            entropy_coef=case["ent"], temperature=case["T"], grad_dtype=kind)
        return dict(loss=r.loss, logprob=r.logprob, kl=r.kl, entropy=r.entropy, grad=r.grad)
    fwd = vsl.token_logprobs(st["logits"], st["tokens"], temperature=case["T"])
    r = vsl.preference_loss(fwd.logprob, st["ref"], st["offsets"], BETA, label_smoothing=SMOOTHING)
    grad = vsl.token_logprobs_grad(st["logits"], st["tokens"], fwd, r.d_logprob, grad_dtype=kind)
    return dict(logprob=fwd.logprob, loss=r.loss, rewards=r.rewards, grad=grad)


def run(st):
    if own:
        return _own(st)
    case = st["case"]
    if case["op"] == "adapters":
        out = _plain_adapters(st)
        return dict(logits=out, stats=_tile_statistics(out)) if case["stats"] else dict(logits=out)
    if case["op"] == "policy":
        return _plain_policy(st)
    if case["op"] == "preference":
        return _plain_preference(st)
    rows = _plain_rows(st)
    out = dict(logprob=rows["lp"].float())
    if case["ent"]:
        out["entropy"] = rows["h"].float()
    if case["grad"] != "none":
        d_h = st["d_entropy"] if case["ent"] else torch.zeros_like(st["d_entropy"])
        out["grad"] = _plain_gradient(st, rows, st["d_logprob"].double(), d_h.double(), case["grad"])
    return out


# ----------------------------------------------------------------------------- what a pass cannot do without


def work(case):
    V = case["S"] * case["V_s"]
    if case["op"] == "adapters":
        R, H, rank = case["R"], case["H"], case["rank"]
        ids = _adapter_of_request(case)
        used = int(ids[ids >= 0].unique().numel())
        rows = int((ids >= 0).sum()) * case["per"]
        stats = R * case["S"] * -(-case["V_s"] // 128) * 32 if case["stats"] else 0
        return dict(bytes=8 * R * V + used * 2 * rank * (V + H) + 2 * R * H + 4 * R + stats,
                    flops=2 * rows * rank * (V + H))
    g = {"none": 0, "fp32": 4, "bf16": 2}[case["grad"]]
    if case["op"] == "preference":
        # a sequence's sum stands between the logprobs and their gradient: the rows that count are read twice.
        # Lengths run from half to the whole of `length`, one row of each does not count.
        low = max(1, case["length"] // 2)
        rows = 2 * case["pairs"] * ((low + case["length"]) / 2 - 1)
        return dict(bytes=rows * V * 8 + 2 * case["pairs"] * case["length"] * V * g, flops=10 * rows * V)
    R = case["R"]
    if case["op"] == "logprobs":
        return dict(bytes=R * V * (4 + (4 + g if g else 0)) + 8 * R, flops=(10 if g else 5) * R * V)
    on = max(1, R - R // 10)
    return dict(bytes=on * V * 4 + R * V * g + 36 * R, flops=10 * on * V)


# ----------------------------------------------------------------------------- the definitions in 64 bits


def _exact_adapters(st):
    out = [x.double() for x in st["logits"]]
    for k in range(st["case"]["n"]):
        rows = (st["ids"] == k).nonzero()[:, 0]
        u = st["scale"][k].double() * (st["hidden"][rows].double() @ st["a"][k].double().T)
        for s, b in enumerate(st["b"]):
            out[s][rows] += u @ b[k].double().T
    if not st["case"]["stats"]:
        return dict(logits=out)
    V_s, records = st["case"]["V_s"], []
    for x in out:
        for first in range(0, V_s, 128):
            block = x[:, first:first + 128]
            quarter = [block[:, q:q + 32].amax(1) if q < block.shape[1] else torch.full_like(block[:, 0], -math.inf)
                       for q in range(0, 128, 32)]
            top = block.amax(1)
            size = block.abs().masked_fill(block == 0, math.inf)
            records.append(torch.stack([*quarter, torch.logsumexp(block, 1).sub(top).exp(), block.amin(1), size.amin(1),
                                        torch.zeros_like(top)], 1))
    return dict(logits=out, stats=torch.stack(records, 1))


def _row_blocks(st):
    """(rows, their logits in 64 bits as a leaf, their tokens, which of them count) a block of rows at a time."""
    R = st["tokens"].numel()
    V = st["case"]["S"] * st["case"]["V_s"]
    step = max(1, 60_000_000 // V)
    for first in range(0, R, step):
        rows = slice(first, min(R, first + step))
        l = torch.cat([x[rows] for x in st["logits"]], 1).double().requires_grad_()
        t = st["tokens"][rows].long()
        on = (t >= 0) & (t < V)
        yield rows, l, t.clamp(0, V - 1), on


def _exact_scores(l, t, T):
    log_p = torch.log_softmax(l / T, 1)
    return log_p.gather(1, t[:, None])[:, 0], -(log_p.exp() * log_p).sum(1)


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "adapters":
        return _exact_adapters(st)
    T, parts = case["T"], []
    d_pref = None
    if case["op"] == "preference":
        with torch.no_grad():
            lp = torch.cat([torch.where(on, _exact_scores(l, t, T)[0], 0.0) for _, l, t, on in _row_blocks(st)])
        lp.requires_grad_()
        at = st["offsets"].tolist()
        s = torch.stack([(lp[i:j] - st["ref"][i:j].double()).sum() for i, j in zip(at[:-1], at[1:])]).view(-1, 2) * BETA
        h = s[:, 0] - s[:, 1]
        loss = -(1 - SMOOTHING) * torch.nn.functional.logsigmoid(h) - SMOOTHING * torch.nn.functional.logsigmoid(-h)
        d_pref, = torch.autograd.grad(loss.sum(), lp)
    for rows, l, t, on in _row_blocks(st):
        lp, ent = _exact_scores(l, t, T)
        zero = torch.zeros_like(lp)
        if case["op"] == "policy":
            w, adv = st["weights"][rows].double(), st["adv"][rows].double()
            on = on & (w != 0)
            ratio = torch.exp(lp - st["old"][rows].double())
            d = st["ref"][rows].double() - lp
            kl = torch.where(on, torch.expm1(d) - d, zero)
            surrogate = torch.minimum(ratio * adv, ratio.clamp(1 - 0.2, 1 + 0.28) * adv)
            rows_loss = torch.where(on, w * (case["kl"] * kl - surrogate - case["ent"] * ent), zero)
            got = dict(loss=rows_loss, logprob=torch.where(on, lp, zero), kl=kl, entropy=torch.where(on, ent, zero))
            objective = rows_loss.sum()
        elif case["op"] == "preference":
            got = dict(logprob=torch.where(on, lp, zero))
            objective = torch.where(on, lp * d_pref[rows], zero).sum()
        else:
            got = dict(logprob=torch.where(on, lp, zero))
            objective = torch.where(on, lp * st["d_logprob"][rows].double(), zero).sum()
            if case["ent"]:
                got["entropy"] = torch.where(on, ent, zero)
                objective = objective + torch.where(on, ent * st["d_entropy"][rows].double(), zero).sum()
        if case["grad"] != "none":
            got["grad"], = torch.autograd.grad(objective, l)
        parts.append({k: v.detach() for k, v in got.items()})
        del l, lp, ent, got, objective
    out = {k: torch.cat([p[k] for p in parts]) for k in parts[0]}
    if case["grad"] != "none":
        out["grad"] = list(out["grad"].split(case["V_s"], 1))
    if case["op"] == "preference":
        out.update(loss=loss.detach(), rewards=s.detach())
    return out
