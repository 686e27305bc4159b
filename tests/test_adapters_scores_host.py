"""CPU checks of the adapters' and losses' calls: what they refuse, before anything reaches a device."""
import ctypes

import pytest
import torch

import vocab_sharded_logits_b200 as v

INVALID, ALIGN, UNSUPPORTED, WORKSPACE = 1, 2, 3, 4
vp = ctypes.c_void_p
WS = v.adapters_workspace_bytes(4, 2, 8)
FAKE = 0x10000                      # never dereferenced: validation fails first


def _arr(*addr):
    return (vp * len(addr))(*addr)


def _adapters(**kw):
    a = dict(logits=_arr(0x10000), out=_arr(0x20000), hidden=FAKE, R=4, H=64, S=1, V_s=512, a=FAKE, b=_arr(0x30000),
             scale=None, n=2, rank=8, ids=FAKE, stats=None, ws=FAKE, ws_bytes=WS, stream=None)
    a.update(kw)
    return v.lib.vsl_adapters_add(*a.values())


def test_adapters_refusals():
    # 3 units (2 adapters and none) of 20 words in the plan, three terms of 16 x 16 bf16 each
    assert WS == (4 + 3 * 20) * 4 + 3 * 3 * 16 * 16 * 2
    for bad in ((0, 2, 8), (4, 0, 8), (4, 2, -1), (4, 2, 264)):
        assert v.adapters_workspace_bytes(*bad) == 0
    for name in ("logits", "out", "hidden", "a", "b", "ids", "ws"):
        assert _adapters(**{name: None}) == INVALID, name
    for name in ("R", "H", "S", "V_s", "n", "rank"):
        assert _adapters(**{name: 0}) == INVALID, name
        assert _adapters(**{name: -8}) == INVALID, name
    assert _adapters(logits=_arr(0)) == INVALID and _adapters(out=_arr(0)) == INVALID and _adapters(b=_arr(0)) == INVALID
    assert _adapters(S=17) == UNSUPPORTED
    assert _adapters(V_s=(1 << 30) + 4) == UNSUPPORTED
    assert _adapters(rank=264) == UNSUPPORTED
    assert _adapters(rank=12) == ALIGN and _adapters(H=60) == ALIGN and _adapters(V_s=510) == ALIGN
    for name in ("hidden", "a", "ws"):
        assert _adapters(**{name: 0x10008}) == ALIGN, name
    assert _adapters(logits=_arr(0x10004)) == ALIGN and _adapters(out=_arr(0x20004)) == ALIGN
    assert _adapters(b=_arr(0x30008)) == ALIGN and _adapters(stats=0x40010) == ALIGN
    assert _adapters(ws_bytes=WS - 1) == WORKSPACE
    two = dict(S=2, logits=_arr(0x10000, 0x20000), b=_arr(0x30000, 0x40000))
    assert _adapters(**two, out=_arr(0x20000, 0x50000)) == INVALID          # another slice's logits
    assert _adapters(**two, out=_arr(0x50000, 0x50000)) == INVALID          # one output twice


def _logprobs(**kw):
    a = dict(logits=_arr(0x10000), R=4, S=1, V_s=512, tokens=FAKE, T=1.0, logprob=FAKE, entropy=None, stats=None,
             stream=None)
    a.update(kw)
    return v.lib.vsl_token_logprobs(*a.values())


def _grad(**kw):
    a = dict(logits=_arr(0x10000), R=4, S=1, V_s=512, tokens=FAKE, T=1.0, stats=FAKE, entropy=None, d_lp=FAKE,
             d_ent=None, grad=_arr(0x20000), kind=0, stream=None)
    a.update(kw)
    return v.lib.vsl_token_logprobs_grad(*a.values())


SIZES = [(dict(R=0), INVALID), (dict(S=0), INVALID), (dict(V_s=0), INVALID), (dict(S=17), UNSUPPORTED),
         (dict(V_s=510), ALIGN), (dict(V_s=(1 << 30) + 4), UNSUPPORTED), (dict(logits=None), INVALID),
         (dict(logits=_arr(0)), INVALID), (dict(logits=_arr(0x10008)), ALIGN)]
BAD_T = [0.0, -1.0, float("nan"), float("inf"), 1e-7, 1e7]


@pytest.mark.parametrize("call", [_logprobs, _grad])
def test_logprob_refusals(call):
    for kw, want in SIZES:
        assert call(**kw) == want, kw
    for t in BAD_T:
        assert call(T=t) == INVALID
    assert call(tokens=None) == INVALID


def test_logprob_output_refusals():
    assert _logprobs(logprob=None) == INVALID and _logprobs(stats=0x10004) == ALIGN
    for name in ("stats", "d_lp", "grad"):
        assert _grad(**{name: None}) == INVALID, name
    assert _grad(d_ent=FAKE) == INVALID                                     # without the entropies
    assert _grad(kind=2) == INVALID and _grad(kind=-1) == INVALID
    assert _grad(grad=_arr(0)) == INVALID and _grad(grad=_arr(0x20008)) == ALIGN and _grad(stats=0x10004) == ALIGN
    assert _grad(grad=_arr(0x10000), kind=1) == INVALID                     # bf16 over the logits
    assert _grad(S=2, logits=_arr(0x10000, 0x30000), grad=_arr(0x30000, 0x40000)) == INVALID


def _policy(sizes=(), **kw):
    i = dict(tokens=FAKE, old=FAKE, adv=FAKE, ref=FAKE, w=None, lo=0.2, hi=0.2, kl=0.1, ent=0.0, T=1.0)
    o = dict(loss=FAKE, logprob=None, kl_out=None, entropy=None, grad=None, kind=0)
    s = dict(logits=_arr(0x10000), R=4, S=1, V_s=512)
    for k, x in kw.items():
        (i if k in i else o if k in o else s)[k] = x
    inputs = v._PolicyInputs(*i.values())
    outputs = v._PolicyOutputs()
    outputs.loss, outputs.grad_type = o["loss"], o["kind"]
    if o["grad"] is not None:
        outputs.grad_slices = o["grad"]
    return v.lib.vsl_policy_loss(*s.values(), ctypes.byref(inputs), ctypes.byref(outputs), None)


def test_policy_refusals():
    for kw, want in SIZES:
        assert _policy(**kw) == want, kw
    for t in BAD_T:
        assert _policy(T=t) == INVALID
    for name in ("tokens", "old", "adv", "loss"):
        assert _policy(**{name: None}) == INVALID, name
    assert _policy(ref=None) == INVALID                                     # a KL term without its reference
    for kw in (dict(lo=-0.1), dict(lo=1.1), dict(lo=float("nan")), dict(hi=-0.1), dict(hi=float("nan")),
               dict(kl=float("inf")), dict(ent=float("nan")), dict(kind=7)):
        assert _policy(**kw) == INVALID, kw
    assert _policy(grad=_arr(0x10000), kind=1) == INVALID and _policy(grad=_arr(0x20004)) == ALIGN
    assert v.lib.vsl_policy_loss(_arr(0x10000), 4, 1, 512, None, None, None) == INVALID


def test_preference_refusals():
    call = lambda **kw: v.lib.vsl_preference_loss(*{**dict(  # noqa: E731
        lp=FAKE, ref=None, at=FAKE, w=None, R=4, pairs=1, beta=0.1, e=0.0, loss=FAKE, rewards=None, d=None,
        stream=None), **kw}.values())
    for kw in (dict(lp=None), dict(at=None), dict(loss=None), dict(R=-1), dict(pairs=0), dict(pairs=-3),
               dict(beta=float("nan")), dict(beta=float("inf")), dict(e=-0.1), dict(e=1.1), dict(e=float("nan"))):
        assert call(**kw) == INVALID, kw
    assert call(pairs=0x40000000) == UNSUPPORTED


def test_binding_checks_tensors_before_the_library():
    x = [torch.zeros(4, 8)]
    ids = torch.zeros(4, dtype=torch.int32)
    f = torch.zeros(4)
    with pytest.raises(ValueError, match="CUDA"):
        v.token_logprobs(x, ids)
    with pytest.raises(ValueError, match="CUDA"):
        v.policy_loss(x, ids, f, f)
    with pytest.raises(ValueError, match="token_ids"):
        v.token_logprobs(x, ids.long())
    with pytest.raises(ValueError, match="slices"):
        v.token_logprobs([torch.zeros(8, 4).T], ids)
    with pytest.raises(ValueError, match="old_logprob"):
        v.policy_loss(x, ids, f[:3], f)
    with pytest.raises(TypeError):
        v.policy_loss(x, ids, f, f, grad_dtype=torch.float16)
    h, a, b = torch.zeros(4, 16).bfloat16(), torch.zeros(2, 8, 16).bfloat16(), [torch.zeros(2, 8, 8).bfloat16()]
    with pytest.raises(TypeError):
        v.adapters_add(x, h.float(), a, b, ids)
    with pytest.raises(ValueError, match="b_slices"):
        v.adapters_add(x, h, a, b + b, ids)
    with pytest.raises(ValueError, match="scale"):
        v.adapters_add(x, h, a, b, ids, scale=torch.ones(3))
    with pytest.raises(ValueError, match="offsets"):
        v.preference_loss(f, None, torch.zeros(4, dtype=torch.int32), 0.1)
    fwd = v.TokenLogprobs(f, None, torch.zeros(4, 2), 1.0)
    with pytest.raises(ValueError, match="entropy"):
        v.token_logprobs_grad(x, ids, fwd, f, d_entropy=f)


def test_adapters_refuse_rows_that_overflow_their_plan():
    assert v.adapters_workspace_bytes((1 << 30) + 1, 2, 8) == 0 and v.adapters_workspace_bytes(1 << 30, 300, 256) > 1 << 40
    assert _adapters(R=(1 << 30) + 1, V_s=4, ws_bytes=1 << 60) == UNSUPPORTED
