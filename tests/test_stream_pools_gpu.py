"""A call on a stream that is not the current one allocates from that stream's pool: a block of the current stream's
could still be in use there, or be handed out again there while the call writes it (GPU)."""
import numpy as np
import pytest
import torch

import vocab_sharded_logits_b200 as vsl

pytestmark = pytest.mark.gpu


def _owner(t):
    """The stream whose pool a tensor's memory comes from."""
    at = t.data_ptr()
    for s in torch.cuda.memory_snapshot():
        if s["address"] <= at < s["address"] + s["total_size"]:
            return s["stream"]
    raise AssertionError("not the allocator's memory")


def _tensors(x):
    if isinstance(x, torch.Tensor):
        return [x]
    if isinstance(x, (list, tuple)):
        return [t for y in x for t in _tensors(y)]
    return [t for y in vars(x).values() if isinstance(y, (torch.Tensor, list, tuple)) for t in _tensors(y)]


def _same(x, y):
    return torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8))  # a NaN equals itself


def _calls(dev):
    R, H, S, V_s, n, rank = 6, 64, 2, 256, 2, 8
    g = torch.Generator(device=dev)
    g.manual_seed(1)
    rand = lambda *s: torch.randn(*s, generator=g, device=dev)  # noqa: E731
    hidden, logits = rand(R, H).bfloat16(), [rand(R, V_s) for _ in range(S)]
    w, a = [rand(V_s, H).bfloat16() for _ in range(S)], rand(n, rank, H).bfloat16()
    b = [rand(n, V_s, rank).bfloat16() for _ in range(S)]
    ids = torch.tensor([0, 1, -1, 0, 1, 1], dtype=torch.int32, device=dev)
    tok, one = torch.arange(R, dtype=torch.int32, device=dev), torch.ones(R, device=dev)
    old = -one                      # made here: a call under another stream would not wait for it
    at = torch.tensor([0, 3, R], dtype=torch.int32, device=dev)
    params = vsl.make_row_params(np.ones(R), np.full(R, 40), np.ones(R), np.arange(R), np.zeros(R), dev)
    fwd = vsl.token_logprobs(logits, tok, entropy=True)
    drafts = torch.zeros(2, 2, dtype=torch.int32, device=dev)
    torch.cuda.synchronize()
    return {
        "logits_local": lambda **k: vsl.logits_local(hidden, w, tile_stats=True, **k),
        "tile_stats": lambda **k: vsl.tile_stats(logits, **k),
        "sample": lambda **k: vsl.sample(logits, params, 3, 4, processed=True, **k),
        "verify_drafts": lambda **k: vsl.verify_drafts(tok, drafts, one, **k),
        "adapters_add": lambda **k: vsl.adapters_add(logits, hidden, a, b, ids, tile_stats=True, **k),
        "token_logprobs": lambda **k: vsl.token_logprobs(logits, tok, entropy=True, **k),
        "token_logprobs_grad": lambda **k: vsl.token_logprobs_grad(logits, tok, fwd, one, one, **k),
        "policy_loss": lambda **k: vsl.policy_loss(logits, tok, old, one, entropy_coef=0.1, **k),
        "preference_loss": lambda **k: vsl.preference_loss(one, None, at, 0.1, **k),
    }


CALLS = ["logits_local", "tile_stats", "sample", "verify_drafts", "adapters_add", "token_logprobs", "token_logprobs_grad",
         "policy_loss", "preference_loss"]


@pytest.mark.parametrize("name", CALLS)
def test_outputs_come_from_the_pool_of_the_calls_stream(cuda_device, name):
    call = _calls(cuda_device)[name]
    side = torch.cuda.Stream()
    want = _tensors(call())
    side.wait_stream(torch.cuda.current_stream())
    got = _tensors(call(stream=side))
    assert torch.cuda.current_stream() != side
    torch.cuda.synchronize()
    assert len(got) == len(want) > 0
    for x, y in zip(got, want):
        assert _owner(x) == side.cuda_stream
        assert _same(x, y)
    # the default stream, given from under another one
    with torch.cuda.stream(side):
        got = _tensors(call(stream=torch.cuda.default_stream()))
        assert torch.cuda.current_stream() == side
    torch.cuda.synchronize()
    for x, y in zip(got, want):
        assert _owner(x) == torch.cuda.default_stream().cuda_stream
        assert _same(x, y)


@pytest.mark.parametrize("name", CALLS)
def test_captured_on_the_stream_it_is_given(cuda_device, name):
    call = _calls(cuda_device)[name]
    want = _tensors(call())
    side = torch.cuda.Stream()
    call(stream=side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = _tensors(call(stream=side))
    graph.replay()
    torch.cuda.synchronize()
    assert all(_same(x, y) for x, y in zip(got, want))
