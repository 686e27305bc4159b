"""Slices given as an iterable that makes its tensors: they live until the call has used them."""
import weakref

import pytest
import torch

import vocab_sharded_logits_b200 as vsl


class Made:
    """Yields new tensors that nothing else holds; float() of it, which the calls take after the slices, looks whether
    they still live."""

    def __init__(self, n):
        self.n, self.refs, self.seen = n, [], []

    def __iter__(self):
        for _ in range(self.n):
            t = torch.zeros(4, 8)
            self.refs.append(weakref.ref(t))
            yield t
            del t

    def __float__(self):
        self.seen.append([r() is not None for r in self.refs])
        return 1.0


def _calls(x):
    ids, f = torch.zeros(4, dtype=torch.int32), torch.zeros(4)
    fwd = vsl.TokenLogprobs(f, None, torch.zeros(4, 2), x)
    return {
        "token_logprobs": lambda s: vsl.token_logprobs(s, ids, temperature=x),
        "token_logprobs_grad": lambda s: vsl.token_logprobs_grad(s, ids, fwd, f),
        "policy_loss": lambda s: vsl.policy_loss(s, ids, f, f, temperature=x),
    }


@pytest.mark.parametrize("name", ["token_logprobs", "token_logprobs_grad", "policy_loss"])
@pytest.mark.parametrize("as_generator", [False, True])
def test_slices_of_an_iterable_live_through_the_call(name, as_generator):
    x = Made(3)
    with pytest.raises(ValueError, match="CUDA"):               # the tensors are on the CPU: nothing is launched
        _calls(x)[name](iter(x) if as_generator else x)
    assert x.seen == [[True] * 3]
    assert [r() for r in x.refs] == [None] * 3                  # and no longer


@pytest.mark.gpu
def test_outputs_given_as_a_generator_come_back_as_a_list(cuda_device):
    g = torch.Generator(device=cuda_device)
    g.manual_seed(1)
    full = [torch.randn(4, 8, generator=g, device=cuda_device) for _ in range(2)]
    ids, one = torch.zeros(4, dtype=torch.int32, device=cuda_device), torch.ones(4, device=cuda_device)
    want = vsl.policy_loss(full, ids, -one, one)
    grad = [torch.empty_like(x) for x in full]
    got = vsl.policy_loss((x.clone() for x in full), ids, -one, one, grad=(x for x in grad))
    assert isinstance(got.grad, list) and all(x is y for x, y in zip(got.grad, grad))
    assert all(torch.equal(x, y) for x, y in zip(got.grad, want.grad)) and torch.equal(got.loss, want.loss)
    same = vsl.policy_loss(full, ids, -one, one, grad=grad)
    assert same.grad is grad
