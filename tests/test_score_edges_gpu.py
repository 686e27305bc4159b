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
