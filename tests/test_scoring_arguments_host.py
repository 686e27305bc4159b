"""Arguments of the scoring calls that raise while they are looked at: the caller sees that error, not another."""
import pytest
import torch

import vocab_sharded_logits_b200 as vsl


class Undecided:
    def __bool__(self):
        raise KeyError("undecided")


def test_an_entropy_flag_without_a_truth_value():
    with pytest.raises(KeyError, match="undecided"):
        vsl.token_logprobs([torch.zeros(4, 8)], torch.zeros(4, dtype=torch.int32), entropy=Undecided())
