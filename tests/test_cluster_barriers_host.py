"""A CTA may touch another CTA's shared memory only once a cluster barrier has shown that the other has started: in
every kernel the first remote access stands behind one, and nothing leaves between a barrier's two halves."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "vocab_sharded_logits_b200", "csrc")
REMOTE = re.compile(r"\b(?:send_part|cluster_ptr|mapa|\w+_dsmem_\w+)\s*(?:<[^;()]*>)?\(")
BARRIER = re.compile(r"\bcluster_(?:wait|sync)\(\)")


def _kernels():
    for name in sorted(os.listdir(CSRC)):
        if not name.endswith((".cu", ".cuh")):
            continue
        with open(os.path.join(CSRC, name)) as f:
            text = re.sub(r"//[^\n]*", "", f.read())
        for k in re.finditer(r"__global__", text):
            at = text.index("{", k.end())
            depth, end = 1, at + 1
            while depth:
                depth += {"{": 1, "}": -1}.get(text[end], 0)
                end += 1
            title = re.findall(r"\b(\w+_kernel)\(", text[k.end():at])
            yield f"{name}:{title[-1] if title else k.start()}", text[at:end]


KERNELS = dict(_kernels())


@pytest.mark.parametrize("name", KERNELS)
def test_remote_accesses_stand_behind_a_cluster_barrier(name):
    body = KERNELS[name]
    remote = REMOTE.search(body)
    if remote:
        barrier = BARRIER.search(body)
        assert barrier and barrier.start() < remote.start(), f"{name}: {remote.group()} before any cluster barrier"


@pytest.mark.parametrize("name", KERNELS)
def test_every_arrival_has_its_wait(name):
    parts = re.split(r"\bcluster_(arrive|wait)\(\)", KERNELS[name])
    halves = parts[1::2]
    assert halves == ["arrive", "wait"] * (len(halves) // 2)
    for between in parts[2::4]:
        assert not re.search(r"\breturn\b", between), f"{name}: leaves between the barrier's halves"


def test_the_kernels_that_exchange_sums_are_among_them():
    found = {n.split(":")[1] for n, body in KERNELS.items() if REMOTE.search(body)}
    assert {"token_logprobs_kernel", "policy_loss_kernel", "adapters_shrink_kernel"} <= found
