"""Without a loadable _binding.so (another torch or Python) the package still imports: the projection, the sampler and
the verification need libvsl.so alone; the calls that do need it say so."""
import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = "vocab_sharded_logits_b200"

SCRIPT = """
import torch, vocab_sharded_logits_b200 as v
assert v.__file__.startswith({at!r})
assert v.lib.vsl_version() and v.adapters_workspace_bytes(4, 2, 8) > 0 and v.tile_stats_shape(2, 3, 200) == (2, 6, 8)
x, i, f = [torch.zeros(4, 8)], torch.zeros(4, dtype=torch.int32), torch.zeros(4)
h = torch.zeros(4, 16).bfloat16()
for call in (lambda: v.logits_local(h, [h]), lambda: v.tile_stats(x), lambda: v.sample(x, torch.zeros(4, 5, dtype=torch.int32), 0, 0),
             lambda: v.verify_drafts(i, torch.zeros(2, 1, dtype=torch.int32))):
    try:
        call()
    except ValueError as e:
        assert "CUDA" in str(e)
    else:
        raise AssertionError
fwd = v.TokenLogprobs(f, None, torch.zeros(4, 2), 1.0)
for call in (lambda: v.token_logprobs(x, i), lambda: v.token_logprobs_grad(x, i, fwd, f), lambda: v.policy_loss(x, i, f, f),
             lambda: v.preference_loss(f, None, i[:3], 0.1), lambda: v.adapters_add(x, h, h[None], [h[None]], i)):
    try:
        call()
    except ImportError as e:
        assert "_binding.so" in str(e)
    else:
        raise AssertionError
print("both kinds", "of calls")
"""


@pytest.mark.parametrize("binding", ["absent", "of another build"])
def test_the_earlier_calls_need_the_library_alone(tmp_path, binding):
    at = tmp_path / PKG
    at.mkdir()
    for name in ("__init__.py", "libvsl.so"):
        shutil.copy(os.path.join(ROOT, PKG, name), at / name)
    if binding != "absent":
        (at / "_binding.so").write_bytes(b"not a shared library")
    run = subprocess.run([sys.executable, "-c", SCRIPT.format(at=str(tmp_path))], cwd=tmp_path, capture_output=True, text=True,
                         env={**os.environ, "PYTHONPATH": str(tmp_path)})
    assert run.returncode == 0 and "both kinds of calls" in run.stdout, run.stderr[-2000:]
