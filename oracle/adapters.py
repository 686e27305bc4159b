"""Oracle of the low-rank adapters beside the projection: float64, row by row.

Test infrastructure only: shares no code with the CUDA path.
"""
import numpy as np


def adapters_add(logits_slices, hidden, a, b_slices, adapter_ids, scale=None):
    """out_s[r] = logits_s[r] + b_s[i] @ (scale[i] * (a[i] @ hidden[r])), i = adapter_ids[r]; a row whose id lies
    outside [0, n) keeps its logits.  Arrays: logits [R, V_s], hidden [R, H], a [n, rank, H], b [n, V_s, rank]."""
    hidden, a = np.asarray(hidden, np.float64), np.asarray(a, np.float64)
    out = [np.array(x, np.float64) for x in logits_slices]
    for r, i in enumerate(np.asarray(adapter_ids)):
        if 0 <= i < a.shape[0]:
            u = a[i] @ hidden[r] * (1.0 if scale is None else float(scale[i]))
            for x, b in zip(out, b_slices):
                x[r] += np.asarray(b[i], np.float64) @ u
    return out


def adapters_add_bound(logits_slices, hidden, a, b_slices, adapter_ids, scale=None):
    """How far a result may be off that forms the products of bf16 values exactly and sums in fp32.

    A fp32 sum of n terms formed by tensor-core steps of 16 is off by at most one truncated step (2^-23 of the
    partial sums' size) for each step and each addition inside it that is not exact: 2^-22 a step covers both.  u: 8
    chains of H / 128 steps, then 8 additions and the scale; the second product: rank / 16 steps for each of three
    bf16 terms of u (which hold its 24 bits), then the sum with the logit (half a step, 2^-24).
    """
    hidden, a = np.abs(np.asarray(hidden, np.float64)), np.abs(np.asarray(a, np.float64))
    n, rank, H = a.shape
    eps_u = (H / 128 + 10) * 2.0 ** -22
    eps_v = (3 * np.ceil(rank / 16) + 2) * 2.0 ** -22
    ref = adapters_add(logits_slices, hidden * 0, a, b_slices, adapter_ids, scale)
    bound = [np.abs(x) * 2.0 ** -24 for x in ref]
    for r, i in enumerate(np.asarray(adapter_ids)):
        if 0 <= i < n:
            u = a[i] @ hidden[r] * (1.0 if scale is None else abs(float(scale[i])))
            for x, b in zip(bound, b_slices):
                term = np.abs(np.asarray(b[i], np.float64)) @ u
                x[r] += term * (eps_u + eps_v + 2.0 ** -23)
    return bound
