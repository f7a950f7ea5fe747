"""What the paged attention may be off by where the softmax weights, not the
output's own rounding, decide: sharper than the bound of kv_reference.py, which
admits a rounding of every weight."""
import torch

from kv_reference import TINY, U


def two_parts(dtype):
    """A weight cut off, which leaves less than 2 U of it; that rounded, half a step U, and its last bit set, a step 2 U."""
    return 2 * U[dtype] * (U[dtype] + 2 * U[dtype])


def attention(q, k, v, scale, dtype, weight, runs=1):
    """One head over n tokens, q [D], k and v [n, D] float64 of `dtype`'s values: (out, lse, tolerance of out).

    weight: relative error that each softmax weight may have for its product
    with v, beside its score's.  runs: how many parts of the tokens are joined."""
    D, n = q.numel(), len(k)
    z, size_z = k @ q * scale, k.abs() @ q.abs() * abs(scale)
    p = torch.softmax(z, 0)
    out = p @ v
    # a score: sums of D products, the scale, the difference to the maximum and exp2f (as in kv_reference.py)
    dz = ((D / 16 + 24) * 2.0 ** -23 * size_z + 2.0 ** -20).max()
    # fp16 weights are held in steps of 2^-24 at 2^-15 of the largest: half a step is 2^-40 of it, and the last bit is set
    floor = 3 * 2.0 ** -40 * p.max() if dtype is torch.float16 else 0.0
    # sums of 16 tokens at a time; the parts' joining
    chain = (n / 16 + 64 + runs) * 2.0 ** -23
    tol = (p * (2 * dz + weight + chain) + floor) @ v.abs() + U[dtype] * out.abs() + TINY[dtype]
    return out, torch.logsumexp(z, 0), tol
