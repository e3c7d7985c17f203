"""How far fp32 results of a projection may be off in norm, and a plain restatement of how they are summed.

The tensor cores add 16 products at a time into fp32 and cut off what does not fit: a running sum s loses between 0 and
one unit of its last place, half of one on average, which is 0.36 * 2^-23 |s| (a unit is 2^-24 to 2^-23 of a
value, 0.72 * 2^-23 on average over its logarithm).  The running sum of m groups of products of random signs grows as the
root of their number: over its course it loses 2/3 m * 0.36 * 2^-23 of its end at most, all in one direction.  A sum ends every 512
products, m = 32, to which an adapter of rank r, in three parts, adds 3 r / 16 groups.  Sums of different runs are off
independently, so the whole is off by as much of its norm as they are.  3 * 2^-23 for the rest: the additions of the runs, the
rounding, and u's own sums, where they matter beside the 3 r / 16."""
import numpy as np


def tolerance(r):
    return 2.0 ** -23 * (0.24 * (32 + 3 * r / 16) + 3)


def off(got, ref):
    return np.linalg.norm(got - ref) / np.linalg.norm(ref)


def cut(x):
    """fp64 to fp32, towards zero."""
    y = x.astype(np.float32)
    return np.where(np.abs(y.astype(np.float64)) > np.abs(x), np.nextafter(y, np.float32(0)), y)


def bf16(x):
    """fp32 to the nearest bf16, as fp32."""
    b = np.asarray(x, np.float32).view(np.uint32).astype(np.uint64)
    return ((b + 0x7fff + ((b >> 16) & 1)) & 0xffff0000).astype(np.uint32).view(np.float32)


def products(X, W, every=512, start=None):
    """X W^T as the tensor cores add it, a new sum every `every` products; `start`: what the last sum begins with is in it."""
    total = np.zeros((X.shape[0], W.shape[0]), np.float32)
    run = np.zeros_like(total)
    for k in range(0, X.shape[1], 16):
        run = cut(run.astype(np.float64) + X[:, k:k + 16].astype(np.float64) @ W[:, k:k + 16].T.astype(np.float64))
        if (k + 16) % every == 0 or k + 16 >= X.shape[1]:
            total = total + run
            run = np.zeros_like(total)
    return total


def linear(X, W, A, B, every=512, parts=3):
    """W x + B (A x) for one adapter, in the order that include/moe.h's operator has: u is held as `parts` bf16 values."""
    y = products(X, W, every)
    left, run = products(X, A, every), np.zeros_like(y)
    split = []
    for _ in range(parts):
        split.append(bf16(left))
        left = left - split[-1]
    for k in range(0, A.shape[0], 16):
        for u in split:
            run = cut(run.astype(np.float64) + u[:, k:k + 16].astype(np.float64) @ B[:, k:k + 16].T.astype(np.float64))
    return y + run
