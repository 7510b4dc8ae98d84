"""Packed batches of trees that the tree operators' tests share."""
import numpy as np


def layout(rng, counts, kind="wide"):
    """(row offsets, owners, parents) of requests of `counts` rows; a wide
    tree's rows hang on any earlier row, a chain's on the one before."""
    off = np.concatenate(([0], np.cumsum(counts))).astype(np.int32)
    owner = np.repeat(np.arange(len(counts)), counts).astype(np.int32)
    par = [(-1 if j == 0 else j - 1 if kind == "chain" else int(rng.integers(0, j)))
           for n in counts for j in range(n)]
    return off, owner, np.array(par, dtype=np.int32)
