"""Rows of logits the row operators' tests share: values, masks, alignment."""
import numpy as np

import oracle
import synth

F32, BF16 = oracle.F32, oracle.BF16
LOWEST = {F32: np.float32(np.finfo(np.float32).min), BF16: np.float32(-3.3895313892515355e38)}

KINDS = ("plain", "ties", "masked", "lowest", "one_left", "equal", "wide", "spikes")


def row_values(rng, kind, V, dtype, sigma=2.5):
    x = (rng.standard_normal(V) * sigma).astype(np.float32)
    if kind == "ties":                       # a handful of distinct values
        x = np.round(x).astype(np.float32)
    elif kind == "masked":                   # about half the row at -inf
        x[rng.random(V) < 0.5] = -np.inf
        x[rng.integers(V)] = 1.0
    elif kind == "lowest":                   # a mask of the type's lowest value
        x[rng.random(V) < 0.5] = LOWEST[dtype]
        x[rng.integers(V)] = 1.0
    elif kind == "one_left":
        x[:] = -np.inf
        x[rng.integers(V)] = -3.0
    elif kind == "equal":
        x[:] = 0.75
    elif kind == "wide":                     # far beyond any temperature's reach
        x *= np.float32(40.0)
    elif kind == "spikes":
        x[rng.integers(V, size=max(1, V // 200))] += 15.0
    return x


def store_rows(rows, dtype, pad=0, shift=0):
    """[n, shift + V + pad] storage, NaN outside the rows."""
    n, V = len(rows), rows[0].shape[0]
    a = np.full((n, shift + V + pad), np.nan, dtype=np.float32)
    for r, x in enumerate(rows):
        a[r, shift:shift + V] = x
    return synth.f32_to_bf16_bits(a) if dtype == BF16 else a


def rows_f64(store, dtype, V, shift):
    return [oracle.row_f64(store[:, shift:], dtype, r, V) for r in range(store.shape[0])]


def largest(x, T):
    """Largest |x| / T over the finite logits that hold any weight."""
    f = x[np.isfinite(x)]
    f = f[f > f.max() - 800.0 * T]
    return float(np.abs(f).max()) / T
