"""The row operators at the edges of what they accept, against the float64
definition. Tolerances are those derived in test_gpu_rows.py unless a test
states its own."""
import math

import numpy as np
import pytest

import oracle
from tests.row_cases import BF16, F32, rows_f64, store_rows
from tests.test_gpu_rows import _check_draws
from tests.workloads import cuda_or_skip, host, to_dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def vsv():
    cuda_or_skip()
    import draft_token_verification_packed_amd as m
    m.lib()
    return m


# ------------------------------------------------------------------- draws

@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("V", [300, 70001])
def test_draws_at_subnormal_temperatures(vsv, dtype, V):
    # bins narrower than the smallest float: only the row's largest elements
    # hold weight, or its subnormal ones where the type has any below T
    rng = np.random.default_rng(2)
    rows = []
    for kind in range(4):
        x = np.zeros(V, dtype=np.float32)
        if kind == 1:
            x[rng.random(V) < 0.7] = -1.0
        elif kind == 2:
            x[rng.random(V) < 0.7] = -0.0
        elif kind == 3:
            x -= (rng.integers(0, 40, V) * 2.0 ** -149).astype(np.float32)
        rows.append(x)
    T = np.array([1.4e-45, 1e-44, 8e-44, 1e-43, 1e-42, 1e-40], dtype=np.float32)
    n = len(rows) * len(T)
    store = store_rows([rows[r % 4] for r in range(n)], dtype)
    a = (np.repeat(T, 4), np.full(n, 0, dtype=np.int32), np.where(np.arange(n) % 2, 0.9, 1.0).astype(np.float32),
         np.where(np.arange(n) % 3, 0.0, 0.05).astype(np.float32), rng.random(n, dtype=np.float32))
    print("subnormal temperatures V=%d dtype=%d" % (V, dtype), flush=True)
    _check_draws(vsv.sample_rows(to_dev(store), *[to_dev(q) for q in a]), rows_f64(store, dtype, V, 0), *a)
