"""Penalties, biases and masks against the float64 definition.

Tolerance: the operator takes a division or product, a product and two
differences and a sum in float32, each within 2^-24 of its result's size, and
one rounding to the logits' type. No intermediate passes
S = max(|x|, |x| rho, |x| / rho) + |f| c + |p| + |b|, so the float32 part is
within 5 * 2^-24 S (2^-21 S is asked), and the rounding adds half a step of the
value."""
import math

import numpy as np
import pytest

import oracle
import synth
from tests.tree_cases import layout
from tests.workloads import cuda_or_skip, host, to_dev

pytestmark = pytest.mark.gpu

HALF = {oracle.F32: 2.0 ** -24, oracle.BF16: 2.0 ** -8}


@pytest.fixture(scope="module")
def vsv():
    cuda_or_skip()
    import draft_token_verification_packed_amd as m
    m.lib()
    return m


def _case(seed, counts, V, dtype, kind="wide", pad=0, H=40, bias=6, masked=0.5, full=0, tokens=None):
    rng = np.random.default_rng(seed)
    off, owner, par = layout(rng, counts, kind)
    B, R, M = len(counts), int(off[-1]), V if tokens is None else tokens
    x = (rng.standard_normal((R, V)) * 4).astype(np.float32)
    x[rng.random((R, V)) < 0.05] = -np.inf
    x[rng.random((R, V)) < 0.05] = 0.0
    x[:, 0] = np.finfo(np.float32).min if dtype == oracle.F32 else -3.3895313892515355e38
    store = np.full((R + full, V + pad), np.nan, dtype=np.float32)
    store[:R, :V] = x
    c = dict(off=off, owner=owner, par=par, V=V, dtype=dtype, kind=kind, R=R, full=full)
    c["store"] = synth.f32_to_bf16_bits(store) if dtype == oracle.BF16 else store
    c["drafts"] = rng.integers(0, M, R + full - B).astype(np.int32)
    c["history"] = rng.integers(0, M, (B, H)).astype(np.int32)
    c["history_len"] = rng.integers(0, H + 1, B).astype(np.int32)
    c["prompt_len"] = (c["history_len"] * rng.random(B)).astype(np.int32)
    c["repetition"] = rng.choice([1.0, 1.25, 0.8, 2.0], B).astype(np.float32)
    c["frequency"] = rng.choice([0.0, 0.5, -0.3], B).astype(np.float32)
    c["presence"] = rng.choice([0.0, 0.7, -1.5], B).astype(np.float32)
    n = rng.integers(0, bias + 1, B)
    c["bias_offsets"] = np.concatenate(([0], np.cumsum(n))).astype(np.int32)
    c["bias_tokens"] = rng.integers(0, M, n.sum()).astype(np.int32)
    value = (rng.standard_normal(n.sum()) * 3).astype(np.float32)
    value[::5] = -np.inf
    c["bias_values"] = value
    allowed = rng.random((R + full, V)) < rng.choice([0.02, 0.5, 1.0, 0.0], R + full)[:, None]
    words = (V + 31) // 32
    bits = np.zeros((R + full, words * 32), dtype=np.uint8)
    bits[:, :V] = allowed
    bits[:, V:] = rng.integers(0, 2, (R + full, words * 32 - V))
    order = rng.permutation(R + full)
    c["mask"] = np.packbits(bits, axis=1, bitorder="little").view(np.int32)[order]
    index = np.argsort(order).astype(np.int32)
    index[rng.random(R + full) >= masked] = -3
    c["mask_index"], c["allowed"] = index, allowed
    return c


def _call(vsv, c, store=None, chain=False, **kw):
    d = {k: to_dev(c[k]) for k in ("history", "history_len", "prompt_len", "repetition", "frequency", "presence",
                                   "bias_offsets", "bias_tokens", "bias_values", "mask", "mask_index")}
    d.update(parents=None if chain else to_dev(c["par"] if not c["full"] else
                                               np.concatenate((c["par"], np.full(c["full"], 9, dtype=np.int32)))),
             vocab=c["V"])
    d.update(kw)
    x = to_dev(c["store"]) if store is None else store
    return vsv.adjust_logits(x, to_dev(c["off"]), to_dev(c["drafts"]), **d)


def _want(c, r, drop=()):
    i, V = int(c["owner"][r]), c["V"]
    x = oracle.row_f64(c["store"], c["dtype"], r, V)
    r0 = int(c["off"][i])
    path = oracle.path_of(c["par"][r0:c["off"][i + 1]], r - r0)
    text = c["history"][i, :c["history_len"][i]].tolist()
    prompt, output = text[:c["prompt_len"][i]], text[c["prompt_len"][i]:]
    output = output + [int(c["drafts"][r0 + j - i - 1]) for j in path[1:]]
    b = slice(c["bias_offsets"][i], c["bias_offsets"][i + 1])
    bias = list(zip(c["bias_tokens"][b].tolist(), c["bias_values"][b].astype(np.float64).tolist()))
    par = [float(c[k][i]) for k in ("repetition", "frequency", "presence")]
    allowed = c["allowed"][r] if c["mask_index"][r] >= 0 else None
    if "history" in drop:
        prompt, output = [], output[c["history_len"][i] - c["prompt_len"][i]:]
    if "bias" in drop:
        bias = []
    if "mask" in drop:
        allowed = None
    if "penalties" in drop:
        par = [1.0, 0.0, 0.0]
    y = oracle.adjust_row(x, prompt, output, *par, bias=bias, allowed=allowed)
    size = np.maximum(np.abs(x), np.maximum(np.abs(x) * par[0], np.abs(x) / par[0]))
    size = size + abs(par[1]) * np.bincount(np.asarray(output, dtype=np.int64), minlength=V) + abs(par[2])
    for t, v in dict(bias).items():
        size[t] += abs(v) if math.isfinite(v) else 0.0
    return y, size


def _check(got, c, drop=()):
    assert got.shape == (c["R"] + c["full"], c["V"])
    got = got.float().cpu().numpy().astype(np.float64)
    top = np.finfo(np.float32).max if c["dtype"] == oracle.F32 else 3.3895313892515355e38
    for r in range(c["R"]):
        y, size = _want(c, r, drop)
        tol = 2.0 ** -21 * size + HALF[c["dtype"]] * np.abs(y)
        near = np.abs(got[r] - y) <= tol
        # the lowest value times a penalty passes the type's range
        near |= (got[r] == -np.inf) & (y < -top)
        both = np.isinf(y) & (got[r] == y)
        assert np.all(near | both), (r, np.flatnonzero(~(near | both))[:5])


BATCHES = [([1], 1), ([2, 1], 31), ([5, 3, 64], 1000), ([4] * 30, 2049), ([6, 1, 17], 8200), ([9, 30], 20011)]


@pytest.mark.parametrize("dtype", [oracle.F32, oracle.BF16])
@pytest.mark.parametrize("kind", ["chain", "wide"])
@pytest.mark.parametrize("counts,V", BATCHES)
def test_rows_match_the_definition(vsv, dtype, kind, counts, V):
    pad = V % 3
    c = _case(V, counts, V, dtype, kind, pad, tokens=max(1, V // 8))
    print("adjust %d requests V=%d dtype=%d %s" % (len(counts), V, dtype, kind), flush=True)
    got = _call(vsv, c)
    _check(got, c)
    if kind == "chain":
        assert np.array_equal(host(_call(vsv, c, chain=True).float()), host(got.float()), equal_nan=True)
    # in place: the same values, and nothing beyond the vocabulary moves
    x = to_dev(c["store"])
    same = _call(vsv, c, store=x, out=x)
    assert same.data_ptr() == x.data_ptr()
    assert np.array_equal(host(same.float()), host(got.float()), equal_nan=True)
    assert np.all(np.isnan(host(x.float())[:, V:]))


@pytest.mark.parametrize("dtype", [oracle.F32, oracle.BF16])
def test_large_batches(vsv, dtype):
    # more rows than workgroups fit the chip
    c = _case(3, [2] * 300, 16500, dtype, "wide", 1, H=90, tokens=900)
    _check(_call(vsv, c), c)


@pytest.mark.parametrize("drop", ["history", "bias", "mask", "penalties"])
def test_parts_left_out(vsv, drop):
    c = _case(8, [5, 1, 12], 3001, oracle.F32)
    kw = dict(history=dict(history=None, history_len=None, prompt_len=None),
              bias=dict(bias_offsets=None, bias_tokens=None, bias_values=None), mask=dict(mask=None, mask_index=None),
              penalties=dict(repetition=None, frequency=None, presence=None))[drop]
    _check(_call(vsv, c, **kw), c, (drop,))


def test_long_chains_and_histories(vsv):
    c = _case(9, [300, 2], 700, oracle.F32, "chain", H=5000, tokens=20)
    _check(_call(vsv, c, chain=True), c)


def test_strided_history_and_masks(vsv):
    c = _case(11, [5, 4], 500, oracle.BF16)
    wide = np.full((2, 77), -5, dtype=np.int32)
    wide[:, 3:43] = c["history"]
    mask = np.zeros((c["mask"].shape[0], 40), dtype=np.int32)
    mask[:, 5:5 + c["mask"].shape[1]] = c["mask"]
    got = _call(vsv, c, history=to_dev(wide)[:, 3:43], mask=to_dev(mask)[:, 5:5 + c["mask"].shape[1]])
    _check(got, c)
    # a wider out, misaligned against the logits
    import torch
    out = torch.full((c["R"], 507), 7.0, dtype=torch.bfloat16, device="cuda")[:, 3:]
    view = _call(vsv, c, out=out)
    _check(view, c)
    assert torch.all(out[:, 500:] == 7.0)


def test_padded_batches_leave_the_rest(vsv):
    import torch
    c = _case(12, [5, 4, 3], 900, oracle.F32, full=6)
    c["off"] = np.concatenate((c["off"], [12, 12])).astype(np.int32)     # requests without rows behind the last
    for k in ("history", "history_len", "prompt_len", "repetition", "frequency", "presence"):
        c[k] = np.concatenate((c[k], c[k][:2]))
    c["bias_offsets"] = np.concatenate((c["bias_offsets"], c["bias_offsets"][-1:], c["bias_offsets"][-1:]))
    c["drafts"] = c["drafts"][:18 - 5]
    out = torch.full((18, 900), 5.0, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    _check(_call(vsv, c, out=out, error_flag=err), c)
    assert torch.all(out[12:] == 5.0) and int(err) == 0


def test_nan_and_infinite_logits(vsv):
    x = np.array([[np.nan, np.inf, -np.inf, 1.0, np.nan, np.inf]], dtype=np.float32)
    import torch
    y = vsv.adjust_logits(to_dev(x), to_dev(np.array([0, 1], dtype=np.int32)), None,
                          history=to_dev(np.array([[0, 1, 2, 3]], dtype=np.int32)),
                          history_len=to_dev(np.array([4], dtype=np.int32)),
                          repetition=to_dev(np.array([2.0], dtype=np.float32)),
                          presence=to_dev(np.array([1.0], dtype=np.float32)),
                          mask=to_dev(np.array([[0b001111]], dtype=np.int32)))
    y = host(y)[0]
    assert np.isnan(y[0]) and y[1] == np.inf and y[2] == -np.inf and y[3] == -0.5
    assert y[4] == -np.inf and y[5] == -np.inf          # masked: whatever stood there


def test_device_conditions(vsv):
    import torch
    def flag(**kw):
        c = _case(13, [3, 2], 60, oracle.F32)
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        drafts, off = c["drafts"], c["off"]
        c["drafts"], c["off"] = kw.pop("drafts", drafts), kw.pop("off", off)
        _call(vsv, c, error_flag=err, **{k: to_dev(v) for k, v in kw.items()})
        return int(err)
    i32, f32 = (lambda *a: np.array(a, dtype=np.int32)), (lambda *a: np.array(a, dtype=np.float32))
    assert flag() == 0
    assert flag(repetition=f32(1, 0)) == vsv.FLAG_PARAMS
    assert flag(frequency=f32(np.nan, 0)) == vsv.FLAG_PARAMS
    assert flag(presence=f32(np.inf, 0)) == vsv.FLAG_PARAMS
    assert flag(bias_offsets=i32(0, 1, 2), bias_tokens=i32(3, 60), bias_values=f32(1, 1)) == vsv.FLAG_TOKEN
    assert flag(bias_offsets=i32(0, 1, 2), bias_tokens=i32(3, 4), bias_values=f32(1, np.nan)) == vsv.FLAG_PARAMS
    assert flag(bias_offsets=i32(0, 5, 2), bias_tokens=i32(3, 4), bias_values=f32(1, 1)) == vsv.FLAG_LAYOUT
    assert flag(drafts=i32(1, 99, 2)) & vsv.FLAG_TOKEN
    assert flag(off=i32(0, 4, 9)) == vsv.FLAG_LAYOUT
    assert flag(parents=i32(-1, 1, 0, -1, 0)) == vsv.FLAG_LAYOUT
    assert flag(history_len=i32(3, 41)) == vsv.FLAG_LAYOUT
    assert flag(history=np.full((2, 40), 60, dtype=np.int32), history_len=i32(3, 4), prompt_len=i32(1, 1)) == vsv.FLAG_TOKEN
    assert flag(mask_index=i32(0, 1, 5, 0, 0)) == vsv.FLAG_LAYOUT


def test_rows_beyond_32_bits(vsv):
    """The last of rows whose elements lie past 2^31 (2^32 bytes), in place."""
    import torch
    V, R = 262144, 8300
    x = torch.zeros((R, V), dtype=torch.bfloat16, device="cuda")
    x[-1] = 2.0
    off = to_dev(np.array([0, R], dtype=np.int32))
    drafts = torch.zeros(R - 1, dtype=torch.int32, device="cuda")
    drafts[-1] = V - 1
    y = vsv.adjust_logits(x, off, drafts, presence=torch.ones(1, device="cuda"), out=x)
    assert y.data_ptr() == x.data_ptr()
    want = torch.full((V,), 2.0, dtype=torch.bfloat16, device="cuda")
    want[0] = want[-1] = 1.0
    assert torch.equal(x[-1], want)
    assert torch.equal(x[0], torch.zeros_like(want))
