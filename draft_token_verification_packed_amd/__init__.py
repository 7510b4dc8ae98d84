"""Packed draft-token verification on MI355X: Python binding of libvspec_verify.

Argument marshalling only. Every step of verification runs in the HIP
kernels of `libvspec_verify.so` (built in-tree by `build.py`); PyTorch is used
for device memory and the current stream. There is no CPU fallback: if the
library is missing or cannot be loaded, every call raises.

Entry points mirror the C ABI in include/vspec_verify.h:
    verify_greedy(logits, row_offsets, row_owner, draft_tokens, relaxed_topk=1)
    verify_greedy_relaxed(logits, row_offsets, row_owner, draft_tokens, topk=1, margin=0.0,
                          from_position=0, after_tokens=0, generated=None, protected_ids=None)
    verify_greedy_static(logits, row_offsets, row_owner, draft_tokens, relaxed_topk=1)
    verify_greedy_tree(logits, row_offsets, row_owner, draft_tokens, parents)
    verify_sampled(logits, row_offsets, row_owner, draft_tokens,
                   temperature, top_k, top_p, min_p, seed, offset=0)
    draft_confidence(draft_logits, selected=None)
    sample_rows(logits, temperature, top_k, top_p, min_p, uniforms)
    top_logits(logits, k, temperature=1.0)
    distill_loss(student_logits, teacher_ids, teacher_logits, teacher_lse=None, temperature=1.0)   (autograd)
    distill_loss_grad(student_logits, teacher_ids, teacher_logits, row_weight=None, teacher_lse=None, temperature=1.0)
    distill_forward / distill_backward: the two halves of distill_loss
    allocate_verify(confidence, draft_tokens, num_requests, num_drafts, row_budget)
    tree_attention(q, k, v, row_offsets, k_cache, v_cache, block_table, length, parents=None, scale=None)
    adjust_logits(logits, row_offsets, draft_tokens, parents=None, history=None, ...)
    plan_pages(block_table, held, length, row_offsets, free_pages, free_count, page_size, num_rows)
    Goodput(max_steps, window_size=20, update_interval=5, switch_min_gain=0.05)
        .observe(accepted_len, verify_len), .step(cost_ms, batch_size)   (host)
    goodput_select(prefix_acceptance, cost_ms, batch_size, current, switch_min_gain)
"""
import ctypes
import itertools
import os

import torch  # load torch's HIP runtime first so the library binds to it
from torch.autograd import forward_ad as _fwd

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libvspec_verify.so")

VSV_F32 = 0
VSV_BF16 = 1
FLAG_LAYOUT = 1
FLAG_TOKEN = 2
FLAG_LOGITS = 4
FLAG_PARAMS = 8
FLAG_PAGES = 32

_STATUS = {0: "VSV_OK", 1: "VSV_EINVAL", 2: "VSV_EUNSUPPORTED", 3: "VSV_EWORKSPACE", 4: "VSV_EHIP",
           5: "VSV_ELIMIT"}
VSV_ELIMIT = 5
STATIC_MAX_ROWS = 16384


class VSVError(RuntimeError):
    def __init__(self, status, msg):
        super().__init__("%s (%s): %s" % (_STATUS.get(status, status), status, msg))
        self.status = status


class Batch(ctypes.Structure):
    _fields_ = [("logits", ctypes.c_void_p), ("dtype", ctypes.c_int32), ("vocab", ctypes.c_int32),
                ("ld", ctypes.c_int64), ("num_requests", ctypes.c_int32), ("num_rows", ctypes.c_int32),
                ("row_offsets", ctypes.c_void_p), ("row_owner", ctypes.c_void_p),
                ("draft_tokens", ctypes.c_void_p)]


class Outputs(ctypes.Structure):
    _fields_ = [("accepted_len", ctypes.c_void_p), ("next_token", ctypes.c_void_p),
                ("out_offsets", ctypes.c_void_p), ("out_tokens", ctypes.c_void_p),
                ("row_token", ctypes.c_void_p), ("row_lse", ctypes.c_void_p),
                ("error_flag", ctypes.c_void_p), ("slow_rows", ctypes.c_void_p)]


class Relax(ctypes.Structure):
    _fields_ = [("topk", ctypes.c_int32), ("margin", ctypes.c_float), ("from_position", ctypes.c_int32),
                ("after_tokens", ctypes.c_int32), ("generated", ctypes.c_void_p), ("protected_ids", ctypes.c_void_p),
                ("num_protected", ctypes.c_int32)]


class Distill(ctypes.Structure):
    _fields_ = [("logits", ctypes.c_void_p), ("dtype", ctypes.c_int32), ("vocab", ctypes.c_int32),
                ("ld", ctypes.c_int64), ("num_rows", ctypes.c_int32), ("num_top", ctypes.c_int32),
                ("ids", ctypes.c_void_p), ("top", ctypes.c_void_p), ("teacher_lse", ctypes.c_void_p),
                ("temperature", ctypes.c_float)]


class Attention(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_void_p) for n in ("q", "k", "v", "k_cache", "v_cache", "out", "lse")] +
                [(n, ctypes.c_int64) for n in ("q_row", "q_head", "k_row", "k_head", "v_row", "v_head", "out_row",
                                               "out_head", "cache_page", "cache_token", "cache_head")] +
                [(n, ctypes.c_int32) for n in ("dtype", "head_dim", "num_heads", "num_kv_heads", "num_requests",
                                               "num_rows")] +
                [(n, ctypes.c_void_p) for n in ("row_offsets", "parents", "length", "block_table")] +
                [("table_ld", ctypes.c_int64), ("table_width", ctypes.c_int32), ("num_pages", ctypes.c_int32),
                 ("page_size", ctypes.c_int32), ("scale", ctypes.c_float)])


class Adjust(ctypes.Structure):
    _fields_ = [("logits", ctypes.c_void_p), ("out", ctypes.c_void_p), ("dtype", ctypes.c_int32),
                ("vocab", ctypes.c_int32), ("ld", ctypes.c_int64), ("out_ld", ctypes.c_int64),
                ("num_requests", ctypes.c_int32), ("num_rows", ctypes.c_int32), ("row_offsets", ctypes.c_void_p),
                ("draft_tokens", ctypes.c_void_p), ("parents", ctypes.c_void_p), ("history", ctypes.c_void_p),
                ("history_ld", ctypes.c_int64), ("history_width", ctypes.c_int32), ("prompt_len", ctypes.c_void_p),
                ("history_len", ctypes.c_void_p), ("repetition", ctypes.c_void_p), ("frequency", ctypes.c_void_p),
                ("presence", ctypes.c_void_p), ("bias_offsets", ctypes.c_void_p), ("bias_tokens", ctypes.c_void_p),
                ("bias_values", ctypes.c_void_p), ("num_bias", ctypes.c_int32), ("mask", ctypes.c_void_p),
                ("mask_ld", ctypes.c_int64), ("num_masks", ctypes.c_int32), ("mask_index", ctypes.c_void_p),
                ("num_drafts", ctypes.c_int32)]


MAX_PROTECTED = 256
MAX_TREE_ROWS = 64
MAX_PLAN_REQUESTS = 8192
MAX_TOP = 256
DISTILL_STATE = 5

SYMBOLS = ("vsv_workspace_bytes", "vsv_workspace_init", "vsv_verify_greedy", "vsv_verify_greedy_relaxed",
           "vsv_verify_greedy_static", "vsv_verify_greedy_tree", "vsv_tree_attention_workspace_bytes", "vsv_tree_attention",
           "vsv_adjust_logits", "vsv_plan_pages",
           "vsv_verify_sampled",
           "vsv_verify_probabilistic", "vsv_draft_confidence", "vsv_sample_workspace_bytes", "vsv_sample_rows",
           "vsv_top_workspace_bytes", "vsv_top_logits",
           "vsv_distill_workspace_bytes", "vsv_distill_forward", "vsv_distill_backward", "vsv_distill_grad",
           "vsv_allocate_verify", "vsv_goodput_init", "vsv_goodput_observe",
           "vsv_goodput_step", "vsv_goodput_select", "vsv_status_string", "vsv_test_withhold_row_word", "vsv_version")

GOODPUT_MAX_STEPS = 32
GOODPUT_MAX_WINDOW = 64


class GoodputState(ctypes.Structure):
    _fields_ = [("max_steps", ctypes.c_int32), ("window_size", ctypes.c_int32), ("update_interval", ctypes.c_int32),
                ("switch_min_gain", ctypes.c_double), ("current", ctypes.c_int32), ("since", ctypes.c_int32),
                ("filled", ctypes.c_int32), ("head", ctypes.c_int32),
                ("reached", (ctypes.c_int32 * GOODPUT_MAX_STEPS) * GOODPUT_MAX_WINDOW),
                ("accepted", (ctypes.c_int32 * GOODPUT_MAX_STEPS) * GOODPUT_MAX_WINDOW),
                ("estimate", ctypes.c_double * GOODPUT_MAX_STEPS)]

_lib = None


def lib():
    """The loaded library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError("libvspec_verify.so is not built; run "
                           "`python -m draft_token_verification_packed_amd.build`")
    L = ctypes.CDLL(LIB_PATH)
    vp, i32, i64, u64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_uint64, ctypes.c_size_t
    L.vsv_workspace_bytes.argtypes = [i32, i32, i32]
    L.vsv_workspace_bytes.restype = sz
    L.vsv_workspace_init.argtypes = [vp, sz, vp]
    L.vsv_workspace_init.restype = ctypes.c_int
    L.vsv_verify_greedy.argtypes = [ctypes.POINTER(Batch), i32, ctypes.POINTER(Outputs), vp, sz, vp]
    L.vsv_verify_greedy.restype = ctypes.c_int
    L.vsv_verify_greedy_relaxed.argtypes = [ctypes.POINTER(Batch), ctypes.POINTER(Relax), ctypes.POINTER(Outputs),
                                            vp, sz, vp]
    L.vsv_verify_greedy_relaxed.restype = ctypes.c_int
    L.vsv_verify_greedy_static.argtypes = [ctypes.POINTER(Batch), i32, ctypes.POINTER(Outputs), vp]
    L.vsv_verify_greedy_static.restype = ctypes.c_int
    L.vsv_verify_greedy_tree.argtypes = [ctypes.POINTER(Batch), vp, ctypes.POINTER(Outputs), vp, vp, sz, vp]
    L.vsv_verify_greedy_tree.restype = ctypes.c_int
    L.vsv_tree_attention_workspace_bytes.argtypes = [ctypes.POINTER(Attention)]
    L.vsv_tree_attention_workspace_bytes.restype = sz
    L.vsv_tree_attention.argtypes = [ctypes.POINTER(Attention), vp, vp, sz, vp]
    L.vsv_tree_attention.restype = ctypes.c_int
    L.vsv_adjust_logits.argtypes = [ctypes.POINTER(Adjust), vp, vp]
    L.vsv_adjust_logits.restype = ctypes.c_int
    L.vsv_plan_pages.argtypes = [vp, i64, i32, vp, vp, vp, i32, i32, vp, i32, vp, i32, vp, vp, vp, vp, vp, vp, vp]
    L.vsv_plan_pages.restype = ctypes.c_int
    L.vsv_verify_sampled.argtypes = [ctypes.POINTER(Batch), vp, vp, vp, vp, u64, u64,
                                     ctypes.POINTER(Outputs), vp, sz, vp]
    L.vsv_verify_sampled.restype = ctypes.c_int
    L.vsv_verify_probabilistic.argtypes = [ctypes.POINTER(Batch), vp, i64, vp, vp, vp, vp, vp, u64, u64,
                                           ctypes.POINTER(Outputs), vp, sz, vp]
    L.vsv_verify_probabilistic.restype = ctypes.c_int
    L.vsv_draft_confidence.argtypes = [vp, i32, i32, i64, i32, vp, vp, vp, vp, vp]
    L.vsv_draft_confidence.restype = ctypes.c_int
    L.vsv_sample_workspace_bytes.argtypes = [i32, i32, i32]
    L.vsv_sample_workspace_bytes.restype = sz
    L.vsv_sample_rows.argtypes = [vp, i32, i32, i64, i32, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    L.vsv_sample_rows.restype = ctypes.c_int
    L.vsv_top_workspace_bytes.argtypes = [i32, i32, i32, i32]
    L.vsv_top_workspace_bytes.restype = sz
    L.vsv_top_logits.argtypes = [vp, i32, i32, i64, i32, i32, ctypes.c_float, vp, vp, vp, vp, vp, sz, vp]
    L.vsv_top_logits.restype = ctypes.c_int
    dp = ctypes.POINTER(Distill)
    L.vsv_distill_workspace_bytes.argtypes = [i32, i32, i32]
    L.vsv_distill_workspace_bytes.restype = sz
    L.vsv_distill_forward.argtypes = [dp, vp, vp, vp, vp, sz, vp]
    L.vsv_distill_forward.restype = ctypes.c_int
    L.vsv_distill_backward.argtypes = [dp, vp, vp, vp, i64, vp]
    L.vsv_distill_backward.restype = ctypes.c_int
    L.vsv_distill_grad.argtypes = [dp, vp, vp, vp, i64, vp, vp, sz, vp]
    L.vsv_distill_grad.restype = ctypes.c_int
    L.vsv_allocate_verify.argtypes = [vp, vp, i32, i32, i32, vp, vp, vp, vp, vp, vp, vp]
    L.vsv_allocate_verify.restype = ctypes.c_int
    gp = ctypes.POINTER(GoodputState)
    L.vsv_goodput_init.argtypes = [gp, i32, i32, i32, ctypes.c_double]
    L.vsv_goodput_init.restype = ctypes.c_int
    L.vsv_goodput_observe.argtypes = [gp, vp, vp, i32]
    L.vsv_goodput_observe.restype = ctypes.c_int
    L.vsv_goodput_step.argtypes = [gp, vp, i32, ctypes.POINTER(i32)]
    L.vsv_goodput_step.restype = ctypes.c_int
    L.vsv_goodput_select.argtypes = [vp, vp, i32, i32, i32, ctypes.c_double]
    L.vsv_goodput_select.restype = i32
    L.vsv_status_string.argtypes = [ctypes.c_int]
    L.vsv_status_string.restype = ctypes.c_char_p
    L.vsv_test_withhold_row_word.argtypes = [i32]
    L.vsv_test_withhold_row_word.restype = ctypes.c_int
    L.vsv_version.argtypes = []
    L.vsv_version.restype = i32
    _lib = L
    return L


def _check(status):
    if status != 0:
        raise VSVError(status, lib().vsv_status_string(status).decode())


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _dtype_code(t):
    if t.dtype == torch.bfloat16:
        return VSV_BF16
    if t.dtype == torch.float32:
        return VSV_F32
    raise TypeError("logits must be bfloat16 or float32")


def _vec(t, n, dtype, name):
    if t is None or not t.is_cuda or t.dtype != dtype or t.dim() != 1 or t.numel() != n or not t.is_contiguous():
        raise ValueError("%s must be a contiguous %s CUDA vector of length %d" % (name, dtype, n))
    return t


def _logits(t, vocab):
    # the column stride only matters when a row holds more than one element
    # (torch gives tensors without elements, or of one column, any strides)
    if not t.is_cuda or t.dim() != 2 or (t.stride(1) != 1 and t.shape[1] > 1 and t.numel() > 0):
        raise ValueError("logits must be a 2-D CUDA tensor with unit column stride")
    v = t.shape[1] if vocab is None else int(vocab)
    if v > t.shape[1]:
        raise ValueError("vocab exceeds the logits width")
    return _dtype_code(t), v, t.stride(0) if t.shape[0] > 1 else max(t.shape[1], 1)


def workspace_bytes(num_requests, num_rows, sampled=False):
    return int(lib().vsv_workspace_bytes(int(num_requests), int(num_rows), int(bool(sampled))))


_ws_cache = {}


def _resolve_stream(stream, device=None):
    if stream is not None:
        return stream
    return torch.cuda.current_stream(device)


def workspace(num_requests, num_rows, sampled=False, device=None, stream=None):
    """A zeroed workspace tensor, cached per (device, stream) and grown on demand.

    The buffer is allocated and zero-filled on the stream the calls run on,
    so the fill is ordered before them and the caching allocator hands its
    memory to no other stream. Calls on one stream run in order and each
    leaves the workspace ready for the next, so the cached buffer serves
    every later call on that stream. Calls that may overlap need workspaces
    of their own (pass `ws`).
    """
    need = workspace_bytes(num_requests, num_rows, sampled)
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    s = _resolve_stream(stream, dev)
    key = (dev.index, s.cuda_stream)
    ws = _ws_cache.get(key)
    if ws is None or ws.numel() < need:
        size = max(need, 4096)
        size = (size + 3) // 4 * 4
        with torch.cuda.stream(s):
            ws = torch.empty(size, dtype=torch.uint8, device=dev)
        _check(lib().vsv_workspace_init(_ptr(ws), ws.numel(), ctypes.c_void_p(s.cuda_stream)))
        _ws_cache[key] = ws
    return ws


def _keep_alive(stream, *tensors):
    """Tell the caching allocator that `tensors` are used on `stream` when it
    is not the current stream, so their memory is not reused before the
    stream's work on them is done."""
    if stream is None or stream == torch.cuda.current_stream(stream.device):
        return
    for t in tensors:
        if t is not None and t.is_cuda:
            t.record_stream(stream)


def _prepare(logits, row_offsets, row_owner, draft_tokens, vocab, stream=None):
    dtype, V, ld = _logits(logits, vocab)
    R = logits.shape[0]
    B = row_offsets.numel() - 1
    _vec(row_offsets, B + 1, torch.int32, "row_offsets")
    _vec(row_owner, R, torch.int32, "row_owner")
    if R - B > 0:
        _vec(draft_tokens, R - B, torch.int32, "draft_tokens")
    dev = logits.device
    # outputs are allocated (and the ones with a fill are filled) on the
    # stream the call runs on, so the fills are ordered before the kernels
    with torch.cuda.stream(_resolve_stream(stream, dev)):
        out = _new_outputs(B, R, dev)
    batch = Batch(_ptr(logits), dtype, V, ld, B, R, _ptr(row_offsets), _ptr(row_owner),
                  _ptr(draft_tokens) if R - B > 0 else None)
    outs = _outputs_struct(out)
    return batch, outs, out, B, R


_OUT_KEYS = ("accepted_len", "next_token", "out_offsets", "out_tokens", "row_token", "row_lse", "error_flag",
             "slow_rows")


def _outputs_struct(out):
    return Outputs(*[_ptr(out[k]) for k in _OUT_KEYS])


def _new_outputs(B, R, dev):
    return dict(accepted_len=torch.empty(B, dtype=torch.int32, device=dev),
               next_token=torch.empty(B, dtype=torch.int32, device=dev),
               out_offsets=torch.empty(B + 1, dtype=torch.int32, device=dev),
               out_tokens=torch.full((max(R, 1),), -1, dtype=torch.int32, device=dev),
               row_token=torch.empty(R, dtype=torch.int32, device=dev),
               row_lse=torch.empty(R, dtype=torch.float32, device=dev),
               error_flag=torch.zeros(1, dtype=torch.int32, device=dev),
               slow_rows=torch.zeros(1, dtype=torch.int32, device=dev))


def verify_greedy(logits, row_offsets, row_owner, draft_tokens, relaxed_topk=1, vocab=None,
                  ws=None, stream=None):
    """Greedy verification of a packed batch; returns a dict of device tensors."""
    batch, outs, out, B, R = _prepare(logits, row_offsets, row_owner, draft_tokens, vocab, stream)
    ws = workspace(B, R, False, logits.device, stream) if ws is None else ws
    _keep_alive(stream, logits, row_offsets, row_owner, draft_tokens, ws)
    _check(lib().vsv_verify_greedy(ctypes.byref(batch), int(relaxed_topk), ctypes.byref(outs),
                                   _ptr(ws), ws.numel(), _stream(stream)))
    return out


def verify_greedy_relaxed(logits, row_offsets, row_owner, draft_tokens, topk=1, margin=0.0, from_position=0,
                          after_tokens=0, generated=None, protected_ids=None, vocab=None, ws=None, stream=None):
    """Greedy verification with relaxed acceptance (vsv_verify_greedy_relaxed):
    top-K and/or a logit margin, gated by draft position and by each
    request's generated-token count (`generated`, int32 [B] device or None),
    never relaxing a protected token (`protected_ids`, int32 device vector
    or None). Returns a dict of device tensors."""
    batch, outs, out, B, R = _prepare(logits, row_offsets, row_owner, draft_tokens, vocab, stream)
    if generated is not None:
        _vec(generated, B, torch.int32, "generated")
    nprot = 0
    if protected_ids is not None:
        nprot = protected_ids.numel()
        if nprot:
            _vec(protected_ids, nprot, torch.int32, "protected_ids")
    relax = Relax(int(topk), float(margin), int(from_position), int(after_tokens), _ptr(generated),
                  _ptr(protected_ids) if nprot else None, int(nprot))
    ws = workspace(B, R, False, logits.device, stream) if ws is None else ws
    _keep_alive(stream, logits, row_offsets, row_owner, draft_tokens, generated, protected_ids, ws)
    _check(lib().vsv_verify_greedy_relaxed(ctypes.byref(batch), ctypes.byref(relax), ctypes.byref(outs), _ptr(ws),
                                           ws.numel(), _stream(stream)))
    return out


def withhold_row_word(row):
    """Test hook (vsv_test_withhold_row_word): later row-per-workgroup verify
    launches leave row `row`'s result word unpublished, so their scan waits
    out its bounded poll and flags VSV_FLAG_STALLED; -1 turns it off."""
    _check(lib().vsv_test_withhold_row_word(int(row)))


def verify_greedy_static(logits, row_offsets, row_owner, draft_tokens, relaxed_topk=1, vocab=None, out=None,
                         stream=None):
    """Greedy verification through the entry point that allocates nothing
    (vsv_verify_greedy_static: library-owned scratch, at most STATIC_MAX_ROWS
    rows). `out`, if given, is a dict of output tensors as returned by
    verify_greedy and is written in place; otherwise outputs are allocated
    here. Returns the output dict."""
    batch, outs, res, B, R = _prepare(logits, row_offsets, row_owner, draft_tokens, vocab, stream)
    if out is not None:
        res = out
        outs = _outputs_struct(res)
    _keep_alive(stream, logits, row_offsets, row_owner, draft_tokens)
    _check(lib().vsv_verify_greedy_static(ctypes.byref(batch), int(relaxed_topk), ctypes.byref(outs),
                                          _stream(stream)))
    return res


def verify_sampled(logits, row_offsets, row_owner, draft_tokens, temperature, top_k, top_p, min_p,
                   seed, offset=0, vocab=None, ws=None, stream=None):
    """Sampled / mixed verification of a packed batch; returns a dict of device tensors."""
    batch, outs, out, B, R = _prepare(logits, row_offsets, row_owner, draft_tokens, vocab, stream)
    _vec(temperature, B, torch.float32, "temperature")
    _vec(top_k, B, torch.int32, "top_k")
    _vec(top_p, B, torch.float32, "top_p")
    _vec(min_p, B, torch.float32, "min_p")
    ws = workspace(B, R, True, logits.device, stream) if ws is None else ws
    _keep_alive(stream, logits, row_offsets, row_owner, draft_tokens, temperature, top_k, top_p, min_p, ws)
    _check(lib().vsv_verify_sampled(ctypes.byref(batch), _ptr(temperature), _ptr(top_k), _ptr(top_p),
                                    _ptr(min_p), int(seed) & (2**64 - 1), int(offset) & (2**64 - 1),
                                    ctypes.byref(outs), _ptr(ws), ws.numel(), _stream(stream)))
    return out


def verify_probabilistic(logits, row_offsets, row_owner, draft_tokens, draft_logits, temperature, top_k, top_p,
                         min_p, draft_temperature, seed, offset=0, vocab=None, ws=None, stream=None):
    """Rejection-sampling verification with probabilistic drafts; draft_logits
    holds the R - B draft rows in the draft tokens' layout. Returns a dict of
    device tensors (row_lse and slow_rows are not written)."""
    batch, outs, out, B, R = _prepare(logits, row_offsets, row_owner, draft_tokens, vocab, stream)
    for t, n in ((temperature, "temperature"), (top_p, "top_p"), (min_p, "min_p"),
                 (draft_temperature, "draft_temperature")):
        _vec(t, B, torch.float32, n)
    _vec(top_k, B, torch.int32, "top_k")
    dld = 0
    if R - B > 0:
        dtype, V, _ = _logits(logits, vocab)
        ddt, _, dld = _logits(draft_logits, vocab if vocab is not None else logits.shape[1])
        if ddt != dtype or draft_logits.shape[0] != R - B or draft_logits.shape[1] < V:
            raise ValueError("draft_logits must be [R - B, >= vocab] of the logits' dtype")
        dld = draft_logits.stride(0) if draft_logits.shape[0] > 1 else max(draft_logits.shape[1], 1)
    ws = workspace(B, R, False, logits.device, stream) if ws is None else ws
    _keep_alive(stream, logits, row_offsets, row_owner, draft_tokens, draft_logits, temperature, top_k, top_p,
                min_p, draft_temperature, ws)
    _check(lib().vsv_verify_probabilistic(ctypes.byref(batch), _ptr(draft_logits) if R - B > 0 else None, int(dld),
                                          _ptr(temperature), _ptr(top_k), _ptr(top_p), _ptr(min_p),
                                          _ptr(draft_temperature), int(seed) & (2**64 - 1),
                                          int(offset) & (2**64 - 1), ctypes.byref(outs), _ptr(ws), ws.numel(),
                                          _stream(stream)))
    return out


def draft_confidence(draft_logits, selected=None, vocab=None, stream=None):
    """(confidence, lse, error_flag) device tensors for every draft row."""
    dtype, V, ld = _logits(draft_logits, vocab)
    D = draft_logits.shape[0]
    if selected is not None:
        _vec(selected, D, torch.int32, "selected")
    dev = draft_logits.device
    with torch.cuda.stream(_resolve_stream(stream, dev)):
        conf = torch.empty(D, dtype=torch.float32, device=dev)
        lse = torch.empty(D, dtype=torch.float32, device=dev)
        flag = torch.zeros(1, dtype=torch.int32, device=dev)
    _keep_alive(stream, draft_logits, selected)
    _check(lib().vsv_draft_confidence(_ptr(draft_logits), dtype, V, ld, D, _ptr(selected), _ptr(conf),
                                      _ptr(lse), _ptr(flag), _stream(stream)))
    return conf, lse, flag


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


class _on:
    """The device of a call's tensors as the current one, and the stream its
    outputs are allocated and its kernels run on: `stream`, or the device's
    current stream. Kernels launch on the current device, so a call on
    another device's tensors switches to it."""

    __slots__ = ("device", "raw", "_swap", "other")

    def __init__(self, device, stream):
        self.device = device
        self._swap = self.other = None
        if stream is None:
            self.raw = _raw_stream(device.index)
            if device.index != torch.cuda.current_device():
                self._swap = torch.cuda.device(device)
        else:
            if stream.device != device:
                raise ValueError("the stream belongs to %s, the tensors to %s" % (stream.device, device))
            self.raw = stream.cuda_stream
            if stream != torch.cuda.current_stream(device) or device.index != torch.cuda.current_device():
                self.other = stream
                self._swap = torch.cuda.stream(stream)   # also switches the device

    def __enter__(self):
        if self._swap is not None:
            self._swap.__enter__()
        return self.raw

    def __exit__(self, *exc):
        if self._swap is not None:
            self._swap.__exit__(*exc)
        return False

    def keep(self, *tensors):
        if self.other is not None:
            for t in tensors:
                if t is not None:
                    t.record_stream(self.other)


def _at(t):
    return None if t is None else t.data_ptr()


def _same_device(device, *tensors):
    for t in tensors:
        if t is not None and t.device != device:
            raise ValueError("a tensor is on %s, the logits on %s" % (t.device, device))


_flag_words = {}
_FLAG_BLOCK = 1024


def _new_flag(device, raw_stream):
    """A zeroed int32 [1] error word of its own: cut from a block that is
    zero-filled on the call's stream once in a thousand calls, or filled by
    the call itself where it is captured (so that a replay starts from 0)."""
    if torch.cuda.is_current_stream_capturing():
        return torch.zeros(1, dtype=torch.int32, device=device)
    key = (device.index, raw_stream)
    block, count = _flag_words.get(key, (None, None))
    i = next(count) if block is not None else _FLAG_BLOCK
    if i >= _FLAG_BLOCK:
        with torch.inference_mode(False):   # later calls may not be in the mode of this one
            block, count = torch.zeros(_FLAG_BLOCK, dtype=torch.int32, device=device), itertools.count()
        i = next(count)
        _flag_words[key] = (block, count)
    return block[i:i + 1]


def _flag(error_flag, device):
    """The caller's sticky error word, if given."""
    if error_flag is not None:
        _vec(error_flag, 1, torch.int32, "error_flag")
        _same_device(device, error_flag)
    return error_flag


def sample_rows(logits, temperature, top_k, top_p, min_p, uniforms, vocab=None, stream=None):
    """One token per row of logits, drawn at the given numbers (vsv_sample_rows).

    `temperature` (0: arg-max), `top_p`, `min_p` and `uniforms` (in [0, 1))
    are float32 vectors with one value per row, `top_k` an int32 one. Returns
    a dict of device vectors: token, logprob (under the filtered law the
    token was drawn from), lse (of the row over its temperature) and
    error_flag."""
    dtype, V, ld = _logits(logits, vocab)
    R, dev = logits.shape[0], logits.device
    for t, n in ((temperature, "temperature"), (top_p, "top_p"), (min_p, "min_p"), (uniforms, "uniforms")):
        _vec(t, R, torch.float32, n)
    _vec(top_k, R, torch.int32, "top_k")
    _same_device(dev, temperature, top_k, top_p, min_p, uniforms)
    on = _on(dev, stream)
    with on as s:
        out = dict(token=torch.empty(R, dtype=torch.int32, device=dev),
                   logprob=torch.empty(R, dtype=torch.float32, device=dev),
                   lse=torch.empty(R, dtype=torch.float32, device=dev),
                   error_flag=_new_flag(dev, s))
        n = lib().vsv_sample_workspace_bytes(R, V, dtype)
        ws = torch.empty(n, dtype=torch.uint8, device=dev) if n else None
        on.keep(logits, temperature, top_k, top_p, min_p, uniforms)
        _check(lib().vsv_sample_rows(_at(logits), dtype, V, ld, R, _at(temperature), _at(top_k), _at(top_p),
                                     _at(min_p), _at(uniforms), _at(out["token"]), _at(out["logprob"]),
                                     _at(out["lse"]), _at(out["error_flag"]), _at(ws), n, s))
    return out


def top_logits(logits, k, temperature=1.0, vocab=None, stream=None):
    """The k first logits of every row (value descending, lowest token first;
    vsv_top_logits). Returns a dict of device tensors: values [R, k] float32,
    ids [R, k] int32, lse [R] of the rows over `temperature`, error_flag.
    values, ids and lse are what distill_loss takes of a teacher."""
    dtype, V, ld = _logits(logits, vocab)
    R, dev, k = logits.shape[0], logits.device, int(k)
    if not 1 <= k <= min(V, MAX_TOP):
        raise ValueError("k must lie in 1 .. min(vocab, %d)" % MAX_TOP)
    on = _on(dev, stream)
    with on as s:
        out = dict(values=torch.empty((R, k), dtype=torch.float32, device=dev),
                   ids=torch.empty((R, k), dtype=torch.int32, device=dev),
                   lse=torch.empty(R, dtype=torch.float32, device=dev),
                   error_flag=_new_flag(dev, s))
        n = lib().vsv_top_workspace_bytes(R, V, dtype, k)
        ws = torch.empty(n, dtype=torch.uint8, device=dev) if n else None
        on.keep(logits)
        _check(lib().vsv_top_logits(_at(logits), dtype, V, ld, R, k, float(temperature), _at(out["values"]),
                                    _at(out["ids"]), _at(out["lse"]), _at(out["error_flag"]), _at(ws), n, s))
    return out


def _distill_args(student_logits, teacher_ids, teacher_logits, teacher_lse, temperature):
    dtype, V, ld = _logits(student_logits, None)
    N, dev = student_logits.shape[0], student_logits.device
    if teacher_ids.dim() != 2 or teacher_ids.shape[0] != N or not 1 <= teacher_ids.shape[1] <= MAX_TOP:
        raise ValueError("teacher_ids must be [rows, 1 .. %d]" % MAX_TOP)
    K = teacher_ids.shape[1]
    for t, dt, n in ((teacher_ids, torch.int32, "teacher_ids"), (teacher_logits, torch.float32, "teacher_logits")):
        if not t.is_cuda or t.dtype != dt or t.shape != (N, K) or not t.is_contiguous():
            raise ValueError("%s must be a contiguous %s CUDA matrix [%d, %d]" % (n, dt, N, K))
    if teacher_lse is not None:
        _vec(teacher_lse, N, torch.float32, "teacher_lse")
    _same_device(dev, teacher_ids, teacher_logits, teacher_lse)
    return Distill(_at(student_logits), dtype, V, ld, N, K, _at(teacher_ids), _at(teacher_logits),
                   _at(teacher_lse), float(temperature))


def _distill_scratch(d, dev):
    n = int(lib().vsv_distill_workspace_bytes(d.num_rows, d.vocab, d.dtype))
    return torch.empty(n // 8, dtype=torch.float64, device=dev) if n else None, n


def _row_weight(row_weight, d, dev):
    if row_weight is not None:
        _vec(row_weight, d.num_rows, torch.float32, "row_weight")
        _same_device(dev, row_weight)
    return row_weight


def _distill_losses(student_logits, teacher_ids, teacher_logits, teacher_lse, temperature, error_flag, stream,
                    with_state):
    d = _distill_args(student_logits, teacher_ids, teacher_logits, teacher_lse, temperature)
    dev = student_logits.device
    _flag(error_flag, dev)
    on = _on(dev, stream)
    with on as s:
        loss = torch.empty(d.num_rows, dtype=torch.float32, device=dev)
        state = torch.empty((d.num_rows, DISTILL_STATE), dtype=torch.float64, device=dev) if with_state else None
        ws, n = _distill_scratch(d, dev)
        on.keep(student_logits, teacher_ids, teacher_logits, teacher_lse, error_flag)
        _check(lib().vsv_distill_forward(ctypes.byref(d), _at(loss), _at(state), _at(error_flag), _at(ws), n, s))
    return loss, state


def distill_forward(student_logits, teacher_ids, teacher_logits, teacher_lse=None, temperature=1.0, error_flag=None,
                    stream=None):
    """(loss [N] float32, state [N, DISTILL_STATE] float64) of every student row
    (vsv_distill_forward); `state` is what distill_backward takes. Device
    conditions set bits in `error_flag` (int32 [1]) if given."""
    return _distill_losses(student_logits, teacher_ids, teacher_logits, teacher_lse, temperature, error_flag, stream,
                           True)


def distill_backward(row_weight, student_logits, teacher_ids, teacher_logits, state, teacher_lse=None,
                     temperature=1.0, stream=None):
    """Gradient [N, V] of sum(row_weight * loss) in the student's logits, in
    their type (vsv_distill_backward)."""
    d = _distill_args(student_logits, teacher_ids, teacher_logits, teacher_lse, temperature)
    dev = student_logits.device
    _row_weight(row_weight, d, dev)
    if (state.dtype != torch.float64 or state.shape != (d.num_rows, DISTILL_STATE) or not state.is_contiguous() or
            state.device != dev):
        raise ValueError("state must be the one distill_forward returned for these rows")
    on = _on(dev, stream)
    with on as s:
        grad = torch.empty((d.num_rows, d.vocab), dtype=student_logits.dtype, device=dev)
        on.keep(row_weight, student_logits, teacher_ids, teacher_logits, teacher_lse, state)
        _check(lib().vsv_distill_backward(ctypes.byref(d), _at(state), _at(row_weight), _at(grad), d.vocab, s))
    return grad


def distill_loss_grad(student_logits, teacher_ids, teacher_logits, row_weight=None, teacher_lse=None,
                      temperature=1.0, error_flag=None, stream=None):
    """(loss [N], gradient [N, V] of sum(row_weight * loss)) in one call
    (vsv_distill_grad); row_weight None counts 1 for every row."""
    d = _distill_args(student_logits, teacher_ids, teacher_logits, teacher_lse, temperature)
    dev = student_logits.device
    _row_weight(row_weight, d, dev)
    _flag(error_flag, dev)
    on = _on(dev, stream)
    with on as s:
        loss = torch.empty(d.num_rows, dtype=torch.float32, device=dev)
        grad = torch.empty((d.num_rows, d.vocab), dtype=student_logits.dtype, device=dev)
        ws, n = _distill_scratch(d, dev)
        on.keep(student_logits, teacher_ids, teacher_logits, teacher_lse, row_weight, error_flag)
        _check(lib().vsv_distill_grad(ctypes.byref(d), _at(row_weight), _at(loss), _at(grad), d.vocab,
                                      _at(error_flag), _at(ws), n, s))
    return loss, grad


class _DistillLoss(torch.autograd.Function):
    @staticmethod
    def forward(ctx, student, ids, top, lse, temperature, error_flag):
        loss, state = distill_forward(student, ids, top, lse, temperature, error_flag)
        ctx.save_for_backward(student, ids, top, lse, state)
        ctx.temperature = temperature
        return loss

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, g):
        student, ids, top, lse, state = ctx.saved_tensors
        # a summed loss hands down one number for every row
        grad = distill_backward(g.contiguous(), student, ids, top, state, lse, ctx.temperature)
        return grad, None, None, None, None, None


def distill_loss(student_logits, teacher_ids, teacher_logits, teacher_lse=None, temperature=1.0, vocab=None,
                 error_flag=None):
    """Distillation loss of every student row [N, V] (bfloat16 or float32)
    against a teacher's top logits, differentiable in the student's logits.

    `teacher_ids` (int32) and `teacher_logits` (float32) are [N, K], K at most
    MAX_TOP, as top_logits returns them; a negative id marks an unused entry,
    and a row without any has loss 0 and gradient 0. Without `teacher_lse` the
    teacher is renormalised over its entries; with it (the teacher's
    log-sum-exp at the same temperature) the rest of its mass is set against
    the student's mass outside the row's ids. Losses are float32 [N]; runs on
    the current stream, its backward on the same one. The teacher gets no
    gradient, and a student that carries a forward-mode tangent is refused.
    Columns at or beyond `vocab` are not part of the rows. A step
    captured into a graph needs leaves of its own (made for the capture, or
    without a live eager graph), as any torch backward pass does."""
    if _fwd.unpack_dual(student_logits).tangent is not None:
        raise NotImplementedError("distill_loss has no forward-mode derivative")
    if vocab is not None and int(vocab) != student_logits.shape[1]:
        if not 1 <= int(vocab) <= student_logits.shape[1]:
            raise ValueError("vocab exceeds the logits width")
        student_logits = student_logits[:, :int(vocab)]
    if student_logits.dim() == 2 and student_logits.shape[0] > 1 and student_logits.stride(0) < student_logits.shape[1]:
        student_logits = student_logits.contiguous()   # one row standing for several
    if not (student_logits.requires_grad and torch.is_grad_enabled()):
        return _distill_losses(student_logits, teacher_ids, teacher_logits, teacher_lse, temperature, error_flag, None,
                               False)[0]
    return _DistillLoss.apply(student_logits, teacher_ids, teacher_logits, teacher_lse, float(temperature), error_flag)


def _in(t, n, dtype, device, name):
    """Address of an input vector (None: 0), checked like _vec and to lie on `device`."""
    if t is None:
        return None
    if t.dtype is not dtype or t.device != device or t.dim() != 1 or t.numel() != n or not t.is_contiguous():
        _vec(t, n, dtype, name)
        _same_device(device, t)
    return t.data_ptr()


def _no_gradient(name, *tensors):
    """Refuses tensors that ask for a derivative (None: not given)."""
    # (tangents live inside a dual level alone: the look at every tensor costs
    # 3 us of a call's 14 to 20)
    backward, forward = torch.is_grad_enabled(), getattr(_fwd, "_current_level", 0) >= 0
    if backward or forward:
        for t in tensors:
            if t is not None and ((backward and t.requires_grad) or (forward and _fwd.unpack_dual(t).tangent is not None)):
                raise NotImplementedError("%s has no derivative" % name)


def _cuda(t, name):
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    return t.device


def _matrix(t, rows, width, device, name):
    """(address, row stride) of an int32 matrix of unit column stride."""
    if (t.dtype is not torch.int32 or t.device != device or t.dim() != 2 or t.shape[0] != rows or t.shape[1] < width or
            (t.shape[1] > 1 and t.stride(1) != 1)):
        raise ValueError("%s must be an int32 matrix [%d, >= %d] on %s with unit column stride" %
                         (name, rows, width, device))
    return t.data_ptr(), t.stride(0) if rows > 1 else max(t.shape[1], 1)


def verify_greedy_tree(logits, row_offsets, row_owner, draft_tokens, parents, vocab=None, ws=None, stream=None):
    """Greedy verification of trees of drafts (vsv_verify_greedy_tree).

    `parents` (int32 [R], a row's parent counted from its request's first
    row; the roots' entries are not read) or None for chains. At most
    MAX_TREE_ROWS rows a request. Returns verify_greedy's dict (without
    slow_rows) with out_rows [R]: the rows of every accepted path at
    out_offsets, -1 behind them."""
    dev = _cuda(logits, "logits")
    dtype, V, ld = _logits(logits, vocab)
    R, B, i32 = logits.shape[0], row_offsets.numel() - 1, torch.int32
    if B < 0:
        raise ValueError("row_offsets must be a vector of B + 1")
    batch = Batch(logits.data_ptr(), dtype, V, ld, B, R, _in(row_offsets, B + 1, i32, dev, "row_offsets"),
                  _in(row_owner, R, i32, dev, "row_owner"),
                  _in(draft_tokens, R - B, i32, dev, "draft_tokens") if R > B else None)
    par = _in(parents, R, i32, dev, "parents")
    on = _on(dev, stream)
    with on as s:
        if ws is None and torch.cuda.is_current_stream_capturing():
            # a graph's own, so that it shares none with another one
            ws = torch.empty(lib().vsv_workspace_bytes(B, R, 0), dtype=torch.uint8, device=dev)
            _check(lib().vsv_workspace_init(ws.data_ptr(), ws.numel(), s))
        elif ws is None:
            ws = _ws_cache.get((dev.index, s))
            if ws is None or ws.numel() < lib().vsv_workspace_bytes(B, R, 0):
                ws = workspace(B, R, False, dev, on.other if on.other is not None else torch.cuda.current_stream(dev))
        words = torch.empty(3 * B + 1 + 4 * R, dtype=i32, device=dev)
        acc, nxt, offs, toks, rows, tok, lse = torch.split_with_sizes(words, (B, B, B + 1, R, R, R, R))
        flag = _new_flag(dev, s)
        base = words.data_ptr()
        r0 = base + 4 * (3 * B + 1)
        outs = Outputs(base, base + 4 * B, base + 8 * B, r0, r0 + 8 * R, r0 + 12 * R, flag.data_ptr(), None)
        on.keep(logits, row_offsets, row_owner, draft_tokens, parents, ws)
        _check(lib().vsv_verify_greedy_tree(ctypes.byref(batch), par, ctypes.byref(outs), r0 + 4 * R, ws.data_ptr(),
                                            ws.numel(), s))
    return dict(accepted_len=acc, next_token=nxt, out_offsets=offs, out_tokens=toks, out_rows=rows, row_token=tok,
                row_lse=lse.view(torch.float32), error_flag=flag)


def _heads(t, shape, dtype, device, name):
    """Strides of a tensor of `shape` with unit last stride (0 for a
    dimension of one, whose stride torch leaves open)."""
    st = t.stride()
    if t.dtype is not dtype or t.device != device or t.shape != shape or (st[-1] != 1 and t.numel()):
        raise ValueError("%s must be a %s tensor %s on %s with unit last stride" % (name, dtype, list(shape), device))
    return st if 1 not in shape else [s if n > 1 else 0 for s, n in zip(st, shape)]


def tree_attention(q, k, v, row_offsets, k_cache, v_cache, block_table, length, parents=None, scale=None, out=None,
                   return_lse=False, error_flag=None, stream=None):
    """Attention of packed draft rows over a paged cache (vsv_tree_attention).

    `q` [R, H, D], and the rows' own `k` and `v` [R, KV, D], may be slices of
    one projection; `k_cache` and `v_cache` [pages, page_size, KV, D] have the
    same strides. Row r of request i sees length[i] cached tokens (pages
    block_table[i]), the rows on its path from the root (`parents` as in
    verify_greedy_tree, None: chains) and itself. All matrices are bfloat16 or
    all float32, D is 64, 128 or (bfloat16) 256, and pointers and strides are
    multiples of 16 bytes. `scale` is D ** -0.5 by default. Returns out
    [R, H, D] (`out` if given, which shares no memory with the inputs), and
    with return_lse also the scores' log-sum-exp [R, H]. Rows of no request,
    and of requests whose offsets or lengths make no sense, are left as they
    are in a given `out` and hold nothing of meaning in a new one. Device
    conditions set bits in `error_flag` (int32 [1]) if given: FLAG_LAYOUT for
    offsets, lengths or parents, FLAG_PAGES for a page that the caches do not
    have. Tensors that ask for
    a derivative, backward or forward, are refused."""
    _no_gradient("tree_attention", q, k, v, k_cache, v_cache, out)
    if q.dim() != 3 or k.dim() != 3 or k_cache.dim() != 4:
        raise ValueError("q and k must be [rows, heads, dim], the caches [pages, page_size, heads, dim]")
    dtype, dev, i32 = _dtype_code(q), _cuda(q, "q"), torch.int32
    R, H, D = q.shape
    KV, (pages, page) = k.shape[1], k_cache.shape[:2]
    B, W = row_offsets.numel() - 1, block_table.shape[-1]
    qs, ks, vs = (_heads(t, s, q.dtype, dev, n) for t, s, n in ((q, (R, H, D), "q"), (k, (R, KV, D), "k"), (v, (R, KV, D), "v")))
    cs = _heads(k_cache, (pages, page, KV, D), q.dtype, dev, "k_cache")
    if _heads(v_cache, (pages, page, KV, D), q.dtype, dev, "v_cache") != cs:
        raise ValueError("k_cache and v_cache must have the same strides")
    off = _in(row_offsets, B + 1, i32, dev, "row_offsets")
    lens = _in(length, B, i32, dev, "length")
    par = _in(parents, R, i32, dev, "parents")
    err = _in(error_flag, 1, i32, dev, "error_flag")
    table, table_ld = _matrix(block_table, B, 0, dev, "block_table")
    if out is not None:
        os_ = _heads(out, (R, H, D), q.dtype, dev, "out")
    on = _on(dev, stream)
    with on as s:
        if out is None:
            out = torch.empty((R, H, D), dtype=q.dtype, device=dev)
            os_ = (H * D if R > 1 else 0, D if H > 1 else 0)
        lse = torch.empty((R, H), dtype=torch.float32, device=dev) if return_lse else None
        a = Attention(q.data_ptr(), k.data_ptr(), v.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), out.data_ptr(),
                      _at(lse), qs[0], qs[1], ks[0], ks[1], vs[0], vs[1], os_[0], os_[1], cs[0], cs[1], cs[2],
                      dtype, D, H, KV, B, R, off, par, lens, table, table_ld, W, pages, page,
                      D ** -0.5 if scale is None else float(scale))
        ref = ctypes.byref(a)
        n = lib().vsv_tree_attention_workspace_bytes(ref)
        ws = torch.empty(n, dtype=torch.uint8, device=dev) if n else None
        on.keep(q, k, v, row_offsets, k_cache, v_cache, block_table, length, parents, out, error_flag)
        _check(lib().vsv_tree_attention(ref, err, _at(ws), n, s))
    return (out, lse) if return_lse else out


def adjust_logits(logits, row_offsets, draft_tokens, parents=None, history=None, history_len=None, prompt_len=None,
                  repetition=None, frequency=None, presence=None, bias_offsets=None, bias_tokens=None,
                  bias_values=None, mask=None, mask_index=None, vocab=None, out=None, error_flag=None, stream=None):
    """Penalties, biases and grammar masks on packed rows of logits
    (vsv_adjust_logits); returns the adjusted rows [R, vocab] in the logits'
    type.

    Row r of request i stands behind the drafts before it (with `parents`:
    behind those on its path from the root). Requests without rows come last;
    `draft_tokens` then holds one draft less than there are rows for every
    request that has some. `history` [B, H] int32 holds each
    request's prompt and output, `prompt_len` and `history_len` [B] how many
    tokens of it are the prompt's and how many there are; `repetition`,
    `frequency` and `presence` are float32 [B]. Biases are lists of tokens and
    values, request i's at bias_offsets[i] .. bias_offsets[i + 1]. `mask`
    [M, (vocab + 31) // 32] int32 allows token v where bit v % 32 of word
    v // 32 is set, and `mask_index` [R] names each row's (negative: none;
    None: row r has mask r). `out` may be a matrix like the logits or the logits
    themselves, of which only the touched elements then move. Rows of no
    request, and of requests whose offsets make no sense, are left as they are
    in a given `out` and hold nothing of meaning in a new one. Device
    conditions set bits in `error_flag` (int32 [1]) if given: FLAG_LAYOUT,
    FLAG_TOKEN and FLAG_PARAMS. Tensors that ask for a derivative,
    backward or forward, are refused."""
    _no_gradient("adjust_logits", logits, repetition, frequency, presence, bias_values, out)
    dtype, V, ld = _logits(logits, vocab)
    R, dev, i32, f32 = logits.shape[0], logits.device, torch.int32, torch.float32
    B = row_offsets.numel() - 1
    off = _in(row_offsets, B + 1, i32, dev, "row_offsets")
    # (requests without rows leave more drafts than R - B)
    D = 0 if draft_tokens is None else draft_tokens.numel()
    if D < R - B or (D > R > B):
        raise ValueError("draft_tokens: %d entries, between %d and %d rows carry drafts" % (D, max(R - B, 0), R))
    drafts = _in(draft_tokens, D, i32, dev, "draft_tokens") if D else None
    D = min(D, R)
    par = _in(parents, R, i32, dev, "parents")
    hist, hist_ld, width, prompt, used = None, 0, 0, None, None
    if history is not None:
        if history_len is None:
            raise ValueError("history needs history_len")
        hist, hist_ld = _matrix(history, B, 0, dev, "history")
        width = history.shape[1]
        used = _in(history_len, B, i32, dev, "history_len")
        prompt = _in(prompt_len, B, i32, dev, "prompt_len")
    rep = _in(repetition, B, f32, dev, "repetition")
    freq = _in(frequency, B, f32, dev, "frequency")
    pres = _in(presence, B, f32, dev, "presence")
    boff, btok, bval, n = None, None, None, 0
    if bias_offsets is not None:
        boff = _in(bias_offsets, B + 1, i32, dev, "bias_offsets")
        n = 0 if bias_tokens is None else bias_tokens.numel()
        if n:
            if bias_values is None:
                raise ValueError("bias_tokens need bias_values")
            btok = _in(bias_tokens, n, i32, dev, "bias_tokens")
            bval = _in(bias_values, n, f32, dev, "bias_values")
    mp, mask_ld, masks, midx = None, 0, 0, None
    if mask is not None:
        masks = mask.shape[0]
        mp, mask_ld = _matrix(mask, masks, (V + 31) // 32, dev, "mask")
        if mask_index is None and masks < R:
            raise ValueError("without mask_index every row needs a row of mask")
        midx = _in(mask_index, R, i32, dev, "mask_index")
    err = _in(error_flag, 1, i32, dev, "error_flag")
    if out is not None:
        odt, _, old = _logits(out, V)
        if odt != dtype or out.shape[0] != R or out.device != dev:
            raise ValueError("out must be a matrix [R, >= vocab] of the logits' type and device")
    on = _on(dev, stream)
    with on as s:
        if out is None:
            out, old = torch.empty((R, V), dtype=logits.dtype, device=dev), V
        a = Adjust(logits.data_ptr(), out.data_ptr(), dtype, V, ld, old, B, R, off, drafts, par, hist, hist_ld, width,
                   prompt, used, rep, freq, pres, boff, btok, bval, n, mp, mask_ld, masks, midx, D)
        on.keep(logits, row_offsets, draft_tokens, parents, history, history_len, prompt_len, repetition, frequency,
                presence, bias_offsets, bias_tokens, bias_values, mask, mask_index, out, error_flag)
        _check(lib().vsv_adjust_logits(ctypes.byref(a), err, s))
    return out[:, :V] if out.shape[1] > V else out


def plan_pages(block_table, held, length, row_offsets, free_pages, free_count, page_size, num_rows, stream=None):
    """Pages and slots for rows to be stored (vsv_plan_pages).

    Request i has `length[i]` tokens stored in its first `held[i]` pages of
    block_table [B, W] and row_offsets[i + 1] - row_offsets[i] rows to store.
    block_table and free_pages (a stack of `free_count[0]` page ids) are
    updated in place; everything is int32. `num_rows` is the most rows there
    may be (the offsets' own end is known to the device alone). Returns a
    dict of device tensors: slot [num_rows] int64 and position [num_rows] (-1
    for rows of no request), held, length and free_count behind the call, and
    error_flag (FLAG_PAGES: the pool ran out, and the requests it could not
    serve are as they were)."""
    R, page = int(num_rows), int(page_size)
    if not 0 <= R < 2 ** 31 or not 0 <= page < 2 ** 31:      # (ctypes would take them modulo 2^32)
        raise ValueError("num_rows and page_size must be within 0 .. 2^31 - 1")
    B, i32, dev = row_offsets.numel() - 1, torch.int32, _cuda(row_offsets, "row_offsets")
    off = _in(row_offsets, B + 1, i32, dev, "row_offsets")
    had = _in(held, B, i32, dev, "held")
    lens = _in(length, B, i32, dev, "length")
    pool = free_pages.numel()
    free = _in(free_pages, pool, i32, dev, "free_pages")
    count = _in(free_count, 1, i32, dev, "free_count")
    table, table_ld = _matrix(block_table, B, 0, dev, "block_table")
    on = _on(dev, stream)
    with on as s:
        slot = torch.empty(R, dtype=torch.int64, device=dev)
        words = torch.empty(R + 2 * B + 1, dtype=i32, device=dev)
        position, new_held, new_length, new_count = torch.split_with_sizes(words, (R, B, B, 1))
        flag = _new_flag(dev, s)
        base = words.data_ptr()
        on.keep(block_table, held, length, row_offsets, free_pages, free_count)
        _check(lib().vsv_plan_pages(table, table_ld, block_table.shape[1], had, lens, off, B, R, free, pool, count,
                                    page, slot.data_ptr(), base, base + 4 * R, base + 4 * (R + B),
                                    base + 4 * (R + 2 * B), flag.data_ptr(), s))
    return dict(slot=slot, position=position, held=new_held, length=new_length, free_count=new_count, error_flag=flag)


def _alloc_outputs(B, K, G, dev, with_drafts):
    return dict(verify_len=torch.empty(B, dtype=torch.int32, device=dev),
                row_offsets=torch.empty(B + 1, dtype=torch.int32, device=dev),
                row_owner=torch.empty(max(G, 1), dtype=torch.int32, device=dev),
                row_source=torch.empty(max(G, 1), dtype=torch.int32, device=dev),
                packed_drafts=(torch.empty(max(G - B, 1), dtype=torch.int32, device=dev) if with_drafts else None),
                prefix=torch.empty(max(B * K, 1), dtype=torch.float32, device=dev))


def _alloc_args(confidence, draft_tokens, B, K, G, out, stream):
    if B * K > 0:
        _vec(confidence, B * K, torch.float32, "confidence")
        if draft_tokens is not None:
            _vec(draft_tokens, B * K, torch.int32, "draft_tokens")
    pd = out["packed_drafts"] if draft_tokens is not None and G > B else None
    return (_ptr(confidence) if B * K > 0 else None, (_ptr(draft_tokens) if pd is not None else None), int(B), int(K), int(G),
            _ptr(out["verify_len"]), _ptr(out["row_offsets"]), _ptr(out["row_owner"]),
            _ptr(out["row_source"]), _ptr(pd), _ptr(out["prefix"]), _stream(stream))


def allocate_verify(confidence, draft_tokens, num_requests, num_drafts, row_budget, stream=None):
    """Verify lengths and packed verify layout for a row budget; returns a dict of device tensors.

    `confidence` and `draft_tokens` are [B * K] request-major device vectors
    (`draft_tokens` may be None). The result's row_offsets, row_owner and
    packed_drafts are the batch layout the verify entry points take.
    """
    B, K, G = int(num_requests), int(num_drafts), int(row_budget)
    dev = confidence.device if confidence is not None else torch.device("cuda", torch.cuda.current_device())
    with torch.cuda.stream(_resolve_stream(stream, dev)):
        out = _alloc_outputs(B, K, G, dev, draft_tokens is not None)
    _keep_alive(stream, confidence, draft_tokens)
    _check(lib().vsv_allocate_verify(*_alloc_args(confidence, draft_tokens, B, K, G, out, stream)))
    return out


def _host_array(x, ctype, np_dtype):
    import numpy as np
    a = np.ascontiguousarray(np.asarray(x, dtype=np_dtype))
    return a, a.ctypes.data_as(ctypes.c_void_p)


class Goodput:
    """Goodput step selection over completed batches (host code; see
    vsv_goodput_* in the header). `observe` takes a batch's accepted and
    verified draft counts, `step` the full-round cost of every candidate
    step count 1 .. max_steps and returns the step count for the next batch."""

    def __init__(self, max_steps, window_size=20, update_interval=5, switch_min_gain=0.05):
        self.state = GoodputState()
        _check(lib().vsv_goodput_init(ctypes.byref(self.state), int(max_steps), int(window_size),
                                      int(update_interval), float(switch_min_gain)))

    def observe(self, accepted_len, verify_len):
        import numpy as np
        a, pa = _host_array(accepted_len, ctypes.c_int32, np.int32)
        k, pk = _host_array(verify_len, ctypes.c_int32, np.int32)
        if a.shape != k.shape or a.ndim != 1:
            raise ValueError("accepted_len and verify_len must be matching vectors")
        _check(lib().vsv_goodput_observe(ctypes.byref(self.state), pa, pk, int(a.size)))

    def step(self, cost_ms, batch_size):
        import numpy as np
        c, pc = _host_array(cost_ms, ctypes.c_double, np.float64)
        if c.size != self.state.max_steps:
            raise ValueError("cost_ms needs one cost per step count 1 .. max_steps")
        out = ctypes.c_int32(0)
        _check(lib().vsv_goodput_step(ctypes.byref(self.state), pc, int(batch_size), ctypes.byref(out)))
        return int(out.value)

    @property
    def estimate(self):
        return [self.state.estimate[j] for j in range(self.state.max_steps)]


def goodput_select(prefix_acceptance, cost_ms, batch_size, current, switch_min_gain=0.05):
    """One stateless scoring (vsv_goodput_select); -1 for invalid arguments."""
    import numpy as np
    p, pp = _host_array(prefix_acceptance, ctypes.c_double, np.float64)
    c, pc = _host_array(cost_ms, ctypes.c_double, np.float64)
    if p.size != c.size:
        raise ValueError("one prefix acceptance and one cost per step count")
    return int(lib().vsv_goodput_select(pp, pc, int(c.size), int(batch_size), int(current), float(switch_min_gain)))


class PreparedCall:
    """One entry-point call with every argument marshalled once.

    `run()` issues the C call on the stream captured at construction; the
    tensors passed in must stay alive (they are referenced here). Used where
    per-call Python overhead would otherwise show next to a ~30 us kernel.
    """

    def __init__(self, fn, args, keep):
        self._fn = fn
        self._args = args
        self._keep = keep

    def run(self):
        _check(self._fn(*self._args))


def prepare_greedy(logits, row_offsets, row_owner, draft_tokens, relaxed_topk=1, vocab=None,
                   out=None, ws=None, stream=None):
    batch, outs, res, B, R = _prepare(logits, row_offsets, row_owner, draft_tokens, vocab, stream)
    if out is not None:
        res = out
        outs = _outputs_struct(res)
    ws = workspace(B, R, False, logits.device, stream) if ws is None else ws
    _keep_alive(stream, logits, row_offsets, row_owner, draft_tokens, ws)
    args = (ctypes.byref(batch), int(relaxed_topk), ctypes.byref(outs), _ptr(ws), ws.numel(), _stream(stream))
    return PreparedCall(lib().vsv_verify_greedy, args, (batch, outs, res, ws, logits)), res


def prepare_sampled(logits, row_offsets, row_owner, draft_tokens, temperature, top_k, top_p, min_p,
                    seed, offset=0, vocab=None, out=None, ws=None, stream=None):
    batch, outs, res, B, R = _prepare(logits, row_offsets, row_owner, draft_tokens, vocab, stream)
    if out is not None:
        res = out
        outs = _outputs_struct(res)
    for t, dt, name in ((temperature, torch.float32, "temperature"), (top_k, torch.int32, "top_k"),
                        (top_p, torch.float32, "top_p"), (min_p, torch.float32, "min_p")):
        _vec(t, B, dt, name)
    ws = workspace(B, R, True, logits.device, stream) if ws is None else ws
    _keep_alive(stream, logits, row_offsets, row_owner, draft_tokens, temperature, top_k, top_p, min_p, ws)
    args = (ctypes.byref(batch), _ptr(temperature), _ptr(top_k), _ptr(top_p), _ptr(min_p),
            int(seed) & (2**64 - 1), int(offset) & (2**64 - 1), ctypes.byref(outs), _ptr(ws), ws.numel(),
            _stream(stream))
    return PreparedCall(lib().vsv_verify_sampled, args,
                        (batch, outs, res, ws, logits, temperature, top_k, top_p, min_p)), res


def prepare_allocate(confidence, draft_tokens, num_requests, num_drafts, row_budget, out=None, stream=None):
    B, K, G = int(num_requests), int(num_drafts), int(row_budget)
    if out is None:
        out = _alloc_outputs(B, K, G, confidence.device, draft_tokens is not None)
    args = _alloc_args(confidence, draft_tokens, B, K, G, out, stream)
    return PreparedCall(lib().vsv_allocate_verify, args, (confidence, draft_tokens, out)), out


def prepare_confidence(draft_logits, selected=None, vocab=None, out=None, stream=None):
    dtype, V, ld = _logits(draft_logits, vocab)
    D = draft_logits.shape[0]
    if selected is not None:
        _vec(selected, D, torch.int32, "selected")
    dev = draft_logits.device
    if out is None:
        out = (torch.empty(D, dtype=torch.float32, device=dev), torch.empty(D, dtype=torch.float32, device=dev),
               torch.zeros(1, dtype=torch.int32, device=dev))
    conf, lse, flag = out
    args = (_ptr(draft_logits), dtype, V, ld, D, _ptr(selected), _ptr(conf), _ptr(lse), _ptr(flag),
            _stream(stream))
    return PreparedCall(lib().vsv_draft_confidence, args, (draft_logits, selected, out)), out
