"""Python binding of the q8moe C ABI (include/q8moe.h): argument marshalling only.

Every computation runs in the CUDA library ``libq8moe.so`` built in-tree for sm_103a (``build.build()``).  There is no
fallback: importing this package without the built library raises ImportError.  Tensors are PyTorch tensors used only
as device memory; the current PyTorch stream is used unless a stream is passed.
"""
from __future__ import annotations

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libq8moe.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is not built; run moe_add_rmsnorm_gb300.build.build() (nvcc, sm_103a)")

lib = ctypes.CDLL(LIB_PATH)

F32ACT_F64SUM = 0
INT8ACT = 1
INT8ACT2 = 2  # the two-word activation (high words, low words in 128ths of the block scale)
QBLOCK = 32

STATUS = {0: "Q8_OK", -1: "Q8_EINVAL", -2: "Q8_EUNSUPPORTED", -3: "Q8_ECUDA", -4: "Q8_ETIMEOUT", -5: "Q8_ENOSPACE"}


class Q8Error(RuntimeError):
    def __init__(self, code, msg):
        super().__init__(f"{STATUS.get(code, code)}: {msg}")
        self.code = code


class q8_mat(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("s", ctypes.c_void_p), ("rows", ctypes.c_int64), ("cols", ctypes.c_int64)]


class q8_act(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("s", ctypes.c_void_p), ("lo", ctypes.c_void_p)]


class q8_shared_expert(ctypes.Structure):
    _fields_ = [("gate", q8_mat), ("up", q8_mat), ("down", q8_mat)]


class q8_moe_plan(ctypes.Structure):
    _fields_ = [("counts", ctypes.c_void_p), ("offsets", ctypes.c_void_p), ("lists", ctypes.c_void_p),
                ("active", ctypes.c_void_p)]


KV_INT8 = 0  # cached words: signed 8-bit integers, a scale a row
KV_E4M3 = 1  # cached words: 8-bit floats of 4 exponent and 3 mantissa bits, a scale a row
KV_ERR_LENGTH, KV_ERR_PAGE, KV_ERR_ROPE, KV_ERR_WAIT = 1, 2, 4, 8  # bits of a batch's error word


class q8_kv_pages(ctypes.Structure):
    device = tensors = None  # the tensors behind it (kv_pages sets them; None: the caller's business)
    _fields_ = [(n, ctypes.c_void_p) for n in ("k", "v", "ks", "vs")] + [
        (n, ctypes.c_int64) for n in ("pages", "page_size", "kv_heads", "head_dim")] + [("words", ctypes.c_int)]


class q8_kv_batch(ctypes.Structure):
    device = tensors = None
    _fields_ = [(n, ctypes.c_void_p) for n in ("row_start", "kv_len", "table")] + [
        (n, ctypes.c_int64) for n in ("seqs", "table_pages", "table_stride")] + [("error", ctypes.c_void_p)]


class q8_model_desc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("layers", "d", "heads", "kv_heads", "head_dim", "experts", "k", "dff",
                                                "vocab", "ctx")] + [
        ("eps", ctypes.c_float), ("rope_theta", ctypes.c_double), ("mode", ctypes.c_int),
        ("embed", ctypes.c_void_p), ("attn_norm", ctypes.c_void_p), ("ffn_norm", ctypes.c_void_p),
        ("q_norm", ctypes.c_void_p), ("k_norm", ctypes.c_void_p), ("final_norm", ctypes.c_void_p),
        ("wq", ctypes.c_void_p), ("wk", ctypes.c_void_p), ("wv", ctypes.c_void_p), ("wo", ctypes.c_void_p),
        ("router", ctypes.c_void_p), ("gate", ctypes.c_void_p), ("up", ctypes.c_void_p), ("down", ctypes.c_void_p),
        ("lm_head", q8_mat), ("k_cache", ctypes.c_void_p), ("v_cache", ctypes.c_void_p),
        ("tok", ctypes.c_void_p), ("pos", ctypes.c_void_p), ("logits", ctypes.c_void_p),
        ("router_f32", ctypes.c_void_p), ("shared_gate", ctypes.c_void_p), ("shared_up", ctypes.c_void_p),
        ("shared_down", ctypes.c_void_p), ("shared_dff", ctypes.c_int64), ("batch", ctypes.c_int64)]


_vp, _i64, _i32, _f32, _sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
_P = ctypes.POINTER
_SIGS = {
    "q8_workspace_create": [_sz, _P(_vp)],
    "q8_workspace_destroy": [_vp],
    "q8_workspace_bytes": [_vp],
    "q8_workspace_check": [_vp, _vp],
    "q8_quantize": [_vp, _i64, _i64, _P(q8_act), _vp],
    "add_rmsnorm_q8": [_vp, _vp, _vp, _i64, _i64, _f32, _vp, _vp, _P(q8_act), _vp],
    "q8_gemv": [_P(q8_mat), _i32, _vp, _P(q8_act), _i64, _vp, _vp, _vp],
    "q8_gemv_blockdots": [_P(q8_mat), _P(q8_act), _i64, _vp, _vp, _vp, _vp],
    "q8_gemv_noalloc": [_P(q8_mat), _i32, _vp, _P(q8_act), _i64, _vp, _vp],
    "q8_set_tensor_core_rows": [_i32],
    "q8_set_grouped_tensor_core_rows": [_i32],
    "q8_set_tensor_core_attention": [_i32],
    "q8_set_persistent_decode": [_i32],
    "q8_set_streamed_batch_attention": [_i32],
    "q8_model_persistent": [_vp],
    "moe_route_topk": [_P(q8_mat), _i32, _vp, _P(q8_act), _i64, _i32, _vp, _vp, _vp, _P(q8_moe_plan), _vp, _vp],
    "moe_route_topk_f32": [_vp, _i64, _i64, _vp, _i64, _i32, _vp, _vp, _vp, _P(q8_moe_plan), _vp, _vp],
    "moe_gate_up": [_P(q8_mat), _P(q8_mat), _i64, _i32, _vp, _P(q8_act), _i64, _i32, _vp, _P(q8_moe_plan), _vp,
                    _P(q8_act), _P(q8_shared_expert), _vp, _vp],
    "moe_down_combine": [_P(q8_mat), _i64, _i32, _vp, _P(q8_act), _i64, _i32, _vp, _vp, _P(q8_moe_plan), _vp, _vp,
                         _vp, _P(q8_shared_expert), _vp, _vp],
    "q8_rope_table": [ctypes.c_double, _i64, _i64, _vp, _vp, _vp],
    "q8_kv_append": [_P(q8_kv_pages), _P(q8_kv_batch), _i64, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _vp, _f32, _vp,
                     _vp, _i64, _vp, _i64, _vp],
    "q8_kv_read": [_P(q8_kv_pages), _P(q8_kv_batch), _i64, _vp, _vp, _i64, _i64, _vp],
    "q8_paged_attention": [_P(q8_kv_pages), _P(q8_kv_batch), _i64, _i64, _vp, _i64, _f32, _vp, _i64, _vp, _vp, _vp],
    "q8_paged_wait_selftest": [_P(q8_kv_pages), _P(q8_kv_batch), _i64, _i64, _vp, _i64, _f32, _vp, _i64, _vp, ctypes.c_uint,
                               _vp],
    "q8_model_create": [_P(q8_model_desc), _P(_vp)],
    "q8_model_destroy": [_vp],
    "decode_step": [_vp, _vp],
    "decode_step_launches": [_vp, _vp],
    "decode_step_trace": [_vp, _vp, _vp],
    "prefill_chunk": [_vp, _vp, _i64, _vp, _vp],
    "prefill_chunk_trace": [_vp, _vp, _i64, _vp, _vp, _vp],
    "q8_model_check": [_vp, _vp],
    "q8_model_wait_selftest": [_vp, ctypes.c_uint, _vp],
    "q8_model_launches_per_step": [_vp],
    "q8_last_error": [],
}
for _name, _args in _SIGS.items():
    _fn = getattr(lib, _name)
    _fn.argtypes = _args
    _fn.restype = ctypes.c_int
lib.q8_workspace_destroy.restype = None
lib.q8_model_destroy.restype = None
lib.q8_workspace_bytes.restype = ctypes.c_size_t
lib.q8_last_error.restype = ctypes.c_char_p
lib.q8_model_launches_per_step.restype = ctypes.c_int64

EXPORTS = tuple(_SIGS)


def last_error() -> str:
    return lib.q8_last_error().decode()


def _check(code):
    if code != 0:
        raise Q8Error(code, last_error())


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is not None:
        return ctypes.c_void_p(int(stream))
    import torch
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def mat(q, s) -> q8_mat:
    """A q8_mat over device tensors q int8 [rows, cols] and s f32 [rows, cols/32]."""
    return q8_mat(q.data_ptr(), s.data_ptr(), q.shape[0], q.shape[1])


def act(q, s, lo=None) -> q8_act:
    return q8_act(q.data_ptr(), s.data_ptr(), lo.data_ptr() if lo is not None else None)


def _actref(q, s, lo=None):
    return ctypes.byref(act(q, s, lo)) if q is not None else None


class Workspace:
    def __init__(self, nbytes: int = 0):
        h = ctypes.c_void_p()
        _check(lib.q8_workspace_create(nbytes, ctypes.byref(h)))
        self.handle = h
        self.device = _lazy_torch().cuda.current_device()

    @property
    def nbytes(self):
        return lib.q8_workspace_bytes(self.handle)

    def check(self, stream=None):
        """Waits for the stream; raises Q8_ETIMEOUT, and makes the workspace usable again, when a bounded wait of a
        q8_paged_attention on it gave up."""
        _check(lib.q8_workspace_check(self.handle, _stream(stream)))

    def close(self):
        if self.handle:
            lib.q8_workspace_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def q8_quantize(x, q, s, stream=None, lo=None):
    """One word per value, or with `lo` the two-word form."""
    rows = x.shape[0] if x.dim() > 1 else 1
    _check(lib.q8_quantize(_ptr(x), rows, x.shape[-1], _actref(q, s, lo), _stream(stream)))


def add_rmsnorm_q8(a, b, w, eps, sum_out=None, y_out=None, yq=None, ys=None, stream=None, yl=None):
    rows = a.shape[0] if a.dim() > 1 else 1
    qa = _actref(yq, ys, yl)
    _check(lib.add_rmsnorm_q8(_ptr(a), _ptr(b), _ptr(w), rows, a.shape[-1], float(eps), _ptr(sum_out), _ptr(y_out),
                              qa, _stream(stream)))


def q8_gemv(q, s, mode, y, x=None, xq=None, xs=None, rows=1, ws=None, stream=None, xl=None):
    W = mat(q, s)
    qa = _actref(xq, xs, xl)
    _check(lib.q8_gemv(ctypes.byref(W), int(mode), _ptr(x), qa, rows, _ptr(y), ws.handle if ws else None,
                       _stream(stream)))


def q8_gemv_noalloc(q, s, mode, y, x=None, xq=None, xs=None, rows=1, stream=None, xl=None):
    """q8_gemv without a workspace: scratch comes from the library's fixed per-device array (see q8moe.h)."""
    W = mat(q, s)
    qa = _actref(xq, xs, xl)
    _check(lib.q8_gemv_noalloc(ctypes.byref(W), int(mode), _ptr(x), qa, rows, _ptr(y), _stream(stream)))


def q8_gemv_blockdots(q, s, xq, xs, dots, y, rows=1, ws=None, stream=None, xl=None):
    """With xl (two words) dots is [2, rows, n, nb]: the words' dots, then the low words'."""
    W = mat(q, s)
    qa = act(xq, xs, xl)
    _check(lib.q8_gemv_blockdots(ctypes.byref(W), ctypes.byref(qa), rows, _ptr(dots), _ptr(y),
                                 ws.handle if ws else None, _stream(stream)))


def set_tensor_core_rows(rows: int):
    """The fewest int8 activation rows (16..64) a dense projection takes to the tensor cores; 0: never; -1 (the
    default): one matrix of at least 2048 x 2048 from 32 rows on."""
    _check(lib.q8_set_tensor_core_rows(int(rows)))


def set_grouped_tensor_core_rows(rows: int):
    """The fewest rows (16..64) an int8 expert group of a chunk needs to take the tensor cores; 0: never (default 32)."""
    _check(lib.q8_set_grouped_tensor_core_rows(int(rows)))


def set_tensor_core_attention(on: bool):
    """Prefill chunks' causal attention on the tensor cores (default) or, with False, the CUDA cores."""
    _check(lib.q8_set_tensor_core_attention(1 if on else 0))


def set_persistent_decode(on: bool):
    """One-sequence int8 decode steps as one persistent launch, or (False, the default) six launches a layer."""
    _check(lib.q8_set_persistent_decode(1 if on else 0))


def set_streamed_batch_attention(min_batch: int):
    """Batch decode steps of at least min_batch sequences (default 8) attend in the streamed form; 0: never."""
    _check(lib.q8_set_streamed_batch_attention(int(min_batch)))


def plan_struct(counts, offsets, lists, active):
    return q8_moe_plan(counts.data_ptr(), offsets.data_ptr(), lists.data_ptr(), active.data_ptr())


def moe_route_topk(rq, rs, mode, k, ids, gates, x=None, xq=None, xs=None, rows=1, logits=None, plan=None, ws=None,
                   stream=None, xl=None):
    R = mat(rq, rs)
    qa = _actref(xq, xs, xl)
    pl = ctypes.byref(plan) if plan is not None else None
    _check(lib.moe_route_topk(ctypes.byref(R), int(mode), _ptr(x), qa, rows, int(k), _ptr(ids), _ptr(gates),
                              _ptr(logits), pl, ws.handle if ws else None, _stream(stream)))


def shared_expert(gate, up, down) -> q8_shared_expert:
    """A shared expert over (q, s) device tensor pairs: gate and up [sdff, d], down [d, sdff]."""
    return q8_shared_expert(mat(*gate), mat(*up), mat(*down))


def moe_route_topk_f32(router, k, ids, gates, x, rows=1, logits=None, plan=None, ws=None, stream=None):
    """The router of f32 values (device f32 [E, d]) over the f32 rows x, then top-k as moe_route_topk."""
    pl = ctypes.byref(plan) if plan is not None else None
    _check(lib.moe_route_topk_f32(_ptr(router), router.shape[0], router.shape[1], _ptr(x), rows, int(k), _ptr(ids),
                                  _ptr(gates), _ptr(logits), pl, ws.handle if ws else None, _stream(stream)))


def moe_gate_up(gq, gs, uq, us, dff, mode, k, ids, h, x=None, xq=None, xs=None, hq=None, hs=None, rows=1, plan=None,
                ws=None, stream=None, xl=None, hl=None, shared=None):
    G, U = mat(gq, gs), mat(uq, us)
    qa = _actref(xq, xs, xl)
    ha = _actref(hq, hs, hl)
    pl = ctypes.byref(plan) if plan is not None else None
    sh = ctypes.byref(shared) if shared is not None else None
    _check(lib.moe_gate_up(ctypes.byref(G), ctypes.byref(U), int(dff), int(mode), _ptr(x), qa, rows, int(k),
                           _ptr(ids), pl, _ptr(h), ha, sh, ws.handle if ws else None, _stream(stream)))


def moe_down_combine(dq, ds, d, mode, k, ids, gates, y, h=None, hq=None, hs=None, rows=1, plan=None, residual=None,
                     expert_out=None, ws=None, stream=None, hl=None, shared=None):
    Dm = mat(dq, ds)
    ha = _actref(hq, hs, hl)
    pl = ctypes.byref(plan) if plan is not None else None
    sh = ctypes.byref(shared) if shared is not None else None
    _check(lib.moe_down_combine(ctypes.byref(Dm), int(d), int(mode), _ptr(h), ha, rows, int(k), _ptr(ids),
                                _ptr(gates), pl, _ptr(residual), _ptr(y), _ptr(expert_out), sh,
                                ws.handle if ws else None, _stream(stream)))


_torch = None


def _lazy_torch():
    """torch, imported on first use (the calls below run once a layer: they look a module up once)."""
    global _torch
    if _torch is None:
        import torch
        _torch = torch
    return _torch


def _refuse(msg):
    raise Q8Error(-1, msg)


_current_device = None


def _device(t, name):
    """The device of tensor t, which has to be the current one (a CUDA tensor's torch has been initialised: the device is
    asked for without that check where this torch has a call for it)."""
    global _current_device
    if _current_device is None:
        _current_device = getattr(_lazy_torch()._C, "_cuda_getDevice", None) or _lazy_torch().cuda.current_device
    d = t.get_device()
    if d < 0 or d != _current_device():
        _refuse(f"{name}: not on the current device")
    return d


_raw_stream = None


def _stream_of(stream, device):
    """The stream of a call on `device`: the one given, or torch's current one (by the handle alone where this torch has
    a call for it: building a Stream object takes longer than the launch)."""
    global _raw_stream
    if stream is not None:
        return int(stream)
    if _raw_stream is None:
        _raw_stream = getattr(_torch._C, "_cuda_getCurrentRawStream", None) or \
            (lambda d: _torch.cuda.current_stream(d).cuda_stream)
    return _raw_stream(device)


def _rows(t, heads, hd, device, name):
    """The address and row stride of f32 rows [rows, heads, hd] whose heads are consecutive."""
    if t.dtype is not _torch.float32 or t.get_device() != device:
        _refuse(f"{name}: not an f32 tensor of the current device")
    shape, stride = t.shape, t.stride()
    if len(shape) != 3 or shape[1] != heads or shape[2] != hd:
        _refuse(f"{name}: {tuple(shape)}, expected [rows, {heads}, {hd}]")
    if stride[2] != 1 or (heads > 1 and stride[1] != hd):
        _refuse(f"{name}: the heads of a row are not consecutive")
    return t.data_ptr(), stride[0] if shape[0] > 1 else heads * hd


def _matrix(t, name):
    """A table of two dimensions (its values are checked by _vec)."""
    if t.dim() != 2:
        _refuse(f"{name}: {tuple(t.shape)}, expected [positions, head_dim/2]")
    return t.shape


def _heads_of(t, name):
    """The heads of rows [rows, heads, hd] (the rest of them is checked by _rows)."""
    if t.dim() != 3:
        _refuse(f"{name}: {tuple(t.shape)}, expected [rows, heads, head_dim]")
    return t.shape[1]


def _vec(t, n, device, name):
    """The address of a contiguous device f32 tensor of n values (None: NULL)."""
    if t is None:
        return None
    if t.dtype is not _torch.float32 or t.get_device() != device or t.numel() != n or not t.is_contiguous():
        _refuse(f"{name}: not a contiguous f32 tensor of {n} values on the current device")
    return t.data_ptr()


def kv_pages(k, ks, v, vs) -> q8_kv_pages:
    """Pages over device tensors: words k and v [pages, kv_heads, page_size, head_dim] (int8 or float8_e4m3fn), scales ks
    and vs f32 [pages, kv_heads, page_size].  The struct keeps the tensors."""
    torch = _lazy_torch()
    kind, shape = k.dtype, k.shape
    if kind is torch.int8:
        words = KV_INT8
    elif kind is torch.float8_e4m3fn:
        words = KV_E4M3
    else:
        _refuse("k: not int8 or e4m3 words")
    if len(shape) != 4 or v.dtype is not kind or v.shape != shape:
        _refuse("k, v: not words [pages, kv_heads, page_size, head_dim] of one type")
    scales = shape[:3]
    if ks.dtype is not torch.float32 or vs.dtype is not torch.float32 or ks.shape != scales or vs.shape != scales:
        _refuse(f"ks, vs: not f32 {tuple(scales)}")
    if not (k.is_contiguous() and v.is_contiguous() and ks.is_contiguous() and vs.is_contiguous()):
        _refuse("pages: not contiguous")
    d = _device(k, "k")
    if v.get_device() != d or ks.get_device() != d or vs.get_device() != d:
        _refuse("pages: not all on the current device")
    p = q8_kv_pages(k.data_ptr(), v.data_ptr(), ks.data_ptr(), vs.data_ptr(), shape[0], shape[2], shape[1], shape[3],
                    words)
    p.device, p.tensors = d, (k, ks, v, vs)
    return p


def kv_batch(row_start, kv_len, table, error=None) -> q8_kv_batch:
    """A batch of sequences over pages (q8moe.h, q8_kv_batch): device int32 row_start [seqs + 1], kv_len [seqs] and table
    [seqs, pages], and optionally an int32 error word.  The struct keeps the tensors."""
    i32 = _lazy_torch().int32
    shape = table.shape
    if len(shape) != 2 or kv_len.dim() != 1 or row_start.dim() != 1:
        _refuse("batch: expected row_start [seqs + 1], kv_len [seqs], table [seqs, pages]")
    seqs, pages = shape
    if kv_len.shape[0] != seqs or row_start.shape[0] != seqs + 1:
        _refuse("batch: expected row_start [seqs + 1], kv_len [seqs], table [seqs, pages]")
    if table.dtype is not i32 or kv_len.dtype is not i32 or row_start.dtype is not i32:
        _refuse("batch: not int32")
    strides = table.stride()
    if not (kv_len.is_contiguous() and row_start.is_contiguous() and (pages <= 1 or strides[1] == 1)):
        _refuse("batch: values not consecutive")
    d = _device(table, "table")
    if kv_len.get_device() != d or row_start.get_device() != d:
        _refuse("batch: not all on the current device")
    e = None
    if error is not None:
        if error.dtype is not i32 or error.numel() != 1 or error.get_device() != d:
            _refuse("error: not one int32 value on the current device")
        e = error.data_ptr()
    b = q8_kv_batch(row_start.data_ptr(), kv_len.data_ptr(), table.data_ptr(), seqs, pages,
                    strides[0] if seqs > 1 else pages, e)
    b.device, b.tensors = d, (row_start, kv_len, table, error)
    return b


def _paged_device(pages, batch, t, name):
    """The device of a call's tensor t, which has to be the current one, the pages' and the batch's."""
    d = _device(t, name)
    if (pages.device not in (d, None)) or (batch.device not in (d, None)):
        _refuse("pages, batch: not on the current device")
    return d


def _ws_of(ws, device):
    """The handle of a call's workspace, which has to be of its device."""
    if ws is None:
        return None
    if ws.device != device:
        _refuse("ws: not on the current device")
    return ws.handle


def q8_rope_table(theta, cos, sin, stream=None):
    """Fills cos and sin (device f32 [positions, head_dim/2]) with the rotation tables of base theta."""
    n, half = _matrix(cos, "cos")
    d = _device(cos, "cos")
    _check(lib.q8_rope_table(float(theta), n, 2 * half, _vec(cos, n * half, d, "cos"), _vec(sin, n * half, d, "sin"),
                             _stream_of(stream, d)))


def q8_kv_append(pages, batch, q, k, v, q_out, q_norm=None, k_norm=None, eps=1e-6, cos=None, sin=None, stream=None):
    """Norms and rotates the rows' query and key heads (q [rows, heads, hd] into q_out; k, v [rows, kv_heads, hd]) and
    quantizes the keys and values into their page slots.  q and q_out may be None (keys and values only)."""
    kv, hd = pages.kv_heads, pages.head_dim
    d = _paged_device(pages, batch, k, "k")
    ka, ks = _rows(k, kv, hd, d, "k")
    va, vs = _rows(v, kv, hd, d, "v")
    rows = k.shape[0]
    if v.shape[0] != rows or (q is None) != (q_out is None):
        _refuse("q, k, v, q_out: rows differ")
    heads, qa, qs, oa, os_ = 0, None, 0, None, 0
    if q is not None:
        heads = _heads_of(q, "q")
        qa, qs = _rows(q, heads, hd, d, "q")
        oa, os_ = _rows(q_out, heads, hd, d, "q_out")
        if q.shape[0] != rows or q_out.shape[0] != rows:
            _refuse("q, k, v, q_out: rows differ")
    positions = _matrix(cos, "cos")[0] if cos is not None else 0
    _check(lib.q8_kv_append(pages, batch, rows, heads, qa, qs, ka, ks, va, vs, _vec(q_norm, hd, d, "q_norm"),
                            _vec(k_norm, hd, d, "k_norm"), eps, _vec(cos, positions * hd // 2, d, "cos"),
                            _vec(sin, positions * hd // 2, d, "sin"), positions, oa, os_, _stream_of(stream, d)))


def q8_kv_read(pages, batch, k_out=None, v_out=None, stream=None):
    """The values of the batch's rows into k_out and v_out [rows, kv_heads, hd] (either may be None; rows and heads any
    multiple of 8 values apart, as in the transposed view of a dense cache [kv_heads, ctx, hd])."""
    kv, hd = pages.kv_heads, pages.head_dim
    one = k_out if k_out is not None else v_out
    if one is None:
        _refuse("k_out and v_out: both None")
    d, shape, strides, f32 = _paged_device(pages, batch, one, "k_out, v_out"), one.shape, one.stride(), _torch.float32
    if len(shape) != 3 or shape[1] != kv or shape[2] != hd or strides[2] != 1 or one.dtype is not f32:
        _refuse(f"k_out, v_out: not f32 [rows, {kv}, {hd}] with consecutive values")
    if one is k_out and v_out is not None:
        if v_out.dtype is not f32 or v_out.get_device() != d or v_out.shape != shape or v_out.stride() != strides:
            _refuse("v_out: not laid out as k_out")
    rows = shape[0]
    _check(lib.q8_kv_read(pages, batch, rows, k_out.data_ptr() if k_out is not None else None,
                          v_out.data_ptr() if v_out is not None else None, strides[0] if rows > 1 else kv * hd,
                          strides[1] if kv > 1 else hd, _stream_of(stream, d)))


def q8_paged_attention(pages, batch, q, out, scale=None, lse=None, ws=None, stream=None):
    """Causal attention of the rows q [rows, heads, hd] over their sequences' cached positions, into out; scale defaults
    to hd^-1/2, lse (optional) is f32 [rows, heads]."""
    hd, d = pages.head_dim, _paged_device(pages, batch, q, "q")
    heads, rows = _heads_of(q, "q"), q.shape[0]
    qa, qs = _rows(q, heads, hd, d, "q")
    oa, os_ = _rows(out, heads, hd, d, "out")
    if out.shape[0] != rows:
        _refuse("out: rows differ")
    _check(lib.q8_paged_attention(pages, batch, rows, heads, qa, qs, hd ** -0.5 if scale is None else scale, oa, os_,
                                  _vec(lse, rows * heads, d, "lse"), _ws_of(ws, d), _stream_of(stream, d)))


def q8_paged_wait_selftest(pages, batch, q, out, polls, ws, stream=None):
    """q8_paged_attention's launches with waits that run out after `polls` polls; the next ws.check() raises Q8_ETIMEOUT."""
    hd, d = pages.head_dim, _paged_device(pages, batch, q, "q")
    heads, rows = _heads_of(q, "q"), q.shape[0]
    qa, qs = _rows(q, heads, hd, d, "q")
    oa, os_ = _rows(out, heads, hd, d, "out")
    if out.shape[0] != rows:
        _refuse("out: rows differ")
    _check(lib.q8_paged_wait_selftest(pages, batch, rows, heads, qa, qs, hd ** -0.5, oa, os_, _ws_of(ws, d), int(polls),
                                      _stream_of(stream, d)))


class Model:
    """A decode model over caller-owned device tensors (see q8_model_desc in include/q8moe.h)."""

    def __init__(self, cfg: dict, t: dict, mode: int, tok, pos, logits=None):
        L = cfg["layers"]
        self._keep = []

        def ptr_array(tensors):
            arr = (ctypes.c_void_p * L)(*[x.data_ptr() for x in tensors])
            self._keep.append(arr)
            return ctypes.cast(arr, ctypes.c_void_p)

        def mat_array(pairs):
            arr = (q8_mat * L)(*[mat(q, s) for q, s in pairs])
            self._keep.append(arr)
            return ctypes.cast(arr, ctypes.c_void_p)

        d = q8_model_desc()
        for key in ("layers", "d", "heads", "kv_heads", "experts", "k", "dff", "vocab", "ctx"):
            setattr(d, key, int(cfg[key]))
        d.head_dim = int(cfg["hd"])
        d.batch = int(cfg.get("batch", 0))  # the batch form: tok, pos [batch], logits [batch, vocab], caches per layer
                                            # [batch, kv, ctx, hd]
        d.eps = float(cfg["eps"])
        d.rope_theta = float(cfg["rope_theta"])
        d.mode = int(mode)
        d.embed = t["embed"].data_ptr()
        d.attn_norm = ptr_array(t["attn_norm"])
        d.ffn_norm = ptr_array(t["ffn_norm"])
        d.q_norm = ptr_array(t["q_norm"])
        d.k_norm = ptr_array(t["k_norm"])
        d.final_norm = t["final_norm"].data_ptr()
        for key in ("wq", "wk", "wv", "wo", "router", "gate", "up", "down"):
            setattr(d, key, mat_array(t[key]))
        d.lm_head = mat(*t["lm_head"])
        d.k_cache = ptr_array(t["k_cache"])
        d.v_cache = ptr_array(t["v_cache"])
        d.tok = tok.data_ptr()
        d.pos = pos.data_ptr()
        d.logits = logits.data_ptr() if logits is not None else None
        if t.get("router_f32") is not None:  # optional: routers of f32 values
            d.router_f32 = ptr_array(t["router_f32"])
        if t.get("shared_gate") is not None:  # optional: a shared expert per layer
            for key in ("shared_gate", "shared_up", "shared_down"):
                setattr(d, key, mat_array(t[key]))
            d.shared_dff = int(t["shared_gate"][0][0].shape[0])
        h = ctypes.c_void_p()
        _check(lib.q8_model_create(ctypes.byref(d), ctypes.byref(h)))
        self.handle = h
        self.tensors = t

    def step(self, stream=None):
        _check(lib.decode_step(self.handle, _stream(stream)))

    def step_launches(self, stream=None):
        _check(lib.decode_step_launches(self.handle, _stream(stream)))

    def step_trace(self, hidden, stream=None):
        """Plain-launch step that also copies the residual stream entering layer 0 and leaving every layer into
        hidden (device f32 [layers + 1, d])."""
        _check(lib.decode_step_trace(self.handle, hidden.data_ptr(), _stream(stream)))

    def prefill(self, tokens, ws, stream=None):
        """tokens: device int32 [rows]; the chunk through every layer (plain launches), last row's token into tok."""
        _check(lib.prefill_chunk(self.handle, tokens.data_ptr(), tokens.numel(), ws.handle, _stream(stream)))

    def prefill_trace(self, tokens, ws, hidden, stream=None):
        """prefill() that also copies the residual rows entering every layer and the final ones into hidden (device
        f32 [layers + 1, rows, d])."""
        _check(lib.prefill_chunk_trace(self.handle, tokens.data_ptr(), tokens.numel(), ws.handle, hidden.data_ptr(),
                                       _stream(stream)))

    def check(self, stream=None):
        _check(lib.q8_model_check(self.handle, _stream(stream)))

    def wait_selftest(self, polls, stream=None):
        """A bounded wait on a barrier nothing arrives on; the next check() raises Q8_ETIMEOUT."""
        _check(lib.q8_model_wait_selftest(self.handle, int(polls), _stream(stream)))

    def launches_per_step(self):
        """Kernels one step launches (the captured graph's kernel nodes; 0 before the first step)."""
        return int(lib.q8_model_launches_per_step(self.handle))

    def persistent(self):
        """Whether the model's decode steps run their layers as one persistent launch."""
        return bool(lib.q8_model_persistent(self.handle))

    def close(self):
        if self.handle:
            lib.q8_model_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
