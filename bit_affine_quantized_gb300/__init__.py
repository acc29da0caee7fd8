"""Python binding of libmoe_gb300 (include/moe.h): argument marshalling only.

Every step of the MoE block runs in the CUDA library; this module turns
torch tensors into device pointers and status codes into exceptions.  It
fails loudly when the compiled library is missing: there is no fallback.
"""
from __future__ import annotations

import ctypes
import math
import os
import re

from .build import LIB_PATH, build as build_library

__all__ = [
    "MoeError", "Dims", "QMat", "BlobLayout", "LayerWeights", "Moe", "load_library", "header_symbols",
    "MOE_OK", "MOE_ERR_INVALID_ARG", "MOE_ERR_UNSUPPORTED", "MOE_ERR_CUDA", "MOE_ERR_BAD_EXPERT_ID",
    "MOE_ERR_TIMEOUT", "MOE_ERR_NONFINITE", "MOE_ERR_WORKSPACE", "build_library", "static_get_error",
    "layer_forward_static", "ExpertCache", "QdenseWeights", "LogitRules", "make_qdense_weights", "make_logit_rules",
    "KvCache", "SampleRules", "make_kv_cache", "make_sample_rules",
]

MOE_OK = 0
MOE_ERR_INVALID_ARG = 1
MOE_ERR_UNSUPPORTED = 2
MOE_ERR_CUDA = 3
MOE_ERR_BAD_EXPERT_ID = 4
MOE_ERR_TIMEOUT = 5
MOE_ERR_NONFINITE = 6
MOE_ERR_WORKSPACE = 7
MOE_PROMPT_MAX_ROWS = 4096

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "moe.h")


class Dims(ctypes.Structure):
    _fields_ = [("hidden", ctypes.c_int), ("inter", ctypes.c_int), ("n_experts", ctypes.c_int),
                ("top_k", ctypes.c_int), ("group", ctypes.c_int)]


class QMat(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("biases", ctypes.c_void_p)]


_BLOB_FIELDS = ("gate_q", "gate_s", "gate_b", "up_q", "up_s", "up_b", "down_q", "down_s", "down_b")


class BlobLayout(ctypes.Structure):
    _fields_ = [(n, ctypes.c_size_t) for n in _BLOB_FIELDS]


class LayerWeights(ctypes.Structure):
    _fields_ = [("dims", Dims), ("router", QMat), ("experts", ctypes.c_void_p), ("expert_stride", ctypes.c_size_t),
                ("layout", BlobLayout), ("shared", ctypes.c_void_p), ("logit_bias", ctypes.c_void_p),
                ("router_scale", ctypes.c_void_p), ("per_expert_scale", ctypes.c_void_p),
                ("post_norm", ctypes.c_void_p), ("layer_scalar", ctypes.c_void_p)]


class HeadWeights(ctypes.Structure):
    _fields_ = [("vocab", ctypes.c_int), ("hidden", ctypes.c_int), ("w", QMat)]


class QdenseWeights(ctypes.Structure):
    device = None  # of the tensors, where make_qdense_weights knows them
    _fields_ = [("channels", ctypes.c_int), ("width", ctypes.c_int), ("q", ctypes.c_void_p),
                ("scales", ctypes.c_void_p)]


class LogitRules(ctypes.Structure):
    device = rows = words = None  # of the tensors, where make_logit_rules knows them
    _fields_ = [("history", ctypes.c_void_p), ("history_len", ctypes.c_void_p), ("prompt_len", ctypes.c_void_p),
                ("history_stride", ctypes.c_int), ("repetition", ctypes.c_void_p), ("presence", ctypes.c_void_p),
                ("frequency", ctypes.c_void_p), ("bias_ids", ctypes.c_void_p), ("bias_values", ctypes.c_void_p),
                ("bias_len", ctypes.c_void_p), ("bias_stride", ctypes.c_int), ("mask", ctypes.c_void_p),
                ("mask_stride", ctypes.c_int)]


class KvCache(ctypes.Structure):
    device = None  # of the tensors, where make_kv_cache knows them
    _fields_ = [("n_pages", ctypes.c_int), ("kv_heads", ctypes.c_int), ("page_rows", ctypes.c_int),
                ("head_dim", ctypes.c_int), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("k_scales", ctypes.c_void_p), ("v_scales", ctypes.c_void_p), ("table", ctypes.c_void_p),
                ("n_seqs", ctypes.c_int), ("table_stride", ctypes.c_int)]


class SampleRules(ctypes.Structure):
    device = rows = None  # of the tensors, where make_sample_rules knows them
    _fields_ = [("uniform", ctypes.c_void_p), ("temperature", ctypes.c_void_p), ("top_k", ctypes.c_void_p),
                ("top_p", ctypes.c_void_p), ("min_p", ctypes.c_void_p)]


class MoeError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {_status_string(status)} ({status})")


_lib = None


def load_library(path: str = LIB_PATH):
    """dlopen the in-tree library (raises if it was not built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it first (bit_affine_quantized_gb300.build_library())")
    lib = ctypes.CDLL(path)
    P, I, Z, V = ctypes.POINTER, ctypes.c_int, ctypes.c_size_t, ctypes.c_void_p
    proto = {
        "moe_status_string": (ctypes.c_char_p, [I]),
        "moe_create": (I, [P(V)]),
        "moe_destroy": (I, [V]),
        "moe_check_weights": (I, [P(LayerWeights)]),
        "moe_workspace_bytes": (Z, [P(Dims), I]),
        "moe_router_topk": (I, [V, V, I, P(LayerWeights), V, V, V, V, Z, V]),
        "moe_route_sort": (I, [V, V, I, P(Dims), V, V, V, V, V]),
        "moe_expert_ffn": (I, [V, V, I, V, V, P(LayerWeights), I, V, V, Z, V]),
        "moe_layer_forward": (I, [V, V, I, P(LayerWeights), V, V, V, V, V, Z, V]),
        "moe_layer_forward_residual": (I, [V, V, I, P(LayerWeights), V, V, V, V, V, Z, V]),
        "moe_selftest_wait_timeout": (I, [V, ctypes.c_ulonglong, V]),
        "moe_set_trace": (I, [V, V, I]),
        "moe_layer_forward_static": (I, [V, P(LayerWeights), V, V, V, V, V]),
        "moe_static_get_error": (I, [P(I)]),
        "moe_selftest_skip_arrival": (I, [V, I, ctypes.c_ulonglong]),
        "moe_layer_forward_stack": (I, [V, V, I, P(LayerWeights), V, Z, V]),
        "moe_get_error": (I, [V, P(I)]),
        "moe_head_forward": (I, [V, V, I, P(HeadWeights), ctypes.c_float, V, V, V]),
        "moe_embed": (I, [V, V, I, P(HeadWeights), V, V]),
        "moe_dense_forward": (I, [V, V, I, P(HeadWeights), V, V, V]),
        "moe_cache_create": (I, [I, I, P(V)]),
        "moe_cache_destroy": (None, [V]),
        "moe_cache_lookup": (I, [V, I, V, I, V, V, V, P(I)]),
        "moe_cache_stats": (I, [V, I, P(ctypes.c_longlong), P(ctypes.c_longlong)]),
        "moe_cache_slot_expert": (I, [V, I, I]),
        "moe_cache_slots": (I, [V]),
        "moe_layer_forward_offload": (I, [V, V, I, V, P(LayerWeights), V, V, Z, V]),
        "moe_norm_quant": (I, [V, V, V, I, I, V, ctypes.c_float, V, V, V, V, V]),
        "moe_qdense_workspace_bytes": (Z, [P(QdenseWeights), I]),
        "moe_qdense_forward": (I, [V, V, V, I, P(QdenseWeights), ctypes.c_float, V, V, V, Z, V]),
        "moe_logits_process": (I, [V, V, Z, I, I, P(LogitRules), V, Z, V, V]),
        "moe_kv_append": (I, [V, V, Z, I, V, Z, V, Z, I, V, V, P(KvCache), V, I, V, Z, V]),
        "moe_kv_read": (I, [V, P(KvCache), V, V, I, V, Z, V, Z, V]),
        "moe_kv_attend_workspace_bytes": (Z, [P(KvCache), I]),
        "moe_kv_attend": (I, [V, V, Z, P(KvCache), V, I, ctypes.c_float, ctypes.c_float, I, V, Z, V, V, Z, V]),
        "moe_sample": (I, [V, V, Z, I, I, P(SampleRules), V, V, V]),
        "moe_prompt_workspace_bytes": (Z, [P(Dims), I]),
        "moe_layer_forward_prompt": (I, [V, V, I, P(LayerWeights), V, V, V, V, V, Z, V]),
    }
    for name, (res, args) in proto.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def _status_string(status: int) -> str:
    try:
        return load_library().moe_status_string(status).decode()
    except Exception:  # library not loadable: still report the number
        return "status"


def header_symbols(path: str = HEADER) -> list[str]:
    """Names of the functions include/moe.h declares."""
    with open(path) as f:
        text = f.read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(moe_[a-z_]+)\s*\(", text)))


def _ptr(t):
    """Device (or host) address of a tensor, or None."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


_raw_stream = None


def _stream(stream, dev=None):
    """Handle of a stream; without one, of device dev's current stream (the current device's)."""
    if stream is None:
        return (_raw_stream or _find_raw_stream())(dev)
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _find_raw_stream():
    """Sets _raw_stream, the handle of a device's current stream: torch's own
    getter where there is one (a Stream object costs several times as much as a
    small call), else through torch.cuda."""
    global _raw_stream
    import torch
    torch.cuda.current_stream()  # torch's device state is set up
    get, now = getattr(torch._C, "_cuda_getCurrentRawStream", None), getattr(torch._C, "_cuda_getDevice", None)
    if get and now:
        _raw_stream = lambda dev: get(now() if dev is None else dev)
    else:
        _raw_stream = lambda dev: torch.cuda.current_stream(dev).cuda_stream
    return _raw_stream


def make_dims(hidden: int, inter: int, n_experts: int, top_k: int, group: int = 64) -> Dims:
    return Dims(hidden, inter, n_experts, top_k, group)


def make_layer_weights(dims: Dims, router_q: int, router_s: int, router_b: int, experts: int, expert_stride: int,
                       layout: dict, shared: int, logit_bias=None, router_scale=None,
                       per_expert_scale=None, post_norm=None, layer_scalar=None) -> LayerWeights:
    """LayerWeights from device addresses; `layout` maps gate_q .. down_b to byte offsets.

    Optional entries (device address, CUDA tensor or None): logit_bias fp32
    [E]; router_scale bf16 [H] and per_expert_scale fp32 [E], the router's
    learned scales; post_norm bf16 [H] and layer_scalar fp32 [1], the layer
    tail, which only the residual calls apply."""
    return LayerWeights(dims, QMat(router_q, router_s, router_b), experts, expert_stride,
                        BlobLayout(*[layout[n] for n in _BLOB_FIELDS]), shared, _ptr(logit_bias),
                        _ptr(router_scale), _ptr(per_expert_scale), _ptr(post_norm), _ptr(layer_scalar))


def make_head_weights(vocab: int, hidden: int, q: int, scales: int, biases: int) -> HeadWeights:
    """HeadWeights from device addresses (or CUDA tensors) of the tied head."""
    return HeadWeights(vocab, hidden, QMat(_ptr(q), _ptr(scales), _ptr(biases)))


_current_device = None


def _device() -> int:
    """The current device, on which the calls of the batched path launch and
    their tensors have to be."""
    return (_current_device or _find_current_device())()


def _find_current_device():
    global _current_device
    import torch
    torch.cuda.current_device()  # torch's device state is set up
    _current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
    return _current_device


def _data(t, what: str, types, n: int, dev: int, width: int = 1):
    """Device address of a tensor on device dev that a call of the batched path
    takes (None stays None), after a check of its type (one of `types`), layout
    and size: n values, or more in rows of `width` (1: a vector)."""
    if t is None:
        return None
    if t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{what}: a contiguous CUDA tensor on device {max(dev, 0)} is wanted, one on {t.device} given")
    if t.dtype not in types:
        raise ValueError(f"{what}: {t.dtype} given, {types[0]} wanted")
    if t.numel() != n:  # (exactly n values lie in memory as the call reads them; t.shape costs more than t.numel())
        _check_rows(t.shape, what, n, width)
    return t.data_ptr()


def _check_rows(shape, what: str, n: int, width: int):
    """Refuses a shape of fewer than n values, or whose last dimensions do not
    make up rows of `width` (flat tensors have no rows; width 1: a vector, the one
    row or column of a matrix too; 0: any)."""
    if math.prod(shape) < n:
        raise ValueError(f"{what}: {math.prod(shape)} elements given, {n} wanted")
    if width == 1:
        fits = max(shape, default=1) == math.prod(shape)
    else:
        size, at = 1, len(shape)
        while at > 0 and size < width:
            at -= 1
            size *= shape[at]
        fits = size == width or len(shape) == 1
    if width and not fits:
        raise ValueError(f"{what}: {tuple(shape)} given, {'a vector' if width == 1 else f'rows of {width}'} wanted")


_DTYPES = {}


def _fill_dtypes():
    import torch
    _DTYPES.update(b16=(torch.bfloat16, torch.int16, torch.uint16), f32=(torch.float32,),
                   i32=(torch.int32, torch.uint32), i8=(torch.int8,), u8=(torch.uint8,))
    return _DTYPES


def _rows(t, what: str, n_rows: int, width: int, dev: int):
    """Device address and row stride of an fp32 matrix on device dev of at least
    n_rows rows and `width` columns."""
    if t.get_device() != dev or t.dtype not in (_DTYPES or _fill_dtypes())["f32"] or t.dim() != 2 \
            or t.shape[0] < n_rows or t.shape[1] < width or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{what}: a float32 matrix on CUDA device {dev} of at least {n_rows} x {width} with adjacent "
                         f"columns is wanted")
    return t.data_ptr(), t.stride(0) if t.shape[0] > 1 else max(width, t.stride(0))


def make_qdense_weights(channels: int, width: int, q, scales) -> QdenseWeights:
    """QdenseWeights from CUDA tensors: q int8 [channels, width], scales fp32
    [channels].  The result keeps the tensors alive."""
    dev, k = max(q.get_device(), 0), _DTYPES or _fill_dtypes()
    w = QdenseWeights(channels, width, _data(q, "q", k["i8"], channels * width, dev, width),
                      _data(scales, "scales", k["f32"], channels, dev))
    _check_rows(q.shape, "q", channels * width, width)
    w.keep, w.device = (q, scales), dev
    return w


def make_logit_rules(history=None, history_len=None, prompt_len=None, repetition=None, presence=None, frequency=None,
                     bias_ids=None, bias_values=None, bias_len=None, mask=None) -> LogitRules:
    """LogitRules from CUDA tensors, any of which may be left out with what
    belongs to it: history int32 [T, L] with history_len (and prompt_len)
    int32 [T] and the penalties fp32 [T]; bias_ids int32 and bias_values fp32
    [T, B] with bias_len int32 [T]; mask int32 words [T, W], or [W] for one
    mask of every row.  The result keeps the tensors alive."""
    rows = []
    for name, t in (("history", history), ("bias_ids", bias_ids)):
        if t is not None:
            if t.dim() != 2:
                raise ValueError(f"{name}: a matrix is wanted")
            rows.append(t.shape[0])
    if mask is not None:
        if mask.dim() not in (1, 2):
            raise ValueError("mask: a vector or a matrix is wanted")
        if mask.dim() == 2:
            rows.append(mask.shape[0])
    T = min(rows) if rows else None
    n = T or 0
    L = history.shape[1] if history is not None else 0
    B = bias_ids.shape[1] if bias_ids is not None else 0
    every = (history, history_len, prompt_len, repetition, presence, frequency, bias_ids, bias_values, bias_len, mask)
    dev = max((t.get_device() for t in every if t is not None), default=-1)
    dev = max(dev, 0)
    k = _DTYPES or _fill_dtypes()
    i32, f32 = k["i32"], k["f32"]
    r = LogitRules(_data(history, "history", i32, n * L, dev, L), _data(history_len, "history_len", i32, n, dev),
                   _data(prompt_len, "prompt_len", i32, n, dev), L, _data(repetition, "repetition", f32, n, dev),
                   _data(presence, "presence", f32, n, dev), _data(frequency, "frequency", f32, n, dev),
                   _data(bias_ids, "bias_ids", i32, n * B, dev, B),
                   _data(bias_values, "bias_values", f32, n * B, dev, B), _data(bias_len, "bias_len", i32, n, dev), B,
                   _data(mask, "mask", i32, 0, dev, 0),
                   mask.shape[1] if mask is not None and mask.dim() == 2 else 0)
    if bias_values is not None:
        _check_rows(bias_values.shape, "bias_values", n * B, B)
    r.device = dev if any(t is not None for t in every) else None
    r.rows, r.words = T, mask.shape[-1] if mask is not None else None
    r.keep = every
    return r


def _heads(t, what: str, n_rows: int, heads: int, dim: int, dev: int):
    """Device address and row stride of bf16 rows on device dev: a tensor of at
    least n_rows x heads x dim, or x (heads * dim), whose rows may lie apart."""
    stride = t.stride()
    if t.get_device() == dev and t.dtype in _DTYPES["b16"]:
        if len(stride) == 3:
            n, h, d = t.shape
            if h == heads and d == dim and stride[2] == 1 and (stride[1] == dim or h == 1) and n >= n_rows:
                return t.data_ptr(), stride[0] if n > 1 else heads * dim
        elif len(stride) == 2:
            n, w = t.shape
            if w == heads * dim and stride[1] == 1 and n >= n_rows:
                return t.data_ptr(), stride[0] if n > 1 else w
    raise ValueError(f"{what}: {tuple(t.shape)} {t.dtype} with strides {stride} on {t.device} given, at least {n_rows} bf16 "
                     f"rows of {heads} x {dim} adjacent values on CUDA device {max(dev, 0)} are wanted")


def make_kv_cache(k, v, table, k_scales=None, v_scales=None) -> KvCache:
    """KvCache from CUDA tensors: k and v [n_pages, kv_heads, page_rows,
    head_dim], bf16, or int8 with k_scales and v_scales fp32 [n_pages,
    kv_heads, page_rows]; table int32 [n_seqs, pages].  The result keeps the
    tensors alive."""
    if k.dim() != 4:
        raise ValueError(f"k: [n_pages, kv_heads, page_rows, head_dim] is wanted, {tuple(k.shape)} given")
    if (k_scales is None) != (v_scales is None):
        raise ValueError("k_scales, v_scales: both or neither are wanted")
    types, dev = _DTYPES or _fill_dtypes(), max(k.get_device(), 0)
    kind = types["b16"] if k_scales is None else types["i8"]
    for name, t, like in (("v", v, k.shape), ("k_scales", k_scales, k.shape[:3]), ("v_scales", v_scales, k.shape[:3])):
        if t is not None and t.shape != like:
            raise ValueError(f"{name}: {tuple(t.shape)} given, {tuple(like)} wanted")
    if table.dim() != 2:
        raise ValueError(f"table: a matrix is wanted, {tuple(table.shape)} given")
    rows = math.prod(k.shape[:3])
    c = KvCache(*k.shape, _data(k, "k", kind, k.numel(), dev, 0), _data(v, "v", kind, k.numel(), dev, 0),
                _data(k_scales, "k_scales", types["f32"], rows, dev, 0),
                _data(v_scales, "v_scales", types["f32"], rows, dev, 0),
                _data(table, "table", types["i32"], table.numel(), dev, 0), *table.shape)
    c.keep, c.device = (k, v, k_scales, v_scales, table), dev
    return c


def make_sample_rules(uniform, temperature=None, top_k=None, top_p=None, min_p=None) -> SampleRules:
    """SampleRules from CUDA tensors of a value per row: uniform, temperature,
    top_p and min_p fp32, top_k int32.  The result keeps the tensors alive."""
    k, dev, n = _DTYPES or _fill_dtypes(), max(uniform.get_device(), 0), uniform.numel()
    every = (uniform, temperature, top_k, top_p, min_p)
    r = SampleRules(*[_data(t, name, k["i32"] if name == "top_k" else k["f32"], n, dev) for t, name in
                      zip(every, ("uniform", "temperature", "top_k", "top_p", "min_p"))])
    r.keep, r.device, r.rows = every, dev, n
    return r


def layer_forward_static(x, w: LayerWeights, y, ids_out=None, logits_out=None, weights_out=None, stream=None):
    """moe_layer_forward_static: one token, no handle, no workspace.

    For hosts that cannot allocate device memory; the library's scratch for
    this call is a fixed static device array (see include/moe.h)."""
    st = load_library().moe_layer_forward_static(_ptr(x), ctypes.byref(w), _ptr(y), _ptr(ids_out), _ptr(logits_out),
                                                 _ptr(weights_out), _stream(stream))
    if st != MOE_OK:
        raise MoeError(st, "moe_layer_forward_static")


def static_get_error() -> int:
    """moe_static_get_error: the device-side status of the static calls on the
    current device since the last read (waits for the device; clears it)."""
    st = ctypes.c_int(0)
    rc = load_library().moe_static_get_error(ctypes.byref(st))
    if rc != MOE_OK:
        raise MoeError(rc, "moe_static_get_error")
    return st.value


class ExpertCache:
    """Host-side slot policy of the expert offload (moe_cache_*): n_layers
    layers of n_slots slots, least frequently used eviction, recency breaking
    ties."""

    def __init__(self, n_layers: int, n_slots: int = 16):
        self.lib = load_library()
        self.c = ctypes.c_void_p()
        st = self.lib.moe_cache_create(n_layers, n_slots, ctypes.byref(self.c))
        if st:
            raise MoeError(st, "moe_cache_create")
        self.n_layers, self.n_slots = n_layers, n_slots

    def lookup(self, layer: int, ids):
        """One step for a sequence of selected expert ids: (slots, [(slot,
        expert) loads])."""
        n = len(ids)
        a = (ctypes.c_int32 * n)(*ids)
        sl, ls, li = (ctypes.c_int32 * n)(), (ctypes.c_int32 * n)(), (ctypes.c_int32 * n)()
        nl = ctypes.c_int()
        st = self.lib.moe_cache_lookup(self.c, layer, a, n, sl, ls, li, ctypes.byref(nl))
        if st:
            raise MoeError(st, "moe_cache_lookup")
        return list(sl), [(ls[i], li[i]) for i in range(nl.value)]

    def stats(self, layer: int):
        h, m = ctypes.c_longlong(), ctypes.c_longlong()
        st = self.lib.moe_cache_stats(self.c, layer, ctypes.byref(h), ctypes.byref(m))
        if st:
            raise MoeError(st, "moe_cache_stats")
        return h.value, m.value

    def slot_expert(self, layer: int, slot: int) -> int:
        return self.lib.moe_cache_slot_expert(self.c, layer, slot)

    def close(self):
        if self.c:
            self.lib.moe_cache_destroy(self.c)
            self.c = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class Moe:
    """One library handle (device error word + router counter) on the current device."""

    def __init__(self):
        self.lib = load_library()
        h = ctypes.c_void_p()
        st = self.lib.moe_create(ctypes.byref(h))
        if st != MOE_OK:
            raise MoeError(st, "moe_create")
        self.h = h

    def close(self):
        if self.h:
            self.lib.moe_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def _check(self, st, what):
        if st != MOE_OK:
            raise MoeError(st, what)

    def workspace_bytes(self, dims: Dims, n_tokens: int) -> int:
        return int(self.lib.moe_workspace_bytes(ctypes.byref(dims), n_tokens))

    def router_topk(self, x, n_tokens, w: LayerWeights, ids, weights, ws, logits=None, stream=None):
        self._check(self.lib.moe_router_topk(self.h, _ptr(x), n_tokens, ctypes.byref(w), _ptr(logits), _ptr(ids),
                                             _ptr(weights), _ptr(ws), ws.numel() * ws.element_size(),
                                             _stream(stream)), "moe_router_topk")

    def route_sort(self, ids, n_tokens, dims: Dims, counts, offsets, perm, pos, stream=None):
        self._check(self.lib.moe_route_sort(self.h, _ptr(ids), n_tokens, ctypes.byref(dims), _ptr(counts),
                                            _ptr(offsets), _ptr(perm), _ptr(pos), _stream(stream)), "moe_route_sort")

    def expert_ffn(self, x, n_tokens, ids, weights, w: LayerWeights, y, ws, include_shared=True, stream=None):
        self._check(self.lib.moe_expert_ffn(self.h, _ptr(x), n_tokens, _ptr(ids), _ptr(weights), ctypes.byref(w),
                                            1 if include_shared else 0, _ptr(y), _ptr(ws),
                                            ws.numel() * ws.element_size(), _stream(stream)), "moe_expert_ffn")

    def layer_forward(self, x, n_tokens, w: LayerWeights, y, ws, ids_out=None, logits_out=None, weights_out=None,
                      stream=None):
        self._check(self.lib.moe_layer_forward(self.h, _ptr(x), n_tokens, ctypes.byref(w), _ptr(y), _ptr(ids_out),
                                               _ptr(logits_out), _ptr(weights_out), _ptr(ws),
                                               ws.numel() * ws.element_size(), _stream(stream)), "moe_layer_forward")

    def layer_forward_residual(self, hidden, n_tokens, w: LayerWeights, ws, y_out=None, x_out=None, ids_out=None,
                               logits_out=None, stream=None):
        """One layer of a residual stack: hidden <- hidden + MoE(rmsnorm(hidden))
        in place, or with the layer's tail hidden <- lambda * (hidden +
        post_norm * y / rms(y)); y_out / x_out receive the block output and
        its normalised input."""
        self._check(self.lib.moe_layer_forward_residual(self.h, _ptr(hidden), n_tokens, ctypes.byref(w), _ptr(y_out),
                                                        _ptr(x_out), _ptr(ids_out), _ptr(logits_out), _ptr(ws),
                                                        ws.numel() * ws.element_size(), _stream(stream)),
                    "moe_layer_forward_residual")

    def prompt_workspace_bytes(self, dims: Dims, n_rows: int) -> int:
        return int(self.lib.moe_prompt_workspace_bytes(ctypes.byref(dims), n_rows))

    def layer_forward_prompt(self, hidden, n_rows, w: LayerWeights, ws, y_out=None, x_out=None, ids_out=None,
                             logits_out=None, stream=None):
        """One residual layer on a whole prompt of up to 4096 rows
        (moe_layer_forward_prompt): the same function as
        layer_forward_residual, row by row, with the expert work grouped over
        all rows; ws of prompt_workspace_bytes(dims, n_rows) bytes."""
        self._check(self.lib.moe_layer_forward_prompt(self.h, _ptr(hidden), n_rows, ctypes.byref(w), _ptr(y_out),
                                                      _ptr(x_out), _ptr(ids_out), _ptr(logits_out), _ptr(ws),
                                                      ws.numel() * ws.element_size(), _stream(stream)),
                    "moe_layer_forward_prompt")

    def layer_forward_stack(self, hidden, layers, ws, stream=None):
        """Single-token layers of a residual stack in one call (hidden bf16 [H]
        updated in place); `layers` is a sequence of LayerWeights."""
        arr = (LayerWeights * len(layers))(*layers)
        self._check(self.lib.moe_layer_forward_stack(self.h, _ptr(hidden), len(layers), arr, _ptr(ws),
                                                     ws.numel() * ws.element_size(), _stream(stream)),
                    "moe_layer_forward_stack")

    def layer_forward_offload(self, hidden, cache: "ExpertCache", layer: int, w: LayerWeights, slots, ws,
                              stream=None):
        """One single-token residual layer with its routed experts in host
        memory (w.experts: pinned host memory), filling the layer's device
        `slots` through `cache` (moe_layer_forward_offload)."""
        self._check(self.lib.moe_layer_forward_offload(self.h, cache.c, layer, _ptr(hidden), ctypes.byref(w),
                                                       _ptr(slots), _ptr(ws), ws.numel() * ws.element_size(),
                                                       _stream(stream)), "moe_layer_forward_offload")

    def head_forward(self, x, n_tokens, hw: HeadWeights, softcap: float = 30.0, logits=None, tokens=None,
                     stream=None):
        """The tied head on n_tokens (<= 8) rows of x: logits (fp32 [T, V])
        and/or greedy tokens (int32 [T])."""
        self._check(self.lib.moe_head_forward(self.h, _ptr(x), n_tokens, ctypes.byref(hw), ctypes.c_float(softcap),
                                              _ptr(logits), _ptr(tokens), _stream(stream)), "moe_head_forward")

    def dense_forward(self, x, n_tokens, w: HeadWeights, y=None, y32=None, stream=None):
        """A dense 4-bit affine projection y = W x on n_tokens (<= 8) rows:
        bf16 [T, N] and/or fp32 [T, N] outputs."""
        self._check(self.lib.moe_dense_forward(self.h, _ptr(x), n_tokens, ctypes.byref(w), _ptr(y), _ptr(y32),
                                               _stream(stream)), "moe_dense_forward")

    def norm_quant(self, hidden, n_rows, q, scales, y=None, norm=None, eps: float = 1e-6, hidden_out=None, x_out=None,
                   stream=None):
        """Residual addition, root-mean-square norm and 8-bit rows of n_rows
        rows (moe_norm_quant): q int8 [T, H] and scales fp32 [T] of the
        normalised hidden (+ y) bf16 [T, H], whose sum goes to hidden_out and
        whose bf16 rows go to x_out where these are given.  H is q's last
        dimension."""
        H, dev, k = q.shape[-1], _device(), _DTYPES or _fill_dtypes()
        n, b16 = n_rows * H, k["b16"]
        st = self.lib.moe_norm_quant(self.h, _data(hidden, "hidden", b16, n, dev, H), _data(y, "y", b16, n, dev, H),
                                     n_rows, H, _data(norm, "norm", b16, H, dev), eps,
                                     _data(hidden_out, "hidden_out", b16, n, dev, H), _data(q, "q", k["i8"], n, dev, H),
                                     _data(scales, "scales", k["f32"], n_rows, dev),
                                     _data(x_out, "x_out", b16, n, dev, H), _stream(stream, dev))
        if st:
            self._check(st, "moe_norm_quant")

    def qdense_workspace_bytes(self, w: QdenseWeights, n_rows: int) -> int:
        return int(self.lib.moe_qdense_workspace_bytes(ctypes.byref(w), n_rows))

    def qdense_forward(self, x, x_scales, n_rows, w: QdenseWeights, ws=None, y=None, y32=None, softcap: float = 0.0,
                       stream=None):
        """A dense 8-bit projection of n_rows 8-bit rows (moe_qdense_forward):
        x int8 [T, K] with x_scales fp32 [T]; outputs y bf16 and/or y32 fp32
        [T, N], through a softcap if one is given; ws of
        qdense_workspace_bytes(w, n_rows) bytes."""
        dev, k = _device(), _DTYPES or _fill_dtypes()
        if w.device is not None and w.device != dev:
            raise ValueError(f"weights on CUDA device {w.device} given, the current device is {dev}")
        f32, N, K = k["f32"], w.channels, w.width
        n, ws_bytes = n_rows * N, 0 if ws is None else ws.numel()
        st = self.lib.moe_qdense_forward(self.h, _data(x, "x", k["i8"], n_rows * K, dev, K),
                                         _data(x_scales, "x_scales", f32, n_rows, dev), n_rows, ctypes.byref(w),
                                         softcap, _data(y, "y", k["b16"], n, dev, N), _data(y32, "y32", f32, n, dev, N),
                                         _data(ws, "ws", k["u8"], ws_bytes, dev), ws_bytes, _stream(stream, dev))
        if st:
            self._check(st, "moe_qdense_forward")

    def logits_process(self, logits, n_rows, vocab, rules: LogitRules, out=None, tokens=None, stream=None):
        """Penalties, biases, a mask (rules: make_logit_rules) and the greedy
        token of n_rows rows of logits (moe_logits_process): fp32 matrices
        whose rows may lie apart (out may be logits itself), tokens int32."""
        if rules.rows is not None and rules.rows < n_rows:
            raise ValueError(f"rules for {rules.rows} rows given, {n_rows} wanted")
        if rules.words is not None and rules.words < (vocab + 31) // 32:
            raise ValueError(f"mask: {rules.words} words given, {(vocab + 31) // 32} wanted")
        dev = _device()
        if rules.device is not None and rules.device != dev:
            raise ValueError(f"rules on CUDA device {rules.device} given, the current device is {dev}")
        at, ld = _rows(logits, "logits", n_rows, vocab, dev)
        to, ld_out = _rows(out, "out", n_rows, vocab, dev) if out is not None else (None, 0)
        st = self.lib.moe_logits_process(self.h, at, ld, n_rows, vocab, ctypes.byref(rules), to, ld_out,
                                         _data(tokens, "tokens", _DTYPES["i32"], n_rows, dev), _stream(stream, dev))
        if st:
            self._check(st, "moe_logits_process")

    def _on_device(self, what, dev):
        now = _device()
        if dev is not None and dev != now:
            raise ValueError(f"{what} on CUDA device {dev} given, the current device is {now}")
        return now

    def kv_append(self, k, v, positions, cache: KvCache, seqs=None, q=None, q_out=None, inv_freq=None, stream=None):
        """Rotary positions on q and k (inv_freq fp32 [r / 2]: the first r
        dimensions of a head; None: none), q_out <- q, and k and v into the
        cache (moe_kv_append).  A row per entry of positions (int32, as seqs;
        None: row t is of sequence t): q bf16 [T, q_heads, head_dim], k and v
        [T, kv_heads, head_dim], or with the last two dimensions as one; rows may
        lie apart, as the parts of one projection's output do."""
        dev, types = self._on_device("cache", cache.device), _DTYPES or _fill_dtypes()
        T, H, D, i32 = positions.numel(), cache.kv_heads, cache.head_dim, types["i32"]
        (kp, lk), (vp, lv) = _heads(k, "k", T, H, D, dev), _heads(v, "v", T, H, D, dev)
        if q is None or q_out is None:  # (the call refuses one without the other)
            q_heads, qp, lq, op, lo = 0, _ptr(q), 0, _ptr(q_out), 0
        else:
            q_heads = q.shape[1] if q.dim() == 3 else q.shape[-1] // D
            (qp, lq), (op, lo) = _heads(q, "q", T, q_heads, D, dev), _heads(q_out, "q_out", T, q_heads, D, dev)
        rot = 0 if inv_freq is None else 2 * inv_freq.numel()
        st = self.lib.moe_kv_append(self.h, qp, lq, q_heads, kp, lk, vp, lv, T,
                                    None if seqs is None else _data(seqs, "seqs", i32, T, dev),
                                    _data(positions, "positions", i32, T, dev), ctypes.byref(cache),
                                    _data(inv_freq, "inv_freq", types["f32"], rot // 2, dev), rot, op, lo,
                                    _stream(stream, dev))
        if st:
            self._check(st, "moe_kv_append")

    def kv_read(self, cache: KvCache, positions, k_out=None, v_out=None, seqs=None, stream=None):
        """Rows of the cache as bf16 [T, kv_heads, head_dim], one per entry of
        positions (moe_kv_read; seqs None: row t is of sequence t)."""
        dev, types = self._on_device("cache", cache.device), _DTYPES or _fill_dtypes()
        T, H, D = positions.numel(), cache.kv_heads, cache.head_dim
        kp, lk = (None, 0) if k_out is None else _heads(k_out, "k_out", T, H, D, dev)
        vp, lv = (None, 0) if v_out is None else _heads(v_out, "v_out", T, H, D, dev)
        st = self.lib.moe_kv_read(self.h, ctypes.byref(cache), _data(seqs, "seqs", types["i32"], T, dev),
                                  _data(positions, "positions", types["i32"], T, dev), T, kp, lk, vp, lv,
                                  _stream(stream, dev))
        if st:
            self._check(st, "moe_kv_read")

    def kv_attend_workspace_bytes(self, cache: KvCache, q_heads: int) -> int:
        return int(self.lib.moe_kv_attend_workspace_bytes(ctypes.byref(cache), q_heads))

    def kv_attend(self, q, lengths, cache: KvCache, out, ws, scale: float, softcap: float = 0.0, window: int = 0,
                  lse=None, stream=None):
        """Attention of one new token per sequence of the cache's table
        (moe_kv_attend): q and out bf16 [n_seqs, q_heads, head_dim], or with the
        last two dimensions as one, lengths int32 and lse fp32 [n_seqs,
        q_heads]; ws of kv_attend_workspace_bytes(cache, q_heads) bytes."""
        dev, types = self._on_device("cache", cache.device), _DTYPES or _fill_dtypes()
        n, D = cache.n_seqs, cache.head_dim
        q_heads = q.shape[1] if q.dim() == 3 else q.shape[-1] // D
        (qp, lq), (op, lo) = _heads(q, "q", n, q_heads, D, dev), _heads(out, "out", n, q_heads, D, dev)
        ws_bytes = ws.numel()
        st = self.lib.moe_kv_attend(self.h, qp, lq, ctypes.byref(cache),
                                    _data(lengths, "lengths", types["i32"], n, dev), q_heads, scale, softcap, window,
                                    op, lo, _data(lse, "lse", types["f32"], n * q_heads, dev, q_heads),
                                    _data(ws, "ws", types["u8"], ws_bytes, dev), ws_bytes, _stream(stream, dev))
        if st:
            self._check(st, "moe_kv_attend")

    def sample(self, logits, n_rows, vocab, rules: SampleRules, tokens, logprobs=None, stream=None):
        """A token per row of logits (an fp32 matrix whose rows may lie apart)
        through the filters of rules (make_sample_rules), and the log of its
        share of what remained (moe_sample): tokens int32, logprobs fp32."""
        if rules.rows is not None and rules.rows < n_rows:
            raise ValueError(f"rules for {rules.rows} rows given, {n_rows} wanted")
        dev, types = self._on_device("rules", rules.device), _DTYPES or _fill_dtypes()
        at, ld = _rows(logits, "logits", n_rows, vocab, dev)
        st = self.lib.moe_sample(self.h, at, ld, n_rows, vocab, ctypes.byref(rules),
                                 _data(tokens, "tokens", types["i32"], n_rows, dev),
                                 _data(logprobs, "logprobs", types["f32"], n_rows, dev), _stream(stream, dev))
        if st:
            self._check(st, "moe_sample")

    def embed(self, ids, n, hw: HeadWeights, out, stream=None):
        """Tied embedding rows (bf16 [n, H]) of int32 token ids on the device."""
        self._check(self.lib.moe_embed(self.h, _ptr(ids), n, ctypes.byref(hw), _ptr(out), _stream(stream)),
                    "moe_embed")

    def set_trace(self, buffer=None, n_launches: int = 0):
        """Record per-launch device timestamps into `buffer` (u64 x 4 x n)."""
        self._check(self.lib.moe_set_trace(self.h, _ptr(buffer), n_launches), "moe_set_trace")

    def selftest_wait_timeout(self, limit_ns: int, stream=None):
        self._check(self.lib.moe_selftest_wait_timeout(self.h, limit_ns, _stream(stream)), "moe_selftest_wait_timeout")

    def selftest_skip_arrival(self, block: int, limit_ns: int):
        """Arms the next fused single-token launch: `block` withholds its
        barrier arrival, every wait gives up after limit_ns (failure test)."""
        self._check(self.lib.moe_selftest_skip_arrival(self.h, block, limit_ns), "moe_selftest_skip_arrival")

    def get_error(self) -> int:
        st = ctypes.c_int(0)
        self._check(self.lib.moe_get_error(self.h, ctypes.byref(st)), "moe_get_error")
        return st.value


def layer_weights_from(dims: Dims, addr: dict) -> LayerWeights:
    """LayerWeights from a dict with router_q/router_s/router_b/experts/stride/
    shared/layout entries and optional logit_bias/router_scale/per_expert_scale/
    post_norm/layer_scalar entries (device addresses and byte offsets)."""
    return make_layer_weights(dims, addr["router_q"], addr["router_s"], addr["router_b"], addr["experts"],
                              addr["stride"], addr["layout"], addr["shared"], addr.get("logit_bias"),
                              addr.get("router_scale"), addr.get("per_expert_scale"), addr.get("post_norm"),
                              addr.get("layer_scalar"))
