"""GB300-native single-pass block drafting with target-context injection and
lossless verification.

This module is a thin ctypes binding over ``libdflash.so`` (built from
``csrc/`` by ``build.py``).  Every function carries the name of the C entry
point it calls and only marshals arguments: torch tensors supply device memory
and the current CUDA stream; all computation runs in the library's kernels.
There is no fallback: if the library is missing, every call raises.
"""

import ctypes
import os
import re
import struct
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libdflash.so")
HEADER_PATH = os.path.join(os.path.dirname(_HERE), "include", "dflash.h")

DFLASH_VERIFY_GREEDY = 0
DFLASH_VERIFY_SAMPLED = 1

ERRORS = {
    -1: "DFLASH_ERR_ARG", -2: "DFLASH_ERR_SHAPE", -3: "DFLASH_ERR_ALIGN",
    -4: "DFLASH_ERR_UNSUPPORTED", -5: "DFLASH_ERR_LAUNCH", -6: "DFLASH_ERR_DEVICE_TIMEOUT",
    -7: "DFLASH_ERR_WORKSPACE", -8: "DFLASH_ERR_CUDA", -9: "DFLASH_ERR_RANGE",
}


class DflashError(RuntimeError):
    def __init__(self, code, where):
        self.code = code
        self.name = ERRORS.get(code, str(code))
        super().__init__(f"{where}: {self.name} ({dflash_strerror(code)})")


class dflash_config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in (
        "hidden", "n_q_heads", "n_kv_heads", "head_dim", "ffn", "vocab", "n_layers", "n_feat",
        "feat_dim", "window", "gamma_max", "topk_max", "batch_max", "append_max")] + [
        ("rope_theta", ctypes.c_float), ("eps", ctypes.c_float), ("mask_id", ctypes.c_int),
        ("weight_format", ctypes.c_int)]


DFLASH_WEIGHTS_BF16 = 0
DFLASH_WEIGHTS_E4M3 = 1

LAYER_MATRICES = ("w_qkv", "w_o", "w_gate", "w_up", "w_down")


class dflash_layer_weights(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in (
        "g_attn", "w_qkv", "w_o", "g_mlp", "w_gate", "w_up", "w_down",
        "s_qkv", "s_o", "s_gate", "s_up", "s_down")]


class dflash_weights(ctypes.Structure):
    _fields_ = [("embed", ctypes.c_void_p), ("lm_head", ctypes.c_void_p), ("w_c", ctypes.c_void_p),
                ("g_c", ctypes.c_void_p), ("g_final", ctypes.c_void_p),
                ("layers", ctypes.POINTER(dflash_layer_weights)), ("s_lm_head", ctypes.c_void_p)]


class dflash_sampling(ctypes.Structure):
    _fields_ = [("temperature", ctypes.c_float), ("top_p", ctypes.c_float),
                ("seeds", ctypes.c_void_p), ("step", ctypes.c_uint64)]


DFLASH_TYPE_BF16, DFLASH_TYPE_F16, DFLASH_TYPE_F32 = 0, 1, 2
DFLASH_CACHE_BF16, DFLASH_CACHE_F16, DFLASH_CACHE_E4M3 = 0, 1, 2

_TYPES = {torch.bfloat16: DFLASH_TYPE_BF16, torch.float16: DFLASH_TYPE_F16,
          torch.float32: DFLASH_TYPE_F32}
_CACHES = {torch.bfloat16: DFLASH_CACHE_BF16, torch.float16: DFLASH_CACHE_F16,
           torch.float8_e4m3fn: DFLASH_CACHE_E4M3, torch.uint8: DFLASH_CACHE_E4M3}


class dflash_paged_cache(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("k_pages", "v_pages", "k_scale", "v_scale")] + [
        (n, ctypes.c_longlong) for n in ("k_page_stride", "v_page_stride")] + [
        (n, ctypes.c_int) for n in ("n_pages", "n_kv_heads", "page_size", "head_dim", "format")] + [
        ("maps", ctypes.c_void_p)]


class dflash_paged_maps(ctypes.Structure):
    _fields_ = [("opaque", ctypes.c_ulonglong * 48)]


class dflash_paged_batch(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("row_start", "kv_len", "page_table")] + [
        ("table_stride", ctypes.c_longlong)] + [
        (n, ctypes.c_int) for n in ("B", "max_pages", "rows")]


class dflash_rows(ctypes.Structure):
    _fields_ = [("ptr", ctypes.c_void_p), ("row_stride", ctypes.c_longlong),
                ("head_stride", ctypes.c_longlong)]


class dflash_logit_rules(ctypes.Structure):
    _fields_ = [("counts", ctypes.c_void_p), ("prompt_mask", ctypes.c_void_p),
                ("req_slot", ctypes.c_void_p), ("slots", ctypes.c_int)] + [
        (n, ctypes.c_void_p) for n in ("draft", "repetition", "frequency", "presence",
                                       "bias_start", "bias_ids", "bias_vals")] + [
        ("n_bias", ctypes.c_int), ("allow", ctypes.c_void_p)]


class dflash_draft_out(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in (
        "topk_ids", "topk_vals", "lse", "logits", "q", "draft")]


_lib = None
_P = ctypes.c_void_p
_I = ctypes.c_int
_SZ = ctypes.c_size_t


def lib():
    """Load libdflash.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                           "block_speculative_decoding_ctx_gb300.build.build()")
    L = ctypes.CDLL(LIB_PATH)
    sig = {
        "dflash_create": (_I, [ctypes.POINTER(dflash_config), ctypes.POINTER(dflash_weights),
                               ctypes.POINTER(_P)]),
        "dflash_destroy": (_I, [_P]),
        "dflash_draft_workspace_bytes": (_SZ, [_P]),
        "dflash_append_workspace_bytes": (_SZ, [_P]),
        "dflash_verify_workspace_bytes": (_SZ, [_I, _I, _I]),
        "dflash_probs_workspace_bytes": (_SZ, [_I, _I]),
        "dflash_ctx_append": (_I, [_P, _I, _I, _P, _P, _P, _P, _P, _P, _I, _P, _SZ, _P]),
        "dflash_draft_block": (_I, [_P, _I, _I, _P, _P, _P, _P, _P, _I, _I,
                                    ctypes.POINTER(dflash_sampling),
                                    ctypes.POINTER(dflash_draft_out), _P, _SZ, _P]),
        "dflash_probs": (_I, [_I, _I, _P, ctypes.c_float, ctypes.c_float, _P, _P, _SZ, _P]),
        "dflash_verify": (_I, [_I, _I, _I, _I, _P, _P, _P, _P, ctypes.c_uint64, _P, _P, _P, _P, _P,
                               _SZ, _P]),
        "dflash_read_status": (_I, [_P, ctypes.POINTER(ctypes.c_int32), _P]),
        "dflash_strerror": (ctypes.c_char_p, [_I]),
        "dflash_selftest_timeout": (_I, [_P, ctypes.c_longlong, _P]),
        "dflash_sample_draft": (_I, [_I, _I, _I, _P, _P, ctypes.c_uint64, _P, _P, _SZ, _P]),
        "dflash_sample_workspace_bytes": (_SZ, [_I, _I]),
        "dflash_profile_enable": (_I, [_P, _I]),
        "dflash_quantize_e4m3": (_I, [_P, _I, _I, _P, _P, _P]),
        "dflash_verify_noalloc": (_I, [_I, _I, _I, _I, _P, _P, _P, _P, ctypes.c_uint64, _P, _P, _P,
                                       _P, _P]),
        "dflash_paged_cache_maps": (_I, [_P, _P]),
        "dflash_paged_workspace_bytes": (_SZ, []),
        "dflash_paged_append": (_I, [_P, _P, _I, _P, _P, _P, _SZ, _P]),
        "dflash_paged_gather": (_I, [_P, _P, _I, _P, _P, _P, _SZ, _P]),
        "dflash_paged_attention_workspace_bytes": (_SZ, [_I, _I, _I, _I]),
        "dflash_paged_attention": (_I, [_P, _P, _I, _I, _P, _P, _P, _I, ctypes.c_float, _I, _I, _P,
                                        _SZ, _P]),
        "dflash_logits_adjust_workspace_bytes": (_SZ, []),
        "dflash_logits_adjust": (_I, [_I, _I, _I, _I, _P, ctypes.c_longlong, ctypes.c_longlong, _P,
                                      ctypes.c_longlong, ctypes.c_longlong, _P, _P, _SZ, _P]),
        "dflash_profile_read": (_I, [_P, ctypes.POINTER(ctypes.c_float),
                                     ctypes.POINTER(ctypes.c_double), ctypes.POINTER(_I), _I,
                                     ctypes.POINTER(_I)]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(L, name)
        fn.restype = res
        fn.argtypes = args
    _lib = L
    return L


def declared_functions():
    """Names of the functions include/dflash.h declares."""
    text = open(HEADER_PATH).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(dflash_\w+)\s*\(", text)))


# ----------------------------------------------------------------- helpers

def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _check(code, where):
    if code != 0:
        raise DflashError(code, where)


def dflash_strerror(code):
    return lib().dflash_strerror(int(code)).decode()


def workspace(nbytes, device="cuda"):
    """A zero-filled, 256-byte-aligned workspace tensor of nbytes bytes."""
    return torch.zeros(max(int(nbytes), 256), dtype=torch.uint8, device=device)


# ------------------------------------------------------------ entry points

class Handle:
    """Owns a dflash_handle and keeps the weight tensors alive."""

    def __init__(self, ptr, keep, cfg):
        self.ptr = ptr
        self._keep = keep
        self.cfg = cfg

    def __del__(self):
        try:
            if self.ptr:
                lib().dflash_destroy(self.ptr)
                self.ptr = None
        except Exception:
            pass


def dflash_create(cfg, weights):
    """cfg: dict with the dflash_config fields (weight_format defaults to
    DFLASH_WEIGHTS_BF16); weights: dict of CUDA tensors (matrices bf16, gains
    float32) with keys embed, lm_head, w_c, g_c, g_final and layers =
    [dict(g_attn, w_qkv, w_o, g_mlp, w_gate, w_up, w_down)].  With
    DFLASH_WEIGHTS_E4M3 the layer matrices and lm_head are uint8 E4M3 codes
    and s_qkv, s_o, s_gate, s_up, s_down (per layer) and s_lm_head their
    float32 row scales."""
    cfg = dict(cfg)
    cfg.setdefault("weight_format", DFLASH_WEIGHTS_BF16)
    c = dflash_config(**{k: cfg[k] for k, _ in dflash_config._fields_})
    layers = (dflash_layer_weights * len(weights["layers"]))()
    for i, lw in enumerate(weights["layers"]):
        for k, _ in dflash_layer_weights._fields_:
            t = lw.get(k)
            setattr(layers[i], k, t.data_ptr() if t is not None else None)
    s_head = weights.get("s_lm_head")
    w = dflash_weights(weights["embed"].data_ptr(), weights["lm_head"].data_ptr(),
                       weights["w_c"].data_ptr(), weights["g_c"].data_ptr(),
                       weights["g_final"].data_ptr(), layers,
                       s_head.data_ptr() if s_head is not None else None)
    out = ctypes.c_void_p()
    _check(lib().dflash_create(ctypes.byref(c), ctypes.byref(w), ctypes.byref(out)), "dflash_create")
    return Handle(out, (weights, layers), dict(cfg))


def dflash_destroy(handle):
    if handle.ptr:
        _check(lib().dflash_destroy(handle.ptr), "dflash_destroy")
        handle.ptr = None


def dflash_draft_workspace_bytes(handle):
    return int(lib().dflash_draft_workspace_bytes(handle.ptr))


def dflash_append_workspace_bytes(handle):
    return int(lib().dflash_append_workspace_bytes(handle.ptr))


def dflash_verify_workspace_bytes(batch, gamma, vocab):
    return int(lib().dflash_verify_workspace_bytes(batch, gamma, vocab))


def dflash_probs_workspace_bytes(rows, vocab):
    return int(lib().dflash_probs_workspace_bytes(rows, vocab))


def dflash_ctx_append(handle, feats, n_new, ctx_len, ring_k, ring_v, ws, req_slot=None,
                      stream=None):
    """feats bf16 [B, n_max, nf, fd]; n_new int32 [B]; ctx_len int64 [B] (in/out)."""
    B, n_max = feats.shape[0], feats.shape[1]
    _check(lib().dflash_ctx_append(handle.ptr, B, n_max, _ptr(feats), _ptr(n_new), _ptr(ctx_len),
                                   _ptr(req_slot), _ptr(ring_k), _ptr(ring_v), ring_k.shape[1],
                                   _ptr(ws), ws.numel(), _stream(stream)), "dflash_ctx_append")


def dflash_draft_block(handle, anchor, ctx_len, ring_k, ring_v, gamma, ws, topk=0, out=None,
                       sampling=None, req_slot=None, stream=None):
    """out: dict with any of topk_ids, topk_vals, lse, logits, q, draft (CUDA tensors).
    sampling: dict(temperature, top_p, seeds (uint64 as int64 tensor), step) or None."""
    out = out or {}
    o = dflash_draft_out(*[out[k].data_ptr() if out.get(k) is not None else None
                           for k, _ in dflash_draft_out._fields_])
    sp = None
    if sampling is not None:
        sp = ctypes.byref(dflash_sampling(float(sampling["temperature"]), float(sampling["top_p"]),
                                          sampling["seeds"].data_ptr(), int(sampling["step"])))
    _check(lib().dflash_draft_block(handle.ptr, anchor.shape[0], gamma, _ptr(anchor), _ptr(ctx_len),
                                    _ptr(req_slot), _ptr(ring_k), _ptr(ring_v), ring_k.shape[1],
                                    topk, sp, ctypes.byref(o), _ptr(ws), ws.numel(),
                                    _stream(stream)), "dflash_draft_block")


def dflash_probs(logits, temperature, top_p, probs, ws, stream=None):
    rows = logits.numel() // logits.shape[-1]
    _check(lib().dflash_probs(rows, logits.shape[-1], _ptr(logits), float(temperature),
                              float(top_p), _ptr(probs), _ptr(ws), ws.numel(), _stream(stream)),
           "dflash_probs")


def dflash_verify(mode, target, draft, accept_len, tokens, ws, q=None, seeds=None, step=0,
                  next_anchor=None, n_append=None, stream=None):
    """target: greedy target logits or sampled p, float32 [B, gamma, V]."""
    B, gamma, V = target.shape
    _check(lib().dflash_verify(int(mode), B, gamma, V, _ptr(target), _ptr(q), _ptr(draft),
                               _ptr(seeds), ctypes.c_uint64(int(step) & (2 ** 64 - 1)),
                               _ptr(accept_len), _ptr(tokens), _ptr(next_anchor), _ptr(n_append),
                               _ptr(ws), ws.numel(), _stream(stream)), "dflash_verify")


def dflash_read_status(ws, stream=None):
    v = ctypes.c_int32(0)
    _check(lib().dflash_read_status(_ptr(ws), ctypes.byref(v), _stream(stream)),
           "dflash_read_status")
    return v.value


def dflash_selftest_timeout(ws, limit_ns=1_000_000, stream=None):
    _check(lib().dflash_selftest_timeout(_ptr(ws), int(limit_ns), _stream(stream)),
           "dflash_selftest_timeout")


def dflash_sample_workspace_bytes(rows, vocab):
    return int(lib().dflash_sample_workspace_bytes(rows, vocab))


def dflash_sample_draft(q, seeds, step, y, ws, stream=None):
    """q float32 [B, G, V]; seeds uint64 (as int64) [B]; y int32 [B, G] out."""
    B, G, V = q.shape
    _check(lib().dflash_sample_draft(B, G, V, _ptr(q), _ptr(seeds), ctypes.c_uint64(int(step) & (2 ** 64 - 1)),
                                     _ptr(y), _ptr(ws), ws.numel(), _stream(stream)),
           "dflash_sample_draft")


def dflash_profile_enable(handle, n_pairs):
    _check(lib().dflash_profile_enable(handle.ptr, int(n_pairs)), "dflash_profile_enable")


PROFILE_KINDS = {0: "gemm", 1: "attention", 2: "norm", 3: "topk", 4: "sampling"}


def dflash_profile_read(handle, cap=128):
    """Per-launch (ms, algorithmic bytes, kind) of the last draft_block call."""
    ms = (ctypes.c_float * cap)()
    by = (ctypes.c_double * cap)()
    kd = (ctypes.c_int * cap)()
    n = ctypes.c_int(0)
    _check(lib().dflash_profile_read(handle.ptr, ms, by, kd, cap, ctypes.byref(n)),
           "dflash_profile_read")
    return [(ms[i], by[i], PROFILE_KINDS.get(kd[i], str(kd[i]))) for i in range(n.value)]


def dflash_verify_noalloc(mode, target, draft, accept_len, tokens, q=None, seeds=None, step=0,
                          next_anchor=None, n_append=None, stream=None):
    """dflash_verify without a workspace, for callers that cannot provide
    device memory: the scratch is a fixed array inside the library (see
    include/dflash.h for its size limit and for why overlapping calls race)."""
    B, gamma, V = target.shape
    _check(lib().dflash_verify_noalloc(int(mode), B, gamma, V, _ptr(target), _ptr(q), _ptr(draft),
                                       _ptr(seeds), ctypes.c_uint64(int(step) & (2 ** 64 - 1)),
                                       _ptr(accept_len), _ptr(tokens), _ptr(next_anchor),
                                       _ptr(n_append), _stream(stream)), "dflash_verify_noalloc")


def dflash_quantize_e4m3(w, codes, scales, stream=None):
    """w bf16 [rows, cols] -> codes uint8 [rows, cols], scales float32 [rows]."""
    rows, cols = w.shape
    _check(lib().dflash_quantize_e4m3(_ptr(w), rows, cols, _ptr(codes), _ptr(scales), _stream(stream)),
           "dflash_quantize_e4m3")


# ------------------------------------------------- the target's side of a cycle
#
# A decoding step makes these calls once a layer, so their argument marshalling
# is kept short: host structs are packed bytes (laid out as the ctypes
# structures above), addresses are plain integers.

_PACK_ROWS = struct.Struct("@Pqq").pack
_PACK_BATCH = struct.Struct("@PPPqiii4x").pack
_PACK_RULES = struct.Struct("@PPPiPPPPPPPiP").pack


_maps_lock = threading.Lock()


class PagedCache:
    """One layer's paged cache (see paged_cache); keeps its tensors alive."""

    def __init__(self, fields, keep, index):
        self.struct = fields
        self.index = index
        self._bytes = bytes(fields)
        self._keep = keep
        self._rows = (fields.n_kv_heads, fields.head_dim)
        self._maps = None

    def _with_maps(self):
        """The struct's bytes with the descriptors that attention needs, made
        once: another thread's call may be reading them."""
        with _maps_lock:
            if self._maps is None:
                maps = dflash_paged_maps()
                _check(lib().dflash_paged_cache_maps(self._bytes, ctypes.byref(maps)), "dflash_paged_cache_maps")
                c = dflash_paged_cache.from_buffer_copy(self._bytes)
                c.maps = ctypes.addressof(maps)
                self._maps = (bytes(c), maps)
        return self._maps[0]


def _misfit(name, t, dtype, shape, index):
    raise ValueError(f"{name}: expected a contiguous {dtype} tensor {tuple(shape)} on cuda:{index}, got "
                     f"{t.dtype} {tuple(t.shape)} on {t.device}")


def _fit(name, t, dtype, shape, index):
    """The tensor's address if it is a contiguous one of this type, shape and
    device; 0 for None."""
    if t is None:
        return 0
    if t.dtype is dtype and t.shape == shape and t.get_device() == index and t.is_contiguous():
        return t.data_ptr()
    _misfit(name, t, dtype, shape, index)


def _c_ints(what, *values):
    """ctypes passes the lower 32 bits of what a C int does not hold."""
    if min(values) < -1 << 31 or max(values) >= 1 << 31:
        raise ValueError(f"{what}: expected less than 2^31, got {values}")


def _current(index, stream):
    """The stream to launch on; the tensors' device must be the current one."""
    if index < 0:
        raise ValueError("expected CUDA tensors")
    if torch._C._cuda_getDevice() != index:
        raise ValueError(f"the tensors are on cuda:{index}, the current device is cuda:{torch.cuda.current_device()}")
    return torch._C._cuda_getCurrentRawStream(index) if stream is None else stream.cuda_stream


def _workspace(ws, index):
    if ws.get_device() != index or not ws.is_contiguous() or ws.element_size() != 1:
        raise ValueError(f"workspace: expected one of dfl.workspace on cuda:{index}")
    return ws.data_ptr()


def paged_cache(k_pages, v_pages, k_scale=None, v_scale=None):
    """A cache for the dflash_paged_* calls: pages [n_pages, n_kv_heads,
    page_size, head_dim] of bfloat16, float16, or E4M3 codes (float8_e4m3fn or
    uint8) with float32 scales [n_pages, n_kv_heads, page_size].  A page is
    contiguous; pages may lie further apart (a slice of a larger tensor)."""
    if k_pages.dim() != 4 or v_pages.shape != k_pages.shape or v_pages.dtype != k_pages.dtype or \
            v_pages.device != k_pages.device:
        raise ValueError("k_pages and v_pages: expected [n_pages, n_kv_heads, page_size, head_dim], alike in "
                         "shape, type and device")
    if k_pages.dtype not in _CACHES:
        raise ValueError(f"no cache of {k_pages.dtype}")
    n, heads, size, hd = k_pages.shape
    for t in (k_pages, v_pages):
        if n and not t[0].is_contiguous():
            raise ValueError("a page is not contiguous")
    fmt = _CACHES[k_pages.dtype]
    if (fmt == DFLASH_CACHE_E4M3) != (k_scale is not None) or (k_scale is None) != (v_scale is None):
        raise ValueError("E4M3 pages come with k_scale and v_scale, 16-bit pages without")
    index = k_pages.get_device()
    shape = (n, heads, size)
    page = heads * size * hd
    c = dflash_paged_cache(k_pages.data_ptr(), v_pages.data_ptr(),
                           _fit("k_scale", k_scale, torch.float32, shape, index),
                           _fit("v_scale", v_scale, torch.float32, shape, index),
                           k_pages.stride(0) if n > 1 else page, v_pages.stride(0) if n > 1 else page,
                           n, heads, size, hd, fmt, None)
    return PagedCache(c, (k_pages, v_pages, k_scale, v_scale), index)


def _rows(name, t, index):
    if t.dim() != 3 or t.get_device() != index or (t.stride(2) != 1 and t.numel()):
        raise ValueError(f"{name}: expected [rows, heads, head_dim] on cuda:{index} with head_dim contiguous")
    return _PACK_ROWS(t.data_ptr(), t.stride(0), t.stride(1))


def _batch(row_start, kv_len, page_table, rows, index):
    B = kv_len.shape[0]
    if page_table.dim() != 2 or page_table.shape[0] != B or page_table.dtype is not torch.int32 or \
            page_table.get_device() != index or (page_table.stride(1) != 1 and page_table.shape[1] > 1 and B):
        raise ValueError(f"page_table: expected int32 [{B}, max_pages] on cuda:{index}")
    pages = page_table.shape[1]
    return _PACK_BATCH(_fit("row_start", row_start, torch.int32, (B + 1,), index),
                       _fit("kv_len", kv_len, torch.int64, (B,), index), page_table.data_ptr(),
                       page_table.stride(0) if B > 1 else pages, B, pages, rows)


def dflash_paged_workspace_bytes():
    return int(lib().dflash_paged_workspace_bytes())


def _paged_move(call, name, cache, k, v, row_start, kv_len, page_table, ws, stream):
    index = cache.index
    if k.shape != v.shape or k.dtype is not v.dtype or k.shape[1:] != cache._rows:
        raise ValueError("k and v: expected [rows, %d, %d] of one type" % cache._rows)
    if k.dtype is not torch.bfloat16 and k.dtype is not torch.float16:
        raise ValueError(f"no rows of {k.dtype}")
    stream = _current(index, stream)
    code = call(cache._bytes, _batch(row_start, kv_len, page_table, k.shape[0], index), _TYPES[k.dtype],
                _rows("k", k, index), _rows("v", v, index), _workspace(ws, index), ws.numel(), stream)
    if code:
        raise DflashError(code, name)


def dflash_paged_append(cache, k, v, row_start, kv_len, page_table, ws, stream=None):
    """Write rows k, v [rows, n_kv_heads, head_dim] into the cache; row_start
    int32 [B + 1], kv_len int64 [B] (new rows counted), page_table int32
    [B, max_pages]."""
    _paged_move(lib().dflash_paged_append, "dflash_paged_append", cache, k, v, row_start, kv_len, page_table, ws,
                stream)


def dflash_paged_gather(cache, k, v, row_start, kv_len, page_table, ws, stream=None):
    """Read the last row_start[b + 1] - row_start[b] positions of every request
    back into k, v [rows, n_kv_heads, head_dim]."""
    _paged_move(lib().dflash_paged_gather, "dflash_paged_gather", cache, k, v, row_start, kv_len, page_table, ws,
                stream)


def dflash_paged_attention_workspace_bytes(n_q_heads, n_kv_heads, head_dim, max_rows):
    _c_ints("heads, head_dim and max_rows", n_q_heads, n_kv_heads, head_dim, max_rows)
    return int(lib().dflash_paged_attention_workspace_bytes(n_q_heads, n_kv_heads, head_dim, max_rows))


def dflash_paged_attention(cache, q, out, row_start, kv_len, page_table, max_rows, ws, lse=None,
                           scale=None, causal=True, window=0, stream=None):
    """q, out [rows, n_q_heads, head_dim]; lse float32 [rows, n_q_heads] or
    None; scale None: 1 / sqrt(head_dim)."""
    index, hd = cache.index, cache._rows[1]
    shape = q.shape
    if out.shape != shape or q.dtype is not out.dtype or len(shape) != 3 or shape[2] != hd:
        raise ValueError(f"q and out: expected [rows, n_q_heads, {hd}] of one type")
    if q.dtype is not torch.bfloat16 and q.dtype is not torch.float16:
        raise ValueError(f"no rows of {q.dtype}")
    if not (0 <= max_rows < 1 << 31 and 0 <= window < 1 << 31):
        raise ValueError(f"max_rows and window: expected 0 to 2^31 - 1, got {max_rows} and {window}")
    stream = _current(index, stream)
    maps = cache._maps
    code = lib().dflash_paged_attention(
        maps[0] if maps is not None else cache._with_maps(), _batch(row_start, kv_len, page_table, shape[0], index), _TYPES[q.dtype], shape[1],
        _rows("q", q, index), _rows("out", out, index), _fit("lse", lse, torch.float32, shape[:2], index) or None,
        max_rows, hd ** -0.5 if scale is None else scale, 1 if causal else 0, window, _workspace(ws, index),
        ws.numel(), stream)
    if code:
        raise DflashError(code, "dflash_paged_attention")


def dflash_logits_adjust_workspace_bytes():
    return int(lib().dflash_logits_adjust_workspace_bytes())


def dflash_logits_adjust(logits, out, ws, counts=None, prompt_mask=None, req_slot=None, draft=None,
                         repetition=None, frequency=None, presence=None, bias_start=None, bias_ids=None,
                         bias_vals=None, allow=None, stream=None):
    """logits [B, G, V] float32, bfloat16 or float16; out float32 [B, G, V]
    (may be logits).  counts int32 [slots, V]; prompt_mask int32
    [slots, ceil(V / 32)] bits; req_slot int32 [B]; draft int32 [B, G - 1];
    repetition, frequency, presence float32 [B]; bias_start int32 [B + 1] with
    bias_ids int32 and bias_vals float32 [n_bias]; allow int32
    [B, G, ceil(V / 32)] bits."""
    shape = logits.shape
    index = logits.get_device()
    if len(shape) != 3 or logits.dtype not in _TYPES or out.shape != shape or \
            out.dtype is not torch.float32 or out.get_device() != index:
        raise ValueError("logits and out: expected [B, G, V], out float32, on one device")
    B, G, V = shape
    _c_ints("B, G and V", B, G, V)
    if not (bias_start is None) == (bias_ids is None) == (bias_vals is None):
        raise ValueError("bias_start, bias_ids and bias_vals come together")
    l_b, l_i, l_v = logits.stride()
    o_b, o_i, o_v = out.stride()
    if V > 1 and (l_v != 1 or o_v != 1):
        raise ValueError("the vocabulary is not contiguous")
    stream = _current(index, stream)
    words = (V + 31) // 32
    slots = counts.shape[0] if counts is not None else prompt_mask.shape[0] if prompt_mask is not None else 0
    n_bias = 0 if bias_ids is None else bias_ids.shape[0]
    i32, f32, per = torch.int32, torch.float32, (B,)
    rules = _PACK_RULES(
        _fit("counts", counts, i32, (slots, V), index),
        _fit("prompt_mask", prompt_mask, i32, (slots, words), index),
        _fit("req_slot", req_slot, i32, per, index), slots,
        _fit("draft", draft, i32, (B, G - 1), index),
        _fit("repetition", repetition, f32, per, index),
        _fit("frequency", frequency, f32, per, index),
        _fit("presence", presence, f32, per, index),
        _fit("bias_start", bias_start, i32, (B + 1,), index),
        _fit("bias_ids", bias_ids, i32, (n_bias,), index),
        _fit("bias_vals", bias_vals, f32, (n_bias,), index), n_bias,
        _fit("allow", allow, i32, (B, G, words), index))
    code = lib().dflash_logits_adjust(B, G, V, _TYPES[logits.dtype], logits.data_ptr(), l_b, l_i, out.data_ptr(),
                                      o_b, o_i, rules, _workspace(ws, index), ws.numel(), stream)
    if code:
        raise DflashError(code, "dflash_logits_adjust")


def quantize_weights_e4m3(weights, stream=None):
    """A copy of a bf16 weight dict (see dflash_create) whose layer matrices
    and lm_head are E4M3 codes with their row scales, made on the device by
    dflash_quantize_e4m3; embed, w_c and the gains are shared."""
    def q(t):
        codes = torch.empty(t.shape, dtype=torch.uint8, device=t.device)
        scales = torch.empty(t.shape[0], dtype=torch.float32, device=t.device)
        dflash_quantize_e4m3(t, codes, scales, stream)
        return codes, scales

    out = {k: v for k, v in weights.items() if k != "layers"}
    out["lm_head"], out["s_lm_head"] = q(weights["lm_head"])
    out["layers"] = []
    for lw in weights["layers"]:
        nl = dict(lw)
        for k in LAYER_MATRICES:
            nl[k], nl["s_" + k[2:]] = q(lw[k])
        out["layers"].append(nl)
    return out
