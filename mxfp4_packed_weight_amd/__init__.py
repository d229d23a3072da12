"""Python binding of libk3moe.so, the MI355X (gfx950) MXFP4 routed-expert path.

Argument marshalling only: every step runs in the HIP kernels behind the C
ABI declared in ``include/k3moe.h``. Functions carry the C names. Device
buffers are torch tensors on a ROCm device (torch provides memory and
streams, nothing else); host buffers of the ``*_host`` calls are numpy arrays.

The library must be built first (``python -m mxfp4_packed_weight_amd._build``
or ``__graft_entry__.build()``); importing works without it, but every call
raises ``K3LibraryMissing`` rather than falling back to anything else.
"""
import ctypes
import os

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libk3moe.so")
_lib = None
_functions = {}  # those called so far

K3_OK, K3_ERR_ARG, K3_ERR_CONFIG, K3_ERR_MEMORY, K3_ERR_DEVICE = 0, 1, 2, 3, 4
K3_MAX_EXPERTS, K3_MAX_TOPK, K3_MAX_SHARED = 4096, 64, 8
K3_WAIT_LIMIT_DEFAULT = 1 << 20
K3_BF16, K3_F16, K3_E4M3 = 0, 1, 2
K3_MAX_REQUESTS, K3_MAX_TREE_WORDS, K3_MAX_ACCEPTED, K3_MAX_HEADS = 4096, 32, 1024, 1024

# (name, restype, argtypes) of every exported symbol in include/k3moe.h
_vp, _i, _sz, _i64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_int64


class k3_cache_stats(ctypes.Structure):
    _fields_ = [(f, ctypes.c_uint64) for f in
                ("requests", "hits", "misses", "inflight_reuses", "evictions", "bytes_copied")]

    def as_dict(self):
        return {f: int(getattr(self, f)) for f, _ in self._fields_}


class k3_kv_cache(ctypes.Structure):
    """One layer's paged cache as the C calls take it; k3_kv_cache_of fills it
    from tensors and keeps them alive."""
    _fields_ = ([(f, ctypes.c_void_p) for f in ("k", "v", "k_scale", "v_scale")]
                + [(f, ctypes.c_int64) for f in ("page_stride", "slot_stride", "head_stride")]
                + [(f, ctypes.c_int32) for f in ("n_pages", "page_size", "n_heads", "head_dim",
                                                 "dtype")])


_stats_p = ctypes.POINTER(k3_cache_stats)
SIGNATURES = [
    ("k3_strerror", ctypes.c_char_p, [_i]),
    ("k3_last_error", ctypes.c_char_p, []),
    ("k3_abi_version", _i, []),
    ("k3_mxfp4_packed_bytes", _sz, [_i, _i]),
    ("k3_mxfp4_pack_host", _i, [_vp, _vp, _i, _i, _vp]),
    ("k3_mxfp4_unpack_host", _i, [_vp, _i, _i, _vp, _vp]),
    ("k3_mxfp4_pack", _i, [_vp, _vp, _i, _i, _vp, _vp]),
    ("k3_mxfp4_unpack", _i, [_vp, _i, _i, _vp, _vp, _vp]),
    ("k3_expert_packed_bytes", _sz, [_i, _i]),
    ("k3_expert_pack_host", _i, [_vp] * 6 + [_i, _i, _vp]),
    ("k3_expert_pack", _i, [_vp] * 6 + [_i, _i, _vp, _vp]),
    ("k3_mxfp4_gemv", _i, [_vp, _vp, _i, _i, _vp, _vp]),
    ("k3_expert_swiglu", _i, [_vp, _vp, _i, _i, _vp, _vp, _vp]),
    ("k3_expert_swiglu_workspace_bytes", _sz, [_i, _i]),
    ("k3_expert_swiglu_ws", _i, [_vp, _vp, _i, _i, _vp, _vp, _vp, _sz, _vp]),
    ("k3_expert_gate_up", _i, [_vp, _vp, _vp, _i, _i, _i, _vp, _vp]),
    ("k3_expert_gate_up_routed", _i, [_vp, _vp, _vp, _i, _i, _i, _i, _vp, _vp, _vp, _vp]),
    ("k3_expert_down", _i, [_vp, _vp, _vp, _i, _i, _i, _vp, _vp]),
    ("k3_moe_combine", _i, [_vp, _vp, _i, _i, _vp, _vp, _vp]),
    ("k3_router", _i, [_vp, _vp, _i, _i, _i, _vp, _vp]),
    ("k3_router_topk", _i, [_vp, _vp, _i, _i, _i, _vp, _vp, _vp]),
    ("k3_router_topk_f32", _i, [_vp, _vp, _i, _i, _i, _vp, _vp, _vp]),
    ("k3_router_topk_scaled", _i, [_vp, _vp, _i, _i, _i, ctypes.c_double, _vp, _vp, _vp]),
    ("k3_moe_workspace_bytes", _sz, [_i, _i, _i, _i, _i]),
    ("k3_moe_layer", _i, [_vp, _vp, _vp, _i, _i, _i, _i, _vp, _vp, _sz, _vp]),
    ("k3_moe_layer_ex", _i, [_vp, _vp, _vp, _i, _i, _i, _i, _vp, _vp, _vp, _vp, _vp,
                             _vp, _sz, _vp]),
    ("k3_moe_layer_noalloc", _i, [_vp, _vp, _vp, _i, _i, _i, _i, _vp, _vp, _vp, _vp, _vp,
                                  _vp]),
    ("k3_moe_permute_workspace_bytes", _sz, [_i, _i]),
    ("k3_moe_permute", _i, [_vp, _i, _i, _i, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    ("k3_moe_batched_workspace_bytes", _sz, [_i, _i, _i, _i, _i]),
    ("k3_moe_layer_from_logits", _i, [_vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _vp, _vp, _vp,
                                      _vp, _vp, _sz, _vp]),
    ("k3_moe_layer_batched", _i, [_vp, _vp, _vp, _i, _i, _i, _i, _i, _vp, _vp, _vp, _vp, _vp,
                                  _sz, _vp]),
    ("k3_mxfp4_quantize_f32", _i, [_vp, _i, _i, _vp, _vp, _vp]),
    ("k3_mxfp4_quantize_bf16", _i, [_vp, _i, _i, _vp, _vp, _vp]),
    ("k3_moe_prefill_workspace_bytes", _sz, [_i, _i, _i, _i, _i]),
    ("k3_moe_prefill", _i, [_vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _vp, _vp, _vp, _vp, _vp,
                            _vp, _vp, _vp, _sz, _vp]),
    ("k3_hbm_read_probe", _i, [_vp, _sz, _vp, _vp]),
    ("k3_set_wait_limit", _i, [_i]),
    ("k3_shared_expert_bytes", _sz, [_i, _i]),
    ("k3_shared_experts", _i, [_vp, _vp, _i, _i, _i, _vp, _vp, _vp]),
    ("k3_moe_layer_shared_workspace_bytes", _sz, [_i, _i, _i, _i, _i, _i]),
    ("k3_moe_layer_shared", _i, [_vp, _vp, _vp, _i, _i, _i, _i, _vp, _i, _i, _vp, _vp, _vp,
                                 _vp, _vp, _vp, _sz, _vp]),
    ("k3_expert_dense_bytes", _sz, [_i, _i]),
    ("k3_expert_dequantize", _i, [_vp, _i, _i, _vp, _vp]),
    ("k3_experts_dense", _i, [_vp, _vp, _vp, _i, _i, _i, _vp, _vp, _vp]),
    ("k3_cache_create", _i, [_i, _sz, _i, ctypes.POINTER(_vp)]),
    ("k3_cache_destroy", None, [_vp]),
    ("k3_cache_set_source", _i, [_vp, _i, _vp]),
    ("k3_cache_pin", _i, [_vp, _i, _i]),
    ("k3_cache_fetch", _i, [_vp, _vp, _i, _vp]),
    ("k3_cache_table", _vp, [_vp]),
    ("k3_cache_get_stats", _i, [_vp, _stats_p]),
    ("k3_cache_histogram", _i, [_vp, _vp]),
    ("k3_cache_trace", _i, [_vp, _vp, _sz, ctypes.POINTER(_sz)]),
    ("k3_cache_replay", _i, [_vp, _sz, _i, _i, _vp, _i, _i, _stats_p]),
    ("k3_cache_replay_opt", _i, [_vp, _sz, _i, _i, _vp, _i, _i, _stats_p]),
    ("k3_moe_layer_from_logits_cached", _i, [_vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _vp, _vp,
                                             _vp, _vp, _vp, _sz, _vp]),
    ("k3_moe_layer_cached", _i, [_vp, _vp, _vp, _i, _i, _i, _i, _vp, _vp, _vp, _vp, _vp,
                                 _vp, _sz, _vp]),
    ("k3_kv_plan", _i, [_vp] * 3 + [_i] * 5 + [_vp] * 11 + [_i, _vp, _vp]),
    ("k3_qk_norm_rope", _i, [_vp, _i64, _vp, _i64, _vp, _i64, _i, _i, _i, _vp, _vp,
                             ctypes.c_float, _vp, _i, _i, _vp, _vp, _i64, _vp, _vp, _vp]),
    ("k3_tree_attention_workspace_bytes", _sz, [_i, _i, _i, _i]),
    ("k3_tree_attention", _i, [_vp, _i64, _i, _i, _i, _vp, _vp, _i, _vp, _vp, _i, _vp, _i,
                               ctypes.c_float, _vp, _i64, _vp, _sz, _vp, _vp]),
    ("k3_kv_commit", _i, [_vp, _i, _i64, _vp, _i, _vp, _vp, _vp, _i, _i, _vp, _vp]),
    ("k3_kv_commit_ex", _i, [_vp, _i, _i64, _vp, _i, _vp, _vp, _vp, _vp, _i, _i, _vp, _vp]),
]


class K3LibraryMissing(RuntimeError):
    pass


class K3Error(RuntimeError):
    def __init__(self, fn, status, detail):
        self.status = status
        super().__init__(f"{fn}: status {status} ({strerror(status)}): {detail}")


def lib():
    """Load libk3moe.so (once). Raises K3LibraryMissing if it is not built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise K3LibraryMissing(
                f"{LIB_PATH} is not built; run __graft_entry__.build() "
                "(there is no fallback implementation)")
        L = ctypes.CDLL(LIB_PATH)
        for name, res, args in SIGNATURES:
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


def strerror(status):
    return lib().k3_strerror(int(status)).decode()


def last_error():
    return lib().k3_last_error().decode()


def _call(name, *args):
    f = _functions.get(name)
    if f is None:
        f = _functions[name] = getattr(lib(), name)
    rc = f(*args)
    if rc != K3_OK:
        raise K3Error(name, rc, last_error())
    return rc


def _dp(t):
    """Device pointer of a torch tensor or a raw address (None -> NULL)."""
    if t is None:
        return None
    if isinstance(t, int):
        return ctypes.c_void_p(t)
    return ctypes.c_void_p(t.data_ptr())


def _hp(a):
    return None if a is None else ctypes.c_void_p(a.ctypes.data)


_current = None


def _stream(stream=None):
    """The handle of a stream, or of the current device's current one (asked
    for without the stream object: 0.3 us instead of 3)."""
    global _current
    if stream is not None:
        return stream.cuda_stream
    if _current is None:
        import torch
        torch.cuda.init()
        _current = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice
    return _current[0](_current[1]())


# ---- layout ---------------------------------------------------------------

def k3_mxfp4_packed_bytes(rows, cols):
    return lib().k3_mxfp4_packed_bytes(rows, cols)


def k3_expert_packed_bytes(hidden, inter):
    return lib().k3_expert_packed_bytes(hidden, inter)


def k3_mxfp4_pack_host(nib, sc):
    nib, sc = np.ascontiguousarray(nib, np.uint8), np.ascontiguousarray(sc, np.uint8)
    rows, cols = nib.shape[0], nib.shape[1] * 2
    out = np.empty(k3_mxfp4_packed_bytes(rows, cols), np.uint8)
    _call("k3_mxfp4_pack_host", _hp(nib), _hp(sc), rows, cols, _hp(out))
    return out


def k3_mxfp4_unpack_host(tiles, rows, cols):
    tiles = np.ascontiguousarray(tiles, np.uint8)
    nib = np.empty((rows, cols // 2), np.uint8)
    sc = np.empty((rows, cols // 32), np.uint8)
    _call("k3_mxfp4_unpack_host", _hp(tiles), rows, cols, _hp(nib), _hp(sc))
    return nib, sc


def k3_expert_pack_host(E, hidden, inter):
    arrs = [np.ascontiguousarray(a, np.uint8) for a in
            (E["gate"][0], E["gate"][1], E["up"][0], E["up"][1], E["down"][0], E["down"][1])]
    out = np.empty(k3_expert_packed_bytes(hidden, inter), np.uint8)
    _call("k3_expert_pack_host", *[_hp(a) for a in arrs], hidden, inter, _hp(out))
    return out


def k3_mxfp4_pack(nib_d, sc_d, rows, cols, tiles_d, stream=None):
    _call("k3_mxfp4_pack", _dp(nib_d), _dp(sc_d), rows, cols, _dp(tiles_d), _stream(stream))


def k3_mxfp4_unpack(tiles_d, rows, cols, nib_d, sc_d, stream=None):
    _call("k3_mxfp4_unpack", _dp(tiles_d), rows, cols, _dp(nib_d), _dp(sc_d), _stream(stream))


def k3_expert_pack(gate_nib, gate_sc, up_nib, up_sc, down_nib, down_sc, hidden, inter,
                   expert_d, stream=None):
    _call("k3_expert_pack", _dp(gate_nib), _dp(gate_sc), _dp(up_nib), _dp(up_sc),
          _dp(down_nib), _dp(down_sc), hidden, inter, _dp(expert_d), _stream(stream))


# ---- compute --------------------------------------------------------------

def _nbytes(t):
    return t.numel() * t.element_size()


def k3_mxfp4_gemv(x, tiles, rows, cols, y, stream=None):
    _call("k3_mxfp4_gemv", _dp(x), _dp(tiles), rows, cols, _dp(y), _stream(stream))


def k3_expert_swiglu(x, expert, hidden, inter, y, h, stream=None):
    _call("k3_expert_swiglu", _dp(x), _dp(expert), hidden, inter, _dp(y), _dp(h),
          _stream(stream))


def k3_expert_swiglu_workspace_bytes(hidden, inter):
    return lib().k3_expert_swiglu_workspace_bytes(hidden, inter)


def k3_expert_swiglu_ws(x, expert, hidden, inter, y, ws, h=None, stream=None):
    _call("k3_expert_swiglu_ws", _dp(x), _dp(expert), hidden, inter, _dp(y), _dp(h), _dp(ws),
          _nbytes(ws), _stream(stream))


def k3_expert_gate_up(x, experts, idx, k, hidden, inter, h, stream=None):
    _call("k3_expert_gate_up", _dp(x), _dp(experts), _dp(idx), k, hidden, inter, _dp(h),
          _stream(stream))


def k3_expert_gate_up_routed(x, logits, experts, n_experts, k, hidden, inter, h, idx, w,
                             stream=None):
    _call("k3_expert_gate_up_routed", _dp(x), _dp(logits), _dp(experts), n_experts, k, hidden,
          inter, _dp(h), _dp(idx), _dp(w), _stream(stream))


def k3_expert_down(h, experts, idx, k, hidden, inter, yp, stream=None):
    _call("k3_expert_down", _dp(h), _dp(experts), _dp(idx), k, hidden, inter, _dp(yp),
          _stream(stream))


def k3_moe_combine(yp, w, k, hidden, y=None, y_f32=None, stream=None):
    _call("k3_moe_combine", _dp(yp), _dp(w), k, hidden, _dp(y), _dp(y_f32), _stream(stream))


def k3_router(x, router_w, T, hidden, n_experts, logits, stream=None):
    _call("k3_router", _dp(x), _dp(router_w), T, hidden, n_experts, _dp(logits),
          _stream(stream))


def k3_router_topk(logits, bias, T, n_experts, k, idx, w, stream=None):
    _call("k3_router_topk", _dp(logits), _dp(bias), T, n_experts, k, _dp(idx), _dp(w),
          _stream(stream))


def k3_router_topk_f32(logits, bias, T, n_experts, k, idx, w, stream=None):
    _call("k3_router_topk_f32", _dp(logits), _dp(bias), T, n_experts, k, _dp(idx), _dp(w),
          _stream(stream))


def k3_router_topk_scaled(logits, bias, T, n_experts, k, routed_scale, idx, w, stream=None):
    _call("k3_router_topk_scaled", _dp(logits), _dp(bias), T, n_experts, k, float(routed_scale),
          _dp(idx), _dp(w), _stream(stream))


def k3_moe_workspace_bytes(T, n_experts, hidden, inter, k):
    return lib().k3_moe_workspace_bytes(T, n_experts, hidden, inter, k)


def k3_moe_layer(x, router_w, experts, n_experts, hidden, inter, k, y, ws, stream=None):
    _call("k3_moe_layer", _dp(x), _dp(router_w), _dp(experts), n_experts, hidden, inter, k,
          _dp(y), _dp(ws), _nbytes(ws), _stream(stream))


def k3_moe_layer_ex(x, router_w, experts, n_experts, hidden, inter, k, y, ws, y_f32=None,
                    idx=None, w=None, logits=None, stream=None):
    _call("k3_moe_layer_ex", _dp(x), _dp(router_w), _dp(experts), n_experts, hidden, inter,
          k, _dp(y), _dp(y_f32), _dp(idx), _dp(w), _dp(logits), _dp(ws), _nbytes(ws),
          _stream(stream))


def k3_moe_layer_noalloc(x, router_w, experts, n_experts, hidden, inter, k, y, y_f32=None,
                         idx=None, w=None, logits=None, stream=None):
    _call("k3_moe_layer_noalloc", _dp(x), _dp(router_w), _dp(experts), n_experts, hidden,
          inter, k, _dp(y), _dp(y_f32), _dp(idx), _dp(w), _dp(logits), _stream(stream))


K3_NOALLOC_SCRATCH_BYTES = 2 << 20


# ---- batched decode -------------------------------------------------------

def k3_moe_permute_workspace_bytes(T, k):
    return lib().k3_moe_permute_workspace_bytes(T, k)


def k3_moe_permute(idx, T, k, n_experts, counts, offsets, pair_token, pair_slot, ws,
                   stream=None):
    _call("k3_moe_permute", _dp(idx), T, k, n_experts, _dp(counts), _dp(offsets),
          _dp(pair_token), _dp(pair_slot), _dp(ws), _nbytes(ws), _stream(stream))


def k3_moe_batched_workspace_bytes(T, n_experts, hidden, inter, k):
    return lib().k3_moe_batched_workspace_bytes(T, n_experts, hidden, inter, k)


def k3_moe_layer_from_logits(X, logits, bias, experts, n_experts, hidden, inter, k, T, Y, ws,
                             Y_f32=None, idx=None, w=None, stream=None):
    _call("k3_moe_layer_from_logits", _dp(X), _dp(logits), _dp(bias), _dp(experts), n_experts,
          hidden, inter, k, T, _dp(Y), _dp(Y_f32), _dp(idx), _dp(w), _dp(ws), _nbytes(ws),
          _stream(stream))


def k3_moe_layer_batched(X, router_w, experts, n_experts, hidden, inter, k, T, Y, ws,
                         Y_f32=None, idx=None, w=None, stream=None):
    _call("k3_moe_layer_batched", _dp(X), _dp(router_w), _dp(experts), n_experts, hidden,
          inter, k, T, _dp(Y), _dp(Y_f32), _dp(idx), _dp(w), _dp(ws), _nbytes(ws),
          _stream(stream))


# ---- prefill --------------------------------------------------------------

def k3_mxfp4_quantize_f32(v, rows, cols, nib, sc, stream=None):
    _call("k3_mxfp4_quantize_f32", _dp(v), rows, cols, _dp(nib), _dp(sc), _stream(stream))


def k3_mxfp4_quantize_bf16(v, rows, cols, nib, sc, stream=None):
    _call("k3_mxfp4_quantize_bf16", _dp(v), rows, cols, _dp(nib), _dp(sc), _stream(stream))


def k3_moe_prefill_workspace_bytes(T, n_experts, hidden, inter, k):
    return lib().k3_moe_prefill_workspace_bytes(T, n_experts, hidden, inter, k)


def k3_moe_prefill(X, logits, bias, experts, n_experts, hidden, inter, k, T, Y, ws, Y_f32=None,
                   idx=None, w=None, h_f32=None, h_nib=None, h_sc=None, stream=None):
    _call("k3_moe_prefill", _dp(X), _dp(logits), _dp(bias), _dp(experts), n_experts, hidden,
          inter, k, T, _dp(Y), _dp(Y_f32), _dp(idx), _dp(w), _dp(h_f32), _dp(h_nib), _dp(h_sc),
          _dp(ws), _nbytes(ws), _stream(stream))


# ---- measurement ------------------------------------------------------------

def k3_hbm_read_probe(buf, nbytes, sink, stream=None):
    _call("k3_hbm_read_probe", _dp(buf), nbytes, _dp(sink), _stream(stream))


def k3_set_wait_limit(polls):
    _call("k3_set_wait_limit", polls)


# ---- shared experts ---------------------------------------------------------

def k3_shared_expert_bytes(hidden, inter):
    return lib().k3_shared_expert_bytes(hidden, inter)


def k3_shared_experts(x, shared, n_shared, hidden, inter, h, ys, stream=None):
    _call("k3_shared_experts", _dp(x), _dp(shared), n_shared, hidden, inter, _dp(h), _dp(ys),
          _stream(stream))


def k3_moe_layer_shared_workspace_bytes(n_experts, hidden, inter, k, n_shared, inter_shared):
    return lib().k3_moe_layer_shared_workspace_bytes(n_experts, hidden, inter, k, n_shared,
                                                     inter_shared)


def k3_moe_layer_shared(x, router_w, experts, n_experts, hidden, inter, k, shared, n_shared,
                        inter_shared, y, ws, y_f32=None, idx=None, w=None, logits=None,
                        stream=None):
    _call("k3_moe_layer_shared", _dp(x), _dp(router_w), _dp(experts), n_experts, hidden, inter,
          k, _dp(shared), n_shared, inter_shared, _dp(y), _dp(y_f32), _dp(idx), _dp(w),
          _dp(logits), _dp(ws), _nbytes(ws), _stream(stream))


# ---- dequantise-then-multiply control -------------------------------------

def k3_expert_dense_bytes(hidden, inter):
    return lib().k3_expert_dense_bytes(hidden, inter)


def k3_expert_dequantize(expert, hidden, inter, dense, stream=None):
    _call("k3_expert_dequantize", _dp(expert), hidden, inter, _dp(dense), _stream(stream))


def k3_experts_dense(x, dense_experts, idx, k, hidden, inter, h, yp, stream=None):
    _call("k3_experts_dense", _dp(x), _dp(dense_experts), _dp(idx), k, hidden, inter, _dp(h),
          _dp(yp), _stream(stream))


# ---- expert cache ---------------------------------------------------------
# A cache is the opaque handle (an int) k3_cache_create returns; host blobs
# are pinned CPU torch tensors or numpy arrays that the caller keeps alive.

def _ids(ids):
    a = np.ascontiguousarray(ids, np.int32)
    return a, ctypes.c_void_p(a.ctypes.data)


def k3_cache_create(n_experts, expert_bytes, n_slots):
    h = _vp()
    _call("k3_cache_create", n_experts, expert_bytes, n_slots, ctypes.byref(h))
    return h.value


def k3_cache_destroy(cache):
    lib().k3_cache_destroy(_vp(cache))


def k3_cache_set_source(cache, expert, host_blob):
    ptr = host_blob.data_ptr() if hasattr(host_blob, "data_ptr") else host_blob.ctypes.data
    _call("k3_cache_set_source", _vp(cache), expert, _vp(ptr))


def k3_cache_pin(cache, expert, pinned=True):
    _call("k3_cache_pin", _vp(cache), expert, int(bool(pinned)))


def k3_cache_fetch(cache, ids, stream=None):
    a, p = _ids(ids)
    _call("k3_cache_fetch", _vp(cache), p, a.size, _stream(stream))


def k3_cache_table(cache):
    """Device address of the cache's expert pointer table (an int)."""
    return lib().k3_cache_table(_vp(cache))


def k3_cache_get_stats(cache):
    st = k3_cache_stats()
    _call("k3_cache_get_stats", _vp(cache), ctypes.byref(st))
    return st.as_dict()


def k3_cache_histogram(cache, n_experts):
    out = np.zeros(n_experts, np.uint64)
    _call("k3_cache_histogram", _vp(cache), _hp(out))
    return out


def k3_cache_trace(cache):
    n = _sz()
    _call("k3_cache_trace", _vp(cache), None, 0, ctypes.byref(n))
    out = np.zeros(max(1, n.value), np.int32)
    _call("k3_cache_trace", _vp(cache), _hp(out), out.size, ctypes.byref(n))
    return out[:n.value]


def k3_cache_replay(trace, n_experts, n_slots, pinned=(), request_size=1):
    t, tp = _ids(trace)
    pn, pp = _ids(pinned)
    st = k3_cache_stats()
    _call("k3_cache_replay", tp, t.size, n_experts, n_slots, pp if pn.size else None,
          pn.size, request_size, ctypes.byref(st))
    return st.as_dict()


def k3_cache_replay_opt(trace, n_experts, n_slots, pinned=(), request_size=1):
    t, tp = _ids(trace)
    pn, pp = _ids(pinned)
    st = k3_cache_stats()
    _call("k3_cache_replay_opt", tp, t.size, n_experts, n_slots, pp if pn.size else None,
          pn.size, request_size, ctypes.byref(st))
    return st.as_dict()


def k3_moe_layer_cached(x, router_w, cache, n_experts, hidden, inter, k, y, ws, y_f32=None,
                        idx=None, w=None, logits=None, stream=None):
    _call("k3_moe_layer_cached", _dp(x), _dp(router_w), _vp(cache), n_experts, hidden, inter,
          k, _dp(y), _dp(y_f32), _dp(idx), _dp(w), _dp(logits), _dp(ws), _nbytes(ws),
          _stream(stream))


def k3_moe_layer_from_logits_cached(X, logits, bias, cache, n_experts, hidden, inter, k, T, Y,
                                    ws, Y_f32=None, idx=None, w=None, stream=None):
    _call("k3_moe_layer_from_logits_cached", _dp(X), _dp(logits), _dp(bias), _vp(cache),
          n_experts, hidden, inter, k, T, _dp(Y), _dp(Y_f32), _dp(idx), _dp(w), _dp(ws),
          _nbytes(ws), _stream(stream))


# ---- paged key/value cache --------------------------------------------------
# Tensors only: strides are read off the rows' tensors, and what the C calls
# cannot see is checked here: types, dense arrays, and that they hold as much
# as the call's sizes say. A cache is the handle that k3_kv_cache_of returns,
# made once per layer.

def _ptr(t):
    return None if t is None else t.data_ptr()


_kv_codes = {}
_int32 = _float32 = None  # torch's, once an array was given


def _array(name, t, dtype, n):
    """Address of a dense array of at least n values."""
    if t.dtype is not dtype:
        raise TypeError(f"{name} is {t.dtype}, not {dtype}")
    if not t.is_contiguous() or t.numel() < n:
        raise ValueError(f"{name}: a dense array of at least {n} values, not {tuple(t.shape)} "
                         f"with strides {t.stride()}")
    return t.data_ptr()


def _ints(name, t, n):
    """The same of int32 (None: NULL)."""
    global _int32
    if t is None:
        return None
    if t.dtype is _int32 and t.is_contiguous() and t.numel() >= n:
        return t.data_ptr()
    import torch
    _int32 = torch.int32
    return _array(name, t, _int32, n)


def _floats(name, t, n):
    """The same of float32 (None: NULL)."""
    global _float32
    if t is None:
        return None
    if _float32 is None:
        import torch
        _float32 = torch.float32
    return _array(name, t, _float32, n)


def _kv_dtype(t):
    if not _kv_codes:
        import torch
        _kv_codes.update({torch.bfloat16: K3_BF16, torch.float16: K3_F16,
                          torch.float8_e4m3fn: K3_E4M3})
    code = _kv_codes.get(t.dtype)
    if code is None:
        raise TypeError(f"bfloat16, float16 or float8_e4m3fn, not {t.dtype}")
    return code


def _heads(name, t, dtype, T, heads, D):
    """Token stride of rows [T, heads, D] or [T, heads * D] with dense heads,
    the first of as many tokens and heads or more."""
    if t.dtype is not dtype:
        raise TypeError(f"{name} is {t.dtype}, not the type of the call's other rows")
    shape, strides = t.shape, t.stride()
    if len(shape) == 2:
        dense = shape[1] >= heads * D
    else:
        dense = (len(shape) == 3 and shape[1] >= heads and shape[2] == D
                 and (shape[1] == 1 or strides[1] == D))
    if not dense or strides[-1] != 1 or shape[0] < T:
        raise ValueError(f"{name}: rows [{T}, {heads}, {D}] with dense heads, "
                         f"not {tuple(shape)} with strides {strides}")
    return strides[0]


def k3_kv_cache_of(k, v, k_scale=None, v_scale=None):
    """The handle of one layer's cache: k, v [pages, page_size, heads, D]
    views in any order in memory with dense rows; fp32 scales [heads] for
    float8_e4m3fn caches (None: 1)."""
    import torch
    if k.dim() != 4 or k.shape != v.shape or k.stride() != v.stride() or k.dtype != v.dtype:
        raise ValueError("k and v: [pages, page_size, heads, D], alike in shape, strides and type")
    if k.stride(3) != 1:
        raise ValueError(f"rows of keys and values are dense, not of stride {k.stride(3)}")
    for s in (k_scale, v_scale):
        if s is not None and (s.dtype != torch.float32 or s.numel() != k.shape[2]
                              or not s.is_contiguous()):
            raise ValueError("scales are float32 [heads]")
    c = k3_kv_cache(_ptr(k), _ptr(v), _ptr(k_scale), _ptr(v_scale), k.stride(0), k.stride(1),
                    k.stride(2), k.shape[0], k.shape[1], k.shape[2], k.shape[3], _kv_dtype(k))
    c.tensors = (k, v, k_scale, v_scale)
    return c


def k3_kv_plan(ctx, new, parents, R, T, n_pages, page_size, blocks, held, ring, ring_state, table,
               held_out, ring_out, cu, kv_lens, slots, positions, mask, words, status,
               stream=None):
    _call("k3_kv_plan", _ints("ctx", ctx, R), _ints("new", new, R), _ints("parents", parents, T), R,
          T, n_pages, page_size, blocks, _ints("held", held, R), _ints("ring", ring, n_pages),
          _ints("ring_state", ring_state, 2), _ints("table", table, R * blocks),
          _ints("held_out", held_out, R), _ints("ring_out", ring_out, 2), _ints("cu", cu, R + 1),
          _ints("kv_lens", kv_lens, R), _ints("slots", slots, T), _ints("positions", positions, T),
          _ints("mask", mask, 0 if parents is None else T * words), words,
          _ints("status", status, 2), _stream(stream))


def k3_qk_norm_rope(q_in, k_in, v_in, T, Hq, wq, wk, eps, inv_freq, rot, interleaved, positions,
                    q_out, cache, slots, stream=None):
    code, dt, H, D = _kv_dtype(q_in), q_in.dtype, cache.n_heads, cache.head_dim
    wq, wk = _array("wq", wq, dt, D), _array("wk", wk, dt, D)
    _call("k3_qk_norm_rope", q_in.data_ptr(), _heads("q_in", q_in, dt, T, Hq, D), k_in.data_ptr(),
          _heads("k_in", k_in, dt, T, H, D), v_in.data_ptr(), _heads("v_in", v_in, dt, T, H, D), code, T,
          Hq, wq, wk, eps, _floats("inv_freq", inv_freq, rot // 2), rot, int(bool(interleaved)),
          _ints("positions", positions, T), q_out.data_ptr(), _heads("q_out", q_out, dt, T, Hq, D),
          ctypes.byref(cache), _ints("slots", slots, T), _stream(stream))


def k3_tree_attention_workspace_bytes(T, Hq, n_heads, head_dim):
    return lib().k3_tree_attention_workspace_bytes(T, Hq, n_heads, head_dim)


def k3_tree_attention(q, T, Hq, cache, table, blocks, cu, kv_lens, R, mask, words, scale, out, ws,
                      lse=None, stream=None):
    code, dt, D = _kv_dtype(q), q.dtype, cache.head_dim
    q_stride, out_stride = _heads("q", q, dt, T, Hq, D), _heads("out", out, dt, T, Hq, D)
    if not ws.is_contiguous():
        raise ValueError(f"ws: dense bytes, not {tuple(ws.shape)} with strides {ws.stride()}")
    _call("k3_tree_attention", q.data_ptr(), q_stride, code, T, Hq, ctypes.byref(cache),
          _ints("table", table, R * blocks), blocks, _ints("cu", cu, R + 1),
          _ints("kv_lens", kv_lens, R), R, _ints("mask", mask, T * words), words, scale, out.data_ptr(),
          out_stride, ws.data_ptr(), _nbytes(ws), _floats("lse", lse, T * Hq), _stream(stream))


def k3_kv_commit(cache, layers, layer_stride, table, blocks, ctx, accepted, n_accepted, most, R,
                 ctx_out, stream=None):
    _call("k3_kv_commit", ctypes.byref(cache), layers, layer_stride,
          _ints("table", table, R * blocks), blocks, _ints("ctx", ctx, R),
          _ints("accepted", accepted, R * most), _ints("n_accepted", n_accepted, R), most, R,
          _ints("ctx_out", ctx_out, R), _stream(stream))


def k3_kv_commit_ex(cache, layers, layer_stride, table, blocks, ctx, kv_lens, accepted, n_accepted, most,
                    R, ctx_out, stream=None):
    _call("k3_kv_commit_ex", ctypes.byref(cache), layers, layer_stride,
          _ints("table", table, R * blocks), blocks, _ints("ctx", ctx, R),
          _ints("kv_lens", kv_lens, R), _ints("accepted", accepted, R * most),
          _ints("n_accepted", n_accepted, R), most, R, _ints("ctx_out", ctx_out, R), _stream(stream))
