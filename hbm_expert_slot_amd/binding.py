"""ctypes binding of libslotcache (include/slotcache.h): argument marshalling only.

Every function keeps the C name and raises SlotCacheError on a non-OK status.
The library is loaded from this package directory; if it is missing the
import of a call fails loudly -- there is no fallback implementation.
"""
import ctypes
import os
import struct

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libslotcache.so")

SC_OK = 0
SC_E_ARG = -1
SC_E_HOST_OOM = -2
SC_E_HIP = -3
SC_E_STATE = -4
SC_E_DEVICE = -5
SC_E_UNSUPPORTED = -6
SC_BYPASS_ROWS = 16
SC_FLAG_BATCH_INVARIANT = 1
SC_FLAG_OVERLAP_FILL = 2
SC_MFMA_MIN_ROWS_GATEUP = 5
SC_MFMA_MIN_ROWS_DOWN = 5
SC_N_KERNELS = 5
SC_N_EVENTS = 2 * SC_N_KERNELS
SC_STATIC_SCRATCH_BYTES = 16777216
SC_DTYPE_F32 = 0
SC_DTYPE_BF16 = 1
SC_DTYPE_F16 = 2
SC_FP4_NV = 0
SC_FP4_MX = 1
SC_FP4_QUANT_WORKSPACE_BYTES = 4096
SC_MOE_MAX_ROWS = 16
SC_SCORE_SOFTMAX = 0
SC_SCORE_SIGMOID = 1
SC_PROMPT_MAX_HEADS = 1024
SC_PROMPT_MAX_SEQS = 65536
SC_PROMPT_MAX_ROWS = 1 << 24
SC_PROMPT_MAX_STRIDE = 1 << 23
SC_PROMPT_PART_KEYS = 2048
SC_KV4_PAGE = 64
SC_KV4_MAX_HEADS = 1024
SC_KV4_MAX_SEQS = 65536
SC_KV4_MAX_WIDTH = 1 << 24
SC_KV4_MAX_ROWS = 16
SC_KV4_MAX_GROUP = 64

EXPORTED = (
    "slotcache_query_sizes", "slotcache_init", "slotcache_backing", "slotcache_set_global_scales",
    "slotcache_preload", "moe_layer_decode", "moe_layer_decode_ev", "slotcache_stats",
    "slotcache_read_state", "slotcache_write_state", "slotcache_read_events",
    "slotcache_read_routing", "slotcache_read_kernel_spans", "slotcache_pin", "slotcache_last_error",
    "slotcache_destroy", "moe_layer_decode_static", "fp4_quantize", "fp4_dequantize", "fp4_linear",
    "moe_layer_workspace_bytes", "moe_layer_prepare", "moe_layer_forward",
    "prompt_attention_workspace_bytes", "prompt_attention",
    "kv4_page_bytes", "kv4_append", "kv4_read", "kv4_attention_workspace_bytes", "kv4_attention",
    "kv4_evict_workspace_bytes", "kv4_evict",
)


class SlotCacheError(RuntimeError):
    def __init__(self, status, message):
        super().__init__("slotcache status %d: %s" % (status, message))
        self.status = status


class sc_config(ctypes.Structure):
    _fields_ = [
        ("n_layers", ctypes.c_int32), ("hidden", ctypes.c_int32), ("inter", ctypes.c_int32),
        ("n_experts", ctypes.c_int32), ("top_k", ctypes.c_int32),
        ("slots_per_layer", ctypes.POINTER(ctypes.c_int32)), ("max_rows", ctypes.c_int32),
        ("n_banks", ctypes.c_int32), ("event_capacity", ctypes.c_int32), ("flags", ctypes.c_uint32),
        ("prefill_stage", ctypes.c_int32),
    ]


class sc_sizes(ctypes.Structure):
    _fields_ = [
        ("blob_bytes", ctypes.c_size_t), ("slot_pool_bytes", ctypes.c_size_t),
        ("state_bytes", ctypes.c_size_t), ("workspace_bytes", ctypes.c_size_t),
        ("backing_bytes_per_bank", ctypes.c_size_t),
    ]


class sc_stats(ctypes.Structure):
    _fields_ = [(n, ctypes.c_uint64) for n in (
        "steps", "bypass_steps", "picks", "lookups", "hits", "misses", "evictions",
        "bytes_filled", "bypass_bytes")] + [("device_error", ctypes.c_uint32), ("reserved", ctypes.c_uint32)]


class sc_event(ctypes.Structure):
    _fields_ = [("step", ctypes.c_int64), ("expert", ctypes.c_int32), ("slot", ctypes.c_int32),
                ("evicted", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class sc_fp4_matrix(ctypes.Structure):
    _fields_ = [("format", ctypes.c_int32), ("rows", ctypes.c_int32), ("cols", ctypes.c_int32),
                ("d_codes", ctypes.c_void_p), ("d_scales", ctypes.c_void_p),
                ("d_global_scale", ctypes.c_void_p)]


class sc_moe_config(ctypes.Structure):
    _fields_ = [("hidden", ctypes.c_int32), ("inter", ctypes.c_int32), ("n_experts", ctypes.c_int32),
                ("top_k", ctypes.c_int32), ("shared_inter", ctypes.c_int32), ("max_rows", ctypes.c_int32),
                ("score", ctypes.c_int32), ("routed_scale", ctypes.c_float)]


class sc_moe_weights(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in (
        "d_router", "d_score_bias", "d_blobs", "d_global_scales", "d_shared_blob", "d_shared_scales")]


class sc_prompt(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "type", "head_dim", "q_heads", "kv_heads", "n_seqs", "rows", "keys")] + [("scale", ctypes.c_float)] + [
        (n, ctypes.c_void_p) for n in ("d_q", "d_k", "d_v", "d_out", "d_lse", "d_starts", "d_key_starts")] + [
        (n, ctypes.c_int64 * 2) for n in ("q_stride", "k_stride", "v_stride", "out_stride")]


class sc_kv4_cache(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("format", "head_dim", "kv_heads", "n_pages")] + [
        (n, ctypes.c_void_p) for n in ("d_pages", "d_weights", "d_positions", "d_k_scale", "d_v_scale")]


class sc_kv4_seqs(ctypes.Structure):
    _fields_ = [("n_seqs", ctypes.c_int32), ("width", ctypes.c_int32), ("ld_table", ctypes.c_int64),
                ("d_table", ctypes.c_void_p), ("d_lens", ctypes.c_void_p)]


class sc_kv4_rows(ctypes.Structure):
    _fields_ = [("type", ctypes.c_int32), ("d_k", ctypes.c_void_p), ("d_v", ctypes.c_void_p)] + [
        (n, ctypes.c_int64) for n in ("k_token", "k_head", "v_token", "v_head")]


class sc_kv4_query(ctypes.Structure):
    _fields_ = [("type", ctypes.c_int32), ("rows", ctypes.c_int32), ("q_heads", ctypes.c_int32),
                ("scale", ctypes.c_float), ("d_q", ctypes.c_void_p), ("d_out", ctypes.c_void_p),
                ("q_stride", ctypes.c_int64 * 3), ("out_stride", ctypes.c_int64 * 3)]


# The same structures as bytes, which cost a call less than ctypes objects.
PROMPT = struct.Struct("@7if7N8q")
KV4_SEQS = struct.Struct("@2iq2N")
KV4_ROWS = struct.Struct("@i4x2N4q")
KV4_QUERY = struct.Struct("@3if2N6q")

_lib = None


def lib():
    """The loaded library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("libslotcache.so is not built; run python -m hbm_expert_slot_amd.build")
        L = ctypes.CDLL(LIB_PATH)
        P = ctypes.c_void_p
        i32, i64, sz = ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
        sig = {
            "slotcache_query_sizes": [ctypes.POINTER(sc_config), ctypes.POINTER(sc_sizes)],
            "slotcache_init": [ctypes.POINTER(sc_config), P, P, P, ctypes.POINTER(P)],
            "slotcache_backing": [P, i32, ctypes.POINTER(P), ctypes.POINTER(sz)],
            "slotcache_set_global_scales": [P, i32, P],
            "slotcache_preload": [P, i32],
            "moe_layer_decode": [P, i32, P, P, i32, P, P],
            "moe_layer_decode_ev": [P, i32, P, P, i32, P, P, P],
            "moe_layer_decode_static": [P, i32, P, P, i32, P, P],
            "slotcache_stats": [P, i32, ctypes.POINTER(sc_stats)],
            "slotcache_read_state": [P, i32, P, P, P, P],
            "slotcache_write_state": [P, i32, P, P, P, i64],
            "slotcache_read_events": [P, i32, P, sz, ctypes.POINTER(sz), ctypes.POINTER(ctypes.c_uint64)],
            "slotcache_read_routing": [P, P, P, ctypes.POINTER(i32), ctypes.POINTER(i32)],
            "slotcache_read_kernel_spans": [P, ctypes.POINTER(ctypes.c_double)],
            "slotcache_pin": [P, i32, P, i32],
            "fp4_quantize": [P, i32, i64, ctypes.POINTER(sc_fp4_matrix), i32, P, P],
            "fp4_dequantize": [ctypes.POINTER(sc_fp4_matrix), P, i32, i64, P],
            "moe_layer_workspace_bytes": [ctypes.POINTER(sc_moe_config), ctypes.POINTER(sz)],
            "moe_layer_prepare": [ctypes.POINTER(sc_moe_config), P, P],
            "moe_layer_forward": [ctypes.POINTER(sc_moe_config), ctypes.POINTER(sc_moe_weights), P, P, i64, i32, P,
                                  i32, i64, P, P, P],
            "prompt_attention_workspace_bytes": [P, ctypes.POINTER(sz)],
            "prompt_attention": [P, P, P],
            "kv4_page_bytes": [i32, i32, ctypes.POINTER(sz)],
            "kv4_append": [P, P, P, i32, P, P, P],
            "kv4_read": [P, P, P, i32, P, P],
            "kv4_attention_workspace_bytes": [P, P, i32, i32, i32, ctypes.POINTER(sz)],
            "kv4_attention": [P, P, P, i32, P, P],
            "kv4_evict_workspace_bytes": [P, P, i32, ctypes.POINTER(sz)],
            "kv4_evict": [P, P, i32, i32, i32, P, P, P],
            "fp4_linear": [ctypes.POINTER(sc_fp4_matrix), P, i32, i64, i32, P, P, i32, i64, P],
        }
        for name, args in sig.items():
            f = getattr(L, name)
            f.argtypes = args
            f.restype = ctypes.c_int
        L.slotcache_last_error.argtypes = []
        L.slotcache_last_error.restype = ctypes.c_char_p
        L.slotcache_destroy.argtypes = [P]
        L.slotcache_destroy.restype = None
        _lib = L
    return _lib


def _check(st):
    if st != SC_OK:
        raise SlotCacheError(st, lib().slotcache_last_error().decode())


def make_config(n_layers, hidden, inter, n_experts, top_k, slots_per_layer, max_rows,
                n_banks=1, event_capacity=0, flags=0, prefill_stage=0):
    arr = (ctypes.c_int32 * n_layers)(*[int(s) for s in slots_per_layer])
    cfg = sc_config(n_layers, hidden, inter, n_experts, top_k,
                    ctypes.cast(arr, ctypes.POINTER(ctypes.c_int32)), max_rows, n_banks,
                    event_capacity, flags, prefill_stage)
    cfg._keep = arr
    return cfg


def slotcache_query_sizes(cfg):
    out = sc_sizes()
    _check(lib().slotcache_query_sizes(ctypes.byref(cfg), ctypes.byref(out)))
    return out


def slotcache_init(cfg, d_slot_pool, d_state, d_workspace):
    h = ctypes.c_void_p()
    _check(lib().slotcache_init(ctypes.byref(cfg), d_slot_pool, d_state, d_workspace, ctypes.byref(h)))
    return h


def slotcache_backing(h, bank):
    p, n = ctypes.c_void_p(), ctypes.c_size_t()
    _check(lib().slotcache_backing(h, bank, ctypes.byref(p), ctypes.byref(n)))
    return p.value, n.value


def slotcache_set_global_scales(h, bank, h_gs_ptr):
    _check(lib().slotcache_set_global_scales(h, bank, h_gs_ptr))


def slotcache_preload(h, layer):
    _check(lib().slotcache_preload(h, layer))


def moe_layer_decode(h, layer, d_logits, d_x, M, d_y, stream):
    _check(lib().moe_layer_decode(h, layer, d_logits, d_x, M, d_y, stream))


def moe_layer_decode_static(h, layer, d_logits, d_x, M, d_y, stream):
    _check(lib().moe_layer_decode_static(h, layer, d_logits, d_x, M, d_y, stream))


def moe_layer_decode_ev(h, layer, d_logits, d_x, M, d_y, stream, events):
    _check(lib().moe_layer_decode_ev(h, layer, d_logits, d_x, M, d_y, stream, events))


def slotcache_stats(h, layer):
    out = sc_stats()
    _check(lib().slotcache_stats(h, layer, ctypes.byref(out)))
    return out


def slotcache_read_state(h, layer, e2s_ptr, s2e_ptr, key_ptr, step_ptr):
    _check(lib().slotcache_read_state(h, layer, e2s_ptr, s2e_ptr, key_ptr, step_ptr))


def slotcache_write_state(h, layer, e2s_ptr, s2e_ptr, key_ptr, step):
    _check(lib().slotcache_write_state(h, layer, e2s_ptr, s2e_ptr, key_ptr, step))


def slotcache_read_events(h, layer, buf_ptr, cap):
    n, tot = ctypes.c_size_t(), ctypes.c_uint64()
    _check(lib().slotcache_read_events(h, layer, buf_ptr, cap, ctypes.byref(n), ctypes.byref(tot)))
    return n.value, tot.value


def slotcache_read_routing(h, ids_ptr, w_ptr):
    M, byp = ctypes.c_int32(), ctypes.c_int32()
    _check(lib().slotcache_read_routing(h, ids_ptr, w_ptr, ctypes.byref(M), ctypes.byref(byp)))
    return M.value, byp.value


def slotcache_pin(h, layer, experts_ptr, n):
    _check(lib().slotcache_pin(h, layer, experts_ptr, n))


def slotcache_read_kernel_spans(h):
    """Execution spans (us) of the kernels of the last timed step."""
    out = (ctypes.c_double * SC_N_KERNELS)()
    _check(lib().slotcache_read_kernel_spans(h, out))
    return list(out)


def fp4_quantize(d_w, w_type, ldw, out, scale_given, d_workspace, stream):
    _check(lib().fp4_quantize(d_w, w_type, ldw, out, scale_given, d_workspace, stream))


def fp4_dequantize(w, d_w, w_type, ldw, stream):
    _check(lib().fp4_dequantize(w, d_w, w_type, ldw, stream))


def fp4_linear(w, d_x, x_type, ldx, M, d_bias, d_y, y_type, ldy, stream):
    _check(lib().fp4_linear(w, d_x, x_type, ldx, M, d_bias, d_y, y_type, ldy, stream))


def moe_layer_workspace_bytes(cfg):
    n = ctypes.c_size_t()
    _check(lib().moe_layer_workspace_bytes(cfg, ctypes.byref(n)))
    return n.value


def moe_layer_prepare(cfg, d_workspace, stream):
    _check(lib().moe_layer_prepare(cfg, d_workspace, stream))


def moe_layer_forward(cfg, w, d_workspace, d_x, ldx, M, d_y, y_type, ldy, d_ids, d_weights, stream):
    _check(lib().moe_layer_forward(cfg, w, d_workspace, d_x, ldx, M, d_y, y_type, ldy, d_ids, d_weights, stream))


def prompt_attention_workspace_bytes(p):
    n = ctypes.c_size_t()
    _check(lib().prompt_attention_workspace_bytes(p, ctypes.byref(n)))
    return n.value


def prompt_attention(p, d_workspace, stream):
    _check(lib().prompt_attention(p, d_workspace, stream))


def kv4_page_bytes(fmt, head_dim):
    n = ctypes.c_size_t()
    _check(lib().kv4_page_bytes(fmt, head_dim, ctypes.byref(n)))
    return n.value


def kv4_append(cache, seqs, rows, tokens, d_starts, d_positions, stream):
    _check(lib().kv4_append(cache, seqs, rows, tokens, d_starts, d_positions, stream))


def kv4_read(cache, seqs, rows, tokens, d_starts, stream):
    _check(lib().kv4_read(cache, seqs, rows, tokens, d_starts, stream))


def kv4_attention_workspace_bytes(cache, seqs, rows, q_heads, accumulate):
    n = ctypes.c_size_t()
    _check(lib().kv4_attention_workspace_bytes(cache, seqs, rows, q_heads, accumulate, ctypes.byref(n)))
    return n.value


def kv4_attention(cache, seqs, query, accumulate, d_workspace, stream):
    _check(lib().kv4_attention(cache, seqs, query, accumulate, d_workspace, stream))


def kv4_evict_workspace_bytes(cache, seqs, keep):
    n = ctypes.c_size_t()
    _check(lib().kv4_evict_workspace_bytes(cache, seqs, keep, ctypes.byref(n)))
    return n.value


def kv4_evict(cache, seqs, keep, recent, sinks, d_new_lens, d_workspace, stream):
    _check(lib().kv4_evict(cache, seqs, keep, recent, sinks, d_new_lens, d_workspace, stream))


def slotcache_last_error():
    return lib().slotcache_last_error().decode()


def slotcache_destroy(h):
    lib().slotcache_destroy(h)
