"""Thin ctypes binding of libtpx.so (include/tpx.h), same names as the C ABI.

Argument marshalling only: torch tensors supply device memory and streams, every
step of the computation runs in the library's CUDA kernels.  Loading fails loudly
if the library has not been built: there is no fallback path.
"""
import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libtpx.so")

TP_OK, TP_ERR_INVALID_ARG, TP_ERR_SHAPE, TP_ERR_ALIGN, TP_ERR_LAYOUT_MISMATCH = 0, 1, 2, 3, 4
TP_ERR_WORKSPACE, TP_ERR_CUDA, TP_ERR_TIMEOUT, TP_ERR_DEVICE_TIMEOUT, TP_ERR_UNSUPPORTED = 5, 6, 7, 8, 9
TP_BF16, TP_FP8_E4M3 = 0, 1
TP_W_GATE_UP, TP_W_DOWN, TP_W_QKV, TP_W_O, TP_W_VOCAB, TP_W_EMBED = 0, 1, 2, 3, 4, 5
TP_F_UNFUSED_REDUCE, TP_F_FP32_COLPAR_OUT = 0x1, 0x2
TP_F_KERNEL_SKINNY, TP_F_KERNEL_TC, TP_F_SERIAL, TP_F_SPLIT_BLOCK = 0x10, 0x20, 0x40, 0x80
TP_F_FP8_ACT = 0x200
TP_F_FP8_HILO = 0x400
TP_F_FOLD_NORM = 0x800
TP_ROPE_HALF, TP_ROPE_INTERLEAVED = 0, 1
TP_ROPE_NONE, TP_ROPE_LINEAR, TP_ROPE_WAVELENGTH, TP_ROPE_YARN = 0, 1, 2, 3

EXPORTS = ["tp_packed_bytes", "tp_describe", "tp_partition_weights", "tp_workspace_bytes",
           "tp_mlp_forward", "tp_proj_forward", "tp_reduce_partials", "tp_colpar_forward",
           "tp_rowpar_partials", "tp_rowpar_forward", "tp_rowpar_forward_noalloc",
           "tp_noalloc_scratch_capacity", "tp_rmsnorm", "tp_selftest_bounded_wait",
           "tp_layer_scratch_bytes", "tp_layer_forward", "tp_selftest_e4m3_decode", "tp_sync", "tp_status_str", "tp_launch_count",
           "tp_lm_head_forward", "tp_embed_lookup", "tp_attn_workspace_bytes", "tp_attn_decode",
           "tp_attn_block_workspace_bytes", "tp_attn_block_forward", "tp_quantize_fp8_per_token",
           "tp_paged_tables", "tp_rope_describe", "tp_rope_forward", "tp_rope_append",
           "tp_paged_attn_workspace_bytes", "tp_paged_attn_decode", "tp_paged_attn_block_workspace_bytes",
           "tp_paged_attn_block_forward", "tp_token_logprobs", "tp_prefix_attn_workspace_bytes",
           "tp_prefix_attn_decode", "tp_sample_tokens"]


class TpxError(RuntimeError):
    def __init__(self, status, where):
        self.status = status
        super().__init__(f"{where}: {status_str(status)} ({status})")


class Shape(ctypes.Structure):
    _fields_ = [("d", ctypes.c_int32), ("ffn", ctypes.c_int32), ("n_q_heads", ctypes.c_int32),
                ("n_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("t", ctypes.c_int32),
                ("wtype", ctypes.c_int32), ("vocab", ctypes.c_int32)]


class PackedDesc(ctypes.Structure):
    _fields_ = [("magic", ctypes.c_uint32), ("layout_version", ctypes.c_uint32),
                ("kind", ctypes.c_int32), ("wtype", ctypes.c_int32), ("shape", Shape),
                ("rows_per_shard", ctypes.c_int64), ("k_per_shard", ctypes.c_int64),
                ("shard_payload_bytes", ctypes.c_uint64), ("scales_offset", ctypes.c_uint64),
                ("shard_stride_bytes", ctypes.c_uint64), ("total_bytes", ctypes.c_uint64)]


class Pages(ctypes.Structure):
    """Geometry of a paged key-value cache (tp_pages)."""
    _fields_ = [("kv_dtype", ctypes.c_int32), ("page_size", ctypes.c_int32), ("n_pages", ctypes.c_int32),
                ("max_pages", ctypes.c_int32), ("table_stride", ctypes.c_int32)]


class RopeParams(ctypes.Structure):
    _fields_ = [("rot_dim", ctypes.c_int32), ("layout", ctypes.c_int32), ("scaling", ctypes.c_int32),
                ("original_len", ctypes.c_int32), ("theta", ctypes.c_double), ("factor", ctypes.c_double),
                ("low_freq_factor", ctypes.c_double), ("high_freq_factor", ctypes.c_double),
                ("beta_fast", ctypes.c_double), ("beta_slow", ctypes.c_double)]


class Rope(ctypes.Structure):
    """A described rotation (tp_rope)."""
    _fields_ = [("magic", ctypes.c_uint32), ("rot_dim", ctypes.c_int32), ("layout", ctypes.c_int32),
                ("mscale", ctypes.c_float), ("step", ctypes.c_uint64 * 128)]


_lib = None


def lib():
    """Load libtpx.so once; raise if it is missing (no CPU or eager fallback exists)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is not built; run __graft_entry__.build()")
        L = ctypes.CDLL(LIB_PATH)
        P, V, I32, U32, SZ = ctypes.POINTER, ctypes.c_void_p, ctypes.c_int32, ctypes.c_uint32, ctypes.c_size_t
        sig = {
            "tp_packed_bytes": (SZ, [P(Shape), I32]),
            "tp_describe": (I32, [P(Shape), I32, P(PackedDesc)]),
            "tp_partition_weights": (I32, [P(Shape), I32, V, V, V, SZ, P(PackedDesc), V]),
            "tp_workspace_bytes": (SZ, [P(Shape), I32, U32]),
            "tp_mlp_forward": (I32, [P(PackedDesc), V, P(PackedDesc), V, V, V, I32, V, V, V, SZ, U32, V]),
            "tp_proj_forward": (I32, [P(PackedDesc), V, P(PackedDesc), V, V, V, I32, V, V, V, V, SZ, U32, V]),
            "tp_reduce_partials": (I32, [V, I32, I32, I32, V, V, V]),
            "tp_colpar_forward": (I32, [P(PackedDesc), V, V, I32, V, V, SZ, U32, V]),
            "tp_rowpar_partials": (I32, [P(PackedDesc), V, V, I32, V, V]),
            "tp_rowpar_forward": (I32, [P(PackedDesc), V, V, V, I32, V, V, SZ, U32, V]),
            "tp_rowpar_forward_noalloc": (I32, [P(PackedDesc), V, V, V, I32, V, U32, V]),
            "tp_noalloc_scratch_capacity": (SZ, []),
            "tp_rmsnorm": (I32, [V, V, ctypes.c_float, I32, I32, V, V]),
            "tp_sync": (I32, [V, I32]),
            "tp_selftest_bounded_wait": (I32, [I32, V]),
            "tp_layer_scratch_bytes": (SZ, [P(Shape), I32]),
            "tp_selftest_e4m3_decode": (I32, [V, V, I32, V]),
            "tp_layer_forward": (I32, [P(PackedDesc), V, P(PackedDesc), V, P(PackedDesc), V, P(PackedDesc), V,
                                       V, I32, V, ctypes.c_float, V, SZ, V, SZ, U32, V]),
            "tp_status_str": (ctypes.c_char_p, [I32]),
            "tp_lm_head_forward": (I32, [P(PackedDesc), V, V, I32, V, V, SZ, U32, V]),
            "tp_embed_lookup": (I32, [P(PackedDesc), V, V, I32, V, V]),
            "tp_attn_workspace_bytes": (SZ, [P(Shape), I32, I32]),
            "tp_attn_decode": (I32, [P(Shape), V, V, V, I32, V, I32, V, V, SZ, V]),
            "tp_attn_block_workspace_bytes": (SZ, [P(Shape), I32, I32, U32]),
            "tp_quantize_fp8_per_token": (I32, [V, I32, I32, V, V, V]),
            "tp_attn_block_forward": (I32, [P(PackedDesc), V, P(PackedDesc), V, V, V, I32, V, V, I32, V, V, V, V,
                                            V, SZ, U32, V]),
            "tp_launch_count": (ctypes.c_uint64, []),
            "tp_paged_tables": (I32, [P(Pages), V, V, I32, V, I32, V, V, V, V, V, V, I32, V, V]),
            "tp_rope_describe": (I32, [P(RopeParams), P(Rope)]),
            "tp_rope_forward": (I32, [P(Shape), P(Rope), V, V, I32, V, V]),
            "tp_rope_append": (I32, [P(Shape), P(Rope), P(Pages), V, V, V, I32, V, V, V, V, V, V]),
            "tp_paged_attn_workspace_bytes": (SZ, [P(Shape)]),
            "tp_paged_attn_decode": (I32, [P(Shape), P(Pages), V, V, V, V, V, V, V, I32, ctypes.c_float, I32, V, V, V,
                                           SZ, V]),
            "tp_paged_attn_block_workspace_bytes": (SZ, [P(Shape), I32, U32]),
            "tp_paged_attn_block_forward": (I32, [P(PackedDesc), V, P(PackedDesc), V, V, V, I32, P(Rope), P(Pages), V, V,
                                                  V, V, V, V, V, V, I32, V, V, V, V, V, SZ, U32, V]),
            "tp_token_logprobs": (I32, [V, ctypes.c_int64, I32, I32, V, I32, V, V, V, V, V, V]),
            "tp_prefix_attn_workspace_bytes": (SZ, [P(Shape), I32]),
            "tp_prefix_attn_decode": (I32, [P(Shape), P(Pages), V, V, V, V, V, V, V, I32, V, V, I32, ctypes.c_float, I32,
                                            V, V, V, SZ, V]),
            "tp_sample_tokens": (I32, [V, ctypes.c_int64, I32, I32, V, V, V, V, V, V, V, V]),
        }
        for name, (res, args) in sig.items():
            f = getattr(L, name)
            f.restype, f.argtypes = res, args
        _lib = L
    return _lib


def status_str(s):
    return lib().tp_status_str(int(s)).decode()


def _check(st, where):
    if st != TP_OK:
        raise TpxError(st, where)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _flat(t, dtype, n):
    """Whether the C call can read n elements one after another from t.data_ptr() on (None: it is not given)."""
    return t is None or (t.dtype is dtype and t.is_contiguous() and t.numel() >= n)


_raw_stream = _device = None


def _stream(stream):
    global _raw_stream, _device
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is None:
        if not torch.cuda.is_available():
            return None
        torch.cuda.init()
        _raw_stream, _device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice
    # the current stream's handle, without a Stream object: a decode step makes many short calls
    return _raw_stream(_device())


def make_shape(d, ffn=0, n_q=0, n_kv=0, hd=0, t=1, wtype=TP_BF16, vocab=0):
    return Shape(d, ffn, n_q, n_kv, hd, t, wtype, vocab)


def tp_packed_bytes(shape, kind):
    return lib().tp_packed_bytes(ctypes.byref(shape), kind)


def tp_describe(shape, kind):
    d = PackedDesc()
    _check(lib().tp_describe(ctypes.byref(shape), kind, ctypes.byref(d)), "tp_describe")
    return d


def tp_workspace_bytes(shape, M, flags=0):
    return lib().tp_workspace_bytes(ctypes.byref(shape), M, flags)


def tp_partition_weights(shape, kind, W0, W1=None, stream=None, packed=None):
    """Returns (packed uint8 device tensor, PackedDesc)."""
    n = tp_packed_bytes(shape, kind)
    if n == 0:
        tp_describe(shape, kind)  # raises with the precise status
    if packed is None:
        packed = torch.empty(n, dtype=torch.uint8, device=W0.device)
    d = PackedDesc()
    _check(lib().tp_partition_weights(ctypes.byref(shape), kind, _ptr(W0), _ptr(W1), _ptr(packed),
                                      packed.numel(), ctypes.byref(d), _stream(stream)),
           "tp_partition_weights")
    return packed, d


def new_workspace(shape, M, device, flags=0):
    """Zero-filled workspace (the ticket counters must start at zero)."""
    return torch.zeros(max(1, tp_workspace_bytes(shape, M, flags)), dtype=torch.uint8, device=device)


def tp_mlp_forward(gu, gu_w, dn, dn_w, x, residual, y, h, ws, flags=0, stream=None):
    M = x.shape[0]
    _check(lib().tp_mlp_forward(ctypes.byref(gu), _ptr(gu_w), ctypes.byref(dn), _ptr(dn_w), _ptr(x),
                                _ptr(residual), M, _ptr(y), _ptr(h), _ptr(ws),
                                0 if ws is None else ws.numel(), flags, _stream(stream)),
           "tp_mlp_forward")
    return y


def tp_proj_forward(qkv, qkv_w, o, o_w, x, residual, y, qkv_out, o_in, ws, flags=0, stream=None):
    M = x.shape[0]
    _check(lib().tp_proj_forward(ctypes.byref(qkv), _ptr(qkv_w), ctypes.byref(o), _ptr(o_w), _ptr(x),
                                 _ptr(residual), M, _ptr(y), _ptr(qkv_out), _ptr(o_in), _ptr(ws),
                                 0 if ws is None else ws.numel(), flags, _stream(stream)),
           "tp_proj_forward")
    return y


def tp_reduce_partials(partials, t, M, d, residual, y, stream=None):
    _check(lib().tp_reduce_partials(_ptr(partials), t, M, d, _ptr(residual), _ptr(y), _stream(stream)),
           "tp_reduce_partials")
    return y


def tp_colpar_forward(desc, w, x, out, flags=0, stream=None, ws=None):
    _check(lib().tp_colpar_forward(ctypes.byref(desc), _ptr(w), _ptr(x), x.shape[0], _ptr(out), _ptr(ws),
                                   0 if ws is None else ws.numel(), flags, _stream(stream)), "tp_colpar_forward")
    return out


def tp_rowpar_partials(desc, w, a, partials, stream=None):
    _check(lib().tp_rowpar_partials(ctypes.byref(desc), _ptr(w), _ptr(a), a.shape[0], _ptr(partials),
                                    _stream(stream)), "tp_rowpar_partials")
    return partials


def tp_rowpar_forward(desc, w, a, residual, y, ws, flags=0, stream=None):
    _check(lib().tp_rowpar_forward(ctypes.byref(desc), _ptr(w), _ptr(a), _ptr(residual), a.shape[0], _ptr(y),
                                   _ptr(ws), 0 if ws is None else ws.numel(), flags, _stream(stream)),
           "tp_rowpar_forward")
    return y


def tp_rowpar_forward_noalloc(desc, w, a, residual, y, flags=0, stream=None):
    """tp_rowpar_forward without a workspace argument: for callers that cannot allocate
    device memory (the library's own static scratch array is used)."""
    _check(lib().tp_rowpar_forward_noalloc(ctypes.byref(desc), _ptr(w), _ptr(a), _ptr(residual), a.shape[0],
                                           _ptr(y), flags, _stream(stream)), "tp_rowpar_forward_noalloc")
    return y


def tp_noalloc_scratch_capacity():
    return lib().tp_noalloc_scratch_capacity()


def tp_rmsnorm(x, out, eps=1e-5, gain=None, stream=None):
    _check(lib().tp_rmsnorm(_ptr(x), _ptr(gain), eps, x.shape[0], x.shape[1], _ptr(out), _stream(stream)),
           "tp_rmsnorm")
    return out


def tp_sync(stream=None, timeout_ms=2000):
    return lib().tp_sync(_stream(stream), timeout_ms)


def tp_selftest_bounded_wait(timeout_us, stream=None):
    _check(lib().tp_selftest_bounded_wait(timeout_us, _stream(stream)), "tp_selftest_bounded_wait")


def tp_layer_scratch_bytes(shape, M):
    return lib().tp_layer_scratch_bytes(ctypes.byref(shape), M)


def tp_layer_forward(qkv, qkv_w, o, o_w, gu, gu_w, dn, dn_w, x, y, scratch, ws, eps=1e-5, flags=0, stream=None):
    _check(lib().tp_layer_forward(ctypes.byref(qkv), _ptr(qkv_w), ctypes.byref(o), _ptr(o_w), ctypes.byref(gu),
                                  _ptr(gu_w), ctypes.byref(dn), _ptr(dn_w), _ptr(x), x.shape[0], _ptr(y), eps,
                                  _ptr(scratch), scratch.numel(), _ptr(ws), ws.numel(), flags, _stream(stream)),
           "tp_layer_forward")
    return y


def tp_selftest_e4m3_decode(codes, out, stream=None):
    _check(lib().tp_selftest_e4m3_decode(_ptr(codes), _ptr(out), codes.numel(), _stream(stream)),
           "tp_selftest_e4m3_decode")
    return out


def tp_launch_count():
    return lib().tp_launch_count()


def tp_lm_head_forward(desc, w, x, logits, ws=None, flags=0, stream=None):
    _check(lib().tp_lm_head_forward(ctypes.byref(desc), _ptr(w), _ptr(x), x.shape[0], _ptr(logits), _ptr(ws),
                                    0 if ws is None else ws.numel(), flags, _stream(stream)), "tp_lm_head_forward")
    return logits


def tp_embed_lookup(desc, w, ids, x, stream=None):
    _check(lib().tp_embed_lookup(ctypes.byref(desc), _ptr(w), _ptr(ids), ids.shape[0], _ptr(x), _stream(stream)),
           "tp_embed_lookup")
    return x


def tp_attn_block_workspace_bytes(shape, M, L, flags=0):
    return lib().tp_attn_block_workspace_bytes(ctypes.byref(shape), M, L, flags)


def new_attn_block_workspace(shape, M, L, device, flags=0):
    """Zero-filled workspace of tp_attn_block_forward (its projection counters start at zero)."""
    return torch.zeros(max(1, tp_attn_block_workspace_bytes(shape, M, L, flags)), dtype=torch.uint8, device=device)


def tp_attn_block_forward(qkv, qkv_w, o, o_w, x, residual, k_cache, v_cache, lens, y, qkv_out, o_in, ws, flags=0,
                          stream=None):
    """k_cache, v_cache: [t, M, n_kv/t, L, hd] bf16; lens: [M] int32 on the device."""
    L = k_cache.shape[3]
    _check(lib().tp_attn_block_forward(ctypes.byref(qkv), _ptr(qkv_w), ctypes.byref(o), _ptr(o_w), _ptr(x),
                                       _ptr(residual), x.shape[0], _ptr(k_cache), _ptr(v_cache), L, _ptr(lens),
                                       _ptr(y), _ptr(qkv_out), _ptr(o_in), _ptr(ws), ws.numel(), flags,
                                       _stream(stream)), "tp_attn_block_forward")
    return y


def tp_quantize_fp8_per_token(x, q, s, stream=None):
    """x: [M, K] bf16; q: [M, K] uint8 codes; s: [M] fp32 (all on the device)."""
    _check(lib().tp_quantize_fp8_per_token(_ptr(x), x.shape[0], x.shape[1], _ptr(q), _ptr(s), _stream(stream)),
           "tp_quantize_fp8_per_token")
    return q, s


def tp_attn_workspace_bytes(shape, M, L):
    return lib().tp_attn_workspace_bytes(ctypes.byref(shape), M, L)


def tp_attn_decode(shape, qkv, k_cache, v_cache, lens, o_in, ws, stream=None):
    """k_cache, v_cache: [t, M, n_kv/t, L, hd] bf16; lens: [M] int32 on the device."""
    L = k_cache.shape[3]
    _check(lib().tp_attn_decode(ctypes.byref(shape), _ptr(qkv), _ptr(k_cache), _ptr(v_cache), L, _ptr(lens),
                                qkv.shape[0], _ptr(o_in), _ptr(ws), ws.numel(), _stream(stream)), "tp_attn_decode")
    return o_in


def make_pages(page_size, n_pages, max_pages, kv_dtype=TP_BF16, table_stride=None):
    """Geometry of a paged cache; max_pages: page ids in a row of the block table."""
    return Pages(kv_dtype, page_size, n_pages, max_pages, max_pages if table_stride is None else table_stride)


def tp_rope_describe(params):
    r = Rope()
    _check(lib().tp_rope_describe(ctypes.byref(params), ctypes.byref(r)), "tp_rope_describe")
    return r


def make_rope(rot_dim, theta=10000.0, layout=TP_ROPE_HALF, scaling=TP_ROPE_NONE, factor=1.0, original_len=0,
              low_freq_factor=1.0, high_freq_factor=4.0, beta_fast=32.0, beta_slow=1.0):
    return tp_rope_describe(RopeParams(rot_dim, layout, scaling, original_len, theta, factor, low_freq_factor,
                                       high_freq_factor, beta_fast, beta_slow))


def tp_paged_tables(pages, lens, add, free_pages, block_table, lens_out, cu_rows, positions, slots, counts, head=None,
                    stream=None):
    """All int32 on the device: lens, add, lens_out [M]; free_pages [n_free]; block_table [M, table_stride]; cu_rows
    [M + 1]; positions, slots [rows]; counts [3]; head: one element or None.  Returns slots.  With no requests nothing
    is written, counts included: keep the set written last as the next step's lens and head."""
    _check(lib().tp_paged_tables(ctypes.byref(pages), _ptr(lens), _ptr(add), lens.shape[0], _ptr(free_pages),
                                 free_pages.shape[0], _ptr(head), _ptr(block_table), _ptr(lens_out), _ptr(cu_rows),
                                 _ptr(positions), _ptr(slots), slots.shape[0], _ptr(counts), _stream(stream)),
           "tp_paged_tables")
    return slots


def tp_rope_forward(shape, rope, qkv, positions, qkv_out, stream=None):
    """qkv, qkv_out (may be qkv): [M, (n_q + 2 n_kv) hd] bf16; positions: [M] int32 on the device."""
    _check(lib().tp_rope_forward(ctypes.byref(shape), ctypes.byref(rope), _ptr(qkv), _ptr(positions), qkv.shape[0],
                                 _ptr(qkv_out), _stream(stream)), "tp_rope_forward")
    return qkv_out


def tp_rope_append(shape, rope, pages, qkv, positions, slots, q_out, k_pages, v_pages, k_scale=None, v_scale=None,
                   stream=None):
    """q_out: [M, n_q hd] bf16; k_pages, v_pages: [t, n_pages, n_kv/t, page_size, hd], bf16 or e4m3 codes with scales
    [n_kv] fp32; positions, slots: [M] int32 on the device.  rope None: append without turning."""
    _check(lib().tp_rope_append(ctypes.byref(shape), None if rope is None else ctypes.byref(rope), ctypes.byref(pages),
                                _ptr(qkv), _ptr(positions), _ptr(slots), qkv.shape[0], _ptr(q_out), _ptr(k_pages),
                                _ptr(v_pages), _ptr(k_scale), _ptr(v_scale), _stream(stream)), "tp_rope_append")
    return q_out


def tp_paged_attn_workspace_bytes(shape):
    return lib().tp_paged_attn_workspace_bytes(ctypes.byref(shape))


def new_paged_attn_workspace(shape, device):
    """Zero-filled workspace of tp_paged_attn_decode (its counters start at zero), for every M and length."""
    return torch.zeros(max(1, tp_paged_attn_workspace_bytes(shape)), dtype=torch.uint8, device=device)


def tp_paged_attn_decode(shape, pages, q, k_pages, v_pages, block_table, lens, o_in, ws, lse=None, scale=0.0, window=0,
                         k_scale=None, v_scale=None, stream=None):
    """q, o_in: [M, n_q hd] bf16; lse: [M, n_q] fp32 or None; block_table: [M, table_stride], lens: [M] int32 on the
    device; the pages as for tp_rope_append."""
    _check(lib().tp_paged_attn_decode(ctypes.byref(shape), ctypes.byref(pages), _ptr(q), _ptr(k_pages), _ptr(v_pages),
                                      _ptr(k_scale), _ptr(v_scale), _ptr(block_table), _ptr(lens), q.shape[0], scale,
                                      window, _ptr(o_in), _ptr(lse), _ptr(ws), ws.numel(), _stream(stream)),
           "tp_paged_attn_decode")
    return o_in


def tp_prefix_attn_workspace_bytes(shape, M):
    return lib().tp_prefix_attn_workspace_bytes(ctypes.byref(shape), M)


def new_prefix_attn_workspace(shape, M, device):
    """Zero-filled workspace of tp_prefix_attn_decode (its counters start at zero), for calls of up to M requests."""
    return torch.zeros(max(1, tp_prefix_attn_workspace_bytes(shape, M)), dtype=torch.uint8, device=device)


def tp_prefix_attn_decode(shape, pages, q, k_pages, v_pages, block_table, lens, cu_groups, prefix_lens, o_in, ws,
                          lse=None, scale=0.0, window=0, k_scale=None, v_scale=None, stream=None):
    """As tp_paged_attn_decode, with the requests cu_groups[g] .. cu_groups[g + 1] - 1 sharing their first
    prefix_lens[g] positions' whole pages; cu_groups [n + 1], prefix_lens [n]: int32 on the device.  All tensors but the
    block table, whose rows are pages.table_stride apart, are contiguous.  pages.max_pages, what a row can name, says
    whether sharing is worth looking at: give the longest request's pages where the host knows them."""
    n_groups = prefix_lens.shape[0]
    if cu_groups.shape[0] != n_groups + 1:
        raise TpxError(TP_ERR_INVALID_ARG, "tp_prefix_attn_decode: cu_groups and prefix_lens")
    M, heads, i32, f32, bf16 = q.shape[0], shape.n_q_heads, torch.int32, torch.float32, torch.bfloat16
    row, held = heads * shape.head_dim, pages.n_pages * pages.page_size * shape.n_kv_heads * shape.head_dim
    kv = bf16 if pages.kv_dtype == TP_BF16 else torch.uint8 if k_pages.dtype is torch.uint8 else torch.float8_e4m3fn
    if not (_flat(q, bf16, M * row) and _flat(o_in, bf16, M * row) and _flat(k_pages, kv, held) and _flat(v_pages, kv, held)
            and _flat(lens, i32, M) and _flat(cu_groups, i32, 1) and _flat(prefix_lens, i32, 0) and _flat(lse, f32, M * heads)
            and _flat(k_scale, f32, shape.n_kv_heads) and _flat(v_scale, f32, shape.n_kv_heads)):
        raise TpxError(TP_ERR_INVALID_ARG, "tp_prefix_attn_decode: a tensor's type, length or strides")
    rows, pitch = block_table.shape, block_table.stride()
    if block_table.dtype is not i32 or len(rows) != 2 or rows[0] < M or rows[1] < pages.max_pages or \
            (pitch[1] != 1 and rows[1] > 1) or (pitch[0] != pages.table_stride and M > 1):
        raise TpxError(TP_ERR_INVALID_ARG, "tp_prefix_attn_decode: block_table")
    _check(lib().tp_prefix_attn_decode(ctypes.byref(shape), ctypes.byref(pages), _ptr(q), _ptr(k_pages), _ptr(v_pages),
                                       _ptr(k_scale), _ptr(v_scale), _ptr(block_table), _ptr(lens), M,
                                       _ptr(cu_groups), _ptr(prefix_lens), n_groups, scale, window,
                                       _ptr(o_in), _ptr(lse), _ptr(ws), ws.numel(), _stream(stream)),
           "tp_prefix_attn_decode")
    return o_in


def tp_paged_attn_block_workspace_bytes(shape, M, flags=0):
    return lib().tp_paged_attn_block_workspace_bytes(ctypes.byref(shape), M, flags)


def new_paged_attn_block_workspace(shape, M, device, flags=0):
    """Zero-filled workspace of tp_paged_attn_block_forward, for calls of up to M rows in any order."""
    return torch.zeros(max(1, tp_paged_attn_block_workspace_bytes(shape, M, flags)), dtype=torch.uint8, device=device)


def tp_paged_attn_block_forward(qkv, qkv_w, o, o_w, x, residual, rope, pages, positions, slots, k_pages, v_pages,
                                block_table, lens, y, qkv_out, q_out, o_in, ws, window=0, k_scale=None, v_scale=None,
                                flags=0, stream=None):
    """x, residual (or None), y: [M, d] bf16; qkv_out [M, (n_q + 2 n_kv) hd], q_out and o_in [M, n_q hd] bf16; the
    cache as for tp_rope_append and tp_paged_attn_decode; lens counts the new token."""
    _check(lib().tp_paged_attn_block_forward(ctypes.byref(qkv), _ptr(qkv_w), ctypes.byref(o), _ptr(o_w), _ptr(x),
                                             _ptr(residual), x.shape[0], None if rope is None else ctypes.byref(rope),
                                             ctypes.byref(pages), _ptr(positions), _ptr(slots), _ptr(k_pages),
                                             _ptr(v_pages), _ptr(k_scale), _ptr(v_scale), _ptr(block_table), _ptr(lens),
                                             window, _ptr(y), _ptr(qkv_out), _ptr(q_out), _ptr(o_in), _ptr(ws),
                                             ws.numel(), flags, _stream(stream)), "tp_paged_attn_block_forward")
    return y


def tp_token_logprobs(logits, ids, logprob, entropy, rank, top_logprob=None, top_id=None, stream=None):
    """logits: [M, vocab] fp32, rows logits.stride(0) apart, a row's logits next to one another; ids, rank: [M] int32;
    logprob, entropy: [M] fp32; top_logprob, top_id: [M, k], both or neither (all on the device; ids, logprob, entropy
    and rank may be None)."""
    if logits.shape[1] > 1 and logits.stride(1) != 1:
        raise TpxError(TP_ERR_INVALID_ARG, "tp_token_logprobs: logits' stride along the vocabulary")
    if (top_logprob is None) != (top_id is None) or (top_id is not None and top_logprob.shape != top_id.shape):
        raise TpxError(TP_ERR_INVALID_ARG, "tp_token_logprobs: top_logprob and top_id")
    k = 0 if top_id is None else top_id.shape[1]
    ldl = logits.stride(0) if logits.shape[0] > 1 else logits.shape[1]
    _check(lib().tp_token_logprobs(_ptr(logits), ldl, logits.shape[0], logits.shape[1], _ptr(ids), k, _ptr(logprob),
                                   _ptr(rank), _ptr(entropy), _ptr(top_logprob), _ptr(top_id), _stream(stream)),
           "tp_token_logprobs")
    return logprob


def tp_sample_tokens(logits, u, ids, temperature=None, top_k=None, top_p=None, min_p=None, logprob=None, stream=None):
    """logits: [M, vocab] fp32, rows logits.stride(0) apart, a row's logits next to one another; u, temperature, top_p,
    min_p, logprob: [M] fp32, ids, top_k: [M] int32, contiguous (all on the device; the settings and logprob may be
    None)."""
    (M, V), (pitch, step), i32, f32 = logits.shape, logits.stride(), torch.int32, torch.float32
    if logits.dtype is not f32 or (V > 1 and step != 1):
        raise TpxError(TP_ERR_INVALID_ARG, "tp_sample_tokens: logits' type, or stride along the vocabulary")
    if not (_flat(u, f32, M) and _flat(ids, i32, M) and _flat(temperature, f32, M) and _flat(top_k, i32, M)
            and _flat(top_p, f32, M) and _flat(min_p, f32, M) and _flat(logprob, f32, M)):
        raise TpxError(TP_ERR_INVALID_ARG, "tp_sample_tokens: a tensor's type, length or strides")
    _check(lib().tp_sample_tokens(_ptr(logits), pitch if M > 1 else V, M, V, _ptr(u), _ptr(temperature), _ptr(top_k),
                                  _ptr(top_p), _ptr(min_p), _ptr(ids), _ptr(logprob), _stream(stream)),
           "tp_sample_tokens")
    return ids
