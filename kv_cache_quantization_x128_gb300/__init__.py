"""Python binding of libkvarn (KVarN tile quantization + paged decode attention on
GB300). Argument marshalling only: every step runs in the CUDA library, whose C
ABI is declared in include/kvarn.h. Tensors are torch CUDA tensors; PyTorch only
provides device memory and streams.

Importing this module loads ``libkvarn.so`` built in-tree by ``build_lib.build()``;
if the library is missing the import fails (there is no fallback).
"""
from __future__ import annotations

import ctypes
import os
import struct

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libkvarn.so")

RECORD_BYTES = 14336
HEAD_DIM = 128
BLOCK_SIZE = 128

KVARN_OK, KVARN_EINVAL, KVARN_EUNSUPPORTED, KVARN_EALIGN, KVARN_ESCRATCH, KVARN_ECUDA = range(6)
FLAG_BAD_SLOTS, FLAG_BAD_BLOCK, FLAG_BAD_LENGTH, FLAG_WAIT_TIMEOUT, FLAG_BAD_INDEX = 0x1, 0x2, 0x4, 0x8, 0x10
KVARN_F16, KVARN_BF16, KVARN_F32 = range(3)
KVARN_MAX_TREE = 64
KVARN_MAX_AXES = 4
KVARN_WAIT_MBARRIER, KVARN_WAIT_GRID = 0, 1

# exported entry points and their C signatures (include/kvarn.h)
_SIGS = {
    "kvarn_record_bytes": (ctypes.c_size_t, []),
    "kvarn_meta_record_bytes": (ctypes.c_size_t, [ctypes.c_void_p]),
    "kvarn_cache_bytes": (ctypes.c_size_t, [ctypes.c_void_p]),
    "kvarn_workspace_bytes": (ctypes.c_size_t, [ctypes.c_void_p, ctypes.c_int32]),
    "kvarn_decode_scratch_bytes": (ctypes.c_size_t, [ctypes.c_void_p, ctypes.c_int32]),
    "kvarn_quantize_tiles": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64,
                                            ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]),
    "kvarn_append_decode": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                           ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p, ctypes.c_void_p,
                                           ctypes.c_void_p, ctypes.c_void_p]),
    "kvarn_decode_attention": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                              ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p, ctypes.c_void_p,
                                              ctypes.c_size_t, ctypes.c_void_p, ctypes.c_void_p]),
    "kvarn_decode_attention_static": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                                     ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32,
                                                     ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]),
    "kvarn_serve_step": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p,
                                        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t,
                                        ctypes.c_void_p, ctypes.c_void_p]),
    "kvarn_prefill_attention": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                               ctypes.c_void_p, ctypes.c_int32, ctypes.c_int32, ctypes.c_void_p,
                                               ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                               ctypes.c_void_p]),
    "kvarn_qk_norm_rope": (ctypes.c_int, [ctypes.c_void_p] * 8 + [ctypes.c_int64] + [ctypes.c_void_p] * 5),
    "kvarn_qk_norm_rope_axes": (ctypes.c_int, [ctypes.c_void_p] * 9 + [ctypes.c_int64] + [ctypes.c_void_p] * 5),
    "kvarn_decode_weights_scratch_bytes": (ctypes.c_size_t, [ctypes.c_void_p, ctypes.c_int32]),
    "kvarn_decode_attention_weights": (ctypes.c_int, [ctypes.c_void_p] * 5 + [ctypes.c_int32, ctypes.c_float]
                                       + [ctypes.c_void_p] * 4 + [ctypes.c_size_t, ctypes.c_void_p, ctypes.c_void_p]),
    "kvarn_evict_tiles": (ctypes.c_int, [ctypes.c_void_p] * 6 + [ctypes.c_int32] * 3 + [ctypes.c_void_p] * 4),
    "kvarn_tree_scratch_bytes": (ctypes.c_size_t, [ctypes.c_void_p, ctypes.c_int32, ctypes.c_int32]),
    "kvarn_tree_attention": (ctypes.c_int, [ctypes.c_void_p] * 7 + [ctypes.c_int32, ctypes.c_int64, ctypes.c_int32]
                             + [ctypes.c_void_p] * 6 + [ctypes.c_size_t, ctypes.c_void_p, ctypes.c_void_p]),
    "kvarn_append_tokens": (ctypes.c_int, [ctypes.c_void_p] * 3 + [ctypes.c_int64] + [ctypes.c_void_p] * 2
                            + [ctypes.c_int32] + [ctypes.c_void_p] * 3 + [ctypes.c_int32] + [ctypes.c_void_p] * 4),
    "kvarn_read_tokens": (ctypes.c_int, [ctypes.c_void_p] * 6 + [ctypes.c_int32, ctypes.c_int64, ctypes.c_int32]
                          + [ctypes.c_void_p] * 4),
    "kvarn_check_bounded_waits": (ctypes.c_int, [ctypes.c_int32, ctypes.c_uint32, ctypes.c_void_p, ctypes.c_size_t,
                                                 ctypes.c_void_p]),
    "kvarn_device_flags": (ctypes.c_int, [ctypes.POINTER(ctypes.c_uint32), ctypes.c_void_p]),
    "kvarn_last_error": (ctypes.c_char_p, []),
}


class KvarnError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"libkvarn status {status}: {message}")
        self.status = status


class KvarnMeta(ctypes.Structure):
    """Mirror of ``kvarn_meta`` (include/kvarn.h)."""
    _fields_ = [
        ("num_kv_heads", ctypes.c_int32),
        ("num_q_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("block_size", ctypes.c_int32),
        ("k_bits", ctypes.c_int32),
        ("v_bits", ctypes.c_int32),
        ("n_iters", ctypes.c_int32),
        ("eps", ctypes.c_float),
        ("num_blocks", ctypes.c_int64),
        ("max_blocks_per_seq", ctypes.c_int32),
        ("layout", ctypes.c_int32),
    ]


class KvarnRope(ctypes.Structure):
    """Mirror of ``kvarn_rope``."""
    _fields_ = [("dtype", ctypes.c_int32), ("rotary_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("norm_eps", ctypes.c_float), ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64),
                ("v_stride", ctypes.c_int64)]


class KvarnAxes(ctypes.Structure):
    """Mirror of ``kvarn_axes``."""
    _fields_ = [("n_axes", ctypes.c_int32), ("reserved", ctypes.c_int32), ("position_stride", ctypes.c_int64),
                ("axis", ctypes.c_uint8 * 64)]


class KvarnScore(ctypes.Structure):
    """Mirror of ``kvarn_score``."""
    _fields_ = [("scale", ctypes.c_float), ("softcap", ctypes.c_float), ("window", ctypes.c_int32),
                ("reserved", ctypes.c_int32), ("slopes", ctypes.c_void_p)]


# bit widths (keys, values) and metadata layout of the presets; k4v2 is
# kvarn_k4v2_g128, k4v2l the same with lean metadata (KVARN_LAYOUT_LEAN)
PRESETS = {"k4v2": (4, 2, 0), "k4v4": (4, 4, 0), "k2v2": (2, 2, 0), "k4v2l": (4, 2, 1)}
KVARN_LAYOUT_LEAN = 1


def make_meta(num_kv_heads: int, num_q_heads: int, num_blocks: int, max_blocks_per_seq: int = 0,
              n_iters: int = 4, eps: float = 1e-6, preset: str = "k4v2") -> KvarnMeta:
    """Head_dim 128, block 128; preset k4v2 (4-bit K, 2-bit V: kvarn_k4v2_g128),
    k4v4, k2v2, or k4v2l (k4v2 with lean metadata)."""
    kb, vb, layout = PRESETS[preset]
    return KvarnMeta(num_kv_heads, num_q_heads, HEAD_DIM, BLOCK_SIZE, kb, vb, n_iters, eps,
                     num_blocks, max_blocks_per_seq, layout)


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    if not os.path.exists(path):
        raise ImportError(f"{path} is missing: build it with "
                          "`python -c 'import __graft_entry__ as g; g.build()'` (needs nvcc)")
    lib = ctypes.CDLL(path)
    for name, (res, args) in _SIGS.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


_lib = load_library()


def _check(status: int):
    if status != KVARN_OK:
        raise KvarnError(status, _lib.kvarn_last_error().decode())


def _ptr(t, name, dtype=None, numel=None):
    """Device address of a contiguous CUDA tensor (None -> NULL)."""
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if numel is not None and t.numel() < numel:
        raise ValueError(f"{name} has {t.numel()} elements, needs {numel}")
    return t.data_ptr()


def _stream(stream):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def record_bytes() -> int:
    return int(_lib.kvarn_record_bytes())


def meta_record_bytes(meta: KvarnMeta) -> int:
    """Bytes of one (block, kv-head) record for the meta's preset."""
    return int(_lib.kvarn_meta_record_bytes(ctypes.byref(meta)))


def cache_bytes(meta: KvarnMeta) -> int:
    return int(_lib.kvarn_cache_bytes(ctypes.byref(meta)))


def workspace_bytes(meta: KvarnMeta, max_seqs: int) -> int:
    return int(_lib.kvarn_workspace_bytes(ctypes.byref(meta), max_seqs))


def decode_scratch_bytes(meta: KvarnMeta, n_seqs: int) -> int:
    return int(_lib.kvarn_decode_scratch_bytes(ctypes.byref(meta), n_seqs))


def kvarn_quantize_tiles(k, v, slot_mapping, cache, meta: KvarnMeta, stream=None):
    """k, v: fp16 [n_tokens, Hkv, 128]; slot_mapping: int64 [n_tokens];
    cache: uint8 [num_blocks, Hkv, meta_record_bytes(meta)]."""
    import torch
    n = int(k.shape[0])
    _check(_lib.kvarn_quantize_tiles(_ptr(k, "k", torch.float16), _ptr(v, "v", torch.float16),
                                     _ptr(slot_mapping, "slot_mapping", torch.int64, n), n,
                                     _ptr(cache, "cache", torch.uint8), ctypes.byref(meta), _stream(stream)))


def kvarn_append_decode(k_new, v_new, seq_lens, seq_lens_out, block_tables, workspace, cache,
                        meta: KvarnMeta, stream=None):
    """k_new, v_new: fp16 [n_seqs, Hkv, 128]; seq_lens (before) / seq_lens_out
    (after, may be None): int32 [n_seqs]; block_tables: int32 [n_seqs,
    max_blocks]; workspace: fp16 [>= n_seqs, Hkv, 2, 128, 128]."""
    import torch
    n = int(k_new.shape[0])
    _check(_lib.kvarn_append_decode(_ptr(k_new, "k_new", torch.float16), _ptr(v_new, "v_new", torch.float16),
                                    _ptr(seq_lens, "seq_lens", torch.int32, n),
                                    _ptr(seq_lens_out, "seq_lens_out", torch.int32, n),
                                    _ptr(block_tables, "block_tables", torch.int32), n,
                                    _ptr(workspace, "workspace", torch.float16),
                                    _ptr(cache, "cache", torch.uint8), ctypes.byref(meta), _stream(stream)))


def kvarn_decode_attention(q, cache, workspace, block_tables, seq_lens, out, scratch, meta: KvarnMeta,
                           stream=None):
    """q, out: fp16 [n_seqs, Hq, 128]; scratch: any CUDA tensor of at least
    decode_scratch_bytes(meta, n_seqs) bytes."""
    import torch
    n = int(q.shape[0])
    nbytes = 0 if scratch is None else scratch.numel() * scratch.element_size()
    _check(_lib.kvarn_decode_attention(_ptr(q, "q", torch.float16), _ptr(cache, "cache", torch.uint8),
                                       _ptr(workspace, "workspace", torch.float16),
                                       _ptr(block_tables, "block_tables", torch.int32),
                                       _ptr(seq_lens, "seq_lens", torch.int32, n), n,
                                       _ptr(out, "out", torch.float16), _ptr(scratch, "scratch"), nbytes,
                                       ctypes.byref(meta), _stream(stream)))


def kvarn_serve_step(q, k_new, v_new, seq_lens, seq_lens_out, block_tables, workspace, cache, out, scratch,
                     meta: KvarnMeta, stream=None):
    """One serving step in one launch: kvarn_append_decode then
    kvarn_decode_attention over seq_lens_out. q, out: fp16 [n_seqs, Hq, 128];
    k_new, v_new: fp16 [n_seqs, Hkv, 128]; seq_lens / seq_lens_out: int32 [n_seqs];
    scratch: at least decode_scratch_bytes(meta, n_seqs) bytes."""
    import torch
    n = int(q.shape[0])
    nbytes = 0 if scratch is None else scratch.numel() * scratch.element_size()
    _check(_lib.kvarn_serve_step(_ptr(q, "q", torch.float16), _ptr(k_new, "k_new", torch.float16),
                                 _ptr(v_new, "v_new", torch.float16), _ptr(seq_lens, "seq_lens", torch.int32, n),
                                 _ptr(seq_lens_out, "seq_lens_out", torch.int32, n),
                                 _ptr(block_tables, "block_tables", torch.int32), n,
                                 _ptr(workspace, "workspace", torch.float16), _ptr(cache, "cache", torch.uint8),
                                 _ptr(out, "out", torch.float16), _ptr(scratch, "scratch"), nbytes,
                                 ctypes.byref(meta), _stream(stream)))


def kvarn_decode_attention_static(q, cache, workspace, block_tables, seq_lens, out, meta: KvarnMeta, stream=None):
    """kvarn_decode_attention without a scratch argument, for callers that cannot
    allocate device memory: the library's built-in 16 MiB device array is used
    instead (shared by all calls on a device; calls overlapping on the GPU race).
    The first call on a device looks up that array's address."""
    import torch
    n = int(q.shape[0])
    _check(_lib.kvarn_decode_attention_static(_ptr(q, "q", torch.float16), _ptr(cache, "cache", torch.uint8),
                                              _ptr(workspace, "workspace", torch.float16),
                                              _ptr(block_tables, "block_tables", torch.int32),
                                              _ptr(seq_lens, "seq_lens", torch.int32, n), n,
                                              _ptr(out, "out", torch.float16), ctypes.byref(meta), _stream(stream)))


def kvarn_prefill_attention(q, k_new, v_new, cu_tokens, seq_lens, max_chunk: int, block_tables, cache, workspace,
                            out, meta: KvarnMeta, stream=None):
    """Chunked prefill: q, out fp16 [n_tokens, Hq, 128]; k_new, v_new fp16
    [n_tokens, Hkv, 128]; cu_tokens int32 [n_seqs + 1]; seq_lens int32 [n_seqs]
    (cached tokens before each chunk); max_chunk >= every chunk length."""
    import torch
    n = int(seq_lens.shape[0])
    _check(_lib.kvarn_prefill_attention(_ptr(q, "q", torch.float16), _ptr(k_new, "k_new", torch.float16),
                                        _ptr(v_new, "v_new", torch.float16),
                                        _ptr(cu_tokens, "cu_tokens", torch.int32, n + 1),
                                        _ptr(seq_lens, "seq_lens", torch.int32, n), n, int(max_chunk),
                                        _ptr(block_tables, "block_tables", torch.int32),
                                        _ptr(cache, "cache", torch.uint8), _ptr(workspace, "workspace", torch.float16),
                                        _ptr(out, "out", torch.float16), ctypes.byref(meta), _stream(stream)))


_CODES = {}


def _dtype_code(t, name):
    if not _CODES:
        import torch
        _CODES.update({torch.float16: KVARN_F16, torch.bfloat16: KVARN_BF16, torch.float32: KVARN_F32})
    code = _CODES.get(t.dtype)
    if code is None:
        raise ValueError(f"{name} must be torch.float16, torch.bfloat16 or torch.float32, got {t.dtype}")
    return code


def _device_call(lead, tensors, stream, call):
    """call(stream handle) with `lead`'s device current: the calls below launch on the
    device of their tensors, on its current stream unless one is given. (The handle of the
    current stream is asked for directly: a Stream object around it costs 2 us a call.)"""
    import torch
    dev = lead.get_device()
    if dev < 0:
        raise ValueError("tensors must be CUDA tensors")
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"tensors are on {lead.device} and on {t.device}")
    if stream is None:
        handle = torch._C._cuda_getCurrentRawStream(dev)
    elif stream.device.index != dev:
        raise ValueError(f"tensors are on {lead.device}, the stream is on {stream.device}")
    else:
        handle = stream.cuda_stream
    if dev == torch._C._cuda_getDevice():
        _check(call(handle))
    else:
        with torch.cuda.device(dev):
            _check(call(handle))


def _heads(t, name, n, heads, dtype):
    """Row stride of a [n, heads, 128] tensor whose rows are contiguous inside."""
    if t.shape != (n, heads, HEAD_DIM):
        raise ValueError(f"{name} must be [{n}, {heads}, {HEAD_DIM}], got {list(t.shape)}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    row, head, one = t.stride()
    if one != 1 or (heads > 1 and head != HEAD_DIM):
        raise ValueError(f"the heads of a row of {name} must be contiguous")
    return row


# kvarn_rope and kvarn_axes as bytes (a ctypes Structure costs 0.3 us a call more)
_ROPE, _AXES = struct.Struct("=iiifqqq"), struct.Struct("=iiq64s")
assert _ROPE.size == ctypes.sizeof(KvarnRope) and _AXES.size == ctypes.sizeof(KvarnAxes)


def _rope_args(q, k, v, q_out, k_out, v_out, meta, q_weight, k_weight, norm_eps, inv_freq, interleaved):
    """The C arguments that the norm and rotation calls share: the rows up to their
    kvarn_rope, and those behind it."""
    import torch
    n, hq, hkv = int(q.shape[0]), meta.num_q_heads, meta.num_kv_heads
    f16 = torch.float16
    dtype = q.dtype
    eps = norm_eps if 0.0 < norm_eps < 1.0 else 0.0    # (refused by the library; what is not a float would not pack)
    rope = _ROPE.pack(_dtype_code(q, "q"), HEAD_DIM if inv_freq is None else 2 * inv_freq.numel(), 1 if interleaved else 0,
                      eps, _heads(q, "q", n, hq, dtype), _heads(k, "k", n, hkv, dtype),
                      0 if v is None else _heads(v, "v", n, hkv, dtype))
    return ((q.data_ptr(), k.data_ptr(), None if v is None else v.data_ptr(), rope),
            (_ptr(q_weight, "q_weight", dtype, HEAD_DIM), _ptr(k_weight, "k_weight", dtype, HEAD_DIM),
             _ptr(inv_freq, "inv_freq", torch.float32), _ptr(q_out, "q_out", f16, n * hq * HEAD_DIM),
             _ptr(k_out, "k_out", f16, n * hkv * HEAD_DIM),
             None if v is None else _ptr(v_out, "v_out", f16, n * hkv * HEAD_DIM), ctypes.byref(meta)))


def kvarn_qk_norm_rope(q, k, v, positions, q_out, k_out, v_out, meta: KvarnMeta, q_weight=None, k_weight=None,
                       norm_eps: float = 1e-6, inv_freq=None, interleaved: bool = False, stream=None):
    """Per-head norm and rotation of projected rows. q [n, Hq, 128], k and v [n, Hkv, 128]
    in fp16, bf16 or fp32, rows at any stride (slices of a fused projection); weights
    [128] of the same type or None (no norm); positions int32 [n]; inv_freq float32
    [rotary_dim / 2] or None (no rotation); outputs fp16, contiguous. v and v_out may be None."""
    import torch
    n = int(q.shape[0])
    rows, rest = _rope_args(q, k, v, q_out, k_out, v_out, meta, q_weight, k_weight, norm_eps, inv_freq, interleaved)
    args = (*rows, *rest[:3], _ptr(positions, "positions", torch.int32, n), n, *rest[3:])
    _device_call(q, (k, v, positions, q_out, k_out, v_out, q_weight, k_weight, inv_freq), stream,
                 lambda st: _lib.kvarn_qk_norm_rope(*args, st))


def kvarn_qk_norm_rope_axes(q, k, v, positions, axes, q_out, k_out, v_out, meta: KvarnMeta, q_weight=None, k_weight=None,
                            norm_eps: float = 1e-6, inv_freq=None, interleaved: bool = False, stream=None):
    """kvarn_qk_norm_rope for tokens with a position on each of several axes (time, height,
    width): positions int32 [n_axes, n] (rows at any stride, or one row expanded; the first starts 16-byte
    aligned, so columns [:, start:end] of longer rows can be given where start is a multiple of four, and
    have to be copied by the caller otherwise); axes: for each of the rotary_dim / 2 pairs its axis, a
    sequence of whole numbers as long as inv_freq."""
    import torch
    n = int(q.shape[0])
    if positions.dim() != 2 or positions.shape[1] != n:
        raise ValueError(f"positions must be [n_axes, {n}], got {list(positions.shape)}")
    if not positions.is_cuda or positions.dtype != torch.int32:
        raise ValueError("positions must be a CUDA tensor of torch.int32")
    if n > 1 and positions.stride(1) != 1:
        raise ValueError("each axis' positions must be contiguous")
    if inv_freq is None:
        raise ValueError("inv_freq is required")
    if len(axes) != inv_freq.numel():
        raise ValueError(f"axes must have {inv_freq.numel()} entries, one for each pair, got {len(axes)}")
    of_pair = bytes(axes if isinstance(axes, (list, tuple)) else [int(x) for x in axes])
    rows, rest = _rope_args(q, k, v, q_out, k_out, v_out, meta, q_weight, k_weight, norm_eps, inv_freq, interleaved)
    split = _AXES.pack(int(positions.shape[0]), 0, positions.stride(0), of_pair)
    args = (*rows, split, *rest[:3], positions.data_ptr(), n, *rest[3:])
    _device_call(q, (k, v, positions, q_out, k_out, v_out, q_weight, k_weight, inv_freq), stream,
                 lambda st: _lib.kvarn_qk_norm_rope_axes(*args, st))


def decode_weights_scratch_bytes(meta: KvarnMeta, n_seqs: int) -> int:
    return int(_lib.kvarn_decode_weights_scratch_bytes(ctypes.byref(meta), n_seqs))


def kvarn_decode_attention_weights(q, cache, workspace, block_tables, seq_lens, weights, out, scratch, meta: KvarnMeta,
                                   decay: float = 1.0, lse=None, stream=None):
    """kvarn_decode_attention that also adds each tile's attention weight to weights (float32
    [n_seqs, Hkv, max_blocks], decay * old + new) and writes the log-sum-exp (float32
    [n_seqs, Hq], or None). q, out: fp16 [n_seqs, Hq, 128]; scratch: at least
    decode_weights_scratch_bytes(meta, n_seqs) bytes."""
    import torch
    n, f16, f32, i32 = int(q.shape[0]), torch.float16, torch.float32, torch.int32
    rows, hkv = n * meta.num_q_heads, meta.num_kv_heads
    args = (_ptr(q, "q", f16, rows * HEAD_DIM), _ptr(cache, "cache", torch.uint8),
            _ptr(workspace, "workspace", f16, n * hkv * 32768),
            _ptr(block_tables, "block_tables", i32, n * meta.max_blocks_per_seq), _ptr(seq_lens, "seq_lens", i32, n), n,
            float(decay), _ptr(weights, "weights", f32, n * hkv * meta.max_blocks_per_seq),
            _ptr(out, "out", f16, rows * HEAD_DIM), _ptr(lse, "lse", f32, rows), _ptr(scratch, "scratch"),
            0 if scratch is None else scratch.numel() * scratch.element_size(), ctypes.byref(meta))
    _device_call(q, (cache, workspace, block_tables, seq_lens, weights, out, lse, scratch), stream,
                 lambda st: _lib.kvarn_decode_attention_weights(*args, st))


def kvarn_evict_tiles(weights, weights_out, seq_lens, seq_lens_out, block_tables, budgets, kept, cache, meta: KvarnMeta,
                      keep_first: int = 1, keep_last: int = 1, stream=None):
    """The tiles of least weight leave the cache, for every sequence and kv-head: at most
    budgets[s] (int32 [n_seqs], negative: all) stay, the first keep_first and last
    keep_last among them. weights, weights_out (may be the same): float32 [n_seqs, Hkv,
    max_blocks]; seq_lens / seq_lens_out: int32 [n_seqs]; kept: int32 [n_seqs, Hkv,
    max_blocks], the old slots by new slot, then the evicted ones, then -1."""
    import torch
    n, f32, i32 = int(seq_lens.shape[0]), torch.float32, torch.int32
    entries = n * meta.num_kv_heads * meta.max_blocks_per_seq
    args = (_ptr(weights, "weights", f32, entries), _ptr(weights_out, "weights_out", f32, entries),
            _ptr(seq_lens, "seq_lens", i32, n), _ptr(seq_lens_out, "seq_lens_out", i32, n),
            _ptr(block_tables, "block_tables", i32, n * meta.max_blocks_per_seq), _ptr(budgets, "budgets", i32, n), n,
            int(keep_first), int(keep_last), _ptr(kept, "kept", i32, entries), _ptr(cache, "cache", torch.uint8),
            ctypes.byref(meta))
    _device_call(seq_lens, (weights, weights_out, seq_lens_out, block_tables, budgets, kept, cache), stream,
                 lambda st: _lib.kvarn_evict_tiles(*args, st))


def tree_scratch_bytes(meta: KvarnMeta, n_seqs: int, max_tree: int) -> int:
    return int(_lib.kvarn_tree_scratch_bytes(ctypes.byref(meta), n_seqs, max_tree))


def kvarn_tree_attention(q, k_new, v_new, tree_mask, cu_tokens, seq_lens, max_tree: int, block_tables, cache, workspace,
                         out, scratch, meta: KvarnMeta, positions=None, scale: float = 0.0, softcap: float = 0.0,
                         window: int = 0, slopes=None, stream=None):
    """Drafted tokens over the quantized cache. q, out: fp16 [n_tokens, Hq, 128]; k_new,
    v_new: fp16 [n_tokens, Hkv, 128]; tree_mask: int64 (or uint64) [n_tokens], bit j = the
    sequence's j-th new token is attended, None = a chain; cu_tokens: int32 [n_seqs + 1];
    seq_lens: int32 [n_seqs], cached tokens; max_tree: at least every sequence's new tokens
    (<= 64); scratch: at least tree_scratch_bytes(meta, n_seqs, max_tree) bytes. Scores:
    scale (0: 1/sqrt(128)), softcap, window and slopes (float32 [Hq]), the last two over
    positions (int32 [n_tokens])."""
    import torch
    n, n_seqs, f16, i32 = int(q.shape[0]), int(seq_lens.shape[0]), torch.float16, torch.int32
    if tree_mask is not None and tree_mask.dtype not in (torch.int64, torch.uint64):
        raise ValueError(f"tree_mask must be 64-bit integers, got {tree_mask.dtype}")
    rows = n * meta.num_kv_heads * HEAD_DIM
    score = KvarnScore(scale, softcap, window, 0, _ptr(slopes, "slopes", torch.float32, meta.num_q_heads))
    args = (_ptr(q, "q", f16, n * meta.num_q_heads * HEAD_DIM), _ptr(k_new, "k_new", f16, rows),
            _ptr(v_new, "v_new", f16, rows), _ptr(tree_mask, "tree_mask", None, n),
            _ptr(positions, "positions", i32, n), _ptr(cu_tokens, "cu_tokens", i32, n_seqs + 1),
            _ptr(seq_lens, "seq_lens", i32, n_seqs), n_seqs, n, int(max_tree),
            _ptr(block_tables, "block_tables", i32, n_seqs * meta.max_blocks_per_seq),
            _ptr(cache, "cache", torch.uint8), _ptr(workspace, "workspace", f16, n_seqs * meta.num_kv_heads * 32768),
            ctypes.byref(score), _ptr(out, "out", f16, n * meta.num_q_heads * HEAD_DIM), _ptr(scratch, "scratch"),
            0 if scratch is None else scratch.numel() * scratch.element_size(), ctypes.byref(meta))
    _device_call(q, (k_new, v_new, tree_mask, positions, cu_tokens, seq_lens, block_tables, cache, workspace, out,
                     scratch, slopes), stream, lambda st: _lib.kvarn_tree_attention(*args, st))


def kvarn_append_tokens(k_new, v_new, cu_tokens, seq_lens, seq_lens_out, block_tables, workspace, cache, meta: KvarnMeta,
                        accepted=None, n_accepted=None, stream=None):
    """Several tokens a sequence into the cache. k_new, v_new: fp16 [n_tokens, Hkv, 128],
    sequence s's rows cu_tokens[s] .. cu_tokens[s + 1] - 1 (int32 [n_seqs + 1]); accepted:
    int32 [n_seqs, max_accept] rows counted from cu_tokens[s] with n_accepted int32
    [n_seqs], or both None: all rows, in order; seq_lens / seq_lens_out: int32 [n_seqs]."""
    import torch
    n, n_seqs, f16, i32 = int(k_new.shape[0]), int(seq_lens.shape[0]), torch.float16, torch.int32
    rows = n * meta.num_kv_heads * HEAD_DIM
    width = 0
    if accepted is not None:
        if accepted.dim() != 2 or accepted.shape[0] != n_seqs or accepted.shape[1] < 1:
            raise ValueError(f"accepted must be [{n_seqs}, max_accept >= 1], got {list(accepted.shape)}")
        width = int(accepted.shape[1])
    args = (_ptr(k_new, "k_new", f16, rows), _ptr(v_new, "v_new", f16, rows),
            _ptr(cu_tokens, "cu_tokens", i32, n_seqs + 1), n, _ptr(accepted, "accepted", i32),
            _ptr(n_accepted, "n_accepted", i32, n_seqs), width, _ptr(seq_lens, "seq_lens", i32, n_seqs),
            _ptr(seq_lens_out, "seq_lens_out", i32, n_seqs),
            _ptr(block_tables, "block_tables", i32, n_seqs * meta.max_blocks_per_seq), n_seqs,
            _ptr(workspace, "workspace", f16, n_seqs * meta.num_kv_heads * 32768), _ptr(cache, "cache", torch.uint8),
            ctypes.byref(meta))
    _device_call(seq_lens, (k_new, v_new, cu_tokens, accepted, n_accepted, seq_lens_out, block_tables, workspace, cache),
                 stream, lambda st: _lib.kvarn_append_tokens(*args, st))


def kvarn_read_tokens(cache, workspace, block_tables, seq_lens, cu_tokens, k_out, v_out, meta: KvarnMeta, first=None,
                      stream=None):
    """Cached tokens first[s] (None: 0) .. first[s] + n - 1 of sequence s, n =
    cu_tokens[s + 1] - cu_tokens[s], as rows cu_tokens[s] .. of k_out and v_out
    [n_tokens, Hkv, 128] (fp16, bf16 or fp32)."""
    import torch
    n, n_seqs, i32 = int(k_out.shape[0]), int(seq_lens.shape[0]), torch.int32
    rows = n * meta.num_kv_heads * HEAD_DIM
    args = (_ptr(cache, "cache", torch.uint8),
            _ptr(workspace, "workspace", torch.float16, n_seqs * meta.num_kv_heads * 32768),
            _ptr(block_tables, "block_tables", i32, n_seqs * meta.max_blocks_per_seq),
            _ptr(seq_lens, "seq_lens", i32, n_seqs), _ptr(first, "first", i32, n_seqs),
            _ptr(cu_tokens, "cu_tokens", i32, n_seqs + 1), n_seqs, n, _dtype_code(k_out, "k_out"),
            _ptr(k_out, "k_out", None, rows), _ptr(v_out, "v_out", k_out.dtype, rows), ctypes.byref(meta))
    _device_call(k_out, (v_out, cache, workspace, block_tables, seq_lens, first, cu_tokens), stream,
                 lambda st: _lib.kvarn_read_tokens(*args, st))


def kvarn_check_bounded_waits(which: int, limit_us: int, scratch=None, stream=None):
    """Runs the library's bounded-wait code against a wait that never completes
    (KVARN_WAIT_MBARRIER or KVARN_WAIT_GRID), giving up after limit_us; the
    timeout shows as FLAG_WAIT_TIMEOUT in kvarn_device_flags(). scratch: a device
    buffer of at least 8 bytes for the grid barrier's words."""
    nbytes = 0 if scratch is None else scratch.numel() * scratch.element_size()
    _check(_lib.kvarn_check_bounded_waits(int(which), int(limit_us), _ptr(scratch, "scratch"), nbytes,
                                          _stream(stream)))


def kvarn_device_flags(stream=None) -> int:
    v = ctypes.c_uint32(0)
    _check(_lib.kvarn_device_flags(ctypes.byref(v), _stream(stream)))
    return int(v.value)
