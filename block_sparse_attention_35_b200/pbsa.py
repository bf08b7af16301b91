"""Thin Python binding of the PBSA C ABI (include/pbsa.h).

Each ``pbsa_*`` function here has the name and argument order of the C function; it only
turns torch tensors into device pointers and the current CUDA stream into ``void*``, and
raises ``PBSAError`` on a non-zero return code.  All work runs in the CUDA kernels of
``libpbsa.so``; there is no CPU fallback, and importing this module fails loudly when the
library has not been built.
"""
from __future__ import annotations

import ctypes
import os
import re
import types
import warnings

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libpbsa.so")
HEADER = os.path.join(os.path.dirname(_HERE), "include", "pbsa.h")

PBSA_OK = 0
PBSA_ERR_ARG = -1
PBSA_ERR_UNSUPPORTED = -2
PBSA_ERR_CUDA = -3
PBSA_ERR_TIMEOUT = -4
PBSA_ERR_DEVICE_CHECK = -5
PBSA_ERR_WORKSPACE = -6
PBSA_OP_SELECT, PBSA_OP_FWD, PBSA_OP_BWD, PBSA_OP_UPDATE = 0, 1, 2, 3
PBSA_KV_CACHE_SPARSE_FORCING, PBSA_KV_CACHE_DENSE = 0, 1
PBSA_DTYPE_BF16, PBSA_DTYPE_FP16, PBSA_DTYPE_FP32 = 0, 1, 2
_DTYPES = {torch.bfloat16: PBSA_DTYPE_BF16, torch.float16: PBSA_DTYPE_FP16,
           torch.float32: PBSA_DTYPE_FP32}
_TORCH = {v: k for k, v in _DTYPES.items()}


class PBSAError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"PBSA error {code}: {msg}")
        self.code = code


class pbsa_config(ctypes.Structure):
    """Mirror of the C struct pbsa_config."""
    _fields_ = [
        ("B", ctypes.c_int), ("H", ctypes.c_int), ("D", ctypes.c_int),
        ("frame_h", ctypes.c_int), ("frame_w", ctypes.c_int),
        ("block_t", ctypes.c_int), ("block_h", ctypes.c_int), ("block_w", ctypes.c_int),
        ("total_cache_size", ctypes.c_int), ("local_cache_size", ctypes.c_int),
        ("persistent_cache_size", ctypes.c_int), ("max_seq_len", ctypes.c_int),
        ("kv_cache_mode", ctypes.c_int), ("use_local_block_sparse_attn", ctypes.c_int),
        ("local_block_sparse_topk_ratio", ctypes.c_float),
        ("sink_frames", ctypes.c_int),
    ]


class pbsa_qk_config(ctypes.Structure):
    """Mirror of the C struct pbsa_qk_config."""
    _fields_ = [
        ("B", ctypes.c_int), ("T", ctypes.c_int), ("Hq", ctypes.c_int), ("Hkv", ctypes.c_int),
        ("D", ctypes.c_int), ("dtype", ctypes.c_int), ("grad_dtype", ctypes.c_int),
        ("rot_dim", ctypes.c_int), ("interleaved", ctypes.c_int), ("n_axes", ctypes.c_int),
        ("axis_pairs", ctypes.c_int * 3), ("table_len", ctypes.c_int), ("eps", ctypes.c_float),
    ]


class pbsa_kv4_config(ctypes.Structure):
    """Mirror of the C struct pbsa_kv4_config."""
    _fields_ = [
        ("B", ctypes.c_int), ("Hq", ctypes.c_int), ("Hkv", ctypes.c_int), ("D", ctypes.c_int),
        ("capacity", ctypes.c_int), ("dtype", ctypes.c_int), ("k_unit", ctypes.c_float),
        ("v_unit", ctypes.c_float),
    ]


class pbsa_kv4_cache(ctypes.Structure):
    """Mirror of the C struct pbsa_kv4_cache (make_kv4_cache fills it from tensors)."""
    _fields_ = [("k_codes", ctypes.c_void_p), ("k_scales", ctypes.c_void_p),
                ("v_codes", ctypes.c_void_p), ("v_scales", ctypes.c_void_p),
                ("pos", ctypes.c_void_p)]


def _dtype(dt):
    if dt not in _DTYPES:
        raise PBSAError(PBSA_ERR_UNSUPPORTED, f"dtype {dt}")
    return _DTYPES[dt]


def make_qk_config(B, T, Hq, Hkv, D, dtype=torch.bfloat16, rot_dim=None, interleaved=False,
                   axis_pairs=None, table_len=0, eps=1e-6, grad_dtype=None) -> pbsa_qk_config:
    """rot_dim None rotates every channel; axis_pairs None is one position component."""
    rot_dim = D if rot_dim is None else rot_dim
    pairs = (rot_dim // 2,) if axis_pairs is None else tuple(axis_pairs)
    if not 1 <= len(pairs) <= 3:
        raise PBSAError(PBSA_ERR_ARG, f"axis_pairs has {len(pairs)} entries, not 1 to 3")
    return pbsa_qk_config(B, T, Hq, Hkv, D, _dtype(dtype),
                          _dtype(dtype if grad_dtype is None else grad_dtype), rot_dim,
                          int(bool(interleaved)), len(pairs),
                          (ctypes.c_int * 3)(*pairs, *(0,) * (3 - len(pairs))), table_len,
                          float(eps))


def make_kv4_config(B, Hq, Hkv, D, capacity, dtype=torch.bfloat16, k_unit=1.0,
                    v_unit=1.0) -> pbsa_kv4_config:
    return pbsa_kv4_config(B, Hq, Hkv, D, capacity, _dtype(dtype), float(k_unit), float(v_unit))


def make_kv4_cache(cfg, k_codes, k_scales, v_codes, v_scales, pos) -> pbsa_kv4_cache:
    """The cache handle of its five device tensors (which it keeps alive)."""
    pbsa_validate_kv4_config(cfg)
    rows = (cfg.B, cfg.Hkv, cfg.capacity)
    dev = pos.device
    for name, t, w in (("k_codes", k_codes, cfg.D // 2), ("k_scales", k_scales, cfg.D // 16),
                       ("v_codes", v_codes, cfg.D // 2), ("v_scales", v_scales, cfg.D // 16)):
        _want(t, name, (*rows, w), torch.uint8, dev)
    _want(pos, "pos", rows, torch.int32, dev)
    c = pbsa_kv4_cache(k_codes.data_ptr(), k_scales.data_ptr(), v_codes.data_ptr(),
                       v_scales.data_ptr(), pos.data_ptr())
    c.tensors = (k_codes, k_scales, v_codes, v_scales, pos)
    c.device, c.index = dev, pos.get_device()
    c.shape = (cfg.B, cfg.Hkv, cfg.capacity, cfg.D)
    return c


def make_config(B, H, D, frame_h, frame_w, total_cache_size, local_cache_size,
                persistent_cache_size, max_seq_len, local_block_sparse_topk_ratio,
                use_local_block_sparse_attn=True, sparse_kv_block_size=(1, 8, 8),
                kv_cache_mode="sparse_forcing", sink_frames=0) -> pbsa_config:
    """Builds a pbsa_config from the SparseForcingAttention constructor arguments (plus
    sink_frames, the length of the sequence's sink)."""
    modes = {"sparse_forcing": PBSA_KV_CACHE_SPARSE_FORCING, "dense": PBSA_KV_CACHE_DENSE}
    if kv_cache_mode not in modes:
        raise PBSAError(PBSA_ERR_UNSUPPORTED, f"kv_cache_mode {kv_cache_mode!r}")
    bt, bh, bw = sparse_kv_block_size
    return pbsa_config(B, H, D, frame_h, frame_w, bt, bh, bw, total_cache_size,
                       local_cache_size, persistent_cache_size, max_seq_len,
                       modes[kv_cache_mode], int(bool(use_local_block_sparse_attn)),
                       float(local_block_sparse_topk_ratio), int(sink_frames))


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with "
                          "`python -m block_sparse_attention_35_b200.build`")
    lib = ctypes.CDLL(LIB_PATH)   # before token_calls, which is linked with it
    P = ctypes.c_void_p
    I = ctypes.c_int
    C = ctypes.POINTER(pbsa_config)
    Z = ctypes.c_size_t
    S = ctypes.POINTER(ctypes.c_int64)
    QC, KC, KK = (ctypes.POINTER(t) for t in (pbsa_qk_config, pbsa_kv4_config, pbsa_kv4_cache))
    sig = {
        "pbsa_validate_config": (I, [C]),
        "pbsa_blocks_per_frame": (I, [C]),
        "pbsa_window_frames": (I, [C]),
        "pbsa_num_slots": (I, [C]),
        "pbsa_sink_slots": (I, [C]),
        "pbsa_topk_count": (I, [C, I]),
        "pbsa_workspace_size": (ctypes.c_size_t, [C, I, I]),
        "pbsa_last_error": (ctypes.c_char_p, []),
        "pbsa_version": (ctypes.c_char_p, []),
        "pbsa_select_blocks": (I, [C, P, I, P, I, I, P, I, P, P, P, ctypes.c_size_t, P]),
        "pbsa_attn_fwd": (I, [C, P, I, P, P, P, P, P, I, I, P, I, P, P, P, P, P, P,
                              ctypes.c_size_t, P, P]),
        "pbsa_attn_bwd": (I, [C, P, I, P, P, P, P, P, I, I, P, I, P, P, P, P, P, P, P, P, P,
                              P, ctypes.c_size_t, P, P]),
        "pbsa_cache_update": (I, [C, P, P, I, I, P, I, I, P, P, P, P, P, P, P, P,
                                  ctypes.c_size_t, P]),
        "pbsa_wait_selftest": (I, [P, ctypes.c_longlong, P]),
        "pbsa_pool_keys": (I, [C, P, I, I, P, P]),
        "pbsa_append_frames": (I, [C, P, P, I, I, P, P, I, P, P, P, P, P, P, P]),
        "pbsa_select_blocks_pooled": (I, [C, P, I, P, I, I, P, I, P, P, P, ctypes.c_size_t, P]),
        "pbsa_qk_workspace_size": (Z, [QC]),
        "pbsa_qk_norm_rope": (I, [QC, P, P, S, P, P, P, P, P, P, P, P, P]),
        "pbsa_qk_norm_rope_bwd": (I, [QC, P, P, S, P, P, P, P, P, P, P, P, P, P, P, P, Z, P, P]),
        "pbsa_validate_kv4_config": (I, [KC]),
        "pbsa_kv4_workspace_size": (Z, [KC, I]),
        "pbsa_kv4_append": (I, [KC, KK, P, P, S, I, P, P, P, P, P]),
        "pbsa_kv4_read": (I, [KC, KK, P, I, P, P, P, P]),
        "pbsa_kv4_attn": (I, [KC, KK, P, S, I, P, P, P, P, P, P, Z, P, P]),
        "pbsa_kv4_evict": (I, [KC, P, P, I, I, P, P, P, P]),
    }
    for name, (res, args) in sig.items():
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args
    return lib


_lib = _load()

# of csrc/token_calls.cpp, where it makes no call: ctypes then makes all of them
_NO_CALLS = types.SimpleNamespace(**{name: lambda *args: None for name in (
    "qk_norm_rope", "qk_norm_rope_bwd", "kv4_append", "kv4_read", "kv4_attn", "kv4_evict")})


def _quick_calls():
    """The module built beside the library, which reads torch's tensors and so belongs to one torch."""
    try:
        from . import token_calls
        if token_calls.torch_version == torch.__version__:
            return token_calls
        why = f"was built for torch {token_calls.torch_version}"
    except ImportError as e:
        why = str(e)
    warnings.warn(f"token_calls.so {why}: the token operators' calls go through ctypes (a few us more each)")
    return _NO_CALLS


_calls = _quick_calls()


def header_symbols(path: str = HEADER):
    """Names of the functions declared in include/pbsa.h."""
    txt = open(path).read()
    return sorted(set(re.findall(r"PBSA_API\s+[\w\s\*]+?\b(pbsa_\w+)\s*\(", txt)))


def library():
    return _lib


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else stream


def _check(rc):
    if rc != PBSA_OK:
        raise PBSAError(rc, _lib.pbsa_last_error().decode())


def _cfg(cfg):
    return ctypes.byref(cfg)


# ------------------------------------------------------------------ host-only queries
def pbsa_validate_config(cfg):
    _check(_lib.pbsa_validate_config(_cfg(cfg)))


def pbsa_blocks_per_frame(cfg) -> int:
    return _lib.pbsa_blocks_per_frame(_cfg(cfg))


def pbsa_window_frames(cfg) -> int:
    return _lib.pbsa_window_frames(_cfg(cfg))


def pbsa_num_slots(cfg) -> int:
    return _lib.pbsa_num_slots(_cfg(cfg))


def pbsa_sink_slots(cfg) -> int:
    return _lib.pbsa_sink_slots(_cfg(cfg))


def pbsa_topk_count(cfg, local_frames: int) -> int:
    k = _lib.pbsa_topk_count(_cfg(cfg), local_frames)
    if k < 0:
        _check(k)
    return k


def pbsa_workspace_size(cfg, op: int, q_frames: int) -> int:
    return int(_lib.pbsa_workspace_size(_cfg(cfg), op, q_frames))


def pbsa_version() -> str:
    return _lib.pbsa_version().decode()


def pbsa_last_error() -> str:
    return _lib.pbsa_last_error().decode()


# ------------------------------------------------------------------ device calls
def pbsa_select_blocks(cfg, q, q_frames, k_local, local_frames, ring_head, idx, idx_stride,
                       cnt, scores, workspace, stream=None):
    _check(_lib.pbsa_select_blocks(
        _cfg(cfg), _ptr(q), q_frames, _ptr(k_local), local_frames, ring_head, _ptr(idx),
        idx_stride, _ptr(cnt), _ptr(scores), _ptr(workspace),
        0 if workspace is None else workspace.numel() * workspace.element_size(),
        _stream(stream)))


def pbsa_attn_fwd(cfg, q, q_frames, k_pers, v_pers, pers_len, k_local, v_local, local_frames,
                  ring_head, idx, idx_stride, cnt, out, lse, mass_local, mass_pers, workspace,
                  status, stream=None):
    _check(_lib.pbsa_attn_fwd(
        _cfg(cfg), _ptr(q), q_frames, _ptr(k_pers), _ptr(v_pers), _ptr(pers_len),
        _ptr(k_local), _ptr(v_local), local_frames, ring_head, _ptr(idx), idx_stride,
        _ptr(cnt), _ptr(out), _ptr(lse), _ptr(mass_local), _ptr(mass_pers), _ptr(workspace),
        0 if workspace is None else workspace.numel() * workspace.element_size(),
        _ptr(status), _stream(stream)))


def pbsa_attn_bwd(cfg, q, q_frames, k_pers, v_pers, pers_len, k_local, v_local, local_frames,
                  ring_head, idx, idx_stride, cnt, out, lse, dout, dq, dk_pers, dv_pers,
                  dk_local, dv_local, workspace, status, stream=None):
    _check(_lib.pbsa_attn_bwd(
        _cfg(cfg), _ptr(q), q_frames, _ptr(k_pers), _ptr(v_pers), _ptr(pers_len),
        _ptr(k_local), _ptr(v_local), local_frames, ring_head, _ptr(idx), idx_stride,
        _ptr(cnt), _ptr(out), _ptr(lse), _ptr(dout), _ptr(dq), _ptr(dk_pers), _ptr(dv_pers),
        _ptr(dk_local), _ptr(dv_local), _ptr(workspace),
        0 if workspace is None else workspace.numel() * workspace.element_size(),
        _ptr(status), _stream(stream)))


def pbsa_cache_update(cfg, k_local, v_local, local_frames, ring_head, mass_local,
                      n_evict_frames, first_frame_global, k_pers, v_pers, pers_len, pers_score,
                      pers_src, upd, n_upd, workspace=None, stream=None):
    _check(_lib.pbsa_cache_update(
        _cfg(cfg), _ptr(k_local), _ptr(v_local), local_frames, ring_head, _ptr(mass_local),
        n_evict_frames, first_frame_global, _ptr(k_pers), _ptr(v_pers), _ptr(pers_len),
        _ptr(pers_score), _ptr(pers_src), _ptr(upd), _ptr(n_upd), _ptr(workspace),
        0 if workspace is None else workspace.numel() * workspace.element_size(),
        _stream(stream)))


def pbsa_wait_selftest(status, timeout_ns: int, stream=None):
    _check(_lib.pbsa_wait_selftest(_ptr(status), int(timeout_ns), _stream(stream)))


def pbsa_append_frames(cfg, k_new, v_new, n_frames, first_global_frame, k_local, v_local,
                       ring_slot, kbar=None, k_pers=None, v_pers=None, pers_len=None,
                       pers_score=None, pers_src=None, stream=None):
    """Appends frames to the cache: sink frames into their slots, the others into the ring
    from ring_slot on, with their key means written to kbar (when given) in the same pass."""
    _check(_lib.pbsa_append_frames(
        _cfg(cfg), _ptr(k_new), _ptr(v_new), n_frames, first_global_frame, _ptr(k_local),
        _ptr(v_local), ring_slot, _ptr(kbar), _ptr(k_pers), _ptr(v_pers), _ptr(pers_len),
        _ptr(pers_score), _ptr(pers_src), _stream(stream)))


def pbsa_pool_keys(cfg, k_local, first_slot, n_frames, kbar, stream=None):
    """Pools the key blocks of ring slots first_slot.. (n_frames, mod W) into kbar
    [B, H, W*NB_f, D] fp32 (row = slot * NB_f + block)."""
    _check(_lib.pbsa_pool_keys(_cfg(cfg), _ptr(k_local), first_slot, n_frames, _ptr(kbar),
                               _stream(stream)))


def pbsa_select_blocks_pooled(cfg, q, q_frames, kbar, local_frames, ring_head, idx, idx_stride,
                              cnt, scores, workspace, stream=None):
    """Block selection with the window's key means read from kbar (see pbsa_pool_keys)."""
    _check(_lib.pbsa_select_blocks_pooled(
        _cfg(cfg), _ptr(q), q_frames, _ptr(kbar), local_frames, ring_head, _ptr(idx),
        idx_stride, _ptr(cnt), _ptr(scores), _ptr(workspace),
        0 if workspace is None else workspace.numel() * workspace.element_size(),
        _stream(stream)))


def pbsa_select_blocks_noalloc(cfg, q, q_frames, k_local, local_frames, ring_head, idx,
                               idx_stride, cnt, scores, stream=None):
    """Block selection without a workspace, for callers that cannot allocate device
    memory (the library keeps the scratch in a static device buffer; see include/pbsa.h)."""
    f = _lib.pbsa_select_blocks_noalloc
    if f.argtypes is None:
        P, I = ctypes.c_void_p, ctypes.c_int
        f.restype = I
        f.argtypes = [ctypes.POINTER(pbsa_config), P, I, P, I, I, P, I, P, P, P]
    _check(f(_cfg(cfg), _ptr(q), q_frames, _ptr(k_local), local_frames, ring_head, _ptr(idx),
             idx_stride, _ptr(cnt), _ptr(scores), _stream(stream)))


# --------------------------------------------- token operators: heads and the 4-bit cache
# These calls check what a pointer cannot show - shapes, types, the device - before they hand
# the pointers on, and run on the current stream of the tensors' device.  Where all is as it
# should be and that device is the current one, csrc/token_calls.cpp makes them; what it leaves
# alone is checked here, with an error that says what does not fit.

def _bad(msg):
    raise PBSAError(PBSA_ERR_ARG, msg)


def _want(t, name, shape, dtype, device, strided=False):
    """Checks a tensor: contiguous, or (strided) only its last dimension contiguous."""
    if t.shape != shape:
        _bad(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != dtype:
        _bad(f"{name}: {t.dtype}, expected {dtype}")
    if t.device != device:
        _bad(f"{name} is on {t.device}, not on {device}")
    if strided:
        if t.stride(-1) != 1:
            _bad(f"{name}: channels are not contiguous")
    elif not t.is_contiguous():
        _bad(f"{name} is not contiguous")


def _want_heads(t, name, shape, dtype, device):
    """Checks a [B, T, H, D] tensor as the library does too: strides and address multiples of 16 bytes."""
    if (t.shape == shape and t.dtype == dtype and t.get_device() == device.index and t.is_contiguous()
            and t.data_ptr() % 16 == 0):
        return   # an ordinary one
    _want(t, name, shape, dtype, device, True)
    if t.numel() and (t.data_ptr() % 16 or any(n > 1 and st * t.element_size() % 16
                                               for n, st in zip(t.shape[:3], t.stride()))):
        _bad(f"{name}: an address or a stride is not a multiple of 16 bytes")


def _strides(*tensors):
    """Batch, token and head strides of [B, T, H, D] tensors (zeros for None, and where there is
    one element: its stride says nothing)."""
    out = []
    for t in tensors:
        out += (0, 0, 0) if t is None else (0 if n == 1 else s for n, s in zip(t.shape[:3], t.stride()))
    return (ctypes.c_int64 * len(out))(*out)


# what torch.cuda.current_stream() and current_device() ask, without the objects around it
_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice


def _launch(index, stream, call, *args):
    """call(*args, stream) with device `index` current; its current stream unless one is given."""
    if index < 0:
        _bad("tensors are not on a CUDA device")
    if _current_device() == index:
        rc = call(*args, _raw_stream(index) if stream is None else _stream(stream))
    else:
        with torch.cuda.device(index):
            rc = call(*args, _raw_stream(index) if stream is None else _stream(stream))
    if rc != PBSA_OK:
        _check(rc)


def _quick(call, kind, cfg, index, stream, *args):
    """Makes an ordinary call through token_calls; False if it is not one."""
    if index < 0 or type(cfg) is not kind or _current_device() != index:
        return False
    rc = call(ctypes.addressof(cfg), index, _raw_stream(index) if stream is None else _stream(stream),
              *args)
    if rc is None:
        return False
    if rc != PBSA_OK:
        _check(rc)
    return True


def _bytes(t):
    return 0 if t is None else t.numel() * t.element_size()


def _want_workspace(t, device):
    if t is not None and (t.device != device or not t.is_contiguous()):
        _bad(f"workspace is not a contiguous tensor on {device}")


def _qk_check(cfg, tensors, q_weight, k_weight, cos, sin, pos, status):
    """tensors: (name, query tensor, key tensor, dtype) of [B, T, H, D] pairs."""
    dev = tensors[0][1].device
    for name, tq, tk, dt in tensors:
        _want(tq, "q" + name if name[:1] == "_" or not name else name + "q",
              (cfg.B, cfg.T, cfg.Hq, cfg.D), dt, dev, True)
        if cfg.Hkv:
            _want(tk, "k" + name if name[:1] == "_" or not name else name + "k",
                  (cfg.B, cfg.T, cfg.Hkv, cfg.D), dt, dev, True)
    for name, tq, tk, _ in tensors[-1:]:   # the outputs: every element its own
        for t in (tq, tk):
            if t is not None and any(st == 0 and n > 1 for st, n in zip(t.stride(), t.shape)):
                _bad("an output has elements that share memory")
    for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
        if w is not None:
            _want(w, name, (cfg.D,), torch.float32, dev)
    if cfg.rot_dim:
        if cos is None or sin is None or pos is None or status is None:
            _bad("cos, sin, pos and status are needed for a rotation")
        table = (cfg.table_len, cfg.rot_dim // 2)
        _want(cos, "cos", table, torch.float32, dev)
        _want(sin, "sin", table, torch.float32, dev)
        _want(pos, "pos", (cfg.B, cfg.T, cfg.n_axes), torch.int32, dev)
    if status is not None:
        _want(status, "status", (1,), torch.int32, dev)
    return dev


def pbsa_qk_workspace_size(cfg) -> int:
    n = _lib.pbsa_qk_workspace_size(_cfg(cfg))
    if n == 0:
        raise PBSAError(PBSA_ERR_ARG, pbsa_last_error())
    return n


def pbsa_qk_norm_rope(cfg, q, k, q_weight, k_weight, cos, sin, pos, q_out, k_out, status,
                      stream=None):
    """RMS norm and rotation of every head; q, k, q_out, k_out may be strided views."""
    i = q.get_device()
    if _quick(_calls.qk_norm_rope, pbsa_qk_config, cfg, i, stream, q, k, q_weight, k_weight, cos, sin,
              pos, q_out, k_out, status):
        return
    dt = _TORCH.get(cfg.dtype)
    if not cfg.Hkv:
        k = k_out = None
    _qk_check(cfg, (("", q, k, dt), ("_out", q_out, k_out, dt)), q_weight, k_weight, cos, sin, pos,
              status)
    _launch(i, stream, _lib.pbsa_qk_norm_rope, _cfg(cfg), q.data_ptr(), _ptr(k),
            _strides(q, k, q_out, k_out), _ptr(q_weight), _ptr(k_weight), _ptr(cos), _ptr(sin), _ptr(pos), q_out.data_ptr(),
            _ptr(k_out), _ptr(status))


def pbsa_qk_norm_rope_bwd(cfg, q, k, q_weight, k_weight, cos, sin, pos, dq_out, dk_out, dq, dk,
                          dq_weight, dk_weight, workspace, status, stream=None):
    """Gradients of pbsa_qk_norm_rope; dq_weight, dk_weight may be None."""
    i = q.get_device()
    if _quick(_calls.qk_norm_rope_bwd, pbsa_qk_config, cfg, i, stream, q, k, q_weight, k_weight, cos,
              sin, pos, dq_out, dk_out, dq, dk, dq_weight, dk_weight, workspace, status):
        return
    dt, gt = _TORCH.get(cfg.dtype), _TORCH.get(cfg.grad_dtype)
    if not cfg.Hkv:
        k = dk_out = dk = None
    _qk_check(cfg, (("", q, k, dt), ("d_out", dq_out, dk_out, gt), ("d", dq, dk, dt)), q_weight,
              k_weight, cos, sin, pos, status)
    for name, w in (("dq_weight", dq_weight), ("dk_weight", dk_weight)):
        if w is not None:
            _want(w, name, (cfg.D,), torch.float32, q.device)
    _want_workspace(workspace, q.device)
    _launch(i, stream, _lib.pbsa_qk_norm_rope_bwd, _cfg(cfg), q.data_ptr(), _ptr(k),
            _strides(q, k, dq_out, dk_out, dq, dk), _ptr(q_weight), _ptr(k_weight), _ptr(cos), _ptr(sin), _ptr(pos), dq_out.data_ptr(),
            _ptr(dk_out), dq.data_ptr(), _ptr(dk), _ptr(dq_weight), _ptr(dk_weight),
            _ptr(workspace), _bytes(workspace), _ptr(status))


def pbsa_validate_kv4_config(cfg):
    _check(_lib.pbsa_validate_kv4_config(_cfg(cfg)))


def pbsa_kv4_workspace_size(cfg, T: int) -> int:
    n = _lib.pbsa_kv4_workspace_size(_cfg(cfg), T)
    if n == 0 and T != 0:
        raise PBSAError(PBSA_ERR_ARG, pbsa_last_error())
    return n


def _kv4_check(cfg, cache):
    if cache.shape != (cfg.B, cfg.Hkv, cfg.capacity, cfg.D):
        _bad(f"cache of shape {cache.shape} does not belong to this configuration")
    return cache.device, cache.index


def pbsa_kv4_append(cfg, cache, k_new, v_new, pos_new, rows, mass, status, stream=None):
    """Quantises the new tokens' keys and values into `rows` (None: row = position)."""
    dev, i = _kv4_check(cfg, cache)
    if _quick(_calls.kv4_append, pbsa_kv4_config, cfg, i, stream, ctypes.addressof(cache), k_new, v_new,
              pos_new, rows, mass, status):
        return
    B, Hkv, T, dt, i32 = cfg.B, cfg.Hkv, k_new.shape[1], _TORCH.get(cfg.dtype), torch.int32
    shape = (B, T, Hkv, cfg.D)
    _want(k_new, "k_new", shape, dt, dev, True)
    _want(v_new, "v_new", shape, dt, dev, True)
    _want(pos_new, "pos_new", (B, T), i32, dev)
    _want(status, "status", (1,), i32, dev)
    if rows is not None:
        _want(rows, "rows", (B, Hkv, T), i32, dev)
    if mass is not None:
        _want(mass, "mass", (B, Hkv, cfg.capacity), torch.float32, dev)
    _launch(i, stream, _lib.pbsa_kv4_append, _cfg(cfg), ctypes.byref(cache), k_new.data_ptr(),
            v_new.data_ptr(), _strides(k_new, v_new), T, pos_new.data_ptr(), _ptr(rows), _ptr(mass), _ptr(status))


def pbsa_kv4_read(cfg, cache, rows, k_out, v_out, status, stream=None):
    """The values of the given rows (None: the first k_out.shape[2] rows)."""
    dev, i = _kv4_check(cfg, cache)
    if _quick(_calls.kv4_read, pbsa_kv4_config, cfg, i, stream, ctypes.addressof(cache), rows, k_out,
              v_out, status):
        return
    n, dt = k_out.shape[2], _TORCH.get(cfg.dtype)
    shape = (cfg.B, cfg.Hkv, n, cfg.D)
    _want(k_out, "k_out", shape, dt, dev)
    _want(v_out, "v_out", shape, dt, dev)
    _want(status, "status", (1,), torch.int32, dev)
    if rows is not None:
        _want(rows, "rows", shape[:3], torch.int32, dev)
    _launch(i, stream, _lib.pbsa_kv4_read, _cfg(cfg), ctypes.byref(cache), _ptr(rows), n,
            _ptr(k_out), v_out.data_ptr(), _ptr(status))


def pbsa_kv4_attn(cfg, cache, q, q_pos, kv_len, out, lse, mass, workspace, status, stream=None):
    """Attention of q [B, T, Hq, D] over the cache; q_pos and mass may be None."""
    dev, i = _kv4_check(cfg, cache)
    if _quick(_calls.kv4_attn, pbsa_kv4_config, cfg, i, stream, ctypes.addressof(cache), q, q_pos,
              kv_len, out, lse, mass, workspace, status):
        return
    B, Hq, T, dt = cfg.B, cfg.Hq, q.shape[1], _TORCH.get(cfg.dtype)
    f32, i32, shape = torch.float32, torch.int32, (B, T, Hq, cfg.D)
    _want(q, "q", shape, dt, dev, True)
    _want(out, "out", shape, dt, dev)
    _want(lse, "lse", (B, Hq, T), f32, dev)
    _want(kv_len, "kv_len", (B,), i32, dev)
    _want(status, "status", (1,), i32, dev)
    if q_pos is not None:
        _want(q_pos, "q_pos", (B, T), i32, dev)
    if mass is not None:
        _want(mass, "mass", (B, cfg.Hkv, cfg.capacity), f32, dev)
    _want_workspace(workspace, dev)
    _launch(i, stream, _lib.pbsa_kv4_attn, _cfg(cfg), ctypes.byref(cache), q.data_ptr(), _strides(q), T,
            _ptr(q_pos), kv_len.data_ptr(), out.data_ptr(), lse.data_ptr(), _ptr(mass), _ptr(workspace),
            _bytes(workspace), _ptr(status))


def pbsa_kv4_evict(cfg, pos, mass, n_sink, keep_from, rows, status, stream=None):
    """Chooses rows.shape[2] rows of every sequence and key head for the next tokens."""
    i = pos.get_device()
    if _quick(_calls.kv4_evict, pbsa_kv4_config, cfg, i, stream, pos, mass, n_sink, keep_from, rows,
              status):
        return
    n, i32, dev = rows.shape[2], torch.int32, pos.device
    B, Hkv = cfg.B, cfg.Hkv
    shape = (B, Hkv, cfg.capacity)
    _want(pos, "pos", shape, i32, dev)
    _want(mass, "mass", shape, torch.float32, dev)
    _want(rows, "rows", (B, Hkv, n), i32, dev)
    _want(status, "status", (1,), i32, dev)
    if keep_from is not None:
        _want(keep_from, "keep_from", (B,), i32, pos.device)
    _launch(i, stream, _lib.pbsa_kv4_evict, _cfg(cfg), _ptr(pos), _ptr(mass), n, n_sink,
            _ptr(keep_from), _ptr(rows), _ptr(status))
