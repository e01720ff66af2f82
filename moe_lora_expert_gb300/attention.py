"""Rotary positions, the paged 8-bit cache and attention over it.

The attention half of a decoder layer, for serving next to ``MoeLoraLayer``:

    cos_sin = rope_table(131072, 128, scaling={"kind": "yarn", "factor": 4.0, "original": 32768}, device="cuda")
    cache = PagedKVCache.create(num_pages=4096, kv_heads=4, page_size=64, head_dim=128)
    q = cache.append(k, v, block_table, seq_lens, q=q, cos_sin=cos_sin)    # k and q rotated on the way
    out = cache.attend(q, block_table, seq_lens)                           # one new token a sequence

Argument marshalling only, as in the package's other bindings: every step runs
in the library's kernels, PyTorch supplies memory and streams.  The arguments
of a call are packed into the C struct's bytes in one go, since the host's
share of a decode step counts.
"""
from __future__ import annotations

import ctypes
import math
import struct
from typing import Dict, Optional

MOE_DTYPE_BF16 = 0
MOE_DTYPE_F16 = 1
MOE_DTYPE_F32 = 2
MOE_DEBUG_STALL_ATTENTION = 4


class RopeArgs(ctypes.Structure):
    _fields_ = [("struct_size", ctypes.c_uint32), ("dtype", ctypes.c_int),
                *[(n, ctypes.c_void_p) for n in ("q", "q_out", "k", "k_out")],
                *[(n, ctypes.c_int64) for n in (
                    "q_stride_token", "q_stride_head", "q_out_stride_token", "q_out_stride_head",
                    "k_stride_token", "k_stride_head", "k_out_stride_token", "k_out_stride_head")],
                *[(n, ctypes.c_void_p) for n in ("positions", "cos_sin", "status")],
                *[(n, ctypes.c_int) for n in ("N", "Hq", "Hk", "D", "rotary_dim", "num_positions",
                                              "interleaved", "inverse")]]


class KvCache(ctypes.Structure):
    _fields_ = [*[(n, ctypes.c_void_p) for n in ("k", "v", "k_scale", "v_scale")],
                *[(n, ctypes.c_int64) for n in ("k_stride_page", "k_stride_head", "k_stride_token",
                                                "v_stride_page", "v_stride_head", "v_stride_token")],
                *[(n, ctypes.c_int) for n in ("num_pages", "kv_heads", "page_size", "head_dim")]]


class KvAppendArgs(ctypes.Structure):
    _fields_ = [("struct_size", ctypes.c_uint32), ("dtype", ctypes.c_int), ("cache", KvCache),
                ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                *[(n, ctypes.c_int64) for n in ("k_stride_token", "k_stride_head", "v_stride_token",
                                                "v_stride_head")],
                ("q", ctypes.c_void_p), ("q_out", ctypes.c_void_p),
                *[(n, ctypes.c_int64) for n in ("q_stride_token", "q_stride_head", "q_out_stride_token",
                                                "q_out_stride_head")],
                *[(n, ctypes.c_void_p) for n in ("block_table", "seq_lens", "cu_q", "positions",
                                                 "cos_sin", "status")],
                *[(n, ctypes.c_int) for n in ("N", "B", "Hq", "table_width", "max_q_len", "rotary_dim",
                                              "num_positions", "interleaved")]]


class PagedAttentionArgs(ctypes.Structure):
    _fields_ = [("struct_size", ctypes.c_uint32), ("dtype", ctypes.c_int), ("cache", KvCache),
                *[(n, ctypes.c_void_p) for n in ("q", "out", "lse")],
                *[(n, ctypes.c_int64) for n in ("q_stride_token", "q_stride_head", "out_stride_token",
                                                "out_stride_head")],
                *[(n, ctypes.c_void_p) for n in ("block_table", "seq_lens", "cu_q", "status", "workspace")],
                ("workspace_bytes", ctypes.c_size_t),
                *[(n, ctypes.c_int) for n in ("N", "B", "Hq", "table_width", "max_q_len", "max_seq_len",
                                              "window", "wait_timeout_ms")],
                ("scale", ctypes.c_float), ("debug_flags", ctypes.c_uint32)]


# The same layouts as bytes (64-bit pointers; the structs have no padding but
# where every 8-byte field is aligned already).
_ROPE = struct.Struct("=Ii4Q8q3Q8i")
_CACHE = struct.Struct("=4Q6q4i")
_HEAD = struct.Struct("=Ii")
_APPEND = struct.Struct("=2Q4q2Q4q6Q8i")
_ATTEND = struct.Struct("=3Q4q6Q8ifI")

# What the entry points use on every call, bound by the first one (torch is
# imported lazily, as in the rest of the package).
_torch = _int32_type = _float32_type = None
_codes: Dict = {}
_rope_fn = _append_fn = _attend_fn = _raw_stream = _empty_like = _capturing = _current_device = None

# Scratch of attention calls: calls on one stream follow one another and share
# it, whatever their cache; a captured call runs when its graph does, so each
# capture has its own.
_workspaces: Dict = {}       # device index: {stream handle: (pointer, bytes, tensor)}
_captured: Dict = {}         # (device index, stream handle): (capture id, workspace) of the latest capture


def _bind():
    global _torch, _int32_type, _float32_type, _rope_fn, _append_fn, _attend_fn, _raw_stream, _empty_like, _capturing
    global _current_device
    import torch
    from . import lib
    L = lib()
    _codes.update({torch.bfloat16: MOE_DTYPE_BF16, torch.float16: MOE_DTYPE_F16, torch.float32: MOE_DTYPE_F32})
    _int32_type, _float32_type = torch.int32, torch.float32
    _append_fn, _attend_fn, _raw_stream = L.moe_kv_append, L.moe_paged_attention, torch._C._cuda_getCurrentRawStream
    _empty_like, _capturing = torch.empty_like, torch.cuda.is_current_stream_capturing
    _current_device = torch._C._cuda_getDevice
    _rope_fn, _torch = L.moe_rope, torch


def _raise(status, what):
    from . import MoeError
    raise MoeError(status, what)


def _elsewhere(index, fn, *args):
    """A call on a device that is not the current one: the library launches on
    the current device, whose stream 0 is another one."""
    with _torch.cuda.device(index):
        return fn(*args)


def _handle(stream, index):
    """The handle of a call's stream on its tensors' device."""
    if stream is None:
        return _raw_stream(index)
    if stream.device_index != index:
        raise ValueError(f"the stream is of cuda:{stream.device_index}, the tensors are on cuda:{index}")
    return stream.cuda_stream


def _record(stream, *tensors):
    """A call on a stream of the caller's choice uses these: their memory is
    not given to others before it is done."""
    for t in tensors:
        if t is not None:
            t.record_stream(stream)


def _dtype_code(dtype, name):
    code = _codes.get(dtype)
    if code is None:
        raise ValueError(f"{name} must be bfloat16, float16 or (moe_rope) float32, got {dtype}")
    return code


def _empty(shape, dtype, device, stream):
    """An output of a call on ``stream``: its memory belongs to that stream."""
    if stream is None:
        return _torch.empty(shape, dtype=dtype, device=device)
    with _torch.cuda.stream(stream):
        return _torch.empty(shape, dtype=dtype, device=device)


def _out_like(x, token, head, N, H, D, dtype, stream):
    """A contiguous output of x's shape (token, head: x's strides) and its pointer."""
    if stream is None and head == D and token == H * D:
        y = _empty_like(x)
    else:
        y = _empty((N, H, D), dtype, x.device, stream)
    return y, y.data_ptr()


def _new_workspace(index, handle):
    """Memory of the stream's own, made ready in its order: of the graph's own
    and as part of it where the stream is being captured."""
    from . import lib
    stream = _torch.cuda.ExternalStream(handle, device=index) if handle else _torch.cuda.default_stream(index)
    with _torch.cuda.stream(stream):
        n = int(lib().moe_paged_attention_workspace_size())
        t = _torch.empty(n, dtype=_torch.uint8, device=_torch.device("cuda", index))
        error = lib().moe_paged_attention_workspace_init(t.data_ptr(), n, handle)
    if error:
        _raise(error, "moe_paged_attention_workspace_init")
    return t.data_ptr(), n, t


def _captured_workspace(index, handle):
    """The workspace of the capture that the stream is in, or None."""
    from . import lib
    capture = ctypes.c_uint64(0)
    error = lib().moe_stream_capture_id(handle, ctypes.byref(capture))
    if error:
        _raise(error, "moe_stream_capture_id")
    if capture.value == 0:
        return None
    held = _captured.get((index, handle))
    if held is None or held[0] != capture.value:
        # the last capture's goes back to its graph, which keeps the memory
        held = _captured[index, handle] = (capture.value, _new_workspace(index, handle))
    return held[1]


def _int32(t, n, name, index):
    """Pointer of an int32 [n] tensor on a call's device."""
    if t.dtype is not _int32_type or t.get_device() != index or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor on cuda:{index}")
    if t.shape != (n,):
        raise ValueError(f"{name} must have shape [{n}], got {tuple(t.shape)}")
    return t.data_ptr()


def _heads(t, N, H, D, dtype, name, index):
    """(pointer, token stride, head stride) of a [N, H, D] tensor."""
    if t.shape != (N, H, D):
        raise ValueError(f"{name} must have shape [{N}, {H}, {D}], got {tuple(t.shape)}")
    if t.dtype is not dtype or t.get_device() != index:
        raise ValueError(f"{name} must be a {dtype} tensor on cuda:{index}")
    st, sh, sd = t.stride()
    if sd != 1:
        raise ValueError(f"{name} must be contiguous along the head dimension")
    return t.data_ptr(), st, sh


def _table(cos_sin, index):
    shape = cos_sin.shape
    if cos_sin.dtype is not _float32_type or cos_sin.get_device() != index or len(shape) != 2 or not cos_sin.is_contiguous():
        raise ValueError(f"cos_sin must be a contiguous float32 tensor [positions, rotary_dim] on cuda:{index}")
    return cos_sin.data_ptr(), shape[0], shape[1]


# ----------------------------------------------------------------------------
# Angles
# ----------------------------------------------------------------------------

def rope_frequencies(rotary_dim: int, base: float = 10000.0, scaling: Optional[Dict] = None):
    """(angle per position of each pair: list of rotary_dim / 2 floats, factor
    on cos and sin).  ``scaling``, for contexts past the trained ones:

    {"kind": "linear", "factor": s}     every angle / s
    {"kind": "ntk", "factor": s}        base * s^(R / (R - 2)): the slowest angle / s, the fastest kept
    {"kind": "yarn", "factor": s, "original": trained length, "beta_fast": 32, "beta_slow": 1,
     "mscale": None}                    angles that turn more than beta_fast times in the trained
                                        length kept, those under beta_slow / s, a ramp between;
                                        cos and sin times mscale (0.1 ln s + 1)
    {"kind": "llama3", "factor": s, "original": trained length, "low": 1, "high": 4}
                                        wavelengths under original / high kept, those over
                                        original / low divided by s, a blend between
    """
    if rotary_dim < 2 or rotary_dim % 2:
        raise ValueError("rotary_dim must be even and at least 2")
    R, sc = rotary_dim, dict(scaling or {"kind": "none"})
    kind = sc.pop("kind", None)
    factor = float(sc.pop("factor", 1.0))
    if not 0 < factor < math.inf or not 0 < base < math.inf:
        raise ValueError("factor and base must be positive and finite")
    if kind in ("yarn", "llama3") and not float(sc.get("original", 0)) > 0:
        raise ValueError(f"scaling kind {kind!r} needs the trained length, original > 0")
    mscale = 1.0
    if kind == "ntk" and R > 2:
        base = base * factor ** (R / (R - 2.0))
    f = [base ** (-2.0 * i / R) for i in range(R // 2)]
    if kind == "linear":
        f = [x / factor for x in f]
    elif kind == "yarn":
        original = float(sc.pop("original"))
        fast, slow = float(sc.pop("beta_fast", 32.0)), float(sc.pop("beta_slow", 1.0))
        if not fast > 0 or not slow > 0 or not base > 1:
            raise ValueError("yarn needs beta_fast > 0, beta_slow > 0 and base > 1")
        pair = lambda turns: R * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(base))
        lo, hi = max(math.floor(pair(fast)), 0), min(math.ceil(pair(slow)), R - 1)
        ramp = [min(max((i - lo) / max(hi - lo, 1e-3), 0.0), 1.0) for i in range(R // 2)]
        f = [x * (1 - r) + x / factor * r for x, r in zip(f, ramp)]
        given = sc.pop("mscale", None)
        mscale = float(given) if given is not None else (0.1 * math.log(factor) + 1.0 if factor > 1 else 1.0)
    elif kind == "llama3":
        original = float(sc.pop("original"))
        low, high = float(sc.pop("low", 1.0)), float(sc.pop("high", 4.0))
        if not low < high:
            raise ValueError("llama3 needs low < high")
        blend = [min(max((original * x / (2 * math.pi) - low) / (high - low), 0.0), 1.0) for x in f]
        f = [x / factor * (1 - b) + x * b for x, b in zip(f, blend)]
    elif kind not in ("none", "ntk"):
        raise ValueError(f"unknown scaling kind {kind!r}")
    if sc:
        raise ValueError(f"unknown scaling arguments {sorted(sc)} for kind {kind!r}")
    return f, mscale


def rope_table(max_positions: int, rotary_dim: int, base: float = 10000.0,
               scaling: Optional[Dict] = None, device=None):
    """float32 [max_positions, rotary_dim]: cosines, then sines, of each
    position's angles, computed in float64.  Made once, at load time."""
    import torch
    f, mscale = rope_frequencies(rotary_dim, base, scaling)
    at = torch.arange(max_positions, dtype=torch.float64, device=device)[:, None]
    at = at * torch.tensor(f, dtype=torch.float64, device=device)
    return torch.cat([at.cos() * mscale, at.sin() * mscale], dim=1).float()


def moe_rope(q, positions, cos_sin, k=None, interleaved=False, inverse=False, q_out=None, k_out=None,
             status=None, stream=None):
    """q [N, Hq, D] (and k [N, Hk, D]) rotated by ``positions`` int32 [N]; the
    columns past the table's rotary_dim are copied.  Returns q_out, or (q_out,
    k_out); pass the inputs as outputs to rotate in place.  ``inverse``: the
    gradient of the forward for an upstream gradient in q's place."""
    if _rope_fn is None:
        _bind()
    N, Hq, D = q.shape
    dtype = q.dtype
    code = _dtype_code(dtype, "q")
    index = q.get_device()
    if index < 0:
        raise ValueError("q must be a CUDA tensor")
    handle = _handle(stream, index)
    qp, q0, q1 = _heads(q, N, Hq, D, dtype, "q", index)
    if q_out is None:
        q_out, op = _out_like(q, q0, q1, N, Hq, D, dtype, stream)
        o0, o1 = Hq * D, D
    else:
        op, o0, o1 = _heads(q_out, N, Hq, D, dtype, "q_out", index)
    kp = kop = k0 = k1 = ko0 = ko1 = Hk = 0
    if k is not None:
        Hk = k.shape[1]
        kp, k0, k1 = _heads(k, N, Hk, D, dtype, "k", index)
        if k_out is None:
            k_out, kop = _out_like(k, k0, k1, N, Hk, D, dtype, stream)
            ko0, ko1 = Hk * D, D
        else:
            kop, ko0, ko1 = _heads(k_out, N, Hk, D, dtype, "k_out", index)
    tp, rows, R = _table(cos_sin, index)
    args = _ROPE.pack(160, code, qp, op, kp, kop, q0, q1, o0, o1, k0, k1, ko0, ko1,
                      _int32(positions, N, "positions", index), tp,
                      0 if status is None else _int32(status, 4, "status", index),
                      N, Hq, Hk, D, R, rows, interleaved, inverse)
    if stream is not None:
        _record(stream, q, k, positions, cos_sin, q_out, k_out, status)
    error = _rope_fn(args, handle) if _current_device() == index else _elsewhere(index, _rope_fn, args, handle)
    if error:
        _raise(error, "moe_rope")
    return q_out if k is None else (q_out, k_out)


class PagedKVCache:
    """A paged cache of e4m3 codes with one float32 scale for each (page, head).

    k, v: uint8 or float8_e4m3fn [num_pages, kv_heads, page_size, head_dim], of
    any strides that keep the last axis contiguous (so a buffer that holds
    [num_pages, page_size, kv_heads, head_dim] goes in as its transpose);
    k_scale, v_scale: float32 [num_pages, kv_heads].  Token j of a sequence is
    at (block_table[b, j // page_size], j % page_size).
    """

    def __init__(self, k, v, k_scale, v_scale):
        if _rope_fn is None:
            _bind()
        torch = _torch
        fp8 = (torch.uint8, torch.float8_e4m3fn)
        index = k.get_device()
        for t, name in ((k, "k"), (v, "v")):
            if t.dtype not in fp8 or not t.is_cuda or t.dim() != 4 or t.shape != k.shape or t.stride(3) != 1:
                raise ValueError(f"{name}: uint8 or float8_e4m3fn CUDA [pages, kv_heads, page_size, head_dim], "
                                 "contiguous along the last axis, k and v alike")
        for t, name in ((k_scale, "k_scale"), (v_scale, "v_scale")):
            if t.dtype != torch.float32 or not t.is_cuda or t.shape != k.shape[:2] or not t.is_contiguous():
                raise ValueError(f"{name} must be a contiguous float32 CUDA tensor {tuple(k.shape[:2])}")
        for t, name in ((v, "v"), (k_scale, "k_scale"), (v_scale, "v_scale")):
            if t.get_device() != index:
                raise ValueError(f"{name} must be on cuda:{index}, as k is")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.num_pages, self.kv_heads, self.page_size, self.head_dim = k.shape
        self.device = k.device
        self.status = torch.zeros(4, dtype=torch.int32, device=k.device)
        torch.cuda.current_stream(k.device).synchronize()           # before a call on another stream writes it
        self._status_ptr = self.status.data_ptr()
        self._tensors = (k, v, k_scale, v_scale, self.status)
        self._bytes = _CACHE.pack(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
                                  *k.stride()[:3], *v.stride()[:3], *k.shape)
        self._index = index
        self._workspaces = _workspaces.setdefault(self._index, {})

    @classmethod
    def create(cls, num_pages: int, kv_heads: int, page_size: int, head_dim: int, tokens_first=False,
               device="cuda"):
        """An empty cache; ``tokens_first``: [page_size, kv_heads] inside a page."""
        import torch
        shape = (num_pages, page_size, kv_heads, head_dim) if tokens_first else (
            num_pages, kv_heads, page_size, head_dim)
        k, v = (torch.zeros(shape, dtype=torch.uint8, device=device) for _ in range(2))
        if tokens_first:
            k, v = k.transpose(1, 2), v.transpose(1, 2)
        ks, vs = (torch.ones((num_pages, kv_heads), dtype=torch.float32, device=device) for _ in range(2))
        return cls(k, v, ks, vs)

    def workspace(self, stream_handle: int):
        """(pointer, bytes, tensor): scratch of the calls on a stream, made by
        the first one.  All caches of a device share it (about 51 MiB a
        stream); it lives as long as the process, as torch's streams do.
        Calls inside a graph capture do not use it: each capture has its own,
        in the graph's memory."""
        ws = self._workspaces.get(stream_handle)
        if ws is None:
            ws = self._workspaces[stream_handle] = _new_workspace(self._index, stream_handle)
        return ws

    def _batch(self, N, block_table, seq_lens, cu_q, max_q_len):
        B, width = block_table.shape
        index = self._index
        if block_table.dtype is not _int32_type or block_table.get_device() != index or not block_table.is_contiguous():
            raise ValueError(f"block_table must be a contiguous int32 tensor [sequences, pages] on cuda:{index}")
        sl = _int32(seq_lens, B, "seq_lens", index)
        if cu_q is None:
            if N != B:
                raise ValueError("without cu_q there is one new token for each sequence")
            return B, width, block_table.data_ptr(), sl, 0, 1
        cu = _int32(cu_q, B + 1, "cu_q", index)
        return B, width, block_table.data_ptr(), sl, cu, N if max_q_len is None else max_q_len

    def append(self, k, v, block_table, seq_lens, cu_q=None, max_q_len=None, q=None, cos_sin=None,
               interleaved=False, positions=None, q_out=None, stream=None):
        """The new tokens' k (rotated by ``cos_sin``) and v, [N, kv_heads,
        head_dim], go into the pages of their sequences: tokens [cu_q[b],
        cu_q[b + 1]) (one each without cu_q) end at seq_lens[b]; a slot whose
        seq_lens is 0 without cu_q stands for no sequence.  ``q`` [N, Hq,
        head_dim] is rotated in the same launch and returned."""
        N, D, H, index = k.shape[0], self.head_dim, self.kv_heads, self._index
        dtype = k.dtype
        code = _dtype_code(dtype, "k")
        handle = _handle(stream, index)
        kp, k0, k1 = _heads(k, N, H, D, dtype, "k", index)
        vp, v0, v1 = _heads(v, N, H, D, dtype, "v", index)
        qp = q0 = q1 = op = o0 = o1 = Hq = 0
        if q is not None:
            Hq = q.shape[1]
            qp, q0, q1 = _heads(q, N, Hq, D, dtype, "q", index)
            if q_out is None:
                q_out, op = _out_like(q, q0, q1, N, Hq, D, dtype, stream)
                o0, o1 = Hq * D, D
            else:
                op, o0, o1 = _heads(q_out, N, Hq, D, dtype, "q_out", index)
        B, width, bt, sl, cu, longest = self._batch(N, block_table, seq_lens, cu_q, max_q_len)
        tp, rows, R = (0, 0, 0) if cos_sin is None else _table(cos_sin, index)
        args = _HEAD.pack(280, code) + self._bytes + _APPEND.pack(
            kp, vp, k0, k1, v0, v1, qp, op, q0, q1, o0, o1, bt, sl, cu,
            0 if positions is None else _int32(positions, N, "positions", index), tp, self._status_ptr,
            N, B, Hq, width, longest, R, rows, interleaved)
        if stream is not None:
            _record(stream, k, v, q, q_out, block_table, seq_lens, cu_q, cos_sin, positions, *self._tensors)
        error = _append_fn(args, handle) if _current_device() == index else _elsewhere(index, _append_fn, args, handle)
        if error:
            _raise(error, "moe_kv_append")
        return q_out

    def attend(self, q, block_table, seq_lens, cu_q=None, max_q_len=None, max_seq_len=None, scale=None,
               window=0, out=None, return_lse=False, lse=None, wait_timeout_ms=0, debug_flags=0, stream=None):
        """Causal attention of q [N, Hq, head_dim] over the cache: rows as in
        ``append``, whose keys have to be in the cache already.  ``window``:
        how many keys a row sees, its own included (0: all).  ``max_q_len``,
        ``max_seq_len``: host-side bounds that size the launch (by default N
        and the block table's width).  Returns out, or (out, lse float32 [N,
        Hq]) with ``return_lse`` or a given ``lse``."""
        N, Hq, D = q.shape
        dtype = q.dtype
        code, index = _dtype_code(dtype, "q"), self._index
        handle = _handle(stream, index)
        qp, q0, q1 = _heads(q, N, Hq, self.head_dim, dtype, "q", index)
        if out is None:
            out, op = _out_like(q, q0, q1, N, Hq, D, dtype, stream)
            o0, o1 = Hq * D, D
        else:
            op, o0, o1 = _heads(out, N, Hq, D, dtype, "out", index)
        if lse is not None:
            if lse.dtype is not _float32_type or lse.shape != (N, Hq) or not lse.is_contiguous() or lse.get_device() != index:
                raise ValueError(f"lse must be a contiguous float32 tensor [{N}, {Hq}] on cuda:{index}")
        elif return_lse:
            lse = _empty((N, Hq), _float32_type, self.device, stream)
        B, width, bt, sl, cu, longest = self._batch(N, block_table, seq_lens, cu_q, max_q_len)
        here = _current_device() == index
        ws = None
        if stream is not None or not here or _capturing():
            ws = _captured_workspace(index, handle)
        if ws is None:
            ws = self._workspaces.get(handle) or self.workspace(handle)
        args = _HEAD.pack(248, code) + self._bytes + _ATTEND.pack(
            qp, op, 0 if lse is None else lse.data_ptr(), q0, q1, o0, o1, bt, sl, cu, self._status_ptr, ws[0], ws[1],
            N, B, Hq, width, longest, width * self.page_size if max_seq_len is None else max_seq_len, window,
            wait_timeout_ms, D ** -0.5 if scale is None else scale, debug_flags)
        if stream is not None:
            _record(stream, q, out, lse, block_table, seq_lens, cu_q, *self._tensors)
        error = _attend_fn(args, handle) if here else _elsewhere(index, _attend_fn, args, handle)
        if error:
            _raise(error, "moe_paged_attention")
        return out if lse is None else (out, lse)

    def device_status(self) -> int:
        """The first problem that a call met on the device since the last
        reading (MOE_OK: none), and clears it.  Waits for the work of all the
        device's streams, since a call may be on any."""
        _torch.cuda.synchronize(self.device)
        code = int(self.status[0].item())
        if code:
            self.status.zero_()
            _torch.cuda.current_stream(self.device).synchronize()   # before a call on another stream writes it
        return code
