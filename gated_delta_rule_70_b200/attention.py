"""Binding of the softmax-attention layer's operators: rotary positions, the append to a paged
8-bit key / value cache and the attention over it (``kda_rope``, ``kda_cache_append``,
``kda_cache_attend`` in ``include/kda.h``).

Argument marshalling only, as in ``gated_delta_rule_70_b200.kda``: work is enqueued on torch's
current stream of the tensors' device, nothing is computed on the host, and there is no fallback.
All tensors of a call live on one device, which need not be the current one.
"""

from __future__ import annotations

import ctypes
import math
import struct
from typing import Optional, Tuple

import torch

from . import kda as _kda

KDA_STATUS_BAD_PAGE, KDA_STATUS_BAD_LENGTH, KDA_STATUS_TIMEOUT_ATTEND = 0x10, 0x20, 0x40
LAYOUTS = {"half": 0, "interleaved": 1}
SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3}


_CODES = {ctypes.c_int32: "i", ctypes.c_uint32: "I", ctypes.c_int64: "q", ctypes.c_float: "f",
          ctypes.c_void_p: "P"}


def _packer(cls):
    """A function from the values of an argument block's fields (addresses as int) to its bytes: a
    call takes them as a pointer, at a fraction of the host time of building the ctypes object."""
    layout = struct.Struct("@" + "".join(_CODES[t] for _, t in cls._fields_))
    assert layout.size <= ctypes.sizeof(cls) < layout.size + 8     # (but for the padding at the end)
    return layout.pack


class RopeConfig(ctypes.Structure):
    """kda_rope_config."""
    _fields_ = [("rot_dim", ctypes.c_int32), ("scaling", ctypes.c_int32), ("base", ctypes.c_double),
                ("factor", ctypes.c_double), ("original_context", ctypes.c_double),
                ("beta_fast", ctypes.c_double), ("beta_slow", ctypes.c_double)]


class RopeArgs(ctypes.Structure):
    """kda_rope_args."""
    _fields_ = [("num_tokens", ctypes.c_int64), ("q_heads", ctypes.c_int32), ("k_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("rot_dim", ctypes.c_int32), ("layout", ctypes.c_int32),
                ("inverse", ctypes.c_int32), ("io_dtype", ctypes.c_int32), ("amplitude", ctypes.c_float),
                ("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("q_out", ctypes.c_void_p),
                ("k_out", ctypes.c_void_p), ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64),
                ("q_out_stride", ctypes.c_int64), ("k_out_stride", ctypes.c_int64),
                ("positions", ctypes.c_void_p), ("frequencies", ctypes.c_void_p)]


class Cache(ctypes.Structure):
    """kda_cache."""
    _fields_ = [(n, ctypes.c_int32) for n in ("num_seqs", "num_kv_heads", "head_dim", "page_tokens",
                                              "num_pages", "max_pages")] + \
               [(n, ctypes.c_void_p) for n in ("k_cache", "v_cache", "k_scale", "v_scale",
                                               "block_table", "seq_lens")]


class CacheAppendArgs(ctypes.Structure):
    """kda_cache_append_args."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_stride", ctypes.c_int64),
                ("v_stride", ctypes.c_int64), ("num_new", ctypes.c_int32), ("io_dtype", ctypes.c_int32),
                ("cu_seqlens", ctypes.c_void_p), ("status", ctypes.c_void_p)]


class CacheAttendArgs(ctypes.Structure):
    """kda_cache_attend_args."""
    _fields_ = [("q", ctypes.c_void_p), ("q_stride", ctypes.c_int64), ("num_new", ctypes.c_int32),
                ("num_heads", ctypes.c_int32), ("io_dtype", ctypes.c_int32), ("flags", ctypes.c_uint32),
                ("scale", ctypes.c_float), ("o", ctypes.c_void_p), ("lse", ctypes.c_void_p),
                ("status", ctypes.c_void_p)]


_pack_rope, _pack_cache = _packer(RopeArgs), _packer(Cache)
_pack_append, _pack_attend = _packer(CacheAppendArgs), _packer(CacheAttendArgs)


def _refuse(t, name, dtype, device):
    """What _check_tensor and _tokens found wrong with a tensor's kind or place."""
    if not isinstance(t, torch.Tensor) or t.dtype != dtype:
        raise ValueError("%s must be a %s tensor" % (name, dtype))
    if t.device != device:
        raise ValueError("%s must live on %s, not on %s" % (name, device, t.device))
    raise ValueError("%s must be contiguous" % name)


def _check_tensor(t, name, dtype, device, shape=None):
    """A contiguous tensor of that type on that device (and of that shape)."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.device == device and t.is_contiguous()):
        _refuse(t, name, dtype, device)
    if shape is not None and t.shape != shape:
        raise ValueError("%s must have the shape %s, not %s" % (name, tuple(shape), tuple(t.shape)))


def _tokens(t, name, dtype, device, heads, d):
    """(number of tokens, elements between tokens) of [.., heads, d] whose tokens lie at one
    distance from one another and whose heads are contiguous."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.device == device):
        _refuse(t, name, dtype, device)
    shape = t.shape
    if len(shape) < 3 or shape[-1] != d or shape[-2] != heads:
        raise ValueError("%s must have the shape [.., %d, %d], not %s" % (name, heads, d, tuple(shape)))
    row = heads * d
    total = t.numel()
    if total == 0:
        return 0, row
    if t.is_contiguous() and row % 8 == 0:
        return total // row, row
    stride = t.stride()
    if stride[-1] != 1 or (heads > 1 and stride[-2] != d):
        raise ValueError("the heads of %s must be contiguous" % name)
    step, count = None, 1
    for size, s in zip(reversed(shape[:-2]), reversed(stride[:-2])):
        if size > 1:
            if step is None:
                step = s
            elif s != step * count:
                raise ValueError("the tokens of %s must lie at one distance" % name)
            count *= size
    if step is None:
        step = row
    if step < row or step % 8:
        raise ValueError("the tokens of %s must lie a multiple of 8 elements apart, without overlap" % name)
    return count, step


def _on_device(device, call, *args):
    """The C call with the tensors' device current, on torch's current stream of it."""
    if device.type != "cuda":
        raise ValueError("KDA tensors must live on a CUDA device")
    if torch.cuda.current_device() == device.index:
        return call(*args, torch._C._cuda_getCurrentRawStream(device.index))
    with torch.cuda.device(device):
        return call(*args, torch._C._cuda_getCurrentRawStream(device.index))


def _empty_like(t):
    """A contiguous tensor of t's shape and type."""
    return torch.empty_like(t) if t.is_contiguous() else torch.empty(t.shape, dtype=t.dtype, device=t.device)


def rope_frequencies(rot_dim: int, base: float = 10000.0, *, scaling: str = "none", factor: float = 1.0,
                     original_context: float = 0.0, beta_fast: float = 32.0, beta_slow: float = 1.0,
                     device=None) -> Tuple[torch.Tensor, float]:
    """The rotation of each channel pair in radians per token, [rot_dim / 2] fp64, and the factor
    on cosine and sine.  ``scaling``: "none", "linear", "ntk" or "yarn" (``kda_rope_frequencies``).
    Made once; ``device``: where the frequencies are to live (default: the CPU)."""
    if scaling not in SCALINGS:
        raise ValueError("scaling must be one of %s" % ", ".join(SCALINGS))
    c = RopeConfig(int(rot_dim), SCALINGS[scaling], base, factor, original_context, beta_fast, beta_slow)
    host = (ctypes.c_double * 128)()
    amplitude = ctypes.c_float(0.0)
    _kda._check(_kda.load_library().kda_rope_frequencies(ctypes.byref(c), host, ctypes.byref(amplitude)),
                "kda_rope_frequencies")
    f = torch.tensor(host[:rot_dim // 2], dtype=torch.float64)
    return (f if device is None else f.to(device)), float(amplitude.value)


def rope(q: torch.Tensor, k: Optional[torch.Tensor], positions: torch.Tensor, frequencies: torch.Tensor, *,
         amplitude: float = 1.0, layout: str = "half", inverse: bool = False,
         out: Optional[Tuple[torch.Tensor, Optional[torch.Tensor]]] = None):
    """Rotary positions: q [.., Hq, d] and k [.., Hk, d] (or None) with ``positions`` int32, one for
    each token, rotated by ``frequencies`` [rot_dim / 2] fp64; returns (q, k) rotated.  Channels from
    rot_dim on pass through.  ``layout``: "half" or "interleaved" pairs.  ``inverse``: the transposed
    map, from the gradient of the outputs to that of the inputs.  ``out``: (q_out, k_out), which may
    be (q, k) themselves.  Tokens may lie apart (parts of one projection's output)."""
    lib = _kda.load_library()
    if layout not in LAYOUTS:
        raise ValueError("layout must be one of %s" % ", ".join(LAYOUTS))
    dev, dt = q.device, q.dtype
    code = _kda._dtype_code(dt)
    heads, d = q.shape[-2:] if q.dim() >= 3 else (0, 0)
    nt, q_step = _tokens(q, "q", dt, dev, heads, d)
    hk, k_step = 0, 0
    if k is not None:
        hk = k.shape[-2] if k.dim() >= 3 else 0
        nk, k_step = _tokens(k, "k", dt, dev, hk, d)
        if nk != nt:
            raise ValueError("q and k must have the same tokens")
    _check_tensor(positions, "positions", torch.int32, dev)
    _check_tensor(frequencies, "frequencies", torch.float64, dev)
    if positions.numel() != nt:
        raise ValueError("positions must have one entry for each of the %d tokens" % nt)
    if frequencies.dim() != 1:
        raise ValueError("frequencies must be a vector")
    if out is None:
        qo = _empty_like(q)
        ko = None if k is None else _empty_like(k)
        qo_step, ko_step = heads * d, hk * d
    else:
        qo, ko = out
        if (ko is None) != (k is None) or qo.shape != q.shape or (k is not None and ko.shape != k.shape):
            raise ValueError("out must be (q_out, k_out) of the shapes of q and k")
        _, qo_step = _tokens(qo, "q_out", dt, dev, heads, d)
        ko_step = 0 if k is None else _tokens(ko, "k_out", dt, dev, hk, d)[1]
    a = _pack_rope(nt, heads, hk, d, 2 * frequencies.numel(), LAYOUTS[layout], int(inverse), code, amplitude,
                   q.data_ptr(), 0 if k is None else k.data_ptr(), qo.data_ptr(),
                   0 if k is None else ko.data_ptr(), q_step, k_step, qo_step, ko_step,
                   positions.data_ptr(), frequencies.data_ptr())
    _kda._check(_on_device(dev, lib.kda_rope, a), "kda_rope")
    return qo, ko


def _cache(k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, device):
    """(kda_cache as bytes, num_seqs, num_kv_heads, head_dim)."""
    if k_cache.dim() != 4 or block_table.dim() != 2:
        raise ValueError("k_cache must be [num_pages, num_kv_heads, page_tokens, head_dim] and "
                         "block_table [num_seqs, max_pages]")
    shape = k_cache.shape
    pages, hk, p, d = shape
    n, columns = block_table.shape
    _check_tensor(k_cache, "k_cache", torch.float8_e4m3fn, device)
    _check_tensor(v_cache, "v_cache", torch.float8_e4m3fn, device, shape)
    _check_tensor(k_scale, "k_scale", torch.float32, device, (pages, hk))
    _check_tensor(v_scale, "v_scale", torch.float32, device, (pages, hk))
    _check_tensor(block_table, "block_table", torch.int32, device)
    _check_tensor(seq_lens, "seq_lens", torch.int32, device, (n,))
    return _pack_cache(n, hk, d, p, pages, columns, k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(),
                       v_scale.data_ptr(), block_table.data_ptr(), seq_lens.data_ptr()), n, hk, d


def _status_word(status, check, device):
    if status is None:
        return torch.empty(1, dtype=torch.int32, device=device) if check else None
    _check_tensor(status, "status", torch.int32, device)
    if status.numel() < 1:
        raise ValueError("status must hold one int32")
    return status


def _device_check(status, what, device):
    """Waits for the call and raises what its status word reports."""
    _kda._check(_on_device(device, _kda.load_library().kda_device_status, status.data_ptr()), what + " (device)")


def cache_append(k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                 k_scale: torch.Tensor, v_scale: torch.Tensor, block_table: torch.Tensor,
                 seq_lens: torch.Tensor, *, cu_seqlens: Optional[torch.Tensor] = None,
                 status: Optional[torch.Tensor] = None, check: bool = False) -> None:
    """Quantises the new tokens' keys and values, k and v [N, T, Hkv, d] (or packed [tokens, Hkv, d]:
    with ``cu_seqlens`` [N + 1], or N equal shares without), into the cache, in place: k_cache,
    v_cache [num_pages, Hkv, page_tokens, d] float8_e4m3fn with k_scale, v_scale [num_pages, Hkv]
    fp32.  ``seq_lens`` [N] counts the new tokens, which are each sequence's last.
    ``status``: a device int32 the call zeroes and sets on a bad page, length or cu_seqlens;
    ``check=True`` waits for the call and raises on it."""
    lib = _kda.load_library()
    dev, dt = k.device, k.dtype
    code = _kda._dtype_code(dt)
    c, n, hk, d = _cache(k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, dev)
    total, k_step = _tokens(k, "k", dt, dev, hk, d)
    tv, v_step = _tokens(v, "v", dt, dev, hk, d)
    if tv != total:
        raise ValueError("k and v must have the same tokens")
    if cu_seqlens is not None:
        _check_tensor(cu_seqlens, "cu_seqlens", torch.int32, dev, (n + 1,))
        new = total
    else:
        new = total // n if n else 0
        if new * n != total or (k.dim() == 4 and total and k.shape[0] != n):
            raise ValueError("k and v must hold the same number of tokens for each of the %d sequences" % n)
    word = _status_word(status, check, dev)
    a = _pack_append(k.data_ptr(), v.data_ptr(), k_step, v_step, new, code,
                     0 if cu_seqlens is None else cu_seqlens.data_ptr(), 0 if word is None else word.data_ptr())
    _kda._check(_on_device(dev, lib.kda_cache_append, c, a), "kda_cache_append")
    if check:
        _device_check(word, "kda_cache_append", dev)


def cache_attend_workspace_size(cache, args) -> int:
    """Bytes of workspace for a kda_cache and a kda_cache_attend_args (ctypes objects or bytes)."""
    p = [x if isinstance(x, bytes) else ctypes.byref(x) for x in (cache, args)]
    return int(_kda.load_library().kda_cache_attend_workspace_size(*p))


def cache_attend(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, k_scale: torch.Tensor,
                 v_scale: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor, *,
                 scale: Optional[float] = None, want_lse: bool = False, out: Optional[torch.Tensor] = None,
                 lse: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                 status: Optional[torch.Tensor] = None, check: bool = False, flags: int = 0):
    """Causal attention of each sequence's last T tokens (already appended), q [N, T, Hq, d], over its
    cache; returns o [N, T, Hq, d], or (o, lse [N, T, Hq] fp32) with ``want_lse`` or ``lse``.
    ``scale``: on the scores, 1 / sqrt(d) if None.  A token that sees nothing gets o = 0 and lse =
    -inf.  ``workspace``: uint8, one for each call that may run at the same time (default: a new one).
    ``status``, ``check`` as in ``cache_append``; ``flags``: raw KDA_FLAG_* bits."""
    lib = _kda.load_library()
    dev, dt = q.device, q.dtype
    code = _kda._dtype_code(dt)
    c, n, _, d = _cache(k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, dev)
    shape = q.shape
    if len(shape) != 4 or shape[0] != n or shape[1] < 1:
        raise ValueError("q must be [%d, T >= 1, heads, %d], not %s" % (n, d, tuple(shape)))
    t, hq = shape[1], shape[2]
    _, q_step = _tokens(q, "q", dt, dev, hq, d)
    if out is None:
        out = _empty_like(q)
    else:
        _check_tensor(out, "out", dt, dev, shape)
    if lse is not None:
        _check_tensor(lse, "lse", torch.float32, dev, (n, t, hq))
    elif want_lse:
        lse = q.new_empty((n, t, hq), dtype=torch.float32)
    word = _status_word(status, check, dev)
    a = _pack_attend(q.data_ptr(), q_step, t, hq, code, int(flags), 1.0 / math.sqrt(d) if scale is None else scale,
                     out.data_ptr(), 0 if lse is None else lse.data_ptr(), 0 if word is None else word.data_ptr())
    if workspace is None:
        size = lib.kda_cache_attend_workspace_size(c, a)
        if size > 0:
            workspace = q.new_empty(size, dtype=torch.uint8)
    else:
        _check_tensor(workspace, "workspace", torch.uint8, dev)
        size = workspace.numel()
    _kda._check(_on_device(dev, lib.kda_cache_attend, c, a, 0 if workspace is None else workspace.data_ptr(), size),
                "kda_cache_attend")
    if check:
        _device_check(word, "kda_cache_attend", dev)
    return out if lse is None else (out, lse)
