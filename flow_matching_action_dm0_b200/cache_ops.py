"""Python-side handle of the operators over key/value caches (argument
marshalling only; the computation runs in ``librtv.so``).

    ops = CacheOps(device=0)                                      # rtv_ops_create
    cache = QuantizedKV.empty(batch, capacity, n_kv_heads, head_dim, device=0)
    ops.write(cache, k, v, start=positions)                       # rtv_kv_write
    k, v = ops.read(cache, n=816, dtype="bf16")                   # rtv_kv_read
    out = ops.cross_attention(q, cache, lens=lens)                # rtv_cross_attention
    out, lse = ops.shared_attention(q, (pk, pv), (k, v), lse=True)   # rtv_shared_attention

Arrays are torch tensors on the handle's GPU, fp32 or bf16: queries
[B][T][Hq][D], keys and values [B][N][Hkv][D] (a shared prefix [N][Hkv][D]),
of any strides with a dense last index and 16-byte steps.  Results are new
tensors unless ``out`` is given.  Work goes to ``stream`` (a torch stream or
its address), or to torch's current stream of the handle's GPU; results and
workspaces are allocated for the stream that the work goes to, as if the call
were made inside ``torch.cuda.stream(stream)``, and tensors given to a call
with a stream may be released at once.  Outputs must not overlap inputs, and
no gradient flows through the calls.
"""

from __future__ import annotations

from typing import NamedTuple, Optional

import torch

from . import _lib as L
from ._lib import RTV_BF16, RTV_F32, RTV_FP8_E4M3, rtv_kv, rtv_queries
from .expert import on_stream

_CODES = {torch.float32: RTV_F32, torch.bfloat16: RTV_BF16}
_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def _place(x, what: str) -> int:
    x = int(x)
    if not -2 ** 31 <= x < 2 ** 31:   # (the C call takes an int; it refuses the negative ones)
        raise ValueError(f"{what}: {x} does not fit 32 bits")
    return x


class QuantizedKV(NamedTuple):
    """Keys and values in E4M3: codes [B][Hkv][capacity][D]
    (torch.float8_e4m3fn) and the scale of each row, fp32 [B][Hkv][capacity];
    a row stands for code * scale."""
    k: torch.Tensor
    v: torch.Tensor
    k_scale: torch.Tensor
    v_scale: torch.Tensor

    @classmethod
    def empty(cls, batch: int, capacity: int, n_kv_heads: int, head_dim: int, device=0) -> "QuantizedKV":
        """A cache of zeros."""
        dev = torch.device("cuda", device) if isinstance(device, int) else torch.device(device)
        codes = torch.zeros((2, batch, n_kv_heads, capacity, head_dim), dtype=torch.uint8, device=dev)
        scales = torch.zeros((2, batch, n_kv_heads, capacity), dtype=torch.float32, device=dev)
        k, v = codes.view(torch.float8_e4m3fn)
        return cls(k, v, scales[0], scales[1])


def _misfit(t, what: str, device: int, dtype, shape):
    """Raises what is wrong with a tensor that is not on the GPU, or not of the type or shape."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{what}: a torch tensor is expected")
    if t.get_device() != device:
        raise ValueError(f"{what}: not on the handle's GPU (cuda:{device})")
    if t.dtype != dtype:
        raise TypeError(f"{what}: dtype {t.dtype} is not taken here")
    raise ValueError(f"{what}: shape {tuple(t.shape)}, expected {tuple(shape)}")


class CacheOps:
    """Handle of the operators on one GPU."""

    def __init__(self, device: int = 0):
        self.device = int(device)
        self.h = L.rtv_ops_create(self.device)
        self._torch_device = torch.device("cuda", self.device)
        self._need = {}      # workspace bytes by shape

    # ------------------------------------------------------------------
    def _on(self, stream):
        return on_stream(stream, self.device)

    def _elsewhere(self, stream, call, *args):
        """The call on that stream, whose queued work keeps the memory of what it is given."""
        with self._on(stream):
            result = call(*args)
            used = torch.cuda.current_stream(self.device)
            for a in args:
                for t in a if isinstance(a, (tuple, list)) else (a,):
                    if isinstance(t, torch.Tensor):
                        t.record_stream(used)
        return result

    def _stream(self) -> int:
        return torch._C._cuda_getCurrentRawStream(self.device)   # torch.cuda.current_stream without its object

    def _rows(self, k, v, what: str, shared: bool = False) -> rtv_kv:
        """Keys and values [B][N][Hkv][D] (shared: [N][Hkv][D]) of one type, shape and strides."""
        dtype = getattr(k, "dtype", None)
        code = _CODES.get(dtype)
        if code is None or k.get_device() != self.device:
            if isinstance(k, torch.Tensor) and code is not None:
                raise ValueError(f"{what}: not on the handle's GPU (cuda:{self.device})")
            raise TypeError(f"{what}: fp32 or bf16 tensors are expected")
        shape, stride = k.shape, k.stride()
        if len(shape) != (3 if shared else 4):
            raise ValueError(f"{what}: {'[N][heads][D]' if shared else '[B][N][heads][D]'} expected")
        if getattr(v, "dtype", None) is not dtype or v.get_device() != self.device or v.shape != shape:
            _misfit(v, what, self.device, dtype, shape)
        if v.stride() != stride:
            raise ValueError(f"{what}: keys and values differ in strides")
        if stride[-1] != 1 and shape[-1] > 1:
            raise ValueError(f"{what}: the last index must be dense")
        if shared:
            n, h, d = shape
            return rtv_kv(k.data_ptr(), v.data_ptr(), None, None, code, 1, n, h, d, 0, stride[0], stride[1])
        b, n, h, d = shape
        return rtv_kv(k.data_ptr(), v.data_ptr(), None, None, code, b, n, h, d, stride[0], stride[1], stride[2])

    def _cache(self, c: QuantizedKV, what: str) -> rtv_kv:
        k, v, ks, vs = c
        shape, stride, fshape, fstride = k.shape, k.stride(), ks.shape, ks.stride()
        if len(shape) != 4:
            raise ValueError(f"{what}: codes [B][heads][capacity][D] expected")
        for t in (k, v):
            if t.dtype is not torch.float8_e4m3fn or t.get_device() != self.device or t.shape != shape:
                _misfit(t, what, self.device, torch.float8_e4m3fn, shape)
        for t in (ks, vs):
            if t.dtype is not torch.float32 or t.get_device() != self.device or t.shape != shape[:3]:
                _misfit(t, what, self.device, torch.float32, shape[:3])
        if v.stride() != stride or vs.stride() != fstride:
            raise ValueError(f"{what}: keys and values differ in strides")
        b, h, n, d = shape
        if stride[3] != 1 and d > 1:
            raise ValueError(f"{what}: the last index must be dense")
        return rtv_kv(k.data_ptr(), v.data_ptr(), ks.data_ptr(), vs.data_ptr(), RTV_FP8_E4M3, b, n, h, d, stride[0],
                      stride[2], stride[1], fstride[0], fstride[2], fstride[1])

    def _ints(self, t, what: str, batch: int) -> Optional[int]:
        if t is None:
            return None
        if not isinstance(t, torch.Tensor) or t.dtype is not torch.int32 or t.get_device() != self.device or \
                t.shape != (batch,):
            _misfit(t, what, self.device, torch.int32, (batch,))
        if batch > 1 and t.stride(0) != 1:
            raise ValueError(f"{what}: must be contiguous")
        return t.data_ptr()

    def _bools(self, t, what: str, shape) -> Optional[int]:
        if t is None:
            return None
        if not isinstance(t, torch.Tensor) or t.dtype is not torch.bool or t.get_device() != self.device or \
                t.shape != shape:
            _misfit(t, what, self.device, torch.bool, shape)
        if t.stride(-1) != 1 and shape[-1] > 1:
            raise ValueError(f"{what}: the last index must be dense")
        return t.data_ptr()

    def _queries(self, q, out, lse, scale):
        code = _CODES.get(getattr(q, "dtype", None))
        if code is None or q.get_device() != self.device:
            if isinstance(q, torch.Tensor) and code is not None:
                raise ValueError(f"q: not on the handle's GPU (cuda:{self.device})")
            raise TypeError("q: an fp32 or bf16 tensor is expected")
        shape, s = q.shape, q.stride()
        if len(shape) != 4:
            raise ValueError("q: [B][T][heads][D] expected")
        b, t, h, d = shape
        if out is None:
            out = torch.empty_like(q, memory_format=torch.contiguous_format)
            o = (t * h * d, h * d, d, 1)
        else:
            if not isinstance(out, torch.Tensor) or out.dtype is not q.dtype or out.get_device() != self.device or \
                    out.shape != shape:
                _misfit(out, "out", self.device, q.dtype, shape)
            o = out.stride()
        if lse is True:
            lse = torch.empty((b, t, h), dtype=torch.float32, device=self._torch_device)
        elif lse is False:
            lse = None
        elif not isinstance(lse, torch.Tensor) or lse.dtype is not torch.float32 or \
                lse.get_device() != self.device or lse.shape != (b, t, h):
            _misfit(lse, "lse", self.device, torch.float32, (b, t, h))
        elif not lse.is_contiguous():
            raise ValueError("lse: must be contiguous")
        if (s[3] != 1 or o[3] != 1) and d > 1:
            raise ValueError("q, out: the last index must be dense")
        desc = rtv_queries(q.data_ptr(), out.data_ptr(), None if lse is None else lse.data_ptr(), code, b, t, h, d,
                           s[0], s[1], s[2], o[0], o[1], o[2], d ** -0.5 if scale is None else scale)
        return desc, out, lse

    def _workspace(self, key, size, *args):
        """(address, bytes, owner) of a workspace for a call of these shapes;
        torch's allocator gives whole 512-byte blocks."""
        need = self._need.get(key)
        if need is None:
            if len(self._need) > 4096:
                self._need.clear()
            need = self._need[key] = size(self.h, *args)
        if not need:
            return None, 0, None
        w = torch.empty(need, dtype=torch.uint8, device=self._torch_device)
        return w.data_ptr(), need, w

    # ------------------------------------------------------------------
    def write(self, cache: QuantizedKV, k, v, start=None, count=None, stream=None):
        """Quantise tokens k, v [B][N][Hkv][D] into the cache: token t of
        element b goes to place start + t.  start: None (0), a number, or an
        int32 tensor [B]; count: int32 tensor [B] of the tokens that are real
        (the rest is not written), or None."""
        if stream is not None:
            return self._elsewhere(stream, self.write, cache, k, v, start, count)
        src, dst = self._rows(k, v, "k, v"), self._cache(cache, "cache")
        first, at = 0, None
        if isinstance(start, torch.Tensor):
            at = self._ints(start, "start", src.batch)
        elif start is not None:
            first = _place(start, "start")
        L.rtv_kv_write(self.h, src, dst, at, first, self._ints(count, "count", src.batch), self._stream())

    def read(self, cache: QuantizedKV, n: Optional[int] = None, first: int = 0, lens=None, dtype="bf16", out=None,
             stream=None):
        """Keys and values [B][n][Hkv][D] of cache tokens first .. first+n-1
        (n None: to the end) in dtype ("f32" or "bf16"), or into out = (k, v).
        Tokens at or past lens[b] (int32 [B]) read as zeros."""
        if stream is not None:
            return self._elsewhere(stream, self.read, cache, n, first, lens, dtype, out)
        src, first = self._cache(cache, "cache"), _place(first, "first")
        if out is None:
            n = src.n_tokens - first if n is None else n
            if n < 0 or dtype not in _TYPES:
                raise ValueError('read: n must not be negative and dtype "f32" or "bf16"')
            kv = torch.empty((2, src.batch, n, src.n_heads, src.head_dim), dtype=_TYPES[dtype],
                             device=self._torch_device)
            out = (kv[0], kv[1])
        elif n is not None and n != out[0].shape[1]:
            raise ValueError(f"read: n is {n}, out holds {out[0].shape[1]} tokens")
        dst = self._rows(out[0], out[1], "out")
        L.rtv_kv_read(self.h, src, first, self._ints(lens, "lens", src.batch), dst, self._stream())
        return out

    def cross_attention(self, q, kv, lens=None, mask=None, scale=None, out=None, lse=False, stream=None):
        """Attention of q [B][T][Hq][D] to kv, (k, v) [B][N][Hkv][D] or a
        QuantizedKV: keys t < lens[b] (int32 [B]) with mask[b][t] (bool
        [B][N]).  scale None: D ** -0.5.  Returns out, or (out, lse) with lse
        True or a tensor [B][T][Hq]."""
        if stream is not None:
            return self._elsewhere(stream, self.cross_attention, q, kv, lens, mask, scale, out, lse)
        desc, out, sums = self._queries(q, out, lse, scale)
        keys = self._cache(kv, "kv") if isinstance(kv, QuantizedKV) else self._rows(kv[0], kv[1], "kv")
        mp = self._bools(mask, "mask", (keys.batch, keys.n_tokens))
        lp = self._ints(lens, "lens", keys.batch)
        wp, wb, keep = self._workspace((q.shape, desc.dtype, keys.dtype, keys.batch, keys.n_tokens, keys.n_heads,
                                        keys.head_dim), L.rtv_cross_attention_workspace, desc, keys)
        L.rtv_cross_attention(self.h, desc, keys, lp, mp, 0 if mp is None else mask.stride(0), wp, wb, self._stream())
        return out if lse is False else (out, sums)

    def shared_attention(self, q, prefix, own=None, prefix_mask=None, own_lens=None, scale=None, out=None, lse=False,
                         stream=None):
        """Attention of q [B][T][Hq][D] to one shared prefix, (k, v)
        [N][Hkv][D] or a QuantizedKV of batch 1, with prefix_mask (bool [N]),
        and to each element's own = (k, v) [B][M][Hkv][D], keys t <
        own_lens[b] (int32 [B]).  Otherwise as cross_attention."""
        if own is None and own_lens is not None:
            raise ValueError("own_lens without own keys")
        if stream is not None:
            return self._elsewhere(stream, self.shared_attention, q, prefix, own, prefix_mask, own_lens, scale, out,
                                   lse)
        desc, out, sums = self._queries(q, out, lse, scale)
        pre = self._cache(prefix, "prefix") if isinstance(prefix, QuantizedKV) else \
            self._rows(prefix[0], prefix[1], "prefix", shared=True)
        mine, key = None, None
        if own is not None:
            mine = self._rows(own[0], own[1], "own")
            key = (mine.dtype, mine.batch, mine.n_tokens, mine.n_heads, mine.head_dim)
        mp = self._bools(prefix_mask, "prefix_mask", (pre.n_tokens,))
        lp = self._ints(own_lens, "own_lens", desc.batch)
        wp, wb, keep = self._workspace((q.shape, desc.dtype, pre.dtype, pre.batch, pre.n_tokens, pre.n_heads,
                                        pre.head_dim, key), L.rtv_shared_attention_workspace, desc, pre, mine)
        L.rtv_shared_attention(self.h, desc, pre, mp, mine, lp, wp, wb, self._stream())
        return out if lse is False else (out, sums)

    # ------------------------------------------------------------------
    def status(self):
        return L.rtv_ops_device_status(self.h)

    def close(self):
        if self.h:
            L.rtv_ops_destroy(self.h)
            self.h = None

    def __del__(self):  # pragma: no cover
        try:
            self.close()
        except Exception:
            pass
