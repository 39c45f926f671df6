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
were made inside ``torch.cuda.stream(stream)``.
"""

from __future__ import annotations

from contextlib import nullcontext
from typing import NamedTuple, Optional

import torch

from . import _lib as L
from ._lib import RTV_BF16, RTV_F32, RTV_FP8_E4M3, rtv_kv, rtv_queries

_CODES = {torch.float32: RTV_F32, torch.bfloat16: RTV_BF16}
_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


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


def _fits(t, what: str, device: int, dtype, shape=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{what}: a torch tensor is expected")
    if t.get_device() != device:
        raise ValueError(f"{what}: not on the handle's GPU (cuda:{device})")
    if dtype is not None and t.dtype not in (dtype if isinstance(dtype, tuple) else (dtype,)):
        raise TypeError(f"{what}: dtype {t.dtype} is not taken here")
    if shape is not None and tuple(t.shape) != shape:
        raise ValueError(f"{what}: shape {tuple(t.shape)}, expected {shape}")


class CacheOps:
    """Handle of the operators on one GPU."""

    def __init__(self, device: int = 0):
        self.device = int(device)
        self.h = L.rtv_ops_create(self.device)
        self._torch_device = torch.device("cuda", self.device)

    # ------------------------------------------------------------------
    def _on(self, stream):
        """Context in which torch allocates for, and names, the call's stream."""
        if stream is None:
            return nullcontext()
        if not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(int(stream), device=self._torch_device) if stream else \
                torch.cuda.default_stream(self._torch_device)
        return torch.cuda.stream(stream)

    def _stream(self) -> int:
        return torch.cuda.current_stream(self._torch_device).cuda_stream

    def _rows(self, k, v, what: str) -> rtv_kv:
        """Keys and values [B][N][Hkv][D] of one type, shape and strides."""
        if k.dim() != 4:
            raise ValueError(f"{what}: [B][N][heads][D] expected")
        _fits(k, what, self.device, (torch.float32, torch.bfloat16))
        b, n, h, d = k.shape
        _fits(v, what, self.device, k.dtype, (b, n, h, d))
        sb, st, sh, sd = k.stride()
        if v.stride() != k.stride():
            raise ValueError(f"{what}: keys and values differ in strides")
        if sd != 1 and d > 1:
            raise ValueError(f"{what}: the last index must be dense")
        return rtv_kv(k.data_ptr(), v.data_ptr(), None, None, _CODES[k.dtype], b, n, h, d, sb, st, sh)

    def _cache(self, c: QuantizedKV, what: str) -> rtv_kv:
        k, v, ks, vs = c
        if k.dim() != 4:
            raise ValueError(f"{what}: codes [B][heads][capacity][D] expected")
        _fits(k, what, self.device, torch.float8_e4m3fn)
        b, h, n, d = k.shape
        _fits(v, what, self.device, torch.float8_e4m3fn, (b, h, n, d))
        _fits(ks, what, self.device, torch.float32, (b, h, n))
        _fits(vs, what, self.device, torch.float32, (b, h, n))
        sb, sh, st, sd = k.stride()
        fb, fh, ft = ks.stride()
        if v.stride() != k.stride() or vs.stride() != ks.stride():
            raise ValueError(f"{what}: keys and values differ in strides")
        if sd != 1 and d > 1:
            raise ValueError(f"{what}: the last index must be dense")
        return rtv_kv(k.data_ptr(), v.data_ptr(), ks.data_ptr(), vs.data_ptr(), RTV_FP8_E4M3, b, n, h, d, sb, st, sh,
                      fb, ft, fh)

    def _ints(self, t, what: str, batch: int) -> Optional[int]:
        if t is None:
            return None
        _fits(t, what, self.device, torch.int32, (batch,))
        if not t.is_contiguous():
            raise ValueError(f"{what}: must be contiguous")
        return t.data_ptr()

    def _queries(self, q, out, lse, scale):
        if not isinstance(q, torch.Tensor) or q.dim() != 4:
            raise ValueError("q: [B][T][heads][D] expected")
        _fits(q, "q", self.device, (torch.float32, torch.bfloat16))
        b, t, h, d = q.shape
        if out is None:
            out = torch.empty((b, t, h, d), dtype=q.dtype, device=self._torch_device)
        else:
            _fits(out, "out", self.device, q.dtype, (b, t, h, d))
        if lse is True:
            lse = torch.empty((b, t, h), dtype=torch.float32, device=self._torch_device)
        elif lse is False:
            lse = None
        if lse is not None:
            _fits(lse, "lse", self.device, torch.float32, (b, t, h))
            if not lse.is_contiguous():
                raise ValueError("lse: must be contiguous")
        s, o = q.stride(), out.stride()
        if (s[3] != 1 or o[3] != 1) and d > 1:
            raise ValueError("q, out: the last index must be dense")
        desc = rtv_queries(q.data_ptr(), out.data_ptr(), None if lse is None else lse.data_ptr(), _CODES[q.dtype], b,
                           t, h, d, s[0], s[1], s[2], o[0], o[1], o[2], d ** -0.5 if scale is None else scale)
        return desc, out, lse

    def _workspace(self, need: int):
        """(address, bytes, owner) of a workspace; torch's allocator gives whole 512-byte blocks."""
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
        src, dst = self._rows(k, v, "k, v"), self._cache(cache, "cache")
        first, at = 0, None
        if isinstance(start, torch.Tensor):
            at = self._ints(start, "start", src.batch)
        elif start is not None:
            first = int(start)
        with self._on(stream):
            L.rtv_kv_write(self.h, src, dst, at, first, self._ints(count, "count", src.batch), self._stream())

    def read(self, cache: QuantizedKV, n: Optional[int] = None, first: int = 0, lens=None, dtype="bf16", out=None,
             stream=None):
        """Keys and values [B][n][Hkv][D] of cache tokens first .. first+n-1
        (n None: to the end) in dtype ("f32" or "bf16"), or into out = (k, v).
        Tokens at or past lens[b] (int32 [B]) read as zeros."""
        src = self._cache(cache, "cache")
        with self._on(stream):
            if out is None:
                n = src.n_tokens - first if n is None else n
                if n < 0 or dtype not in _TYPES:
                    raise ValueError('read: n must not be negative and dtype "f32" or "bf16"')
                kv = torch.empty((2, src.batch, n, src.n_heads, src.head_dim), dtype=_TYPES[dtype],
                                 device=self._torch_device)
                out = (kv[0], kv[1])
            dst = self._rows(out[0], out[1], "out")
            L.rtv_kv_read(self.h, src, first, self._ints(lens, "lens", src.batch), dst, self._stream())
        return out

    def cross_attention(self, q, kv, lens=None, mask=None, scale=None, out=None, lse=False, stream=None):
        """Attention of q [B][T][Hq][D] to kv, (k, v) [B][N][Hkv][D] or a
        QuantizedKV: keys t < lens[b] (int32 [B]) with mask[b][t] (bool
        [B][N]).  scale None: D ** -0.5.  Returns out, or (out, lse) with lse
        True or a tensor [B][T][Hq]."""
        want_lse = lse is not False
        with self._on(stream):
            desc, out, lse = self._queries(q, out, lse, scale)
            keys = self._cache(kv, "kv") if isinstance(kv, QuantizedKV) else self._rows(kv[0], kv[1], "kv")
            mp, ms = None, 0
            if mask is not None:
                _fits(mask, "mask", self.device, torch.bool, (keys.batch, keys.n_tokens))
                ms, dense = mask.stride()
                if dense != 1 and keys.n_tokens > 1:
                    raise ValueError("mask: the last index must be dense")
                mp = mask.data_ptr()
            lp = self._ints(lens, "lens", keys.batch)
            wp, wb, keep = self._workspace(L.rtv_cross_attention_workspace(self.h, desc, keys))
            L.rtv_cross_attention(self.h, desc, keys, lp, mp, ms, wp, wb, self._stream())
        return (out, lse) if want_lse else out

    def shared_attention(self, q, prefix, own=None, prefix_mask=None, own_lens=None, scale=None, out=None, lse=False,
                         stream=None):
        """Attention of q [B][T][Hq][D] to one shared prefix, (k, v)
        [N][Hkv][D] or a QuantizedKV of batch 1, with prefix_mask (bool [N]),
        and to each element's own = (k, v) [B][M][Hkv][D], keys t <
        own_lens[b] (int32 [B]).  Otherwise as cross_attention."""
        want_lse = lse is not False
        if own is None and own_lens is not None:
            raise ValueError("own_lens without own keys")
        with self._on(stream):
            desc, out, lse = self._queries(q, out, lse, scale)
            if isinstance(prefix, QuantizedKV):
                pre = self._cache(prefix, "prefix")
            else:
                pk, pv = prefix
                if pk.dim() != 3:
                    raise ValueError("prefix: [N][heads][D] expected")
                pre = self._rows(pk[None], pv[None], "prefix")
            mine = None if own is None else self._rows(own[0], own[1], "own")
            mp = None
            if prefix_mask is not None:
                _fits(prefix_mask, "prefix_mask", self.device, torch.bool, (pre.n_tokens,))
                if not prefix_mask.is_contiguous():
                    raise ValueError("prefix_mask: must be contiguous")
                mp = prefix_mask.data_ptr()
            lp = self._ints(own_lens, "own_lens", desc.batch)
            wp, wb, keep = self._workspace(L.rtv_shared_attention_workspace(self.h, desc, pre, mine))
            L.rtv_shared_attention(self.h, desc, pre, mp, mine, lp, wp, wb, self._stream())
        return (out, lse) if want_lse else out

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
