"""Operators on a paged KV cache: append rows (with the queries' and keys' norm and rotation), read
rows back, copy pages, and keep count of a pool's pages.

These are the calls around ``BatchDecodePagedKV.run``: a step appends its tokens' K and V, decodes,
and now and then a sequence forks, ends, or the pool is compacted.  Like decode.py, this module
checks shapes and marshals pointers; the work runs in libpkd's CUDA kernels, asynchronously on the
current stream (or ``stream``), and every call can be captured in a CUDA graph.
"""
from __future__ import annotations

import ctypes
import struct
from array import array
from typing import Optional

import numpy as np
import torch

from . import _lib as L
from .decode import (_DTYPE_CODE, CODE_DTYPES, SCALE_DTYPES, current_device, forward_ad, new_output,
                     pool_views, raw_stream, refuse_gradients, weight_views)

_POOL = "4Pq3q3q2Pq5i2fi"  # pkd_paged_pool
_APPEND = struct.Struct("@" + _POOL + "4P8q3P2PPqPqd6i")  # pkd_append_args
_GATHER = struct.Struct("@" + _POOL + "2P4q2PPq2i")  # pkd_gather_args
_EVICT = struct.Struct("@" + _POOL + "P3q4P4i")  # pkd_evict_args
_IO_DTYPES = (torch.float16, torch.bfloat16)


_INT32 = torch.int32


def _index(t, name: str, dev: int, n: Optional[int] = None) -> int:
    """Address of a contiguous int32 tensor on CUDA device `dev` (of n entries)."""
    if not isinstance(t, torch.Tensor) or t.dtype is not _INT32 or t.dim() != 1 or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous 1-D int32 tensor")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, the rows are on cuda:{dev}")
    if n is not None and t.shape[0] != n:
        raise ValueError(f"{name} has {t.shape[0]} entries, expected {n}")
    return t.data_ptr()


def _status(status, dev: int) -> int:
    if status is None:
        return 0
    if status.numel() != 1 or status.element_size() != 4 or status.get_device() != dev:
        raise ValueError(f"status must be one 32-bit integer on cuda:{dev}")
    return status.data_ptr()


def _rows(t, name: str, dtype, dev: int, shape):
    """(address, token stride, head stride) of rows [tokens, heads, head_dim]."""
    if t.shape != shape or t.dtype is not dtype or t.get_device() != dev:
        raise ValueError(f"{name} must be a {dtype} tensor of shape {shape} on cuda:{dev}")
    st0, st1, st2 = t.stride()
    if st2 != 1:
        raise ValueError(f"{name} must have its last axis contiguous")
    # the stride of an axis of one entry is never used; any value will do
    return t.data_ptr(), st0 if shape[0] > 1 else 0, st1 if shape[1] > 1 else 0


def _pool_fields(cache, scales, indptr, indices, kv_layout, k_scale, v_scale, dev, io_dtype):
    """pkd_paged_pool's fields, num_kv_heads and head_dim."""
    if kv_layout != "NHD" and kv_layout != "HND":
        raise ValueError("kv_layout must be 'NHD' or 'HND'")
    first = cache[0] if isinstance(cache, (tuple, list)) else cache
    if first.get_device() != dev:
        raise ValueError(f"paged_kv_cache is on {first.device}, the rows are on cuda:{dev}")
    k, v, (s0, s1, s2), ps, hkv = pool_views(cache, kv_layout)
    shape, kv_dtype = first.shape, first.dtype
    pages, d = shape[0], shape[-1]
    ks = vs = f0 = f1 = f2 = 0
    if scales is not None:
        if kv_dtype not in CODE_DTYPES:
            raise ValueError("kv_block_scales belongs to a 4-bit cache (uint8 or float4_e2m1fn_x2 codes)")
        d *= 2
        sf = scales[0] if isinstance(scales, (tuple, list)) else scales
        ks, vs, (f0, f1, f2), sps, shkv = pool_views(scales, kv_layout, "kv_block_scales")
        if (sf.dtype not in SCALE_DTYPES or sf.get_device() != dev
                or (sf.shape[0], sps, shkv, 16 * sf.shape[-1]) != (pages, ps, hkv, d)):
            raise ValueError("kv_block_scales must be float8_e4m3fn (or uint8) of the cache's shape "
                             "with a last axis of head_dim / 16, on its device")
        code = L.DTYPE_E2M1
    elif kv_dtype is io_dtype or kv_dtype is torch.float8_e4m3fn:
        code = _DTYPE_CODE[kv_dtype]
    else:
        raise ValueError(f"a cache of {kv_dtype} does not go with rows of {io_dtype} (a 4-bit "
                         "cache needs kv_block_scales)")
    ip, ix = _index(indptr, "kv_indptr", dev), _index(indices, "kv_indices", dev)
    return (k, v, ks, vs, pages, s0, s1, s2, f0, f1, f2, ip, ix, indices.shape[0],
            max(0, indptr.shape[0] - 1), code, hkv, d, ps, 1.0 if k_scale is None else float(k_scale),
            1.0 if v_scale is None else float(v_scale), 0), hkv, d


def _launch(call, dev: int, stream, *args) -> None:
    """call(*args, stream) with the tensors' device current and an error raised."""
    if stream is None:
        s = raw_stream(dev)
    elif stream.device.index != dev:
        raise ValueError(f"the stream is on {stream.device}, the tensors are on cuda:{dev}")
    else:
        s = stream.cuda_stream
    if current_device() == dev:
        rc = call(*args, s)
    else:
        with torch.cuda.device(dev):
            rc = call(*args, s)
    if rc:
        L.check(rc)


def append_paged_kv(q: Optional[torch.Tensor], k: Optional[torch.Tensor], v: Optional[torch.Tensor],
                    batch_indices: torch.Tensor, positions: torch.Tensor, paged_kv_cache,
                    kv_indptr: Optional[torch.Tensor], kv_indices: Optional[torch.Tensor],
                    kv_layout: str = "NHD", *, q_weight: Optional[torch.Tensor] = None,
                    k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
                    cos_sin_cache: Optional[torch.Tensor] = None,
                    rope_positions: Optional[torch.Tensor] = None, interleaved: bool = False,
                    kv_block_scales=None, k_scale: Optional[float] = None,
                    v_scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                    status: Optional[torch.Tensor] = None, stream=None) -> Optional[torch.Tensor]:
    """Norm and rotate new queries and keys, and write K and V into their page slots (pkd_append).

    ``q [tokens, num_qo_heads, head_dim]``, ``k`` / ``v [tokens, num_kv_heads, head_dim]``, fp16 or
    bf16, may be views of one projection's output (any token and head stride, head_dim contiguous).
    Row t is token ``positions[t]`` of sequence ``batch_indices[t]`` (device int32); a negative
    batch index marks padding: its rows are not written, and whatever they hold is not used (they may
    be read).  ``kv_indptr [batch + 1]`` and ``kv_indices`` (device int32) are the page table that
    ``BatchDecodePagedKV.plan`` takes.

    Each head of q (k) is divided by its root mean square and multiplied by ``q_weight``
    (``k_weight``, ``[head_dim]``, the rows' type or float32) if that is given.  With
    ``cos_sin_cache`` (float32 ``[positions, rotary_dim]``, cosines then sines, see
    ``make_cos_sin_cache``) the first rotary_dim dims of q and k are rotated in pairs
    (i, i + rotary_dim / 2), or (2i, 2i + 1) if ``interleaved``, at ``rope_positions`` (default:
    ``positions``).

    ``paged_kv_cache`` (5-D, or a (k, v) pair) receives k / k_scale and v / v_scale in the rows' type
    or float8_e4m3fn, rounded once, or as 4-bit codes with ``kv_block_scales`` as
    ``BatchDecodePagedKV.run`` reads them.
    Returns q's rows (``out``, which may be ``q``, but overlap neither other rows of it nor k or v; a
    fresh tensor's padding rows are undefined), or None without q.  ``q`` may be None, or ``k`` and ``v`` with the cache and page table.

    ``status`` (one int32 on the device) receives STATUS_BAD_TOKEN for a row that has no slot in
    its sequence or no entry in ``cos_sin_cache``, STATUS_BAD_PAGE for a page id outside the pool;
    such rows write nothing to the cache.  Two rows of a call must not share a slot."""
    first = q if q is not None else k
    if first is None or (k is None) != (v is None):
        raise ValueError("append needs q, or k and v, or all three")
    if not isinstance(first, torch.Tensor) or first.dim() != 3 or first.dtype not in _IO_DTYPES:
        raise ValueError("q, k and v must be fp16 or bf16 tensors [tokens, heads, head_dim]")
    dev, dtype = first.get_device(), first.dtype
    if dev < 0:
        raise ValueError("q, k and v must be CUDA tensors")
    if (torch.is_grad_enabled()
            and (first.requires_grad or (k is not None and (k.requires_grad or v.requires_grad))
                 or (q_weight is not None and q_weight.requires_grad)
                 or (k_weight is not None and k_weight.requires_grad)
                 or (cos_sin_cache is not None and cos_sin_cache.requires_grad))) or forward_ad._current_level >= 0:
        refuse_gradients("append", q, k, v, q_weight, k_weight, cos_sin_cache)
    n, hq, d = first.shape
    if k is not None:
        pool, hkv, pd = _pool_fields(paged_kv_cache, kv_block_scales, kv_indptr, kv_indices, kv_layout,
                                     k_scale, v_scale, dev, dtype)
        if pd != d:
            raise ValueError(f"the cache's head_dim is {pd}, the rows' is {d}")
        kp, k0, k1 = _rows(k, "k", dtype, dev, (n, hkv, d))
        vp, v0, v1 = _rows(v, "v", dtype, dev, (n, hkv, d))
    else:
        pool = (0,) * 14 + (0, 0, 0, d, 0, 1.0, 1.0, 0)
        kp = k0 = k1 = vp = v0 = v1 = 0
    if q is not None:
        qp, q0, q1 = _rows(q, "q", dtype, dev, (n, hq, d))
        if out is None:
            out = new_output((n, hq, d), q, dtype, stream)
        op, o0, o1 = _rows(out, "out", dtype, dev, (n, hq, d))
    elif out is not None:
        raise ValueError("out without q")
    else:
        hq = qp = q0 = q1 = op = o0 = o1 = 0
    weight_f32 = qw = kw = 0
    if q_weight is not None:
        qw, weight_f32 = _weight(q_weight, "q_weight", dtype, dev, d)
    if k_weight is not None:
        kw, f32 = _weight(k_weight, "k_weight", dtype, dev, d)
        if q_weight is not None and f32 != weight_f32:
            raise ValueError("q_weight and k_weight must have one dtype")
        weight_f32 = f32
    rotary = rows = cs = rp = 0
    if cos_sin_cache is not None:
        c = cos_sin_cache
        if c.dim() != 2 or c.dtype is not torch.float32 or not c.is_contiguous() or c.get_device() != dev:
            raise ValueError(f"cos_sin_cache must be a contiguous float32 [positions, rotary_dim] tensor on cuda:{dev}")
        rows, rotary = c.shape
        cs = c.data_ptr()
        if rope_positions is not None:
            rp = _index(rope_positions, "rope_positions", dev, n)
    elif rope_positions is not None:
        raise ValueError("rope_positions without cos_sin_cache")
    args = _APPEND.pack(
        *pool, qp, kp, vp, op, q0, q1, k0, k1, v0, v1, o0, o1,
        _index(batch_indices, "batch_indices", dev, n), _index(positions, "positions", dev, n),
        rp, qw, kw, cs, rows, _status(status, dev), n,
        eps, hq, _DTYPE_CODE[dtype], weight_f32, rotary, 1 if interleaved else 0, 0)
    _launch(L.lib().pkd_append, dev, stream, args)
    return out


def _weight(w, name: str, dtype, dev: int, d: int):
    """(address, whether it is float32) of a norm's weights."""
    f32 = w.dtype is not dtype
    if f32 and w.dtype is not torch.float32 or w.shape != (d,) or w.get_device() != dev or not w.is_contiguous():
        raise ValueError(f"{name} must be a contiguous [{d}] tensor of {dtype} or float32 on cuda:{dev}")
    return w.data_ptr(), 1 if f32 else 0


def gather_paged_kv(batch_indices: torch.Tensor, positions: torch.Tensor, paged_kv_cache,
                    kv_indptr: torch.Tensor, kv_indices: torch.Tensor, kv_layout: str = "NHD", *,
                    kv_block_scales=None, k_scale: Optional[float] = None,
                    v_scale: Optional[float] = None, out_dtype=None, out=None,
                    status: Optional[torch.Tensor] = None, stream=None):
    """Read token rows of a paged cache back (pkd_gather): returns ``(k, v)``, each
    ``[tokens, num_kv_heads, head_dim]`` in ``out_dtype`` (default: the cache's type if it has 16
    bits, else bf16), the stored values times k_scale / v_scale, rounded once.

    Row t is token ``positions[t]`` of sequence ``batch_indices[t]``; a row with a negative batch
    index (padding), or without a slot (``status``, as in ``append_paged_kv``), is left as it was
    in ``out = (k, v)``, and undefined in fresh tensors.  The cache arguments are those of
    ``append_paged_kv``.  For prefill over a cached prefix, and for moving a cache elsewhere."""
    first = paged_kv_cache[0] if isinstance(paged_kv_cache, (tuple, list)) else paged_kv_cache
    dev = first.get_device()
    if dev < 0:
        raise ValueError("the cache must be a CUDA tensor")
    second = None if first is paged_kv_cache else paged_kv_cache[1]
    if (torch.is_grad_enabled() and (first.requires_grad or (second is not None and second.requires_grad))
            ) or forward_ad._current_level >= 0:
        refuse_gradients("gather", first, second)
    if out is not None:
        k, v = out
        if out_dtype is not None and out_dtype != k.dtype:
            raise ValueError(f"out is {k.dtype}, out_dtype is {out_dtype}")
        out_dtype = k.dtype
    elif out_dtype is None:
        out_dtype = first.dtype if first.dtype in _IO_DTYPES else torch.bfloat16
    if out_dtype not in _IO_DTYPES:
        raise ValueError("out_dtype must be fp16 or bf16")
    pool, hkv, d = _pool_fields(paged_kv_cache, kv_block_scales, kv_indptr, kv_indices, kv_layout,
                                k_scale, v_scale, dev, out_dtype)
    n = batch_indices.shape[0]
    if out is None:
        k, v = new_output((n, hkv, d), first, out_dtype, stream), new_output((n, hkv, d), first, out_dtype, stream)
    kp, k0, k1 = _rows(k, "k out", out_dtype, dev, (n, hkv, d))
    vp, v0, v1 = _rows(v, "v out", out_dtype, dev, (n, hkv, d))
    args = _GATHER.pack(*pool, kp, vp, k0, k1, v0, v1, _index(batch_indices, "batch_indices", dev),
                        _index(positions, "positions", dev, n), _status(status, dev), n,
                        _DTYPE_CODE[out_dtype], 0)
    _launch(L.lib().pkd_gather, dev, stream, args)
    return k, v


def evict_paged_kv(paged_kv_cache, key_weights: torch.Tensor, kv_lens: torch.Tensor, kv_indptr: torch.Tensor,
                   kv_indices: torch.Tensor, budget: int, kv_layout: str = "NHD", *, num_sink_tokens: int = 0,
                   num_recent: int = 0, kv_block_scales=None, return_kept: bool = False,
                   status: Optional[torch.Tensor] = None, stream=None) -> Optional[torch.Tensor]:
    """Cut every sequence back to ``budget`` tokens, in place (pkd_evict): each kv head keeps its first
    ``num_sink_tokens``, its newest ``num_recent`` and the tokens with the largest ``key_weights``
    (float32 ``[pages, num_kv_heads, page_size]``, what ``BatchDecodePagedKV.run`` adds to).
    ``kv_lens`` (device int32 ``[batch]``) are the sequences' lengths, which the call reads and leaves as
    they are; the new ones are ``min(kv_lens, budget)``, and the pages behind may be freed
    (``PageAllocator.free``).

    The first tokens stay in place, the newest lie at the end in order, the others in any slots
    between (those that can stay do), so append later keys with ``rope_positions`` of their own and
    decode without window, ALIBI or ROPE_LLAMA.  Weights move with their tokens, and slots without a
    token have weight 0 afterwards.  ``return_kept=True`` returns int32 ``[batch, num_kv_heads,
    budget]``: the slot whose token each slot now holds, -1 behind the end.

    ``status`` receives STATUS_BAD_TOKEN for a sequence longer than its pages (or of negative length),
    STATUS_BAD_PAGE for one with a page id outside the pool; it is left alone.  The sequences must
    own their pages alone."""
    first = paged_kv_cache[0] if isinstance(paged_kv_cache, (tuple, list)) else paged_kv_cache
    dev = first.get_device()
    if dev < 0:
        raise ValueError("the cache must be a CUDA tensor")
    if not isinstance(key_weights, torch.Tensor):
        raise ValueError("key_weights must be a CUDA float32 tensor")
    second = None if first is paged_kv_cache else paged_kv_cache[1]
    if (torch.is_grad_enabled() and (first.requires_grad or key_weights.requires_grad
                                     or (second is not None and second.requires_grad))
            ) or forward_ad._current_level >= 0:
        refuse_gradients("evict", first, second, key_weights)
    io = first.dtype if first.dtype in _IO_DTYPES else torch.bfloat16
    pool, hkv, _ = _pool_fields(paged_kv_cache, kv_block_scales, kv_indptr, kv_indices, kv_layout, None, None, dev, io)
    batch, ps = pool[14], pool[18]
    budget, sinks, recent = int(budget), int(num_sink_tokens), int(num_recent)
    if not (1 <= budget <= 2 ** 30 and 0 <= sinks and 0 <= recent and sinks + recent <= budget):
        raise ValueError("budget must lie in [1, 2^30], num_sink_tokens and num_recent must be >= 0 and fit "
                         "it together")
    lens = _index(kv_lens, "kv_lens", dev, batch)
    weights = weight_views(key_weights, first.shape[0], hkv, ps, dev)
    heads, middle = batch * hkv, budget - sinks - recent
    kept = new_output((batch, hkv, budget), first, _INT32, stream) if return_kept else None
    moves = new_output((3 * heads * middle,), first, _INT32, stream)
    args = _EVICT.pack(*pool, *weights, lens, 0 if kept is None else kept.data_ptr(), moves.data_ptr(),
                       _status(status, dev), budget, sinks, recent, 0)
    _launch(L.lib().pkd_evict, dev, stream, args)
    return kept


def _page_ids(x, name: str) -> np.ndarray:
    """Host page ids as contiguous int32, refused where a value would change on the way."""
    a = x.detach().cpu().numpy() if isinstance(x, torch.Tensor) else np.asarray(x)
    if a.dtype != np.int32 and a.size:
        if a.dtype.kind not in "iu" or a.min() < -2 ** 31 or a.max() >= 2 ** 31:
            raise ValueError(f"{name} must be 32-bit integers")
    return np.ascontiguousarray(a, dtype=np.int32)


def _host_ids(x, name: str):
    """(address, count, what to keep alive) of host page ids."""
    if isinstance(x, torch.Tensor) and x.dtype is _INT32 and x.device.type == "cpu" and x.is_contiguous():
        if x.dim() != 1:
            raise ValueError(f"{name} must be a list of page ids")
        return x.data_ptr(), x.shape[0], x
    a = _page_ids(x, name)
    if a.ndim != 1:
        raise ValueError(f"{name} must be a list of page ids")
    return a.ctypes.data, a.shape[0], a


def copy_pages(pools, src_pages, dst_pages, stream=None) -> None:
    """Copy pages ``dst_pages[i] <- src_pages[i]`` in every tensor of ``pools`` (pkd_copy_pages):
    one launch for all layers' pools and scales.  Every pool has its pages on axis 0, the same
    number of them, each page one contiguous block.  The ids are host integers (a list, a numpy
    array or a CPU tensor); a destination may appear once and may be no source."""
    if isinstance(pools, torch.Tensor):
        pools = (pools,)
    sp, n, keep_src = _host_ids(src_pages, "src_pages")
    dp, n_dst, keep_dst = _host_ids(dst_pages, "dst_pages")
    if n != n_dst:
        raise ValueError("src_pages and dst_pages must be lists of one length")
    if not len(pools):
        return
    try:
        dev, pages = pools[0].get_device(), pools[0].shape[0]
        bases, strides, sizes = [], [], []
        for t in pools:
            if t.get_device() != dev or dev < 0 or t.shape[0] != pages:
                raise ValueError(f"every pool must hold {pages} pages on axis 0, on one CUDA device")
            if t.is_contiguous():
                page = stride = t.nbytes // (pages or 1)
            else:
                if pages > 0 and not t[0].is_contiguous():
                    raise ValueError("a page of a pool must be one contiguous block")
                page = t.nbytes // (pages or 1)
                stride = t.stride(0) * t.element_size() if pages > 1 else page
            bases.append(t.data_ptr())
            strides.append(stride)
            sizes.append(page)
    except IndexError:
        raise ValueError("every pool must have its pages on axis 0") from None
    bases, strides, sizes = array("q", bases), array("q", strides), array("q", sizes)
    _launch(L.lib().pkd_copy_pages, dev, stream, bases.buffer_info()[0], strides.buffer_info()[0],
            sizes.buffer_info()[0], len(sizes), pages, sp, dp, n)


def make_cos_sin_cache(max_position: int, rotary_dim: int, rope_theta: float = 1e4,
                       rope_scale: float = 1.0, device="cuda") -> torch.Tensor:
    """The table ``append_paged_kv`` rotates by: float32 ``[max_position, rotary_dim]``, cosines of
    the angles p / rope_scale * rope_theta^(-2i / rotary_dim) in the first half of a row, their
    sines in the second (the angles of plan()'s ROPE_LLAMA), computed in 64 bits."""
    if rotary_dim <= 0 or rotary_dim % 16 != 0 or max_position < 0:
        raise ValueError("rotary_dim must be a positive multiple of 16 and max_position >= 0")
    rate = rope_theta ** (-np.arange(0, rotary_dim, 2, dtype=np.float64) / rotary_dim) / rope_scale
    angle = np.arange(max_position, dtype=np.float64)[:, None] * rate
    return torch.from_numpy(np.concatenate([np.cos(angle), np.sin(angle)], axis=1)
                            .astype(np.float32)).to(device)


class PageAllocator:
    """Which pages of a pool are free, and how many sequences share each (pkd_pages_*): host
    bookkeeping for growing, forking and ending sequences and for compacting a pool.  Page ids are
    numpy int32 arrays; free pages are handed out lowest id first.  One thread at a time."""

    def __init__(self, num_pages: int):
        h = ctypes.c_void_p()
        if num_pages >= 2 ** 31:  # (ctypes would take it modulo 2^64)
            raise ValueError("num_pages must lie in [0, 2^31)")
        L.check(L.lib().pkd_pages_create(ctypes.byref(h), int(num_pages)))
        self._h, self.num_pages = h, int(num_pages)

    def __del__(self):
        h = getattr(self, "_h", None)
        if h is not None and h.value:
            try:
                L.lib().pkd_pages_destroy(h)
            except Exception:
                pass
            self._h = None

    @property
    def num_free(self) -> int:
        n = ctypes.c_int64()
        L.check(L.lib().pkd_pages_count(self._h, ctypes.byref(n), None))
        return n.value

    def uses(self) -> np.ndarray:
        """How many sequences use each page."""
        u = np.zeros(self.num_pages, dtype=np.int32)
        L.check(L.lib().pkd_pages_count(self._h, None, u.ctypes.data))
        return u

    def alloc(self, n: int) -> np.ndarray:
        """n free pages; PkdError, and nothing taken, if fewer are free."""
        if n < 0 or n > self.num_pages:
            raise ValueError(f"n must lie in [0, {self.num_pages}]")
        out = np.empty(n, dtype=np.int32)
        L.check(L.lib().pkd_pages_alloc(self._h, n, out.ctypes.data))
        return out

    def free(self, pages) -> None:
        """One use less of each page; PkdError, and nothing changed, if one is not in use."""
        p = _page_ids(pages, "pages")
        L.check(L.lib().pkd_pages_free(self._h, p.ctypes.data, p.size))

    def fork(self, pages, kv_len: int, page_size: int):
        """A second sequence with the first kv_len tokens of one that owns ``pages``: returns
        ``(its pages, src, dst)``.  Full pages are shared; a partly filled last page gets a page of
        its own, and src / dst (arrays of one id, else empty) is the copy to make with
        ``copy_pages`` before either sequence appends."""
        p = _page_ids(pages, "pages")
        if not 0 <= kv_len < 2 ** 63 or not 1 <= page_size < 2 ** 31:  # (ctypes would cut them to size)
            raise ValueError("kv_len must lie in [0, 2^63) and page_size in [1, 2^31)")
        out = np.empty(-(-kv_len // page_size) if kv_len <= p.size * page_size else 0, dtype=np.int32)
        s, d = ctypes.c_int32(), ctypes.c_int32()
        L.check(L.lib().pkd_pages_fork(self._h, p.ctypes.data, p.size, kv_len, page_size,
                                       out.ctypes.data, ctypes.byref(s), ctypes.byref(d)))
        ids = [x.value for x in (s, d) if x.value >= 0]
        return out, np.array(ids[:1], dtype=np.int32), np.array(ids[1:], dtype=np.int32)

    def compact(self):
        """Move the pages in use to the lowest ids: returns ``(src, dst, remap)``.  Copy the pages
        (``copy_pages``), then replace every page table's ids by ``remap[ids]``."""
        src, dst, remap = (np.empty(self.num_pages, dtype=np.int32) for _ in range(3))
        n = ctypes.c_int64()
        L.check(L.lib().pkd_pages_compact(self._h, src.ctypes.data, dst.ctypes.data, ctypes.byref(n),
                                          remap.ctypes.data))
        return src[:n.value].copy(), dst[:n.value].copy(), remap
