"""The paged key/value cache of a speculative decoder and the operators on it.

    cache = PagedCache(n_layers, n_pages, page_size, n_q_heads, n_kv_heads, head_dim)
    seq = cache.new_sequence()
    cache.reserve([seq], T)                  # pages for T more rows
    table, lens = cache.tables([seq])
    out, lse = cache.attend(layer, q, k, v, table, lens, mask=mask)
    accept, path = verify_sample(target, draft, tokens, u, noise, parents=parents)
    lens = cache.commit(table, lens, path, accept)
    cache.advance([seq], accepted)           # once the host knows the counts
    other = cache.fork(seq)

The arithmetic runs in libqmm.so's kernels (qmm_tree_attention,
qmm_cache_commit, qmm_cache_copy, qmm_verify_sample of include/qmm.h).  What
stays on the host is bookkeeping: which pages are free, which sequence holds
which page, and how many sequences share one.
"""
from __future__ import annotations

import ctypes
import functools
import struct

from ._lib import (QMM_DT_BF16, QMM_DT_F16, QMM_DT_F32, QMM_ERR_DEVICE, QMM_OK, QMM_TREE_MAX_T, QmmError, load, qmm_attn_args,
                   qmm_cache_desc, qmm_sample_args)


# The argument structs of the C calls, packed in one go: filling a ctypes
# structure field by field costs more than a small kernel.
_ATTN = struct.Struct("@IiiiPPPP12qPPqifPPPq")
_SAMPLE = struct.Struct("@IIiiqPqqPqqPPPPPPPPPq")
assert _ATTN.size == ctypes.sizeof(qmm_attn_args) and _SAMPLE.size == ctypes.sizeof(qmm_sample_args)
_raw_stream = None
_CODES = {}


def _stream_ptr(stream, device_index) -> int:
    """The address of `stream`, or of the device's current stream."""
    global _raw_stream
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is None:
        import torch
        _raw_stream = torch._C._cuda_getCurrentRawStream
    return _raw_stream(device_index)


def _check(func: str, rc: int):
    if rc != QMM_OK:
        raise QmmError(func, rc)


def _dtype(dtype):
    if not _CODES:
        import torch
        _CODES.update({torch.bfloat16: QMM_DT_BF16, torch.float16: QMM_DT_F16, torch.float32: QMM_DT_F32})
    if dtype not in _CODES:
        raise TypeError(f"dtype must be bfloat16, float16 or float32, not {dtype}")
    return _CODES[dtype]


def _refuse(name, t, dtype, shape, device):
    if not t.is_cuda or t.dtype != dtype:
        raise TypeError(f"{name} must be a CUDA tensor of {dtype}, not {t.dtype} on {t.device}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {shape}, not {tuple(t.shape)}")
    raise ValueError(f"{name} must be on cuda:{device}, not {t.device}")


def _flat(name, t, dtype, shape, device):
    """Refuses a tensor that is not on that GPU, not contiguous, or of another type or shape."""
    if t.shape != shape or t.dtype is not dtype or t.get_device() != device:
        _refuse(name, t, dtype, shape, device)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _strided(name, t, dtype, shape, device):
    """The same for one whose last dimension alone has to be contiguous."""
    if t.shape != shape or t.dtype is not dtype or t.get_device() != device:
        _refuse(name, t, dtype, shape, device)
    if t.stride(-1) != 1 and t.shape[-1] > 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")


def _rows(name, t):
    """Refuses a tensor whose last dimension is not contiguous."""
    if t.stride(-1) != 1 and t.shape[-1] > 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")


# ------------------------------------------------------------------ raw C names
def qmm_cache_create(dtype, n_layers, n_pages, page_size, n_q_heads, n_kv_heads, head_dim, max_batch,
                     k_pool, v_pool, stream=None) -> int:
    """A handle over the two pools (CUDA tensors, which must outlive it)."""
    d = qmm_cache_desc(ctypes.sizeof(qmm_cache_desc), dtype, n_layers, page_size, n_q_heads, n_kv_heads, head_dim,
                       max_batch, n_pages, k_pool.data_ptr(), v_pool.data_ptr())
    h = ctypes.c_void_p()
    _check("qmm_cache_create", load().qmm_cache_create(ctypes.byref(h), ctypes.byref(d),
                                                       _stream_ptr(stream, k_pool.device.index)))
    return h.value


def qmm_cache_destroy(h) -> None:
    _check("qmm_cache_destroy", load().qmm_cache_destroy(h))


def qmm_cache_sync_status(h, stream=None) -> int:
    import torch
    return load().qmm_cache_sync_status(h, _stream_ptr(stream, torch.cuda.current_device()))


def qmm_tree_attention(h, layer, q, k_new, v_new, page_table, lens, out, lse=None, mask=None, n_tokens=None,
                       scale=None, stream=None) -> None:
    """q, out CUDA [B, T, Hq, D]; k_new, v_new [B, T, Hkv, D]; page_table int32
    [B, pages]; lens, n_tokens int32 [B]; mask int64 [B, T]; lse fp32 [B, T, Hq]
    or None; asynchronous."""
    _tree_attention(h, layer, q, k_new, v_new, page_table, lens, out, lse, mask, n_tokens, scale, stream, q.stride(),
                    k_new.stride(), v_new.stride(), out.stride(), page_table.stride(0))


def _tree_attention(h, layer, q, k, v, table, lens, out, lse, mask, n_tokens, scale, stream, qs, ks, vs, os, ld_table):
    B, T, _, D = q.shape
    rc = load().qmm_tree_attention(h, _ATTN.pack(
        _ATTN.size, layer, B, T, q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
        qs[0], qs[1], qs[2], ks[0], ks[1], ks[2], vs[0], vs[1], vs[2], os[0], os[1], os[2],
        0 if lse is None else lse.data_ptr(), table.data_ptr(), ld_table, table.shape[1],
        D ** -0.5 if scale is None else scale, lens.data_ptr(), 0 if n_tokens is None else n_tokens.data_ptr(),
        0 if mask is None else mask.data_ptr(), 0 if mask is None else mask.stride(0)),
        _stream_ptr(stream, q.device.index))
    if rc:
        _check("qmm_tree_attention", rc)


def qmm_cache_commit(h, page_table, lens, path, accept, lens_out, stream=None) -> None:
    """Compacts the accepted branches (path int32 [B, T], accept int32 [B, 2]); asynchronous."""
    B, T = path.shape
    rc = load().qmm_cache_commit(
        h, B, T, page_table.data_ptr(), page_table.stride(0), page_table.shape[1], lens.data_ptr(), path.data_ptr(),
        path.stride(0), accept.data_ptr(), lens_out.data_ptr(), _stream_ptr(stream, lens.device.index))
    if rc:
        _check("qmm_cache_commit", rc)


def qmm_cache_copy(h, src, dst, rows=None, stream=None) -> None:
    """Copies pages src[i] to dst[i] (int32), their first rows[i] rows; asynchronous."""
    _check("qmm_cache_copy", load().qmm_cache_copy(
        h, src.numel(), src.data_ptr(), dst.data_ptr(), rows.data_ptr() if rows is not None else None,
        _stream_ptr(stream, src.device.index)))


def qmm_debug_set_cache_wait_limit(h, ns: int) -> None:
    _check("qmm_debug_set_cache_wait_limit", load().qmm_debug_set_cache_wait_limit(h, ns))


@functools.lru_cache(maxsize=256)
def qmm_verify_sample_workspace(B: int, T: int, V: int) -> int:
    """Bytes of device workspace qmm_verify_sample needs for those sizes (and them alone)."""
    n = ctypes.c_int64()
    _check("qmm_verify_sample_workspace", load().qmm_verify_sample_workspace(B, T, V, ctypes.byref(n)))
    return n.value


def qmm_verify_sample(target, draft, tokens, u, noise, accept, path, workspace, parents=None, temperature=None,
                      n_tokens=None, stream=None) -> None:
    """target [B, T, V] and draft [B, T or T - 1, V] (or None) fp32, bf16 or f16;
    the other arguments as in qmm_sample_args; asynchronous."""
    B, T, V = target.shape
    ts = target.stride()
    ds = (0, 0) if draft is None else draft.stride()
    rc = load().qmm_verify_sample(_SAMPLE.pack(
        _SAMPLE.size, _dtype(target.dtype), B, T, V, target.data_ptr(), ts[0], ts[1],
        0 if draft is None else draft.data_ptr(), ds[0], ds[1], tokens.data_ptr(),
        0 if parents is None else parents.data_ptr(), 0 if n_tokens is None else n_tokens.data_ptr(), u.data_ptr(),
        noise.data_ptr(), 0 if temperature is None else temperature.data_ptr(), accept.data_ptr(), path.data_ptr(),
        workspace.data_ptr(), workspace.numel() * workspace.element_size()), _stream_ptr(stream, target.device.index))
    if rc:
        _check("qmm_verify_sample", rc)


# ------------------------------------------------------------------ convenience
def verify_sample(target, draft, tokens, u, noise, parents=None, temperature=None, n_tokens=None, stream=None):
    """(accept, path) of a drafted tree under rejection sampling; see
    qmm_verify_sample.  accept[:, 0] nodes are accepted, path[b, :accept[b, 0]]
    names them, accept[:, 1] is the token that follows them."""
    import torch
    if stream is not None:  # the results are allocated on the stream that writes them
        with torch.cuda.stream(stream):
            return verify_sample(target, draft, tokens, u, noise, parents, temperature, n_tokens)
    if target.dim() != 3 or not target.is_cuda:
        raise ValueError("target must be a CUDA tensor [B, T, V]")
    B, T, V = target.shape
    at = target.get_device()
    _rows("target", target)
    if draft is not None:
        if draft.dim() != 3 or draft.shape[1] not in (T, T - 1):
            raise ValueError(f"draft must hold {T} or {T - 1} rows a sequence")
        _strided("draft", draft, target.dtype, (B, draft.shape[1], V), at)
        if draft.shape[1] == 0:
            draft = None
    i32, f32, nodes = torch.int32, torch.float32, (B, T)
    # the usual call's checks in one expression; what fails is named after it
    if (tokens.shape != nodes or tokens.dtype is not i32 or tokens.get_device() != at or not tokens.is_contiguous()
            or u.shape != nodes or u.dtype is not f32 or u.get_device() != at or not u.is_contiguous()
            or noise.shape != (B, V) or noise.dtype is not f32 or noise.get_device() != at
            or not noise.is_contiguous()):
        _flat("tokens", tokens, i32, nodes, at)
        _flat("u", u, f32, nodes, at)
        _flat("noise", noise, f32, (B, V), at)
    if parents is not None:
        _flat("parents", parents, i32, nodes, at)
    if temperature is not None:
        _flat("temperature", temperature, f32, (B,), at)
    if n_tokens is not None:
        _flat("n_tokens", n_tokens, i32, (B,), at)
    if torch._C._cuda_getDevice() != at:
        _check("verify_sample", QMM_ERR_DEVICE)
    dev = target.device
    accept = torch.empty((B, 2), dtype=i32, device=dev)
    path = torch.empty((B, T), dtype=i32, device=dev)
    ws = torch.empty(qmm_verify_sample_workspace(B, T, V), dtype=torch.uint8, device=dev)
    qmm_verify_sample(target, draft, tokens, u, noise, accept, path, ws, parents, temperature, n_tokens)
    return accept, path


def tree_mask(parents):
    """int64 [B, T] visibility words of drafted trees from parents [B, T] (CPU
    values; a node sees itself and its ancestors; roots have parent -1)."""
    import torch
    words = []
    for row in parents.tolist():
        seen = []
        for i, par in enumerate(row):
            if par >= i:
                raise ValueError(f"parent {par} of node {i} does not come before it")
            seen.append((seen[par] if par >= 0 else 0) | 1 << i)
        words.append([w - (1 << 64) if w >> 63 else w for w in seen])
    return torch.tensor(words, dtype=torch.int64)


class Sequence:
    """One sequence's pages, in order, and its number of cached rows."""

    def __init__(self):
        self.pages: list[int] = []
        self.length = 0


class PagedCache:
    """Key and value pools [n_layers, n_pages, n_kv_heads, page_size, head_dim], a
    handle for the kernels, and the host's page bookkeeping."""

    def __init__(self, n_layers: int, n_pages: int, page_size: int, n_q_heads: int, n_kv_heads: int, head_dim: int,
                 dtype=None, max_batch: int = 64, k_pool=None, v_pool=None, device="cuda", stream=None):
        import torch
        dtype = torch.bfloat16 if dtype is None else dtype
        shape = (n_layers, n_pages, n_kv_heads, page_size, head_dim)
        pools = []
        for name, pool in (("k_pool", k_pool), ("v_pool", v_pool)):
            if pool is None:
                pool = torch.zeros(shape, dtype=dtype, device=device)
            _flat(name, pool, dtype, shape, pools[0].get_device() if pools else max(0, pool.get_device()))
            pools.append(pool)
        self.k_pool, self.v_pool = pools
        self.n_layers, self.n_pages, self.page_size = n_layers, n_pages, page_size
        self.n_q_heads, self.n_kv_heads, self.head_dim, self.dtype = n_q_heads, n_kv_heads, head_dim, dtype
        self.handle = None
        self._device = pools[0].get_device()
        if torch._C._cuda_getDevice() != self._device:
            _check("PagedCache", QMM_ERR_DEVICE)
        self.handle = qmm_cache_create(_dtype(dtype), n_layers, n_pages, page_size, n_q_heads, n_kv_heads, head_dim,
                                       max_batch, self.k_pool, self.v_pool, stream)
        self._users = [0] * n_pages
        self._free = list(range(n_pages - 1, -1, -1))

    # -------------------------------------------------------------- operators
    def attend(self, layer: int, q, k, v, page_table, lens, mask=None, n_tokens=None, scale=None, out=None,
               lse=None, stream=None):
        """(out, lse): the nodes' attention over cache and tree; their keys and
        values are written behind the cached rows.  See qmm_tree_attention."""
        import torch
        if stream is not None:  # the results are allocated on the stream that writes them
            with torch.cuda.stream(stream):
                return self.attend(layer, q, k, v, page_table, lens, mask, n_tokens, scale, out, lse)
        if q.dim() != 4:
            raise ValueError("q must be [B, T, n_q_heads, head_dim]")
        B, T, _, _ = q.shape
        dt, Hq, D, i32, at = self.dtype, self.n_q_heads, self.head_dim, torch.int32, self._device
        wide, new, seqs = (B, T, Hq, D), (B, T, self.n_kv_heads, D), (B,)
        qs, ks, vs, table = q.stride(), k.stride(), v.stride(), page_table.shape
        # all of a usual call's checks in one expression; what fails is named after it
        if (q.shape != wide or k.shape != new or v.shape != new or q.dtype is not dt or k.dtype is not dt
                or v.dtype is not dt or q.get_device() != at or k.get_device() != at or v.get_device() != at
                or qs[3] != 1 or ks[3] != 1 or vs[3] != 1 or len(table) != 2 or table[0] != B
                or page_table.dtype is not i32 or page_table.get_device() != at or page_table.stride(1) != 1
                or lens.shape != seqs or lens.dtype is not i32 or lens.get_device() != at
                or not lens.is_contiguous()):
            _strided("q", q, dt, wide, at)
            _strided("k", k, dt, new, at)
            _strided("v", v, dt, new, at)
            self._table(page_table, lens, B)
        if mask is not None:
            _strided("mask", mask, torch.int64, (B, T), at)
        if n_tokens is not None:
            _flat("n_tokens", n_tokens, i32, seqs, at)
        if out is None:
            out = torch.empty(wide, dtype=dt, device=q.device)
        else:
            _strided("out", out, dt, wide, at)
        if lse is None:
            lse = torch.empty((B, T, Hq), dtype=torch.float32, device=q.device)
        else:
            _flat("lse", lse, torch.float32, (B, T, Hq), at)
        _tree_attention(self.handle, layer, q, k, v, page_table, lens, out, lse, mask, n_tokens, scale, None, qs, ks,
                        vs, out.stride(), page_table.stride(0))
        return out, lse

    def commit(self, page_table, lens, path, accept, lens_out=None, stream=None):
        """The new lengths: the accepted branches' rows move behind the cached ones
        in every layer.  See qmm_cache_commit."""
        import torch
        if stream is not None:  # lens_out is allocated on the stream that writes it
            with torch.cuda.stream(stream):
                return self.commit(page_table, lens, path, accept, lens_out)
        i32, seqs, table, nodes, at = torch.int32, lens.shape, page_table.shape, path.shape, self._device
        B = seqs[0]
        # the usual call's checks in one expression; what fails is named after it
        if (len(seqs) != 1 or lens.dtype is not i32 or lens.get_device() != at or not lens.is_contiguous()
                or len(table) != 2 or table[0] != B or page_table.dtype is not i32 or page_table.get_device() != at
                or page_table.stride(1) != 1 or len(nodes) != 2 or nodes[0] != B or path.dtype is not i32
                or path.get_device() != at or path.stride(1) != 1 or accept.shape != (B, 2)
                or accept.dtype is not i32 or accept.get_device() != at or not accept.is_contiguous()):
            self._table(page_table, lens, B)
            if path.dim() != 2:
                raise ValueError("path must be [B, T]")
            _strided("path", path, i32, (B, path.shape[1]), at)
            _flat("accept", accept, i32, (B, 2), at)
        if lens_out is None:
            lens_out = torch.empty_like(lens)
        else:
            _flat("lens_out", lens_out, i32, (B,), at)
        qmm_cache_commit(self.handle, page_table, lens, path, accept, lens_out)
        return lens_out

    def copy_pages(self, src, dst, rows=None, stream=None):
        """Copies the first rows[i] rows (None: all) of page src[i] to page dst[i]
        in every layer.  See qmm_cache_copy."""
        import torch
        shape, i32, at = (src.numel(),), torch.int32, self._device
        _flat("src", src, i32, shape, at)
        _flat("dst", dst, i32, shape, at)
        if rows is not None:
            _flat("rows", rows, i32, shape, at)
        qmm_cache_copy(self.handle, src, dst, rows, stream)

    def sync_status(self, stream=None) -> int:
        return qmm_cache_sync_status(self.handle, stream)

    def _table(self, page_table, lens, B):
        import torch
        if page_table.dim() != 2:
            raise ValueError("page_table must be [B, pages]")
        _strided("page_table", page_table, torch.int32, (B, page_table.shape[1]), self._device)
        _flat("lens", lens, torch.int32, (B,), self._device)

    # -------------------------------------------------------------- bookkeeping
    @property
    def free_pages(self) -> int:
        return len(self._free)

    def new_sequence(self) -> Sequence:
        return Sequence()

    def _take(self, n):
        if n > len(self._free):
            raise MemoryError(f"{n} pages wanted, {len(self._free)} free")
        pages = [self._free.pop() for _ in range(n)]
        for p in pages:
            self._users[p] = 1
        return pages

    def reserve(self, seqs, rows: int, stream=None) -> None:
        """Pages of their own for `rows` more rows of every sequence: fresh ones
        where more are needed, and a copy of a partly filled last page that
        others share, made on `stream` (None: the current one), which has to be the
        one that writes the sequences' rows.  Nothing is taken when there are too
        few."""
        need, shared, left = [], [], list(self._users)
        for s in seqs:
            tail = s.length // self.page_size
            shared.append([])
            for i in range(tail, len(s.pages)):
                if left[s.pages[i]] > 1:
                    left[s.pages[i]] -= 1
                    shared[-1].append(i)
            need.append(max(0, -(-(s.length + rows) // self.page_size) - len(s.pages)))
        total = sum(need) + sum(map(len, shared))
        if total > len(self._free):
            raise MemoryError(f"{total} pages wanted, {len(self._free)} free")
        copies = []
        for s, n, at in zip(seqs, need, shared):
            for i in at:
                (fresh,) = self._take(1)
                used = min(max(s.length - i * self.page_size, 0), self.page_size)
                if used:
                    copies.append((s.pages[i], fresh, used))
                self._users[s.pages[i]] -= 1
                s.pages[i] = fresh
            s.pages += self._take(n)
        self._copy(copies, stream)

    def _copy(self, copies, stream=None):
        import torch
        if stream is not None:  # the page ids are allocated on the stream that reads them
            with torch.cuda.stream(stream):
                return self._copy(copies)
        if copies:
            t = torch.tensor(copies, dtype=torch.int32).t().contiguous().to(self.k_pool.device)
            self.copy_pages(t[0], t[1], t[2])

    def advance(self, seqs, counts) -> None:
        """The host's record of `counts` committed rows a sequence."""
        for s, n in zip(seqs, counts):
            if s.length + int(n) > len(s.pages) * self.page_size:
                raise ValueError("more rows than the sequence has pages for")
            s.length += int(n)

    def fork(self, seq: Sequence) -> Sequence:
        """A second sequence with the same cached rows: pages are shared until
        reserve() gives one of them rows of its own."""
        other = Sequence()
        other.length = seq.length
        other.pages = seq.pages[:-(-seq.length // self.page_size)]
        for p in other.pages:
            self._users[p] += 1
        return other

    def free(self, seq: Sequence) -> None:
        """Return the sequence's pages; those that others share stay."""
        for p in seq.pages:
            self._users[p] -= 1
            if self._users[p] == 0:
                self._free.append(p)
        seq.pages, seq.length = [], 0

    def tables(self, seqs, stream=None):
        """(page_table, lens) CUDA tensors for calls over `seqs` on `stream` (None: the
        current one)."""
        import torch
        if stream is not None:  # allocated on the stream that reads them
            with torch.cuda.stream(stream):
                return self.tables(seqs)
        width = max(1, max(len(s.pages) for s in seqs))
        rows = [s.pages + [0] * (width - len(s.pages)) for s in seqs]
        dev = self.k_pool.device
        return (torch.tensor(rows, dtype=torch.int32).to(dev),
                torch.tensor([s.length for s in seqs], dtype=torch.int32).to(dev))

    def close(self):
        if self.handle:
            qmm_cache_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
