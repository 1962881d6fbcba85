"""Token trees over a paged key/value cache: the binding of the ``specverify_tree_*``, ``specverify_verify_tree`` and
``specverify_cache_*`` calls of ``include/specverify.h``.

:class:`KVCache` and :class:`TokenTree` describe a program's buffers once (they hold the tensors and check them);
:class:`SpecTree` is the handle. A serving step::

    st = SpecTree(max_batch, max_moves)
    cache = KVCache(k, v, page_table, mass=mass, pos=pos)        # one layer's, or all layers'
    tree = TokenTree(row_off, nodes, parent, tokens)
    out, lse = st.attention(q, layer_cache, tree, lens)           # in every layer
    n, emitted, path = st.verify(tree, logits)
    new_lens, new_seen = st.commit(cache, lens, n, path, seen=seen)
    st.accumulate(q, lse, layer_cache, tree, lens, n, path)       # in every layer
    mass_out, pos_out, kept = st.evict(cache, new_lens, new_seen, budget, sink=4, recent=256)

Every call is asynchronous on ``stream`` (default: the current stream of the handle's device). Output tensors that are
not passed in are allocated for that stream.
"""
from __future__ import annotations

import contextlib
import ctypes

import torch

FP32, BF16, FP16 = 0, 1, 2
MAX_NODES = 128

_DTYPES = {torch.bfloat16: BF16, torch.float16: FP16}
_LOGITS = {torch.float32: FP32, torch.bfloat16: BF16}


class SpecverifyCache(ctypes.Structure):
    """Mirror of ``specverify_cache`` (include/specverify.h)."""
    _fields_ = [("dtype", ctypes.c_int32), ("layers", ctypes.c_int32), ("num_pages", ctypes.c_int64),
                ("page_size", ctypes.c_int32), ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("layer_stride", ctypes.c_int64), ("page_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64),
                ("token_stride", ctypes.c_int64), ("mass", ctypes.c_void_p), ("pos", ctypes.c_void_p),
                ("mass_layer_stride", ctypes.c_int64), ("mass_page_stride", ctypes.c_int64),
                ("mass_head_stride", ctypes.c_int64), ("mass_token_stride", ctypes.c_int64),
                ("page_table", ctypes.c_void_p), ("table_stride", ctypes.c_int64), ("max_pages", ctypes.c_int32)]


class SpecverifyTree(ctypes.Structure):
    """Mirror of ``specverify_tree``."""
    _fields_ = [("B", ctypes.c_int32), ("max_nodes", ctypes.c_int32), ("row_off", ctypes.c_void_p),
                ("nodes", ctypes.c_void_p), ("parent", ctypes.c_void_p), ("tokens", ctypes.c_void_p)]


def bind(lib):
    """Declares the calls' argument types on the loaded library."""
    vp, i32, i64, f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float
    lib.specverify_tree_create.argtypes = [ctypes.POINTER(vp), ctypes.c_int, i32, i64]
    lib.specverify_tree_destroy.argtypes = [vp]
    lib.specverify_tree_status.argtypes = [vp, vp, ctypes.POINTER(i32)]
    lib.specverify_tree_workspace_bytes.argtypes = [vp, ctypes.POINTER(ctypes.c_size_t)]
    lib.specverify_tree_set_wait_limit.argtypes = [vp, ctypes.c_uint64]
    lib.specverify_tree_attention.argtypes = [vp, vp, vp, vp, vp, i64, i32, i64, i64, f32, vp, i64, i64, vp, vp]
    lib.specverify_verify_tree.argtypes = [vp, vp, vp, i32, i64, i64, i64, vp, vp, vp, vp]
    lib.specverify_tree_commit.argtypes = [vp, vp, i32, i32, vp, vp, vp, vp, vp, vp, vp]
    lib.specverify_cache_accumulate.argtypes = [vp, vp, vp, vp, vp, vp, vp, i64, i32, i64, i64, vp, f32, vp]
    lib.specverify_cache_evict.argtypes = [vp, vp, i32, vp, vp, i32, i32, i32, vp, vp, vp, vp]
    for name in ("tree_create", "tree_destroy", "tree_status", "tree_workspace_bytes", "tree_set_wait_limit",
                 "tree_attention", "verify_tree", "tree_commit", "cache_accumulate", "cache_evict"):
        getattr(lib, "specverify_" + name).restype = ctypes.c_int


def _need(ok: bool, what: str):
    if not ok:
        raise ValueError(what)


def _fits(bits=32, **values):
    """Whole numbers that the call would cut to their lowest bits are refused here."""
    for name, x in values.items():
        _need(-(1 << (bits - 1)) <= x < 1 << (bits - 1), f"{name} must fit {bits} bits, not {x}")


def _ints(name, t, index, shape, dtype=torch.int32):
    """The address of a contiguous integer tensor of that shape on CUDA device `index`."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != index or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on cuda:{index}, not "
                         f"{t.dtype} {tuple(t.shape)} on {t.device}")
    return t.data_ptr()


def _strides(t):
    """Strides with 0 for dimensions of one, whose stride says nothing."""
    return tuple(0 if n == 1 else s for n, s in zip(t.shape, t.stride()))


class KVCache:
    """A paged cache's buffers.

    ``k`` and ``v``: [pages, kv heads, page size, head size], or with a leading layers dimension, bfloat16 or float16, of
    the same strides; the last dimension is contiguous, the others may have any stride of a multiple of 16 bytes (a
    token-major pool is passed as ``pool.transpose(-3, -2)``). ``page_table``: int32 [B, pages of a sequence]. ``mass``
    (float32) and ``pos`` (int32): one value for each slot and head, [.., pages, kv heads, page size], of the same strides.
    """

    def __init__(self, k, v, page_table, mass=None, pos=None):
        _need(k.dim() in (4, 5) and v.shape == k.shape, "k and v must have one shape, [(layers,) pages, heads, page, d]")
        _need(k.dtype in _DTYPES and v.dtype == k.dtype, "k and v must both be bfloat16 or both float16")
        _need(_strides(k) == _strides(v) and k.stride(-1) == 1, "k and v must have the same strides and a contiguous head")
        _need(k.is_cuda and v.device == k.device, "k and v must be on one CUDA device")
        _need(page_table.dim() == 2 and page_table.dtype == torch.int32 and page_table.stride(1) == 1
              and page_table.device == k.device, "page_table must be int32 [B, pages] on the cache's device")
        pages, heads, page, d = k.shape[-4:]
        _need(d in (64, 128), "the head size must be 64 or 128")
        _need(page >= 8 and page % 8 == 0, "the page size must be a multiple of 8")
        _need(pages >= 1 and heads >= 1 and page_table.shape[1] >= 1, "the cache is empty")
        _need(k.dim() == 4 or k.shape[0] >= 1, "the cache has no layers")
        ks = _strides(k)
        _need(all(s % 8 == 0 for s in ks[:-1]) and k.data_ptr() % 16 == 0 and v.data_ptr() % 16 == 0,
              "k and v must be aligned to 16 bytes, strides and all")
        _need(all(s > 0 or n == 1 for s, n in zip(ks, k.shape)), "k and v must not be expanded")
        for name, t, dt in (("mass", mass, torch.float32), ("pos", pos, torch.int32)):
            if t is not None:
                _need(t.dtype == dt and t.shape == k.shape[:-1] and t.device == k.device,
                      f"{name} must be {dt}, of k's shape without the head, on its device")
                _need(all(s > 0 or n == 1 for s, n in zip(t.stride(), t.shape)), f"{name} must not be expanded")
        _need(mass is None or pos is None or _strides(mass) == _strides(pos), "mass and pos must have the same strides")
        self.k, self.v, self.page_table, self.mass, self.pos = k, v, page_table, mass, pos
        self.device, self.dtype, self.head_dim, self.kv_heads = k.device, k.dtype, d, heads
        self.index = k.get_device()
        self.layers, self.batch = (k.shape[0] if k.dim() == 5 else 1), page_table.shape[0]
        self.capacity = page * page_table.shape[1]
        self.values = next((t for t in (mass, pos) if t is not None), None)
        ks = (0,) * (5 - k.dim()) + ks
        ms = (0,) * 4 if self.values is None else (0,) * (5 - k.dim()) + _strides(self.values)
        self.struct = SpecverifyCache(
            _DTYPES[k.dtype], self.layers, pages, page, heads, d, k.data_ptr(), v.data_ptr(), *ks[:4],
            None if mass is None else mass.data_ptr(), None if pos is None else pos.data_ptr(), *ms,
            page_table.data_ptr(), page_table.stride(0) if page_table.shape[0] > 1 else page_table.shape[1],
            page_table.shape[1])
        self.ref = ctypes.byref(self.struct)


class TokenTree:
    """The buffers of a batch of drafted trees: ``row_off`` int64 [B], ``nodes`` int32 [B], ``parent`` and ``tokens`` int32
    [B, max nodes] (tokens only for :meth:`SpecTree.verify`). Their contents may change from step to step."""

    def __init__(self, row_off, nodes, parent, tokens=None):
        _need(parent.dim() == 2 and 1 <= parent.shape[1] <= MAX_NODES, f"parent must be [B, 1 to {MAX_NODES}]")
        _need(parent.is_cuda, "a tree's buffers must be on a CUDA device")
        B, index = parent.shape[0], parent.get_device()
        self.batch, self.max_nodes, self.device, self.index = B, parent.shape[1], parent.device, index
        self.row_off, self.nodes, self.parent, self.tokens = row_off, nodes, parent, tokens
        self.struct = SpecverifyTree(
            B, self.max_nodes, _ints("row_off", row_off, index, (B,), torch.int64), _ints("nodes", nodes, index, (B,)),
            _ints("parent", parent, index, parent.shape),
            None if tokens is None else _ints("tokens", tokens, index, parent.shape))
        self.ref = ctypes.byref(self.struct)


class SpecTree:
    """The handle of the token-tree calls on one CUDA device.

    ``max_batch``: sequences of a call at most. ``max_moves``: see :meth:`evict`. Calls of one handle follow one another on
    one stream; use a handle for each concurrently used stream and for each captured graph that may run beside another."""

    def __init__(self, max_batch: int, max_moves: int = 0, device: int | None = None):
        from . import _check, load
        self.lib, self.check = load(), _check
        self.index = torch.cuda.current_device() if device is None else int(device)
        self.device = torch.device("cuda", self.index)
        _fits(max_batch=max_batch, device=self.index)
        _fits(64, max_moves=max_moves)
        h = ctypes.c_void_p()
        _check(self.lib.specverify_tree_create(ctypes.byref(h), self.index, max_batch, max_moves), "specverify_tree_create")
        self.h = h
        self.max_batch, self.max_moves = max_batch, max_moves

    def close(self):
        if getattr(self, "h", None) is not None:
            self.check(self.lib.specverify_tree_destroy(self.h), "specverify_tree_destroy")
            self.h = None

    def __del__(self):
        with contextlib.suppress(Exception):
            self.close()

    def _stream(self, stream):
        return torch._C._cuda_getCurrentRawStream(self.index) if stream is None else stream.cuda_stream

    def _on(self, *described):
        for x in described:
            if x.index != self.index:
                raise ValueError(f"the handle is on {self.device}, the call's buffers on {x.device}")

    def _empty(self, stream, shape, dtype):
        if stream is None:
            return torch.empty(shape, dtype=dtype, device=self.device)
        with torch.cuda.stream(stream):
            return torch.empty(shape, dtype=dtype, device=self.device)

    def _rows(self, name, x, cache):
        """Address, rows, heads and strides of queries or outputs."""
        rows, heads, d = x.shape
        if (x.dtype is not cache.dtype or d != cache.head_dim or x.get_device() != self.index or heads < 1
                or heads % cache.kv_heads):
            raise ValueError(f"{name} must be [rows, heads, {cache.head_dim}] of {cache.dtype} on {self.device}, heads a "
                             f"multiple of {cache.kv_heads}, not {x.dtype} {tuple(x.shape)} on {x.device}")
        a, b, one = x.stride()
        if one != 1:
            raise ValueError(f"{name} must have a contiguous last dimension")
        return x.data_ptr(), rows, heads, a if rows > 1 else 0, b if heads > 1 else 0

    def _lse(self, lse, rows, heads):
        if (lse.dtype is not torch.float32 or lse.shape != (rows, heads) or lse.get_device() != self.index
                or not lse.is_contiguous()):
            raise ValueError(f"lse must be contiguous float32 [{rows}, {heads}] on {self.device}")
        return lse.data_ptr()

    def attention(self, q, cache: KVCache, tree: TokenTree, lens, *, scale=None, out=None, lse=None, stream=None):
        """Attention of the tree's nodes over the cache and their ancestors; returns (out like q, lse [rows, heads]).

        ``q`` [rows, heads, head size], ``lens`` int32 [B]: committed tokens; ``scale`` defaults to head size ** -0.5.
        ``out`` and ``lse``: buffers to use. Rows that belong to no sequence are not written."""
        self._on(cache, tree)
        B = tree.batch
        if cache.layers != 1 or cache.batch != B:
            raise ValueError("attention takes one layer's cache with a page table row for each sequence of the tree")
        qp, rows, heads, qr, qh = self._rows("q", q, cache)
        if out is None:
            out = self._empty(stream, q.shape, q.dtype)
        elif out.shape != q.shape:
            raise ValueError("out must have q's shape")
        op, _, _, orow, oh = self._rows("out", out, cache)
        if lse is None:
            lse = self._empty(stream, (rows, heads), torch.float32)
        rc = self.lib.specverify_tree_attention(
            self.h, cache.ref, tree.ref, _ints("lens", lens, self.index, (B,)), qp, rows, heads, qr, qh,
            cache.head_dim ** -0.5 if scale is None else scale, op, orow, oh, self._lse(lse, rows, heads),
            self._stream(stream))
        if rc:
            self.check(rc, "specverify_tree_attention")
        return out, lse

    def verify(self, tree: TokenTree, target, *, n=None, tokens=None, path=None, stream=None):
        """Greedy verify of the trees against target logits [rows, V] (float32 or bfloat16, rows aligned to 16 bytes);
        returns (n_accepted [B], emitted tokens [B, max nodes], accepted path [B, max nodes]), padded with -1."""
        self._on(tree)
        if (tree.tokens is None or target.dim() != 2 or target.dtype not in _LOGITS or target.stride(1) != 1
                or target.get_device() != self.index):
            raise ValueError("verify takes a tree with tokens and 2-D float32 or bfloat16 logits with unit column stride on "
                             f"{self.device}")
        B, T, at = tree.batch, tree.max_nodes, self.index
        n = self._empty(stream, (B,), torch.int32) if n is None else n
        tokens = self._empty(stream, (B, T), torch.int32) if tokens is None else tokens
        path = self._empty(stream, (B, T), torch.int32) if path is None else path
        rows, V = target.shape
        rc = self.lib.specverify_verify_tree(
            self.h, tree.ref, target.data_ptr(), _LOGITS[target.dtype], V, target.stride(0) if rows > 1 else -(-V // 8) * 8,
            rows, _ints("n", n, at, (B,)), _ints("tokens", tokens, at, (B, T)), _ints("path", path, at, (B, T)),
            self._stream(stream))
        if rc:
            self.check(rc, "specverify_verify_tree")
        return n, tokens, path

    def commit(self, cache: KVCache, lens, n, path, *, seen=None, new_lens=None, new_seen=None, stream=None):
        """Moves the accepted path's keys and values (every layer of the cache) behind the committed tokens; returns
        (new_lens, new_seen). ``seen`` int32 [B], the tokens of each sequence so far, is needed where the cache has
        ``pos``; new_seen is None without it."""
        self._on(cache)
        B, at = cache.batch, self.index
        if path.dim() != 2 or not 1 <= path.shape[1] <= MAX_NODES:
            raise ValueError(f"path must be [B, 1 to {MAX_NODES}]")
        if seen is None and cache.pos is not None:
            raise ValueError("a cache with positions needs `seen`")
        new_lens = self._empty(stream, (B,), torch.int32) if new_lens is None else new_lens
        if seen is not None and new_seen is None:
            new_seen = self._empty(stream, (B,), torch.int32)
        T = path.shape[1]
        rc = self.lib.specverify_tree_commit(
            self.h, cache.ref, B, T, _ints("lens", lens, at, (B,)), None if seen is None else _ints("seen", seen, at, (B,)),
            _ints("n", n, at, (B,)), _ints("path", path, at, (B, T)), _ints("new_lens", new_lens, at, (B,)),
            None if new_seen is None else _ints("new_seen", new_seen, at, (B,)), self._stream(stream))
        if rc:
            self.check(rc, "specverify_tree_commit")
        return new_lens, new_seen

    def accumulate(self, q, lse, cache: KVCache, tree: TokenTree, lens, n, path, *, scale=None, stream=None):
        """Adds to the cache's ``mass`` the attention weight that the accepted nodes gave each slot; ``q`` and ``lse`` are
        those of :meth:`attention`, ``lens`` the lengths before the commit, which has run. Returns the mass."""
        self._on(cache, tree)
        B, at = tree.batch, self.index
        if cache.layers != 1 or cache.mass is None or cache.batch != B:
            raise ValueError("accumulate takes one layer's cache, its mass and a page table row for each sequence of the tree")
        qp, rows, heads, qr, qh = self._rows("q", q, cache)
        rc = self.lib.specverify_cache_accumulate(
            self.h, cache.ref, tree.ref, _ints("lens", lens, at, (B,)), _ints("n", n, at, (B,)),
            _ints("path", path, at, (B, tree.max_nodes)), qp, rows, heads, qr, qh, self._lse(lse, rows, heads),
            cache.head_dim ** -0.5 if scale is None else scale, self._stream(stream))
        if rc:
            self.check(rc, "specverify_cache_accumulate")
        return cache.mass

    def evict(self, cache: KVCache, lens, seen, budget: int, *, sink: int = 0, recent: int = 0, mass_out=None, pos_out=None,
              new_lens=None, stream=None):
        """Cuts sequences of more than ``budget`` tokens down to it, in every layer and key head by itself: the first
        ``sink`` and the last ``recent`` positions stay, then the slots of the largest mass. ``mass_out`` and ``pos_out``
        default to the cache's own. Returns (mass_out, pos_out, new_lens). The handle's ``max_moves`` must be at least
        layers * B * kv heads * min(budget, slots of a sequence - budget)."""
        self._on(cache)
        B, at = cache.batch, self.index
        if cache.mass is None or cache.pos is None:
            raise ValueError("evict needs the cache's mass and pos")
        mass_out = cache.mass if mass_out is None else mass_out
        pos_out = cache.pos if pos_out is None else pos_out
        for name, t, like in (("mass_out", mass_out, cache.mass), ("pos_out", pos_out, cache.pos)):
            if t is not like and (t.dtype is not like.dtype or t.shape != like.shape or _strides(t) != _strides(like)
                                  or t.get_device() != at):
                raise ValueError(f"{name} must be laid out as the cache's")
        _fits(budget=budget, sink=sink, recent=recent)
        new_lens = self._empty(stream, (B,), torch.int32) if new_lens is None else new_lens
        rc = self.lib.specverify_cache_evict(
            self.h, cache.ref, B, _ints("lens", lens, at, (B,)), _ints("seen", seen, at, (B,)), budget, sink, recent,
            mass_out.data_ptr(), pos_out.data_ptr(), _ints("new_lens", new_lens, at, (B,)), self._stream(stream))
        if rc:
            self.check(rc, "specverify_cache_evict")
        return mass_out, pos_out, new_lens

    def device_status(self, stream=None) -> int:
        """Synchronises, returns the sticky status bits (``STATUS_BITS``) and clears them."""
        v = ctypes.c_int32()
        self.check(self.lib.specverify_tree_status(self.h, self._stream(stream), ctypes.byref(v)), "specverify_tree_status")
        return v.value

    def set_wait_limit(self, ns: int):
        """Bounds every wait inside the kernels of the calls that follow, in nanoseconds; 0: the default, about two
        seconds. A wait that runs out ends its call with the status bit ``timeout`` and its outputs undefined."""
        _need(0 <= ns < 1 << 63, f"a wait's limit must be a number of nanoseconds, not {ns}")
        self.check(self.lib.specverify_tree_set_wait_limit(self.h, int(ns)), "specverify_tree_set_wait_limit")

    def workspace_bytes(self) -> int:
        v = ctypes.c_size_t()
        self.check(self.lib.specverify_tree_workspace_bytes(self.h, ctypes.byref(v)), "specverify_tree_workspace_bytes")
        return v.value
