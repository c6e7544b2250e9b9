"""Paged KV cache around the decode step (C ABI in include/mk_cache.h).

Argument checks and marshalling only; the work is done by the CUDA library.
Arguments are torch CUDA tensors; calls are asynchronous on the stream the object
was made with.  Where that is not torch's current stream, the caller orders the
two and keeps a call's tensors until the stream has passed it.
"""
from __future__ import annotations

import ctypes
import math

from . import (_addr, _check, lib, mk_append_desc, mk_append_rows, mk_attn_batch, mk_attn_desc,
               mk_kv_desc)


def _stream(stream, device):
    """The cudaStream_t of a torch stream, an integer, or (None) torch's current
    stream on the device."""
    if stream is None:
        import torch

        return torch.cuda.current_stream(device).cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _want(t, what, dtype, device, ndim=None):
    """t is a contiguous tensor of this type on this device."""
    import torch

    if not isinstance(t, torch.Tensor) or t.dtype != getattr(torch, dtype):
        raise TypeError(f"{what} has to be a torch.{dtype} tensor")
    if t.device != device:
        raise ValueError(f"{what} is on {t.device}, not on {device}")
    if (ndim is not None and t.dim() != ndim) or not t.is_contiguous():
        raise ValueError(f"{what} has to be contiguous"
                         + (f" with {ndim} dimensions" if ndim is not None else ""))
    return t


def _batch(device, page_tables, seq_lens, q_offsets, group_starts, prefix_lens, n_tokens):
    _want(page_tables, "page_tables", "int32", device, 2)
    _want(seq_lens, "seq_lens", "int32", device, 1)
    n = seq_lens.numel()
    if page_tables.shape[0] != n:
        raise ValueError("seq_lens has an entry for each table row")
    if (group_starts is None) != (prefix_lens is None):
        raise ValueError("group_starts and prefix_lens come together")
    groups = 0
    if group_starts is not None:
        _want(group_starts, "group_starts", "int32", device, 1)
        _want(prefix_lens, "prefix_lens", "int32", device, 1)
        groups = prefix_lens.numel()
        if group_starts.numel() != groups + 1:
            raise ValueError("group_starts has one entry more than prefix_lens")
    if q_offsets is not None:
        _want(q_offsets, "q_offsets", "int32", device, 1)
        if q_offsets.numel() != n + 1:
            raise ValueError("q_offsets has one entry more than there are sequences")
    if n_tokens is None:
        n_tokens = n
    b = mk_attn_batch(n, n_tokens, groups, page_tables.shape[1], page_tables.data_ptr(), seq_lens.data_ptr(),
                      _addr(q_offsets), _addr(group_starts), _addr(prefix_lens))
    b.keep, b.device = (page_tables, seq_lens, q_offsets, group_starts, prefix_lens), device
    return b


def _layers(layers, n_kv_heads, page_size, head_dim):
    """(the (k_cache, v_cache) tensors of each layer, checked; device; pages)."""
    layers = [tuple(kv) for kv in layers]
    if not layers:
        raise ValueError("no layers")
    dev, pages = layers[0][0].device, layers[0][0].shape[0]
    for k, v in layers:
        for t, what in ((k, "k_cache"), (v, "v_cache")):
            _want(t, what, "bfloat16", dev)
            if t.numel() != pages * n_kv_heads * page_size * head_dim:
                raise ValueError(f"{what} is not [{pages}][{n_kv_heads}][{page_size}]"
                                 f"[{head_dim}]")
    if dev.type != "cuda":
        raise ValueError("the caches have to be CUDA tensors")
    return layers, dev, pages


def _pointers(tensors):
    return (ctypes.c_void_p * len(tensors))(*[t.data_ptr() for t in tensors])


class KvCache:
    """Who holds which page of a set of paged pools.

    pools: the K and V pool of every layer, each a contiguous tensor whose first
    dimension is num_pages (the l{i}.kpool / l{i}.vpool of a Decoder).
    page_tables int32 [n_seqs][max_pages_per_seq] (-1: unused), seq_lens int32
    [n_seqs] and page_refs int32 [num_pages] (holders of each page) are the
    caller's and are updated in place.

    A call that is refused on the device changes nothing, and neither do the
    calls behind it, until sync() raises its MkError."""

    def __init__(self, pools, page_tables, seq_lens, page_refs, page_size: int, stream=None):
        import torch

        pools = list(pools)
        if not pools or not all(isinstance(p, torch.Tensor) and p.is_cuda and p.is_contiguous()
                                for p in pools):
            raise ValueError("pools have to be contiguous CUDA tensors")
        dev, shape = pools[0].device, pools[0].shape
        page_bytes = pools[0][0].numel() * pools[0].element_size() if shape[0] else 0
        if any(p.device != dev or p.shape != shape or p.dtype != pools[0].dtype for p in pools):
            raise ValueError("pools have to agree in device, shape and type")
        _want(page_tables, "page_tables", "int32", dev, 2)
        _want(seq_lens, "seq_lens", "int32", dev, 1)
        _want(page_refs, "page_refs", "int32", dev, 1)
        if seq_lens.numel() != page_tables.shape[0] or page_refs.numel() != shape[0]:
            raise ValueError("seq_lens has an entry for each table row, page_refs for each page")
        self.handle = None
        self.device, self._index, self._int32 = dev, page_refs.get_device(), torch.int32
        self.pools, self.page_tables = pools, page_tables
        self.seq_lens, self.page_refs = seq_lens, page_refs
        self.n_seqs, self.max_pages_per_seq = page_tables.shape
        self.page_size = page_size
        self._page_heads = shape[1] if len(shape) == 4 and shape[2] == page_size else None
        ptrs = (ctypes.c_void_p * len(pools))(*[p.data_ptr() for p in pools])
        desc = mk_kv_desc(len(pools), shape[0], page_size, self.n_seqs, self.max_pages_per_seq,
                          page_bytes, ptrs, page_tables.data_ptr(), seq_lens.data_ptr(),
                          page_refs.data_ptr())
        self._lib = lib()
        h = ctypes.c_void_p()
        with torch.cuda.device(dev):
            _check(self._lib.mk_kv_create(ctypes.byref(desc), _stream(stream, dev),
                                          ctypes.byref(h)), "mk_kv_create")
        self.handle = h.value

    def _two(self, a, b, what_a, what_b):
        for t, what in ((a, what_a), (b, what_b)):
            # the quick look first: these calls take a few microseconds
            if not (getattr(t, "dtype", None) is self._int32 and t.get_device() == self._index
                    and t.dim() == 1 and t.is_contiguous()):
                _want(t, what, "int32", self.device, 1)
        n = a.numel()
        if n != b.numel():
            raise ValueError(f"{what_a} and {what_b} have different lengths")
        return self.handle, n, a.data_ptr(), b.data_ptr()

    def copy_pages(self, src_pages, dst_pages):
        """Copies page src_pages[i] over page dst_pages[i] in every pool."""
        _check(self._lib.mk_kv_copy_pages(*self._two(src_pages, dst_pages, "src_pages",
                                                     "dst_pages")), "mk_kv_copy_pages")

    def fork(self, src_seqs, dst_seqs):
        """Makes sequence dst_seqs[i] a copy of src_seqs[i] that shares its full pages."""
        _check(self._lib.mk_kv_fork(*self._two(src_seqs, dst_seqs, "src_seqs", "dst_seqs")),
               "mk_kv_fork")

    def resize(self, seqs, new_lens):
        """Sets the lengths of sequences: takes or releases pages; 0 frees a sequence."""
        _check(self._lib.mk_kv_resize(*self._two(seqs, new_lens, "seqs", "new_lens")),
               "mk_kv_resize")

    def keep(self, seqs, starts, offsets, picks, n_kv_heads: int = None):
        """Moves, in every pool, the tokens at starts[i] + picks[j] of sequence seqs[i], j from
        offsets[i] to offsets[i + 1], to starts[i], starts[i] + 1, ...: a drafted tree's accepted
        path.  Lengths do not change.  n_kv_heads: of a page; None: the pools' second dimension
        (pools [pages][heads][tokens][dims])."""
        _, n, s, b = self._two(seqs, starts, "seqs", "starts")
        for t, what in ((offsets, "offsets"), (picks, "picks")):
            if not (getattr(t, "dtype", None) is self._int32 and t.get_device() == self._index
                    and t.dim() == 1 and t.is_contiguous()):
                _want(t, what, "int32", self.device, 1)
        if offsets.numel() != n + 1:
            raise ValueError("offsets has one entry more than there are sequences")
        if n_kv_heads is None:
            n_kv_heads = self._page_heads
            if n_kv_heads is None:
                raise ValueError("n_kv_heads is needed: the pools are not [pages][heads][tokens][dims]")
        _check(self._lib.mk_kv_keep(self.handle, n, s, b, offsets.data_ptr(), picks.numel(),
                                    picks.data_ptr(), n_kv_heads), "mk_kv_keep")

    def compact(self, page_map=None):
        """Moves the held pages to the lowest ids; page_map (int32 [num_pages]) receives
        each page's new id, -1 for free pages."""
        if page_map is not None:
            _want(page_map, "page_map", "int32", self.device, 1)
            if page_map.numel() != self.page_refs.numel():
                raise ValueError("page_map has an entry for each page")
        _check(self._lib.mk_kv_compact(self.handle, _addr(page_map)), "mk_kv_compact")

    def sync(self):
        """Waits for the stream; raises the MkError of the first refused call."""
        _check(self._lib.mk_kv_sync(self.handle), "mk_kv_sync")

    def read(self, seqs):
        """(lengths, table rows) of sequences as numpy arrays (synchronises)."""
        rows = [int(i) for i in seqs]
        if any(not 0 <= i < self.n_seqs for i in rows):
            raise ValueError(f"seqs are numbers of table rows, 0 to {self.n_seqs - 1}")
        self.sync()
        return (self.seq_lens[rows].cpu().numpy(), self.page_tables[rows].cpu().numpy())

    def close(self):
        if self.handle:
            self._lib.mk_kv_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class PrefixAttention:
    """Attention of a batch's query tokens over paged K and V, reading the pages
    that a group of sequences shares once for all of them.

    layers: (k_cache, v_cache) of each layer, contiguous bf16 [num_pages]
    [n_kv_heads][page_size][head_dim].  max_tokens bounds a call's query tokens
    (it sizes the workspace).  scale: of the scores, None for 1 / sqrt(head_dim)."""

    def __init__(self, n_q_heads: int, n_kv_heads: int, head_dim: int, page_size: int, layers,
                 max_tokens: int, max_seqs: int = 1024, max_groups: int = 512,
                 scale: float = None, stream=None):
        import torch

        if scale is not None and not ctypes.c_float(scale).value > 0.0:
            raise ValueError("scale has to be positive, in 32 bits")
        layers, dev, pages = _layers(layers, n_kv_heads, page_size, head_dim)
        self.handle = None
        self.device, self.layers, self.max_tokens = dev, layers, max_tokens
        self.heads, self.head_dim = n_q_heads, head_dim
        self._index, self._bf16, self._f32 = layers[0][0].get_device(), torch.bfloat16, torch.float32
        self._int32 = torch.int32
        self._lib = lib()
        n = len(layers)
        ks, vs = _pointers([k for k, _ in layers]), _pointers([v for _, v in layers])
        desc = mk_attn_desc(n_q_heads, n_kv_heads, head_dim, page_size, pages, max_tokens,
                            max_seqs, max_groups, n, ks, vs, scale or 0.0)
        h = ctypes.c_void_p()
        with torch.cuda.device(dev):
            _check(self._lib.mk_attn_create(ctypes.byref(desc), _stream(stream, dev),
                                            ctypes.byref(h)), "mk_attn_create")
        self.handle = h.value

    def batch(self, page_tables, seq_lens, q_offsets=None, group_starts=None, prefix_lens=None,
              n_tokens: int = None):
        """The batch of a call, to be kept as long as its tensors stay in place (their
        contents may change between calls).  q_offsets None: one query token each.
        n_tokens: rows of q and out; None: with q_offsets max_tokens, else one each."""
        if n_tokens is None and q_offsets is not None:
            n_tokens = self.max_tokens
        return _batch(self.device, page_tables, seq_lens, q_offsets, group_starts, prefix_lens,
                      n_tokens)

    def run(self, layer: int, batch, q, out, lse=None, tree=None):
        """out [n_tokens][n_q_heads][head_dim] = attention of q over the layer's pools;
        lse (fp32 [n_tokens][n_q_heads]) receives the logarithm of the softmax sums.  q may
        have a token stride of its own (the q part of a fused projection).  tree (int32 [n_tokens]
        [words], see tree_rows): which of its sequence's query tokens each one sees, a bit for
        each; None: those before it and itself."""
        rows = (batch.n_tokens, self.heads, self.head_dim)
        if batch.device != self.device:
            raise ValueError(f"the batch is on {batch.device}, not on {self.device}")
        if (q.shape != rows or q.dtype is not self._bf16 or q.get_device() != self._index
                or q.stride(2) != 1 or (self.heads > 1 and q.stride(1) != self.head_dim)):
            raise ValueError(f"q has to be bfloat16 {rows} with contiguous heads on {self.device}")
        # the quick look first: a call takes some tens of microseconds
        if not (out.dtype is self._bf16 and out.get_device() == self._index
                and out.is_contiguous()):
            _want(out, "out", "bfloat16", self.device)
        if out.shape != rows:
            raise ValueError(f"out has to be {rows}")
        if lse is not None:
            if not (lse.dtype is self._f32 and lse.get_device() == self._index
                    and lse.is_contiguous()):
                _want(lse, "lse", "float32", self.device)
            if lse.shape != rows[:2]:
                raise ValueError(f"lse has to be {rows[:2]}")
        stride = q.stride(0) if rows[0] > 1 else self.heads * self.head_dim
        to = None if lse is None else lse.data_ptr()
        if tree is None:
            _check(self._lib.mk_prefix_attention(self.handle, layer, ctypes.byref(batch),
                                                 q.data_ptr(), stride, out.data_ptr(), to),
                   "mk_prefix_attention")
            return
        if not (tree.dtype is self._int32 and tree.get_device() == self._index
                and tree.dim() == 2 and tree.is_contiguous()):
            _want(tree, "tree", "int32", self.device, 2)
        if tree.shape[0] != rows[0]:
            raise ValueError("tree has a row for each query token")
        _check(self._lib.mk_tree_attention(self.handle, layer, ctypes.byref(batch),
                                           tree.data_ptr(), tree.shape[1], q.data_ptr(), stride,
                                           out.data_ptr(), to), "mk_tree_attention")

    def set_wait_limit_ns(self, ns: int):
        """How long a wait inside a kernel of the calls behind this one lasts before the call
        is given up, which sync() then raises; 2 seconds unless set."""
        _check(self._lib.mk_attn_set_wait_limit_ns(self.handle, ns), "mk_attn_set_wait_limit_ns")

    def sync(self):
        """Waits for the stream; raises the MkError of the first device error."""
        _check(self._lib.mk_attn_sync(self.handle), "mk_attn_sync")

    def close(self):
        if self.handle:
            self._lib.mk_attn_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def tree_rows(parents):
    """(tree, depths) of drafted trees, on the host, for PrefixAttention.run and, added to the
    context's length, for KvAppend's positions.  parents: for each sequence its tokens' parents,
    numbers of earlier tokens of the same sequence, -1 for a token that follows the context.
    tree: int32 [tokens][words], each token's ancestors and itself; depths: int32 [tokens]."""
    import numpy as np
    import torch

    words = max([1] + [-(-len(p) // 32) for p in parents])
    rows = np.zeros((sum(len(p) for p in parents), 4 * words), np.uint8)
    depths = np.zeros(len(rows), np.int32)
    first = 0
    for tokens in parents:
        for i, p in enumerate(tokens):
            if not -1 <= p < i:
                raise ValueError(f"token {i} has parent {p}: parents come before their children")
            if p >= 0:
                rows[first + i] = rows[first + p]
                depths[first + i] = depths[first + p] + 1
            rows[first + i, i // 8] |= 1 << i % 8
        first += len(tokens)
    return torch.from_numpy(rows.view("<i4")), torch.from_numpy(depths)


def rope_frequencies(rotary_dim: int, base: float = 10000.0, scaling: str = None,
                     factor: float = 1.0, old_context: int = None, low: float = 1.0,
                     high: float = 4.0):
    """Turning rates of rotary_dim / 2 pairs in radians a position, for KvAppend, of a context that
    is `factor` times as long as the one a model was trained with.

    scaling None: base ** (-2 i / rotary_dim).  "linear": those over factor.  "base": of a base
    grown by factor ** (rotary_dim / (rotary_dim - 2)), so that the slowest pair turns 1 / factor
    as fast and the fastest as before.  "parts": pairs that turn at least `high` times over
    old_context keep their rate, those that turn at most `low` times take it over factor, those
    between a blend that is linear in their turns."""
    if rotary_dim < 0 or rotary_dim % 2:
        raise ValueError("rotary_dim has to be even")
    if not (base > 0.0 and factor > 0.0):
        raise ValueError("base and factor have to be positive")
    if scaling == "base":
        if rotary_dim < 4:
            raise ValueError("scaling of the base takes two pairs at least")
        base *= factor ** (rotary_dim / (rotary_dim - 2))
    rates = [base ** (-2.0 * i / rotary_dim) for i in range(rotary_dim // 2)]
    if scaling in (None, "base"):
        return rates
    if scaling == "linear":
        return [f / factor for f in rates]
    if scaling != "parts":
        raise ValueError(f"scaling is None, 'linear', 'base' or 'parts', not {scaling!r}")
    if old_context is None or not low < high:
        raise ValueError("scaling by parts takes old_context, and low below high")

    def part(f):
        kept = min(1.0, max(0.0, (old_context * f / (2.0 * math.pi) - low) / (high - low)))
        return f * kept + f / factor * (1.0 - kept)

    return [part(f) for f in rates]


class KvAppend:
    """Norms and rotates the heads of a batch's tokens and appends their keys and values to the
    pages: prompts, drafted tokens, or single tokens.

    layers: (k_cache, v_cache) of each layer as for PrefixAttention.  rotary_dim: the head's first
    dims that turn (None: all).  interleaved: pairs are neighbours, else halves.  frequencies:
    radians a position of each pair (see rope_frequencies), None: of rope_base.  magnitude: of
    the cosines and sines.  norm_eps: 0 or above; under 2^-100 heads of any size are normed, else
    those whose elements are below 2^60."""

    def __init__(self, n_q_heads: int, n_kv_heads: int, head_dim: int, page_size: int, layers,
                 rotary_dim: int = None, interleaved: bool = False, rope_base: float = 10000.0,
                 frequencies=None, magnitude: float = 1.0, norm_eps: float = 1e-6, stream=None):
        import torch

        rotary_dim = head_dim if rotary_dim is None else rotary_dim
        if not ctypes.c_float(magnitude).value > 0.0:
            raise ValueError("magnitude has to be positive, in 32 bits")
        rates = None
        if frequencies is not None:
            rates = [float(f) for f in frequencies]
            if len(rates) != rotary_dim // 2:
                raise ValueError(f"frequencies has {len(rates)} entries for {rotary_dim // 2} pairs")
            rates = (ctypes.c_double * max(1, len(rates)))(*rates)
        layers, dev, pages = _layers(layers, n_kv_heads, page_size, head_dim)
        self.handle = None
        self.device, self.layers = dev, layers
        self.heads, self.kv_heads, self.head_dim = n_q_heads, n_kv_heads, head_dim
        self._index, self._bf16 = layers[0][0].get_device(), torch.bfloat16
        self._int32 = torch.int32
        self._lib = lib()
        desc = mk_append_desc(n_q_heads, n_kv_heads, head_dim, page_size, pages, rotary_dim,
                              int(bool(interleaved)), len(layers),
                              _pointers([k for k, _ in layers]), _pointers([v for _, v in layers]),
                              rates, rope_base, magnitude, norm_eps)
        h = ctypes.c_void_p()
        with torch.cuda.device(dev):
            _check(self._lib.mk_append_create(ctypes.byref(desc), _stream(stream, dev),
                                              ctypes.byref(h)), "mk_append_create")
        self.handle = h.value

    def batch(self, page_tables, seq_lens, q_offsets=None, n_tokens: int = None):
        """The batch of a call, as PrefixAttention.batch makes it (whose batches run() takes
        too), of at most 1024 sequences.  n_tokens: rows of q, k and v; needed with q_offsets."""
        if q_offsets is not None and n_tokens is None:
            raise ValueError("n_tokens is needed with q_offsets")
        return _batch(self.device, page_tables, seq_lens, q_offsets, None, None, n_tokens)

    def _stride(self, t, what, shape):
        stride = t.stride()
        if (t.shape != shape or t.dtype is not self._bf16 or t.get_device() != self._index
                or stride[2] != 1 or (shape[1] > 1 and stride[1] != shape[2])):
            raise ValueError(f"{what} has to be bfloat16 {tuple(shape)} with contiguous heads on "
                             f"{self.device}")
        return stride[0] if shape[0] > 1 else shape[1] * shape[2]

    def _gain(self, t, what):
        if not (t.dtype is self._bf16 and t.get_device() == self._index and t.is_contiguous()):
            _want(t, what, "bfloat16", self.device, 1)
        if t.numel() != self.head_dim:
            raise ValueError(f"{what} has an entry for each of the head's {self.head_dim} dims")
        return t.data_ptr()

    def run(self, layer: int, batch, k, v, q=None, q_out=None, positions=None, q_norm=None,
            k_norm=None):
        """k, v [n_tokens][n_kv_heads][head_dim] go to the layer's pages, q [n_tokens][n_q_heads]
        [head_dim] to q_out (which may be q itself).  They may have token strides of their own,
        as parts of a fused projection.  positions (int32 [n_tokens]): what the heads turn to,
        None: the tokens' places.  q_norm, k_norm: gains of the norm, None: no norm."""
        n = batch.n_tokens
        if batch.device != self.device:
            raise ValueError(f"the batch is on {batch.device}, not on {self.device}")
        if (q is None) != (q_out is None):
            raise ValueError("q and q_out come together")
        kv = (n, self.kv_heads, self.head_dim)
        k_stride, v_stride = self._stride(k, "k", kv), self._stride(v, "v", kv)
        q_at = q_to = at = None
        q_stride = q_out_stride = 0
        if q is not None:
            shape = (n, self.heads, self.head_dim)
            q_stride, q_out_stride = self._stride(q, "q", shape), self._stride(q_out, "q_out", shape)
            q_at, q_to = q.data_ptr(), q_out.data_ptr()
        if positions is not None:
            if not (positions.dtype is self._int32 and positions.get_device() == self._index
                    and positions.is_contiguous()):
                _want(positions, "positions", "int32", self.device, 1)
            if positions.shape != (n,):
                raise ValueError("positions has an entry for each token")
            at = positions.data_ptr()
        rows = mk_append_rows(
            q_at, k.data_ptr(), v.data_ptr(), q_to, q_stride, k_stride, v_stride, q_out_stride,
            None if q_norm is None else self._gain(q_norm, "q_norm"),
            None if k_norm is None else self._gain(k_norm, "k_norm"), at)
        _check(self._lib.mk_append_tokens(self.handle, layer, ctypes.byref(batch),
                                          ctypes.byref(rows)), "mk_append_tokens")

    def sync(self):
        """Waits for the stream; raises the MkError of the first device error."""
        _check(self._lib.mk_append_sync(self.handle), "mk_append_sync")

    def close(self):
        if self.handle:
            self._lib.mk_append_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
