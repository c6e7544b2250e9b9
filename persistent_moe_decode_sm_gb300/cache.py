"""Paged KV cache around the decode step (C ABI in include/mk_cache.h).

Argument checks and marshalling only; the work is done by the CUDA library.
Arguments are torch CUDA tensors; calls are asynchronous on the stream the object
was made with.  Where that is not torch's current stream, the caller orders the
two and keeps a call's tensors until the stream has passed it.
"""
from __future__ import annotations

import ctypes

from . import _addr, _check, lib, mk_kv_desc


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
        self.device = dev
        self.pools, self.page_tables = pools, page_tables
        self.seq_lens, self.page_refs = seq_lens, page_refs
        self.n_seqs, self.max_pages_per_seq = page_tables.shape
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
        _want(a, what_a, "int32", self.device, 1)
        _want(b, what_b, "int32", self.device, 1)
        if a.numel() != b.numel():
            raise ValueError(f"{what_a} and {what_b} have different lengths")
        return self.handle, a.numel(), a.data_ptr(), b.data_ptr()

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
        self.sync()
        rows = [int(i) for i in seqs]
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
