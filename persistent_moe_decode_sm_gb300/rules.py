"""Penalties, biases and masks on logits, and the greedy tokens under them (C ABI in
include/mk_rules.h).

Argument checks and marshalling only; the work is done by the CUDA library.  Arguments are torch
CUDA tensors; calls are asynchronous on the stream the object was made with."""
from __future__ import annotations

import ctypes

from . import _addr, _check, lib, mk_rules_batch
from .cache import _stream, _want


class TokenRules:
    """Rules on the logits of up to max_rows rows over a vocabulary.  The workspace lies on
    `device` (None: torch's current one)."""

    def __init__(self, vocab: int, max_rows: int, device=None, stream=None):
        import torch

        self.handle = None
        self.device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
        if self.device.type != "cuda":
            raise ValueError("the device has to be a CUDA device")
        if self.device.index is None:
            self.device = torch.device("cuda", torch.cuda.current_device())
        self._index = self.device.index
        self.vocab, self.max_rows = vocab, max_rows
        self._f32, self._bf16, self._int32 = torch.float32, torch.bfloat16, torch.int32
        self._lib = lib()
        self.stream = _stream(stream, self.device)
        h = ctypes.c_void_p()
        with torch.cuda.device(self.device):
            _check(self._lib.mk_rules_create(vocab, max_rows, self.stream, ctypes.byref(h)),
                   "mk_rules_create")
        self.handle = h.value

    def batch(self, n_rows: int, tokens=None, ranges=None, prompt_lens=None, path_offsets=None,
              path_tokens=None, repetition=None, presence=None, frequency=None, bias_offsets=None,
              bias_tokens=None, bias=None, allowed=None, allowed_rows=None):
        """What holds for the rows of a call, to be kept as long as its tensors stay in place
        (their contents may change between calls), by these rules or others with the same
        vocabulary and device.

        tokens int32, ranges int32 [n_rows][2] (begin and end of a row's history in tokens; rows
        may share one), prompt_lens int32 [n_rows] (of it, not generated); path_offsets int32
        [n_rows + 1] into path_tokens (drafted tokens behind the history); repetition, presence,
        frequency float32 [n_rows]; bias_offsets int32 [n_rows + 1] into bias_tokens (rising
        within a row) and bias (float32); allowed int32 [masks][(vocab + 31) // 32], a bit for
        each token that may follow, allowed_rows int32 [n_rows] (a row's mask, -1: none; without
        it mask i is of row i)."""
        for what, together in (("tokens and ranges", (tokens, ranges)),
                               ("path_offsets and path_tokens", (path_offsets, path_tokens)),
                               ("bias_offsets, bias_tokens and bias", (bias_offsets, bias_tokens, bias))):
            given = sum(t is not None for t in together)
            if given not in (0, len(together)):
                raise ValueError(what + " come together")
        if prompt_lens is not None and ranges is None:
            raise ValueError("prompt_lens comes with ranges")
        if allowed_rows is not None and allowed is None:
            raise ValueError("allowed_rows comes with allowed")
        words = (self.vocab + 31) // 32
        for t, what, dtype, shape in (
                (tokens, "tokens", "int32", (None,)), (ranges, "ranges", "int32", (n_rows, 2)),
                (prompt_lens, "prompt_lens", "int32", (n_rows,)),
                (path_offsets, "path_offsets", "int32", (n_rows + 1,)),
                (path_tokens, "path_tokens", "int32", (None,)),
                (repetition, "repetition", "float32", (n_rows,)),
                (presence, "presence", "float32", (n_rows,)),
                (frequency, "frequency", "float32", (n_rows,)),
                (bias_offsets, "bias_offsets", "int32", (n_rows + 1,)),
                (bias_tokens, "bias_tokens", "int32", (None,)), (bias, "bias", "float32", (None,)),
                (allowed, "allowed", "int32", (None, words)),
                (allowed_rows, "allowed_rows", "int32", (n_rows,))):
            if t is None:
                continue
            _want(t, what, dtype, self.device, len(shape))
            if any(want is not None and got != want for got, want in zip(t.shape, shape)):
                raise ValueError(f"{what} has shape {tuple(t.shape)}, not {shape}")
        if bias is not None and bias.numel() != bias_tokens.numel():
            raise ValueError("bias has an entry for each of bias_tokens")
        if allowed is not None and allowed_rows is None and allowed.shape[0] < n_rows:
            raise ValueError("allowed has a mask for each row, or allowed_rows says which")

        def count(t):
            return 0 if t is None else t.shape[0]

        arrays = (tokens, ranges, prompt_lens, path_offsets, path_tokens, repetition, presence,
                  frequency, bias_offsets, bias_tokens, bias, allowed, allowed_rows)
        b = mk_rules_batch(n_rows, count(tokens), count(path_tokens), count(bias_tokens),
                           count(allowed), *[_addr(t) for t in arrays])
        b.keep, b.vocab, b.device = arrays, self.vocab, self.device
        return b

    def run(self, batch, logits, out=None, tokens=None):
        """out float32 [n_rows][vocab] (None: not wanted; logits itself: in place) = logits, float32
        or bfloat16 with any row stride, under the batch's rules; tokens int32 [n_rows] (None: not
        wanted) the largest one's id in each row, -1 where none may follow."""
        _check(self._lib.mk_rules_apply(self.handle, ctypes.byref(batch),
                                        *self._args(batch, logits, out, tokens)), "mk_rules_apply")

    def follow(self, batch, logits, tokens):
        """run() in place behind a decode step, whose own greedy tokens `tokens` holds: a row that is
        refused on the device gets -1 there and does not keep the step's."""
        at, _, _, _, to = self._args(batch, logits, logits, tokens)
        _check(self._lib.mk_rules_follow(self.handle, ctypes.byref(batch), at, to), "mk_rules_follow")

    def check(self, batch, logits, out=None, tokens=None):
        """Raises what run() raises for these arguments; nothing is enqueued."""
        _check(self._lib.mk_rules_check(self.handle, ctypes.byref(batch),
                                        *self._args(batch, logits, out, tokens)), "mk_rules_check")

    def _args(self, batch, logits, out, tokens):
        """What mk_rules_apply takes behind the batch, checked."""
        n = batch.n_rows
        # the library knows a mask's length by the vocabulary alone
        if batch.vocab != self.vocab or batch.device != self.device:
            raise ValueError("the batch was made by rules with another vocabulary or on another device")
        stride, half = logits.stride(), logits.dtype is self._bf16
        if (logits.shape != (n, self.vocab) or not (half or logits.dtype is self._f32)
                or logits.get_device() != self._index or (self.vocab > 1 and stride[1] != 1)):
            raise ValueError(f"logits has to be float32 or bfloat16 {(n, self.vocab)} with contiguous "
                             f"rows on {self.device}")
        for t, what, dtype, shape in ((out, "out", self._f32, (n, self.vocab)), (tokens, "tokens", self._int32, (n,))):
            if t is not None and (t.dtype is not dtype or t.shape != shape or t.get_device() != self._index
                                  or not t.is_contiguous()):
                raise ValueError(f"{what} has to be contiguous {dtype} {shape} on {self.device}")
        return (logits.data_ptr(), half, stride[0] if n > 1 else self.vocab,
                None if out is None else out.data_ptr(), None if tokens is None else tokens.data_ptr())

    def sync(self):
        """Waits for the stream; raises the MkError of the first device error."""
        _check(self._lib.mk_rules_sync(self.handle), "mk_rules_sync")

    def close(self):
        if self.handle:
            self._lib.mk_rules_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
