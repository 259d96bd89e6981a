"""Python handle on the native block manager (include/pa_block_manager.h).

Host-only: the manager never touches the GPU, so it works without one.  It hands out the slots
that pa_cache_append writes, the block tables pa_attention reads, and the (source, destination)
pairs pa_copy_blocks must copy before a shared block is written.
"""

from __future__ import annotations

import ctypes
from typing import List, Optional, Sequence, Tuple

import numpy as np

from . import _lib

NO_SPACE = -1
BAD_ARG = -2


class NoSpace(RuntimeError):
    """Not enough free or evictable blocks; the manager is unchanged."""


class BlockManager:
    def __init__(self, num_blocks: int, block_size: int = 16):
        self._L = _lib.load()
        self._h = self._L.pa_bm_create(int(num_blocks), int(block_size))
        if not self._h:
            raise ValueError("num_blocks and block_size must be positive")
        self.num_blocks = int(num_blocks)
        self.block_size = int(block_size)

    def __del__(self):
        h = getattr(self, "_h", None)
        if h:
            self._L.pa_bm_destroy(h)
            self._h = None

    @staticmethod
    def _check(rc: int) -> int:
        if rc == NO_SPACE:
            raise NoSpace("not enough free blocks")
        if rc < 0:
            raise ValueError("bad argument (unknown or duplicate sequence, bad count)")
        return rc

    def num_free(self) -> int:
        return int(self._L.pa_bm_num_free(self._h))

    def append(self, seq: int, n: int) -> Tuple[np.ndarray, List[Tuple[int, int]]]:
        """Reserve slots for n new tokens; returns (slots, copy-on-write pairs)."""
        slots = np.empty(max(n, 1), dtype=np.int64)
        pairs = np.empty(2, dtype=np.int32)
        rc = self._check(self._L.pa_bm_append(self._h, int(seq), int(n),
                                               slots.ctypes.data, pairs.ctypes.data, 1))
        return slots[:n], [(int(pairs[0]), int(pairs[1]))] if rc else []

    def append_tokens(self, seq: int, tokens: Sequence[int]
                      ) -> Tuple[np.ndarray, List[Tuple[int, int]], int]:
        """Like append, with token ids (makes full blocks cacheable; a new sequence reuses the
        longest cached prefix).  Returns (slots, copy pairs, tokens already cached)."""
        toks = np.ascontiguousarray(np.asarray(tokens, dtype=np.int32))
        n = int(toks.shape[0])
        slots = np.empty(max(n, 1), dtype=np.int64)
        pairs = np.empty(2, dtype=np.int32)
        cached = ctypes.c_int32(0)
        rc = self._check(self._L.pa_bm_append_tokens(self._h, int(seq), toks.ctypes.data, n,
                                                      slots.ctypes.data, pairs.ctypes.data, 1,
                                                      ctypes.byref(cached)))
        return slots[:n], ([(int(pairs[0]), int(pairs[1]))] if rc else []), int(cached.value)

    def cached_prefix(self, tokens: Sequence[int]) -> int:
        """Leading tokens a new sequence with these ids would find in the prefix cache."""
        toks = np.ascontiguousarray(np.asarray(tokens, dtype=np.int32))
        return self._check(self._L.pa_bm_cached_prefix(self._h, toks.ctypes.data,
                                                        int(toks.shape[0])))

    def fork(self, parent: int, child: int) -> None:
        self._check(self._L.pa_bm_fork(self._h, int(parent), int(child)))

    def free(self, seq: int) -> None:
        self._check(self._L.pa_bm_free(self._h, int(seq)))

    def block_table(self, seq: int) -> np.ndarray:
        n = self._check(self._L.pa_bm_block_table(self._h, int(seq), None, 0))
        out = np.empty(max(n, 1), dtype=np.int32)
        self._L.pa_bm_block_table(self._h, int(seq), out.ctypes.data, n)
        return out[:n]

    def evict(self, seq: int, keep: int, width: Optional[int] = None) -> np.ndarray:
        """Reduce the sequence to `keep` positions; returns its new block table, padded with -1 to
        `width` entries (evict_keys' dst_tables row beside the table from before the call).  For
        several sequences in one evict_keys call use evict_batch: tables of separate calls may name
        each other's blocks."""
        need = -(-max(int(keep), 0) // self.block_size)
        out = np.full(max(need, 1) if width is None else int(width), -1, dtype=np.int32)
        n = self._check(self._L.pa_bm_evict(self._h, int(seq), int(keep), out.ctypes.data,
                                            int(out.shape[0])))
        return out[:n] if width is None else out

    def evict_batch(self, seqs: Sequence[int], keeps: Sequence[int],
                    width: Optional[int] = None) -> np.ndarray:
        """Reduce the sequences to keeps[i] positions each; returns their new block tables, int32
        [len(seqs), width] padded with -1: dst_tables of one evict_keys call, whose block_tables are
        the tables from before this call.  No block written for one is read for another."""
        ids = np.ascontiguousarray(np.asarray(seqs, dtype=np.int64).reshape(-1))
        kp = np.ascontiguousarray(np.asarray(keeps, dtype=np.int64).reshape(-1))
        if ids.shape != kp.shape:
            raise ValueError("seqs and keeps must have the same length")
        if width is None:
            width = max([-(-max(int(k), 0) // self.block_size) for k in kp] + [1])
        out = np.full((ids.shape[0], int(width)), -1, dtype=np.int32)
        self._check(self._L.pa_bm_evict_batch(self._h, ids.ctypes.data, kp.ctypes.data,
                                              int(ids.shape[0]), out.ctypes.data, int(width)))
        return out

    def num_tokens(self, seq: int) -> int:
        return int(self._check(self._L.pa_bm_num_tokens(self._h, int(seq))))

    def refcount(self, block: int) -> int:
        return int(self._check(self._L.pa_bm_refcount(self._h, int(block))))

    def tables(self, seqs: Sequence[int], width: Optional[int] = None) -> np.ndarray:
        """Block tables of several sequences as one int32 array padded with -1."""
        rows = [self.block_table(s) for s in seqs]
        w = max([len(r) for r in rows] + [1]) if width is None else width
        out = np.full((len(rows), w), -1, dtype=np.int32)
        for i, r in enumerate(rows):
            out[i, :len(r)] = r
        return out
