"""Paged entry cache of an HCA decode, and the plan of a batch that shares
prefixes (cf-1.com/news/5231315 §4.4: requests that share a prefix share its
cached state).

``PagedEntries`` owns the pools of some layers, the page table and the page
counts, and sequences the ``kv_pages_*`` calls on them; ``PrefixGroups`` tells
``hca_prefix_attn_fwd`` which sequences hold the same first pages.
"""
from __future__ import annotations

import torch

from . import ops


class PrefixGroups:
    """Groups of a batch's sequences: ``groups`` is a list of (members, shared),
    where the members' first ``shared`` entries lie in the same pages.  A
    sequence belongs to one group at most; those in none are not attended."""

    def __init__(self, groups, B, device="cuda"):
        off, seq, shared = [0], [], []
        for members, n in groups:
            members = [int(b) for b in members]
            if not members or int(n) < 0:
                raise ValueError("a group needs a member and a shared length >= 0")
            seq += members
            off.append(len(seq))
            shared.append(int(n))
        if any(b < 0 or b >= B for b in seq) or len(set(seq)) != len(seq):
            raise ValueError("group members must be distinct sequences of the batch")
        self.B, self.G, self.n_seq = int(B), len(shared), len(seq)
        self.off, self.seq, self.shared = (torch.tensor(v or [0], dtype=torch.int32).to(device)
                                           for v in (off, seq, shared))
        # int32 [B], 1 for a sequence of some group; None where all are
        self.attended = None
        if self.n_seq < self.B:
            listed = set(seq)
            self.attended = torch.tensor([int(b in listed) for b in range(self.B)], dtype=torch.int32).to(device)
        # what a call passes on (this object owns the tensors behind the pointers)
        self.dev = self.off.get_device()
        self.off_ptr, self.seq_ptr, self.shared_ptr = (t.data_ptr() for t in (self.off, self.seq, self.shared))

    @staticmethod
    def singles(B, device="cuda"):
        """Every sequence by itself: nothing is shared."""
        return PrefixGroups([([b], 0) for b in range(B)], B, device=device)


class PagedEntries:
    """Pools [L, N, P, D] of N pages of P entries for L layers, shared by R rows
    (sequences) of up to max_entries entries.

    Row lists and entry counts are device int32 tensors (or host lists, which
    are copied to the device first); nothing is read back, so every call can be
    captured in a CUDA graph when given tensors.  ``status`` is the device word
    in which a refused call records why (``layer.raise_on_status``)."""

    def __init__(self, L, N, P, D, R, max_entries, dtype=torch.bfloat16, device="cuda"):
        self.P, self.R, self.N = P, R, N
        self.max_pages = max(1, -(-max_entries // P))
        self.pool = torch.zeros((L, N, P, D), dtype=dtype, device=device)
        self.refcount = torch.zeros((N,), dtype=torch.int32, device=device)
        self.table = torch.full((R, self.max_pages), -1, dtype=torch.int32, device=device)
        self.held = torch.zeros((R,), dtype=torch.int32, device=device)
        self.n_live = torch.zeros((1,), dtype=torch.int32, device=device)
        self.status = torch.zeros((1,), dtype=torch.int32, device=device)
        # one list item per row at most does useful work
        self.ws = torch.empty((ops.kv_pages_workspace_size(N, R) // 4,), dtype=torch.int32, device=device)

    def _list(self, v, stream=None):
        if torch.is_tensor(v):
            return v
        # The copy lives until the call returns, its kernels read it later: it is made on
        # their stream, where its memory comes back into use behind them alone.
        with torch.cuda.stream(stream):
            return torch.tensor([int(x) for x in v], dtype=torch.int32).to(self.pool.device)

    def _rows(self, v, stream=None):
        v = self._list(v, stream)
        if v.numel() > self.R:
            raise ValueError(f"a list of {v.numel()} rows for a cache of {self.R}")
        return v

    def reserve(self, rows, n_entries, stream=None):
        """Grow rows so that they hold n_entries entries each."""
        ops.kv_pages_reserve(self._rows(rows, stream), self._list(n_entries, stream), self.P, self.table, self.held,
                             self.refcount, self.ws, self.status, stream)

    def fork(self, src, dst, n_entries, stream=None):
        """Empty rows dst take the first n_entries entries of rows src."""
        ops.kv_pages_fork(self._list(src, stream), self._rows(dst, stream), self._list(n_entries, stream), self.pool,
                          self.table, self.held, self.refcount, self.ws, self.status, stream)

    def forked(self):
        """Whether the cache's last call, a fork, was made (a refused one changes
        nothing): bool [1] on the device."""
        return self.ws[:1] > 0

    def free(self, rows, stream=None):
        """Rows give up their pages."""
        ops.kv_pages_free(self._rows(rows, stream), self.table, self.held, self.refcount, self.status, stream)

    def compact(self, stream=None):
        """Move the pages in use to the lowest ids; n_live receives their number."""
        ops.kv_pages_compact(self.pool, self.table, self.held, self.refcount, self.n_live, self.ws, stream=stream)
