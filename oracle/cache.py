"""The target's cache in plain numpy and Python (oracle side): rotary positions of packed rows, causal attention of
new rows over the rows before them, and the life of a paged cache's blocks.

Rotary positions (Su et al., RoFormer): pair j of a head's leading rot elements turns by position * f_j, f_j =
theta^(-2j / rot); scaled kinds as `frequencies` states.  Attention: new row i of n, with L rows in the cache
(the new ones included), stands at p = L - n + i and sees the keys max(0, p - window + 1) .. p.

Pages: a block is free when no table entry maps it; the lowest free ids go first, in sequence order.  Everything is
one step at a time here: a dictionary of contents shows what each sequence reads back.
"""
from __future__ import annotations

import math
from typing import Dict, List, Optional, Sequence, Tuple

import numpy as np


def frequencies(rot: int, theta: float, kind: str = "none", factor: float = 1.0, low: float = 0.0, high: float = 0.0,
                original: int = 0) -> np.ndarray:
    """Radians a position of each pair.  linear: f / factor.  bands: kept from `high` turns in `original` positions
    on, slowed up to `low`, linear in the turns between.  ramp: kept up to the (floored) pair that makes `high` turns,
    slowed from the (ceiled) pair that makes `low`, linear in the pair number between."""
    out = []
    for j in range(rot // 2):
        f = theta ** (-2.0 * j / rot)
        keep = 1.0
        if kind == "linear":
            keep = 0.0
        elif kind == "bands":
            keep = (original * f / (2.0 * math.pi) - low) / (high - low)
        elif kind == "ramp":
            pair = lambda turns: rot * math.log(original / (2.0 * math.pi * turns)) / (2.0 * math.log(theta))
            lo, hi = max(math.floor(pair(high)), 0), min(math.ceil(pair(low)), rot - 1)
            keep = 1.0 - (j - lo) / max(hi - lo, 1e-3)
        keep = min(max(keep, 0.0), 1.0)
        out.append(keep * f + (1.0 - keep) * f / factor)
    return np.array(out, dtype=np.float64)


def rotate(x: np.ndarray, pos: Sequence[int], freq: np.ndarray, interleaved: bool, mscale: float = 1.0) -> np.ndarray:
    """x [n, H, dh] at positions pos [n]; 2 len(freq) leading elements rotate."""
    x = np.asarray(x, dtype=np.float64)
    half = len(freq)
    first = np.arange(half) * 2 if interleaved else np.arange(half)
    second = first + 1 if interleaved else first + half
    ang = np.asarray(pos, dtype=np.float64)[:, None, None] * freq
    c, s = mscale * np.cos(ang), mscale * np.sin(ang)
    y = x.copy()
    y[..., first] = x[..., first] * c - x[..., second] * s
    y[..., second] = x[..., second] * c + x[..., first] * s
    return y


def rows_of(row_start: Sequence[int], n_rows: int) -> List[Tuple[int, int]]:
    """The packed rows [lo, hi) of each request by its own two starts; (0, 0), none, where they break
    0 <= lo <= hi <= n_rows."""
    return [(a, z) if 0 <= a <= z <= n_rows else (0, 0) for a, z in zip(row_start, row_start[1:])]


def chunk_attention(q: np.ndarray, k: np.ndarray, v: np.ndarray, scale: float, window: int = 0
                    ) -> Tuple[np.ndarray, np.ndarray, np.ndarray]:
    """q [n, Hq, dh], k and v [L, Hkv, dh] with the new rows last.  Returns the output, and for error bounds the
    probability-weighted mean of |v| and, per row and head, the largest sum |q_i k_i| scale of a visible key."""
    q, k, v = (np.asarray(t, dtype=np.float64) for t in (q, k, v))
    n, Hq, dh = q.shape
    L, Hkv = k.shape[0], k.shape[1]
    G = Hq // Hkv
    out, mean_abs, reach = np.zeros((n, Hq, dh)), np.zeros((n, Hq, dh)), np.zeros((n, Hq))
    pos = L - n + np.arange(n)
    j = np.arange(L)
    sees = j[None, :] <= pos[:, None]
    if window:
        sees &= j[None, :] > pos[:, None] - window
    any_ = sees.any(1)
    for h in range(Hq):
        kh, vh = k[:, h // G], v[:, h // G]
        s = np.where(sees, q[:, h] @ kh.T * scale, -np.inf)
        m = np.where(any_, s.max(1, initial=-np.inf), 0.0)
        p = np.exp(s - m[:, None])
        z = p.sum(1)
        p /= np.where(z == 0, 1.0, z)[:, None]
        out[:, h], mean_abs[:, h] = p @ vh, p @ np.abs(vh)
        reach[:, h] = np.where(sees, np.abs(q[:, h]) @ np.abs(kh).T * scale, 0.0).max(1, initial=0.0)
    return out, mean_abs, reach


class OutOfBlocks(Exception):
    pass


class Pages:
    """Tables, lengths and counts of a paged cache."""

    def __init__(self, n_seqs: int, per_seq: int, block_size: int, n_blocks: int):
        self.n_seqs, self.per, self.bs, self.n_blocks = n_seqs, per_seq, block_size, n_blocks
        self.table = [[-1] * per_seq for _ in range(n_seqs)]
        self.len = [0] * n_seqs
        self.ref = [0] * n_blocks

    def _blocks(self, rows: int) -> int:
        return -(-rows // self.bs)

    def _drop(self, s: int, c: int):
        if self.table[s][c] >= 0:
            self.ref[self.table[s][c]] -= 1
            self.table[s][c] = -1

    def fork(self, src: Sequence[int], dst: Sequence[int]) -> List[int]:
        """Returns the pairs that were refused."""
        refused = []
        for i, (s, d) in enumerate(zip(src, dst)):
            if not (0 <= s < self.n_seqs and 0 <= d < self.n_seqs) or d in src or d in list(dst)[:i]:
                refused.append(i)
        for i, (s, d) in enumerate(zip(src, dst)):
            if i in refused:
                continue
            for c in range(self.per):
                self._drop(d, c)
            for c in range(self._blocks(self.len[s])):
                self.table[d][c] = self.table[s][c]
                self.ref[self.table[s][c]] += 1
            self.len[d] = self.len[s]
        return refused

    def release(self, keep: Sequence[int]):
        for s, k in enumerate(keep):
            if k >= 0:
                for c in range(self._blocks(k), self.per):
                    self._drop(s, c)
                self.len[s] = min(self.len[s], k)

    def reserve(self, n_new: Sequence[int]) -> List[Tuple[int, int, int]]:
        """Returns the copies (block, to block, rows).  Raises OutOfBlocks with nothing changed."""
        writers: Dict[int, List[int]] = {}
        for s, n in enumerate(n_new):
            if n > 0 and self.len[s] + n > self.per * self.bs:
                raise OutOfBlocks
            if n > 0 and self.len[s] % self.bs:
                writers.setdefault(self.table[s][self.len[s] // self.bs], []).append(s)
        copying = set()
        for blk, who in writers.items():
            if self.ref[blk] > 1:
                copying |= set(who[:-1] if len(who) == self.ref[blk] else who)
        wanted = []                                    # (sequence, column, copied block or -1)
        for s, n in enumerate(n_new):
            if n <= 0:
                continue
            if s in copying:
                wanted.append((s, self.len[s] // self.bs, self.table[s][self.len[s] // self.bs]))
            for c in range(self._blocks(self.len[s]), self._blocks(self.len[s] + n)):
                if self.table[s][c] < 0:
                    wanted.append((s, c, -1))
        free = [b for b in range(self.n_blocks) if self.ref[b] == 0]
        if len(wanted) > len(free):
            raise OutOfBlocks
        copies = []
        for (s, c, old), blk in zip(wanted, free):
            if old >= 0:
                self.ref[old] -= 1
                copies.append((old, blk, self.len[s] % self.bs))
            self.table[s][c] = blk
            self.ref[blk] += 1
        return copies

    def compact(self) -> List[Tuple[int, int]]:
        """Returns the moves (block, to block)."""
        live = [b for b in range(self.n_blocks) if self.ref[b] > 0]
        u = len(live)
        moves = list(zip([b for b in live if b >= u], [b for b in range(u) if self.ref[b] == 0]))
        to = dict(moves)
        for row in self.table:
            for c, b in enumerate(row):
                row[c] = to.get(b, b)
        for a, z in moves:
            self.ref[z], self.ref[a] = self.ref[a], 0
        return moves
