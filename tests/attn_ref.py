"""Plain 64-bit forms of the attention-layer operators (include/gdnattn.h), written from
their definitions, and the seeded inputs of their tests.  numpy on the CPU."""
from __future__ import annotations

import math

import numpy as np
import torch


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().cpu().double().numpy()


# ------------------------------------------------------------------ cache inputs
class CacheCase:
    """A cache of ``layers`` layers whose sequence b holds lens[b] committed tokens and has
    pages for ``room`` more, in a random order, under a random slot map.  Rows that no token
    owns hold NaN (keys) and infinity (values); block-table entries past the owned ones are
    out of range."""

    def __init__(self, lens, room, Hkv, d, page, dtype, layers=1, seed=0, spare=3, extra_slots=2):
        g = self.g = torch.Generator().manual_seed(seed)
        self.lens, self.page, self.Hkv, self.d, self.layers = list(lens), page, Hkv, d, layers
        self.B, self.dtype = len(self.lens), dtype
        owned = [-(-(x + room) // page) for x in self.lens]
        self.n_page, self.n_slot = sum(owned) + spare, self.B + extra_slots
        self.max_pages = max(owned + [1]) + 1
        order = torch.randperm(self.n_page, generator=g)
        self.state_idx = torch.randperm(self.n_slot, generator=g)[:self.B].to(torch.int32)
        shape = (layers, self.n_page, Hkv, page, d)
        k, v = torch.full(shape, float("nan")), torch.full(shape, float("inf"))
        self.block_table = torch.full((self.n_slot, self.max_pages), 1 << 30, dtype=torch.int32)
        self.seq_len = torch.zeros(self.n_slot, dtype=torch.int32)
        self.n_owned = torch.zeros(self.n_slot, dtype=torch.int32)
        self.ref = torch.zeros(self.n_page, dtype=torch.int32)
        at = 0
        for b, n in enumerate(owned):
            s, ids = int(self.state_idx[b]), order[at:at + n]
            at += n
            self.block_table[s, :n] = ids.to(torch.int32)
            self.seq_len[s], self.n_owned[s] = self.lens[b], n
            self.ref[ids] = 1
            tokens = self.lens[b] + room
            for x, scale in ((k, 1.3), (v, 1.0)):
                rows = scale * torch.randn(layers, tokens, Hkv, d, generator=g)
                pos = torch.arange(tokens)
                x[:, ids[pos // page], :, pos % page] = rows.transpose(0, 1)
        self.k, self.v = k.to(dtype).contiguous(), v.to(dtype).contiguous()
        self.free_list = torch.zeros(self.n_page, dtype=torch.int32)
        self.free_list[:self.n_page - at] = order[at:].to(torch.int32)
        self.free_count = torch.tensor([self.n_page - at], dtype=torch.int32)

    def init(self):
        return {n: getattr(self, n) for n in ("k", "v", "block_table", "seq_len", "n_owned", "ref",
                                              "free_list", "free_count")}

    def dims(self, lib):
        return lib.PageDims(n_slot=self.n_slot, max_pages=self.max_pages, n_page=self.n_page, page=self.page,
                            n_layer=self.layers, Hkv=self.Hkv, d=self.d,
                            dtype=lib.DTYPE_BF16 if self.dtype == torch.bfloat16 else lib.DTYPE_F32)

    def cell(self, b, token):
        """Page and row of a token of sequence b."""
        s = int(self.state_idx[b])
        return int(self.block_table[s, token // self.page]), token % self.page

    def rows(self, x, b, n, layer=0):
        """[n, Hkv, d] first n tokens of sequence b of a cache tensor."""
        s, pos = int(self.state_idx[b]), torch.arange(n)
        ids = self.block_table[s][pos // self.page].long()
        return f64(x[layer][ids, :, pos % self.page])


# ------------------------------------------------------------------------ trees
def random_parents(B, T, g, width=4):
    t = torch.arange(T)
    back = 1 + torch.randint(0, width, (B, T), generator=g)
    p = torch.where(t == 0, -1, (t - back).clamp(min=-1))
    return p.to(torch.int32)


def ancestors(parents, n):
    """Words and depths of the first n tokens of one tree (lists of Python integers)."""
    words, depth = [], []
    for t in range(n):
        p = int(parents[t])
        words.append((words[p] if p >= 0 else 0) | 1 << t)
        depth.append(depth[p] + 1 if p >= 0 else 0)
    return words, depth


def as_int64(words):
    return [w - (1 << 64) if w >= 1 << 63 else w for w in words]


# ----------------------------------------------------------------------- verify
def attention(q, k, v, words, ln, scale):
    """q [n, Hq, d], k, v [ln + n, Hkv, d], words: one integer per row (bit u: draft token u is
    seen).  Returns out, lse, and per element the quantities the error bounds need:
    A = sum_j p_j |v_j| / l and, per row, S = max_j sum_i |q_i k_ji| scale over seen j."""
    n, Hq, d = q.shape
    Hkv = k.shape[1]
    G, total = Hq // Hkv, ln + n
    out, A = np.zeros((n, Hq, d)), np.zeros((n, Hq, d))
    lse, S = np.full((n, Hq), -np.inf), np.zeros((n, Hq))
    for t in range(n):
        seen = np.concatenate([np.ones(ln, bool), np.array([(words[t] >> u) & 1 for u in range(n)], bool)])
        if not seen.any():
            continue
        for h in range(Hq):
            kk, vv = k[:total, h // G][seen], v[:total, h // G][seen]
            s = kk @ q[t, h] * scale
            m = s.max()
            p = np.exp(s - m)
            l = p.sum()
            out[t, h], A[t, h] = p @ vv / l, p @ np.abs(vv) / l
            lse[t, h], S[t, h] = m + math.log(l), (np.abs(kk) @ np.abs(q[t, h])).max() * scale
    return out, lse, A, S


def verify_bounds(A, S, lse, keys, d, bf16):
    """Absolute bounds on the errors of out and lse.  A score is a sum of d exact products
    (bf16) or d fused multiply-adds (fp32) in fp32, scaled and exponentiated with relative
    error 2^-22: |ds| <= (d + 8) 2^-24 S.  The sums over the keys add keys 2^-24.  With bf16
    inputs the output is rounded once, a relative 2^-8, which the second product's roundings
    (2^-16) hardly add to."""
    es = (d + 8) * 2.0 ** -24 * S
    rel = 2 * es + (keys + 16) * 2.0 ** -23
    if bf16:
        rel = rel + 2.0 ** -8
    finite = np.where(np.isfinite(lse), np.abs(lse), 0.0)
    return A * rel[..., None] * 1.01 + 1e-30, es + (keys + 16) * 2.0 ** -24 + 2.0 ** -21 * (1 + finite)


# ------------------------------------------------------------------------ stage
def norm_rotate(x, w, eps, cos, sin, rot, pairs):
    """x [H, d] normalised, weighted, its first rot dims turned; and a bound on the size of
    the terms each element is a difference of."""
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w
    out, size = y.copy(), np.abs(y)
    i = np.arange(0, rot, 2) if pairs else np.arange(rot // 2)
    j = i + 1 if pairs else i + rot // 2
    out[:, i], out[:, j] = y[:, i] * cos - y[:, j] * sin, y[:, j] * cos + y[:, i] * sin
    both = np.abs(y[:, i]) + np.abs(y[:, j])
    size[:, i], size[:, j] = both, both
    return out, size


# ------------------------------------------------------------------------- pool
class Pool:
    """The page pool, row by row, in Python integers."""

    BAD_SLOT, BAD_LEN, NO_ROOM, BAD_PAGE, NO_PAGES = 8, 4, 2, 64, 512

    def __init__(self, case):
        self.table = case.block_table.clone().numpy()
        self.len, self.owned = case.seq_len.clone().numpy(), case.n_owned.clone().numpy()
        self.ref, self.list = case.ref.clone().numpy(), case.free_list.clone().numpy()
        self.count, self.page, self.max_pages = int(case.free_count), case.page, case.max_pages
        self.k, self.v, self.status = case.k.clone(), case.v.clone(), 0

    def _slot_bad(self, s):
        return not 0 <= s < len(self.len)

    def _pop(self):
        self.count -= 1
        return int(self.list[self.count])

    def reserve(self, slots, extra):
        out = False
        for s in slots:
            if self._slot_bad(s):
                self.status |= self.BAD_SLOT
                continue
            want = -(-(int(self.len[s]) + extra) // self.page)
            if want > self.max_pages:
                self.status |= self.NO_ROOM
                continue
            need = max(0, want - int(self.owned[s]))
            if need and (out or need > self.count):
                out = True
                self.status |= self.NO_PAGES
                continue
            for _ in range(need):
                p = self._pop()
                self.table[s, self.owned[s]] = p
                self.ref[p] = 1
                self.owned[s] += 1

    def fork(self, src, dst):
        copies = []
        for a, z in zip(src, dst):
            pair = (-1, -1)
            if self._slot_bad(a) or self._slot_bad(z) or self.owned[z]:
                self.status |= self.BAD_SLOT
            else:
                full, tail = divmod(int(self.len[a]), self.page)
                if tail and self.count == 0:
                    self.status |= self.NO_PAGES
                else:
                    self.table[z, :full] = self.table[a, :full]
                    for p in self.table[a, :full]:
                        self.ref[p] += 1
                    if tail:
                        p = self._pop()
                        pair = (int(self.table[a, full]), p)
                        self.table[z, full], self.ref[p] = p, 1
                    self.len[z], self.owned[z] = self.len[a], full + (1 if tail else 0)
            copies.append(pair)
        for a, z in copies:
            if a >= 0:
                self.k[:, z], self.v[:, z] = self.k[:, a], self.v[:, a]
        return copies

    def release(self, slots):
        for s in slots:
            if self._slot_bad(s):
                self.status |= self.BAD_SLOT
                continue
            for c in range(int(self.owned[s])):
                p = int(self.table[s, c])
                self.ref[p] -= 1
                if self.ref[p] == 0:
                    self.list[self.count] = p
                    self.count += 1
            self.len[s] = self.owned[s] = 0
