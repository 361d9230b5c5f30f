"""Bounds on the verify's errors that stay below what a wrong page of values does over long contexts,
and values made for showing such pages."""
from __future__ import annotations

import numpy as np
import torch


def verify_bounds(out, A, S, keys, d, bf16):
    """Absolute bound on the error of out, whose exact value is ``out``; A and S as attn_ref.attention
    gives them.

    Scores: a sum of d products in fp32, |ds| <= es = (d + 8) 2^-24 S, so each weight is off by a relative
    es + 2^-21 (the exponential's argument and value), and out by twice that of A.
    Sums, bf16: an accumulator of the values' product takes 8 MMAs for 64 keys (16 keys each, the weights'
    first terms, then their second); an MMA's sum of 16 products and the accumulator is taken as off by
    2^-22 of their magnitudes (it need not round as separate additions do): keys 2^-25, and 16 MMAs more
    for the joined parts.  The denominator adds a few terms a tile, keys 2^-30, and 32 additions.
    Sums, fp32: one rounding per key and column, 2^-24; as many parts.
    bf16 besides: a weight's two terms leave 2^-16 of it, and the output is rounded once, 2^-8 of itself."""
    es = (d + 8) * 2.0 ** -24 * S
    rel = 2 * es + 2.0 ** -20 + ((1.05 * keys + 200) * 2.0 ** -25 + 2.0 ** -16 if bf16 else (1.05 * keys + 100) * 2.0 ** -24)
    return 1.01 * (A * rel[..., None] + (2.0 ** -8 * np.abs(out) if bf16 else 0.0)) + 1e-30


def page_marks(tokens, Hkv, d, group, g):
    """Values [tokens, Hkv, d] >= 0 whose columns each belong to some groups of ``group`` neighbouring tokens:
    group i has one value per token, in column (i + 5 h) mod d.  Nothing cancels in a sum over them, so a
    group's share of its column is its share of the softmax there."""
    v = torch.zeros(tokens, Hkv, d)
    at = torch.arange(tokens) // group
    for h in range(Hkv):
        v[torch.arange(tokens), h, (at + 5 * h) % d] = 1 + torch.rand(tokens, generator=g)
    return v
