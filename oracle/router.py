"""Balance loss, per-expert counts and the gradients of router and combine,
written out in float64 (the formulas of include/moe.h).

Pins (tests/test_router_cpu.py): every gradient against central differences
of the value it belongs to; a uniform routing has loss 1; sequences with no
token, masked tokens and rows of -inf by hand.
"""
from __future__ import annotations

import numpy as np


def softmax_rows(logits):
    """p [T, E] and lse [T]; a row of nothing but -inf has p = 0 and lse = 0."""
    l = np.asarray(logits, dtype=np.float64)
    top = l.max(axis=1, keepdims=True) if l.size else np.zeros((l.shape[0], 1))
    dead = np.isneginf(top)
    z = np.where(dead, 0.0, np.exp(l - np.where(dead, 0.0, top)))
    total = z.sum(axis=1, keepdims=True)
    p = np.divide(z, total, out=np.zeros_like(z), where=~dead)
    lse = np.where(dead, 0.0, np.where(dead, 0.0, top) + np.log(np.where(dead, 1.0, total)))
    return p, lse[:, 0]


def tokens_of(T, seq_offsets=None, mask=None):
    """The tokens of each sequence, as lists of indices."""
    off = [0, T] if seq_offsets is None else [int(v) for v in seq_offsets]
    return [[t for t in range(a, b) if mask is None or mask[t]] for a, b in zip(off[:-1], off[1:])]


def balance(logits, idx, seq_offsets=None, mask=None):
    """loss [2], counts [S, E], prob [S, E], coef [S + 1]."""
    l = np.asarray(logits)
    T, E = l.shape
    k = np.asarray(idx).shape[1]
    seqs = tokens_of(T, seq_offsets, mask)
    some = sum(len(t) > 0 for t in seqs)
    n = sum(len(t) for t in seqs)
    counts = np.zeros((len(seqs), E), dtype=np.int64)
    prob = np.zeros((len(seqs), E))
    coef = np.zeros(len(seqs) + 1)
    coef[-1] = 1.0 / max(n, 1)
    loss = np.zeros(2)
    for s, t in enumerate(seqs):
        if not t:
            continue
        p, lse = softmax_rows(l[t])
        prob[s] = p.mean(axis=0)
        for e in np.asarray(idx)[t].ravel():
            if 0 <= e < E:
                counts[s, e] += 1
        coef[s] = E / (k * len(t) ** 2 * some)
        loss[0] += E / (k * len(t) * some) * (counts[s] * prob[s]).sum()
        loss[1] += (lse ** 2).sum() / n
    return loss, counts, prob, coef


def router_backward(logits, idx, gate=None, dgate=None, counts=None, coef=None, dloss=None, seq_offsets=None,
                    mask=None):
    l = np.asarray(logits)
    T, E = l.shape
    out = np.zeros((T, E))
    for s, ts in enumerate(tokens_of(T, seq_offsets, mask)):
        for t in ts:
            if dloss is not None:
                p, lse = softmax_rows(l[t:t + 1])
                c = np.asarray(counts[s], dtype=np.float64)
                out[t] = (dloss[0] * coef[s] * p[0] * (c - (c * p[0]).sum())
                          + 2 * dloss[1] * coef[-1] * lse[0] * p[0])
            if dgate is not None:
                g, dg = np.asarray(gate[t], dtype=np.float64), np.asarray(dgate[t], dtype=np.float64)
                for j, e in enumerate(idx[t]):
                    if 0 <= e < E:
                        out[t, e] += g[j] * (dg[j] - (g * dg).sum())
    return out


def combine_backward(y_perm, idx, gate, inv_perm, slot, dout, dy0):
    """dgate [T, k] and dy_perm (dy0 with the written rows replaced)."""
    T, k = np.asarray(idx).shape
    dgate = np.zeros((T, k))
    dy = np.array(dy0, dtype=np.float64)
    n = T * k
    for t in range(T):
        for j in range(k):
            q, e = int(inv_perm[t * k + j]), int(idx[t, j])
            if not 0 <= q < n or (slot is not None and (not 0 <= e < len(slot) or slot[e] < 0)):
                continue
            dgate[t, j] = np.asarray(dout[t], dtype=np.float64) @ np.asarray(y_perm[q], dtype=np.float64)
            dy[q] = float(gate[t, j]) * np.asarray(dout[t], dtype=np.float64)
    return dgate, dy
