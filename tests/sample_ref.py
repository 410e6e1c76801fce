"""Sampled decoding in 64 bits, position by position, as gdn.h defines it."""
import math

import numpy as np


def values(bits):
    """bf16 patterns (uint16) as float64."""
    return (np.asarray(bits, np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def draw(x, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(token, logp, distance of u's place to the nearest border, as a share of the mass) of one position x [V]."""
    x = np.asarray(x, np.float64)
    order = np.argsort(np.where(np.isnan(x), np.inf, -x), kind="stable")
    order = order[~np.isnan(x[order])]
    if order.size == 0:
        return 0, -math.inf, 1.0
    v = x[order]
    if v[0] == -math.inf:
        return int(order[0]), -math.inf, 1.0
    if not temperature > 0:
        return int(order[0]), 0.0, 1.0
    order, v = order[v > -math.inf], v[v > -math.inf]
    if v[0] == math.inf:
        w = (v == math.inf).astype(np.float64)
    elif temperature == math.inf:
        w = np.ones_like(v)
    else:
        w = np.exp((v - v[0]) / np.float64(np.float32(temperature)))
    keep = np.ones(v.size, bool)
    if min_p > 0:
        keep = w >= np.float64(np.float32(min(min_p, 1.0)))
    n = int(keep.sum())
    if top_k > 0:
        n = min(n, top_k)
    w = w[:n]
    if top_p < 1:
        run = np.cumsum(w)
        n = 1 + int((run[:-1] < max(0.0, np.float64(np.float32(top_p))) * run[-1]).sum())
        w = w[:n]
    run = np.cumsum(w)
    u = np.float64(np.float32(u))
    at = min(max(u, 0.0) if u == u else 0.0, 1 - 2.0 ** -24) * run[-1]  # the nearest fp32 in [0, 1)
    j = min(int((run <= at).sum()), int(np.flatnonzero(w > 0)[-1]))
    border = float(np.min(np.abs(run - at))) / run[-1]
    return int(order[j]), -math.log1p((run[-1] - w[j]) / w[j]), border


def accept(tokens, draft, active):
    """keep and next of tokens [B][T]."""
    B, T = tokens.shape
    keep, nxt = np.zeros(B, np.int32), np.full(B, -1, np.int32)
    for b in range(B):
        if active[b]:
            k = 1
            while k < T and draft[b, k] == tokens[b, k - 1]:
                k += 1
            keep[b], nxt[b] = k, tokens[b, k - 1]
    return keep, nxt
