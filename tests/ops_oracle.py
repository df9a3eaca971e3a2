"""The serving operators in 64 bits on the CPU, straight from their
definitions: what the kernels' tests compare against."""

from __future__ import annotations

import math

import numpy as np
import torch

PAGE = 64


def rotate(x, positions, inv_freq, interleaved, magnitude):
    """x [tokens][heads][hd], rotated; also the sum |a| + |b| of each element's pair."""
    x = x.double()
    half = inv_freq.numel()
    out, reach = x.clone(), torch.zeros_like(x)
    for i in range(half):
        lo, hi = (2 * i, 2 * i + 1) if interleaved else (i, half + i)
        angle = positions.double() * float(inv_freq[i])
        cos, sin = angle.cos()[:, None] * magnitude, angle.sin()[:, None] * magnitude
        a, b = x[..., lo], x[..., hi]
        out[..., lo], out[..., hi] = a * cos - b * sin, b * cos + a * sin
        reach[..., lo] = reach[..., hi] = (a.abs() + b.abs()) * magnitude
    return out, reach


def attention(q, k_pool, v_pool, table, positions, group_start, prefix_lens, scale):
    """(out, lse, sum of weight x |v|, largest |score|), rows of no group NaN."""
    b, hq, hd = q.shape
    hkv = k_pool.shape[1]
    g = hq // hkv
    out = torch.full((b, hq, hd), math.nan, dtype=torch.float64)
    lse = torch.full((b, hq), math.nan, dtype=torch.float64)
    mass = torch.zeros((b, hq, hd), dtype=torch.float64)
    high = torch.zeros((b, hq), dtype=torch.float64)
    for n in range(len(prefix_lens)):
        for i in range(group_start[n], group_start[n + 1]):
            seen = positions[i] + 1
            if seen <= 0:
                out[i], lse[i] = 0.0, -math.inf
                continue
            ks, vs = [], []
            for t in range(seen):
                row = group_start[n] if t < prefix_lens[n] else i
                page = int(table[row, t // PAGE])
                ks.append(k_pool[page, :, t % PAGE])
                vs.append(v_pool[page, :, t % PAGE])
            k, v = torch.stack(ks).double(), torch.stack(vs).double()     # [seen][hkv][hd]
            for h in range(hq):
                s = (k[:, h // g] @ q[i, h].double()) * scale
                lse[i, h] = torch.logsumexp(s, 0)
                w = (s - lse[i, h]).exp()
                out[i, h] = w @ v[:, h // g]
                mass[i, h] = w @ v[:, h // g].abs()
                high[i, h] = s.abs().max()
    return out, lse, mass, high


def kept(x, temperature, k, p, m):
    """(ids in descending order of logit, their weights), the kept ones only."""
    x = np.where(np.isnan(x), -np.inf, x.astype(np.float64))
    if not (x > -np.inf).any():
        return np.zeros(0, dtype=np.int64), np.zeros(0)
    top = x.max()
    if top == np.inf:
        w = (x == np.inf).astype(np.float64)
    else:
        w = np.exp((x - top) / temperature)
    order = np.lexsort((np.arange(len(x)), -x))
    order = order[x[order] > -np.inf]
    if k > 0:
        order = order[:k]
    ws = w[order]
    if p < 1:
        before = np.concatenate(([0.0], np.cumsum(ws)[:-1]))
        n = max(1, int((before < p * ws.sum()).sum()))
        order, ws = order[:n], ws[:n]
    n = max(1, int((ws >= m).sum()))
    return order[:n], ws[:n]


def sample(x, u, temperature=1.0, k=0, p=1.0, m=0.0):
    """(token, log-probability) of one row."""
    x = np.asarray(x, dtype=np.float64)
    if temperature == 0:
        y = np.where(np.isnan(x), -np.inf, x)
        if not (y > -np.inf).any():
            return -1, -math.inf
        return int(np.argmax(y)), 0.0
    ids, w = kept(x, float(temperature), k, float(p), float(m))
    if len(ids) == 0:
        return -1, -math.inf
    by_id = np.argsort(ids)
    cum = np.cumsum(w[by_id])
    j = int(np.searchsorted(cum, float(u) * cum[-1], side="right"))
    j = min(j, len(ids) - 1)
    return int(ids[by_id[j]]), float(math.log(w[by_id[j]] / cum[-1]))
