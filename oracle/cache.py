"""The 4-bit key/value cache in plain numpy float64: what its operators compute,
written from their definition.

A cache is held as the values that it stands for, kv[0 or 1][page, head, row,
channel], and the sums of the keys of each page; ``tile_values`` decodes the
bytes of a cache tile from the documented layout, byte by byte.
"""
from __future__ import annotations

import numpy as np
import torch


def bf16(x: np.ndarray) -> np.ndarray:
    """Nearest bfloat16 (half to even) of float32 values, as float64."""
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).bfloat16().double().numpy()


def quantise(x: np.ndarray):
    """Codes, scale and zero of x [..., D] (float32 values): one scale and zero
    for each group of 64 channels. The operator is defined in float32 steps."""
    f = np.float32
    with np.errstate(all="ignore"):
        g = np.asarray(x, f).reshape(*x.shape[:-1], -1, 64)
        zero = bf16(g.min(-1))
        rng = (g.max(-1) - zero.astype(f)).astype(f)
        scale = bf16(rng * f(1 / 15))
        scale[scale < 2.0 ** -126] = 0
        bad = ~np.isfinite(rng)
        inv = np.where(scale > 0, 1 / np.where(scale > 0, scale, 1), 0).astype(f)
        t = ((g - zero.astype(f)[..., None]).astype(f) * inv[..., None]).astype(f)
        code = np.clip(np.rint(np.where(bad[..., None], 0, t)), 0, 15).astype(np.int64)
    scale[bad] = zero[bad] = np.nan
    return code.reshape(x.shape), scale, zero


def held(x: np.ndarray) -> np.ndarray:
    """What the cache holds of x [..., D]."""
    code, scale, zero = quantise(x)
    return (zero[..., None] + scale[..., None] * code.reshape(*scale.shape, 64)).reshape(x.shape)


def tile_values(tile: np.ndarray):
    """Keys and values [64, D] of the bytes of a cache tile [72 D], by the layout's formulas."""
    D = tile.shape[0] // 72
    sz = torch.from_numpy(tile[64 * D:].copy()).view(torch.bfloat16).double().numpy().reshape(2, 64, D // 64, 2)
    k, v = np.empty((64, D)), np.empty((64, D))
    for r in range(64):
        for c in range(D):
            kb = r * (D // 2) + ((c % 32) // 8) * (D // 8) + (c // 32) * 4 + (c % 8) // 2
            vb = (32 * D + (r // 2) * D + (((c % 32) // 4) ^ (2 * ((r // 2) % 4))) * (D // 8) + (c // 32) * 4
                  + (r % 2) * 2 + (c % 4) // 2)
            for n, (out, byte) in enumerate(((k, kb), (v, vb))):
                s, z = sz[n, r, c // 64]
                out[r, c] = z + s * ((int(tile[byte]) >> (4 * (c % 2))) & 15)
    return k, v


def new_cache(num_pages: int, H_kv: int, D: int, block_size: int):
    """An unwritten cache: NaN everywhere, so that whatever reads a token that was never written shows."""
    return {"kv": np.full((2, num_pages, H_kv, block_size, D), np.nan), "k_sum": np.full((num_pages, H_kv, D), np.nan)}


def _page(table, num_pages, b, block):
    if not 0 <= block < table.shape[1]:
        return -1
    p = int(table[b, block])
    return p if 0 <= p < num_pages else -1


def _step(start, count, b, T, capacity):
    s, c = int(start[b]), T if count is None else int(count[b])
    if s < 0:
        return 0, 0
    return min(s, capacity), max(0, min(c, T))


def write(cache, k, v, table, start, count=None):
    """k, v [B, T, H_kv, D] into the cache at start[b] + t; k_sum of every page that got a token."""
    _, pages, _, bs, _ = cache["kv"].shape
    B, T = k.shape[:2]
    for b in range(B):
        s, n = _step(start, count, b, T, table.shape[1] * bs)
        for block in range(s // bs, (s + n - 1) // bs + 1 if n else 0):
            p = _page(table, pages, b, block)
            if p < 0:
                continue
            lo, hi = max(s, block * bs), min(s + n, (block + 1) * bs)
            for i, x in enumerate((k, v)):
                cache["kv"][i, p, :, lo - block * bs:hi - block * bs] = held(x[b, lo - s:hi - s]).transpose(1, 0, 2)
            cache["k_sum"][p] = cache["kv"][0, p, :, :hi - block * bs].sum(1)


def read(cache, table, start, T, count=None, k_out=None, v_out=None):
    _, pages, Hk, bs, D = cache["kv"].shape
    B = table.shape[0]
    out = [np.zeros((B, T, Hk, D)) if x is None else x.copy() for x in (k_out, v_out)]
    for b in range(B):
        s, n = _step(start, count, b, T, table.shape[1] * bs)
        for t in range(n):
            p = _page(table, pages, b, (s + t) // bs)
            for i in range(2):
                out[i][b, t] = cache["kv"][i, p, :, (s + t) % bs] if p >= 0 else 0.0
    return out


def block_topk(q, k_sum, table, start, topk, bs, count=None, force_diag=False):
    """idx [B, H_kv, topk], and the scores of the present blocks (float64 rounded
    to float32) as lists of dicts [b][h]. The order: forced blocks, NaN scores,
    scores from the largest on; the lower block first where these are equal."""
    B, T, H, D = q.shape
    pages, Hk = k_sum.shape[:2]
    idx = np.full((B, Hk, topk), -1, np.int32)
    scores = []
    for b in range(B):
        s, n = _step(start, count, b, T, table.shape[1] * bs)
        total = min(s + n, table.shape[1] * bs)
        scores.append([])
        for h in range(Hk):
            qs = q[b, :n, h * (H // Hk):(h + 1) * (H // Hk)].sum((0, 1))
            sc, forced = {}, set()
            for j in range(-(-total // bs)):
                p = _page(table, pages, b, j)
                if p >= 0:
                    sc[j] = np.float32((qs @ k_sum[p, h]) / min(bs, total - j * bs))
                    if force_diag and n and (j + 1) * bs > s:
                        forced.add(j)
            rank = {j: (0, 0.0, j) if j in forced else (1, 0.0, j) if np.isnan(x) else (2, -x, j) for j, x in sc.items()}
            best = sorted(sc, key=rank.get)[:topk]
            idx[b, h, :len(best)] = sorted(best)
            scores[b].append(sc)
    return idx, scores


def attn(cache, q, table, start, idx=None, scale=None, count=None, out=None):
    """o [B, T, H, D]; rows without a visible token are zeros, rows t >= count[b] as
    in ``out``. For error bounds also the sum of the softmax weights times the
    size of what a value is made of, and each row's largest sum |q k| scale. A
    value is zero + scale code; with m the largest |value| of its group, |zero|
    <= m + scale and scale <= 2 m / 14, so |zero| + |scale code| <= |v| + 2
    |zero| <= |v| + 2.3 m."""
    kv = cache["kv"]
    _, pages, Hk, bs, D = kv.shape
    B, T, H, _ = q.shape
    G = H // Hk
    scale = 1 / np.sqrt(D) if scale is None else scale
    o = np.zeros(q.shape) if out is None else out.astype(np.float64).copy()
    size, logit = np.zeros(q.shape), np.zeros((B, T, H))
    for b in range(B):
        s, n = _step(start, count, b, T, table.shape[1] * bs)
        for h in range(Hk):
            blocks = range(table.shape[1]) if idx is None else [j for j in idx[b, h] if j >= 0]
            blocks = [j for j in blocks if _page(table, pages, b, j) >= 0 and j * bs < s + n]
            if n and not blocks:
                o[b, :n, h * G:(h + 1) * G] = 0
                continue
            if not n:
                continue
            pos = np.concatenate([np.arange(j * bs, (j + 1) * bs) for j in blocks])
            k, v = (np.concatenate([kv[i, _page(table, pages, b, j), h] for j in blocks]) for i in range(2))
            m = np.abs(v.reshape(len(v), -1, 64)).max(-1)
            parts = np.abs(v) + 2.3 * np.repeat(m, 64, -1)
            for t in range(n):
                see = pos <= s + t
                for g in range(h * G, (h + 1) * G):
                    if not see.any():
                        o[b, t, g] = 0
                        continue
                    x = (k[see] @ q[b, t, g]) * scale
                    w = np.exp(x - x.max())
                    w /= w.sum()
                    o[b, t, g] = w @ v[see]
                    size[b, t, g] = w @ parts[see]
                    logit[b, t, g] = (np.abs(k[see]) @ np.abs(q[b, t, g])).max() * scale
    return o, size, logit
