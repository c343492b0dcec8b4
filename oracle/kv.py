"""Oracle of the 4-bit key/value cache and the attention over it (test
infrastructure; numpy only, no code shared with the library).

The definitions are those of include/moe.h ("key/value cache in 4 bits"):
quantisation in IEEE fp32 arithmetic, step for step, so records can be compared
byte for byte; attention in fp64.
"""
from __future__ import annotations

import numpy as np

BLOCK = 16
NIBBLE_ELEMENT = (0, 2, 4, 6, 1, 3, 5, 7)


def f16_down(x):
    """fp32 -> fp16, the largest value not above x."""
    h = x.astype(np.float16)
    return np.where(h.astype(np.float32) > x, np.nextafter(h, np.float16(-np.inf)), h).astype(np.float16)


def f16_up(x):
    h = x.astype(np.float16)
    return np.where(h.astype(np.float32) < x, np.nextafter(h, np.float16(np.inf)), h).astype(np.float16)


def quantise(x):
    """x fp32 [..., D]: codes uint8 [..., D/64, 64], scale and bias fp16 [..., D/64]."""
    g = np.clip(np.asarray(x, np.float32), np.float32(-65504), np.float32(65504))
    g = g.reshape(g.shape[:-1] + (-1, 64))
    lo, hi = g.min(-1), g.max(-1)
    bias = f16_down(lo)
    b32 = bias.astype(np.float32)
    scale = f16_up((hi - b32) / np.float32(15))
    s32 = scale.astype(np.float32)[..., None]
    with np.errstate(divide="ignore", invalid="ignore"):
        q = np.where(s32 > 0, np.rint((g - b32[..., None]) / s32), np.float32(0))
    return np.nan_to_num(q).astype(np.uint8), scale, bias


def values(codes, scale, bias):
    """fp64 [..., D]; exact."""
    v = scale.astype(np.float64)[..., None] * codes + bias.astype(np.float64)[..., None]
    return v.reshape(v.shape[:-2] + (-1,))


def empty_pages(n_pages, n_kv_heads, head_dim, page_tokens, fill=0):
    return np.full((n_pages, n_kv_heads, page_tokens // BLOCK, 18 * head_dim), fill, np.uint8)


def _row_bytes(codes):
    """[NG, 64] codes of one row: its D/2 code bytes."""
    ng = codes.shape[0]
    words = np.zeros(8 * ng, np.uint32)
    for j in range(ng):
        for i in range(8):
            w = 0
            for n in range(8):
                w |= int(codes[j, 8 * i + NIBBLE_ELEMENT[n]]) << (4 * n)
            words[i * ng + j] = w
    return words.view(np.uint8)


def _spans(d, side, r):
    """Byte ranges of row r's codes and affine words in a record; side 0 K, 1 V."""
    c = side * 8 * d + r * d // 2
    a = (16 + side) * d + r * d // 16
    return slice(c, c + d // 2), slice(a, a + d // 16)


def append(pages, page_tokens, k, v, slots):
    """In place; k, v fp32 [n][H][D]."""
    d = k.shape[-1]
    for side, x in enumerate((k, v)):
        codes, scale, bias = quantise(x)
        for t, slot in enumerate(slots):
            if slot < 0:
                continue
            page, place = divmod(int(slot), page_tokens)
            for h in range(x.shape[1]):
                rec = pages[page, h, place // BLOCK]
                cs, as_ = _spans(d, side, place % BLOCK)
                rec[cs] = _row_bytes(codes[t, h])
                rec[as_] = np.stack([scale[t, h], bias[t, h]], -1).view(np.uint8).reshape(-1)


def read(pages, page_tokens, slots):
    """k, v fp64 [n][H][D], exact; zeros where a slot is negative."""
    n, H, d = len(slots), pages.shape[1], pages.shape[3] // 18
    ng = d // 64
    out = np.zeros((2, n, H, d))
    slots = np.asarray(slots, np.int64)
    live = slots >= 0
    page, place = np.divmod(np.where(live, slots, 0), page_tokens)
    rec = pages[page, :, place // BLOCK]  # [n, H, bytes]
    r = place % BLOCK
    for side in (0, 1):
        code = np.stack([rec[t, :, _spans(d, side, r[t])[0]] for t in range(n)]) if n else np.zeros((0, H, d // 2), np.uint8)
        aff = np.stack([rec[t, :, _spans(d, side, r[t])[1]] for t in range(n)]) if n else np.zeros((0, H, d // 16), np.uint8)
        words = np.ascontiguousarray(code).view(np.uint32).reshape(n, H, 8, ng)
        half = np.ascontiguousarray(aff).view(np.float16).reshape(n, H, ng, 2).astype(np.float64)
        for pos, e in enumerate(NIBBLE_ELEMENT):
            q = (words >> np.uint32(4 * pos)) & np.uint32(15)  # [n, H, i, j]
            val = q.astype(np.float64).transpose(0, 1, 3, 2) * half[..., :1] + half[..., 1:]  # [n, H, j, i]
            for j in range(ng):
                out[side, :, :, 64 * j + e:64 * j + 64:8] = val[:, :, j]
    out[:, ~live] = 0
    return out[0], out[1]


def attend(pages, page_tokens, q, table, kv_len, q_start, scale, causal=True, window=0):
    """q fp64 [n_q][Hq][D]. Returns out fp64, lse fp64, and what bounds of its error need: mag = sum_j w_j |V_j|
    (per output element), dot = scale * max_j sum_d |q_d K_jd| (per row) and seen (keys per row)."""
    n_q, Hq, d = q.shape
    H = pages.shape[1]
    G = Hq // H
    out, mag = np.zeros((n_q, Hq, d)), np.zeros((n_q, Hq, d))
    lse, dot, seen = np.full((n_q, Hq), -np.inf), np.zeros((n_q, Hq)), np.zeros((n_q, Hq))
    top = np.zeros((n_q, Hq))
    for b, n_kv in enumerate(kv_len):
        a, e = int(q_start[b]), int(q_start[b + 1])
        if n_kv == 0 or e == a:
            continue
        t = np.arange(n_kv)
        K, V = read(pages, page_tokens, table[b][t // page_tokens].astype(np.int64) * page_tokens + t % page_tokens)
        pos = n_kv - (e - a) + np.arange(e - a)
        see = np.ones((e - a, n_kv), bool)
        if causal:
            see &= t[None] <= pos[:, None]
        if window:
            see &= t[None] > pos[:, None] - window
        for hq in range(Hq):
            h = hq // G
            z = scale * (q[a:e, hq] @ K[:, h].T)
            z = np.where(see, z, -np.inf)
            m = z.max(1, keepdims=True)
            p = np.exp(z - np.where(np.isfinite(m), m, 0))
            l = p.sum(1, keepdims=True)
            some = l[:, 0] > 0
            w = np.divide(p, l, out=np.zeros_like(p), where=l > 0)
            out[a:e, hq] = w @ V[:, h]
            mag[a:e, hq] = w @ np.abs(V[:, h])
            lse[a:e, hq][some] = (m[:, 0] + np.log(np.where(some, l[:, 0], 1)))[some]
            ad = np.where(see, abs(scale) * (np.abs(q[a:e, hq]) @ np.abs(K[:, h]).T), 0)
            dot[a:e, hq] = ad.max(1)
            seen[a:e, hq] = see.sum(1)
            top[a:e, hq] = np.where(see[:, :, None], np.abs(V[None, :, h]), 0).max((1, 2)) if n_kv * (e - a) * d < 2e7 else np.abs(V[:, h]).max()
    return out, lse, dict(mag=mag, dot=dot, seen=seen, top=top)
