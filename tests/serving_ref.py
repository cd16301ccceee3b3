"""Plain restatements, on the CPU, of the serving-step operators (include/pn.h,
"4-bit cache"): 64-bit floats and Python integers, no code of the library."""
from __future__ import annotations

import numpy as np


# ---------------------------------------------------------------- 4-bit rule --
def quantise(x: np.ndarray):
    """fp32 [..., D] -> codes [..., D] (0..15) and fp16 scales [..., D / 64]: the
    group's first largest-magnitude value / -8 as fp16; codes rint(x / d) + 8
    limited to 0..15, fp32 quotients, ties to even."""
    x = x.astype(np.float32)
    g = x.reshape(x.shape[:-1] + (x.shape[-1] // 64, 64))
    first = np.abs(g).argmax(-1)
    a = np.take_along_axis(g, first[..., None], -1)
    d = np.clip(a * np.float32(-0.125), np.float32(-65504), np.float32(65504)).astype(np.float16)
    d = np.where(d == 0, np.float16(0), d)
    with np.errstate(divide="ignore", invalid="ignore"):
        n = np.rint(g / d.astype(np.float32))
    n = np.where(d == 0, np.float32(0), np.clip(n, -8, 7)) + 8
    return n.astype(np.uint8).reshape(x.shape), d[..., 0]


def dequantise(n: np.ndarray, d: np.ndarray) -> np.ndarray:
    g = n.reshape(n.shape[:-1] + (n.shape[-1] // 64, 64)).astype(np.float64) - 8
    return (g * d.astype(np.float64)[..., None]).reshape(n.shape)


# ------------------------------------------------------------- record layout --
def code_place(D: int, r: int, d: int):
    """(byte, shift) in a record of the codes of value d of token r: K and V."""
    h, g = divmod(r, 8)
    j, rest = divmod(d, 64)
    i, c = divmod(rest, 8)
    per = 2 if D >= 128 else 1
    planes = D // 64 // per
    plane, s = divmod(j, per)
    k_index = 0
    for size, at in ((2, h), (planes, plane), (8, g), (4, i // 2), (per, s), (2, i % 2)):
        k_index = k_index * size + at
    v_index = 0
    for size, at in ((2, h), (planes, plane), (8, i), (4, g // 2), (2, g % 2), (per, s)):
        v_index = v_index * size + at
    bit = 16 * (c % 2) + 4 * (c // 2)
    return (4 * k_index + bit // 8, bit % 8), (8 * D + D // 2 + 4 * v_index + bit // 8, bit % 8)


def place_tables(D: int):
    """Byte and shift of every (token, value), for K and for V: four [16][D] arrays."""
    t = np.array([[sum(code_place(D, r, d), ()) for d in range(D)] for r in range(16)])
    return t[..., 0], t[..., 1], t[..., 2], t[..., 3]


def write_tokens(cache: np.ndarray, slots, kn, kd, vn, vd) -> None:
    """Writes tokens (codes [T][heads][D], scales [T][heads][D / 64]) into cache
    uint8 [pages][heads][page / 16][17 D]."""
    D = cache.shape[3] // 17
    page = cache.shape[2] * 16
    kb, ks, vb, vs = place_tables(D)
    for t, slot in enumerate(slots):
        slot = int(slot)
        if slot < 0:
            continue
        r = slot % 16
        for h in range(cache.shape[1]):
            rec = cache[slot // page, h, slot % page // 16]
            for byte, shift, n in ((kb[r], ks[r], kn[t, h]), (vb[r], vs[r], vn[t, h])):
                for sh in (0, 4):
                    at = shift == sh
                    rec[byte[at]] = (rec[byte[at]] & (0xF0 if sh == 0 else 0x0F)) | (n[at] << sh)
            G = D // 64
            for base, d in ((8 * D, kd[t, h]), (16 * D + D // 2, vd[t, h])):
                rec[base + 2 * G * r: base + 2 * G * (r + 1)] = d.astype(np.float16).view(np.uint8)


# ---------------------------------------------------------------------- plan --
def plan(lens, add, held, table, free, ring, page, capacity):
    """Request by request; table and free are written like the call does."""
    B, F = len(lens), len(free)
    most = table.shape[1]
    head, tail = (int(x) for x in ring)
    avail = tail - head
    out = dict(slots=[-1] * capacity, positions=[-1] * capacity, requests=[-1] * capacity, starts=[0], lens=[], held=[])
    taken = wanted = back = refused = 0
    give = []
    for b in range(B):
        start = out["starts"][-1]
        if add[b] < 0:
            give += [int(p) for p in table[b, :held[b]]]
            back += int(held[b])
            out["lens"].append(0)
            out["held"].append(0)
            out["starts"].append(start)
            continue
        end = start + int(add[b])
        out["starts"].append(end)
        pages = -(-(int(lens[b]) + int(add[b])) // page)
        fits = pages <= most and end <= capacity
        need = max(pages - int(held[b]), 0) if fits else 0
        ok = fits and (need == 0 or wanted + need <= avail)
        if ok:
            for i in range(need):
                table[b, held[b] + i] = free[(head + wanted + i) % F]
            taken += need
        else:
            refused += 1
        wanted += need
        out["lens"].append(int(lens[b]) + (int(add[b]) if ok else 0))
        out["held"].append(int(held[b]) + (need if ok else 0))
        for t in range(start, min(end, capacity)):
            out["requests"][t] = b
            if ok:
                pos = int(lens[b]) + t - start
                out["positions"][t] = pos
                out["slots"][t] = int(table[b, pos // page]) * page + pos % page
    for i, p in enumerate(give):
        free[(tail + i) % F] = p
    out["ring"] = [head + taken, tail + back]
    out["refused"] = [refused]
    return out


# ------------------------------------------------------------------- append --
def norm_rotate_f32(x, weight, eps, cos, sin, positions, interleaved):
    """The documented fp32 arithmetic, each operation rounded by itself.  x fp32 [T][H][D]."""
    f = np.float32
    x = x.astype(f)
    if weight is not None:
        p = x * x
        while p.shape[-1] > 1:
            half = p.shape[-1] // 2
            p = p[..., :half] + p[..., half:]
        x = x * (f(1) / np.sqrt(p * f(1.0 / x.shape[-1]) + f(eps))) * weight.astype(f)
    if cos is not None:
        x = x.copy()
        half = cos.shape[1]
        for t, pos in enumerate(positions):
            if not 0 <= pos < cos.shape[0]:
                continue
            c, s = cos[pos].astype(f), sin[pos].astype(f)
            first = slice(0, 2 * half, 2) if interleaved else slice(0, half)
            second = slice(1, 2 * half, 2) if interleaved else slice(half, 2 * half)
            a, b = x[t, :, first].copy(), x[t, :, second].copy()
            x[t, :, first] = a * c - b * s
            x[t, :, second] = b * c + a * s
    return x


# ---------------------------------------------------------------- attention --
def attention(q, k, v, scale, window, sinks):
    """One request, 64 bits: q [n][H][D] at the last n of the L cached tokens k, v
    [L][KV][D].  Returns out, lse and two bounds' ingredients per row: sum p |v|
    [n][H][D], and the largest scale * sum |q| |k| over the tokens seen [n][H]."""
    n, H, D = q.shape
    L, KV = k.shape[0], k.shape[1]
    out, lse = np.zeros((n, H, D)), np.full((n, H), -np.inf)
    size, reach = np.zeros((n, H, D)), np.zeros((n, H))
    for i in range(n):
        p = L - n + i
        t = np.arange(L)
        see = t <= p
        if window:
            see &= (t > p - window) | (t < sinks)
        if not see.any():
            continue
        for h in range(H):
            kk, vv = k[see, h // (H // KV)], v[see, h // (H // KV)]
            x = scale * (kk @ q[i, h])
            top = x.max()
            e = np.exp(x - top)
            lse[i, h] = top + np.log(e.sum())
            w = e / e.sum()
            out[i, h] = w @ vv
            size[i, h] = w @ np.abs(vv)
            reach[i, h] = (abs(scale) * (np.abs(kk) @ np.abs(q[i, h]))).max()
    return out, lse, size, reach


# ------------------------------------------------------------------- verify --
def verify(tokens, target, draft, uniforms, counts):
    """Exact integers for the weights; fp32 for the acceptance test."""
    B, K = tokens.shape
    V = target.shape[2]
    accepted, out = [], np.full((B, K + 1), -1, np.int32)
    for b in range(B):
        count = K if counts is None else min(max(int(counts[b]), 0), K)
        n = 0
        while n < count:
            x = int(tokens[b, n])
            if not 0 <= x < V:
                break
            q = np.float32(1) if draft is None else draft[b, n, x]
            if not uniforms[b, n] * q < target[b, n, x]:
                break
            out[b, n] = x
            n += 1
        accepted.append(n)

        def whole(w):
            w = np.where(w > 0, np.minimum(w, np.float32(1)), np.float32(0))
            return [int(z) for z in np.rint(w * np.float32(2.0 ** 42))]

        row = target[b, n]
        rest = row.copy()
        if n < count:
            if draft is not None:
                rest = row - draft[b, n]
            elif 0 <= tokens[b, n] < V:
                rest[tokens[b, n]] = 0
        w = whole(rest)
        if sum(w) == 0:
            w = whole(row)
        total = sum(w)
        if total == 0:
            continue
        at = min(max(int(np.floor(np.float64(uniforms[b, K]) * np.float64(total))), 0), total - 1)
        s = 0
        for j, z in enumerate(w):
            s += z
            if s > at:
                out[b, n] = j
                break
    return np.array(accepted, np.int32), out
