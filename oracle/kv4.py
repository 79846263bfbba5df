"""Reference of the paged 4-bit window cache (include/hq_kv4.h) in numpy.

Codes and scales follow the fp32 steps of the format one by one, each sum and
product rounded once, so that pages can be compared byte for byte; values,
attention and eviction are computed in 64 bits from the bytes of the pages.
Everything here runs on the CPU and shares no code with the CUDA path.
"""
from __future__ import annotations

import numpy as np

TILE, UNIT, UNIT_BYTES = 128, 16, 2112
F32 = np.float32


def bf16_round(x: np.ndarray) -> np.ndarray:
    """fp32 values rounded to bf16 (nearest, ties to even), as fp32; finite inputs."""
    b = np.ascontiguousarray(x, F32).view(np.uint32).astype(np.uint64)
    b = ((b + 0x7FFF + ((b >> 16) & 1)) >> 16).astype(np.uint32) << 16
    return b.view(F32)


def signs_of(mask) -> np.ndarray:
    """The +-1 diagonal of a 128-bit mask (4 words)."""
    i = np.arange(TILE)
    m = np.asarray(mask, np.uint32)
    return 1.0 - 2.0 * ((m[i // 32] >> (i % 32)) & 1)


def fwht(x: np.ndarray) -> np.ndarray:
    """Unnormalised transform of the last axis, stages 1, 2, .. 64 in the input's own type."""
    x = x.copy()
    h = 1
    while h < TILE:
        y = x.reshape(x.shape[:-1] + (TILE // (2 * h), 2, h))
        a, b = y[..., 0, :].copy(), y[..., 1, :].copy()
        y[..., 0, :], y[..., 1, :] = a + b, a - b
        h *= 2
    return x


def quantize(x: np.ndarray, mask):
    """Rows [..., 128] fp32 -> codes uint8, scales fp32 (bf16 values), row out of range."""
    with np.errstate(all="ignore"):
        z = fwht(np.asarray(x, F32) * signs_of(mask).astype(F32))
        top = np.abs(z).max(-1)                    # NaN if any is
        bad = ~np.isfinite(top)
        s = bf16_round(np.where(bad, F32(0), top) * F32(0.011785113019775793))
        s = np.where(s < F32(2.0 ** -126), F32(0), s)
        inv = np.where(s > 0, F32(1) / (s * F32(11.313708498984761)), F32(0)).astype(F32)
        zz = np.where(s[..., None] > 0, z, F32(0))
        t = np.floor(zz.astype(np.float64) * inv[..., None].astype(np.float64)) + 8   # exact products
    return np.clip(t, 0, 15).astype(np.uint8), s.astype(F32), bad


def new_pages(n_pages, n_kv, page_tokens, fill=0):
    return np.full((n_pages, n_kv, page_tokens // UNIT, UNIT_BYTES), fill, np.uint8)


def _bits(s):
    return (np.ascontiguousarray(s, F32).view(np.uint32) >> 16).astype(np.uint16)


def put(pages, page, h, t, which, codes, scale):
    """One row's codes and scale into token t of a page (which: 0 K, 1 V)."""
    unit, k = pages[page, h, t // UNIT], t % UNIT
    packed = codes[0::2] | (codes[1::2] << 4)
    if which == 0:
        unit[k * 64:k * 64 + 64] = packed
    else:
        for j in range(8):
            at = 1024 + (k // 2) * 128 + j * 16 + (k % 2) * 8
            unit[at:at + 8] = packed[8 * j:8 * j + 8]
    at = 2048 + 32 * which + 2 * k
    unit[at:at + 2] = _bits(np.array([scale]))[:1].view(np.uint8)


def append(pages, table, k, v, seq, pos, mask):
    """Writes rows; returns (out of range, bad place) as hq_kv4_append reports them."""
    P = pages.shape[2] * UNIT
    rng = page_bad = False
    coded = [quantize(x, mask) for x in (k, v)]
    for i, (b, p) in enumerate(zip(seq, pos)):
        if b < 0:
            continue
        if b >= table.shape[0] or p < 0 or p >= table.shape[1] * P or not \
                0 <= table[b, p // P] < pages.shape[0]:
            page_bad = True
            continue
        for which in range(2):
            c, s, bad = coded[which]
            rng |= bool(bad[i].any())
            for h in range(pages.shape[1]):
                put(pages, table[b, p // P], h, p % P, which, c[i, h], s[i, h])
    return rng, page_bad


def raw_rows(pages, page, which):
    """Codes [n_kv][page tokens][128] and scales [n_kv][page tokens] of one page."""
    u = pages[page]                                                    # [n_kv][units][2112]
    nh, n = u.shape[:2]
    if which == 0:
        b = u[..., :1024].reshape(nh, n * UNIT, 64)
    else:
        b = u[..., 1024:2048].reshape(nh, n, 8, 8, 2, 8).transpose(0, 1, 2, 4, 3, 5)
        b = b.reshape(nh, n * UNIT, 64)
    c = np.stack([b & 15, b >> 4], -1).reshape(nh, n * UNIT, TILE)
    s = np.ascontiguousarray(u[..., 2048 + 32 * which:2080 + 32 * which]).view(np.uint16)
    s = (s.astype(np.uint32) << 16).view(F32).reshape(nh, n * UNIT)
    return c, s


def rotated(pages, table, b, n, which):
    """Sequence b's first n rows in the transformed domain, [n_kv][n][128] in 64 bits."""
    P = pages.shape[2] * UNIT
    got = [raw_rows(pages, table[b, j], which) for j in range(-(-n // P))]
    if not got:
        return np.zeros((pages.shape[1], 0, TILE))
    c = np.concatenate([g[0] for g in got], 1)[:, :n].astype(np.float64)
    s = np.concatenate([g[1] for g in got], 1)[:, :n].astype(np.float64)
    with np.errstate(invalid="ignore"):
        return (c - 7.5) * s[..., None]


def back(y, mask):
    """Transformed rows -> values, in 64 bits."""
    return fwht(np.asarray(y, np.float64)) * signs_of(mask) / np.sqrt(128.0)


def read32(pages, page, h, t, which, mask):
    """One row as the fp32 steps of hq_kv4_read give it."""
    c, s = raw_rows(pages, page, which)
    sf = F32(s[h, t]) * F32(0.08838834764831845)
    return fwht(c[h, t].astype(F32) - F32(7.5)) * signs_of(mask).astype(F32) * sf     # exact sums


def attention(pages, table, lengths, q, mask, scale, cap=0.0, mass=None):
    """q [B, q_len, Hq, 128] in 64 bits -> dict of out, lse, mass, and what the error bound
    goes by: size [B, q_len, Hq, 128] = sum of p |V'| in the transformed domain, zeta [B, q_len, Hq] =
    |scale| |q| max |Khat|, and zeta_codes = |scale| |q| max of s max(|c|, 7.5 sqrt(128)), |c| of a
    row's codes, and scales = sum of p s over V's scales."""
    B, q_len, Hq, _ = q.shape
    nh = pages.shape[1]
    G = Hq // nh
    out, size = np.zeros(q.shape), np.zeros(q.shape)
    lse, zeta = np.full(q.shape[:3], -np.inf), np.zeros(q.shape[:3])
    zeta_codes, scales = np.zeros(q.shape[:3]), np.zeros(q.shape[:3])
    add = np.zeros((B, nh, table.shape[1] * pages.shape[2] * UNIT))
    for b in range(B):
        n = int(lengths[b])
        K, V = (rotated(pages, table, b, n, w) for w in (0, 1))
        codes = [raw_rows(pages, table[b, j], 0) for j in range(-(-n // (pages.shape[2] * UNIT)))]
        S = np.concatenate([s * np.maximum(np.linalg.norm(c.astype(np.float64), axis=-1),
                                           7.5 * np.sqrt(128.0)) for c, s in codes],
                           1)[:, :n] if n else np.zeros((nh, 0))
        sv = [raw_rows(pages, table[b, j], 1)[1] for j in range(-(-n // (pages.shape[2] * UNIT)))]
        sv = np.concatenate(sv, 1)[:, :n].astype(np.float64) if n else np.zeros((nh, 0))
        for j in range(q_len):
            m = n - q_len + j + 1
            if m <= 0:
                continue
            for hq in range(Hq):
                h = hq // G
                y = fwht(q[b, j, hq] * signs_of(mask)) / np.sqrt(128.0)
                z = (K[h, :m] @ y) * scale
                if cap > 0:
                    z = cap * np.tanh(z / cap)
                top = z.max()
                e = np.exp(z - top)
                p = e / e.sum()
                out[b, j, hq] = back(p @ V[h, :m], mask)
                size[b, j, hq] = p @ np.abs(V[h, :m])
                scales[b, j, hq] = p @ sv[h, :m]
                lse[b, j, hq] = top + np.log(e.sum())
                size_q = abs(scale) * np.linalg.norm(y)
                zeta[b, j, hq] = size_q * np.linalg.norm(K[h, :m], axis=-1).max()
                zeta_codes[b, j, hq] = size_q * S[h, :m].max()
                add[b, h, :m] += p
    total = add if mass is None else add + mass
    return dict(out=out, lse=lse, mass=total, added=add, size=size, zeta=zeta,
                zeta_codes=zeta_codes, scales=scales)


def keep(mass, n, budget, recent):
    """The positions one head keeps, in order."""
    if n <= budget:
        return np.arange(n)
    old = n - recent
    m = np.where(np.isnan(mass[:old]), -np.inf, mass[:old]).astype(np.float64) + 0.0
    nan = np.isnan(mass[:old])
    order = sorted(range(old), key=lambda i: (nan[i], -m[i], i))
    return np.array(sorted(order[:budget - recent]) + list(range(old, n)), np.int64)
