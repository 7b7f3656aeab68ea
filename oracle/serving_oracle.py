"""Float64 oracle of the serving operators around the paged round-robin cache: the rotary embedding,
the 4-bit K/V format, the read-back of a cache, and attention with modified scores.  NumPy only,
written from the definitions, one row and one position at a time where that is practical; shares no
code with the CUDA path."""
import numpy as np

PAGE = 16
GROUP = 64


# ---------------------------------------------------------------- rotary embedding
def rotate(x, pos, inv_freq, pairs):
    """x [N, H, d] rotated at positions pos [N] by angles pos * inv_freq, in float64."""
    y = np.array(x, dtype=np.float64)
    h = len(inv_freq)
    ang = np.asarray(pos, dtype=np.float64)[:, None] * np.asarray(inv_freq, dtype=np.float64)
    c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
    i = np.arange(h)
    a, b = (2 * i, 2 * i + 1) if pairs else (i, i + h)
    u, w = y[..., a].copy(), y[..., b].copy()
    y[..., a] = u * c - w * s
    y[..., b] = w * c + u * s
    return y


# ---------------------------------------------------------------- 4-bit records
def to_bf16(x):
    """Nearest bf16 (ties to even) of float64 values, as float64."""
    f = np.asarray(x, dtype=np.float32)
    u = f.view(np.uint32).astype(np.uint64)
    r = ((u + 0x7FFF + ((u >> 16) & 1)) & 0xFFFF0000).astype(np.uint32)
    return np.where(np.isfinite(f), r.view(np.float32), f).astype(np.float64)


def q4_codes(row):
    """Codes, scales and minima of one head's row [d]: (n [d], scale [d / 64], minimum [d / 64])."""
    d = len(row)
    n, sc, mn = np.zeros(d, int), np.zeros(d // GROUP), np.zeros(d // GROUP)
    for g in range(d // GROUP):
        x = np.asarray(row[g * GROUP:(g + 1) * GROUP], dtype=np.float64)
        if not np.isfinite(x).all():
            sc[g], mn[g] = 0.0, np.nan
            continue
        mn[g] = to_bf16(x.min())
        sc[g] = max(0.0, to_bf16((x.max() - mn[g]) / 15))   # the minimum's rounding may pass the maximum
        if sc[g] > 0:
            n[g * GROUP:(g + 1) * GROUP] = np.clip(np.rint((x - mn[g]) / sc[g]), 0, 15)
    return n, sc, mn


def q4_values(n, sc, mn):
    return np.repeat(mn, GROUP) + np.repeat(sc, GROUP) * n


def q4_place(dim, d):
    """(byte, shift) of a dim's code within a row of d / 2 bytes."""
    g, c, i = dim // GROUP, (dim % GROUP) // 8, dim % 8
    word = c if d == 64 else 2 * c + g
    return 4 * word + i // 2, 4 * (i % 2)


def q4_read(record, t, d):
    """Values [d] of token t of one record (uint8 [9 d])."""
    row = record[t * (d // 2):(t + 1) * (d // 2)].astype(int)
    n = np.array([(row[q4_place(k, d)[0]] >> q4_place(k, d)[1]) & 15 for k in range(d)])
    pairs = record[8 * d + t * (d // 16):8 * d + (t + 1) * (d // 16)].copy().view(np.uint16)
    f = (pairs.astype(np.uint32) << 16).view(np.float32).astype(np.float64).reshape(-1, 2)
    return q4_values(n, f[:, 0], f[:, 1])


def q4_minima(record, t, d):
    """Each dim's group minimum of token t."""
    pairs = record[8 * d + t * (d // 16):8 * d + (t + 1) * (d // 16)].copy().view(np.uint16)
    f = (pairs.astype(np.uint32) << 16).view(np.float32).astype(np.float64).reshape(-1, 2)
    return np.repeat(f[:, 1], GROUP)


def q4_write(record, t, row):
    """Stores one head's row as token t of a record, in place."""
    d = len(row)
    n, sc, mn = q4_codes(row)
    for k in range(d):
        at, sh = q4_place(k, d)
        at += t * (d // 2)
        record[at] = (int(record[at]) & ~(15 << sh) & 255) | (int(n[k]) << sh)
    bits = (np.stack([sc, mn], -1).astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)
    record[8 * d + t * (d // 16):8 * d + (t + 1) * (d // 16)] = bits.reshape(-1).view(np.uint8)


# ---------------------------------------------------------------- placement
def slot(p, cp, I, table):
    """(rank, page, row) of position p, by dealing groups of I positions in turn."""
    rank = (p // I) % cp
    before = sum(min(I, p - g * I) for g in range(rank, p // I + 1, cp) if g * I < p)
    return rank, int(table[rank][before // PAGE]), before % PAGE


# ---------------------------------------------------------------- attention
def bounds(i, kv_len, window=0, kv_start=None, prefix=0):
    lo = max(0, i - window + 1 if window else 0, 0 if kv_start is None else kv_start)
    return lo, min(kv_len, max(i + 1, prefix))


def attend(q, k, v, i, lo, hi, scale, softcap=0.0, slopes=None):
    """One query row q [Hq, d] at position i over keys j in [lo, hi) of k, v [Hkv, L, d].
    Returns (out [Hq, d], lse [Hq], weight-averaged |v| [Hq, d], the largest scale * sum |q||k|)."""
    Hq, d = q.shape
    G = Hq // k.shape[0]
    out, lse, absv, big = np.zeros((Hq, d)), np.full(Hq, -np.inf), np.zeros((Hq, d)), 0.0
    if hi <= lo:
        return out, lse, absv, big
    j = np.arange(lo, hi)
    for h in range(Hq):
        kk, vv = k[h // G, lo:hi], v[h // G, lo:hi]
        s = scale * (kk @ q[h])
        big = max(big, float((scale * (np.abs(kk) @ np.abs(q[h]))).max()))
        if softcap:
            s = softcap * np.tanh(s / softcap)
        if slopes is not None:
            s = s - slopes[h] * np.abs(i - j)
        m = s.max()
        w = np.exp(s - m)
        out[h], absv[h], lse[h] = w @ vv / w.sum(), w @ np.abs(vv) / w.sum(), m + np.log(w.sum())
    return out, lse, absv, big
