"""Float64 oracle of beam search over an encoder's states: cross attention, the selection of the best
continuations, and the reordering of the beams' paged caches.  NumPy only, written from the definitions,
one sequence, one row and one beam at a time; shares no code with the CUDA path."""
import numpy as np

from oracle import serving_oracle as so

PAGE = so.PAGE


# ---------------------------------------------------------------- cross attention
def cross(q, k, v, scale, ranges=None):
    """Rows q [T, Hq, d] over the keys k, v [S, Hkv, d] of one sequence; ranges [T, 2]: each row's keys.
    Returns (out, lse, weight-averaged |v|, per row and head the largest scale * sum |q||k|)."""
    T, Hq, d = q.shape
    S, G = k.shape[0], Hq // k.shape[1]
    out, lse = np.zeros((T, Hq, d)), np.full((T, Hq), -np.inf)
    absv, big = np.zeros((T, Hq, d)), np.zeros((T, Hq))
    for i in range(T):
        lo, hi = (0, S) if ranges is None else (max(0, int(ranges[i][0])), min(S, int(ranges[i][1])))
        if lo >= hi:
            continue
        for h in range(Hq):
            kk, vv = k[lo:hi, h // G], v[lo:hi, h // G]
            s = scale * (kk @ q[i, h])
            big[i, h] = scale * (np.abs(kk) @ np.abs(q[i, h])).max()
            m = s.max()
            w = np.exp(s - m)
            out[i, h], absv[i, h], lse[i, h] = w @ vv / w.sum(), w @ np.abs(vv) / w.sum(), m + np.log(w.sum())
    return out, lse, absv, big


# ---------------------------------------------------------------- selection
def select(logits, scores, M, eos=-1):
    """One sequence: logits [K, V], scores [K].  Returns (candidates, beams that go on), lists of (score, beam, token)."""
    K, V = logits.shape
    flat = np.full((K, V), -np.inf)
    for k in range(K):
        x = np.where(np.isnan(logits[k]), -np.inf, np.asarray(logits[k], dtype=np.float64))
        m = x.max()
        if m == -np.inf or not np.isfinite(scores[k]):
            continue
        if m == np.inf:
            flat[k] = np.where(x == np.inf, scores[k] - np.log((x == np.inf).sum()), -np.inf)
        else:
            flat[k] = scores[k] + (x - m - np.log(np.exp(x - m).sum()))
    flat = flat.reshape(-1)
    order = np.lexsort((np.arange(K * V), -flat))[:M]
    best = [(float(flat[i]), int(i // V), int(i % V)) for i in order]
    return best, [c for c in best if c[2] != eos][:K]


# ---------------------------------------------------------------- reordering
def held(n, rank, cp, I):
    """Tokens of n that a rank holds."""
    return sum(1 for p in range(n) if (p // I) % cp == rank)


def reorder(parents, lens, tables, own, caches, cp, I):
    """parents [B, K], lens [B], tables and own [cp, B K, columns], caches: arrays [.., cp, pool, Hkv, 16, d] (rows) or
    uint8 [.., cp, pool, Hkv, 9 d] (4-bit records).  Returns the new tables and caches."""
    out, new = tables.copy(), [c.copy() for c in caches]
    K = len(parents[0])
    for b, n in enumerate(lens):
        for r in range(cp):
            full, rest = divmod(held(n, r, cp, I), PAGE)
            for j, p in enumerate(parents[b]):
                out[r, b * K + j, :full] = tables[r, b * K + p, :full]
                if full < tables.shape[2]:
                    out[r, b * K + j, full] = own[r, b * K + j, full]
                if rest == 0:
                    continue
                src, dst = tables[r, b * K + p, full], own[r, b * K + j, full]
                for old, c in zip(caches, new):
                    if c.dtype == np.uint8:
                        d = c.shape[-1] // 9
                        for a, z in ((0, rest * d // 2), (8 * d, 8 * d + rest * d // 16)):
                            c[..., r, dst, :, a:z] = old[..., r, src, :, a:z]
                    else:
                        c[..., r, dst, :, :rest, :] = old[..., r, src, :, :rest, :]
    return out, new
