"""Plain definitions of the cache operators in 64 bits (NumPy), with the error bounds
their roundings allow.  Test infrastructure: one sequence, head and row at a time."""
import math

import numpy as np

D = 128
U16, U32 = 2.0 ** -8, 2.0 ** -24      # half a step of bf16 and of fp32, relative to the value


def gather(x, table, b, h, t):
    """Rows t of (b, h): contiguous [B, Hkv, N, w] or pages [n, Hkv, P, w] behind table."""
    t = np.asarray(t, np.int64)
    if table is None:
        return x[b, h, t]
    P = x.shape[2]
    return x[table[b][t // P], h, t % P]


# ---------------------------------------------------------------- rotary positions
def rotate(x, pos, freqs, rot, interleaved, mscale):
    """fp32 arithmetic of the definition, step by step: x [heads, 128] float32 (bf16
    values) at one position; returns float32 before the rounding to bf16."""
    turn = (np.asarray(freqs, np.uint64) * np.uint64(pos % (1 << 64))).astype(np.int64)
    ang = turn.astype(np.float64) * 2.0 ** -63 * math.pi
    c, s = (np.cos(ang) * mscale).astype(np.float32), (np.sin(ang) * mscale).astype(np.float32)
    y = x.copy()
    i1 = np.arange(0, rot, 2) if interleaved else np.arange(rot // 2)
    i2 = i1 + 1 if interleaved else i1 + rot // 2
    a, b = x[:, i1], x[:, i2]
    y[:, i1] = a * c - b * s
    y[:, i2] = b * c + a * s
    return y


def rotate64(x, pos, freq, rot, interleaved, mscale):
    """The definition in 64 bits from the frequencies in radians."""
    ang = (pos * freq) % (2 * math.pi)
    c, s = np.cos(ang) * mscale, np.sin(ang) * mscale
    x = x.astype(np.float64)
    y = x.copy()
    i1 = np.arange(0, rot, 2) if interleaved else np.arange(rot // 2)
    i2 = i1 + 1 if interleaved else i1 + rot // 2
    y[:, i1] = x[:, i1] * c - x[:, i2] * s
    y[:, i2] = x[:, i2] * c + x[:, i1] * s
    return y


# ---------------------------------------------------------------- attention of a chunk
def score_error(q, K):
    """Largest error of an fp32 score of q [128] with K [n, 128]: 128 exact products
    summed in some order (each partial sum rounded, or cut: one step), then scaled
    and its maximum subtracted (two more roundings, of the score's size)."""
    mag = np.abs(K) @ np.abs(q) / math.sqrt(D)
    return (2 * 128 + 8) * U32 * mag


def attend(q, K, V, cu, lens, table):
    """q [T, Hq, 128], caches as float64 arrays.  Returns out, lse, and their bounds."""
    T, Hq, _ = q.shape
    Hkv = K.shape[1]
    G = Hq // Hkv
    out, lse = np.zeros((T, Hq, D)), np.zeros((T, Hq))
    tol, ltol = np.zeros((T, Hq, D)), np.zeros((T, Hq))
    for b in range(len(lens)):
        n = cu[b + 1] - cu[b]
        for h in range(Hq):
            rows = np.arange(max(0, int(lens[b])))
            Kb, Vb = gather(K, table, b, h // G, rows), gather(V, table, b, h // G, rows)
            for i in range(n):
                r, at = cu[b] + i, lens[b] - n + i
                if at < 0:
                    lse[r, h] = -math.inf
                    continue
                k, v = Kb[: at + 1], Vb[: at + 1]
                s = k @ q[r, h] / math.sqrt(D)
                m = s.max()
                p = np.exp(s - m)
                l = p.sum()
                es = score_error(q[r, h], k).max()
                # the probabilities' own rounding, exp's (2^-21) and the sums'
                each = U16 + 2 * es + 2.0 ** -21 + (at + 9) * U32
                out[r, h] = p @ v / l
                lse[r, h] = m + math.log(l)
                tol[r, h] = (each * 1.01) * (p @ np.abs(v)) / l + U16 * np.abs(out[r, h]) + es * np.abs(out[r, h]) + 1e-30
                ltol[r, h] = es + 2.0 ** -21 + (at + 9) * U32 + 4 * U32 * (abs(m) + abs(lse[r, h]))
    return out, lse, tol, ltol


def accumulate_chunk(q, K, lse, cu, lens, mass, table):
    T, Hq, _ = q.shape
    G = Hq // K.shape[1]
    mass, tol = mass.astype(np.float64), np.zeros(mass.shape)
    for b in range(len(lens)):
        n = cu[b + 1] - cu[b]
        for h in range(Hq):
            Kb = gather(K, table, b, h // G, np.arange(max(0, int(lens[b]))))
            for i in range(n):
                r, at = cu[b] + i, lens[b] - n + i
                if at < 0 or lse[r, h] == -math.inf:
                    continue
                p = np.exp(Kb[: at + 1] @ q[r, h] / math.sqrt(D) - lse[r, h])
                mass[b, h // G, : at + 1] += p
                es = score_error(q[r, h], Kb[: at + 1]) + 4 * U32 * abs(lse[r, h])
                tol[b, h // G, : at + 1] += p * (1.01 * es + 2.0 ** -21)
    return mass, tol + (len(q) * Hq + 4) * U32 * np.abs(mass)


def accumulate_kept(q, K, idx, lens, mass, table):
    B, Hq, _ = q.shape
    Hkv = K.shape[1]
    G = Hq // Hkv
    mass, tol = mass.astype(np.float64), np.zeros(mass.shape)
    for b in range(B):
        for h in range(Hq):
            t = idx[b, h if idx.shape[1] == Hq else h // G]
            t = t[(t >= 0) & (t < lens[b])]
            if not len(t):
                continue
            k = gather(K, table, b, h // G, t)
            s = k @ q[b, h] / math.sqrt(D)
            p = np.exp(s - s.max())
            p /= p.sum()
            mass[b, h // G, t] += p
            es = score_error(q[b, h], k).max()
            tol[b, h // G, t] += p * (2.02 * es + 2.0 ** -20 + (len(t) + 9) * U32)
    return mass, tol + (G + 4) * U32 * np.abs(mass)


# ---------------------------------------------------------------- eviction
def evict_select(mass, lens, keep, n_sink, n_recent):
    """kept [B, Hkv, keep] (old slots ascending, -1 behind) and the new lengths."""
    B, Hkv, N = mass.shape
    kept = np.full((B, Hkv, keep), -1, np.int32)
    for b in range(B):
        L = int(lens[b])
        k = min(keep, L)
        for h in range(Hkv):
            def rank(t):
                if t < n_sink or t >= L - n_recent:
                    return (0, 0.0, t)
                x = float(mass[b, h, t])
                return (2, 0.0, t) if x != x else (1, -x, t)
            kept[b, h, :k] = sorted(sorted(range(L), key=rank)[:k])
    return kept, np.minimum(lens, keep).astype(np.int32)
