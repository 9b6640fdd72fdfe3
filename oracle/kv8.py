"""CPU oracle of the 8-bit KV cache path -- TEST INFRASTRUCTURE ONLY.

Plain numpy in float64, straight from the definitions, one sequence, head and
block at a time; shares no code with the CUDA library.
"""
from __future__ import annotations

import numpy as np

E_MIN, E_MAX = -110, 119


def turns(rope_dims, base=10000.0, scaling="none", factor=1.0, orig_len=0.0, fast=32.0, slow=1.0):
    """Turns per token of each pair."""
    out = []
    for p in range(rope_dims // 2):
        t = base ** (-2.0 * p / rope_dims)
        if scaling == "linear":
            t /= factor
        elif scaling == "parts":
            r = orig_len * t / (2.0 * np.pi)
            g = min(max((r - slow) / (fast - slow), 0.0), 1.0)
            t = t * (g + (1.0 - g) / factor)
        out.append(t / (2.0 * np.pi))
    return np.array(out)


def norm_rope(x, pos, turn, rope_off, layout, gain=None, eps=1e-6, norm=True, mscale=1.0):
    """x [R][n][d] at positions pos [R] -> (values, |a| + |b| of each rotated
    element and |x| of the others, the scale its rounding errors go by)."""
    y = np.array(x, dtype=np.float64)
    if norm:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps)
        if gain is not None:
            y = y * np.asarray(gain, dtype=np.float64)
    mag = np.abs(y)
    out = y.copy()
    half = len(turn)
    for p in range(half):
        a, b = (rope_off + p, rope_off + half + p) if layout == "half" else \
            (rope_off + 2 * p, rope_off + 2 * p + 1)
        ang = 2.0 * np.pi * np.mod(np.asarray(pos, dtype=np.float64) * turn[p], 1.0)
        c, s = np.cos(ang)[:, None] * mscale, np.sin(ang)[:, None] * mscale
        out[..., a] = y[..., a] * c - y[..., b] * s
        out[..., b] = y[..., a] * s + y[..., b] * c
        mag[..., a] = mag[..., b] = (np.abs(y[..., a]) + np.abs(y[..., b])) * abs(mscale)
    return out, mag


def e4m3_table():
    """Values of the 256 codes (0x7f and 0xff are NaN)."""
    v = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = np.nan if (c & 0x7f) == 0x7f else (m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10))
        v[c] = -x if c & 0x80 else x
    return v


_TAB = e4m3_table()
_POS = _TAB[:127]


def e4m3_encode(y):
    """Nearest code, ties to the even one, saturating; NaN becomes 0."""
    y = np.asarray(y, dtype=np.float64)
    a = np.minimum(np.abs(np.where(np.isnan(y), 0.0, y)), 448.0)
    hi = np.clip(np.searchsorted(_POS, a), 1, 126)
    lo = hi - 1
    dl, dh = a - _POS[lo], _POS[hi] - a
    code = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    return (code + np.where(np.signbit(y) & ~np.isnan(y), 128, 0)).astype(np.uint8)


def exponent(amax):
    """Least e with amax <= 448 * 2^e, in range."""
    if amax <= 0:
        return E_MIN
    e = E_MIN
    while e < E_MAX and amax > 448.0 * 2.0 ** e:
        e += 1
    return e


def append(x, n_old, n_new, codes, exps, block):
    """x [B][T][H][d] (fp64) into codes [B][H][N][d] and exps [B][H][N/block],
    in place."""
    B, T, H, d = x.shape
    N = codes.shape[2]
    for b in range(B):
        end = min(n_old[b] + n_new[b], N)
        for i in range(n_old[b] // block, -(-end // block)):
            s0 = i * block
            lo, hi = max(n_old[b], s0), min(end, s0 + block)
            if lo >= hi:
                continue
            for h in range(H):
                new = x[b, lo - n_old[b]: hi - n_old[b], h]
                fin = np.abs(new[np.isfinite(new)])
                e = exponent(fin.max() if fin.size else 0.0)
                if lo > s0:
                    was = int(exps[b, h, i]) - 127
                    e = max(e, was)
                    if e > was:
                        codes[b, h, s0:lo] = e4m3_encode(_TAB[codes[b, h, s0:lo]] * 2.0 ** (was - e))
                codes[b, h, lo:hi] = e4m3_encode(new * 2.0 ** -e)
                exps[b, h, i] = e + 127


def values(codes, exps, block):
    """Stored values [..][N][d] of codes and exponent bytes."""
    e = np.repeat(exps.astype(np.float64) - 127.0, block, axis=-1)
    return _TAB[codes] * 2.0 ** e[..., None]


def attend(q, n_vis, K, V, block, scale, sink=None):
    """q [B Q][n_q][d], K and V [B][H][N][d] -> out [B Q][n_q][d], the block
    weights [B][H][N/block], and for tolerances: sum p |v| as out, and the
    largest sum |q||k| * scale of each row's visible slots [B Q][n_q]."""
    R, n_q, d = q.shape
    B, H, N, _ = K.shape
    Q, G = R // B, n_q // H
    out, mag = np.zeros((R, n_q, d)), np.zeros((R, n_q, d))
    load = np.zeros((R, n_q))
    w = np.zeros((B, H, N // block))
    for r in range(R):
        n = min(max(int(n_vis[r]), 0), N)
        if n == 0:
            continue
        for h in range(n_q):
            k, v = K[r // Q, h // G, :n], V[r // Q, h // G, :n]
            s = scale * (k @ q[r, h])
            load[r, h] = abs(scale) * (np.abs(k) @ np.abs(q[r, h])).max()
            top = s.max() if sink is None else max(s.max(), sink[h])
            p = np.exp(s - top)
            den = p.sum() + (0.0 if sink is None else np.exp(sink[h] - top))
            p = p / den
            out[r, h] = p @ v
            mag[r, h] = p @ np.abs(v)
            w[r // Q, h // G] += np.add.reduceat(np.pad(p, (0, N - n)), np.arange(0, N, block))
    return out, w, mag, load


def evict(acc, n_tok, keep, recent, block):
    """(kept [B][H][keep], acc_out, n_tok_out) of the eviction; kept is the
    list of moves as well."""
    B, H, NB = acc.shape
    kept = np.full((B, H, keep), -1, dtype=np.int32)
    acc_out = np.zeros_like(acc)
    n_out = np.array(n_tok).copy()
    for b in range(B):
        nb = -(-int(n_tok[b]) // block)
        for h in range(H):
            if nb <= keep:
                src = list(range(nb))
            else:
                old = range(nb - recent)
                order = sorted(old, key=lambda i: (np.isnan(acc[b, h, i]), -acc[b, h, i] if not
                                                   np.isnan(acc[b, h, i]) else 0.0, i))
                stay = sorted(order[: keep - recent]) + list(range(nb - recent, nb))
                up = [i for i in stay[:-1] if i >= keep - 1]
                src = [i if i in set(stay) else up.pop(0) for i in range(keep - 1)] + [nb - 1]
            kept[b, h, : len(src)] = src
            acc_out[b, h, : len(src)] = acc[b, h, src]
        if nb > keep:
            n_out[b] = int(n_tok[b]) - (nb - keep) * block
    return kept, acc_out, n_out
