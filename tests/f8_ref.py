"""The block-scaled 8-bit cache in plain numpy, one block at a time: the rules td.h states, sharing
no code with the library. fp32 where td.h says fp32 (the scale ratios), otherwise 64 bits."""
import numpy as np

import oracle

BLOCKS = (16, 32, 64, 128)


def _table():
    v = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = np.nan if (c & 0x7f) == 0x7f else m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        v[c] = -x if c & 0x80 else x
    return v


VALUE = _table()                                  # value of every code
_POS = VALUE[:127]                                # 0 .. 448, ascending
_MID = (_POS[:-1] + _POS[1:]) / 2


def encode(x):
    """Codes of x (any float array): nearest, ties to the even code, saturating; NaN -> 0x7f."""
    x = np.asarray(x, np.float64)
    a = np.abs(np.where(np.isnan(x), 0.0, x))
    c = np.searchsorted(_MID, a, side="left")     # the lower neighbour at a tie
    tie = (c < 126) & (a == _MID[np.minimum(c, 125)])
    c = np.where(tie & (c % 2 == 1), c + 1, c).astype(np.uint8)
    c = np.where(np.signbit(x), c | 0x80, c).astype(np.uint8)
    return np.where(np.isnan(x), np.uint8(0x7f), c)


def pow2_scale(amax):
    """The least 2^k, k >= -126, with amax <= 448 * 2^k."""
    if amax == 0:
        return 2.0 ** -126
    m, e = np.frexp(np.float64(amax))             # amax = m 2^e, m in [0.5, 1); 448 = 0.875 * 2^9
    return 2.0 ** max(int(e) - 9 + (1 if m > 0.875 else 0), -126)


def append(codes, scales, x, lens, block):
    """Rows x [B, H, T, D] (float64 values of the stored elements) into codes uint8 [B, H, S, D] and
    scales float32 [B, H, NB], in place; sequences that do not fit are left alone."""
    B, H, T, D = x.shape
    S = codes.shape[2]
    for b in range(B):
        L = int(lens[b])
        if L < 0 or L + T > S:
            continue
        for j in range(L // block, (L + T - 1) // block + 1):
            r0, r1 = max(L, j * block), min(L + T, (j + 1) * block)
            for h in range(H):
                new = x[b, h, r0 - L:r1 - L]
                fin = np.abs(new[np.isfinite(new)])
                s = np.float32(pow2_scale(fin.max() if fin.size else 0.0))
                if r0 > j * block:
                    old = scales[b, h, j]
                    if s > old:
                        r = np.float32(old) / s
                        part = codes[b, h, j * block:r0]
                        v = VALUE[part].astype(np.float32) * r
                        part[...] = encode(v)
                    s = max(s, old)
                inv = np.float32(1.0) / s
                with np.errstate(over="ignore", invalid="ignore"):
                    y = (new.astype(np.float32) * inv).astype(np.float64)
                y = np.where(np.isfinite(new), y, np.nan)
                codes[b, h, r0:r1] = encode(y)
                scales[b, h, j] = s


def values(codes, scales, block):
    """code * scale in float64 [B, H, S, D] (a NaN code gives NaN)."""
    S = codes.shape[2]
    return VALUE[codes] * np.repeat(scales.astype(np.float64), block, axis=2)[:, :, :S, None]


def rotate(x, cos, sin):
    """Pairs (i, i + D/2) of x [..., D] turned by cos, sin [..., D/2], in 64 bits."""
    h = x.shape[-1] // 2
    lo, hi = x[..., :h], x[..., h:]
    return np.concatenate([lo * cos - hi * sin, hi * cos + lo * sin], axis=-1)


def rotate_keys(x, cos, sin):
    """The keys' rotation as td.h states it: every product and sum rounded to fp32."""
    h = x.shape[-1] // 2
    lo, hi = x[..., :h].astype(np.float32), x[..., h:].astype(np.float32)
    cos, sin = cos.astype(np.float32), sin.astype(np.float32)
    return np.concatenate([lo * cos - hi * sin, hi * cos + lo * sin], axis=-1)


def attention(q, k, v, lens, scale):
    """The oracle's exact attention and lse over float64 values, and per output the sums its
    tolerance needs: (out, lse, status, sum_j w_j |v_j| + 2^-21 sum_j |v_j|, largest
    scale * sum_i |q_i k_i|). v is zero behind the lengths."""
    orc = oracle.load()
    lens = np.ascontiguousarray(lens, np.int32)
    out, lse, st = orc.attention(q, k, v, lens, scale)
    absv, _, _ = orc.attention(q, k, np.abs(v), lens, scale)
    B, Hq, T, _ = q.shape
    G, S = Hq // k.shape[1], k.shape[2]
    absv = absv + 2.0 ** -21 * np.repeat(np.abs(v).sum(axis=2), G, axis=1)[:, :, None]
    big = np.zeros((B, Hq, T))
    for b in range(B):
        n = min(max(int(lens[b]), 0), S)
        for h in range(Hq):
            if n:
                big[b, h] = abs(scale) * (np.abs(q[b, h]) @ np.abs(k[b, h // G, :n]).T).max(axis=1)
    return out, lse, st, absv, big


def bounds(out, lse, absv, big, D, n):
    """How far the kernel's outputs may be from the exact ones.

    A score is a D-term dot product in fp32 (each product exact, at most 2^-23 of the terms' sum of
    magnitudes lost at each of D additions, 2^-22 for the scales and the exponent): off by at most
    e = (D + 4) 2^-23 big, so a weight by a factor e^(2e). A probability is rounded to fp16, 2^7
    above its place: by 2^-11 of it, or below fp16's least normal 2^-14 by an absolute 2^-25, which
    is 2^-32 of the sum of probabilities (the reference key's alone is 2^7). With every key's weight
    w_j |v_j| + 2^-21 |v_j| in absv, 2^-11 absv covers both. The sums over n keys run in fp32 (n 2^-24
    of the terms' magnitudes, in pieces of a warp's share: n / 4 additions at most), and the output
    is rounded to bf16 (2^-8)."""
    e = (D + 4) * 2.0 ** -23 * big
    grow = np.expm1(2 * e) + 2.0 ** -11 + n * 2.0 ** -25
    return (2.0 ** -8 * np.abs(out) + (1 + 2.0 ** -8) * grow[..., None] * absv + 1e-30,
            e + n * 2.0 ** -25 + 2.0 ** -21 * (1 + np.abs(np.where(np.isfinite(lse), lse, 0.0))))
