"""Attention under any mask in numpy, 64 bits, with the sums that parity.value_bound takes."""
import numpy as np
import torch

from parity import assert_lse_close, assert_out_close, value_bound


def attend(q, k, v, see, scale):
    """q [H, T, D] of one kv head's query heads, k and v [S, D], see [T, S] -> out [H, T, D], lse [H, T] and
    parity.value_stats' three sums. Unseen rows of k and v may hold anything."""
    j = np.flatnonzero(see.any(0))
    H, T, D = q.shape
    out, lse = np.zeros((H, T, D)), np.full((H, T), -np.inf)
    s1, s2, a = np.zeros((H, T, D)), np.zeros((H, T)), np.zeros((H, T, D))
    if j.size:
        x = scale * np.einsum("htd,jd->htj", q, k[j])
        x = np.where(see[None][:, :, j], x, -np.inf)
        m = x.max(-1, keepdims=True)
        p = np.exp(x - np.where(np.isfinite(m), m, 0.0))
        tot = p.sum(-1, keepdims=True)
        w = p / np.where(tot > 0, tot, 1.0)
        out = w @ v[j]
        with np.errstate(divide="ignore"):
            lse = (m + np.log(tot))[..., 0]
        s1, s2, a = np.sqrt((w * w) @ (v[j] ** 2)), np.sqrt((w * w).sum(-1)), w @ np.abs(v[j])
    return out, lse, (s1, s2, a)


def check(out, lse, q, k, v, see, scale, what=""):
    """Torch results [B, Hq, T, D] and [B, Hq, T] against attend() on the torch inputs; see [B, T, S]."""
    B, Hq, T, D = q.shape
    Hkv = k.shape[1]
    G = Hq // Hkv
    bf16 = q.dtype == torch.bfloat16
    for b in range(B):
        for h in range(Hkv):
            heads = slice(h * G, (h + 1) * G)
            ref, rl, stats = attend(q[b, heads].double().numpy(), k[b, h].double().numpy(), v[b, h].double().numpy(),
                                    see[b], scale)
            name = f"{what} sequence {b} kv head {h}"
            got = out[b, heads].double().numpy()
            if bf16:
                assert_out_close(out[b, heads], ref, "bf16", what=name)
                err = np.abs(got - ref)
                bound = value_bound(ref, stats)
                assert np.all(err <= bound), f"{name}: worst err/bound {float((err / bound).max()):.2f}"
            else:
                # fp32 products, sums and weights: a few roundings of 2^-24 on scores of up to about 30, so weights
                # to 1e-5, of the values' weighted magnitude
                err = np.abs(got - ref)
                bound = 2e-5 * stats[2] + 1e-6
                assert np.all(err <= bound), f"{name}: worst err/bound {float((err / bound).max()):.2f}"
            if lse is not None:
                assert_lse_close(lse[b, heads], rl, what=name)


def window_mask(lens, T, S, window, sinks):
    """see [B, T, S] of a sliding window with sinks; lengths as the library clamps them."""
    L = np.clip(np.asarray(lens, np.int64), 0, S)[:, None, None]
    p = L - T + np.arange(T)[None, :, None]
    j = np.arange(S)[None, None, :]
    return (j <= p) & ((j > p - window) | (j < sinks))


def rising_keys(q, S, rise, g, period=None):
    """Keys [Hkv, S, D] over which the scores q k D^-1/2 of every row of q [Hkv, T, D] rise by `rise` (base 2) from the first
    to the last (with a period: and again from each multiple of it on), give or take a hundredth and the rows' noise; q is
    made alike within a head: a direction and a little of its own per row."""
    Hkv, T, D = q.shape
    u = torch.randn(Hkv, 1, D, generator=g)
    u *= D ** 0.5 / u.norm(dim=-1, keepdim=True)
    q.copy_(u + 0.002 * q)
    n = S if period is None else period
    ramp = (torch.arange(S) % n / (n - 1.0) * rise / 1.4426950408889634)[None, :, None]
    return u * ramp * D ** -0.5 + 0.002 * torch.randn(Hkv, S, D, generator=g)


def check_large(out, lse, q, k, v, see, scale, what=""):
    """check() for values far from 1: the value bound alone, whose terms all follow the values' size, and lse."""
    G = q.shape[1] // k.shape[1]
    for b in range(q.shape[0]):
        for h in range(k.shape[1]):
            heads = slice(h * G, (h + 1) * G)
            ref, rl, stats = attend(q[b, heads].double().numpy(), k[b, h].double().numpy(), v[b, h].double().numpy(),
                                    see[b], scale)
            got = out[b, heads].double().numpy()
            name = f"{what} sequence {b} kv head {h}"
            assert np.isfinite(got).all(), f"{name}: not finite"
            err, bound = np.abs(got - ref), value_bound(ref, stats)
            assert np.all(err <= bound), f"{name}: worst err/bound {float((err / bound).max()):.2f}"
            assert_lse_close(lse[b, heads], rl, what=name)
