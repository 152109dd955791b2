"""A NaN in a key makes the rows that see it NaN in out and in lse, whichever kernel takes the call and however the keys are
cut and merged, and changes no other row by a bit. (-inf in lse says "no keys", and a caller who joins parts by it would
leave the part out.)"""
import numpy as np
import pytest
import torch

from masked_ref import window_mask

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def td():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from decode_attention_split_gb300 import build
    build.build()
    import decode_attention_split_gb300 as td
    return td


def attend(td, kind, q, k, v, lens, window, sinks, split):
    T = q.shape[2]
    a = (k.cuda(), v.cuda(), torch.tensor(lens, dtype=torch.int32).cuda())
    kw = dict(return_lse=True) if kind == "prompt" else dict(return_lse=True, split=split)
    w = () if window is None else (window, sinks)
    name = {"prompt": "td_prefill_attn", "token": "td_decode_attn" if T == 1 else "td_verify_attn"}[kind]
    call = getattr(td, name + ("" if window is None else "_window"))
    q = q.cuda()
    out, lse = call(q[:, :, 0].contiguous() if T == 1 and kind == "token" else q, *a, *w, **kw)
    torch.cuda.synchronize()
    return out.cpu().view(q.shape), lse.cpu().view(q.shape[:-1])


# kind, dtype, D, query heads a kv head, T, lengths, split: the cluster kernel, the persistent one with one chunk and with
# several (merged by the last CTA; 24 rows by the last tickets' CTAs), the CUDA-core kernel, the prompt's
SHAPES = [
    ("token", "bf16", 128, 4, 1, [17, 1], 0),
    ("token", "bf16", 128, 4, 1, [900, 17], 0),
    ("token", "bf16", 64, 12, 1, [900, 333], 0),
    ("token", "bf16", 128, 4, 1, [900, 17], 96),
    ("token", "bf16", 128, 4, 1, [900, 17], 1024),
    ("token", "bf16", 64, 12, 1, [900, 17], 64),
    ("token", "bf16", 128, 4, 6, [900, 401], 0),
    ("token", "bf16", 128, 4, 6, [900, 401], 64),
    ("token", "bf16", 128, 4, 6, [900, 401], 160),
    ("token", "bf16", 128, 4, 6, [900, 401], 1024),
    ("token", "bf16", 64, 3, 5, [900, 401], 48),
    ("token", "bf16", 128, 4, 6, [900] * 20, 0),
    ("token", "f32", 64, 2, 1, [900, 17], 0),
    ("token", "f32", 128, 3, 4, [900, 401], 0),
    ("token", "f32", 64, 8, 3, [900, 401], 64),
    ("prompt", "bf16", 128, 2, 200, [900, 401], 0),
    ("prompt", "bf16", 64, 3, 129, [900, 129], 0),
    ("prompt", "bf16", 128, 1, 1, [65, 1], 0),
]


@pytest.mark.parametrize("window,sinks", [(None, 0), (300, 4), (1000, 0)])
@pytest.mark.parametrize("shape", SHAPES)
def test_nan_keys(td, shape, window, sinks):
    kind, dtype, D, G, T, lens, split = shape
    B, Hkv, S = len(lens), 2, 1000
    g = torch.Generator().manual_seed(T + D)
    q = torch.randn(B, Hkv * G, T, D, generator=g).to(DT[dtype])
    k, v = (torch.randn(B, Hkv, S, D, generator=g).to(DT[dtype]) for _ in range(2))
    see = window_mask(lens, T, S, S if window is None else window, sinks)
    want, want_lse = attend(td, kind, q, k, v, lens, window, sinks, split)
    assert want.isfinite().all() and want_lse.isfinite().all()
    # the last key, one that a warp has alone (16 keys a warp), sinks, keys that some tokens' windows have passed
    for j in (-1, 16, 0, 3, 601, 640, 101):
        bad = k.clone()
        hit = np.zeros((B, Hkv, T), bool)
        for b, L in enumerate(lens):
            at = L - 1 if j < 0 else j
            if at < L:
                bad[b, b % Hkv, at, 5] = float("nan")
                hit[b, b % Hkv] = see[b, :, at]
        out, lse = attend(td, kind, q, bad, v, lens, window, sinks, split)
        hit = torch.from_numpy(hit).repeat_interleave(G, dim=1)
        assert out[hit].isnan().all() and lse[hit].isnan().all(), f"key {j}"
        assert torch.equal(out[~hit], want[~hit]) and torch.equal(lse[~hit], want_lse[~hit]), f"key {j}"


@pytest.mark.parametrize("T,split", [(1, 0), (1, 64), (6, 0), (6, 64)])
def test_nan_key_scales_of_an_8_bit_cache(td, T, split):
    """The same merges."""
    B, Hkv, G, S, D, L = 1, 2, 4, 512, 128, 500
    g = torch.Generator().manual_seed(T)
    q = torch.randn(B, Hkv * G, T, D, generator=g).bfloat16().cuda()
    kc, vc = (torch.randint(-127, 128, (B, Hkv, S, D), generator=g, dtype=torch.int8).cuda() for _ in range(2))
    ks, vs = (torch.rand(B, Hkv, S, generator=g).cuda() / 64 for _ in range(2))
    lens = torch.tensor([L], dtype=torch.int32).cuda()
    call = td.td_decode_attn_q8 if T == 1 else td.td_verify_attn_q8
    qq = q[:, :, 0].contiguous() if T == 1 else q
    want, want_lse = (x.cpu() for x in call(qq, kc, ks, vc, vs, lens, split=split, return_lse=True))
    ks[0, 1, 77] = float("nan")
    out, lse = (x.cpu() for x in call(qq, kc, ks, vc, vs, lens, split=split, return_lse=True))
    assert out[:, G:].isnan().all() and lse[:, G:].isnan().all()
    assert torch.equal(out[:, :G], want[:, :G]) and torch.equal(lse[:, :G], want_lse[:, :G])
