"""The normed append, windowed and shared-prefix attention at the ends of what their calls allow: the smallest sizes, caches
past 2^32 bytes, CTAs that take full and partly filled tiles in turn, steps in a row and captured ones."""
import numpy as np
import pytest
import torch

from decode_attention_split_gb300.workloads import rope_tables
from masked_ref import check, window_mask

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def td():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from decode_attention_split_gb300 import build
    build.build()
    import decode_attention_split_gb300 as td
    return td


def ints(*x):
    return torch.tensor(x, dtype=torch.int32).cuda()


def draw(g, *s, dtype=torch.bfloat16):
    return torch.randn(*s, generator=g).to(dtype).cuda()


def prefix_see(B, T, Pmax, P, S, lens):
    own = np.arange(S)[None, None] < np.asarray(lens)[:, None, None] - T + 1 + np.arange(T)[None, :, None]
    return np.concatenate([np.broadcast_to(np.arange(Pmax) < P, (B, T, Pmax)), own], axis=2)


def check_prefix(out, lse, q, kp, vp, P, k, v, lens, picks):
    """The sequences of `picks` against plain attention over prefix and own keys."""
    T = q.shape[2]
    see = prefix_see(len(picks), T, kp.shape[1], P, k.shape[2], [lens[b] for b in picks])
    both = [torch.cat([a[None].expand(len(picks), -1, -1, -1), x[picks]], dim=2).cpu() for a, x in ((kp, k), (vp, v))]
    check(out[picks].cpu(), lse[picks].cpu(), q[picks].cpu(), *both, see, q.shape[-1] ** -0.5)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("P,L", [(1, 1), (0, 1), (1, 0), (0, 0)])
def test_one_key_each(td, D, P, L):
    """One sequence, one head, caches of one row."""
    g = torch.Generator().manual_seed(D)
    q, kp, vp = draw(g, 1, 1, 1, D), draw(g, 1, 1, D), draw(g, 1, 1, D)
    k, v = draw(g, 1, 1, 1, D), draw(g, 1, 1, 1, D)
    out, lse = td.td_decode_attn_prefix(q[:, :, 0], kp, vp, ints(P), k, v, ints(L), return_lse=True)
    check_prefix(out[:, :, None], lse[:, :, None], q, kp, vp, P, k, v, [L], [0])
    see = window_mask([L], 1, 1, 1, 0)
    out, lse = td.td_decode_attn_window(q[:, :, 0], k, v, ints(L), 1, 0, return_lse=True)
    check(out.cpu()[:, :, None], lse.cpu()[:, :, None], q.cpu(), k.cpu(), v.cpu(), see, D ** -0.5)
    out, lse = td.td_prefill_attn_window(q, k, v, ints(L), 1, 0, return_lse=True)
    check(out.cpu(), lse.cpu(), q.cpu(), k.cpu(), v.cpu(), see, D ** -0.5)
    f = [x.float() for x in (q, k, v)]
    out, lse = td.td_decode_attn_window(f[0][:, :, 0], f[1], f[2], ints(L), 1, 0, return_lse=True)
    check(out.cpu()[:, :, None], lse.cpu()[:, :, None], *(x.cpu() for x in f), see, D ** -0.5)


@pytest.mark.parametrize("D,B,G,T,P", [(64, 593, 16, 1, 700), (128, 593, 16, 1, 130), (64, 200, 8, 6, 513), (128, 200, 8, 6, 400)])
def test_full_and_partly_filled_tiles_in_turn(td, D, B, G, T, P):
    """More tiles of rows than the GPU holds CTAs, a kv head's last tile partly filled: a CTA's warps have rows in one of its
    tiles and none in the next, and again."""
    Hkv, S = 8, 20
    g = torch.Generator().manual_seed(B)
    lens = [T + i % (S - T + 1) for i in range(B)]
    q, kp, vp = draw(g, B, Hkv * G, T, D), draw(g, Hkv, P, D), draw(g, Hkv, P, D)
    k, v = draw(g, B, Hkv, S, D), draw(g, B, Hkv, S, D)
    out, lse = td.td_verify_attn_prefix(q, kp, vp, ints(P), k, v, ints(*lens), return_lse=True)
    check_prefix(out, lse, q, kp, vp, P, k, v, lens, list(range(0, B, 29)) + [B - 2, B - 1])
    for _ in range(5):
        again = td.td_verify_attn_prefix(q, kp, vp, ints(P), k, v, ints(*lens), return_lse=True)
        assert torch.equal(again[0], out) and torch.equal(again[1], lse)


def test_long_prefix_offsets(td):
    """A prefix of 1M rows and 20 kv heads (5 GB each of K and V), and own caches as long: the last heads lie past 2^32 bytes."""
    Hkv, D, N = 20, 128, 1 << 20
    kp, vp = (torch.zeros(Hkv, N, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    k, v = (torch.zeros(1, Hkv, N, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    g = torch.Generator().manual_seed(3)
    q = draw(g, 1, Hkv, D)
    for h in (0, Hkv - 1):
        q[0, h] = 4.0
        kp[h, N - 3], k[0, h, N - 2] = 8.0, 8.0                 # scores of 362 and its equal beside zeros: half the weight each
        vp[h, N - 3], v[0, h, N - 2] = 1.0 + h, 3.0 + h
    out, lse = td.td_decode_attn_prefix(q, kp, vp, ints(N), k, v, ints(N), return_lse=True)
    for h in (0, Hkv - 1):
        assert torch.equal(out[0, h], torch.full_like(out[0, h], 2.0 + h))
        assert abs(float(lse[0, h]) - (32 * D ** 0.5 + np.log(2.0))) < 2e-3 + 1e-5 * 363
    out, lse = td.td_decode_attn_window(q, k, v, ints(N), 3, 0, return_lse=True)
    p = td.td_prefill_attn_window(q[:, :, None].contiguous(), k, v, ints(N), 3, 0)
    for h in (0, Hkv - 1):
        assert torch.equal(out[0, h], torch.full_like(out[0, h], 3.0 + h)) and torch.equal(p[0, h, 0], out[0, h])


def test_long_window_and_append_offsets_in_fp32(td):
    Hkv, D, N = 10, 128, 1 << 20
    k, v = (torch.zeros(1, Hkv, N, D, device="cuda") for _ in range(2))
    g = torch.Generator().manual_seed(4)
    cos, sin = (torch.ones(64, D // 2).cuda(), torch.zeros(64, D // 2).cuda())
    w, lens = torch.ones(D).cuda(), ints(N - 40)
    kn, vn = draw(g, 1, Hkv, 40, D, dtype=torch.float32), draw(g, 1, Hkv, 40, D, dtype=torch.float32)
    pos = torch.arange(40, dtype=torch.int32).cuda().view(1, 40, 1)
    td.td_norm_rope_kv_append(kn, vn, k, v, lens, w, cos, sin, eps=1e-6, positions=pos)
    assert int(lens) == N
    want = kn * torch.rsqrt((kn * kn).mean(-1, keepdim=True) + 1e-6)
    assert float((k[:, :, N - 40:] - want).abs().max()) < 1e-5 and torch.equal(v[:, :, N - 40:], vn)
    assert not k[:, :, :N - 40].any()
    q = draw(g, 1, Hkv, 4, D, dtype=torch.float32)
    out, lse = td.td_verify_attn_window(q, k, v, lens, 30, 0, return_lse=True)
    tail = [x[:, :, N - 64:].cpu() for x in (k, v)]
    check(out.cpu(), lse.cpu(), q.cpu(), *tail, window_mask([64], 4, 64, 30, 0), D ** -0.5)


def _window_steps(td, sync, seed):
    """A prompt and then tokens and chunks of a windowed layer; each step's queries come from the step before."""
    D, Hq, Hkv, B, S, window, sinks = 128, 8, 2, 3, 256, 40, 4
    g = torch.Generator().manual_seed(seed)
    kc, vc = draw(g, B, Hkv, S, D), draw(g, B, Hkv, S, D)
    w = torch.ones(D).cuda()
    cos, sin = (t.cuda() for t in rope_tables(S, D))
    lens = ints(0, 5, 17)
    outs = []
    carry = torch.zeros(B, Hq, 1, D, dtype=torch.bfloat16, device="cuda")
    for T in (150, 1, 6, 1, 1, 33, 1, 6, 2):
        q, kn, vn = draw(g, B, Hq, T, D) + carry, draw(g, B, Hkv, T, D), draw(g, B, Hkv, T, D)

        def step():
            if sync:
                torch.cuda.synchronize()
        step()
        r = td.td_norm_rope_kv_append(kn, vn, kc, vc, lens, w, cos, sin, q=q, q_weight=w)
        step()
        if T > 30:
            out = td.td_prefill_attn_window(r, kc, vc, lens, window, sinks)
        elif T > 1:
            out = td.td_verify_attn_window(r, kc, vc, lens, window, sinks)
        else:
            out = td.td_decode_attn_window(r[:, :, 0].contiguous(), kc, vc, lens, window, sinks)[:, :, None]
        step()
        outs.append(out)
        carry = out[:, :, -1:].contiguous()
    torch.cuda.synchronize()
    return outs, kc, vc, lens


def test_windowed_steps_in_a_row_give_what_steps_one_by_one_give(td):
    for seed in range(4):
        a, ka, va, la = _window_steps(td, False, seed)
        b, kb, vb, lb = _window_steps(td, True, seed)
        assert all(torch.equal(x, y) for x, y in zip(a, b))
        assert torch.equal(ka, kb) and torch.equal(va, vb) and torch.equal(la, lb)


def test_graph_of_windowed_and_prefix_prompts(td):
    """Captured prompt and verify calls, replayed over other inputs in the same buffers."""
    D, Hq, Hkv, T, S, P = 64, 6, 2, 130, 300, 200
    g = torch.Generator().manual_seed(5)
    q, k, v = draw(g, 2, Hq, T, D), draw(g, 2, Hkv, S, D), draw(g, 2, Hkv, S, D)
    kp, vp, lens, plen = draw(g, Hkv, P, D), draw(g, Hkv, P, D), ints(300, 140), ints(P)
    q6 = q[:, :, :6].contiguous()
    ws = torch.empty(td.td_prefix_workspace_bytes(2, Hq, Hkv, P, S, D, 6), dtype=torch.uint8, device="cuda")
    wsw = torch.zeros(td.td_window_workspace_bytes(2, Hq, Hkv, S, D, 70, 3, q_len=6), dtype=torch.uint8, device="cuda")

    def calls(outs):
        td.td_prefill_attn_window(q, k, v, lens, 70, 3, out=outs[0], lse=outs[1])
        td.td_verify_attn_window(q6, k, v, lens, 70, 3, out=outs[2], lse=outs[3], workspace=wsw)
        td.td_verify_attn_prefix(q6, kp, vp, plen, k, v, lens, out=outs[4], lse=outs[5], workspace=ws)

    def buffers():
        return [x for t in (q, q6, q6) for x in (torch.empty_like(t), torch.empty(t.shape[:3], device="cuda"))]
    got, want = buffers(), buffers()
    calls(want)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls(got)
    for i in range(3):
        for t in (q, q6, k, v, kp, vp):
            t.copy_(draw(g, *t.shape))
        lens.copy_(ints(300 - 7 * i, 131 + i))
        plen.fill_(P - 60 * i)
        graph.replay()
        calls(want)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), i
