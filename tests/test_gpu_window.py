"""Attention over a sliding window with sinks on the GPU against plain masked attention in 64 bits
(masked_ref), the bounds of parity.py. Rows that no token of a call sees hold NaN in every test."""
import numpy as np
import pytest
import torch

from decode_attention_split_gb300.workloads import rope_tables
from masked_ref import check, check_large, rising_keys, window_mask

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


class Problem:
    def __init__(self, dtype, D, Hq, Hkv, T, S, lens, window, sinks, seed=0):
        g = torch.Generator().manual_seed(seed)
        B = len(lens)
        self.T, self.S, self.lens, self.window, self.sinks = T, S, lens, window, sinks
        self.q = torch.randn(B, Hq, T, D, generator=g).to(DT[dtype])
        k, v = torch.randn(B, Hkv, S, D, generator=g), torch.randn(B, Hkv, S, D, generator=g)
        k = torch.where(torch.rand(B, Hkv, S, 1, generator=g) < 0.02, 4 * k, k)
        self.see = window_mask(lens, T, S, window, sinks)
        hidden = torch.from_numpy(~self.see.any(1))[:, None, :, None]
        self.k, self.v = (x.masked_fill(hidden, float("nan")).to(DT[dtype]) for x in (k, v))
        self.scale = D ** -0.5

    def status(self):
        bits = 0
        for L in self.lens:
            bits |= (8 if L < 0 else 0) | (1 if L > self.S else 0)
            bits |= 4 if self.T > 1 and min(max(L, 0), self.S) < self.T else 0
        return bits

    def run(self, td, prompt=False, **kw):
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        lens = torch.tensor(self.lens, dtype=torch.int32).cuda()
        q, decode = self.q.cuda(), self.T == 1 and not prompt
        call = td.td_prefill_attn_window if prompt else td.td_decode_attn_window if decode else td.td_verify_attn_window
        out, lse = call(q[:, :, 0].contiguous() if decode else q, self.k.cuda(), self.v.cuda(), lens, self.window, self.sinks,
                        scale=self.scale, dev_status=st, return_lse=True, **kw)
        torch.cuda.synchronize()
        assert int(st) == self.status()
        return out.cpu().view(self.q.shape), lse.cpu().view(self.q.shape[:-1])

    def check(self, out, lse, what=""):
        check(out, lse, self.q, self.k, self.v, self.see, self.scale, what)


# sizes of window and sinks around the 16-row boxes, the 64-row stages and the lengths
SHAPES = [(1, 0), (1, 1), (5, 0), (16, 4), (33, 16), (64, 17), (100, 64), (63, 65), (200, 130), (290, 4), (299, 1), (300, 0),
          (1000, 0), (7, 300), (250, 51), (128, 4)]


@pytest.mark.parametrize("window,sinks", SHAPES)
@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("bf16", 64), ("f32", 64), ("f32", 128)])
def test_decode(td, dtype, D, window, sinks):
    """Few groups: the cluster kernel (bf16)."""
    p = Problem(dtype, D, 6, 2, 1, 300, [300, 1, 0, 77, 299, 304, -3, window + sinks + 1, window + sinks], window, sinks, seed=1)
    p.check(*p.run(td))


@pytest.mark.parametrize("window,sinks", SHAPES)
@pytest.mark.parametrize("dtype,D,G,T", [("bf16", 128, 4, 6), ("bf16", 64, 3, 2), ("bf16", 128, 2, 5), ("f32", 64, 3, 4),
                                         ("bf16", 128, 7, 9)])
def test_verify(td, dtype, D, G, T, window, sinks):
    p = Problem(dtype, D, 2 * G, 2, T, 300, [300, T, 150, T - 1, 299], window, sinks, seed=2)
    p.check(*p.run(td))


@pytest.mark.parametrize("dtype,D,G,T", [("bf16", 128, 4, 1), ("bf16", 64, 12, 1), ("bf16", 128, 4, 6), ("f32", 64, 8, 1),
                                         ("bf16", 64, 5, 3), ("bf16", 128, 8, 5)])
@pytest.mark.parametrize("window,sinks", [(100, 4), (500, 20), (1, 0), (3000, 70)])
def test_many_sequences(td, dtype, D, G, T, window, sinks):
    """Many groups: the persistent kernel, several items a CTA."""
    S = 1500
    lens = [int(x) for x in np.random.default_rng(3).integers(T, S + 1, size=40)] + [S, T]
    p = Problem(dtype, D, 4 * G, 4, T, S, lens, window, sinks, seed=3)
    p.check(*p.run(td))


@pytest.mark.parametrize("split", [16, 48, 64, 160, 1024])
@pytest.mark.parametrize("dtype,T", [("bf16", 1), ("bf16", 6), ("f32", 1), ("f32", 3)])
def test_given_split(td, dtype, T, split):
    for window, sinks in ((100, 4), (333, 70), (40, 0)):
        p = Problem(dtype, 128 if T == 6 else 64, 4, 1, T, 700, [700, 431, T], window, sinks, seed=4)
        p.check(*p.run(td, split=split), what=f"window {window}")


@pytest.mark.parametrize("L", [5000, 32768])
def test_long_context(td, L):
    """The window of a token far into its context, most of which holds NaN."""
    p = Problem("bf16", 128, 6, 2, 1, L, [L], 4096, 4, seed=5)
    p.check(*p.run(td))


def test_window_of_the_whole_cache_is_the_plain_call(td):
    """The same keys, in the same chunks where those are multiples of 16: the same bits."""
    for T in (1, 6):
        p = Problem("bf16", 128, 8, 2, T, 512, [512, 400], 512, 0, seed=6)
        out, lse = p.run(td)
        q = p.q.cuda()
        args = (p.k.cuda(), p.v.cuda(), torch.tensor(p.lens, dtype=torch.int32).cuda(), p.scale)
        plain, plain_lse = td.td_decode_attn(q[:, :, 0].contiguous(), *args, return_lse=True) if T == 1 else \
            td.td_verify_attn(q, *args, return_lse=True)
        assert torch.equal(out, plain.cpu().view(out.shape)) and torch.equal(lse, plain_lse.cpu().view(lse.shape))


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (5, 3), (64, 4), (100, 70), (128, 0), (200, 64), (333, 130),
                                          (1000, 5), (20, 1000)])
@pytest.mark.parametrize("B,Hq,Hkv,D,S,T,lens", [
    (1, 4, 2, 128, 300, 300, [300]),
    (2, 6, 2, 64, 520, 260, [400, 260]),
    (1, 2, 2, 128, 1000, 129, [1000]),
    (2, 3, 1, 128, 700, 200, [455, 190]),             # the second chunk is longer than its sequence
    (3, 2, 1, 64, 70, 1, [70, 0, 33]),
])
def test_prompt(td, B, Hq, Hkv, D, S, T, lens, window, sinks):
    p = Problem("bf16", D, Hq, Hkv, T, S, lens, window, sinks, seed=7)
    # a tile's tokens share its weights' zeros: what one of them sees has to be finite for all
    p.check(*p.run(td, prompt=True))


def test_prompt_matches_verify(td):
    p = Problem("bf16", 128, 24, 8, 256, 1024, [1000], 300, 4, seed=8)
    a, la = p.run(td, prompt=True)
    b, lb = p.run(td)
    p.check(a, la)
    p.check(b, lb)


@pytest.mark.parametrize("rise", [7, 9, 31, 34, 90, 200])
@pytest.mark.parametrize("size", [0, 100])
@pytest.mark.parametrize("D,window,sinks", [(128, 1000, 0), (64, 300, 4), (128, 257, 70)])
def test_prompt_of_rising_scores(td, D, window, sinks, size, rise):
    """A row's maximum moves many tiles after its first, by less and by more than its reference is let to lag (its sums are
    rescaled then), under values of magnitude 2^size: as far as the plain call stays finite, so does this one."""
    B, Hkv, G, T, S = 1, 2, 2, 200, 700
    g = torch.Generator().manual_seed(rise)
    p = Problem("bf16", D, Hkv * G, Hkv, T, S, [S], window, sinks, seed=17)
    q = torch.randn(Hkv, G * T, D, generator=g)
    p.k = rising_keys(q, S, rise, g)[None].bfloat16()
    p.q = q.view(B, Hkv * G, T, D).bfloat16()
    p.v = (torch.randn(B, Hkv, S, D, generator=g) * 2.0 ** size).bfloat16()
    out, lse = p.run(td, prompt=True)
    check_large(out, lse, p.q, p.k, p.v, p.see, p.scale)
    plain = td.td_prefill_attn(p.q.cuda(), p.k.cuda(), p.v.cuda(), torch.tensor([S], dtype=torch.int32).cuda())
    assert plain.isfinite().all()


@pytest.mark.parametrize("scale", [0.0, -0.05])
def test_zero_and_negative_scale(td, scale):
    for prompt, T in ((False, 1), (False, 4), (True, 200)):
        p = Problem("bf16", 128, 4, 2, T, 400, [390], 90, 5, seed=9)
        p.scale = scale
        p.check(*p.run(td, prompt=prompt))


def test_a_layer_from_prompt_to_tokens(td):
    """A windowed layer as it is used: the prompt's rows normed, rotated and appended, its attention, then a verify chunk
    and single tokens; each attention against the plain one over the rows in the cache."""
    D, Hq, Hkv, S, window, sinks = 128, 8, 2, 260, 48, 4
    g = torch.Generator().manual_seed(13)

    def draw(*s):
        return torch.randn(*s, generator=g).bfloat16().cuda()
    kc, vc = draw(2, Hkv, S, D), draw(2, Hkv, S, D)
    lens = torch.tensor([0, 17], dtype=torch.int32).cuda()
    w = (1 + 0.1 * torch.randn(D, generator=g)).cuda()
    cos, sin = (t.cuda() for t in rope_tables(S, D))
    for step, T in enumerate((200, 6, 1, 1, 3)):
        q = td.td_norm_rope_kv_append(draw(2, Hkv, T, D), draw(2, Hkv, T, D), kc, vc, lens, w, cos, sin,
                                      q=draw(2, Hq, T, D), q_weight=w)
        if T > 100:
            out, lse = td.td_prefill_attn_window(q, kc, vc, lens, window, sinks, return_lse=True)
        elif T > 1:
            out, lse = td.td_verify_attn_window(q, kc, vc, lens, window, sinks, return_lse=True)
        else:
            out, lse = td.td_decode_attn_window(q[:, :, 0].contiguous(), kc, vc, lens, window, sinks, return_lse=True)
        torch.cuda.synchronize()
        check(out.cpu().view(q.shape), lse.cpu().view(q.shape[:-1]), q.cpu(), kc.cpu(), vc.cpu(),
              window_mask(lens.tolist(), T, S, window, sinks), D ** -0.5, f"step {step}")
    assert lens.tolist() == [211, 228]


def test_types_in_turn_on_kept_workspaces(td):
    """Both types of one shape without a workspace: their layouts differ (24 rows are one row block in bf16, six in fp32)."""
    lens = [4000, 3000, 2000, 1000, 500, 4000, 100, 3999]
    p = {dt: Problem(dt, 128, 32, 8, 6, 4000, lens, 2500, 16, seed=15) for dt in DT}
    want = {dt: [x.clone() for x in p[dt].run(td, workspace=torch.zeros(
        td.td_window_workspace_bytes(8, 32, 8, 4000, 128, 2500, 16, q_len=6), dtype=torch.uint8, device="cuda"))] for dt in DT}
    for dt in ("bf16", "f32", "bf16", "f32"):
        assert all(torch.equal(x, y) for x, y in zip(p[dt].run(td), want[dt])), dt


def test_the_largest_batch(td):
    lens = [(11 * i) % 41 for i in range(1024)]
    p = Problem("bf16", 64, 2, 1, 1, 40, lens, 9, 2, seed=14)
    p.check(*p.run(td))


def test_own_workspace_streams_and_graph(td):
    """One workspace for calls of one shape; a captured step replayed while the lengths move on the device."""
    window, sinks, S = 100, 4, 500
    p = Problem("bf16", 128, 8, 2, 1, S, [90, 450], S, 0, seed=10)      # finite rows everywhere below the lengths
    n = td.td_window_workspace_bytes(2, 8, 2, S, 128, window, sinks)
    assert n > 0 and td.td_window_workspace_bytes(2, 8, 2, S, 128, 0, 0) == 0
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    q, k, v = p.q[:, :, 0].contiguous().cuda(), p.k.cuda().nan_to_num(), p.v.cuda().nan_to_num()
    lens = torch.tensor(p.lens, dtype=torch.int32).cuda()
    out, lse = torch.empty_like(q), torch.empty(2, 8, device="cuda")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(2):
        td.td_decode_attn_window(q, k, v, lens, window, sinks, out=out, lse=lse, workspace=ws, stream=s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        td.td_decode_attn_window(q, k, v, lens, window, sinks, out=out, lse=lse, workspace=ws)
        lens += 1
    for i in range(4):
        graph.replay()
        torch.cuda.synchronize()
        check(out.cpu()[:, :, None], lse.cpu()[:, :, None], p.q, k.cpu(), v.cpu(),
              window_mask([x + i for x in p.lens], 1, S, window, sinks), 128 ** -0.5, f"replay {i}")
    with pytest.raises(RuntimeError, match="workspace"):
        td.td_decode_attn_window(q, k, v, lens, window, sinks, workspace=ws[:256])


def test_capture_needs_its_own_workspace(td):
    p = Problem("bf16", 64, 2, 1, 1, 64, [64], 8, 1)
    q, k, v = p.q[:, :, 0].contiguous().cuda(), p.k.cuda(), p.v.cuda()
    lens = torch.tensor(p.lens, dtype=torch.int32).cuda()
    out = torch.empty_like(q)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        with pytest.raises(ValueError, match="captured"):
            td.td_decode_attn_window(q, k, v, lens, 8, 1, out=out)
        out.zero_()


def test_two_streams_at_once(td):
    """The kept workspaces are one per stream."""
    ps = [Problem("bf16", 128, 8, 2, 1, 3000, [3000, 2500, 1], 700 + 100 * i, 4, seed=20 + i) for i in range(2)]
    args = [(p.q[:, :, 0].contiguous().cuda(), p.k.cuda(), p.v.cuda(), torch.tensor(p.lens, dtype=torch.int32).cuda())
            for p in ps]
    streams = [torch.cuda.Stream() for _ in ps]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(20):
        for i, (p, a, s) in enumerate(zip(ps, args, streams)):
            outs[i].append(td.td_decode_attn_window(*a, p.window, p.sinks, stream=s, return_lse=True))
    torch.cuda.synchronize()
    for p, got in zip(ps, outs):
        for out, lse in got:
            p.check(out.cpu()[:, :, None], lse.cpu()[:, :, None])
