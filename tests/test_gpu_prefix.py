"""Attention over a shared prefix and each sequence's own keys on the GPU against plain masked attention over
both in 64 bits (masked_ref), the bounds of parity.py. Rows that no token sees hold NaN in every test."""
import threading

import numpy as np
import pytest
import torch

from decode_attention_split_gb300.workloads import rope_tables
from masked_ref import check, check_large, rising_keys

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def td():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from decode_attention_split_gb300 import build
    build.build()
    import decode_attention_split_gb300 as td
    return td


class Problem:
    def __init__(self, D, Hq, Hkv, T, Pmax, P, S, lens, seed=0):
        g = torch.Generator().manual_seed(seed)
        B = len(lens)
        self.T, self.Pmax, self.P, self.S, self.lens = T, Pmax, P, S, lens
        bf = torch.bfloat16
        self.q = torch.randn(B, Hq, T, D, generator=g).to(bf)
        kp, vp = torch.randn(Hkv, Pmax, D, generator=g), torch.randn(Hkv, Pmax, D, generator=g)
        kp = torch.where(torch.rand(Hkv, Pmax, 1, generator=g) < 0.02, 4 * kp, kp)
        k, v = torch.randn(B, Hkv, S, D, generator=g), torch.randn(B, Hkv, S, D, generator=g)
        self.n = min(max(P, 0), Pmax)
        L = np.clip(np.asarray(lens, np.int64), 0, S)[:, None, None]
        own = np.arange(S)[None, None] < L - T + 1 + np.arange(T)[None, :, None]
        self.see = np.concatenate([np.broadcast_to(np.arange(Pmax) < self.n, (B, T, Pmax)), own], axis=2)
        hidden = torch.from_numpy(~own.any(1))[:, None, :, None]
        self.k, self.v = (x.masked_fill(hidden, float("nan")).to(bf) for x in (k, v))
        kp[:, self.n:], vp[:, self.n:] = float("nan"), float("nan")
        self.kp, self.vp = kp.to(bf), vp.to(bf)
        self.scale = D ** -0.5

    def status(self):
        bits = (8 if self.P < 0 else 0) | (1 if self.P > self.Pmax else 0)
        for L in self.lens:
            bits |= (8 if L < 0 else 0) | (1 if L > self.S else 0)
            bits |= 4 if self.T > 1 and min(max(L, 0), self.S) < self.T else 0
        return bits

    def args(self):
        q = self.q.cuda()
        return (q[:, :, 0].contiguous() if self.T == 1 else q, self.kp.cuda(), self.vp.cuda(),
                torch.tensor([self.P], dtype=torch.int32).cuda(), self.k.cuda(), self.v.cuda(),
                torch.tensor(self.lens, dtype=torch.int32).cuda())

    def run(self, td, **kw):
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        call = td.td_decode_attn_prefix if self.T == 1 else td.td_verify_attn_prefix
        out, lse = call(*self.args(), scale=self.scale, dev_status=st, return_lse=True, **kw)
        torch.cuda.synchronize()
        assert int(st) == self.status()
        return out.cpu().view(self.q.shape), lse.cpu().view(self.q.shape[:-1])

    def check(self, out, lse, what=""):
        B = len(self.lens)
        both = [torch.cat([p[None].expand(B, -1, -1, -1), x], dim=2) for p, x in ((self.kp, self.k), (self.vp, self.v))]
        check(out, lse, self.q, *both, self.see, self.scale, what)


PREFIXES = [0, 1, 63, 64, 65, 128, 130, 500, 999, 1000, 1001, -2]


@pytest.mark.parametrize("P", PREFIXES)
@pytest.mark.parametrize("D,Hq,Hkv", [(128, 6, 2), (64, 5, 1), (64, 16, 2)])
def test_decode(td, D, Hq, Hkv, P):
    p = Problem(D, Hq, Hkv, 1, 1000, P, 200, [200, 1, 0, 77, 201, -1], seed=1)
    p.check(*p.run(td))


@pytest.mark.parametrize("P", PREFIXES)
@pytest.mark.parametrize("D,G,T", [(128, 4, 6), (64, 7, 5), (128, 8, 20), (64, 1, 2), (128, 3, 4)])
def test_verify(td, D, G, T, P):
    """Row counts of a sequence that divide 128, do not, and pass it; the last sequence is shorter than its chunk."""
    p = Problem(D, 2 * G, 2, T, 1000, P, 150, [150, T, 99, T - 1], seed=2)
    p.check(*p.run(td))


@pytest.mark.parametrize("D,G,T,B", [(128, 4, 1, 70), (64, 8, 1, 64), (128, 1, 3, 90), (64, 3, 6, 33), (128, 16, 1, 41)])
@pytest.mark.parametrize("P", [17, 700, 2048])
def test_many_sequences(td, D, G, T, B, P):
    """Several tiles of 128 rows a kv head, the last one partly filled; many groups of own keys."""
    lens = [int(x) for x in np.random.default_rng(3).integers(T, 301, size=B)]
    p = Problem(D, 3 * G, 3, T, 2048, P, 300, lens, seed=3)
    p.check(*p.run(td))


def test_more_tiles_than_slots(td):
    """600 sequences: more tiles of rows than the GPU holds CTAs, one chunk each."""
    B = 600
    p = Problem(64, 16 * 8, 8, 1, 192, 130, 16, [1 + i % 16 for i in range(B)], seed=4)
    out, lse = p.run(td)
    for b in range(0, B, 37):
        q = Problem.__new__(Problem)
        q.__dict__.update(p.__dict__, lens=p.lens[b:b + 1], q=p.q[b:b + 1], k=p.k[b:b + 1], v=p.v[b:b + 1], see=p.see[b:b + 1])
        q.check(out[b:b + 1], lse[b:b + 1], f"sequence {b}")


def test_long_prefix(td):
    p = Problem(128, 6, 2, 1, 33000, 32003, 100, [100, 3, 0], seed=5)
    p.check(*p.run(td))


@pytest.mark.parametrize("scale", [0.0, -0.05])
def test_zero_and_negative_scale(td, scale):
    for T in (1, 4):
        p = Problem(128, 4, 2, T, 300, 290, 100, [90, 100], seed=6)
        p.scale = scale
        p.check(*p.run(td))


def test_a_large_maximum_late_in_the_prefix(td):
    """Scores that rise by hundreds from tile to tile: the running maximum moves and the sums are rescaled."""
    p = Problem(128, 8, 2, 1, 640, 640, 64, [64, 1], seed=7)
    ramp = torch.linspace(0, 6, 640)[None, :, None]
    p.kp = (p.q[0, 0, 0].float() * ramp + 0.1 * p.kp.float()).to(torch.bfloat16)
    p.check(*p.run(td))


@pytest.mark.parametrize("rise", [7, 9, 31, 34, 90, 200])
@pytest.mark.parametrize("size", [0, 100])
@pytest.mark.parametrize("D,G,T", [(128, 4, 1), (64, 3, 6)])
def test_rising_scores(td, D, G, T, size, rise):
    """The same, by less and by more than the reference is let to lag, under values of magnitude 2^size."""
    period = 384                    # three tiles of keys, and with two kv heads and 76 periods so is a chunk
    B, Hkv, P, S = 2, 2, 76 * period, 100
    g = torch.Generator().manual_seed(rise)
    p = Problem(D, Hkv * G, Hkv, T, P, P, S, [S, S - 7], seed=8)
    q = torch.randn(Hkv, B * G * T, D, generator=g)
    p.kp = rising_keys(q, P, rise, g, period).bfloat16()
    p.q = q.view(Hkv, B, G, T, D).transpose(0, 1).reshape(B, Hkv * G, T, D).bfloat16()
    p.k, p.v = p.k.nan_to_num(), (p.v.nan_to_num().float() * 2.0 ** size).bfloat16()
    p.vp = (p.vp.float() * 2.0 ** size).bfloat16()
    out, lse = p.run(td)
    both = [torch.cat([a[None].expand(B, -1, -1, -1), x], dim=2) for a, x in ((p.kp, p.k), (p.vp, p.v))]
    check_large(out, lse, p.q, *both, p.see, p.scale)
    plain = td.td_verify_attn(p.q.cuda(), *(x.cuda() for x in both), torch.tensor([P + S] * B, dtype=torch.int32).cuda())
    assert plain.isfinite().all()


@pytest.mark.parametrize("T", [1, 5])
def test_nan_reaches_the_rows_that_see_it_and_no_other(td, T):
    D, Hq, Hkv, S = 128, 8, 2, 100
    p = Problem(D, Hq, Hkv, T, 500, 500, S, [100, 60, T], seed=31)
    clean, clean_lse = p.run(td)
    p.kp[1, 300, 7] = float("nan")                    # a key of the prefix, kv head 1
    out, lse = p.run(td)
    assert torch.equal(out[:, :4], clean[:, :4]) and torch.equal(lse[:, :4], clean_lse[:, :4])
    assert out[:, 4:].isnan().all() and lse[:, 4:].isnan().all()
    p = Problem(D, Hq, Hkv, T, 500, 500, S, [100, 60, T], seed=31)
    p.v[1, 0, 20, 5] = float("nan")                   # a value element of sequence 1, kv head 0
    p.k[2, 1, 0, 0] = float("inf")                    # a key of sequence 2, kv head 1
    out, lse = p.run(td)
    assert out[1, :4, :, 5].isnan().all() and torch.equal(out[1, :4, :, 6:], clean[1, :4, :, 6:])
    # its scores are infinite with the query element's sign: infinity makes a row NaN, minus infinity weighs nothing
    up = (p.q[2, 4:, :, 0] > 0)
    sees = torch.from_numpy(p.see[2, :, p.Pmax])
    assert torch.equal(out[2, 4:].isnan().all(-1), up & sees)
    assert out[2, 4:].isfinite().all(-1).equal(~(up & sees))
    assert torch.equal(out[0], clean[0]) and torch.equal(out[1, 4:], clean[1, 4:]) and torch.equal(out[2, :4], clean[2, :4])


def test_a_long_chunk_behind_a_prefix(td):
    """A hundred new tokens a sequence: many row blocks over the own keys, tiles of rows inside one sequence."""
    p = Problem(64, 6, 2, 100, 400, 333, 180, [180, 100, 133], seed=32)
    p.check(*p.run(td))


@pytest.mark.parametrize("D,T,P", [(128, 1, 5), (64, 6, 0), (128, 3, 2000)])
def test_long_own_keys_of_few_sequences(td, D, T, P):
    """Each row's own keys in many runs (more parts than the join takes at a time), behind a short prefix or none."""
    p = Problem(D, 4, 1, T, 2000, P, 20000, [20000, 0 if T == 1 else T, 13001], seed=34)
    p.check(*p.run(td))


def test_any_workspace_contents(td):
    p = Problem(128, 8, 2, 6, 700, 650, 300, [300, 6, 90, 2], seed=35)
    q = p.q.shape
    want = p.run(td)
    for fill in (0, 255, 127):
        n = td.td_prefix_workspace_bytes(q[0], q[1], 2, 700, 300, 128, 6)
        got = p.run(td, workspace=torch.full((n,), fill, dtype=torch.uint8, device="cuda"))
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_the_largest_batch(td):
    B = 1024
    lens = [(7 * i) % 33 for i in range(B)]
    p = Problem(64, 2, 1, 1, 100, 77, 32, lens, seed=33)
    out, lse = p.run(td)
    p.check(out, lse)


def test_empty_everywhere(td):
    p = Problem(128, 4, 2, 1, 64, 0, 32, [0, 0], seed=8)
    out, lse = p.run(td)
    assert torch.equal(out, torch.zeros_like(out)) and torch.isneginf(lse).all()


def test_the_split_point_does_not_matter(td):
    """The same keys as prefix and own keys, cut at different places, and as one plain cache."""
    D, Hq, Hkv, N = 128, 8, 2, 600
    g = torch.Generator().manual_seed(9)
    q = torch.randn(1, Hq, D, generator=g).bfloat16().cuda()
    k, v = (torch.randn(1, Hkv, N, D, generator=g).bfloat16().cuda() for _ in range(2))
    want, lse = td.td_decode_attn(q, k, v, torch.tensor([N], dtype=torch.int32).cuda(), return_lse=True)
    for cut in (1, 64, 333, 599):
        out, got = td.td_decode_attn_prefix(q, k[0, :, :cut].contiguous(), v[0, :, :cut].contiguous(),
                                            torch.tensor([cut], dtype=torch.int32).cuda(), k[:, :, cut:].contiguous(),
                                            v[:, :, cut:].contiguous(), torch.tensor([N - cut], dtype=torch.int32).cuda(),
                                            return_lse=True)
        # two roundings to bf16 of values below 1, and weights rounded to bf16 in different chunks
        assert float((out.float() - want.float()).abs().max()) <= 2 * 2.0 ** -8
        assert float((got - lse).abs().max()) <= 1e-4


def _steps(td, sync, steps=12, seed=10):
    """Steps of a batch behind a prefix: rows normed, rotated behind the prefix and appended, then attended; every
    step's queries come from the step before."""
    D, Hq, Hkv, B, P, S = 128, 8, 2, 6, 300, 64
    g = torch.Generator().manual_seed(seed)

    def draw(*s):
        return torch.randn(*s, generator=g).bfloat16().cuda()
    kp, vp = draw(Hkv, P, D), draw(Hkv, P, D)
    kc, vc = draw(B, Hkv, S, D), draw(B, Hkv, S, D)
    q = draw(B, Hq, 1, D)
    kn, vn = [draw(B, Hkv, 1, D) for _ in range(steps)], [draw(B, Hkv, 1, D) for _ in range(steps)]
    w = torch.ones(D).cuda()
    cos, sin = (t.cuda() for t in rope_tables(P + S, D))
    lens = torch.arange(B, dtype=torch.int32).cuda()
    plen = torch.tensor([P], dtype=torch.int32).cuda()
    outs = []
    for i in range(steps):
        pos = (plen + lens)[:, None, None].contiguous()
        if sync:
            torch.cuda.synchronize()
        r = td.td_norm_rope_kv_append(kn[i], vn[i], kc, vc, lens, w, cos, sin, positions=pos, q=q, q_weight=w)
        if sync:
            torch.cuda.synchronize()
        out = td.td_decode_attn_prefix(r[:, :, 0].contiguous(), kp, vp, plen, kc, vc, lens)
        if sync:
            torch.cuda.synchronize()
        outs.append(out)
        q = (out + q[:, :, 0])[:, :, None].contiguous()
    torch.cuda.synchronize()
    return outs, kc, vc, lens


def test_steps_in_a_row_give_what_steps_one_by_one_give(td):
    """The launches overlap their neighbours' ends: the same bits as with a synchronisation between all calls."""
    for seed in range(4):
        a, ka, va, la = _steps(td, False, seed=seed)
        b, kb, vb, lb = _steps(td, True, seed=seed)
        assert all(torch.equal(x, y) for x, y in zip(a, b))
        assert torch.equal(ka, kb) and torch.equal(va, vb) and torch.equal(la, lb)


def test_graph_of_a_step(td):
    """Append and attention captured, replayed with the lengths moving on the device."""
    p = Problem(128, 8, 2, 1, 400, 333, 64, [5, 20, 1], seed=11)
    q, kp, vp, plen, k, v, lens = p.args()
    k, v = k.nan_to_num(), v.nan_to_num()
    g = torch.Generator().manual_seed(12)
    kn, vn = (torch.randn(3, 2, 1, 128, generator=g).bfloat16().cuda() for _ in range(2))
    ws = torch.zeros(td.td_prefix_workspace_bytes(3, 8, 2, 400, 64, 128), dtype=torch.uint8, device="cuda")
    out, lse = torch.empty_like(q), torch.empty(3, 8, device="cuda")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    td.td_decode_attn_prefix(q, kp, vp, plen, k, v, lens, out=out, lse=lse, workspace=ws, stream=s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        td.td_kv_append(kn, vn, k, v, lens)
        td.td_decode_attn_prefix(q, kp, vp, plen, k, v, lens, out=out, lse=lse, workspace=ws)
    for i in range(3):
        plen.fill_(333 - 50 * i)
        graph.replay()
        torch.cuda.synchronize()
        want = Problem(128, 8, 2, 1, 400, 333 - 50 * i, 64, [x + i + 1 for x in p.lens], seed=11)
        want.q, want.k, want.v, want.kp, want.vp = p.q, k.cpu(), v.cpu(), p.kp, p.vp
        want.check(out.cpu()[:, :, None], lse.cpu()[:, :, None], f"replay {i}")
    with pytest.raises(RuntimeError, match="workspace"):
        td.td_decode_attn_prefix(q, kp, vp, plen, k, v, lens, workspace=ws[:-256])


def test_two_streams_at_once(td):
    ps = [Problem(128, 8, 2, 1, 1500, 1400 + i, 200, [200, 50, 0], seed=20 + i) for i in range(2)]
    args = [p.args() for p in ps]
    streams = [torch.cuda.Stream() for _ in ps]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            outs[i].append(td.td_decode_attn_prefix(*args[i], stream=s, return_lse=True))
    torch.cuda.synchronize()
    for p, got in zip(ps, outs):
        for out, lse in got:
            assert torch.equal(out, got[0][0]) and torch.equal(lse, got[0][1])
        p.check(got[0][0].cpu()[:, :, None], got[0][1].cpu()[:, :, None])


def test_two_threads_on_one_stream(td):
    """Calls of two threads share a stream and, without one of their own, a workspace."""
    ps = [Problem(128, 8, 2, 1, 1500, 1400 + i, 200, [200, 50 + i, 0], seed=40 + i) for i in range(2)]
    args = [p.args() for p in ps]
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = [[], []]

    def work(i):
        for _ in range(200):
            outs[i].append(td.td_decode_attn_prefix(*args[i], stream=stream, return_lse=True))
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for p, got in zip(ps, outs):
        assert len(got) == 200
        for out, lse in got:
            assert torch.equal(out, got[0][0]) and torch.equal(lse, got[0][1])
        p.check(got[0][0].cpu()[:, :, None], got[0][1].cpu()[:, :, None])


def test_capture_needs_its_own_workspace(td):
    p = Problem(64, 2, 1, 1, 64, 64, 32, [3], seed=30)
    args = p.args()
    out = torch.empty_like(args[0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        with pytest.raises(ValueError, match="captured"):
            td.td_decode_attn_prefix(*args, out=out)
        out.zero_()
