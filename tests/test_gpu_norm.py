"""td_norm_rope_kv_append on the GPU against the formula in numpy, 64 bits.

Bound on an element y = a c - b s (a, b normed, c, s its angle): the sum of D <= 128 squares is off by at most
20 roundings in a row (16 products of one lane, 4 exchanges), of which the root takes half; rsqrt adds 2 steps
of 2^-23 and eps, the mean and two products one rounding each: (10 + 4 + 4) * 2^-24 < 2^-19 relative on a and b.
Two products and a sum add 3 * 2^-24 of |a c| + |b s|. So |err| <= 2^-18.5 (|a c| + |b s|) + u |y|, u half a step
of the element type (bf16 2^-8, fp32 2^-24), and u again of the first term."""
import numpy as np
import pytest
import torch

from decode_attention_split_gb300.workloads import rope_tables

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
U = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


@pytest.fixture(scope="module")
def td():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from decode_attention_split_gb300 import build
    build.build()
    import decode_attention_split_gb300 as td
    return td


class Problem:
    def __init__(self, dtype, D, T, Smax, lens, Hq=3, Hkv=2, A=0, seed=0, rows=None):
        rng = np.random.default_rng(seed)
        B = len(lens)
        self.dtype, self.T, self.Smax, self.D, self.A = dtype, T, Smax, D, A
        self.lens = lens

        def draw(*s):
            return torch.from_numpy(rng.normal(size=s) * np.exp(2.0 * rng.normal(size=s[:-1] + (1,)))).to(DT[dtype])
        self.q, self.kn, self.vn = draw(B, Hq, T, D), draw(B, Hkv, T, D), draw(B, Hkv, T, D)
        self.kc, self.vc = draw(B, Hkv, Smax, D), draw(B, Hkv, Smax, D)
        self.qw = torch.from_numpy(rng.normal(size=D)).float()
        self.kw = torch.from_numpy(1 + 0.3 * rng.normal(size=D)).float()
        self.cos, self.sin = rope_tables(Smax if rows is None else rows, D)
        self.pos = self.axes = None
        if A:
            self.pos = torch.from_numpy(rng.integers(0, self.cos.shape[0], size=(B, T, A))).int()
            self.axes = torch.from_numpy(rng.integers(0, A, size=D // 2)).int()
        self.eps = 1e-5

    def call(self, td, advance=True, q=True, stream=None, inplace=False, st=None):
        c = lambda t: None if t is None else t.cuda()
        self.g = dict(kc=c(self.kc), vc=c(self.vc), lens=torch.tensor(self.lens, dtype=torch.int32).cuda(), q=c(self.q),
                      st=torch.zeros(1, dtype=torch.int32, device="cuda") if st is None else st)
        g = self.g
        g["q_out"] = td.td_norm_rope_kv_append(
            c(self.kn), c(self.vn), g["kc"], g["vc"], g["lens"], c(self.kw), c(self.cos), c(self.sin), eps=self.eps,
            positions=c(self.pos), axes=c(self.axes), q=g["q"] if q else None, q_weight=c(self.qw) if q else None,
            q_out=g["q"] if q and inplace else None, advance=advance, dev_status=g["st"], stream=stream)
        return g

    def formula(self, x, w, L, b):
        """x [H, T, D] normed and rotated, and the sums of magnitudes its bound takes."""
        h = self.D // 2
        x = x.double().numpy()
        y = x * w.double().numpy() / np.sqrt((x * x).mean(-1, keepdims=True) + self.eps)
        c, s = np.ones((self.T, h)), np.zeros((self.T, h))
        for t in range(self.T):
            for i in range(h):
                if self.pos is None:
                    p = L + t
                else:
                    a = 0 if self.axes is None else int(self.axes[i])
                    p = int(self.pos[b, t, a]) if 0 <= a < self.A else -1
                if 0 <= p < self.cos.shape[0]:
                    c[t, i], s[t, i] = self.cos[p, i], self.sin[p, i]
        lo, hi = y[..., :h], y[..., h:]
        ref = np.concatenate([lo * c - hi * s, hi * c + lo * s], -1)
        mag = np.concatenate([abs(lo * c) + abs(hi * s), abs(hi * c) + abs(lo * s)], -1)
        return ref, mag

    def close(self, got, ref, mag):
        u = U[self.dtype]
        err = np.abs(got.double().numpy() - ref)
        bound = 2.0 ** -18.5 * mag * (1 + u) + u * np.abs(ref) + 1e-38
        assert np.all(err <= bound), float((err / bound).max())

    def check(self, advance=True, q=True):
        g = {k: None if v is None else v.cpu() for k, v in self.g.items()}
        kc, vc = self.kc.clone(), self.vc.clone()
        over = False
        for b, L in enumerate(self.lens):
            if L < 0 or L + self.T > self.Smax:
                over = True
                assert int(g["lens"][b]) == L
                continue
            assert int(g["lens"][b]) == L + (self.T if advance else 0)
            self.close(g["kc"][b, :, L:L + self.T], *self.formula(self.kn[b], self.kw, L, b))
            kc[b, :, L:L + self.T] = g["kc"][b, :, L:L + self.T]
            vc[b, :, L:L + self.T] = self.vn[b]
            if q:
                self.close(g["q_out"][b], *self.formula(self.q[b], self.qw, L, b))
        # every other row of the caches, bit for bit
        bits = torch.int16 if self.dtype == "bf16" else torch.int32
        assert torch.equal(g["kc"].view(bits), kc.view(bits)) and torch.equal(g["vc"].view(bits), vc.view(bits))
        assert bool(int(g["st"]) & 2) == over


CASES = [
    # dtype, D, T, Smax, lengths, Hq, Hkv, axes
    ("bf16", 128, 1, 64, [0, 1, 63, 64, -1, 17], 3, 2, 0),
    ("bf16", 64, 1, 40, [5, 39], 15, 5, 0),
    ("f32", 128, 1, 50, [0, 49, 7], 4, 1, 0),
    ("f32", 64, 1, 33, [32, 33, 3], 7, 7, 0),
    ("bf16", 128, 2, 64, [0, 61, 62, 63], 5, 1, 0),
    ("bf16", 64, 7, 64, [3, 57, 58], 3, 3, 0),
    ("f32", 128, 16, 64, [0, 48], 3, 2, 0),
    ("bf16", 128, 33, 100, [0, 67, 68], 24, 8, 0),
    ("f32", 64, 100, 333, [7, 233, 234], 3, 1, 0),
    ("bf16", 64, 301, 700, [1, 399], 16, 2, 0),
    ("bf16", 128, 1, 64, [0, 9, 63], 32, 8, 1),
    ("bf16", 128, 45, 100, [0, 9], 8, 4, 3),
    ("f32", 128, 5, 64, [3, 59], 3, 2, 16),
    ("bf16", 128, 1, 16, list(range(16)), 64, 8, 0),
    ("f32", 64, 1, 8, [i % 9 for i in range(77)], 1, 1, 2),
]


@pytest.mark.parametrize("advance", [True, False])
@pytest.mark.parametrize("case", CASES)
def test_against_formula(td, case, advance):
    dtype, D, T, Smax, lens, Hq, Hkv, A = case
    p = Problem(dtype, D, T, Smax, lens, Hq, Hkv, A, seed=T + D, rows=50 if A else None)
    p.call(td, advance)
    p.check(advance)


@pytest.mark.parametrize("T", [1, 40])
def test_without_queries(td, T):
    p = Problem("bf16", 128, T, 64, [0, 24])
    p.call(td, q=False)
    assert p.g["q_out"] is None
    p.check(q=False)


@pytest.mark.parametrize("dtype,D,T,Hkv,A", [("bf16", 128, 32, 1, 0), ("bf16", 64, 300, 8, 0), ("f32", 128, 16, 3, 3),
                                              ("f32", 64, 1000, 2, 1), ("bf16", 128, 2000, 8, 0)])
def test_chunks_without_queries(td, dtype, D, T, Hkv, A):
    """No queries and no weights of theirs, in chunks of one head a CTA and of several: the keys and values are those of
    the call with queries, bit for bit."""
    p = Problem(dtype, D, T, T + 9, [0, 9, 10], Hkv=Hkv, A=A, rows=50 if A else None, seed=T)
    g = p.call(td, q=False)
    assert g["q_out"] is None
    kc, vc, lens = g["kc"].clone(), g["vc"].clone(), g["lens"].clone()
    assert int(g["st"]) == td.DEV_APPEND_OVERFLOW
    if T < 500:
        p.check(q=False)
    g = p.call(td)
    bits = torch.int16 if dtype == "bf16" else torch.int32
    assert torch.equal(g["kc"].view(bits), kc.view(bits)) and torch.equal(g["vc"].view(bits), vc.view(bits))
    assert torch.equal(g["lens"], lens)


@pytest.mark.parametrize("dtype,T", [("bf16", 1), ("f32", 19)])
def test_queries_in_place(td, dtype, T):
    p = Problem(dtype, 64, T, 64, [4, 11])
    g = p.call(td, inplace=True)
    assert g["q_out"].data_ptr() == g["q"].data_ptr()
    p.check()


def test_queries_of_a_sequence_that_does_not_fit_stay(td):
    p = Problem("bf16", 128, 3, 16, [13, 14])
    g = p.call(td, inplace=True)
    assert torch.equal(g["q"][1].cpu(), p.q[1])
    p.check()


@pytest.mark.parametrize("T", [9, 100])
def test_a_chunk_longer_than_the_cache_is_left_out(td, T):
    """Its tokens have neither cache rows nor table rows."""
    p = Problem("bf16", 128, T, 8, [0, 3])
    g = p.call(td, inplace=True)
    assert torch.equal(g["q"].cpu(), p.q)
    p.check()


@pytest.mark.parametrize("T", [1, 21, 50])
def test_bad_positions_leave_their_pairs(td, T):
    p = Problem("bf16", 128, T, 64, [2, 30], A=3, rows=40)
    p.pos[0, T // 2, 1] = 40
    p.pos[1, 0, 2] = -1
    p.axes[5] = 3
    p.axes[9] = -2
    g = p.call(td)
    # the second sequence's 50 tokens do not fit behind its 30 rows
    assert int(g["st"]) == td.DEV_BAD_POSITION | (td.DEV_APPEND_OVERFLOW if 30 + T > 64 else 0)
    p.check()


def test_positions_equal_to_the_rows_give_the_same_bits(td):
    a = Problem("bf16", 128, 9, 64, [2, 30], seed=3)
    b = Problem("bf16", 128, 9, 64, [2, 30], seed=3)
    b.pos = (torch.tensor(b.lens)[:, None, None] + torch.arange(9)[None, :, None]).int()
    b.A = 1
    ga, gb = a.call(td), b.call(td)
    assert torch.equal(ga["kc"], gb["kc"]) and torch.equal(ga["q_out"], gb["q_out"])


def test_rows_of_zeros_nan_and_infinity(td):
    p = Problem("f32", 64, 4, 16, [5], Hq=1, Hkv=1)
    p.kn[0, 0, 0] = 0.0
    p.kn[0, 0, 1, 3] = float("nan")
    p.kn[0, 0, 2, 3] = float("inf")
    g = p.call(td, q=False)
    k = g["kc"][0, 0, 5:9].cpu()
    assert torch.equal(k[0], torch.zeros(64))
    assert k[1].isnan().all()
    other = [i for i in range(64) if i not in (3, 35)]
    assert k[2, [3, 35]].isnan().all() and torch.equal(k[2, other], torch.zeros(62))
    ref, mag = p.formula(p.kn[0], p.kw, 5, 0)
    p.close(k[3], ref[0, 3], mag[0, 3])


def test_stream_and_graph(td):
    """Captured once, replayed twice with the lengths moving on the device; each replay as an eager call."""
    p = Problem("bf16", 128, 2, 64, [0, 20], seed=4)
    s = torch.cuda.Stream()
    g = p.call(td, stream=s)
    torch.cuda.synchronize()
    p.check()
    args = [t.cuda() for t in (p.kn, p.vn, p.kc, p.vc)]
    lens = torch.tensor(p.lens, dtype=torch.int32).cuda()
    kw, qw, cos, sin, q = (t.cuda() for t in (p.kw, p.qw, p.cos, p.sin, p.q))
    q_out = torch.empty_like(q)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        td.td_norm_rope_kv_append(*args, lens, kw, cos, sin, eps=p.eps, q=q, q_weight=qw, q_out=q_out)
    for i in range(2):
        graph.replay()
        torch.cuda.synchronize()
        for b, L in enumerate(p.lens):
            at = L + 2 * i
            assert int(lens[b]) == at + 2
            p.close(args[2][b, :, at:at + 2].cpu(), *p.formula(p.kn[b], p.kw, at, b))
            p.close(q_out[b].cpu(), *p.formula(p.q[b], p.qw, at, b))


def test_a_plain_append_of_normed_rows_is_the_same_cache(td):
    """Unit weights on rows whose mean square is 1 - eps exactly: the call is td_rope_kv_append bit for bit."""
    p = Problem("f32", 64, 3, 32, [4], Hq=2, Hkv=1)
    sign = torch.from_numpy(np.random.default_rng(1).choice([-1.0, 1.0], size=(1, 1, 3, 64))).float()
    p.kn, p.kw, p.eps = sign, torch.ones(64), 3.0          # mean square 1, plus 3: divided by 2 exactly
    g = p.call(td, q=False)
    kc, vc, lens = p.kc.cuda(), p.vc.cuda(), torch.tensor(p.lens, dtype=torch.int32).cuda()
    td.td_rope_kv_append((sign / 2).cuda(), p.vn.cuda(), kc, vc, lens, p.cos.cuda(), p.sin.cuda())
    err = (g["kc"] - kc).abs().max()
    assert float(err) <= 2.0 ** -22 and torch.equal(g["vc"], vc) and torch.equal(g["lens"], lens)
