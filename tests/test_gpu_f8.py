"""The block-scaled 8-bit cache on the GPU against a plain numpy reference (f8_ref): appended codes
and scales bit for bit, read-back bit for bit, attention within a derived bound."""
import math

import numpy as np
import pytest
import torch

import f8_ref
from decode_attention_split_gb300.workloads import rope_tables

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def td():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from decode_attention_split_gb300 import build
    build.build()
    import decode_attention_split_gb300 as td
    return td


DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def f8(codes):
    return torch.from_numpy(codes).view(torch.float8_e4m3fn).cuda()


def codes_of(t):
    return t.view(torch.uint8).cpu().numpy()


def status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def rows(rng, *shape, dtype="bf16", spread=1.0):
    x = rng.normal(size=shape) * np.exp(spread * rng.normal(size=shape[:-1] + (1,)))
    return torch.from_numpy(x).to(DT[dtype])


def filled(rng, B, H, S, D, block, lens=None):
    """A cache as appends leave it (numpy codes, scales), random bytes and NaN scales behind the lengths."""
    NB = -(-S // block)
    x = np.zeros((B, H, NB * block, D))
    x[:, :, :S] = rows(rng, B, H, S, D).double().numpy()
    x = x.reshape(B, H, NB, block, D)
    m, e = np.frexp(np.abs(x).max(axis=(3, 4)))        # f8_ref.pow2_scale of every block
    scales = np.ldexp(1.0, e - 9 + (m > 0.875)).astype(np.float32)
    codes = f8_ref.encode(x / scales[..., None, None]).reshape(B, H, NB * block, D)[:, :, :S].copy()
    if lens is not None:
        for b, L in enumerate(lens):
            L = min(max(int(L), 0), S)
            codes[b, :, L:] = rng.integers(0, 256, size=codes[b, :, L:].shape, dtype=np.uint8)
            scales[b, :, -(-L // block):] = np.nan
    return codes, scales


def same_bits(a, b):
    """Equal codes, any two NaN codes alike."""
    nan = (a & 0x7f) == 0x7f
    return np.array_equal(nan, (b & 0x7f) == 0x7f) and np.array_equal(a[~nan], b[~nan])


# ------------------------------------------------------------------------------- append

APPEND = [
    # dtype, D, block, T, Smax, lengths
    ("bf16", 128, 64, 1, 256, [0, 1, 63, 64, 65, 200, 255]),
    ("bf16", 64, 16, 1, 100, [0, 15, 16, 17, 99, 100, -1]),          # a partial last block; two that do not fit
    ("f32", 128, 32, 1, 96, [0, 5, 31, 95]),
    ("f32", 64, 128, 1, 256, [127, 128, 3]),
    ("bf16", 128, 16, 5, 96, [0, 12, 90, 91, 92]),                   # blocks cut by the chunk; exactly full; too long
    ("bf16", 64, 32, 16, 128, [0, 17, 112, 113]),
    ("bf16", 128, 64, 17, 300, [0, 50, 283, 284]),                   # the first length of the tiled kernel
    ("bf16", 128, 16, 100, 333, [0, 7, 233]),
    ("bf16", 64, 64, 150, 400, [1, 63, 64]),
    ("f32", 128, 128, 200, 500, [0, 100, 300, 301]),
    ("f32", 64, 16, 33, 200, [0, 31]),
    ("bf16", 64, 128, 40, 512, [120, 128, 0]),
    ("bf16", 64, 16, 70, 64, [0, 3]),                                # longer than the cache: nothing fits
    ("bf16", 64, 16, 9, 8, [0, -1]),
    ("bf16", 128, 32, 4, 128, [0, 30, 124, 125]),                    # the most rows of the first kernel for few heads
    ("f32", 128, 16, 12, 64, [(5 * i) % 53 for i in range(70)]),     # and for many
    ("bf16", 64, 64, 13, 64, [(5 * i) % 53 for i in range(70)]),
]


@pytest.mark.parametrize("dtype,D,block,T,S,lens", APPEND)
@pytest.mark.parametrize("advance", [True, False])
def test_append_bit_exact(td, dtype, D, block, T, S, lens, advance):
    rng = np.random.default_rng(D + block + T)
    B, H = len(lens), 3
    kc, ks = filled(rng, B, H, S, D, block, lens)
    vc, vs = filled(rng, B, H, S, D, block, lens)
    kn, vn = rows(rng, B, H, T, D, dtype=dtype), rows(rng, B, H, T, D, dtype=dtype, spread=3.0)
    d = [f8(kc), torch.from_numpy(ks).cuda(), f8(vc), torch.from_numpy(vs).cuda(),
         torch.tensor(lens, dtype=torch.int32, device="cuda")]
    st = status()
    td.td_kv_append_f8(kn.cuda(), vn.cuda(), *d, block, advance=advance, dev_status=st)
    torch.cuda.synchronize()
    fits = [0 <= L and L + T <= S for L in lens]
    f8_ref.append(kc, ks, kn.double().numpy(), lens, block)
    f8_ref.append(vc, vs, vn.double().numpy(), lens, block)
    assert np.array_equal(codes_of(d[0]), kc) and np.array_equal(codes_of(d[2]), vc)
    assert np.array_equal(d[1].cpu().numpy(), ks, equal_nan=True)
    assert np.array_equal(d[3].cpu().numpy(), vs, equal_nan=True)
    assert d[4].cpu().tolist() == [L + T if ok and advance else L for L, ok in zip(lens, fits)]
    assert int(st.item()) == (0 if all(fits) else td.DEV_APPEND_OVERFLOW)


@pytest.mark.parametrize("T", [1, 3, 20])
@pytest.mark.parametrize("old", [2.0 ** -9, 0.0037, 1.0, 2.0 ** -126])
def test_append_grows_a_held_block(td, T, old):
    """A block that holds rows at a smaller scale (powers of two or not) has them brought to the larger
    one; one whose scale is larger keeps it."""
    rng = np.random.default_rng(T)
    B, H, S, D, block = 1, 2, 128, 128, 64
    kc, ks = filled(rng, B, H, S, D, block)
    ks[:] = old
    kn = rows(rng, B, H, T, D)
    kn[:, 0] *= 2.0 ** -20       # head 0's rows are small: its scale is kept
    d = [f8(kc), torch.from_numpy(ks).cuda()]
    lens = torch.tensor([37], dtype=torch.int32, device="cuda")
    td.td_kv_append_f8(kn.cuda(), kn.cuda(), *d, d[0].clone(), d[1].clone(), lens, block)
    torch.cuda.synchronize()
    f8_ref.append(kc, ks, kn.double().numpy(), [37], block)
    assert same_bits(codes_of(d[0]), kc) and np.array_equal(d[1].cpu().numpy(), ks)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 2, 30])
def test_append_extremes(td, dtype, T):
    """Zero rows, the largest and least magnitudes, NaN and infinities."""
    rng = np.random.default_rng(7)
    B, H, S, D, block = 8, 1, 64, 64, 16
    x = rows(rng, B, H, T, D, dtype=dtype)
    x[0] = 0
    x[1] = torch.finfo(DT[dtype]).max
    x[2] *= 2.0 ** -125
    x[3, :, :, 5] = float("nan")
    x[4, :, :, 6] = float("inf")
    x[4, :, :, 7] = float("-inf")
    x[5] = float("nan")
    x[6] = 448.0
    x[7] = -448.0 * (1 + 2.0 ** -7)
    kc, ks = np.zeros((B, H, S, D), np.uint8), np.zeros((B, H, S // block), np.float32)
    d = [f8(kc), torch.from_numpy(ks).cuda()]
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    td.td_kv_append_f8(x.cuda(), x.cuda(), *d, d[0].clone(), d[1].clone(), lens, block)
    torch.cuda.synchronize()
    f8_ref.append(kc, ks, x.double().numpy(), [0] * B, block)
    assert np.array_equal(d[1].cpu().numpy(), ks)
    assert same_bits(codes_of(d[0]), kc)


def test_filled_is_an_append(td):
    """The tests' caches are what the reference's append stores."""
    codes, scales = filled(np.random.default_rng(1), 1, 2, 70, 64, 16)
    x = rows(np.random.default_rng(1), 1, 2, 70, 64).double().numpy()
    kc, ks = np.zeros_like(codes), np.zeros_like(scales)
    f8_ref.append(kc, ks, x, [0], 16)
    assert np.array_equal(kc, codes) and np.array_equal(ks, scales)


def test_append_nothing_else_is_written(td):
    """Bytes of other heads, sequences and rows, and the scales of untouched blocks, stay."""
    rng = np.random.default_rng(8)
    B, H, S, D, block, T = 3, 2, 200, 128, 32, 70
    buf = torch.from_numpy(rng.integers(0, 256, size=B * H * S * D + 512, dtype=np.uint8)).cuda()
    codes = buf[256:-256].view(torch.float8_e4m3fn).view(B, H, S, D)
    before = buf.clone()
    sc = torch.ones(B, H, 7, device="cuda")
    vc, vs = codes.clone(), sc.clone()
    x = rows(rng, B, H, T, D).cuda()
    lens = [33, 131, -5]
    td.td_kv_append_f8(x, x, codes, sc, vc, vs, torch.tensor(lens, dtype=torch.int32, device="cuda"), block)
    torch.cuda.synchronize()
    changed = (buf != before).cpu().numpy()
    assert not changed[:256].any() and not changed[-256:].any()
    c = changed[256:-256].reshape(B, H, S, D)
    assert c[0, :, 33:103].any() and not c[0, :, :32].any() and not c[0, :, 103:].any()
    assert not c[1:].any()       # 131 + 70 > 200, and a negative length
    touched = sc.cpu().numpy() != 1
    assert not touched[1:].any() and not touched[0, :, 0].any() and not touched[0, :, 4:].any()


# --------------------------------------------------------------------- append with rotation

ROPE = [
    # dtype, D, block, T, lengths, axes
    ("bf16", 128, 64, 1, [0, 37, 64], 0),
    ("bf16", 64, 16, 1, [3, 100], 3),
    ("f32", 128, 32, 1, [3, 31], 2),
    ("bf16", 128, 64, 6, [60, 0], 0),
    ("bf16", 128, 32, 40, [0, 31], 0),
    ("bf16", 128, 64, 70, [1, 10], 3),
    ("bf16", 64, 128, 33, [120, 0], 16),
    ("f32", 64, 16, 50, [9, 0], 1),
    ("f32", 128, 128, 20, [127, 5], 3),
    ("bf16", 128, 16, 2, [5, 15], 0),
    ("bf16", 64, 64, 12, [(11 * i) % 200 for i in range(270)], 2),   # many heads: the first kernel's longest chunk
]


@pytest.mark.parametrize("dtype,D,block,T,lens,A", ROPE)
@pytest.mark.parametrize("inplace", [False, True])
def test_rope_append(td, dtype, D, block, T, lens, A, inplace):
    rng = np.random.default_rng(D + T + A)
    B, H, Hq, S, R = len(lens), 2, 6, 256, 300
    kc, ks = filled(rng, B, H, S, D, block, lens)
    vc, vs = filled(rng, B, H, S, D, block, lens)
    kn, vn, q = rows(rng, B, H, T, D, dtype=dtype), rows(rng, B, H, T, D, dtype=dtype), rows(rng, B, Hq, T, D, dtype=dtype)
    cos, sin = rope_tables(R, D)
    pos = axes = None
    at = np.asarray(lens)[:, None, None] + np.arange(T)[None, :, None] + np.zeros(D // 2, np.int64)
    if A:
        pos = torch.from_numpy(rng.integers(0, R, size=(B, T, A), dtype=np.int32))
        # runs of one axis, with a change inside a run of four pairs
        ax = np.sort(rng.integers(0, A, size=D // 2)) if A > 1 else np.zeros(D // 2, np.int64)
        axes = torch.from_numpy(ax.astype(np.int32)) if A > 1 else None
        at = pos.numpy()[:, :, ax]
    c, s = cos.double().numpy(), sin.double().numpy()
    i = np.arange(D // 2)
    c, s = c[at, i][:, None], s[at, i][:, None]               # [B, 1, T, D/2]
    d = [f8(kc), torch.from_numpy(ks).cuda(), f8(vc), torch.from_numpy(vs).cuda(),
         torch.tensor(lens, dtype=torch.int32, device="cuda")]
    qd, st = q.cuda(), status()
    got = td.td_rope_kv_append_f8(kn.cuda(), vn.cuda(), *d, block, cos.cuda(), sin.cuda(),
                                  positions=None if pos is None else pos.cuda(),
                                  axes=None if axes is None else axes.cuda(), q=qd, q_out=qd if inplace else None,
                                  dev_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0 and d[4].cpu().tolist() == [L + T for L in lens]
    assert inplace == (got is qd) and (inplace or torch.equal(qd.cpu(), q))
    # values: quantised as they are
    f8_ref.append(vc, vs, vn.double().numpy(), lens, block)
    assert np.array_equal(codes_of(d[2]), vc) and np.array_equal(d[3].cpu().numpy(), vs, equal_nan=True)
    # queries: fp32 rotation (two roundings of 2^-24 of the larger product), rounded once into dtype
    want = f8_ref.rotate(q.double().numpy(), c, s)
    pair = np.hypot(*np.split(q.double().numpy(), 2, axis=-1))
    u = torch.finfo(DT[dtype]).eps / 2
    tol = u * np.abs(want) * (1 + 2.0 ** -10) + (1 + u) * 2.0 ** -22 * np.concatenate([pair, pair], -1)
    assert np.all(np.abs(got.double().cpu().numpy() - want) <= tol)
    # keys: the fp32 formula's codes bit for bit, and so within its error and half a step of the exact
    # rotation
    exact = f8_ref.rotate(kn.double().numpy(), c, s)
    y = f8_ref.rotate_keys(kn.double().numpy(), c, s)
    kp = np.hypot(*np.split(kn.double().numpy(), 2, axis=-1))
    assert np.all(np.abs(y - exact) <= 2.0 ** -22 * np.concatenate([kp, kp], -1))
    f8_ref.append(kc, ks, y.astype(np.float64), lens, block)
    assert np.array_equal(d[1].cpu().numpy(), ks, equal_nan=True)
    assert np.array_equal(codes_of(d[0]), kc)


@pytest.mark.parametrize("T", [1, 20])
def test_rope_append_bad_positions(td, T):
    """Positions and axes out of range leave their pairs unrotated and raise the status bit; without q
    the call writes keys and values alone."""
    rng = np.random.default_rng(4)
    B, H, S, D, block, R = 2, 1, 64, 64, 16, 50
    kn = rows(rng, B, H, T, D)
    cos, sin = rope_tables(R, D)
    pos = torch.from_numpy(rng.integers(0, R, size=(B, T, 2), dtype=np.int32))
    pos[0, 0, 0], pos[1, 0, 1] = -1, R
    axes = torch.zeros(D // 2, dtype=torch.int32)
    axes[10:20], axes[20], axes[21] = 1, 2, -1
    ok = ((axes >= 0) & (axes < 2)).numpy()
    p = pos.numpy()[:, :, np.where(ok, axes.numpy(), 0)]
    good = ok & (p >= 0) & (p < R)
    i = np.arange(D // 2)
    pc = np.clip(p, 0, R - 1)
    c = np.where(good, cos.double().numpy()[pc, i], 1.0)[:, None]
    s = np.where(good, sin.double().numpy()[pc, i], 0.0)[:, None]
    kc, ks, vc, vs = td.make_f8_cache(B, H, S, D, block)
    st = status()
    out = td.td_rope_kv_append_f8(kn.cuda(), kn.cuda(), kc, ks, vc, vs, torch.zeros(B, dtype=torch.int32, device="cuda"),
                                  block, cos.cuda(), sin.cuda(), positions=pos.cuda(), axes=axes.cuda(), dev_status=st)
    torch.cuda.synchronize()
    assert out is None and int(st.item()) == td.DEV_BAD_POSITION
    rc, rs = np.zeros((B, H, S, D), np.uint8), np.zeros((B, H, S // block), np.float32)
    y = f8_ref.rotate_keys(kn.double().numpy(), c, s)
    f8_ref.append(rc, rs, y.astype(np.float64), [0] * B, block)
    assert np.array_equal(codes_of(kc), rc) and np.array_equal(ks.cpu().numpy(), rs)


LONG = [
    # dtype, D, block, T, lengths, Hq, Hkv, axes: chunks whose CTAs take their heads in several rounds
    ("bf16", 128, 32, 1531, [0, 5, 32, 100, 333, 640, 777], 32, 8, 3),   # 11 million keys; six rounds of four heads
    ("f32", 64, 64, 2000, [0, 1, 63, 64], 24, 8, 0),                     # five of two heads
    ("bf16", 64, 16, 3000, [7, 128], 24, 8, 0),                          # three of eight heads, a warp each
]


@pytest.mark.parametrize("dtype,D,block,T,lens,Hq,H,A", LONG)
def test_rope_append_long(td, dtype, D, block, T, lens, Hq, H, A):
    """Prompts: the keys' codes are the fp32 formula's bit for bit (an operation rounded otherwise moves
    about one code in a million), the values' codes theirs, the queries td_rope_kv_append's."""
    B, S = len(lens), 4096
    rng, g = np.random.default_rng(T), torch.Generator(device="cuda").manual_seed(T)

    def new(h):
        x = torch.randn(B, h, T, D, generator=g, device="cuda") * torch.randn(B, h, T, 1, generator=g, device="cuda").exp()
        return x.to(DT[dtype])

    kn, vn, q = new(H), new(H), new(Hq)
    kc, ks = filled(rng, B, H, S, D, block, lens)
    cos, sin = (t.cuda() for t in rope_tables(S, D))
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    d = [f8(kc), torch.from_numpy(ks).cuda(), f8(kc), torch.from_numpy(ks).cuda(), ln]
    at = ln.long()[:, None, None] + torch.arange(T, device="cuda")[None, :, None] + torch.zeros(D // 2, dtype=torch.long, device="cuda")
    pos = axes = None
    if A:
        pos = torch.randint(0, S, (B, T, A), generator=g, device="cuda", dtype=torch.int32)
        axes = (torch.arange(D // 2, device="cuda") * A // (D // 2)).to(torch.int32)
        at = pos.long()[:, :, axes.long()]
    c, s = torch.gather(cos[None].expand(B, -1, -1), 1, at)[:, None], torch.gather(sin[None].expand(B, -1, -1), 1, at)[:, None]
    got = td.td_rope_kv_append_f8(kn, vn, *d, block, cos, sin, positions=pos, axes=axes, q=q, advance=False)
    torch.cuda.synchronize()
    y = f8_ref.rotate_keys(kn.double().cpu().numpy(), c.cpu().numpy(), s.cpu().numpy())
    for x, codes, scales in ((vn.double().cpu().numpy(), d[2], d[3]), (y.astype(np.float64), d[0], d[1])):
        wc, ws = kc.copy(), ks.copy()
        f8_ref.append(wc, ws, x, lens, block)
        assert np.array_equal(scales.cpu().numpy(), ws, equal_nan=True)
        moved = int((codes_of(codes) != wc).sum())
        assert moved == 0
    # queries: two roundings of 2^-24 of the larger product, then one into dtype
    lo, hi = q.double().split(D // 2, dim=-1)
    want, pair = torch.cat([lo * c - hi * s, hi * c + lo * s], -1), torch.hypot(lo, hi)
    u = torch.finfo(DT[dtype]).eps / 2
    tol = u * want.abs() * (1 + 2.0 ** -10) + (1 + u) * 2.0 ** -22 * torch.cat([pair, pair], -1)
    assert bool(((got.double() - want).abs() <= tol).all())
    if not A:
        cache = [torch.empty(B, H, S, D, dtype=DT[dtype], device="cuda") for _ in range(2)]
        assert torch.equal(got, td.td_rope_kv_append(kn, vn, *cache, ln, cos, sin, q=q, advance=False))


# ------------------------------------------------------------------------------ read-back

READ = [
    # dtype, D, block, Smax, rows, lengths, starts
    ("bf16", 128, 64, 300, 300, [300, 0, 1, 299], None),
    ("bf16", 64, 16, 100, 37, [100, 50, 3], [0, 20, 2]),
    ("f32", 128, 32, 200, 65, [200, 64], [150, 63]),
    ("f32", 64, 128, 256, 256, [130, 256], [0, -10]),
    ("bf16", 128, 16, 70, 1, [70, 12], [69, 12]),
    ("bf16", 128, 16, 70, 200, [90, -3], [1, 0]),          # a length past Smax, a negative one
]


@pytest.mark.parametrize("dtype,D,block,S,N,lens,starts", READ)
def test_read_bit_exact(td, dtype, D, block, S, N, lens, starts):
    rng = np.random.default_rng(N)
    B, H = len(lens), 3
    kc, ks = filled(rng, B, H, S, D, block, lens)
    vc, vs = filled(rng, B, H, S, D, block, lens)
    vs *= np.float32(0.3)                              # scales need not be powers of two
    st = status()
    outs = [torch.full((B, H, N, D), 7.0, dtype=DT[dtype], device="cuda") for _ in range(2)]
    start = None if starts is None else torch.tensor(starts, dtype=torch.int32, device="cuda")
    td.td_kv_read_f8(f8(kc), torch.from_numpy(ks).cuda(), f8(vc), torch.from_numpy(vs).cuda(),
                     torch.tensor(lens, dtype=torch.int32, device="cuda"), block, start=start, k_out=outs[0],
                     v_out=outs[1], dev_status=st)
    torch.cuda.synchronize()
    for out, codes, scales in ((outs[0], kc, ks), (outs[1], vc, vs)):
        v = f8_ref.VALUE[codes].astype(np.float32) * np.repeat(scales, block, axis=2)[:, :, :S, None]
        want = torch.full((B, H, N, D), 7.0, dtype=DT[dtype])
        for b, L in enumerate(lens):
            L, a = min(max(L, 0), S), 0 if starts is None else starts[b]
            t0, t1 = max(0, -a), min(N, L - a)
            if t1 > t0:
                want[b, :, t0:t1] = torch.from_numpy(v[b, :, a + t0:a + t1]).to(DT[dtype])
        assert torch.equal(out.cpu(), want)
    bits = (td.DEV_SEQLEN_CLAMPED if max(lens) > S else 0) | (td.DEV_NEGATIVE_SEQLEN if min(lens) < 0 else 0)
    assert int(st.item()) == bits


def test_read_makes_zeroed_outputs(td):
    rng = np.random.default_rng(1)
    kc, ks = filled(rng, 1, 2, 64, 64, 16)
    lens = torch.tensor([20], dtype=torch.int32, device="cuda")
    args = (f8(kc), torch.from_numpy(ks).cuda(), f8(kc), torch.from_numpy(ks).cuda(), lens, 16)
    k, v = td.td_kv_read_f8(*args, rows=30, dtype=torch.float32)
    assert k.shape == (1, 2, 30, 64) and k.dtype == torch.float32 and torch.equal(k, v)
    assert not k[:, :, 20:].any() and k[:, :, :20].any()
    assert td.td_kv_read_f8(*args)[0].shape == (1, 2, 64, 64)
    with pytest.raises(ValueError):
        td.td_kv_read_f8(*args, rows=5, k_out=k, v_out=v)


# ------------------------------------------------------------------------------ attention

def attend(td, q, cache, lens, block, scale, split=0, **kw):
    st = status()
    q = q.cuda()
    d = [f8(cache[0]), torch.from_numpy(cache[1]).cuda(), f8(cache[2]), torch.from_numpy(cache[3]).cuda(),
         torch.tensor(lens, dtype=torch.int32, device="cuda")]
    if q.shape[2] == 1:
        out, lse = td.td_decode_attn_f8(q[:, :, 0].contiguous(), *d, block, scale, split, return_lse=True, dev_status=st, **kw)
        out, lse = out[:, :, None], lse[:, :, None]
    else:
        out, lse = td.td_verify_attn_f8(q, *d, block, scale, split, return_lse=True, dev_status=st, **kw)
    torch.cuda.synchronize()
    return out.double().cpu().numpy(), lse.double().cpu().numpy(), int(st.item())


def check(td, q, cache, lens, block, scale, split=0):
    """Against the exact attention over the values the codes stand for (those before the lengths)."""
    kc, ks, vc, vs = cache
    S, D = kc.shape[2:]
    k, v = f8_ref.values(kc, ks, block), f8_ref.values(vc, vs, block)
    for b, L in enumerate(lens):
        k[b, :, min(max(L, 0), S):] = 0
        v[b, :, min(max(L, 0), S):] = 0
    out, lse, st = attend(td, q, cache, lens, block, scale, split)
    ref, rlse, rst, absv, big = f8_ref.attention(q.double().numpy(), k, v, lens, scale)
    assert st == rst
    tol, ltol = f8_ref.bounds(ref, rlse, absv, big, D, max(max(lens), 1))
    assert np.all(np.abs(out - ref) <= tol), float((np.abs(out - ref) / tol).max())
    none = np.isneginf(rlse)
    assert np.array_equal(np.isneginf(lse), none) and np.all(np.abs(lse[~none] - rlse[~none]) <= ltol[~none])


ATTN = [
    # D, Hq, Hkv, Smax, T, block, lengths, split
    (128, 24, 8, 520, 1, 64, [520, 100], 0),
    (128, 24, 8, 520, 1, 16, [519, 16], 64),
    (64, 15, 5, 300, 1, 32, [300, 64, 1], 0),
    (64, 15, 5, 300, 1, 128, [299, 0, 17], 16),
    (128, 32, 4, 260, 1, 16, [260, 5], 0),           # 8 rows: one n tile
    (128, 36, 4, 260, 1, 64, [260, 33], 0),          # 9 rows: two n tiles
    (64, 34, 2, 400, 1, 32, [400, 31], 48),          # 17 rows: three
    (64, 25, 1, 300, 1, 32, [300, 3], 0),            # 25 rows: two row blocks
    (128, 32, 8, 200, 6, 64, [200, 70], 0),          # verify, 24 rows
    (128, 32, 8, 300, 6, 16, [4, 6, 300, 0], 0),     # shorter than the chunk; empty
    (64, 8, 1, 400, 1, 16, [400, 399, 31, 2], 32),
    (128, 24, 8, 4096, 1, 128, [4096, 1500, 0], 0),
    (128, 4, 2, 300, 4, 32, [300, 70], 0),
    (64, 6, 2, 77, 11, 16, [77, 40], 0),             # 33 rows over two blocks that wrap tokens
    (128, 8, 1, 1000, 12, 64, [1000, 333], 0),       # 96 rows over four blocks
    (64, 3, 3, 2048, 3, 64, [2048, 1], 112),
    (128, 2, 2, 1, 1, 16, [1, 0], 0),                # a cache of one row
    (128, 24, 8, 600, 1, 64, [(37 * i) % 601 for i in range(40)], 0),
    # ragged: equal runs of stages that cross from group to group, several groups in one run
    (128, 16, 8, 2048, 1, 64, [2048, 130, 128, 0, 1, 1999, 640] + [(331 * i) % 1500 for i in range(33)], 0),
    (64, 24, 8, 2000, 3, 16, [2000, 127, 1025] + [(97 * i) % 700 for i in range(30)], 0),    # 9 rows
    (128, 32, 8, 3000, 6, 32, [3000, 5, 300, 2500, 77, 1000, 129, 0], 0),                    # 24 rows, a batch of 8
    (64, 2, 2, 3000, 1, 128, [3000] + [5] * 100, 0),
    # whole groups, a CTA each: a short sequence up to the longest that is left whole, and one past it
    (128, 24, 8, 640, 1, 64, [640], 0),
    (128, 24, 8, 641, 1, 64, [641], 0),
    (64, 15, 5, 512, 1, 32, [1], 0),
    (128, 32, 8, 520, 1, 16, [0] + [391 + i * 17 % 130 for i in range(31)], 0),
    (64, 15, 5, 512, 1, 128, [(i % 7 > 0) * (300 + i * 37 % 213) for i in range(64)], 0),    # over two rounds
    (128, 8, 8, 4000, 1, 64, [4000 - 64 * i for i in range(20)], 0),
    (64, 6, 2, 300, 2, 16, [300, 0, 1, 2], 0),
]


@pytest.mark.parametrize("T", [1, 6])
def test_captured_attention(td, T):
    """Captured alone, with its merge, and replayed on changed queries."""
    rng = np.random.default_rng(20 + T)
    lens, block = [1500, 40], 64
    kc, ks = filled(rng, 2, 2, 1500, 128, block, lens)
    d = [f8(kc), torch.from_numpy(ks).cuda(), f8(kc), torch.from_numpy(ks).cuda(),
         torch.tensor(lens, dtype=torch.int32, device="cuda")]
    q = rows(rng, 2, 8, T, 128).cuda()
    out, ws = torch.empty_like(q), td.make_workspace(2, 8, 2, 1500, 128, T)
    td.td_verify_attn_f8(q, *d, block, out=out, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        td.td_verify_attn_f8(q, *d, block, out=out, workspace=ws)
    for _ in range(3):
        q.copy_(rows(rng, 2, 8, T, 128))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, td.td_verify_attn_f8(q, *d, block))


@pytest.mark.parametrize("B", [1, 9])
def test_captured_attention_on_changed_lengths(td, B):
    """Short groups left whole and long ones cut, by one captured call: the lengths are read when it runs."""
    rng = np.random.default_rng(30 + B)
    Hq, Hkv, S, D, block = 15, 5, 1800, 64, 32
    kc, ks = filled(rng, B, Hkv, S, D, block)
    lens = torch.full((B,), 100, dtype=torch.int32, device="cuda")
    d = [f8(kc), torch.from_numpy(ks).cuda(), f8(kc), torch.from_numpy(ks).cuda(), lens]
    q = rows(rng, B, Hq, 1, D, spread=0.3)
    qd, ws = q[:, :, 0].contiguous().cuda(), td.make_workspace(B, Hq, Hkv, S, D, 1)
    out = torch.empty_like(qd)
    td.td_decode_attn_f8(qd, *d, block, out=out, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        td.td_decode_attn_f8(qd, *d, block, out=out, workspace=ws)
    v = f8_ref.values(kc, ks, block)
    for L in (1800, 100, 640, 0, 641, 1024, 1):
        now = [max(L - 130 * b, 0) for b in range(B)]
        lens.copy_(torch.tensor(now, dtype=torch.int32))
        out.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        ref, rlse, _, absv, big = f8_ref.attention(q.double().numpy(), v, v, now, 1 / math.sqrt(D))
        tol, _ = f8_ref.bounds(ref, rlse, absv, big, D, max(max(now), 1))
        assert np.all(np.abs(out[:, :, None].double().cpu().numpy() - ref) <= tol), L


@pytest.mark.parametrize("D,Hq,Hkv,S,T,block,lens,split", ATTN)
def test_attention_against_oracle(td, D, Hq, Hkv, S, T, block, lens, split):
    rng = np.random.default_rng(D + S + T)
    B = len(lens)
    kc, ks = filled(rng, B, Hkv, S, D, block, lens)      # random bytes, NaN codes among them, behind the lengths
    vc, vs = filled(rng, B, Hkv, S, D, block, lens)
    q = rows(rng, B, Hq, T, D, spread=0.3)
    check(td, q, (kc, ks, vc, vs), lens, block, 1 / math.sqrt(D), split)


@pytest.mark.parametrize("T", [1, 5])
@pytest.mark.parametrize("what", ["big q", "small q", "big v", "small v", "mixed v", "zero blocks", "odd scales", "negative scale"])
def test_attention_magnitudes(td, T, what):
    """Query rows and scales far from 1, values whose blocks differ by large factors, blocks of zeros."""
    rng = np.random.default_rng(len(what) + T)
    B, Hq, Hkv, S, D, block = 2, 8, 2, 500, 128, 32
    lens = [500, 130]
    kc, ks = filled(rng, B, Hkv, S, D, block, lens)
    vc, vs = filled(rng, B, Hkv, S, D, block, lens)
    q = rows(rng, B, Hq, T, D, spread=0.3)
    scale = 1 / math.sqrt(D)
    if what == "big q":
        q, scale = q * 2.0 ** 40, scale * 2.0 ** -40
    elif what == "small q":
        q, scale = q * 2.0 ** -60, scale * 2.0 ** 60
    elif what == "big v":
        vs *= np.float32(2.0 ** 40)
    elif what == "small v":
        vs *= np.float32(2.0 ** -40)
    elif what == "mixed v":
        vs *= (2.0 ** rng.integers(-12, 12, size=vs.shape)).astype(np.float32)
    elif what == "zero blocks":
        for c, s in ((kc, ks), (vc, vs)):
            c[:, :, 64:128] = 0
            s[:, :, 2:4] = 2.0 ** -126
    elif what == "odd scales":
        ks *= np.float32(0.7)
        vs *= np.float32(1.3)
    else:
        scale = -scale
    check(td, q, (kc, ks, vc, vs), lens, block, scale)


@pytest.mark.parametrize("T", [1, 5])
def test_attention_largest_values(td, T):
    """Values up to 2^116, whose sums over 500 keys are inside fp32 (2^125), and one key of the largest
    value a cache holds of finite rows, 448 * 2^119: the output itself."""
    rng = np.random.default_rng(T)
    B, Hq, Hkv, S, D, block, lens = 2, 8, 2, 500, 128, 32, [500, 130]
    kc, ks = filled(rng, B, Hkv, S, D, block, lens)
    vc, vs = filled(rng, B, Hkv, S, D, block, lens)
    vs *= np.float32(2.0 ** 116 / np.nanmax(448 * vs))
    check(td, rows(rng, B, Hq, T, D, spread=0.3), (kc, ks, vc, vs), lens, block, 1 / math.sqrt(D))
    vc[:], vs[:] = 0x7e, 2.0 ** 119
    out, _, _ = attend(td, rows(rng, B, Hq, T, D), (kc, ks, vc, vs), [T, 1], block, 0.1)
    assert np.all(out[0, :, 0] == 448 * 2.0 ** 119) and np.all(out[1, :, T - 1] == 448 * 2.0 ** 119)


@pytest.mark.parametrize("T,Hq,split", [(1, 8, 0), (1, 8, 64), (6, 8, 0), (6, 8, 64), (3, 2, 0)])
def test_attention_nan_values_reach_only_the_rows_that_see_them(td, T, Hq, split):
    """A NaN value code gives NaN in its element for the rows that see it, and nothing else."""
    rng = np.random.default_rng(T)
    B, Hkv, S, D, block = 1, 2, 256, 128, 16
    L = 200
    kc, ks = filled(rng, B, Hkv, S, D, block, [L])
    vc, vs = filled(rng, B, Hkv, S, D, block, [L])
    vc[0, 1, L - 1, 7] = 0x7f          # seen by the last token alone
    if T > 2:
        vc[0, 1, L - 2, 64] = 0xff     # by the last two
    q = rows(rng, B, Hq, T, D)
    out, lse, _ = attend(td, q, (kc, ks, vc, vs), [L], block, 0.1, split)
    clean = vc.copy()
    clean[(clean & 0x7f) == 0x7f] = 0
    want, wlse, _ = attend(td, q, (kc, ks, clean, vs), [L], block, 0.1, split)
    G = Hq // Hkv
    nan = np.zeros(out.shape, bool)
    nan[0, G:, T - 1, 7] = True
    if T > 2:
        nan[0, G:, T - 2:, 64] = True
    assert np.array_equal(np.isnan(out), nan) and np.array_equal(out[~nan], want[~nan])
    assert np.array_equal(lse, wlse)


@pytest.mark.parametrize("T,split", [(1, 0), (1, 32), (4, 0), (4, 32)])
def test_attention_nan_keys(td, T, split):
    """A NaN key makes the rows that see it NaN (lse +inf) however the keys are split."""
    rng = np.random.default_rng(T)
    B, Hq, Hkv, S, D, block, L = 1, 8, 2, 300, 64, 32, 290
    kc, ks = filled(rng, B, Hkv, S, D, block, [L])
    vc, vs = filled(rng, B, Hkv, S, D, block, [L])
    kc[0, 0, L - 1, 3] = 0x7f
    kc[0, 1, 40, 3] = 0xff
    q = rows(rng, B, Hq, T, D)
    out, lse, _ = attend(td, q, (kc, ks, vc, vs), [L], block, 0.1, split)
    assert np.isnan(out[0, 4:]).all() and np.isposinf(lse[0, 4:]).all()
    assert np.isnan(out[0, :4, T - 1]).all() and np.isposinf(lse[0, :4, T - 1]).all()
    assert np.isfinite(out[0, :4, :T - 1]).all() and np.isfinite(lse[0, :4, :T - 1]).all()


@pytest.mark.parametrize("T,split", [(1, 0), (1, 96), (5, 0)])
def test_attention_stale_bytes_are_never_used(td, T, split):
    rng = np.random.default_rng(9)
    lens, block = [700, 333], 64
    kc, ks = filled(rng, 2, 8, 1024, 128, block, lens)
    vc, vs = filled(rng, 2, 8, 1024, 128, block, lens)
    q = rows(rng, 2, 24, T, 128)
    ref = attend(td, q, (kc, ks, vc, vs), lens, block, 0.09, split)
    for b, L in enumerate(lens):
        kc[b, :, L:], vc[b, :, L:] = 0x7f, 0xff
        ks[b, :, -(-L // block):], vs[b, :, -(-L // block):] = np.inf, -np.inf
    got = attend(td, q, (kc, ks, vc, vs), lens, block, 0.09, split)
    assert all(np.array_equal(a, b) for a, b in zip(got, ref))


def test_attention_statuses(td):
    rng = np.random.default_rng(3)
    kc, ks = filled(rng, 3, 2, 64, 64, 16)
    q = rows(rng, 3, 4, 2, 64)
    out, lse, st = attend(td, q, (kc, ks, kc, ks), [70, -2, 1], 16, 0.1)
    assert st == td.DEV_SEQLEN_CLAMPED | td.DEV_NEGATIVE_SEQLEN | td.DEV_VERIFY_SHORT
    assert not out[1].any() and np.isneginf(lse[1]).all() and np.isneginf(lse[2, :, 0]).all()


def test_attention_long_cache_offsets(td):
    """Offsets past 2^32 bytes: the last kv head of a cache of 5.4 GB, 1M keys."""
    Hkv, S, D, block = 40, 1 << 20, 128, 128
    g = torch.Generator(device="cuda").manual_seed(1)
    kc = torch.zeros(1, Hkv, S, D, dtype=torch.uint8, device="cuda")
    kc[0, -1] = torch.randint(0, 0x48, (S, D), generator=g, device="cuda", dtype=torch.uint8)
    ks = torch.full((1, Hkv, S // block), 0.25, device="cuda")
    vc = kc.flip(3).contiguous()
    f = [t.view(torch.float8_e4m3fn) for t in (kc, vc)]
    lens = torch.tensor([S - 2], dtype=torch.int32, device="cuda")
    new = torch.full((1, Hkv, 1, D), 3.0, dtype=torch.bfloat16, device="cuda")
    td.td_kv_append_f8(new, new, f[0], ks, f[1], ks.clone(), lens, block)
    q = torch.randn(1, Hkv, D, generator=g, device="cuda").to(torch.bfloat16)
    out, lse = td.td_decode_attn_f8(q, f[0], ks, f[1], ks, lens, block, scale=0.05, return_lse=True)
    k = f[0][0, -1, :S - 1].double() * 0.25
    v = f[1][0, -1, :S - 1].double() * 0.25
    assert torch.equal(k[-1], torch.full((D,), 3.0, dtype=torch.float64, device="cuda"))
    x = k @ q[0, -1].double() * 0.05
    want, wl = torch.softmax(x, 0) @ v, torch.logsumexp(x, 0)
    # 2^-8 output, 2^-11 probabilities, scores off by at most (D + 4) 2^-23 of their terms' magnitudes
    e = (D + 4) * 2.0 ** -23 * float((k.abs() @ q[0, -1].double().abs()).max()) * 0.05
    tol = 2.0 ** -8 * want.abs() + (math.expm1(2 * e) + 2.0 ** -11 + 2.0 ** -12) * (torch.softmax(x, 0) @ v.abs())
    assert bool(((out[0, -1].double() - want).abs() <= tol).all())
    assert abs(float(lse[0, -1]) - float(wl)) <= e + 2.0 ** -12 * (1 + abs(float(wl)))
    r, _ = td.td_kv_read_f8(f[0], ks, f[1], ks, lens, block, rows=3, start=lens - 3)
    assert torch.equal(r[0, -1].double(), k[-3:])


# -------------------------------------------------------------------------- used together

def test_generation_run(td):
    """A prompt appended in two chunks and prefilled over its read-back, then tokens decoded and a
    chunk verified, each against the exact attention over what the cache holds."""
    rng = np.random.default_rng(0)
    B, Hq, Hkv, S, D, block = 2, 8, 2, 400, 128, 32
    cache = td.make_f8_cache(B, Hkv, S, D, block)
    lens = torch.tensor([0, 3], dtype=torch.int32, device="cuda")
    first = rows(rng, B, Hkv, 3, D).cuda()
    td.td_kv_append_f8(first, first, *cache, torch.zeros(B, dtype=torch.int32, device="cuda"), block)
    cos, sin = (t.cuda() for t in rope_tables(S, D))
    scale = 1 / math.sqrt(D)

    def values():
        return [f8_ref.values(codes_of(cache[i]), np.nan_to_num(cache[i + 1].cpu().numpy()), block) for i in (0, 2)]

    for T in (150, 45):
        q, k, v = (rows(rng, B, h, T, D).cuda() for h in (Hq, Hkv, Hkv))
        qr = td.td_rope_kv_append_f8(k, v, *cache, lens, block, cos, sin, q=q)
        ko, vo = td.td_kv_read_f8(*cache, lens, block)
        out = td.td_prefill_attn(qr, ko, vo, lens, scale).double().cpu().numpy()
        kv = values()
        # the read-back rounds code * scale to bf16 exactly: 4 significant bits
        n = lens.cpu().tolist()
        for b in range(B):
            assert np.array_equal(ko[b, :, :n[b]].double().cpu().numpy(), kv[0][b, :, :n[b]])
        ref, _, _, absv, _ = f8_ref.attention(qr.double().cpu().numpy(), *kv, n, scale)
        # bf16 probabilities and output, as the prefill's own tests allow at most
        assert np.all(np.abs(out - ref) <= 2e-2 + 1e-2 * np.abs(ref))
    for T in (1, 1, 5, 1):
        q, k, v = (rows(rng, B, h, T, D).cuda() for h in (Hq, Hkv, Hkv))
        qr = td.td_rope_kv_append_f8(k, v, *cache, lens, block, cos, sin, q=q)
        if T == 1:
            out, lse = td.td_decode_attn_f8(qr[:, :, 0].contiguous(), *cache, lens, block, return_lse=True)
        else:
            out, lse = td.td_verify_attn_f8(qr, *cache, lens, block, return_lse=True)
        n = lens.cpu().tolist()
        ref, rl, _, absv, big = f8_ref.attention(qr.double().cpu().numpy(), *values(), n, scale)
        tol, ltol = f8_ref.bounds(ref, rl, absv, big, D, max(n))
        assert np.all(np.abs(out.double().cpu().numpy().reshape(ref.shape) - ref) <= tol)
        assert np.all(np.abs(lse.double().cpu().numpy().reshape(rl.shape) - rl) <= ltol)
    assert lens.cpu().tolist() == [203, 206]


def test_captured_step_replays(td):
    """An append and a decode captured in a graph, replayed as the lengths advance on the device."""
    rng = np.random.default_rng(5)
    B, Hq, Hkv, S, D, block = 3, 8, 2, 300, 64, 16
    kc, ks = filled(rng, B, Hkv, S, D, block)
    q, k, v = (rows(rng, B, h, 1, D).cuda() for h in (Hq, Hkv, Hkv))

    def state():
        return [f8(kc), torch.from_numpy(ks).cuda(), f8(kc), torch.from_numpy(ks).cuda(),
                torch.tensor([0, 14, 200], dtype=torch.int32, device="cuda")]

    def step(s, out, ws):
        td.td_kv_append_f8(k, v, *s, block)
        td.td_decode_attn_f8(q[:, :, 0].contiguous(), *s, block, out=out, workspace=ws)

    ws = td.make_workspace(B, Hq, Hkv, S, D)
    a, b = state(), state()
    oa, ob = torch.empty(B, Hq, D, dtype=torch.bfloat16, device="cuda"), torch.empty(B, Hq, D, dtype=torch.bfloat16, device="cuda")
    step(state(), oa, ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(a, oa, ws)
    for _ in range(5):
        g.replay()
        step(b, ob, None)
        torch.cuda.synchronize()
        assert torch.equal(oa, ob) and torch.equal(a[4], b[4]) and torch.equal(a[0].view(torch.uint8), b[0].view(torch.uint8))


def test_capture_wants_a_workspace(td):
    cache = td.make_f8_cache(1, 2, 64, 64, 16)
    lens = torch.full((1,), 9, dtype=torch.int32, device="cuda")
    q = torch.zeros(1, 4, 64, dtype=torch.bfloat16, device="cuda")
    td.td_decode_attn_f8(q, *cache, lens, 16)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    out = torch.empty_like(q)
    ws = td.make_workspace(1, 4, 2, 64, 64)
    with torch.cuda.graph(g):
        with pytest.raises(ValueError):
            td.td_decode_attn_f8(q, *cache, lens, 16, out=out)
        td.td_decode_attn_f8(q, *cache, lens, 16, out=out, workspace=ws)
    g.replay()
    torch.cuda.synchronize()


def test_two_streams(td):
    """Calls of one shape on two streams at once, each with the workspace kept for its stream."""
    rng = np.random.default_rng(6)
    lens, block = [900, 1024], 64
    kc, ks = filled(rng, 2, 4, 1024, 128, block, lens)
    vc, vs = filled(rng, 2, 4, 1024, 128, block, lens)
    d = [f8(kc), torch.from_numpy(ks).cuda(), f8(vc), torch.from_numpy(vs).cuda(),
         torch.tensor(lens, dtype=torch.int32, device="cuda")]
    q = rows(rng, 2, 16, 1, 128)[:, :, 0].contiguous().cuda()
    want = td.td_decode_attn_f8(q, *d, block)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[] for _ in streams]
    for _ in range(20):
        for s, o in zip(streams, outs):
            o.append(td.td_decode_attn_f8(q, *d, block, stream=s))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for got in outs for o in got)


def test_two_streams_many_rows(td):
    """Verify chunks of 24 rows that fill the GPU, on two streams at once: neither waits for the other."""
    rng = np.random.default_rng(16)
    lens, block = [2048, 1500, 2047], 32
    kc, ks = filled(rng, 3, 4, 2048, 64, block, lens)
    d = [f8(kc), torch.from_numpy(ks).cuda(), f8(kc), torch.from_numpy(ks).cuda(),
         torch.tensor(lens, dtype=torch.int32, device="cuda")]
    q = rows(rng, 3, 16, 6, 64).cuda()
    st = status()
    want, wl = td.td_verify_attn_f8(q, *d, block, return_lse=True)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for _ in range(30):
        for s in streams:
            outs.append(td.td_verify_attn_f8(q, *d, block, stream=s, return_lse=True, dev_status=st))
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    assert all(torch.equal(o, want) and torch.equal(l, wl) for o, l in outs)


def test_streams_are_taken_as_torch_streams_or_handles(td):
    rng = np.random.default_rng(17)
    s = torch.cuda.Stream()
    x = rows(rng, 2, 2, 20, 64).cuda()
    torch.cuda.synchronize()
    got = []
    for stream in (None, s, s.cuda_stream, 0, torch.cuda.default_stream()):
        cache = td.make_f8_cache(2, 2, 64, 64, 16)
        lens = torch.zeros(2, dtype=torch.int32, device="cuda")
        torch.cuda.synchronize()
        td.td_kv_append_f8(x, x, *cache, lens, 16, stream=stream)
        k, v = td.td_kv_read_f8(*cache, lens, 16, stream=stream)
        out = td.td_decode_attn_f8(x[:, :, 0].contiguous(), *cache, lens, 16, stream=stream)
        torch.cuda.synchronize()
        got.append((lens, k, v, out))
    assert got[0][0].tolist() == [20, 20]
    for g in got[1:]:
        assert all(torch.equal(a, b) for a, b in zip(g, got[0]))
    with pytest.raises((TypeError, ValueError)):
        td.td_kv_append_f8(x, x, *cache, lens, 16, stream="x")


def test_one_workspace_for_calls_of_one_shape(td):
    """A workspace serves one shape's calls in turn, decode kinds mixed: each leaves it as it found it."""
    rng = np.random.default_rng(18)
    B, Hq, Hkv, S, D, block = 3, 32, 4, 900, 128, 16
    lens = [900, 250, 0]
    kc, ks = filled(rng, B, Hkv, S, D, block, lens)
    for T in (1, 3):
        ws = td.make_workspace(B, Hq, Hkv, S, D, T)
        q = rows(rng, B, Hq, T, D).cuda()
        d = [f8(kc), torch.from_numpy(ks).cuda(), f8(kc), torch.from_numpy(ks).cuda()]
        bf = torch.from_numpy(rng.normal(size=(B, Hkv, S, D))).to(torch.bfloat16).cuda()
        n = torch.tensor(lens, dtype=torch.int32, device="cuda")
        first = None
        for _ in range(3):
            a = td.td_verify_attn_f8(q, *d, n, block, workspace=ws)
            b = td.td_verify_attn(q, bf, bf, n, workspace=ws, split=0)
            first = first or (a, b)
            assert torch.equal(a, first[0]) and torch.equal(b, first[1])


@pytest.mark.parametrize("D,Hq,Hkv,S,T,block,lens,split", ATTN)
def test_attention_stays_inside_its_workspace(td, D, Hq, Hkv, S, T, block, lens, split):
    """A workspace of exactly the bytes asked for gives the same bits, and nothing behind it is written."""
    rng = np.random.default_rng(D + S + T)
    B = len(lens)
    kc, ks = filled(rng, B, Hkv, S, D, block, lens)
    q = rows(rng, B, Hq, T, D, spread=0.3)
    want = attend(td, q, (kc, ks, kc, ks), lens, block, 0.1, split)
    n = td.td_f8_workspace_bytes(B, Hq, Hkv, S, D, T, split)
    buf = torch.zeros(n + 65536, dtype=torch.uint8, device="cuda")
    buf[n:] = 0xa5
    for _ in range(2):
        got = attend(td, q, (kc, ks, kc, ks), lens, block, 0.1, split, workspace=buf[:n])
        assert all(np.array_equal(a, b) for a, b in zip(got, want))
    assert bool((buf[n:] == 0xa5).all())
    assert n <= td.td_decode_workspace_bytes(B, Hq, Hkv, S, D, T, split)


def _memory_of_call(td, B, splits):
    Hkv, S, D, block, T = 8, 4864, 128, 128, 6
    cache = td.make_f8_cache(B, Hkv, S, D, block)
    lens = torch.full((B,), 700, dtype=torch.int32, device="cuda")
    q = torch.zeros(B, 4 * Hkv, T, D, dtype=torch.bfloat16, device="cuda")
    out = torch.empty_like(q)
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    for split in splits:
        td.td_verify_attn_f8(q, *cache, lens, block, split=split, out=out)
    torch.cuda.synchronize()
    return torch.cuda.memory_allocated() - before


def test_workspaces_are_small(td):
    """What a call keeps does not grow with the batch: 608 blocks of 24 rows (7.7 MB) and 16 bytes a group."""
    assert td.td_f8_workspace_bytes(64, 32, 8, 32768, 128, 6) < 9 << 20
    assert td.td_f8_workspace_bytes(1024, 8, 1, 32768, 128, 3) < 9 << 20
    assert _memory_of_call(td, 64, [0]) < 9 << 20


def test_kept_workspaces_are_bounded(td):
    """Splits of the caller's that ask for 247, 123, 84 and 62 MB: 256 MB of them are kept at most."""
    assert _memory_of_call(td, 8, [16, 32, 48, 64]) <= 256 << 20


def test_largest_batch(td):
    rng = np.random.default_rng(19)
    B, Hkv, S, D, block = 1024, 1, 40, 64, 16
    lens = [(7 * i) % 41 for i in range(B)]
    kc, ks = filled(rng, B, Hkv, S, D, block, lens)
    check(td, rows(rng, B, 3, 1, D, spread=0.3), (kc, ks, kc, ks), lens, block, 0.125)


def test_misaligned_pointers_are_refused(td):
    from decode_attention_split_gb300._lib import TDError
    kc, ks, vc, vs = td.make_f8_cache(1, 2, 64, 64, 16)
    lens = torch.zeros(1, dtype=torch.int32, device="cuda")
    buf = torch.zeros(2 * 64 + 4, device="cuda")
    x = buf[1:-3].view(1, 2, 1, 64)
    y = buf[:-4].view(1, 2, 1, 64)
    raw = torch.zeros(2 * 64 * 64 + 16, dtype=torch.uint8, device="cuda")
    odd = raw[8:-8].view(torch.float8_e4m3fn).view(1, 2, 64, 64)
    for call in (lambda: td.td_kv_append_f8(x, y, kc, ks, vc, vs, lens, 16),
                 lambda: td.td_kv_append_f8(y, y, odd, ks, vc, vs, lens, 16),
                 lambda: td.td_kv_read_f8(kc, ks, odd, vs, lens, 16),
                 lambda: td.td_decode_attn_f8(torch.zeros(1, 4, 64, dtype=torch.bfloat16, device="cuda"), kc, ks, odd, vs, lens, 16)):
        with pytest.raises(TDError) as e:
            call()
        assert e.value.status == 2


def test_repeat_calls_are_equal(td):
    rng = np.random.default_rng(10)
    lens = [5000, 17, 2600, 4096]
    kc, ks = filled(rng, 4, 2, 5000, 128, 64, lens)
    q = rows(rng, 4, 24, 2, 128)
    a = attend(td, q, (kc, ks, kc, ks), lens, 64, 0.09)
    for _ in range(5):
        b = attend(td, q, (kc, ks, kc, ks), lens, 64, 0.09)
        assert all(np.array_equal(x, y) for x, y in zip(a, b))


def test_binding_refuses(td):
    cache = td.make_f8_cache(2, 2, 64, 128, 16)
    lens = torch.zeros(2, dtype=torch.int32, device="cuda")
    x = torch.zeros(2, 2, 1, 128, device="cuda")
    q = torch.zeros(2, 4, 128, dtype=torch.bfloat16, device="cuda")
    bad = [
        lambda: td.td_kv_append_f8(x, x.bfloat16(), *cache, lens, 16),
        lambda: td.td_kv_append_f8(x[:, :1], x[:, :1], *cache, lens, 16),
        lambda: td.td_kv_append_f8(x.half(), x.half(), *cache, lens, 16),
        lambda: td.td_kv_append_f8(x.transpose(1, 2), x, *cache, lens, 16),
        lambda: td.td_kv_append_f8(x, x, *cache, lens.cpu(), 16),
        lambda: td.td_kv_append_f8(x, x, *cache, lens, 32),
        lambda: td.td_decode_attn_f8(q.float(), *cache, lens, 16),
        lambda: td.td_decode_attn_f8(q[:1], *cache, lens, 16),
        lambda: td.td_decode_attn_f8(q, *cache, lens, 16, out=torch.empty_like(q).float()),
        lambda: td.td_decode_attn_f8(q, *cache, lens, 16, lse=torch.empty(2, 3, device="cuda")),
        lambda: td.td_decode_attn_f8(q, *cache, lens, 16, workspace=torch.zeros(64, device="cuda")),
        lambda: td.td_verify_attn_f8(q, *cache, lens, 16),
        lambda: td.td_rope_kv_append_f8(x, x, *cache, lens, 16, torch.zeros(63, 64, device="cuda"), torch.zeros(63, 64, device="cuda")),
        lambda: td.td_kv_read_f8(*cache, lens, 16, start=lens.long()),
    ]
    for call in bad:
        with pytest.raises((TypeError, ValueError)):
            call()
    from decode_attention_split_gb300._lib import TDError
    for call in (lambda: td.td_decode_attn_f8(q, *cache, lens, 16, split=24),
                 lambda: td.td_decode_attn_f8(q, *cache, lens, 16, workspace=torch.zeros(256, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(TDError):
            call()
