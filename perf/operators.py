"""Cases for the 8-bit KV cache held in blocks (e4m3 codes, one fp32 scale per block of tokens and head).

Operators: the append that quantises new rows (with and without a rotation first, the rotation
taking one position per token or one per axis), the read-back into bf16 or fp32 rows, and the
decode and verify attention over the cache. ``run`` makes one call; with ``own`` false it is
computed in elementary torch operations in 32 bits, with ``own`` true by the library.

The cache: codes float8_e4m3fn [B, Hkv, Smax, D], scales fp32 [B, Hkv, ceil(Smax / block)]; a row
reads back as code * scale. An append gives each block it writes the scale
    s = max(old scale if the block already holds rows, 2^k),  k the least with max|x| <= 448 * 2^k
(k >= -126), brings the block's older codes to it (code * (old / s), rounded), and stores its
rows as x * (1 / s), rounded to nearest even.

Lengths are spread over their range by a fixed rule and dealt to the sequences by the seed, so
that a case's work does not depend on the seed.
"""
import math

import torch

own = False

F8 = torch.float8_e4m3fn
NEW = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # the next token's rows of a small batch of a 360M-style layer: a call's own latency
        dict(name="append token 360m x8", op="append", B=8, Hq=15, Hkv=5, D=64, Smax=1024, block=16, T=1, lo=1, hi=900,
             dtype="bf16"),
        # ragged prompts of an odd length behind a shared prefix, rows still in fp32
        dict(name="append prompts f32 x8", op="append", B=8, Hq=15, Hkv=5, D=64, Smax=2048, block=32, T=777, lo=0, hi=1000,
             dtype="f32"),
        # a 4k prompt chunk of the 3B-style layer that starts inside a block
        dict(name="append prompt 3b 4k", op="append", B=1, Hq=24, Hkv=8, D=128, Smax=8192, block=64, T=4096, lo=1003,
             hi=1003, dtype="bf16"),
        # one decode step's rotation and cache write for a batch of 32, three position axes
        dict(name="rope token axes x32", op="rope", B=32, Hq=32, Hkv=8, D=128, Smax=1024, block=64, T=1, lo=1, hi=1000,
             dtype="bf16", axes=3),
        # a long prompt rotated at its cache positions
        dict(name="rope prompt 3b 8k", op="rope", B=1, Hq=24, Hkv=8, D=128, Smax=16384, block=64, T=8000, lo=100, hi=100,
             dtype="bf16", axes=0),
        # prompts of images and text: three axes, odd lengths
        dict(name="rope images axes x4", op="rope", B=4, Hq=32, Hkv=8, D=128, Smax=4096, block=32, T=1531, lo=0, hi=777,
             dtype="bf16", axes=3),
        # a whole 8k context back in bf16, as a prefill over it wants
        dict(name="read 3b 8k", op="read", B=1, Hq=24, Hkv=8, D=128, Smax=16384, block=64, rows=8192, lo=8192, hi=8192,
             first=0, dtype="bf16"),
        # windows of ragged sequences in fp32, most of them starting inside a block
        dict(name="read windows f32 x16", op="read", B=16, Hq=15, Hkv=5, D=64, Smax=2048, block=16, rows=500, lo=1,
             hi=2048, first=300, dtype="f32"),
        # one token over 4k keys of the 360M-style layer: a decode call's latency
        dict(name="decode 360m 4k", op="decode", B=1, Hq=15, Hkv=5, D=64, Smax=4096, block=32, T=1, lo=4096, hi=4096),
        # one token over the 3B-style layer's full 32k context
        dict(name="decode 3b 32k", op="decode", B=1, Hq=24, Hkv=8, D=128, Smax=32768, block=64, T=1, lo=32768, hi=32768),
        # a ragged batch of 32 with up to 8k keys each
        dict(name="decode ragged x32", op="decode", B=32, Hq=32, Hkv=8, D=128, Smax=8192, block=64, T=1, lo=1, hi=8192),
        # a speculative-verify chunk of six tokens over 16k keys, eight sequences
        dict(name="verify six 16k x8", op="verify", B=8, Hq=32, Hkv=8, D=128, Smax=16400, block=16, T=6, lo=16390, hi=16390),
    ]


def _logint(rng, a, b):
    return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))


def draw(rng):
    op = rng.choice(["append", "append", "rope", "rope", "read", "decode", "decode", "verify", "verify"])
    D = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 3, 5, 8])
    G = rng.choice([1, 2, 3, 4, 7, 8])
    block = rng.choice([16, 32, 64, 128])
    Hq = Hkv * G
    c = dict(op=op, Hq=Hq, Hkv=Hkv, D=D, block=block)
    if op in ("append", "rope"):
        T = rng.choice([1, 1, rng.randint(2, 16), _logint(rng, 17, 4000)])
        most = int(20e6 / (T * (Hq + 2 * Hkv) * D))
        B = _logint(rng, 1, 64) if T <= 16 else rng.randint(1, max(1, min(6, most)))
        hi = rng.randint(1, 2000)
        Smax = (hi + T + 3 * block + block - 1) // block * block
        c.update(B=B, T=T, lo=rng.randint(0, hi), hi=hi, Smax=Smax, dtype=rng.choice(["bf16", "bf16", "f32"]))
        if op == "rope":
            c["axes"] = rng.choice([0, 2, 3])
    elif op == "read":
        rows = _logint(rng, 1, 6000)
        hi = _logint(rng, 1, 8000)
        c.update(B=rng.randint(1, 4) if rows > 1000 else _logint(rng, 1, 32), rows=rows, lo=rng.randint(0, hi), hi=hi,
                 Smax=hi + rng.randint(0, 200), first=rng.choice([0, rng.randint(1, 500)]), dtype=rng.choice(["bf16", "f32"]))
    else:
        hi = _logint(rng, 1 if op == "decode" else 16, 30000)
        T = 1 if op == "decode" else rng.randint(2, 12)
        most = max(1, min(64, 130000 // hi, 3000000 // (hi * G * T)))
        c.update(B=_logint(rng, 1, most), T=T, lo=rng.choice([0, hi, rng.randint(0, hi)]), hi=hi,
                 Smax=hi + rng.randint(0, 100))
    return c


# ------------------------------------------------------------------------------ the inputs

def _lengths(case):
    """The case's lengths: spread over [lo, hi] by the golden ratio, hi among them."""
    lo, hi, B = case["lo"], case["hi"], case["B"]
    return [hi - int((i * 0.6180339887498949) % 1.0 * (hi - lo + 1)) for i in range(B)]


def _window(case):
    """Blocks of the cache that T new rows of a sequence can touch."""
    return (case["T"] + case["block"] - 2) // case["block"] + 1


def _starts(case):
    """First row read back of each sequence: `first` rows on, and back by a few for the odd ones."""
    return [max(0, case["first"] - 7 * (i % 5)) for i in range(case["B"])]


def _pow2_scale(amax):
    """The least 2^k (k >= -126) with amax <= 448 * 2^k."""
    m, e = torch.frexp(amax)
    k = torch.where(m <= 0.875, e - 9, e - 8)
    k = torch.where(amax > 0, k, torch.full_like(k, -126)).clamp(min=-126)
    return ((k.int() + 127) << 23).view(torch.float32)


def _rows(B, H, N, D, g, heavy, dev):
    """Rows of a cache: channels of different strength, and now and then a row eight times the others."""
    x = torch.randn(B, H, N, D, generator=g, device=dev)
    x *= torch.exp(0.5 * torch.randn(1, H, 1, D, generator=g, device=dev))
    if heavy:
        x *= 1.0 + 7.0 * (torch.rand(B, H, N, 1, generator=g, device=dev) < 0.01)
    return x


def _filled(B, H, S, D, block, g, heavy, dev):
    """A cache of S rows as appends leave it: codes and scales."""
    NB = -(-S // block)
    x = _rows(B, H, NB * block, D, g, heavy, dev).view(B, H, NB, block, D)
    s = _pow2_scale(x.abs().amax(dim=(3, 4)))
    x /= s[..., None, None]
    codes = x.to(F8).view(B, H, NB * block, D)
    return (codes if NB * block == S else codes[:, :, :S].contiguous()), s


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    B, Hq, Hkv, D, S, block = (case[k] for k in ("B", "Hq", "Hkv", "D", "Smax", "block"))
    order = torch.randperm(B, generator=g, device=dev)
    lens = torch.tensor(_lengths(case), dtype=torch.int32, device=dev)[order]
    kc, ks = _filled(B, Hkv, S, D, block, g, case["op"] in ("decode", "verify"), dev)
    vc, vs = _filled(B, Hkv, S, D, block, g, False, dev)
    st = dict(case=case, kc=kc, ks=ks, vc=vc, vs=vs, lens=lens)
    if case["op"] in ("append", "rope"):
        dt = NEW[case["dtype"]]
        st["k_new"] = _rows(B, Hkv, case["T"], D, g, False, dev).to(dt)
        st["v_new"] = _rows(B, Hkv, case["T"], D, g, False, dev).to(dt)
    if case["op"] == "rope":
        st["q"] = torch.randn(B, Hq, case["T"], D, generator=g, device=dev).to(dt)
        st["q_out"] = torch.empty_like(st["q"])
        A, T = case["axes"], case["T"]
        inv = 500000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64, device=dev) / D)
        ang = torch.arange(S, dtype=torch.float64, device=dev)[:, None] * inv
        st["cos"], st["sin"] = ang.cos().float(), ang.sin().float()
        st["pos"] = st["axis"] = None
        if A:
            # time runs with the tokens, the other axes over a grid's rows and columns
            pos = torch.randint(0, min(S, 64), (B, T, A), generator=g, device=dev, dtype=torch.int32)
            pos[:, :, 0] = (lens[:, None] + torch.arange(T, device=dev, dtype=torch.int32)) % S
            st["pos"] = pos
            st["axis"] = (torch.arange(D // 2, device=dev) * A // (D // 2)).to(torch.int32)
    if case["op"] == "read":
        dt = NEW[case["dtype"]]
        st["start"] = torch.tensor(_starts(case), dtype=torch.int32, device=dev)[order]
        st["k_out"] = torch.zeros(B, Hkv, case["rows"], D, dtype=dt, device=dev)
        st["v_out"] = torch.zeros(B, Hkv, case["rows"], D, dtype=dt, device=dev)
    if case["op"] in ("decode", "verify"):
        st["q"] = torch.randn(B, Hq, case["T"], D, generator=g, device=dev).to(torch.bfloat16)
        if case["op"] == "decode":
            st["q"] = st["q"][:, :, 0].contiguous()
        st["out"] = torch.empty_like(st["q"])
        st["lse"] = torch.empty(st["q"].shape[:-1], dtype=torch.float32, device=dev)
    return st


# ------------------------------------------------------------------------------ one pass

def run(st):
    case = st["case"]
    if own:
        return _own(st, case)
    return {"append": _append, "rope": _rope_append, "read": _read, "decode": _attend, "verify": _attend}[case["op"]](st, case)


def _own(st, case):
    import decode_attention_split_gb300 as td
    cache = (st["kc"], st["ks"], st["vc"], st["vs"], st["lens"], case["block"])
    if case["op"] == "append":
        td.td_kv_append_f8(st["k_new"], st["v_new"], *cache, advance=False)
        return {"k_codes": st["kc"], "k_scales": st["ks"], "v_codes": st["vc"], "v_scales": st["vs"]}
    if case["op"] == "rope":
        td.td_rope_kv_append_f8(st["k_new"], st["v_new"], *cache, st["cos"], st["sin"], positions=st["pos"],
                                axes=st["axis"], q=st["q"], q_out=st["q_out"], advance=False)
        return {"q": st["q_out"], "k_codes": st["kc"], "k_scales": st["ks"], "v_codes": st["vc"], "v_scales": st["vs"]}
    if case["op"] == "read":
        k, v = td.td_kv_read_f8(*cache, start=st["start"], k_out=st["k_out"], v_out=st["v_out"])
        return {"k": k, "v": v}
    call = td.td_decode_attn_f8 if case["op"] == "decode" else td.td_verify_attn_f8
    out, lse = call(st["q"], *cache, out=st["out"], lse=st["lse"])
    return {"out": out, "lse": lse}


def _write(codes, scales, new, lens, T, block):
    """Quantises rows new [B, H, T, D] into codes and scales behind the first lens[b] rows."""
    B, H, S, D = codes.shape
    n = (T + block - 2) // block + 1
    j0 = (lens // block).long()                                                   # first block touched
    blk = j0[:, None] + torch.arange(n, device=codes.device)                      # [B, n]
    row = (j0 * block)[:, None] + torch.arange(n * block, device=codes.device)    # [B, n * block]
    t = row - lens[:, None].long()
    fresh = (t >= 0) & (t < T)
    x = torch.gather(new.float(), 2, t.clamp(0, T - 1)[:, None, :, None].expand(B, H, -1, D))
    x = torch.where(fresh[:, None, :, None], x, torch.zeros_like(x)).view(B, H, n, block, D)
    touched = fresh.view(B, n, block).any(-1)
    s_old = torch.gather(scales, 2, blk[:, None].expand(B, H, n))
    s = _pow2_scale(x.abs().amax(dim=(3, 4)))
    held = (blk * block < lens[:, None])[:, None]
    s = torch.where(held, torch.maximum(s, s_old), s)
    s = torch.where(touched[:, None], s, s_old)
    at = row[:, None, :, None].expand(B, H, -1, D)
    bytes_ = codes.view(torch.uint8)
    old = torch.gather(bytes_, 2, at)
    moved = (old.view(F8).float().view(B, H, n, block, D) * (s_old / s)[..., None, None]).to(F8)
    put = (x * (1.0 / s)[..., None, None]).clamp(-448, 448).to(F8)
    got = torch.where(fresh.view(B, 1, n, block, 1), put.view(torch.uint8), moved.view(torch.uint8)).view(B, H, n * block, D)
    write = fresh | ((t < 0) & touched.repeat_interleave(block, dim=1))
    bytes_.scatter_(2, at, torch.where(write[:, None, :, None], got, old))
    scales.scatter_(2, blk[:, None].expand(B, H, n), s)


def _append(st, case):
    _write(st["kc"], st["ks"], st["k_new"], st["lens"], case["T"], case["block"])
    _write(st["vc"], st["vs"], st["v_new"], st["lens"], case["T"], case["block"])
    return {"k_codes": st["kc"], "k_scales": st["ks"], "v_codes": st["vc"], "v_scales": st["vs"]}


def _turn(x, c, s):
    h = x.shape[-1] // 2
    lo, hi = x[..., :h].float(), x[..., h:].float()
    return torch.cat([lo * c - hi * s, hi * c + lo * s], dim=-1)


def _rope_append(st, case):
    T, h = case["T"], case["D"] // 2
    lens = st["lens"].long()
    if st["pos"] is None:
        at = (lens[:, None] + torch.arange(T, device=lens.device))[:, :, None].expand(-1, -1, h)
    else:
        at = st["pos"].long()[:, :, st["axis"].long()]                             # [B, T, h]
    c, s = torch.gather(st["cos"][None].expand(at.shape[0], -1, -1), 1, at), torch.gather(st["sin"][None].expand(at.shape[0], -1, -1), 1, at)
    c, s = c[:, None], s[:, None]
    st["q_out"].copy_(_turn(st["q"], c, s))
    _write(st["kc"], st["ks"], _turn(st["k_new"], c, s), st["lens"], T, case["block"])
    _write(st["vc"], st["vs"], st["v_new"], st["lens"], T, case["block"])
    return {"q": st["q_out"], "k_codes": st["kc"], "k_scales": st["ks"], "v_codes": st["vc"], "v_scales": st["vs"]}


def _values(codes, scales, block):
    return codes.float() * scales.repeat_interleave(block, dim=2)[:, :, :codes.shape[2], None]


def _read(st, case):
    N = case["rows"]
    row = st["start"].long()[:, None] + torch.arange(N, device=st["lens"].device)
    keep = (row < st["lens"][:, None])[:, None, :, None]
    at = row.clamp(max=case["Smax"] - 1)
    blk = (at // case["block"])[:, None].expand(-1, case["Hkv"], -1)
    at = at[:, None, :, None].expand(-1, case["Hkv"], -1, case["D"])
    for codes, scales, out in ((st["kc"], st["ks"], st["k_out"]), (st["vc"], st["vs"], st["v_out"])):
        x = torch.gather(codes.view(torch.uint8), 2, at).view(F8).float() * torch.gather(scales, 2, blk)[..., None]
        out.copy_(torch.where(keep, x.to(out.dtype), out))
    return {"k": st["k_out"], "v": st["v_out"]}


def _attend(st, case):
    B, Hq, Hkv, D, T, S = (case[k] for k in ("B", "Hq", "Hkv", "D", "T", "Smax"))
    q = st["q"].float().view(B, Hkv, Hq // Hkv * T, D) * (1.0 / math.sqrt(D))
    k, v = _values(st["kc"], st["ks"], case["block"]), _values(st["vc"], st["vs"], case["block"])
    key = torch.arange(S, device=q.device)
    v = torch.where((key < st["lens"][:, None])[:, None, :, None], v, torch.zeros_like(v))
    see = st["lens"][:, None] - T + 1 + torch.arange(T, device=q.device)          # keys each token sees
    see = see.repeat(1, Hq // Hkv)[:, None, :, None]                               # rows are (head in group, token)
    x = (q @ k.transpose(2, 3)).masked_fill(key >= see, float("-inf"))
    m = x.amax(-1, keepdim=True).clamp(min=-3e38)
    p = torch.exp(x - m)
    total = p.sum(-1, keepdim=True)
    out = (p @ v) / torch.where(total > 0, total, torch.ones_like(total))
    lse = torch.where(total > 0, m + torch.log(total), torch.full_like(total, float("-inf")))
    return {"out": out.to(torch.bfloat16).view(st["q"].shape), "lse": lse.view(st["lse"].shape)}


# ------------------------------------------------------------------------------ the floor and the exact values

def work(case):
    B, Hq, Hkv, D, block = (case[k] for k in ("B", "Hq", "Hkv", "D", "block"))
    L = _lengths(case)
    if case["op"] in ("append", "rope"):
        T, e = case["T"], 2 if case["dtype"] == "bf16" else 4
        rows = B * Hkv * T * 2
        scales = sum(-(-(n % block + T) // block) for n in L) * Hkv * 2 * 4
        total = rows * D * (e + 1) + scales + 4 * B
        if case["op"] == "append":
            return {"bytes": total, "flops": 3 * rows * D}
        total += 2 * B * Hq * T * D * e
        total += (D // 2) * (4 + 4 * case["axes"] + 4 * T) + 4 * B * T * case["axes"]
        return {"bytes": total, "flops": 3 * rows * D + 3 * B * (Hq + Hkv) * T * D}
    if case["op"] == "read":
        rows = sum(max(0, min(case["rows"], n - s)) for n, s in zip(L, _starts(case))) * Hkv * 2
        e = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": rows * (D * (1 + e) + 4.0 / block) + 8 * B, "flops": rows * D}
    T = case["T"]
    kv = sum(L) * Hkv * 2 * (D + 4.0 / block)
    return {"bytes": kv + B * Hq * T * (4 * D + 4) + 4 * B, "flops": sum(L) * Hq * T * 4 * D}


def _two_to(k):
    """2^k in 64 bits, exactly."""
    return ((k.long() + 1023) << 52).view(torch.float64)


def _round_e4m3(x):
    """Values of x (64 bits, at most 448) to e4m3's grid, ties to even: 8 steps to a binade, 2^-9 the least."""
    m, e = torch.frexp(x)
    step = _two_to((e - 4).clamp(min=-9))
    return torch.round(x / step) * step


def _exact_write(codes, scales, new, lens, T, block):
    """Block by block and sequence by sequence, in 64 bits: the code values and scales afterwards."""
    c, s = codes.double(), scales.double().clone()
    for b, L in enumerate(lens):
        a = L
        while a < L + T:
            j = a // block
            z = min(L + T, (j + 1) * block)
            x = new[b, :, a - L:z - L]
            big = x.abs().flatten(1).amax(1)
            k = torch.ceil(torch.log2(big.clamp(min=2.0 ** -110) / 448.0))
            k = torch.where(big > 448.0 * _two_to(k), k + 1, torch.where(big <= 448.0 * _two_to(k - 1), k - 1, k))
            one = torch.where(big > 0, _two_to(k.clamp(min=-126)), torch.full_like(big, 2.0 ** -126))
            if j * block < a:
                one = torch.maximum(one, s[b, :, j])
                c[b, :, j * block:a] = _round_e4m3(c[b, :, j * block:a] * (s[b, :, j] / one)[:, None, None])
            s[b, :, j] = one
            c[b, :, a:z] = _round_e4m3(x / one[:, None, None])
            a = z
    return c, s


def exact(case, seed):
    st = prepare(case, seed)
    lens = st["lens"].tolist()
    B, Hq, Hkv, D, block = (case[k] for k in ("B", "Hq", "Hkv", "D", "block"))
    if case["op"] in ("append", "rope"):
        T, kn, q = case["T"], st["k_new"].double(), None
        if case["op"] == "rope":
            h = D // 2
            rows = []
            for b, L in enumerate(lens):
                if st["pos"] is None:
                    c, s = st["cos"][L:L + T].double(), st["sin"][L:L + T].double()
                else:
                    i = torch.arange(h, device=kn.device)
                    p = torch.stack([st["pos"][b, :, a] for a in st["axis"].tolist()], dim=1).long()
                    c, s = st["cos"][p, i].double(), st["sin"][p, i].double()
                z = torch.complex(c, s)
                turned = [torch.complex(x[b, ..., :h].double(), x[b, ..., h:].double()) * z for x in (st["q"], st["k_new"])]
                rows.append([torch.cat([y.real, y.imag], dim=-1) for y in turned])
            q, kn = torch.stack([r[0] for r in rows]), torch.stack([r[1] for r in rows])
        kc, ks = _exact_write(st["kc"], st["ks"], kn, lens, T, block)
        vc, vs = _exact_write(st["vc"], st["vs"], st["v_new"].double(), lens, T, block)
        got = {"k_codes": kc, "k_scales": ks, "v_codes": vc, "v_scales": vs}
        return got if q is None else {"q": q, **got}
    if case["op"] == "read":
        k, v = st["k_out"].double(), st["v_out"].double()
        for b, (L, a) in enumerate(zip(lens, st["start"].tolist())):
            for out, codes, scales in ((k, st["kc"], st["ks"]), (v, st["vc"], st["vs"])):
                n = max(0, min(case["rows"], L - a))
                j = (a + torch.arange(n, device=out.device)) // block
                out[b, :, :n] = codes[b, :, a:a + n].double() * scales[b][:, j, None].double()
        return {"k": k, "v": v}
    T, G = case["T"], Hq // Hkv
    q = st["q"].double().view(B, Hkv, G, T, D)
    out = torch.zeros(B, Hkv, G, T, D, dtype=torch.float64, device=q.device)
    lse = torch.full((B, Hkv, G, T), float("-inf"), dtype=torch.float64, device=q.device)
    for b, L in enumerate(lens):
        j = torch.arange(L, device=q.device) // block
        k = st["kc"][b, :, :L].double() * st["ks"][b][:, j, None].double()
        v = st["vc"][b, :, :L].double() * st["vs"][b][:, j, None].double()
        for t in range(T):
            n = L - T + t + 1
            if n > 0:
                x = torch.einsum("hgd,hjd->hgj", q[b, :, :, t], k[:, :n]) / math.sqrt(D)
                lse[b, :, :, t] = torch.logsumexp(x, dim=-1)
                out[b, :, :, t] = torch.einsum("hgj,hjd->hgd", torch.softmax(x, dim=-1), v[:, :n])
    return {"out": out.view(st["q"].shape), "lse": lse.view(st["lse"].shape)}
