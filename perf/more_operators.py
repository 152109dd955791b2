"""Cases for three operators of a serving step: the new rows' norms with their rotation and cache write,
attention over a sliding window with a few first tokens that stay visible, and attention of a batch that
shares a long prefix.

``norm``: every head's query and key row is divided by its root mean square, sqrt(mean(x^2) + eps), and
multiplied by a weight per dimension; then it is rotated to its position (pairs (x[i], x[i + D/2])), and
keys and values go into the cache behind each sequence's length.

``window``: the query of token t (position P = length - T + t) attends keys j <= P with j > P - window or
j < sinks: for one token, a short chunk, or a prompt.

``prefix``: the queries of B sequences attend the keys of one shared prefix [Hkv, Pmax, D] and then the
sequence's own keys, causal among its last T.

``run`` makes one call; with ``own`` false it is computed in elementary torch operations in 32 bits, with
``own`` true by the library. Lengths are spread over their range by a fixed rule and dealt to the
sequences by the seed, so that a case's work does not depend on the seed.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6


def listed():
    return [
        # the next token's rows of a small batch of a 360M-style layer: a call's own latency
        dict(name="norm token 360m x8", op="norm", B=8, Hq=15, Hkv=5, D=64, Smax=1024, T=1, lo=1, hi=900, dtype="bf16",
             axes=0),
        # a 4k prompt chunk of the 3B-style layer on top of a thousand tokens
        dict(name="norm prompt 3b 4k", op="norm", B=1, Hq=24, Hkv=8, D=128, Smax=8192, T=4096, lo=1003, hi=1003,
             dtype="bf16", axes=0),
        # prompts of images and text in fp32: three position axes, odd lengths
        dict(name="norm images f32 x4", op="norm", B=4, Hq=32, Hkv=8, D=128, Smax=2048, T=777, lo=0, hi=500, dtype="f32",
             axes=3),
        # one token far into a long context of the 3B-style layer, most of which its window has left behind
        dict(name="window decode 3b 32k", op="window", B=1, Hq=24, Hkv=8, D=128, Smax=32768, T=1, lo=32768, hi=32768,
             window=4096, sinks=4, dtype="bf16"),
        # a ragged batch, some sequences shorter than the window
        dict(name="window decode ragged x32", op="window", B=32, Hq=32, Hkv=8, D=128, Smax=8192, T=1, lo=1, hi=8192,
             window=1024, sinks=4, dtype="bf16"),
        # fp32 rows, an odd window, no sinks: the smallest attention call
        dict(name="window decode f32 x4", op="window", B=4, Hq=4, Hkv=2, D=64, Smax=1024, T=1, lo=200, hi=1000, window=250,
             sinks=0, dtype="f32"),
        # a speculative-verify chunk of six tokens, eight sequences
        dict(name="window verify six x8", op="window", B=8, Hq=32, Hkv=8, D=128, Smax=16400, T=6, lo=7000, hi=16390,
             window=2048, sinks=16, dtype="bf16"),
        # an 8k prompt whose tokens see a thousand others each
        dict(name="window prompt 3b 8k", op="prompt", B=1, Hq=24, Hkv=8, D=128, Smax=8192, T=8000, lo=8100, hi=8100,
             window=1024, sinks=4, dtype="bf16"),
        # four short conversations behind one system prompt, 360M-style layer
        dict(name="prefix decode 360m x4", op="prefix", B=4, Hq=15, Hkv=5, D=64, Pmax=1024, P=1000, Smax=256, T=1, lo=1,
             hi=200, dtype="bf16"),
        # sixty-four users of one 8k prompt, up to 512 tokens of their own
        dict(name="prefix decode 8k x64", op="prefix", B=64, Hq=32, Hkv=8, D=128, Pmax=8192, P=8192, Smax=512, T=1, lo=1,
             hi=512, dtype="bf16"),
        # sixteen continuations of one 32k document of an odd length, 3B-style layer
        dict(name="prefix decode 3b 32k x16", op="prefix", B=16, Hq=24, Hkv=8, D=128, Pmax=32768, P=32003, Smax=1024, T=1,
             lo=1, hi=1000, dtype="bf16"),
        # verify chunks of six tokens of sixteen sequences behind a 4k prompt
        dict(name="prefix verify six x16", op="prefix", B=16, Hq=32, Hkv=8, D=128, Pmax=5000, P=4321, Smax=800, T=6, lo=6,
             hi=777, dtype="bf16"),
    ]


def _logint(rng, a, b):
    return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "window", "window", "window", "prompt", "prefix", "prefix", "prefix"])
    D = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 3, 5, 8])
    G = rng.choice([1, 2, 3, 4, 7, 8])
    Hq = Hkv * G
    c = dict(op=op, Hq=Hq, Hkv=Hkv, D=D, dtype="bf16")
    if op == "norm":
        T = rng.choice([1, 1, rng.randint(2, 16), _logint(rng, 17, 4000)])
        most = int(20e6 / (T * (Hq + 2 * Hkv) * D))
        hi = rng.randint(1, 2000)
        c.update(B=_logint(rng, 1, 64) if T <= 16 else rng.randint(1, max(1, min(6, most))), T=T, lo=rng.randint(0, hi),
                 hi=hi, Smax=hi + T + rng.randint(0, 100), dtype=rng.choice(["bf16", "bf16", "f32"]),
                 axes=rng.choice([0, 0, 1, 3]))
    elif op == "window":
        T = rng.choice([1, 1, rng.randint(2, 12)])
        hi = _logint(rng, T, 30000)
        window = _logint(rng, 1, 8000)
        sinks = rng.choice([0, 1, 4, rng.randint(0, 200)])
        see = min(hi, window + sinks + T)
        most = max(1, min(64, 60000 // see, 300000 // hi, 3000000 // (hi * G * T)))
        c.update(B=_logint(rng, 1, most), T=T, lo=rng.choice([T, hi, rng.randint(T, hi)]), hi=hi,
                 Smax=hi + rng.randint(0, 100), window=window, sinks=sinks,
                 dtype=rng.choice(["bf16", "bf16", "bf16", "f32"]))
    elif op == "prompt":
        T = _logint(rng, 17, 4000)
        hi = T + rng.randint(0, 1000)
        c.update(B=1 if T > 1000 else rng.randint(1, 3), T=T, lo=rng.randint(T, hi), hi=hi, Smax=hi + rng.randint(0, 100),
                 window=_logint(rng, 1, 2000), sinks=rng.choice([0, 1, 4, rng.randint(0, 200)]))
    else:
        T = rng.choice([1, 1, rng.randint(2, 8)])
        P = _logint(rng, 16, 30000)
        hi = _logint(rng, T, 1000)
        most = max(1, min(64, 30000 // hi, int(4e6) // (P * G * T)))
        c.update(B=_logint(rng, 1, most), T=T, lo=rng.choice([T, rng.randint(T, hi)]), hi=hi, P=P,
                 Pmax=P + rng.randint(0, 100), Smax=hi + rng.randint(0, 100))
    return c


# ------------------------------------------------------------------------------ the inputs

def _lengths(case):
    """The case's lengths: spread over [lo, hi] by the golden ratio, hi among them."""
    lo, hi, B = case["lo"], case["hi"], case["B"]
    return [hi - int((i * 0.6180339887498949) % 1.0 * (hi - lo + 1)) for i in range(B)]


def _rows(shape, g, dev):
    """Rows of heads [.., H, N, D]: channels of different strength, and now and then a row four times the others."""
    x = torch.randn(shape, generator=g, device=dev)
    x *= torch.exp(0.4 * torch.randn(shape[-3], 1, shape[-1], generator=g, device=dev))
    x *= 1.0 + 3.0 * (torch.rand(*shape[:-1], 1, generator=g, device=dev) < 0.01)
    return x


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    B, Hq, Hkv, D, S, T = (case[k] for k in ("B", "Hq", "Hkv", "D", "Smax", "T"))
    dt = TYPES[case["dtype"]]
    order = torch.randperm(B, generator=g, device=dev)
    lens = torch.tensor(_lengths(case), dtype=torch.int32, device=dev)[order]
    k, v = _rows((B, Hkv, S, D), g, dev), torch.randn(B, Hkv, S, D, generator=g, device=dev)
    st = dict(case=case, lens=lens)
    if case["op"] == "norm":
        st.update(k=k.to(dt), v=v.to(dt))
        st["k_new"] = (2.0 * _rows((B, Hkv, T, D), g, dev)).to(dt)
        st["v_new"] = torch.randn(B, Hkv, T, D, generator=g, device=dev).to(dt)
        st["q"] = (2.0 * _rows((B, Hq, T, D), g, dev)).to(dt)
        st["q_out"] = torch.empty_like(st["q"])
        st["qw"] = 1.0 + 0.3 * torch.randn(D, generator=g, device=dev)
        st["kw"] = 1.0 + 0.3 * torch.randn(D, generator=g, device=dev)
        inv = 500000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64, device=dev) / D)
        ang = torch.arange(S, dtype=torch.float64, device=dev)[:, None] * inv
        st["cos"], st["sin"] = ang.cos().float(), ang.sin().float()
        st["pos"] = st["axis"] = None
        A = case["axes"]
        if A:
            # time runs with the tokens (behind a prefix of other rows), the other axes over a grid's rows and columns
            pos = torch.randint(0, min(S, 64), (B, T, A), generator=g, device=dev, dtype=torch.int32)
            pos[:, :, 0] = (lens[:, None] + torch.arange(T, device=dev, dtype=torch.int32) + 11) % S
            st["pos"] = pos
            st["axis"] = (torch.arange(D // 2, device=dev) * A // (D // 2)).to(torch.int32)
        return st
    q = _rows((B, Hq, T, D), g, dev)
    if case["op"] in ("window", "prompt") and case["sinks"]:
        # the first tokens draw the queries' attention, as they do in models that lean on them
        u = torch.randn(Hkv, 1, D, generator=g, device=dev)
        k[:, :, :case["sinks"]] = 0.3 * k[:, :, :case["sinks"]] + u
        q += 0.5 * u.repeat_interleave(Hq // Hkv, dim=0)
    if case["op"] == "prefix":
        st["kp"] = _rows((Hkv, case["Pmax"], D), g, dev).to(dt)
        st["vp"] = torch.randn(Hkv, case["Pmax"], D, generator=g, device=dev).to(dt)
        st["plen"] = torch.tensor([case["P"]], dtype=torch.int32, device=dev)
    st.update(k=k.to(dt), v=v.to(dt), q=q.to(dt))
    if T == 1 and case["op"] != "prompt":
        st["q"] = st["q"][:, :, 0].contiguous()
    st["out"] = torch.empty_like(st["q"])
    st["lse"] = torch.empty(st["q"].shape[:-1], dtype=torch.float32, device=dev)
    return st


# ------------------------------------------------------------------------------ one pass

def run(st):
    case = st["case"]
    if own:
        return _own(st, case)
    return {"norm": _norm, "window": _window, "prompt": _window, "prefix": _prefix}[case["op"]](st, case)


def _own(st, case):
    import decode_attention_split_gb300 as td
    if case["op"] == "norm":
        td.td_norm_rope_kv_append(st["k_new"], st["v_new"], st["k"], st["v"], st["lens"], st["kw"], st["cos"], st["sin"],
                                  eps=EPS, positions=st["pos"], axes=st["axis"], q=st["q"], q_weight=st["qw"],
                                  q_out=st["q_out"], advance=False)
        return {"q": st["q_out"], "k": st["k"], "v": st["v"]}
    if case["op"] == "prefix":
        call = td.td_decode_attn_prefix if case["T"] == 1 else td.td_verify_attn_prefix
        out, lse = call(st["q"], st["kp"], st["vp"], st["plen"], st["k"], st["v"], st["lens"], out=st["out"], lse=st["lse"])
        return {"out": out, "lse": lse}
    call = td.td_prefill_attn_window if case["op"] == "prompt" else \
        td.td_decode_attn_window if case["T"] == 1 else td.td_verify_attn_window
    out, lse = call(st["q"], st["k"], st["v"], st["lens"], case["window"], case["sinks"], out=st["out"], lse=st["lse"])
    return {"out": out, "lse": lse}


def _turn(x, c, s):
    h = x.shape[-1] // 2
    lo, hi = x[..., :h], x[..., h:]
    return torch.cat([lo * c - hi * s, hi * c + lo * s], dim=-1)


def _norm(st, case):
    B, Hkv, T, D = st["k_new"].shape
    lens = st["lens"].long()
    row = lens[:, None] + torch.arange(T, device=lens.device)                      # [B, T]
    if st["pos"] is None:
        at = row[:, :, None].expand(-1, -1, D // 2)
    else:
        at = st["pos"].long()[:, :, st["axis"].long()]                              # [B, T, D/2]
    c, s = (torch.gather(t[None].expand(B, -1, -1), 1, at)[:, None] for t in (st["cos"], st["sin"]))

    def normed(x, w):
        x = x.float()
        return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w
    st["q_out"].copy_(_turn(normed(st["q"], st["qw"]), c, s))
    to = row[:, None, :, None].expand(B, Hkv, T, D)
    st["k"].scatter_(2, to, _turn(normed(st["k_new"], st["kw"]), c, s).to(st["k"].dtype))
    st["v"].scatter_(2, to, st["v_new"])
    return {"q": st["q_out"], "k": st["k"], "v": st["v"]}


def _window(st, case):
    """Sequence by sequence and kv head by kv head, over the keys that any of its tokens sees."""
    B, Hq, Hkv, D, T, W, C = (case[k] for k in ("B", "Hq", "Hkv", "D", "T", "window", "sinks"))
    G = Hq // Hkv
    q = st["q"].view(B, Hkv, G, T, D)
    out, lse = st["out"].view(B, Hkv, G, T, D), st["lse"].view(B, Hkv, G, T)
    t = torch.arange(T, device=q.device)
    key = torch.arange(case["Smax"], device=q.device)
    for h in range(Hkv):
        for b0 in range(0, B, 8 if T < 100 else 1):
            b1 = min(B, b0 + (8 if T < 100 else 1))
            p = (st["lens"][b0:b1, None] - T + t)[:, None, :, None]                 # positions
            see = (key <= p) & ((key > p - W) | (key < C))                          # [b, 1, T, Smax]
            k, v = st["k"][b0:b1, h, None].float(), st["v"][b0:b1, h, None].float()
            x = (q[b0:b1, h].float() * (1.0 / math.sqrt(D))) @ k.transpose(2, 3)    # [b, G, T, Smax]
            x.masked_fill_(~see, float("-inf"))
            m = x.amax(-1, keepdim=True)
            x.sub_(m).exp_()
            total = x.sum(-1, keepdim=True)
            out[b0:b1, h] = ((x @ v) / total).to(out.dtype)
            lse[b0:b1, h] = (m + torch.log(total))[..., 0]
    return {"out": st["out"], "lse": st["lse"]}


def _prefix(st, case):
    B, Hq, Hkv, D, T, S = (case[k] for k in ("B", "Hq", "Hkv", "D", "T", "Smax"))
    G = Hq // Hkv
    q = st["q"].view(B, Hkv, G * T, D).float() * (1.0 / math.sqrt(D))
    kp, vp = st["kp"][:, :case["P"]].float(), st["vp"][:, :case["P"]].float()
    shared = q.transpose(0, 1).reshape(Hkv, B * G * T, D) @ kp.transpose(1, 2)      # one product for all sequences
    key = torch.arange(S, device=q.device)
    see = st["lens"][:, None] - T + 1 + torch.arange(T, device=q.device)            # own keys each token sees
    see = see.repeat(1, G)[:, None, :, None]                                         # rows are (head in group, token)
    mine = (q @ st["k"].float().transpose(2, 3)).masked_fill_(key >= see, float("-inf"))
    m = torch.maximum(shared.amax(-1).view(Hkv, B, G * T).transpose(0, 1), mine.amax(-1))
    shared.sub_(m.transpose(0, 1).reshape(Hkv, B * G * T, 1)).exp_()
    mine.sub_(m[..., None]).exp_()
    total = shared.sum(-1).view(Hkv, B, G * T).transpose(0, 1) + mine.sum(-1)
    out = (shared @ vp).view(Hkv, B, G * T, D).transpose(0, 1) + mine @ st["v"].float()
    st["out"].view(B, Hkv, G * T, D).copy_(out / total[..., None])
    st["lse"].view(B, Hkv, G * T).copy_(m + torch.log(total))
    return {"out": st["out"], "lse": st["lse"]}


# ------------------------------------------------------------------------------ the floor and the exact values

def work(case):
    B, Hq, Hkv, D, T = (case[k] for k in ("B", "Hq", "Hkv", "D", "T"))
    L = _lengths(case)
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "norm":
        rows = B * T * (2 * Hq + 4 * Hkv)                                           # read and written
        tables = B * T * D * 4 + B * T * case["axes"] * 4
        return {"bytes": rows * D * e + tables + 2 * D * 4 + 4 * B, "flops": B * T * (Hq + Hkv) * D * 7}
    ends = B * Hq * T * (2 * D * e + 4) + 4 * B
    if case["op"] == "prefix":
        return {"bytes": (case["P"] + sum(L)) * Hkv * 2 * D * e + ends,
                "flops": (B * case["P"] + sum(L)) * Hq * T * 4 * D}
    W, C = case["window"], case["sinks"]
    keys = pairs = 0
    for n in L:
        first = n - T - W + 1                                                       # first key in the first token's window
        keys += n if first <= C else C + n - first
        pairs += sum(min(p + 1, W) + max(0, min(C, p + 1 - W)) for p in range(n - T, n))
    return {"bytes": keys * Hkv * 2 * D * e + ends, "flops": pairs * Hq * 4 * D}


def exact(case, seed):
    """From the definitions in 64 bits, one token and one group of heads at a time."""
    st = prepare(case, seed)
    lens = st["lens"].tolist()
    B, Hq, Hkv, D, T = (case[k] for k in ("B", "Hq", "Hkv", "D", "T"))
    G = Hq // Hkv
    dev = st["lens"].device
    if case["op"] == "norm":
        h = D // 2
        q, k, v = torch.empty(st["q"].shape, dtype=torch.float64, device=dev), st["k"].double(), st["v"].double()
        for b, L in enumerate(lens):
            if st["pos"] is None:
                c, s = st["cos"][L:L + T].double(), st["sin"][L:L + T].double()
            else:
                i = torch.arange(h, device=dev)
                p = torch.stack([st["pos"][b, :, a] for a in st["axis"].tolist()], dim=1).long()
                c, s = st["cos"][p, i].double(), st["sin"][p, i].double()
            z = torch.complex(c, s)
            got = []
            for x, w in ((st["q"][b].double(), st["qw"].double()), (st["k_new"][b].double(), st["kw"].double())):
                y = x / torch.sqrt(x.square().sum(-1, keepdim=True) / D + EPS) * w
                y = torch.complex(y[..., :h].contiguous(), y[..., h:].contiguous()) * z
                got.append(torch.cat([y.real, y.imag], dim=-1))
            q[b] = got[0]
            k[b, :, L:L + T] = got[1]
            v[b, :, L:L + T] = st["v_new"][b].double()
        return {"q": q, "k": k, "v": v}
    q = st["q"].double().view(B, Hkv, G, T, D)
    out = torch.empty(B, Hkv, G, T, D, dtype=torch.float64, device=dev)
    lse = torch.empty(B, Hkv, G, T, dtype=torch.float64, device=dev)
    step = max(1, min(T, 250))
    for b, L in enumerate(lens):
        k, v = st["k"][b].double(), st["v"][b].double()
        if case["op"] == "prefix":
            k = torch.cat([st["kp"][:, :case["P"]].double(), k[:, :L]], dim=1)
            v = torch.cat([st["vp"][:, :case["P"]].double(), v[:, :L]], dim=1)
            base, W, C = case["P"] + L - T, case["P"] + L, 0
        else:
            base, W, C = L - T, case["window"], case["sinks"]
        for t0 in range(0, T, step):
            t1 = min(T, t0 + step)
            # the keys that these tokens see between them: the sinks, and the window of the first to the end of the last
            a, z = max(0, base + t0 - W + 1), base + t1
            j = torch.arange(z, device=dev)
            j = j[(j < C) | (j >= a)]
            p = base + torch.arange(t0, t1, device=dev)[:, None]
            hidden = (j > p) | ((j <= p - W) & (j >= C))
            x = torch.einsum("hgtd,hjd->hgtj", q[b, :, :, t0:t1], k[:, j]) / math.sqrt(D)
            x = x.masked_fill(hidden, float("-inf"))
            lse[b, :, :, t0:t1] = torch.logsumexp(x, dim=-1)
            out[b, :, :, t0:t1] = torch.einsum("hgtj,hjd->hgtd", torch.softmax(x, dim=-1), v[:, j])
    return {"out": out.view(st["q"].shape), "lse": lse.view(st["lse"].shape)}
