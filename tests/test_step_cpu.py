"""The normed append, windowed attention and shared-prefix attention without a GPU: what the C calls and
the binding refuse before any launch."""
import re

import pytest
import torch

from decode_attention_split_gb300 import api
from decode_attention_split_gb300 import build as td_build

FAKE = 0x10000  # a 16-byte aligned address the host never dereferences
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3
NAN = float("nan")


@pytest.fixture(scope="module")
def lib():
    td_build.build()
    from decode_attention_split_gb300 import _lib
    return _lib.lib()


def _call(fn, order, defaults, kw):
    a = {**defaults, **kw}
    return fn(*[a[k] for k in order])


NORM = ("dtype", "q", "qo", "Hq", "qw", "kn", "vn", "kw", "eps", "cos", "sin", "rows", "pos", "axes", "A", "kc", "vc",
        "sl", "B", "Hkv", "T", "Smax", "D", "adv", "st", "stream")


@pytest.mark.parametrize("kw,expect", [
    (dict(dtype=2), UNSUPPORTED),
    (dict(kn=None), INVALID),
    (dict(vc=None), INVALID),
    (dict(kw=None), INVALID),
    (dict(sl=None), INVALID),
    (dict(sin=None), INVALID),
    (dict(q=None), INVALID),                          # q_out without q
    (dict(qo=None), INVALID),
    (dict(qw=None), INVALID),
    (dict(Hq=0), INVALID),
    (dict(T=0), INVALID),
    (dict(B=0), INVALID),
    (dict(eps=0.0), INVALID),
    (dict(eps=-1.0), INVALID),
    (dict(eps=NAN), INVALID),
    (dict(eps=float("inf")), INVALID),
    (dict(rows=63), INVALID),                         # fewer table rows than cache rows
    (dict(axes=FAKE), INVALID),                       # axes without positions
    (dict(pos=FAKE, A=0, rows=1), INVALID),
    (dict(pos=FAKE, A=2, rows=0), INVALID),
    (dict(pos=FAKE, A=17, rows=8), UNSUPPORTED),
    (dict(pos=FAKE + 2, A=2, rows=8), UNSUPPORTED),
    (dict(D=96), UNSUPPORTED),
    (dict(D=256), UNSUPPORTED),
    (dict(B=65536), UNSUPPORTED),
    (dict(T=(1 << 20) + 1), UNSUPPORTED),
    (dict(Smax=(1 << 30) + 1, rows=(1 << 30) + 1), UNSUPPORTED),
    (dict(Hkv=4097), UNSUPPORTED),
    (dict(kn=FAKE + 8), UNSUPPORTED),
    (dict(kw=FAKE + 4), UNSUPPORTED),
    (dict(qw=FAKE + 4), UNSUPPORTED),
    (dict(cos=FAKE + 4), UNSUPPORTED),
    (dict(st=FAKE + 1), UNSUPPORTED),
])
def test_norm_append_refuses(lib, kw, expect):
    d = dict(dtype=1, q=FAKE, qo=FAKE, Hq=4, qw=FAKE, kn=FAKE, vn=FAKE, kw=FAKE, eps=1e-6, cos=FAKE, sin=FAKE, rows=64,
             pos=None, axes=None, A=0, kc=FAKE, vc=FAKE, sl=FAKE, B=2, Hkv=2, T=1, Smax=64, D=128, adv=1, st=None,
             stream=None)
    assert _call(lib.td_norm_rope_kv_append, NORM, d, kw) == expect


def rows(*s, dtype=torch.bfloat16):
    return torch.zeros(*s, dtype=dtype)


def norm_args(**kw):
    a = dict(k_new=rows(2, 2, 3, 128), v_new=rows(2, 2, 3, 128), k_cache=rows(2, 2, 64, 128),
             v_cache=rows(2, 2, 64, 128), seq_lens=torch.zeros(2, dtype=torch.int32), k_weight=torch.ones(128),
             cos_t=torch.zeros(64, 64), sin_t=torch.zeros(64, 64), q=rows(2, 4, 3, 128), q_weight=torch.ones(128))
    a.update(kw)
    return a


@pytest.mark.parametrize("kw,error", [
    (dict(v_new=rows(2, 2, 4, 128)), ValueError),
    (dict(k_cache=rows(2, 3, 64, 128), v_cache=rows(2, 3, 64, 128)), ValueError),
    (dict(k_cache=torch.zeros(2, 2, 64, 128)), TypeError),
    (dict(k_new=rows(2, 2, 3, 128, dtype=torch.float16), v_new=rows(2, 2, 3, 128, dtype=torch.float16),
          k_cache=rows(2, 2, 64, 128, dtype=torch.float16), v_cache=rows(2, 2, 64, 128, dtype=torch.float16)), TypeError),
    (dict(seq_lens=torch.zeros(2)), TypeError),
    (dict(seq_lens=torch.zeros(3, dtype=torch.int32)), TypeError),
    (dict(k_weight=rows(128)), TypeError),
    (dict(k_weight=torch.ones(64)), TypeError),
    (dict(q_weight=None), TypeError),
    (dict(q=None), ValueError),
    (dict(q=rows(2, 4, 2, 128)), ValueError),
    (dict(q_out=rows(2, 4, 2, 128)), TypeError),
    (dict(cos_t=torch.zeros(63, 64), sin_t=torch.zeros(63, 64)), TypeError),
    (dict(cos_t=torch.zeros(64, 32), sin_t=torch.zeros(64, 32)), TypeError),
    (dict(axes=torch.zeros(64, dtype=torch.int32)), ValueError),
    (dict(positions=torch.zeros(2, 3, dtype=torch.int32)), TypeError),
    (dict(positions=torch.zeros(2, 3, 2, dtype=torch.int64)), TypeError),
    (dict(positions=torch.zeros(2, 3, 2, dtype=torch.int32), axes=torch.zeros(63, dtype=torch.int32)), TypeError),
    (dict(eps="x"), TypeError),
    (dict(dev_status=torch.zeros(1)), TypeError),
    (dict(k_new=None), TypeError),
    (dict(), ValueError),                             # all in order, but not on a GPU
])
def test_norm_append_binding_refuses(lib, kw, error):
    with pytest.raises(error):
        api.td_norm_rope_kv_append(**norm_args(**kw))


WINDOW = ("dtype", "q", "k", "v", "sl", "B", "Hq", "Hkv", "T", "Smax", "D", "scale", "window", "sinks", "split", "out",
          "lse", "ws", "wsb", "st", "stream")


@pytest.mark.parametrize("kw,expect", [
    (dict(window=0), INVALID),
    (dict(window=-5), INVALID),
    (dict(sinks=-1), INVALID),
    (dict(q=None), INVALID),
    (dict(sl=None), INVALID),
    (dict(out=None), INVALID),
    (dict(Hq=5), INVALID),
    (dict(T=0), INVALID),
    (dict(split=-16), INVALID),
    (dict(scale=NAN), INVALID),
    (dict(Smax=0), INVALID),
    (dict(split=40), UNSUPPORTED),
    (dict(dtype=2), UNSUPPORTED),
    (dict(D=96), UNSUPPORTED),
    (dict(T=65), UNSUPPORTED),
    (dict(B=1025), UNSUPPORTED),
])
def test_window_attention_refuses(lib, kw, expect):
    d = dict(dtype=1, q=FAKE, k=FAKE, v=FAKE, sl=FAKE, B=2, Hq=4, Hkv=2, T=3, Smax=64, D=128, scale=1.0, window=8, sinks=2,
             split=0, out=FAKE, lse=None, ws=FAKE, wsb=1 << 24, st=None, stream=None)
    assert _call(lib.td_verify_attn_window, WINDOW, d, kw) == expect
    if "T" not in kw:
        order = tuple(k for k in WINDOW if k != "T")
        assert _call(lib.td_decode_attn_window, order, d, kw) == expect


PROMPT = ("q", "k", "v", "sl", "B", "Hq", "Hkv", "T", "Smax", "D", "scale", "window", "sinks", "out", "lse", "st", "stream")


@pytest.mark.parametrize("kw,expect", [
    (dict(window=0), INVALID),
    (dict(sinks=-1), INVALID),
    (dict(k=None), INVALID),
    (dict(Hq=5), INVALID),
    (dict(scale=NAN), INVALID),
    (dict(T=65), UNSUPPORTED),
    (dict(D=96), UNSUPPORTED),
    (dict(q=FAKE + 8), UNSUPPORTED),
    (dict(Smax=(1 << 30) + 1), UNSUPPORTED),
])
def test_window_prefill_refuses(lib, kw, expect):
    d = dict(q=FAKE, k=FAKE, v=FAKE, sl=FAKE, B=2, Hq=4, Hkv=2, T=3, Smax=64, D=128, scale=1.0, window=8, sinks=2, out=FAKE,
             lse=None, st=None, stream=None)
    assert _call(lib.td_prefill_attn_window, PROMPT, d, kw) == expect


def attn_args(decode=False, **kw):
    a = dict(q=rows(2, 4, 128) if decode else rows(2, 4, 3, 128), k_cache=rows(2, 2, 64, 128), v_cache=rows(2, 2, 64, 128),
             seq_lens=torch.zeros(2, dtype=torch.int32), window=8, sinks=2)
    a.update(kw)
    return a


BAD_ATTN = [
    (dict(q=rows(2, 4, 3, 64)), ValueError),
    (dict(q=rows(3, 4, 3, 128)), ValueError),
    (dict(q=rows(2, 4)), ValueError),
    (dict(v_cache=rows(2, 2, 65, 128)), ValueError),
    (dict(k_cache=torch.zeros(2, 2, 64, 128)), TypeError),
    (dict(seq_lens=torch.zeros(2, dtype=torch.int64)), TypeError),
    (dict(out=rows(2, 4, 2, 128)), TypeError),
    (dict(out=torch.zeros(2, 4, 3, 128)), TypeError),
    (dict(lse=torch.zeros(2, 4)), TypeError),
    (dict(lse=rows(2, 4, 3)), TypeError),
    (dict(window="8"), TypeError),
    (dict(sinks=2.5), TypeError),
    (dict(window=1 << 40), ValueError),
    (dict(), ValueError),                             # all in order, but not on a GPU
]


@pytest.mark.parametrize("kw,error", BAD_ATTN + [(dict(workspace=torch.zeros(8)), TypeError)])
def test_window_binding_refuses(lib, kw, error):
    with pytest.raises(error):
        api.td_verify_attn_window(**attn_args(**kw))


@pytest.mark.parametrize("kw,error", BAD_ATTN + [
    (dict(q=torch.zeros(2, 4, 3, 128), k_cache=torch.zeros(2, 2, 64, 128), v_cache=torch.zeros(2, 2, 64, 128)), TypeError)])
def test_window_prefill_binding_refuses(lib, kw, error):
    with pytest.raises(error):
        api.td_prefill_attn_window(**attn_args(**kw))


def test_decode_and_verify_take_their_own_queries(lib):
    with pytest.raises(ValueError):
        api.td_decode_attn_window(**attn_args())
    with pytest.raises(ValueError):
        api.td_verify_attn_window(**attn_args(decode=True))


PREFIX = ("q", "kp", "vp", "pl", "k", "v", "sl", "B", "Hq", "Hkv", "T", "Pmax", "Smax", "D", "scale", "out", "lse", "ws",
          "wsb", "st", "stream")


@pytest.mark.parametrize("kw,expect", [
    (dict(kp=None), INVALID),
    (dict(vp=None), INVALID),
    (dict(pl=None), INVALID),
    (dict(T=0), INVALID),
    (dict(Hq=5), INVALID),
    (dict(B=0), INVALID),
    (dict(Smax=0), INVALID),
    (dict(T=65), UNSUPPORTED),
    (dict(D=96), UNSUPPORTED),
    (dict(B=1025), UNSUPPORTED),
])
def test_prefix_attention_refuses(lib, kw, expect):
    d = dict(q=FAKE, kp=FAKE, vp=FAKE, pl=FAKE, k=FAKE, v=FAKE, sl=FAKE, B=2, Hq=4, Hkv=2, T=3, Pmax=100, Smax=64, D=128,
             scale=1.0, out=FAKE, lse=None, ws=FAKE, wsb=1 << 24, st=None, stream=None)
    assert _call(lib.td_verify_attn_prefix, PREFIX, d, kw) == expect
    if "T" not in kw:
        order = tuple(k for k in PREFIX if k != "T")
        assert _call(lib.td_decode_attn_prefix, order, d, kw) == expect


@pytest.mark.parametrize("kw,error", [(k, e) for k, e in BAD_ATTN if "window" not in k and "sinks" not in k] + [
    (dict(k_prefix=rows(3, 100, 128)), ValueError),
    (dict(k_prefix=rows(2, 100, 64), v_prefix=rows(2, 100, 64)), ValueError),
    (dict(v_prefix=rows(2, 99, 128)), ValueError),
    (dict(k_prefix=torch.zeros(2, 100, 128), v_prefix=torch.zeros(2, 100, 128)), TypeError),
    (dict(prefix_len=torch.zeros(1)), TypeError),
    (dict(prefix_len=torch.zeros(2, dtype=torch.int32)), TypeError),
    (dict(prefix_len=100), TypeError),
    (dict(q=torch.zeros(2, 4, 3, 128), k_cache=torch.zeros(2, 2, 64, 128), v_cache=torch.zeros(2, 2, 64, 128)), TypeError),
])
def test_prefix_binding_refuses(lib, kw, error):
    a = attn_args(k_prefix=rows(2, 100, 128), v_prefix=rows(2, 100, 128), prefix_len=torch.zeros(1, dtype=torch.int32))
    del a["window"], a["sinks"]
    a.update(kw)
    with pytest.raises(error):
        api.td_verify_attn_prefix(**a)
    if a["q"].dim() == 4:
        with pytest.raises(ValueError):
            api.td_decode_attn_prefix(**a)


def test_kernels_have_no_spills(lib):
    """Register gate (ptxas), as for the other kernels."""
    log = open(td_build.PTXAS_LOG).read()
    entries = re.findall(r"Compiling entry function '(\w+)'.*?\n(?:.*?\n)*?\s+(\d+) bytes stack frame, (\d+) bytes "
                         r"spill stores, (\d+) bytes spill loads", log)
    for k, n in (("norm_append_kernel", 4), ("norm_append_rows_kernel", 4), ("mma_kernelILi64", 10), ("mma_kernelILi128", 10),
                 ("cluster_kernelILi64", 6), ("cluster_kernelILi128", 6), ("Li1EEEvNS_11SplitParams", 6), ("14prefill_kernel", 4),
                 ("13prefix_kernel", 6), ("join_kernel", 8)):
        assert [(int(st), int(ld)) for name, _, st, ld in entries if k in name] == [(0, 0)] * n, k
