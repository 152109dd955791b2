"""The block-scaled 8-bit cache without a GPU: what the C calls and the binding refuse before any
launch, and the plain reference against itself."""
import ctypes
import inspect
import re

import numpy as np
import pytest
import torch

import f8_ref
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


CACHE = dict(kc=FAKE, ks=FAKE, vc=FAKE, vs=FAKE, sl=FAKE, B=2, Hkv=2, Smax=64, D=128, block=32, st=None, stream=None)
APPEND = ("dtype", "kn", "vn", "kc", "ks", "vc", "vs", "sl", "B", "Hkv", "T", "Smax", "D", "block", "adv", "st", "stream")


@pytest.mark.parametrize("kw,expect", [
    (dict(dtype=2), UNSUPPORTED),
    (dict(kn=None), INVALID),
    (dict(vs=None), INVALID),
    (dict(sl=None), INVALID),
    (dict(T=0), INVALID),
    (dict(B=0), INVALID),
    (dict(T=(1 << 30) + 1), UNSUPPORTED),
    (dict(Smax=(1 << 30) + 1), UNSUPPORTED),
    (dict(D=96), UNSUPPORTED),
    (dict(block=8), UNSUPPORTED),
    (dict(block=48), UNSUPPORTED),
    (dict(block=256), UNSUPPORTED),
    (dict(block=-16), UNSUPPORTED),
    (dict(B=65536), UNSUPPORTED),
    (dict(Hkv=16385), UNSUPPORTED),
    (dict(kc=FAKE + 8), UNSUPPORTED),
    (dict(vn=FAKE + 4), UNSUPPORTED),
    (dict(ks=FAKE + 2), UNSUPPORTED),
    (dict(st=FAKE + 1), UNSUPPORTED),
])
def test_append_refuses(lib, kw, expect):
    d = dict(CACHE, dtype=1, kn=FAKE, vn=FAKE, T=1, adv=1)
    assert _call(lib.td_kv_append_f8, APPEND, d, kw) == expect


ROPE = ("dtype", "q", "qo", "Hq", "kn", "vn", "cos", "sin", "rows", "pos", "axes", "A", "kc", "ks", "vc", "vs", "sl", "B",
        "Hkv", "T", "Smax", "D", "block", "adv", "st", "stream")


@pytest.mark.parametrize("kw,expect", [
    (dict(cos=None), INVALID),
    (dict(sin=None), INVALID),
    (dict(q=FAKE), INVALID),                          # q without q_out
    (dict(q=FAKE, qo=FAKE, Hq=0), INVALID),
    (dict(rows=63), INVALID),                         # fewer table rows than cache rows
    (dict(axes=FAKE), INVALID),                       # axes without positions
    (dict(pos=FAKE, A=0, rows=1), INVALID),
    (dict(pos=FAKE, A=3, rows=0), INVALID),
    (dict(pos=FAKE, A=17, rows=8), UNSUPPORTED),
    (dict(pos=FAKE + 2, A=3, rows=8), UNSUPPORTED),
    (dict(cos=FAKE + 4), UNSUPPORTED),
    (dict(q=FAKE, qo=FAKE + 8, Hq=2), UNSUPPORTED),
    (dict(block=0), UNSUPPORTED),
    (dict(D=80), UNSUPPORTED),
])
def test_rope_append_refuses(lib, kw, expect):
    d = dict(CACHE, dtype=1, q=None, qo=None, Hq=0, kn=FAKE, vn=FAKE, cos=FAKE, sin=FAKE, rows=64, pos=None, axes=None,
             A=0, T=1, adv=1)
    assert _call(lib.td_rope_kv_append_f8, ROPE, d, kw) == expect


READ = ("dtype", "kc", "ks", "vc", "vs", "sl", "start", "B", "Hkv", "N", "Smax", "D", "block", "ko", "vo", "st", "stream")


@pytest.mark.parametrize("kw,expect", [
    (dict(dtype=5), UNSUPPORTED),
    (dict(ko=None), INVALID),
    (dict(ks=None), INVALID),
    (dict(N=0), INVALID),
    (dict(block=24), UNSUPPORTED),
    (dict(D=32), UNSUPPORTED),
    (dict(vo=FAKE + 8), UNSUPPORTED),
    (dict(start=FAKE + 2), UNSUPPORTED),
    (dict(N=(1 << 30) + 1), UNSUPPORTED),
])
def test_read_refuses(lib, kw, expect):
    d = dict(CACHE, dtype=1, start=None, N=8, ko=FAKE, vo=FAKE)
    assert _call(lib.td_kv_read_f8, READ, d, kw) == expect


VERIFY = ("q", "kc", "ks", "vc", "vs", "sl", "B", "Hq", "Hkv", "T", "Smax", "D", "block", "scale", "split", "out", "lse",
          "ws", "wsb", "st", "stream")


@pytest.mark.parametrize("kw,expect", [
    (dict(q=None), INVALID),
    (dict(vs=None), INVALID),
    (dict(Hq=5), INVALID),
    (dict(split=-16), INVALID),
    (dict(scale=NAN), INVALID),
    (dict(split=40), UNSUPPORTED),                    # chunks start at multiples of 16 rows
    (dict(block=8), UNSUPPORTED),
    (dict(D=96), UNSUPPORTED),
    (dict(T=65), UNSUPPORTED),
    (dict(B=1025), UNSUPPORTED),
    (dict(ks=FAKE + 2), UNSUPPORTED),
])
def test_attention_refuses(lib, kw, expect):
    d = dict(CACHE, q=FAKE, Hq=4, T=1, scale=0.1, split=0, out=FAKE, lse=None, ws=FAKE, wsb=1 << 20)
    assert _call(lib.td_verify_attn_f8, VERIFY, d, kw) == expect
    if "T" not in kw:  # the decode entry point is the verify call with T = 1
        assert _call(lib.td_decode_attn_f8, tuple(k for k in VERIFY if k != "T"), d, kw) == expect


def _args():
    codes = torch.zeros(1, 2, 32, 64, dtype=torch.uint8).view(torch.float8_e4m3fn)
    return dict(k_codes=codes, k_scales=torch.zeros(1, 2, 2), v_codes=codes.clone(), v_scales=torch.zeros(1, 2, 2),
                seq_lens=torch.zeros(1, dtype=torch.int32), block=16)


def _calls():
    """The four calls with arguments that a GPU's tensors would pass."""
    x, t, q = torch.zeros(1, 2, 1, 64), torch.zeros(32, 32), torch.zeros(1, 4, 64, dtype=torch.bfloat16)
    return {
        "append": (api.td_kv_append_f8, dict(k_new=x, v_new=x.clone())),
        "rope": (api.td_rope_kv_append_f8, dict(k_new=x, v_new=x.clone(), cos_t=t, sin_t=t.clone())),
        "read": (api.td_kv_read_f8, dict()),
        "decode": (api.td_decode_attn_f8, dict(q=q)),
        "verify": (api.td_verify_attn_f8, dict(q=q[:, :, None])),
    }


@pytest.mark.parametrize("name", ["append", "rope", "read", "decode", "verify"])
def test_binding_refuses_cpu_tensors(name):
    """Shapes and types are checked first: what is left to refuse is the device."""
    fn, own = _calls()[name]
    with pytest.raises(ValueError, match="CUDA"):
        fn(**own, **_args())


@pytest.mark.parametrize("change", [
    dict(block=48), dict(block=32), dict(block=16.0), dict(block=None),
    dict(k_scales=torch.zeros(1, 2, 3)), dict(v_scales=torch.zeros(1, 2, 1)), dict(k_scales=torch.zeros(1, 2, 2).double()),
    dict(k_codes=torch.zeros(1, 2, 32, 64, dtype=torch.int8)), dict(k_codes=None), dict(k_codes=[1.0]),
    dict(seq_lens=torch.zeros(1, dtype=torch.int64)), dict(seq_lens=torch.zeros(2, dtype=torch.int32)),
    dict(v_codes=torch.zeros(1, 2, 16, 64, dtype=torch.float8_e4m3fn)),
    dict(k_codes=torch.zeros(2, 32, 64, dtype=torch.float8_e4m3fn)),
    dict(dev_status=torch.zeros(1)), dict(dev_status=torch.zeros(0, dtype=torch.int32)),
])
@pytest.mark.parametrize("name", ["append", "rope", "read", "decode", "verify"])
def test_binding_checks_the_cache(name, change):
    fn, own = _calls()[name]
    with pytest.raises((TypeError, ValueError)) as e:
        fn(**own, **{**_args(), **change})
    assert "CUDA" not in str(e.value)


@pytest.mark.parametrize("name,change", [
    ("append", dict(v_new=torch.zeros(1, 2, 1, 64).bfloat16())),
    ("append", dict(k_new=torch.zeros(1, 1, 1, 64), v_new=torch.zeros(1, 1, 1, 64))),
    ("append", dict(k_new=torch.zeros(1, 2, 64), v_new=torch.zeros(1, 2, 64))),
    ("append", dict(k_new=torch.zeros(1, 2, 1, 64).half(), v_new=torch.zeros(1, 2, 1, 64).half())),
    ("rope", dict(cos_t=torch.zeros(31, 32), sin_t=torch.zeros(31, 32))),
    ("rope", dict(sin_t=torch.zeros(32, 16))),
    ("rope", dict(axes=torch.zeros(32, dtype=torch.int32))),
    ("rope", dict(positions=torch.zeros(1, 1, 3))),
    ("rope", dict(positions=torch.zeros(1, 2, 3, dtype=torch.int32))),
    ("rope", dict(positions=torch.zeros(1, 1, 3, dtype=torch.int32), axes=torch.zeros(31, dtype=torch.int32))),
    ("rope", dict(q=torch.zeros(1, 4, 1, 64).bfloat16())),
    ("rope", dict(q=torch.zeros(1, 4, 2, 64))),
    ("rope", dict(q_out=torch.zeros(1, 4, 1, 64))),
    ("rope", dict(q=torch.zeros(1, 4, 1, 64), q_out=torch.zeros(1, 5, 1, 64))),
    ("read", dict(k_out=torch.zeros(1, 2, 5, 64))),
    ("read", dict(k_out=torch.zeros(1, 2, 5, 64), v_out=torch.zeros(1, 2, 6, 64))),
    ("read", dict(k_out=torch.zeros(1, 2, 5, 64), v_out=torch.zeros(1, 2, 5, 64), rows=6)),
    ("read", dict(rows=0)),
    ("read", dict(dtype=torch.float16)),
    ("read", dict(dtype=None)),
    ("read", dict(start=torch.zeros(1, dtype=torch.int64))),
    ("decode", dict(q=torch.zeros(1, 4, 64))),
    ("decode", dict(q=torch.zeros(2, 4, 64, dtype=torch.bfloat16))),
    ("decode", dict(q=torch.zeros(1, 4, 32, dtype=torch.bfloat16))),
    ("decode", dict(q=torch.zeros(1, 4, 1, 64, dtype=torch.bfloat16))),
    ("decode", dict(out=torch.zeros(1, 4, 64))),
    ("decode", dict(lse=torch.zeros(1, 3))),
    ("decode", dict(workspace=torch.zeros(64))),
    ("decode", dict(scale="x")),
    ("decode", dict(split=1 << 40)),
    ("verify", dict(q=torch.zeros(1, 4, 64, dtype=torch.bfloat16))),
])
def test_binding_checks_the_rest(name, change):
    fn, own = _calls()[name]
    with pytest.raises((TypeError, ValueError)) as e:
        fn(**{**own, **_args(), **change})
    assert "CUDA" not in str(e.value)


@pytest.mark.parametrize("args", [(0, 4, 2, 64, 128, 1, 0), (1, 5, 2, 64, 128, 1, 0), (1, 4, 2, 64, 96, 1, 0),
                                  (1, 4, 2, 64, 128, 65, 0), (1, 4, 2, 64, 128, 1, -1), (1025, 4, 2, 64, 128, 1, 0)])
def test_workspace_of_refused_shapes(lib, args):
    assert lib.td_f8_workspace_bytes(*args) == 0


def test_binding_names_stand_in_the_package():
    import decode_attention_split_gb300 as td
    for n in ("td_kv_append_f8", "td_rope_kv_append_f8", "td_kv_read_f8", "td_decode_attn_f8", "td_verify_attn_f8",
              "make_f8_cache"):
        assert inspect.getdoc(getattr(td, n))


def test_make_f8_cache_shapes():
    kc, ks, vc, vs = api.make_f8_cache(2, 3, 100, 64, 32, device="cpu")
    assert kc.shape == vc.shape == (2, 3, 100, 64) and kc.dtype == torch.float8_e4m3fn
    assert ks.shape == vs.shape == (2, 3, 4) and ks.dtype == torch.float32
    with pytest.raises(ValueError):
        api.make_f8_cache(2, 3, 100, 64, 20, device="cpu")


def test_library_is_installed_though_the_binding_fails(monkeypatch, tmp_path):
    """libtd.so needs neither Python's nor torch's headers: a binding that does not compile raises with
    the library in place, and no earlier library's binding is left beside it."""
    (tmp_path / "td_one.cu").write_text('extern "C" int td_one(void) { return 41; }\n')
    (tmp_path / "binding.cpp").write_text("#include <no_such_header.h>\n")
    out = tmp_path / "_build"
    out.mkdir()
    (out / "_td_torch.so").write_bytes(b"an earlier one")
    for name, at in dict(CSRC=tmp_path, BUILD=out, LIB=out / "libtd.so", BINDING=out / "_td_torch.so",
                         BINDING_SRC=tmp_path / "binding.cpp", PTXAS_LOG=out / "ptxas.log").items():
        monkeypatch.setattr(td_build, name, str(at))
    with pytest.raises(RuntimeError, match="no_such_header"):
        td_build.build(force=True)
    assert ctypes.CDLL(str(out / "libtd.so")).td_one() == 41
    assert sorted(p.name for p in out.iterdir()) == ["libtd.so", "ptxas.log"]
    assert not td_build.up_to_date()


def test_f8_kernels_have_no_spills(lib):
    """Register gate (ptxas), as for the other kernels."""
    log = open(td_build.PTXAS_LOG).read()
    entries = re.findall(r"Compiling entry function '(\w+)'.*?\n(?:.*?\n)*?\s+(\d+) bytes stack frame, (\d+) bytes "
                         r"spill stores, (\d+) bytes spill loads", log)
    seen = [n for n, _, st, ld in entries if re.search(r"_f8_|_f8E|merge_f8", n) and (int(st), int(ld)) == (0, 0)]
    for k, n in (("split_attn_f8_kernel", 6), ("merge_f8_kernel", 2), ("read_f8_kernel", 4), ("append_f8_tiles_kernel", 8)):
        assert sum(k in x for x in seen) == n, k


def test_f8_row_kernels_have_no_spills(lib):
    """The same gate for the token append, whose CTAs of 1024 threads leave it 64 registers, and the
    launch that advances the lengths."""
    log = open(td_build.PTXAS_LOG).read()
    entries = re.findall(r"Compiling entry function '(\w+)'.*?\n(?:.*?\n)*?\s+(\d+) bytes stack frame, (\d+) bytes "
                         r"spill stores, (\d+) bytes spill loads", log)
    for k, n in (("append_f8_rows_kernel", 8), ("advance_f8_kernel", 1)):
        assert [(int(st), int(ld)) for name, _, st, ld in entries if k in name] == [(0, 0)] * n, k


def test_reference_codes_agree_with_torch():
    """encode and VALUE against torch's e4m3 conversions, ties and the least values included."""
    x = np.concatenate([f8_ref.VALUE[:127], f8_ref._MID, -f8_ref._MID, np.linspace(-460, 460, 4001),
                        np.random.default_rng(0).normal(size=4000) * 2.0 ** np.random.default_rng(1).integers(-14, 9, 4000)])
    x = np.clip(x, -448, 448).astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(f8_ref.encode(x), want)
    got = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(got, f8_ref.VALUE, equal_nan=True)


def test_reference_scale_is_the_least():
    rng = np.random.default_rng(2)
    for a in np.concatenate([448 * 2.0 ** np.arange(-130, 100, 7), np.nextafter(448 * 2.0 ** np.arange(-100, 100, 9), np.inf),
                             np.exp(rng.uniform(-80, 80, 200))]):
        s = f8_ref.pow2_scale(a)
        assert a <= 448 * s and (s == 2.0 ** -126 or a > 448 * s / 2)


def test_reference_append_in_pieces():
    """Appending token by token or at once stores the same block but for codes rounded below 2^-6
    of a scale that grew afterwards, and both read back within half a step of what was written."""
    rng = np.random.default_rng(3)
    x = rng.normal(size=(1, 2, 40, 64)) * np.exp(rng.normal(size=(1, 2, 40, 1)))
    x = x.astype(np.float32).astype(np.float64)
    one, many = [(np.zeros((1, 2, 64, 64), np.uint8), np.zeros((1, 2, 4), np.float32)) for _ in range(2)]
    f8_ref.append(*one, x, [5], 16)
    for t in range(40):
        f8_ref.append(*many, x[:, :, t:t + 1], [5 + t], 16)
    assert np.array_equal(one[1][:, :, :3], many[1][:, :, :3])
    for codes, scales in (one, many):
        v = f8_ref.values(codes, scales, 16)[:, :, 5:45]
        s = np.repeat(scales, 16, axis=2)[:, :, 5:45, None]
        # half a step: 2^-4 of the value, at least half of 2^-9 scales; below 2^-6 scales a piecewise
        # append rounds again at each growth (at most half a step each, halving towards the past)
        assert np.all(np.abs(v - x) <= 2.0 ** -4 * np.abs(x) + 2.0 ** -9 * s)
