"""The tensor-core prefill and the shared-prefix attention give the same bits call after call while another stream keeps memory busy, so that
its copies land late and in ever different orders (a wait that lets a product's reader pass too early shows here)."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def td():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from decode_attention_split_gb300 import build
    build.build()
    import decode_attention_split_gb300 as td
    return td


@pytest.mark.parametrize("D,T,L,window", [(128, 700, 2047, 0), (64, 129, 1999, 0), (128, 700, 2047, 300), (64, 1, 1500, 700)])
def test_prefill_repeats_itself(td, D, T, L, window):
    g = torch.Generator(device="cuda").manual_seed(D + T)
    q = torch.randn(2, 8, T, D, generator=g, device="cuda").bfloat16()
    # keys that grow along the cache: the running maximum moves in many tiles
    ramp = torch.linspace(0.2, 2.0, L, device="cuda")[None, None, :, None]
    k = (torch.randn(2, 4, L, D, generator=g, device="cuda") * ramp).bfloat16()
    v = torch.randn(2, 4, L, D, generator=g, device="cuda").bfloat16()
    lens = torch.tensor([L, L - 5], dtype=torch.int32, device="cuda")
    a = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    b = torch.empty_like(a)

    def call():
        if window:
            return td.td_prefill_attn_window(q, k, v, lens, window, 4, return_lse=True)
        return td.td_prefill_attn(q, k, v, lens, return_lse=True)
    want = call()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = []
    for _ in range(60):
        with torch.cuda.stream(side):
            b.copy_(a)
        got.append(call())
    torch.cuda.synchronize()
    assert all(torch.equal(x, want[0]) and torch.equal(y, want[1]) for x, y in got)


@pytest.mark.parametrize("D,T,L,window", [(128, 700, 2047, 1500), (64, 257, 1999, 1200)])
def test_windowed_prefill_of_rising_scores_repeats_itself(td, D, T, L, window):
    """Scores that rise by more than the reference is let to lag (2^32) from one tile of keys to the next but one: rows are
    rescaled in most tiles."""
    g = torch.Generator(device="cuda").manual_seed(D + T)
    q = torch.ones(2, 8, T, D, device="cuda")
    q += 0.1 * torch.randn(2, 8, T, D, generator=g, device="cuda")
    ramp = 20 * torch.arange(L, device="cuda") / 64 * 0.6931 * D ** -0.5          # base 2: 20 a tile of 64 keys
    k = (ramp[None, None, :, None] + torch.randn(2, 4, L, D, generator=g, device="cuda")).bfloat16()
    q, v = q.bfloat16(), torch.randn(2, 4, L, D, generator=g, device="cuda").bfloat16()
    lens = torch.tensor([L, L - 5], dtype=torch.int32, device="cuda")
    a = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    b = torch.empty_like(a)
    want = td.td_prefill_attn_window(q, k, v, lens, window, 4, return_lse=True)
    torch.cuda.synchronize()
    assert want[0].isfinite().all()
    side = torch.cuda.Stream()
    got = []
    for _ in range(60):
        with torch.cuda.stream(side):
            b.copy_(a)
        got.append(td.td_prefill_attn_window(q, k, v, lens, window, 4, return_lse=True))
    torch.cuda.synchronize()
    assert all(torch.equal(x, want[0]) and torch.equal(y, want[1]) for x, y in got)


@pytest.mark.parametrize("D,G,T,B,P", [(128, 4, 6, 33, 2048), (64, 3, 6, 33, 1999), (128, 4, 1, 70, 2047), (64, 8, 1, 40, 300)])
def test_prefix_attention_repeats_itself(td, D, G, T, B, P):
    Hkv, S = 3, 300
    g = torch.Generator(device="cuda").manual_seed(D + T)

    def rows(*s):
        return torch.randn(*s, generator=g, device="cuda")
    q = rows(B, Hkv * G, T, D).bfloat16()
    ramp = torch.linspace(0.2, 6.0, P, device="cuda")[None, :, None]   # scores that rise by more than the lag the maximum is let
    kp, vp = (rows(Hkv, P, D) * ramp).bfloat16(), rows(Hkv, P, D).bfloat16()
    k, v = rows(B, Hkv, S, D).bfloat16(), rows(B, Hkv, S, D).bfloat16()
    lens = torch.randint(T, S + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    plen = torch.tensor([P], dtype=torch.int32, device="cuda")
    a = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    b = torch.empty_like(a)
    want = td.td_verify_attn_prefix(q, kp, vp, plen, k, v, lens, return_lse=True)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = []
    for _ in range(150):
        with torch.cuda.stream(side):
            b.copy_(a)
        got.append(td.td_verify_attn_prefix(q, kp, vp, plen, k, v, lens, return_lse=True))
    torch.cuda.synchronize()
    assert all(torch.equal(x, want[0]) and torch.equal(y, want[1]) for x, y in got)
