"""The tensor-core prefill gives the same bits call after call while another stream keeps memory busy, so that
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
