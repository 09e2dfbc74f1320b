"""GPU tests of the gated delta rule and the state cache where offsets pass 32 bits: the
last sequence of a large call is compared, bit for bit, with a call on it alone (no kernel's
sums depend on what else the call holds)."""
import pytest
import torch

from helpers import has_gpu

ssd = pytest.importorskip("mamba_ssd_chunked_03_amd.ssd")
pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not has_gpu(), reason="needs a GPU")]

FIELDS = ("dq", "dk", "dv", "dg", "dbeta")


def test_training_pair_past_2_31_elements():
    """v, its gradient, the kept states (P x 32 a chunk and head) and Z: each past 2^31
    elements in front of the last sequence; v past 2^32 bytes."""
    H, G, P, N, tail = 128, 1, 128, 16, 150
    T = (1 << 31) // (H * P) + 64 + tail
    gen = torch.Generator(device="cuda").manual_seed(3)
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    unit = lambda *s: torch.nn.functional.normalize(rand(*s), dim=-1).bfloat16()  # noqa: E731
    q, k = unit(1, T, G, N), unit(1, T, G, N)
    v, dout = (torch.empty(1, T, H, P, dtype=torch.bfloat16, device="cuda").normal_(generator=gen) for _ in range(2))
    g, beta = -torch.rand(1, T, H, generator=gen, device="cuda"), torch.rand(1, T, H, generator=gen, device="cuda")
    init, d_final = rand(2, H, P, N), rand(2, H, P, N)
    cu = torch.tensor([0, T - tail, T], dtype=torch.int32, device="cuda")
    ws = torch.empty(ssd.delta_workspace_bytes(k, v, cu, backward=True), dtype=torch.uint8, device="cuda")
    assert v[:, :-tail].numel() > 1 << 31 and ws.numel() > 1 << 33
    out, final = ssd.delta_fwd(q, k, v, g, beta, init=init, cu_seqlens=cu, workspace=ws, save_for_backward=True)
    d = ssd.delta_bwd(q, k, v, g, beta, dout, init=init, d_final=d_final, cu_seqlens=cu, workspace=ws, from_saved=True)
    last = lambda x: x[:, -tail:].contiguous()  # noqa: E731
    a = tuple(last(x) for x in (q, k, v, g, beta))
    out1, final1 = ssd.delta_fwd(*a, init=init[1:])
    d1 = ssd.delta_bwd(*a, last(dout), init=init[1:], d_final=d_final[1:])
    assert torch.equal(last(out), out1) and torch.equal(final[1:], final1)
    for n in FIELDS:
        assert torch.equal(last(d[n]), d1[n]), n
    assert torch.equal(d["d_init"][1:], d1["d_init"])
    assert torch.isfinite(final).all() and torch.isfinite(d["d_init"]).all()


@pytest.mark.parametrize("fmt", ["int8", "float8_e4m3fn"])
def test_slots_past_2_31_elements(fmt):
    """A decode step on, and a cache's, last slots behind more than 2^31 values."""
    H, P, N, n = 64, 128, 128, 3
    nslots = (1 << 31) // (H * P * N) + 8
    gen = torch.Generator(device="cuda").manual_seed(4)
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    small = rand(n, H, P, N)
    slots = torch.tensor([nslots - 1, nslots - 3, nslots - 2], dtype=torch.int32, device="cuda")
    at = slots.long()
    codes = torch.empty(nslots, H, P, N, dtype=getattr(torch, fmt), device="cuda")
    scales = torch.empty(nslots, H, P, device="cuda")
    few_c, few_s = torch.empty(n, H, P, N, dtype=codes.dtype, device="cuda"), torch.empty(n, H, P, device="cuda")
    ssd.state_cache_write(small, codes, scales, slots=slots)
    ssd.state_cache_write(small, few_c, few_s)
    # (slot n of the small cache holds sequence n, the large one's slots[n])
    assert torch.equal(codes.view(torch.int8)[at], few_c.view(torch.int8)) and torch.equal(scales[at], few_s)
    got = ssd.state_cache_read(codes, scales, slots=slots)
    assert torch.equal(got, ssd.state_cache_read(few_c, few_s))
    del codes, scales
    states = torch.empty(nslots, H, P, N, device="cuda")
    assert states[:-8].numel() >= 1 << 31
    states[at] = small
    a = (rand(n, 1, 4, N).bfloat16(), rand(n, 1, 4, N).bfloat16(), rand(n, 1, H, P).bfloat16(),
         -torch.rand(n, 1, H, generator=gen, device="cuda"), torch.rand(n, 1, H, generator=gen, device="cuda"))
    out = ssd.delta_step(*a, states, slots=slots)
    alone = small.clone()
    assert torch.equal(out, ssd.delta_step(*a, alone)) and torch.equal(states[at], alone)


def test_reading_into_many_states_past_2_31_elements():
    """One slot read many times: the states written pass 2^31 values."""
    H, P, N = 8, 128, 128
    n = (1 << 31) // (H * P * N) + 3
    x = torch.randn(2, H, P, N, device="cuda")
    codes, scales = torch.empty(2, H, P, N, dtype=torch.int8, device="cuda"), torch.empty(2, H, P, device="cuda")
    ssd.state_cache_write(x, codes, scales)
    slots = (torch.arange(n, device="cuda", dtype=torch.int32) % 2).contiguous()
    got = ssd.state_cache_read(codes, scales, slots=slots)
    two = ssd.state_cache_read(codes, scales)
    assert torch.equal(got[-2:], two[(torch.arange(n - 2, n) % 2).tolist()]) and torch.equal(got[:2], two)
    many = torch.empty(n, H, P, N, dtype=torch.int8, device="cuda")
    ms = torch.empty(n, H, P, device="cuda")
    ssd.state_cache_write(got, many, ms)
    assert torch.equal(many[-1], ssd_codes(two[(n - 1) % 2]))


def ssd_codes(state):
    c, s = torch.empty(1, *state.shape, dtype=torch.int8, device="cuda"), torch.empty(1, *state.shape[:2], device="cuda")
    ssd.state_cache_write(state[None].contiguous(), c, s)
    return c[0]
