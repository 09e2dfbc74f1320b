"""GPU parity of the 8-bit state cache (through the C ABI) with the fp64 oracle.

Codes, scales and what is read back are decided exactly: a code is the nearest of x / scale
(ties to even), the scale one rounded division (int8) or a power of two (e4m3), and a value
read back is one rounded product (exact for e4m3).  So everything is compared for equality,
against the oracle's values rounded to fp32 once."""
import numpy as np
import pytest
import torch

from delta_cases import cuda, f64, make, oracle_fwd
from helpers import has_gpu
from oracle import delta

ssd = pytest.importorskip("mamba_ssd_chunked_03_amd.ssd")
pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not has_gpu(), reason="needs a GPU")]

DTYPE = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}


def cache(nslots, H, P, N, fmt):
    codes = torch.full((nslots, H, P, N), 1, dtype=torch.int8, device="cuda").view(DTYPE[fmt])
    return codes, torch.full((nslots, H, P), 3.0, device="cuda")


def values(shape, seed):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(*shape, generator=gen) * torch.exp(3 * torch.randn(*shape[:-1], 1, generator=gen))
    x[0, 0, 0] = 0.0
    x[0, 0, 1] = 1e-30 * torch.randn(shape[-1], generator=gen)
    x[0, 0, 2, 1:] = 0.0
    # values on borders between codes: halves of the scale's multiples (scale 1: max 127)
    x[0, 0, 3] = (torch.randint(-254, 255, (shape[-1],), generator=gen) / 2).float()
    x[0, 0, 3, 0] = 127.0
    return x


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("shape", [(1, 1, 16, 16), (3, 2, 32, 32), (2, 5, 64, 64), (4, 8, 64, 128), (1, 3, 128, 128)])
def test_write_and_read(fmt, shape):
    n = shape[0]
    x = values(shape, sum(shape))
    codes, scales = cache(n + 3, *shape[1:], fmt)
    slots = torch.randperm(n + 3, generator=torch.Generator().manual_seed(1))[:n].to(torch.int32)
    ssd.state_cache_write(x.cuda(), codes, scales, slots=slots.cuda())
    back, ref_scale = delta.quantise(f64(x), fmt)
    at = slots.long().cuda()
    assert np.array_equal(f64(scales[at]), ref_scale)
    got = ssd.state_cache_read(codes, scales, slots=slots.cuda())
    assert np.array_equal(f64(got), back.astype(np.float32).astype(np.float64))
    rest = [i for i in range(n + 3) if i not in slots.tolist()]  # other slots as they were
    assert bool((codes[rest].view(torch.int8) == 1).all()) and bool((scales[rest] == 3.0).all())


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_error_bounds(fmt):
    x = values((2, 4, 64, 128), 5)
    codes, scales = cache(2, 4, 64, 128, fmt)
    ssd.state_cache_write(x.cuda(), codes, scales)
    got, s = f64(ssd.state_cache_read(codes, scales)), f64(scales)[..., None]
    err = np.abs(got - f64(x))
    bound = s / 2 if fmt == "int8" else np.maximum(2.0 ** -4 * np.abs(f64(x)), 2.0 ** -10 * s)
    assert (err <= bound + 2.0 ** -24 * np.abs(got)).all()


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_slots_outside_and_twice(fmt):
    x = values((6, 2, 16, 32), 7)
    slots = torch.tensor([2, -1, 2, 4, 0, -(2**31)], dtype=torch.int32)
    codes, scales = cache(4, 2, 16, 32, fmt)
    ssd.state_cache_write(x.cuda(), codes, scales, slots=slots.cuda())  # writes slots 2 (sequence 0) and 0
    back, _ = delta.quantise(f64(x), fmt)
    got = f64(ssd.state_cache_read(codes, scales, slots=slots.cuda()))
    want = back.astype(np.float32).astype(np.float64)
    assert np.array_equal(got[[0, 2, 4]], want[[0, 0, 4]])
    assert not got[[1, 3, 5]].any()  # outside: zeros
    assert bool((scales[[1, 3]] == 3.0).all())


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_bad_rows_stay_visible(fmt):
    x = values((1, 2, 16, 64), 9)
    x[0, 1, 3, 5] = float("inf")
    x[0, 1, 4, 6] = float("nan")
    codes, scales = cache(1, 2, 16, 64, fmt)
    ssd.state_cache_write(x.cuda(), codes, scales)
    got = ssd.state_cache_read(codes, scales).cpu()
    assert bool(torch.isnan(got[0, 1, 3:5]).all())
    keep = torch.ones(1, 2, 16, dtype=torch.bool)
    keep[0, 1, 3:5] = False
    x[~keep] = 0.0
    back, _ = delta.quantise(f64(x), fmt)
    assert np.array_equal(f64(got[keep]), back[keep.numpy()].astype(np.float32).astype(np.float64))


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_park_and_resume(fmt):
    """The operators together: a prompt's final states are parked, taken up as the initial states
    of the rest of the sequence (chunked), then as the states of a decode step.  The oracle runs
    on the same rounded states, so the tolerances are those of the delta rule alone
    (test_gpu_delta.py): 2-norm 2e-5 for states of bf16 inputs, 1e-5 more for the step."""
    d = make(2, 200, 4, 2, 64, 128, seed=10)
    part = lambda a, b: {n: d[n][:, a:b].contiguous() for n in ("q", "k", "v", "g", "beta")}  # noqa: E731
    one = cuda(dict(d, **part(0, 100)))
    args = lambda c: (c["q"], c["k"], c["v"], c["g"], c["beta"])  # noqa: E731
    _, S = ssd.delta_fwd(*args(one), init=one["init"])
    codes, scales = cache(5, 4, 64, 128, fmt)
    slots = torch.tensor([4, 1], dtype=torch.int32, device="cuda")
    ssd.state_cache_write(S, codes, scales, slots=slots)
    S1 = ssd.state_cache_read(codes, scales, slots=slots)
    parked, _ = delta.quantise(f64(S), fmt)
    assert np.array_equal(f64(S1), parked.astype(np.float32).astype(np.float64))
    two = cuda(dict(d, **part(100, 199)))
    o2, S2 = ssd.delta_fwd(*args(two), init=S1)
    o3 = ssd.delta_step(*args(cuda(part(199, 200))), S2)
    ro, rS = oracle_fwd(dict(d, init=S1, **part(100, 200)))
    norm = np.linalg.norm
    assert norm(f64(S2) - rS) / norm(rS) <= 2e-5 + 1e-5
    assert norm(f64(o2) - ro[:, :99]) / norm(ro) <= 6.8e-3 and norm(f64(o3) - ro[:, 99:]) / norm(ro[:, 99:]) <= 6.8e-3


def test_scan_states_park_too():
    """ssd_fwd's final states have the same layout and are parked the same way."""
    from mamba_ssd_chunked_03_amd import inputs
    from helpers import gpu_fwd
    inp = inputs.make_inputs(2, 100, 4, 64, 128, 2, io="bf16", init="randn", seed=3)
    _, S = gpu_fwd(ssd, inp, 64)
    codes, scales = cache(2, 4, 64, 128, "int8")
    ssd.state_cache_write(S, codes, scales)
    back, _ = delta.quantise(f64(S), "int8")
    assert np.array_equal(f64(ssd.state_cache_read(codes, scales)), back.astype(np.float32).astype(np.float64))
