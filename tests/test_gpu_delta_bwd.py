"""GPU parity of the gated delta rule's backward with the fp64 oracle, through the C ABI.

Errors are relative 2-norms per tensor, counted as in test_gpu_delta.py: a product of the
bf16 path is off by 6e-6 of its terms (mean; 1.2e-5 at most), of the fp32 path by 1.1e-6.
A gradient comes out of ten of them in a row (four of the forward chain, four of the
backward chain, two of its own): 6e-5 and 1.1e-5 for dbeta, d_init and, fp32, dq, dk, dv.
dg sums row products over the chunk whose terms exceed it by up to 2: 1.2e-4 and 2.2e-5.
bf16 dq, dk, dv: one rounding, 2^-8 of each value at most, on top of the products' 6e-5:
4e-3."""
import numpy as np
import pytest
import torch

from delta_cases import cuda, f64, make, oracle_bwd, oracle_fwd
from helpers import has_gpu
from test_gpu_delta import CASES, OUT_TOL, STATE_TOL, rel

ssd = pytest.importorskip("mamba_ssd_chunked_03_amd.ssd")
pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not has_gpu(), reason="needs a GPU")]

TOL = {"bf16": dict(dq=4e-3, dk=4e-3, dv=4e-3, dg=1.2e-4, dbeta=6e-5, d_init=6e-5),
       "f32": dict(dq=1.1e-5, dk=1.1e-5, dv=1.1e-5, dg=2.2e-5, dbeta=1.1e-5, d_init=1.1e-5)}
NAMES = ("dq", "dk", "dv", "dg", "dbeta", "d_init")


def args(c):
    return c["q"], c["k"], c["v"], c["g"], c["beta"]


def run_bwd(d, **kw):
    c = cuda(d)
    return ssd.delta_bwd(*args(c), c["dout"], scale=d["scale"], init=c["init"], d_final=c["d_final"],
                         cu_seqlens=c["cu"], **kw)


def check(got, ref, io, names=NAMES):
    errs = {n: rel(f64(got[n]), ref[n]) for n in names}
    assert all(errs[n] <= TOL[io][n] for n in names), errs


@pytest.mark.parametrize("case", CASES, ids=str)
def test_bwd_matches_oracle(case):
    *sizes, io, lengths = case
    d = make(*sizes, io=io, lengths=lengths, seed=sum(sizes) + 1)
    check(run_bwd(d), oracle_bwd(d), io)


@pytest.mark.parametrize("P", [16, 32, 64, 128])
@pytest.mark.parametrize("N", [16, 32, 64, 128])
@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_bwd_every_size(P, N, io):
    d = make(1, 140, 2, 1, P, N, io=io, lengths=[75, 65], seed=P + N)
    check(run_bwd(d), oracle_bwd(d), io)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("gates", ["zero_beta", "resets", "strong"])
def test_bwd_gates(io, gates):
    d = make(1, 200, 4, 2, 64, 128, io=io, gates=gates, lengths=[130, 70], seed=17)
    check(run_bwd(d), oracle_bwd(d), io)


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_saved_forward_equals_recompute(io):
    d = make(1, 300, 6, 2, 64, 128, io=io, lengths=[1, 0, 170, 129], seed=18)
    c = cuda(d)
    g0 = run_bwd(d)
    ws = torch.full((ssd.delta_workspace_bytes(c["k"], c["v"], c["cu"], backward=True),), 0xFF, dtype=torch.uint8,
                    device="cuda")
    o0, S0 = ssd.delta_fwd(*args(c), scale=d["scale"], init=c["init"], cu_seqlens=c["cu"])
    o, S = ssd.delta_fwd(*args(c), scale=d["scale"], init=c["init"], cu_seqlens=c["cu"], workspace=ws,
                         save_for_backward=True)
    assert torch.equal(o, o0) and torch.equal(S, S0)
    for _ in range(2):  # the kept context is not used up
        g = run_bwd(d, workspace=ws, from_saved=True)
        for n in NAMES:
            assert torch.equal(g[n], g0[n]), n


def test_bwd_without_states():
    d = make(2, 90, 4, 2, 64, 128, init=False, d_final=False, seed=19)
    got = run_bwd(d)
    assert got["d_init"] is None
    check(got, oracle_bwd(d), "bf16", NAMES[:-1])


def test_bwd_empty():
    d = make(2, 0, 2, 1, 16, 32, seed=1)
    assert torch.equal(run_bwd(d)["d_init"].cpu(), d["d_final"])
    d = make(1, 0, 2, 1, 16, 32, lengths=[0, 0], seed=1)
    assert torch.equal(run_bwd(d)["d_init"].cpu(), d["d_final"])


def test_bwd_rows_behind_the_last_sequence_and_guard_bands():
    d = make(1, 200, 4, 2, 64, 128, lengths=[100, 50, 50], seed=20)
    short = dict(d, cu=torch.tensor([0, 100, 150], dtype=torch.int32), init=d["init"][:2], d_final=d["d_final"][:2])
    for n in ("q", "k", "v", "g", "beta", "dout"):
        short[n] = short[n].clone()
        short[n][:, 150:] = float("nan")
    pad, bufs, grads = 64, {}, {}
    for n, like in (("dq", "q"), ("dk", "k"), ("dv", "v"), ("dg", "g"), ("dbeta", "beta"), ("d_init", "init")):
        t = short[like]
        bufs[n] = torch.full((t.numel() + 2 * pad,), -7.0, dtype=t.dtype, device="cuda")
        grads[n] = bufs[n][pad:-pad].view(t.shape)
    run_bwd(short, grads=grads)
    ref = oracle_bwd(d)
    for n in NAMES:
        assert bool((bufs[n][:pad] == -7.0).all()) and bool((bufs[n][-pad:] == -7.0).all()), n
        if n == "d_init":
            assert rel(f64(grads[n]), ref[n][:2]) <= TOL["bf16"][n]
        else:
            assert bool((grads[n][:, 150:] == -7.0).all()), n
            assert rel(f64(grads[n][:, :150]), ref[n][:, :150]) <= TOL["bf16"][n], n


def test_bwd_against_differences():
    """Directional derivatives of the fp32 forward, by central differences: the forward is off by
    5e-6 of its 2-norm at most (STATE_TOL), a step h divides that into 2 h; h = 1/16 along a
    direction of the input's own size makes 5e-6 / (1/8) = 4e-5 of |loss terms| against a
    third-order remainder of h^2 / 6 = 6.5e-4 relative: tolerance 2e-3 of |dout| |o| + ..., which
    bounds the terms."""
    d = make(1, 100, 2, 1, 32, 32, io="f32", seed=21)
    got = run_bwd(d)
    gen = torch.Generator().manual_seed(5)

    def loss(dd):
        o, S = ssd.delta_fwd(*args(cuda(dd)), scale=d["scale"], init=dd["init"].cuda())
        return float((f64(o) * f64(d["dout"])).sum() + (f64(S) * f64(d["d_final"])).sum())

    o, S = oracle_fwd(d)
    size = np.linalg.norm(o) * np.linalg.norm(f64(d["dout"])) + np.linalg.norm(S) * np.linalg.norm(f64(d["d_final"]))
    for n, grad in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("g", "dg"), ("beta", "dbeta"), ("init", "d_init")):
        u = torch.randn(d[n].shape, generator=gen)
        u *= d[n].norm() / u.norm()
        h = 1.0 / 16
        diff = (loss(dict(d, **{n: d[n] + h * u})) - loss(dict(d, **{n: d[n] - h * u}))) / (2 * h)
        want = float((f64(got[grad]) * f64(u)).sum())
        assert abs(diff - want) <= 2e-3 * size, (n, diff, want)


def test_shared_heads_sum_their_gradients():
    """Groups' keys against the same keys written out per head: dq, dk are the heads' sums."""
    d = make(1, 130, 4, 1, 64, 64, io="f32", seed=22)
    wide = dict(d, q=d["q"].repeat_interleave(4, 2).contiguous(), k=d["k"].repeat_interleave(4, 2).contiguous())
    g, gw = run_bwd(d), run_bwd(wide)
    for n in ("dq", "dk"):
        assert rel(f64(g[n])[:, :, 0], f64(gw[n]).sum(2)) <= 2 * TOL["f32"][n]
    for n in ("dv", "dg", "dbeta", "d_init"):
        assert torch.equal(g[n], gw[n]), n


def test_captured_training_pair_replays():
    d = make(1, 200, 4, 2, 64, 128, lengths=[120, 80], seed=23)
    c = cuda(d)
    ws = torch.empty(ssd.delta_workspace_bytes(c["k"], c["v"], c["cu"], backward=True), dtype=torch.uint8,
                     device="cuda")
    out, final = torch.empty_like(c["v"]), torch.empty_like(c["init"])
    grads = {n: torch.empty_like(c[k]) for n, k in (("dq", "q"), ("dk", "k"), ("dv", "v"), ("dg", "g"),
                                                    ("dbeta", "beta"), ("d_init", "init"))}

    def call():
        ssd.delta_fwd(*args(c), init=c["init"], cu_seqlens=c["cu"], workspace=ws, out=out, final=final,
                      save_for_backward=True)
        ssd.delta_bwd(*args(c), c["dout"], init=c["init"], d_final=c["d_final"], cu_seqlens=c["cu"], workspace=ws,
                      from_saved=True, grads=grads)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for seed in (24, 25, 26):
        n = cuda(make(1, 200, 4, 2, 64, 128, lengths=[120, 80], seed=seed))
        for x in ("q", "k", "v", "g", "beta", "init", "dout", "d_final"):
            c[x].copy_(n[x])
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (out, final, *grads.values())]
        ws.fill_(0xFF)
        call()
        torch.cuda.synchronize()
        for a, b in zip(got, (out, final, *grads.values())):
            assert torch.equal(a, b)


def test_layer_run_with_the_gated_norm():
    """The operators as a layer uses them: delta rule, then the framework's gated RMSNorm on its
    output, and both backwards; against the two oracles chained.  The norm's own tolerances
    (4e-3 forward, 1e-2 backward, normwise) on top of the delta rule's."""
    from oracle import norm as onorm
    d = make(1, 150, 8, 2, 64, 128, seed=27)
    c = cuda(d)
    gen = torch.Generator().manual_seed(1)
    z = torch.randn(1, 150, 512, generator=gen).bfloat16()
    wt = torch.rand(512, generator=gen) + 0.5
    dn = torch.randn(1, 150, 512, generator=gen).bfloat16()
    ws = torch.empty(ssd.delta_workspace_bytes(c["k"], c["v"], backward=True), dtype=torch.uint8, device="cuda")
    o, S = ssd.delta_fwd(*args(c), init=c["init"], workspace=ws, save_for_backward=True)
    y = ssd.gated_rmsnorm_fwd(o.view(1, 150, 512), z.cuda(), wt.cuda(), 512)
    dy, dz, dwt = ssd.gated_rmsnorm_bwd(dn.cuda(), o.view(1, 150, 512), z.cuda(), wt.cuda(), 512)
    g = ssd.delta_bwd(*args(c), dy.view_as(o), init=c["init"], d_final=c["d_final"], workspace=ws, from_saved=True)
    ro, _ = oracle_fwd(d)
    ry, _ = onorm.fwd(ro.reshape(150, 512), f64(z)[0], f64(wt), 512, 1e-5)
    assert rel(f64(y)[0], ry) <= OUT_TOL["bf16"] + 4e-3
    rdy, _, _ = onorm.bwd(f64(dn)[0], ro.reshape(150, 512), f64(z)[0], f64(wt), 512, 1e-5)
    ref = oracle_bwd(dict(d, dout=torch.from_numpy(rdy).view(1, 150, 8, 64)))
    for n in NAMES:
        assert rel(f64(g[n]), ref[n]) <= OUT_TOL["bf16"] + 1e-2 + TOL["bf16"][n], n


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_first_gates_without_a_state_have_no_gradient(io):
    """A sequence's first gate decays its initial state alone: without one its gradient is zero,
    not what rounding leaves of sums that cancel."""
    lengths = [1, 70, 1, 0, 130]
    d = make(1, sum(lengths), 4, 2, 32, 64, io=io, lengths=lengths, init=False, seed=11)
    c = cuda(d)
    got = ssd.delta_bwd(c["q"], c["k"], c["v"], c["g"], c["beta"], c["dout"], scale=d["scale"], cu_seqlens=c["cu"],
                        d_final=c["d_final"])
    first = [0, 1, 71, 72]
    assert (got["dg"][0, first] == 0).all()
    assert (got["dg"][0, 2:71].abs().amax(0) > 0).all()


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_gradients_of_many_sequences_are_those_of_each(io):
    """Few chunks and groups give each head a workgroup, many do not: the same bits."""
    B = 26
    d = make(B, 130, 6, 2, 32, 64, io=io, seed=12)
    c = cuda(d)
    whole = run_bwd(d)
    for b in (0, 7, B - 1):
        one = ssd.delta_bwd(*(x[b:b + 1] for x in args(c)), c["dout"][b:b + 1], scale=d["scale"],
                            init=c["init"][b:b + 1], d_final=c["d_final"][b:b + 1])
        for n in NAMES:
            assert torch.equal(one[n], whole[n][b:b + 1]), (b, n)


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_gates_of_a_few_tokens(io):
    """dg of short sequences with an initial state, sums that can cancel: the error is held against
    the terms' absolute values, of which <|init|, |d_final|> for every token is a part.  A product
    is off by at most 3 x 2^-18 of its terms with bf16 io (two planes an operand), by 2^-26 and
    fp32 sums of at most 128 + 64 terms (2^-20 together) with fp32 io; <S, dS> by fp32 rounding."""
    lengths = [1, 2, 3, 1, 4]
    d = make(1, sum(lengths), 2, 1, 32, 32, io=io, lengths=lengths, seed=21)
    got, ref = f64(run_bwd(d)["dg"]), oracle_bwd(d)["dg"]
    init, dfin = f64(d["init"]), f64(d["d_final"])
    terms = np.sqrt(sum(l * (np.abs(init[s]) * np.abs(dfin[s])).sum((-1, -2)) ** 2 for s, l in enumerate(lengths)).sum())
    assert np.linalg.norm(got - ref) <= (3 * 2.0 ** -18 if io == "bf16" else 2.0 ** -20) * terms


@pytest.mark.parametrize("sizes", [(24, 130, 16, 4, 64, 128), (40, 70, 32, 4, 128, 64), (30, 200, 12, 4, 32, 16)], ids=str)
def test_large_batches_are_their_sequences(sizes):
    """Two tiles of headdim a workgroup of the chains, several heads a wave of the chunk matrices
    (a group's three or four, and two) and a group's heads in one workgroup of the gradients
    give the bits of the forms that one sequence takes."""
    d = make(*sizes, io="bf16", seed=sum(sizes))
    c = cuda(d)
    ws = torch.empty(ssd.delta_workspace_bytes(c["k"], c["v"], backward=True), dtype=torch.uint8, device="cuda")
    out, final = ssd.delta_fwd(*args(c), scale=d["scale"], init=c["init"], workspace=ws, save_for_backward=True)
    whole = run_bwd(d, workspace=ws, from_saved=True)
    for b in (0, sizes[0] // 2, sizes[0] - 1):
        a, init, dfin = [x[b:b + 1] for x in args(c)], c["init"][b:b + 1], c["d_final"][b:b + 1]
        o1, f1 = ssd.delta_fwd(*a, scale=d["scale"], init=init)
        one = ssd.delta_bwd(*a, c["dout"][b:b + 1], scale=d["scale"], init=init, d_final=dfin)
        assert torch.equal(out[b:b + 1], o1) and torch.equal(final[b:b + 1], f1)
        for n in NAMES:
            assert torch.equal(one[n], whole[n][b:b + 1]), (b, n)
