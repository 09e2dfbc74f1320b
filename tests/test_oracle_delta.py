"""Pins of the delta rule's oracle (CPU): a hand-worked case, the projection property, an
independent autograd of the same recurrence, finite differences, packed against separate
sequences; and of the state cache's rounding."""
import math

import numpy as np
import pytest
import torch

from delta_cases import f64, make, oracle_bwd, oracle_fwd
from oracle import delta


def test_hand_worked():
    # one head, P = 1, N = 2: S = [1, 2], exp(g) = 1/2, k = [1, 0], v = 3, beta = 1/4, q = [2, 1]
    # D = [1/2, 1], r = 3 - 1/2 = 5/2, S = [1/2 + 5/8, 1] = [9/8, 1], o = 2 (9/4 + 1) = 13/2
    a = lambda *x: np.array(x, dtype=float)  # noqa: E731
    o, S = delta.fwd(a(2, 1).reshape(1, 1, 1, 2), a(1, 0).reshape(1, 1, 1, 2), a(3).reshape(1, 1, 1, 1),
                     a(math.log(0.5)).reshape(1, 1, 1), a(0.25).reshape(1, 1, 1), 2.0, a(1, 2).reshape(1, 1, 1, 2))
    assert np.allclose(o, 6.5) and np.allclose(S, [[[[9 / 8, 1]]]])


def test_beta_one_unit_key_reads_back_the_value():
    d = make(1, 5, 4, 2, 8, 16, io="f32", gates="ones", seed=1)
    d["q"] = d["k"].clone()
    o, _ = oracle_fwd(d)  # after the write S_t k_t = v_t
    assert np.allclose(o / d["scale"], f64(d["v"]), atol=1e-6)


@pytest.mark.parametrize("gates", ["usual", "zero_beta"])
def test_gradients_against_autograd(gates):
    d = make(1, 9, 4, 2, 3, 5, io="f32", lengths=[4, 0, 1, 4], gates=gates, seed=2)
    names = ("q", "k", "v", "g", "beta", "init")
    leaf = {n: d[n].double().requires_grad_() for n in names}
    cu = d["cu"].tolist()
    loss = 0.0
    for s in range(4):
        S = leaf["init"][s]
        for t in range(cu[s], cu[s + 1]):
            k, q = leaf["k"][0, t].repeat_interleave(2, 0), leaf["q"][0, t].repeat_interleave(2, 0)
            S = S * leaf["g"][0, t].exp()[:, None, None]
            u = leaf["beta"][0, t][:, None] * (leaf["v"][0, t] - torch.einsum("hpn,hn->hp", S, k))
            S = S + torch.einsum("hp,hn->hpn", u, k)
            loss = loss + (d["dout"][0, t].double() * d["scale"] * torch.einsum("hpn,hn->hp", S, q)).sum()
        loss = loss + (d["d_final"][s].double() * S).sum()
    loss.backward()
    ref = oracle_bwd(d)
    for n in names:
        got = ref["d_init" if n == "init" else "d" + n]
        assert np.allclose(got, leaf[n].grad.numpy(), rtol=1e-10, atol=1e-12), n


def test_gradients_against_differences():
    d = make(1, 6, 2, 1, 3, 4, io="f32", seed=3)
    ref = oracle_bwd(d)

    def loss(dd):
        o, S = oracle_fwd(dd)
        return (o * f64(d["dout"])).sum() + (S * f64(d["d_final"])).sum()

    rng = np.random.default_rng(0)
    for n in ("q", "k", "v", "g", "beta", "init"):
        # along a random direction, central differences: error O(h^2) = 1e-10 of third derivatives
        x = d[n].double()
        u = torch.from_numpy(rng.standard_normal(tuple(x.shape)))
        h = 1e-5
        diff = (loss(dict(d, **{n: x + h * u})) - loss(dict(d, **{n: x - h * u}))) / (2 * h)
        want = (ref["d_init" if n == "init" else "d" + n] * u.numpy()).sum()
        assert abs(diff - want) <= 1e-7 * max(1.0, abs(want)), n


def test_packed_equals_separate():
    d = make(1, 12, 2, 1, 4, 4, io="f32", lengths=[5, 0, 7], seed=4)
    o, S = oracle_fwd(d)
    for s, (a, b) in enumerate([(0, 5), (5, 5), (5, 12)]):
        one = dict(d, cu=None, init=d["init"][s:s + 1], **{n: d[n][:, a:b] for n in ("q", "k", "v", "g", "beta")})
        o1, S1 = oracle_fwd(one)
        assert np.array_equal(o[:, a:b], o1) and np.array_equal(S[s:s + 1], S1)


def test_quantise():
    x = np.array([[127.0, -63.5, 0.5, 1.5], [0.0, 0.0, 0.0, 0.0], [448.0, 1.0625, 1.1875, -0.001]])
    back, scale = delta.quantise(x[:2], "int8")
    assert scale.tolist() == [1.0, 0.0] and back.tolist() == [[127.0, -64.0, 0.0, 2.0], [0.0] * 4]
    back, scale = delta.quantise(x, "e4m3")
    # 127 <= 448 / 2: scale 1/2 would do for 224, 1/4 for 112: 127 needs 1/2
    assert scale.tolist() == [0.5, 0.0, 1.0]
    # ties of 3 bits: 1.0625 -> 1.0 (even), 1.1875 -> 1.25 (even); 0.001 -> 2^-9 multiples: 0.001953125 * round(.512)
    assert back[2].tolist() == [448.0, 1.0, 1.25, -0.001953125]
    t = torch.randn(1000) * torch.exp(3 * torch.randn(1000))
    back, scale = delta.quantise(f64(t)[:, None], "e4m3")  # one-element rows: x / scale in (224, 448]
    want = (t / torch.from_numpy(scale).float()).to(torch.float8_e4m3fn).float() * torch.from_numpy(scale).float()
    assert np.array_equal(back[:, 0], f64(want))
