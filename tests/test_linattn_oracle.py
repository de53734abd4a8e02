"""Pins of the linear attention oracle (CPU): the quadratic closed form, the undecayed
cumulative sum, split invariance, and the SSD oracle where the two recurrences coincide."""
import math

import pytest
import torch

from oracle import linattn_oracle as LO
from oracle import oracle as O


def _inp(T=13, H=4, Hk=2, K=8, V=16, nseq=1, seed=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    return r(T, H, K), r(T, Hk, K), r(T, Hk, V), -torch.rand(Hk, generator=g, dtype=torch.float64), r(nseq, Hk, V, K)


def test_closed_form():
    q, k, v, g, s0 = _inp()
    got = LO.linattn(q, k, v, g, 0.5, s0)
    T, H, Hk = q.shape[0], q.shape[1], k.shape[1]
    for t in range(T):
        for h in range(H):
            kv = h // (H // Hk)
            y = math.exp(g[kv] * (t + 1)) * (s0[0, kv] @ q[t, h])
            for s in range(t + 1):
                y = y + math.exp(g[kv] * (t - s)) * (q[t, h] @ k[s, kv]) * v[s, kv]
            assert torch.allclose(got["o"][t, h], 0.5 * y, rtol=0, atol=1e-12)
    assert bool((got["o_mag"] + 1e-12 >= got["o"].abs()).all())


def test_no_decay_is_a_cumulative_sum():
    q, k, v, g, _ = _inp()
    got = LO.linattn(q, k, v, torch.zeros_like(g), 1.0)
    assert torch.allclose(got["final"][0], torch.einsum("thv,thk->hvk", v, k), atol=1e-12)


def test_packed_sequences_and_splits():
    q, k, v, g, s0 = _inp(T=12, nseq=3)
    whole = LO.linattn(q, k, v, g, 1.0, s0, [5, 0, 7])
    assert torch.equal(whole["final"][1], s0[1])
    a = LO.linattn(q[5:9], k[5:9], v[5:9], g, 1.0, s0[2:3])
    b = LO.linattn(q[9:], k[9:], v[9:], g, 1.0, a["final"])
    assert torch.allclose(torch.cat([a["o"], b["o"]]), whole["o"][5:], atol=1e-12)
    assert torch.allclose(b["final"][0], whole["final"][2], atol=1e-12)


def test_equals_the_ssd_oracle_with_unit_dt():
    # dt = softplus(dt_raw + dt_bias) = 1 makes the SSD recurrence this one: x = v, B = k, C = q
    T, H, K, V = 9, 3, 16, 16
    q, k, v, g, s0 = _inp(T, H, H, K, V)
    f = lambda t: t.float()  # noqa: E731
    q, k, v, g, s0 = f(q), f(k), f(v), f(g), f(s0)
    raw = torch.full((T, H), math.log(math.e - 1.0))
    y, fin = O.ssd_scan(v, raw, torch.zeros(H), g, k, q, torch.zeros(H), init_state=s0, batch=1)
    got = LO.linattn(q, k, v, g, 1.0, s0)
    # dt_raw is rounded to float: dt is off 1 by at most 2^-24, times the 9 steps
    assert torch.allclose(torch.as_tensor(y).view_as(got["o"]), got["o"], atol=2e-5)
    assert torch.allclose(torch.as_tensor(fin), got["final"], atol=2e-5)


@pytest.mark.parametrize("mistake", ["transposed", "late"])
def test_planted_mistakes_fail(mistake):
    q, k, v, g, s0 = _inp(K=16)
    good = LO.linattn(q, k, v, g, 1.0, s0)
    if mistake == "transposed":
        bad = LO.linattn(q, v, k, g, 1.0, s0.transpose(2, 3).contiguous())
    else:
        bad = LO.linattn(q, torch.roll(k, 1, 0), torch.roll(v, 1, 0), g, 1.0, s0)
    assert not torch.allclose(bad["o"], good["o"], atol=1e-3)
