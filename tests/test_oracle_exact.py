"""Pins of the oracle's exact losses and gradients: torch's fp64 autograd,
central differences, and closed forms at the edges (CPU)."""
import numpy as np
import pytest
import torch

import oracle


def _rng(seed):
    return np.random.default_rng(seed)


def test_logprobs_against_torch():
    z = _rng(0).normal(size=(5, 40))
    z[1, ::3] = -np.inf
    y = np.array([0, 1, -1, 39, 7])
    got = oracle.token_logprobs(z, y, top=40)
    lp = torch.log_softmax(torch.from_numpy(z), 1)
    for t in range(5):
        assert got["logp"][t] == pytest.approx(float(lp[t, y[t]]) if y[t] >= 0 else 0.0, abs=1e-13)
    np.testing.assert_allclose(got["entropy"], torch.special.entr(lp.exp()).sum(1).numpy(),
                               atol=1e-13)
    order = torch.sort(torch.from_numpy(z), dim=1, descending=True, stable=True)
    live = np.isfinite(order.values.numpy())
    assert (got["top_ids"][live] == order.indices.numpy()[live]).all()
    assert (got["top_ids"][~live] == -1).all() and np.isneginf(got["top_logp"][~live]).all()


def test_logprobs_edges():
    z = np.array([[2.0, 2.0, 1.0, 2.0], [-np.inf] * 4, [0.0, np.nan, 1.0, 0.0],
                  [np.inf, 0.0, 0.0, 0.0], [-3e38, -3e38, -np.inf, -np.inf]])
    got = oracle.token_logprobs(z, np.array([2, 0, 0, 1, 1]), top=3)
    assert got["top_ids"].tolist() == [[0, 1, 3], [-1] * 3, [-1] * 3, [-1] * 3, [0, 1, -1]]
    assert np.isneginf(got["logp"][1]) and got["entropy"][1] == 0.0
    assert np.isnan(got["logp"][2:4]).all() and np.isnan(got["entropy"][2:4]).all()
    assert got["entropy"][4] == pytest.approx(np.log(2)) and got["logp"][4] == pytest.approx(
        -np.log(2))


@pytest.mark.parametrize("tau", [1.0, 0.5, 3.0])
def test_distill_against_autograd_and_differences(tau):
    r = _rng(1)
    T, V, k = 4, 23, 5
    z = r.normal(size=(T, V))
    ids = np.stack([r.choice(V, k, replace=False) for _ in range(T)])
    ids[1, 1] = ids[1, 0]           # listed twice
    ids[2, 3:] = -1
    vals = r.normal(size=(T, k))
    vals[0, 2] = -np.inf
    w = np.array([1.0, 0.3, 2.0, 0.0])
    got = oracle.distill(z, ids, vals, tau, w)
    zt = torch.from_numpy(z).requires_grad_()
    kept = torch.from_numpy(ids >= 0)
    q = torch.softmax(torch.where(kept, torch.from_numpy(vals) / tau, -torch.inf), 1)
    lp = torch.log_softmax(zt / tau, 1).gather(1, torch.from_numpy(ids).clamp(min=0))
    loss = tau ** 2 * (torch.xlogy(q, q) - q * lp).sum(1)
    (loss * torch.from_numpy(w)).sum().backward()
    np.testing.assert_allclose(got["loss"][:3], loss.detach().numpy()[:3], rtol=1e-12)
    np.testing.assert_allclose(got["dZ"], zt.grad.numpy(), atol=1e-14)
    assert got["loss"][3] == 0.0 and (got["dZ"][3] == 0).all()
    h = 1e-5
    for t, j in ((0, 3), (1, int(ids[1, 0])), (2, 20)):
        zp, zm = z.copy(), z.copy()
        zp[t, j] += h
        zm[t, j] -= h
        d = (oracle.distill(zp, ids, vals, tau, w)["loss"][t]
             - oracle.distill(zm, ids, vals, tau, w)["loss"][t]) / (2 * h)
        assert got["dZ"][t, j] == pytest.approx(w[t] * d, abs=1e-8)


def test_distill_of_its_own_teacher_is_a_stationary_point():
    # the teacher keeps every token and agrees with the student: loss and gradient 0
    z = _rng(2).normal(size=(3, 11))
    ids = np.tile(np.arange(11), (3, 1))
    got = oracle.distill(z, ids, z, 2.0)
    assert np.abs(got["loss"]).max() < 1e-14 and np.abs(got["dZ"]).max() < 1e-15


@pytest.mark.parametrize("heads,kv", [(3, 3), (4, 2), (4, 1)])
def test_attention_against_autograd_and_differences(heads, kv):
    r = _rng(3)
    cu = np.array([1, 6, 6, 7, 16])     # a row in front, an empty and a one-token sequence
    T, dh = 18, 4
    Q, E = r.normal(size=(2, T, heads * dh))
    K, V = r.normal(size=(2, T, kv * dh))
    got = oracle.exact_attention(Q, K, V, cu, heads, kv, E=E)
    qt, kt, vt = (torch.from_numpy(x).requires_grad_() for x in (Q, K, V))
    total = 0.0
    for a, b in zip(cu[:-1], cu[1:]):
        if a == b:
            continue
        sp = lambda t, n: t[a:b].view(b - a, n, dh).transpose(0, 1)  # noqa: E731
        o = torch.nn.functional.scaled_dot_product_attention(
            sp(qt, heads), sp(kt, kv).repeat_interleave(heads // kv, 0),
            sp(vt, kv).repeat_interleave(heads // kv, 0), is_causal=True)
        o = o.transpose(0, 1).reshape(b - a, -1)
        np.testing.assert_allclose(got["O"][a:b], o.detach().numpy(), atol=1e-12)
        total = total + (o * torch.from_numpy(E[a:b])).sum()
    total.backward()
    inside = np.zeros(T, bool)
    inside[1:16] = True
    for name, g in (("dQ", qt.grad), ("dK", kt.grad), ("dV", vt.grad)):
        np.testing.assert_allclose(got[name][inside], g.numpy()[inside], atol=1e-12)
        assert np.isnan(got[name][~inside]).all()
    # one-token sequences: o = v, and nothing moves the one-entry softmax: dp and
    # delta are the same 4-term sum in two orders, apart by at most
    # 2 x 4 x 2^-53 x sum |e v| < 1e-14 for these values
    assert np.abs(got["dQ"][6]).max() < 1e-14
    h = 1e-5
    for x, name, at in ((Q, "dQ", (9, 3)), (K, "dK", (8, 1)), (V, "dV", (7, 2))):
        f = []
        for s in (h, -h):
            x[at] += s
            f.append(np.nansum(oracle.exact_attention(Q, K, V, cu, heads, kv)["O"] * E))
            x[at] -= s
        assert got[name][at] == pytest.approx((f[0] - f[1]) / (2 * h), abs=1e-7)
