"""Exact causal attention and its gradients on the GPU against the fp64 oracle.

Tolerances, elementwise and from the arithmetic. fp32 tensors: a score is a sum
of d_h products (relative error at most d_h 2^-24 of the sum of their sizes,
far less in practice) and an exponential turns its absolute error into a
relative one; everything after is sums of such terms. F32 = 2e-5 of the sum of
the terms' sizes covers scores up to ~30. bf16 tensors add half a step (2^-8
relative) wherever the kernels round: the probabilities p and ds that enter a
product, the output o that delta = <o, e> is formed from, and the result.
"""
import ctypes

import numpy as np
import pytest
import torch

import oracle
import zeroth_order_transformer_dust_b200 as dust
from _util import np64

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
F32 = 2e-5
HALF = {"f32": 0.0, "bf16": 2.0 ** -8}


@pytest.fixture(scope="module")
def ctx(cuda_ok):
    return dust.Context(0)


def _inputs(T, heads, kv, dh, dtype, seed, fused=False, sd=1.0):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: (sd * torch.randn(*s, generator=gen)).to(DT[dtype]).cuda()  # noqa: E731
    if fused:
        q, k, v = r(T, (heads + 2 * kv) * dh).split([heads * dh, kv * dh, kv * dh], 1)
    else:
        q, k, v = r(T, heads * dh), r(T, kv * dh), r(T, kv * dh)
    return q, k, v, r(T, heads * dh)


def _sizes(Q, K, V, E, O, cu, heads, kv, scale):
    """Sums of the sizes of the terms behind every output: {name: (of all
    terms, of the terms that bf16 kernels round)}."""
    Q, K, V, E, O = (np64(x) for x in (Q, K, V, E, O))
    dh = Q.shape[1] // heads
    grp = heads // kv
    z = {n: np.zeros(x.shape) for n, x in (("O", Q), ("dQ", Q), ("dK", K), ("dV", K))}
    rnd = {n: x.copy() for n, x in z.items()}
    for a, b in zip(cu[:-1], cu[1:]):
        n = b - a
        low = np.tril(np.ones((n, n), dtype=bool))
        for h in range(heads):
            c, g = slice(h * dh, h * dh + dh), slice(h // grp * dh, h // grp * dh + dh)
            q, k, v, e, o = Q[a:b, c], K[a:b, g], V[a:b, g], E[a:b, c], O[a:b, c]
            if n == 0:
                continue
            s = np.where(low, scale * q @ k.T, -np.inf)
            p = np.exp(s - s.max(1, keepdims=True))
            p /= p.sum(1, keepdims=True)
            z["O"][a:b, c] += p @ np.abs(v)
            rnd["O"][a:b, c] += p @ np.abs(v)
            dl = np.abs(o * e).sum(1, keepdims=True)
            big = p * (np.abs(e) @ np.abs(v).T + dl)
            ds = np.abs(p * (e @ v.T - (o * e).sum(1, keepdims=True))) + p * dl
            z["dQ"][a:b, c] += scale * big @ np.abs(k)
            rnd["dQ"][a:b, c] += scale * ds @ np.abs(k)
            z["dK"][a:b, g] += scale * big.T @ np.abs(q)
            rnd["dK"][a:b, g] += scale * ds.T @ np.abs(q)
            z["dV"][a:b, g] += p.T @ np.abs(e)
            rnd["dV"][a:b, g] += p.T @ np.abs(e)
    return z, rnd


def _check(ctx, lengths, heads, kv, dh, dtype, fused=False, scale=None, sd=1.0, first=0, tail=0,
           **kw):
    cu = first + np.concatenate([[0], np.cumsum(lengths)]).astype(np.int64)
    T = int(cu[-1]) + tail
    q, k, v, e = _inputs(T, heads, kv, dh, dtype, seed=T + dh, fused=fused, sd=sd)
    outside = np.ones(T, dtype=bool)
    outside[first:cu[-1]] = False
    for x in (q, k, v, e):          # rows of no sequence are not read
        x[torch.from_numpy(outside).cuda()] = float("nan")
    shape = dict(n_heads=heads, n_kv_heads=kv, scale=scale, **kw)
    if "seq_len" not in kw:
        shape.update(cu_seqlens=torch.from_numpy(cu.astype(np.int32)).cuda(),
                     max_len=max(1, max(lengths)))
    fwd = ctx.attn_forward(q, k, v, out={
        "O": torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda"),
        "lse": torch.full((T, heads), 7.0, device="cuda")}, **shape)
    bwd = ctx.attn_backward(q, k, v, fwd["O"], fwd["lse"], e, out={
        n: torch.full(x.shape, 7.0, dtype=x.dtype, device="cuda")
        for n, x in (("dQ", q), ("dK", k), ("dV", v))}, **shape)
    ref = oracle.exact_attention(np64(q), np64(k), np64(v), cu, heads, kv, scale, E=np64(e))
    sc = dh ** -0.5 if scale is None else scale
    z, rnd = _sizes(q, k, v, e, fwd["O"], cu, heads, kv, sc)
    got = {n: np64(x) for n, x in {**fwd, **bwd}.items()}
    inside = ~outside
    for name in ("O", "dQ", "dK", "dV"):
        tol = F32 * z[name] + HALF[dtype] * (rnd[name] + np.abs(ref[name])) + 1e-30
        err = np.abs(got[name] - ref[name])
        assert np.all(err[inside] <= tol[inside]), (name, np.max((err / tol)[inside]))
    err = np.abs(got["lse"] - ref["lse"])[inside]
    assert np.all(err <= F32 * (1 + np.abs(ref["lse"][inside])))
    for name, x in got.items():     # left as they were
        assert (x[outside] == 7.0).all(), name


CASES = [
    ([1], 1, 1), ([2, 1, 1], 2, 1), ([63], 1, 1), ([64, 65], 2, 2), ([127, 128, 129], 1, 1),
    ([5, 0, 200, 1], 4, 2), ([300], 8, 1), ([257, 130], 3, 3),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dh", [32, 64, 128])
@pytest.mark.parametrize("lengths,heads,kv", CASES)
def test_packed_sequences(ctx, dtype, dh, lengths, heads, kv):
    _check(ctx, lengths, heads, kv, dh, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dh", [32, 64, 128])
def test_slices_of_a_fused_projection_with_rows_of_no_sequence(ctx, dtype, dh):
    # NaN rows in front of the first and behind the last sequence
    _check(ctx, [70, 0, 190, 3], 4, 2, dh, dtype, fused=True, first=5, tail=77)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_uniform_lengths_scale_and_large_scores(ctx, dtype):
    _check(ctx, [96, 96, 96], 2, 2, 64, dtype, seq_len=96)
    _check(ctx, [150], 2, 1, 128, dtype, scale=0.3, sd=1.5)
    _check(ctx, [600], 1, 1, 64, dtype)


def test_unaligned_rows(ctx):
    # bf16 rows at odd strides and addresses
    gen = torch.Generator().manual_seed(0)
    T, heads, dh = 140, 2, 64
    buf = torch.randn(4, 1 + T * 131, generator=gen).to(torch.bfloat16).cuda()
    q, k, v, e = (b[1:].view(T, 131)[:, :128] for b in buf)
    a = ctx.attn_forward(q, k, v, n_heads=heads)
    b = ctx.attn_forward(*(x.contiguous() for x in (q, k, v)), n_heads=heads)
    torch.testing.assert_close(a["O"].float(), b["O"].float(), rtol=2e-2, atol=2e-2)
    ga = ctx.attn_backward(q, k, v, b["O"], b["lse"], e, n_heads=heads)
    gb = ctx.attn_backward(*(x.contiguous() for x in (q, k, v)), b["O"], b["lse"],
                           e.contiguous(), n_heads=heads)
    for name in ga:
        torch.testing.assert_close(ga[name].float(), gb[name].float(), rtol=2e-2, atol=4e-2)


def test_gradients_into_slices_of_one_tensor(ctx):
    T, heads, kv, dh = 100, 4, 2, 64
    q, k, v, e = _inputs(T, heads, kv, dh, "bf16", 3)
    f = ctx.attn_forward(q, k, v, n_heads=heads, n_kv_heads=kv)
    ref = ctx.attn_backward(q, k, v, f["O"], f["lse"], e, n_heads=heads, n_kv_heads=kv)
    fused = torch.zeros(T, (heads + 2 * kv) * dh, dtype=torch.bfloat16, device="cuda")
    dq, dk, dv = fused.split([heads * dh, kv * dh, kv * dh], 1)
    ctx.attn_backward(q, k, v, f["O"], f["lse"], e, n_heads=heads, n_kv_heads=kv,
                      out={"dQ": dq, "dK": dk, "dV": dv})
    assert torch.equal(dq, ref["dQ"]) and torch.equal(dk, ref["dK"]) and torch.equal(dv, ref["dV"])


def test_gradient_against_differences(ctx):
    # d/dx of sum <o, e> in fp32: rounding of the sum (~1e-4) over 2h and the
    # third derivative's h^2 stay below 1e-2 for h = 0.05
    T, dh, h = 40, 32, 0.05
    q, k, v, e = _inputs(T, 2, 1, dh, "f32", 9)
    f = ctx.attn_forward(q, k, v, n_heads=2, n_kv_heads=1)
    g = ctx.attn_backward(q, k, v, f["O"], f["lse"], e, n_heads=2, n_kv_heads=1)
    for x, name, at in ((q, "dQ", (7, 3)), (k, "dK", (12, 1)), (v, "dV", (0, 31))):
        y = []
        for s in (h, -2 * h, h):
            x[at] += s
            o = ctx.attn_forward(q, k, v, n_heads=2, n_kv_heads=1)["O"]
            y.append(float((o.double() * e.double()).sum()))
        assert abs((y[0] - y[1]) / (2 * h) - float(g[name][at])) < 1e-2


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_repeatable_in_a_graph_and_on_another_stream(ctx, dtype):
    q, k, v, e = _inputs(333, 4, 2, 64, dtype, 5)
    cu = torch.tensor([0, 200, 333], dtype=torch.int32, device="cuda")
    kw = dict(n_heads=4, n_kv_heads=2, cu_seqlens=cu, max_len=200)
    f = ctx.attn_forward(q, k, v, **kw)
    want = {**f, **ctx.attn_backward(q, k, v, f["O"], f["lse"], e, **kw)}
    again = ctx.attn_backward(q, k, v, f["O"], f["lse"], e, **kw)
    for n in again:
        assert torch.equal(again[n], want[n])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = dust.Context(0, stream=side)
    got = other.attn_backward(q, k, v, f["O"], f["lse"], e, **kw)
    side.synchronize()
    for n in again:
        assert torch.equal(got[n], want[n])
    other.close()
    # two graphs of one context, replayed at the same time on two streams
    graphs, outs = [], []
    for _ in range(2):
        out = {n: torch.zeros_like(x) for n, x in want.items()}
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            ff = {n: out[n] for n in ("O", "lse")}
            ctx.attn_forward(q, k, v, out=ff, asynchronous=True, **kw)
            ctx.attn_backward(q, k, v, out["O"], out["lse"], e, asynchronous=True,
                              out={n: out[n] for n in ("dQ", "dK", "dV")}, **kw)
        graphs.append(g)
        outs.append(out)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for out in outs:
        for n in want:
            assert torch.equal(out[n], want[n]), n
    ctx.check()


def test_bad_offsets_are_reported_and_skipped(ctx):
    q, k, v, e = _inputs(100, 2, 2, 64, "bf16", 1)
    for cu, max_len in (([0, 40, 30, 100], 64), ([0, 40, 101], 64), ([-1, 40, 100], 64),
                        ([0, 70, 100], 64)):
        cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
        with pytest.raises(dust.DustError) as err:
            ctx.attn_forward(q, k, v, n_heads=2, cu_seqlens=cu, max_len=max_len)
        assert err.value.status == 4
    f = ctx.attn_forward(q, k, v, n_heads=2)
    with pytest.raises(dust.DustError) as err:
        ctx.attn_backward(q, k, v, f["O"], f["lse"], e, n_heads=2,
                          cu_seqlens=torch.tensor([0, 200], dtype=torch.int32, device="cuda"))
    assert err.value.status == 4


def test_refusals(ctx):
    q, k, v, e = _inputs(24, 4, 2, 64, "bf16", 1)
    ok = dict(n_heads=4, n_kv_heads=2)
    f = ctx.attn_forward(q, k, v, **ok)
    for bad in (dict(n_heads=3, n_kv_heads=1), dict(n_heads=4, n_kv_heads=3), dict(n_heads=4),
                dict(ok, seq_len=7), dict(ok, scale=0.0), dict(ok, scale=-1.0),
                dict(ok, seq_len=24, cu_seqlens=torch.zeros(2, dtype=torch.int32, device="cuda"))):
        with pytest.raises(ValueError):
            ctx.attn_forward(q, k, v, **bad)
    for bad in (dict(ok, scale=float("inf")), dict(n_heads=16, n_kv_heads=8)):  # 16-wide heads
        with pytest.raises(dust.DustError) as err:
            ctx.attn_forward(q, k, v, **bad)
        assert err.value.status == 1
    with pytest.raises(TypeError):
        ctx.attn_forward(q, k.float(), v, **ok)
    with pytest.raises(TypeError):
        ctx.attn_backward(q, k, v, f["O"].float(), f["lse"], e, **ok)
    with pytest.raises(ValueError):
        ctx.attn_backward(q, k, v, f["O"], f["lse"][:, :2], e, **ok)
    with pytest.raises(TypeError):
        ctx.attn_forward(q, k, v, cu_seqlens=torch.zeros(2, dtype=torch.int64, device="cuda"), **ok)
    for out in ({"dQ": q}, {"dQ": e}, {"dK": k}, {"dV": k}):
        with pytest.raises(dust.DustError, match="overlap"):
            ctx.attn_backward(q, k, v, f["O"], f["lse"], e, out=out, **ok)
    with pytest.raises(dust.DustError, match="overlap"):
        ctx.attn_forward(q, k, v, out={"O": q}, **ok)
    same = torch.empty_like(k)
    with pytest.raises(dust.DustError, match="apart"):
        ctx.attn_backward(q, k, v, f["O"], f["lse"], e, out={"dK": same, "dV": same}, **ok)
    empty = ctx.attn_forward(q[:0], k[:0], v[:0], **ok)
    assert empty["O"].shape == (0, 256)
    assert ctx.attn_backward(q[:0], k[:0], v[:0], empty["O"], empty["lse"], e[:0],
                             **ok)["dQ"].shape == (0, 256)


def test_the_estimator_converges_to_the_exact_gradient(ctx):
    # attn_grad's g for each projection against attn_backward, as a user would
    # compare them: with K draws of D = 64 channels the estimate's cosine with
    # the gradient is about 1 / sqrt(1 + (D + 1) / K)
    T, L, heads, dh, K = 96, 48, 1, 64, 16384
    q, k, v, e = _inputs(T, heads, heads, dh, "f32", 21)
    x = torch.randn(T, 32, device="cuda")
    f = ctx.attn_forward(q, k, v, n_heads=heads, seq_len=L)
    ex = ctx.attn_backward(q, k, v, f["O"], f["lse"], e, n_heads=heads, seq_len=L)
    for which, name in (("q", "dQ"), ("k", "dK"), ("v", "dV")):
        g = ctx.attn_grad(x, q, k, v, e, seq_len=L, n_heads=heads, which=which, K=K, sigma=1e-3,
                          want_G=False, want_g=True)["g"]
        cos = torch.nn.functional.cosine_similarity(g.flatten().double(),
                                                    ex[name].flatten().double(), dim=0)
        assert float(cos) > 0.99, which


def test_cosine_against_the_exact_gradient_follows_the_law(ctx):
    # for a linear response and n Gaussian channels cos(K) = 1 / sqrt(1 + (n + 1) / K)
    # per token; value noise is exactly linear, so its curve is the law's within
    # the sampling noise of 96 tokens x 64 channels
    from zeroth_order_transformer_dust_b200.alignment import attn_cosine_vs_k
    T, L, dh = 96, 48, 64
    q, k, v, e = _inputs(T, 1, 1, dh, "f32", 22)
    x = torch.randn(T, 16, device="cuda")
    for which in ("q", "k", "v"):
        res = attn_cosine_vs_k(ctx, x, q, k, v, e, seq_len=L, n_heads=1, which=which,
                               ks=[64, 512, 4096], sigma=1e-3)
        assert res["K"] == [64, 512, 4096] and res["cos_g"] == sorted(res["cos_g"])
        assert res["cos_g"][-1] > 0.97
        if which == "v":
            for K, c in zip(res["K"], res["cos_g"]):
                assert abs(c - (1 + (dh + 1) / K) ** -0.5) < 0.03


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dh", [64, 128])
def test_cuda_core_form(monkeypatch, dtype, dh):
    # what a context without tensor cores runs, at widths they otherwise take
    monkeypatch.setenv("DUST_DISABLE_TC", "1")
    c = dust.Context(0)
    _check(c, [130, 1, 64], 4, 2, dh, dtype, fused=True, first=3, tail=9)
    c.close()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_growing_scores_move_the_maximum(ctx, dtype):
    # keys that grow along the sequence: the running maximum moves by far more
    # than the rescaling threshold in every tile, and shrinking ones never move it
    T, heads, dh = 520, 2, 64
    q, k, v, e = _inputs(T, heads, heads, dh, dtype, 4)
    ramp = torch.linspace(0.1, 6.0, T, device="cuda")[:, None]
    for r in (ramp, ramp.flip(0)):
        kk = (k.float() * r).to(k.dtype)
        f = ctx.attn_forward(q, kk, v, n_heads=heads)
        g = ctx.attn_backward(q, kk, v, f["O"], f["lse"], e, n_heads=heads)
        ref = oracle.exact_attention(np64(q), np64(kk), np64(v), [0, T], heads, heads, E=np64(e))
        z, rnd = _sizes(q, kk, v, e, f["O"], [0, T], heads, heads, dh ** -0.5)
        # scores reach ~100: exponents carry |s| 2^-23 more than F32 covers
        slack = 100 * 2.0 ** -22
        for name, x in {**f, **g}.items():
            if name == "lse":
                assert np.all(np.abs(np64(x) - ref["lse"]) <= 5e-5 * (1 + np.abs(ref["lse"])))
                continue
            tol = (F32 + slack) * z[name] + HALF[dtype] * (rnd[name] + np.abs(ref[name])) + 1e-30
            assert np.all(np.abs(np64(x) - ref[name]) <= tol), name


def test_offsets_past_32_bits(ctx):
    # two sequences whose rows lie more than 2^31 elements into their tensors
    ld, T, dh = 1 << 20, 2200, 64
    buf = torch.zeros(T * ld, dtype=torch.bfloat16, device="cuda").view(T, ld)
    gen = torch.Generator().manual_seed(2)
    x = torch.randn(150, 4 * dh, generator=gen).to(torch.bfloat16).cuda()
    buf[2050:, :4 * dh] = x
    cu = torch.tensor([2050, 2180, 2200], dtype=torch.int32, device="cuda")
    kw = dict(n_heads=1, cu_seqlens=cu, max_len=130)
    part = lambda t: t.split(dh, 1)  # noqa: E731
    q, k, v, e = part(buf[:, :4 * dh])
    f = ctx.attn_forward(q, k, v, out={"O": buf[:, 4 * dh:5 * dh]}, **kw)
    g = ctx.attn_backward(q, k, v, f["O"], f["lse"], e, **kw)
    q, k, v, e = (t.contiguous() for t in part(x))
    kw["cu_seqlens"] = cu - 2050
    f2 = ctx.attn_forward(q, k, v, **kw)
    g2 = ctx.attn_backward(q, k, v, f2["O"], f2["lse"], e, **kw)
    assert torch.equal(f["O"][2050:], f2["O"]) and torch.equal(f["lse"][2050:], f2["lse"])
    for n in g2:
        assert torch.equal(g[n][2050:], g2[n]), n


@pytest.mark.parametrize("dtype,dh", [("bf16", 64), ("bf16", 128), ("f32", 64), ("f32", 32)])
def test_what_lies_around_a_sequence_does_not_change_its_bits(ctx, dtype, dh):
    # rows behind (and before) a sequence share its last tile; whether they are a
    # neighbour's ordinary rows, huge ones, or nobody's, the sequence's results are
    # those of a call on it alone
    n, pad, heads, kv = 300, 100, 2, 1
    base = _inputs(n + 2 * pad, heads, kv, dh, dtype, 31)
    shape = dict(n_heads=heads, n_kv_heads=kv)
    alone = [x[pad:pad + n].contiguous() for x in base]
    f = ctx.attn_forward(*alone[:3], **shape)
    want = {**f, **ctx.attn_backward(*alone[:3], f["O"], f["lse"], alone[3], **shape)}
    for size in (1.0, 60.0, 1e4):
        for cu in ([0, pad, pad + n, n + 2 * pad], [pad, pad + n]):
            q, k, v, e = (x.clone() for x in base)
            for x in (q, k, v, e):
                x[:pad] *= size
                x[pad + n:] *= size
            kw = dict(shape, max_len=n, cu_seqlens=torch.tensor(cu, dtype=torch.int32,
                                                                device="cuda"))
            f = ctx.attn_forward(q, k, v, **kw)
            got = {**f, **ctx.attn_backward(q, k, v, f["O"], f["lse"], e, **kw)}
            for name, x in want.items():
                assert torch.equal(got[name][pad:pad + n], x), (name, size, cu)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dh", [32, 64, 128])
@pytest.mark.parametrize("ld", [0, 131, -7])
def test_one_row_has_no_stride(ctx, dtype, dh, ld):
    # through the C ABI: the stride of a tensor of one row is not used, whatever it is
    heads, kv = 2, 1
    q, k, v, e = _inputs(1, heads, kv, dh, dtype, 6)
    f = ctx.attn_forward(q, k, v, n_heads=heads, n_kv_heads=kv)
    want = {**f, **ctx.attn_backward(q, k, v, f["O"], f["lse"], e, n_heads=heads, n_kv_heads=kv)}
    got = {name: torch.full_like(x, 7.0) for name, x in want.items()}
    L = dust.load_library()
    code = dust.DUST_F32 if dtype == "f32" else dust.DUST_BF16
    d = dust.DustAttnDims(1, None, 1, 1, heads, kv, dh, code, 0.0, 0, *[ld] * 8)
    work = [torch.empty(max(1, L.dust_attn_work_bytes(ctypes.byref(d), b)), dtype=torch.uint8,
                        device="cuda") for b in (0, 1)]
    ctx._bind_stream()
    ctx._check(L.dust_attn_forward(ctx._h, ctypes.byref(d), *(
        x.data_ptr() for x in (q, k, v, got["O"], got["lse"], work[0]))))
    ctx._check(L.dust_attn_backward(ctx._h, ctypes.byref(d), *(
        x.data_ptr() for x in (q, k, v, got["O"], got["lse"], e, got["dQ"], got["dK"], got["dV"],
                               work[1]))))
    for name in want:
        assert torch.equal(got[name], want[name]), name


@pytest.mark.parametrize("dtype,dh", [("bf16", 32), ("bf16", 64), ("bf16", 128), ("f32", 64),
                                      ("f32", 128)])
def test_scores_of_minus_infinity_in_the_first_tiles(ctx, dtype, dh):
    # finite inputs, but the last channel takes the first 140 keys' scores below
    # fp32's range (-2^129 scale): p = 0 there, and the rows behind attend to the
    # rest. (The first 140 rows have no other key; they are not looked at.)
    T, cut = 500, 140
    q, k, v, e = _inputs(T, 1, 1, dh, dtype, 17)
    q[:, -1] = 2.0 ** 64
    k[:, -1] = 0.0
    k[:cut, -1] = -2.0 ** 65
    kw = dict(n_heads=1, scale=0.1)
    f = ctx.attn_forward(q, k, v, **kw)
    g = ctx.attn_backward(q, k, v, f["O"], f["lse"], e, **kw)
    ref = oracle.exact_attention(np64(q), np64(k), np64(v), [0, T], 1, 1, kw["scale"], E=np64(e))
    z, rnd = _sizes(q, k, v, e, torch.from_numpy(ref["O"]), [0, T], 1, 1, kw["scale"])
    for name, x in (("O", f["O"]), ("dQ", g["dQ"])):
        tol = F32 * z[name] + HALF[dtype] * (rnd[name] + np.abs(ref[name])) + 1e-30
        assert np.all((np.abs(np64(x) - ref[name]) <= tol)[cut:]), name
    err = np.abs(np64(f["lse"]) - ref["lse"])[cut:]
    assert np.all(err <= F32 * (1 + np.abs(ref["lse"][cut:])))


# Sequences of 9 to 14 tiles: every ring of stages is worked through several
# times, in three heads' turns on the key side, with a ragged last tile. The
# tolerances hold at these lengths: a chain of n fp32 roundings is off by about
# sqrt(n) 2^-24 of the sum of the terms' sizes (2.3e-6 for 1500), and an
# accumulation that truncates once per 16 terms, n / 16 times, by at most
# n / 16 x 2^-23 of it (1.1e-5), both below F32.
@pytest.mark.parametrize("dtype,dh", [("bf16", 64), ("bf16", 128), ("f32", 64), ("bf16", 32),
                                      ("f32", 128)])
def test_sequences_of_many_tiles(ctx, dtype, dh):
    _check(ctx, [1409, 0, 1190, 37], 3, 1, dh, dtype, fused=True, first=1, tail=3)


@pytest.mark.parametrize("dtype,dh", [("bf16", 128), ("bf16", 64), ("f32", 64)])
def test_growing_scores_over_many_tiles(ctx, dtype, dh):
    # the maximum of a row moves in every one of up to ten tiles, or in the first alone
    T = 1250
    q, k, v, e = _inputs(T, 1, 1, dh, dtype, 14)
    ramp = torch.linspace(0.1, 6.0, T, device="cuda")[:, None]
    for r in (ramp, ramp.flip(0)):
        kk = (k.float() * r).to(k.dtype)
        f = ctx.attn_forward(q, kk, v, n_heads=1)
        g = ctx.attn_backward(q, kk, v, f["O"], f["lse"], e, n_heads=1)
        ref = oracle.exact_attention(np64(q), np64(kk), np64(v), [0, T], 1, 1, E=np64(e))
        z, rnd = _sizes(q, kk, v, e, f["O"], [0, T], 1, 1, dh ** -0.5)
        slack = 100 * 2.0 ** -22   # as in the test of one head width above
        for name, x in {**f, **g}.items():
            if name == "lse":
                assert np.all(np.abs(np64(x) - ref["lse"]) <= 5e-5 * (1 + np.abs(ref["lse"])))
                continue
            tol = (F32 + slack) * z[name] + HALF[dtype] * (rnd[name] + np.abs(ref[name])) + 1e-30
            assert np.all(np.abs(np64(x) - ref[name]) <= tol), name


@pytest.mark.parametrize("dtype,dh", [("bf16", 64), ("bf16", 128), ("f32", 64), ("f32", 32)])
@pytest.mark.parametrize("cu", [[0, 40, 30, 100], [0, 40, 101], [-1, 40, 100], [0, 70, 100],
                                [0, 40, 200, 100, 100]])
def test_bad_sequences_stay_as_they_were_and_good_ones_are_computed(ctx, dtype, dh, cu):
    T, max_len = 100, 64
    shape = dict(n_heads=2, n_kv_heads=1, max_len=max_len)
    q, k, v, e = _inputs(T, 2, 1, dh, dtype, 1)
    offsets = torch.tensor(cu, dtype=torch.int32, device="cuda")
    new = lambda: {name: torch.full((T, w), 7.0, dtype=dt, device="cuda")  # noqa: E731
                   for name, w, dt in (("O", 2 * dh, q.dtype), ("lse", 2, torch.float32),
                                       ("dQ", 2 * dh, q.dtype), ("dK", dh, q.dtype),
                                       ("dV", dh, q.dtype))}
    part = lambda out, names: {n: out[n] for n in names}  # noqa: E731
    want, got = new(), new()
    good = [(a, b) for a, b in zip(cu[:-1], cu[1:]) if 0 <= a <= b <= T and b - a <= max_len]
    for a, b in good:
        kw = dict(shape, cu_seqlens=torch.tensor([a, b], dtype=torch.int32, device="cuda"))
        ctx.attn_forward(q, k, v, out=part(want, ("O", "lse")), **kw)
        ctx.attn_backward(q, k, v, want["O"], want["lse"], e, out=part(want, ("dQ", "dK", "dV")),
                          **kw)
    for call in (lambda: ctx.attn_forward(q, k, v, out=part(got, ("O", "lse")),
                                          cu_seqlens=offsets, **shape),
                 lambda: ctx.attn_backward(q, k, v, want["O"], want["lse"], e,
                                           out=part(got, ("dQ", "dK", "dV")),
                                           cu_seqlens=offsets, **shape)):
        with pytest.raises(dust.DustError) as err:
            call()
        assert err.value.status == 4
    ctx.check()                               # reported once
    for name in want:
        assert torch.equal(got[name], want[name]), name
