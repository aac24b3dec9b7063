"""Scores and distillation of a head's logits on the GPU against the fp64 oracle.

Tolerances, from the kernels' arithmetic (u = 2^-24, one fp32 rounding). An
exponential exp((z - m)/tau) carries the rounding of z - m and of its scaling
(|d| u each for an exponent d, and terms with |d| > 30 weigh nothing), the
hardware exponential's 2^-22, and its share of the sums (at most ~64 roundings
a thread and join): below 5e-6 relative, so log s is within 5e-6. A log
probability adds the rounding of its own size. The entropy log s - u/s has the
same relative error on terms that sum to at most its value plus log s. A
gradient entry w tau (p - q) has 5e-6 of p and of q, then the one rounding to
its type (half a step, eps / 2 of the value).
"""
import math

import numpy as np
import pytest
import torch

import oracle
import zeroth_order_transformer_dust_b200 as dust
from _util import np64

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
E32 = 2.0 ** -23


@pytest.fixture(scope="module")
def ctx(cuda_ok):
    return dust.Context(0)


def _logits(T, V, dtype, seed=0, pitch=None, offset=0, sd=3.0):
    """T x V logits in rows of `pitch`, the first `offset` elements into a buffer."""
    pitch = pitch or V
    gen = torch.Generator().manual_seed(seed)
    buf = (torch.randn(offset + T * pitch, generator=gen) * sd).to(DT[dtype]).cuda()
    return buf[offset:].view(T, pitch)[:, :V]


def _check_scores(got, Z, tokens, top):
    ref = oracle.token_logprobs(np64(Z), tokens, top)
    for name in ("logp", "entropy") + (("top_logp",) if top else ()):
        g, r = np64(got[name]), ref[name]
        assert (np.isnan(g) == np.isnan(r)).all(), name
        assert (g[np.isinf(r)] == r[np.isinf(r)]).all(), name
        ok = np.isfinite(r)
        assert np.all(np.abs(g[ok] - r[ok]) <= 1e-5 + 4 * E32 * np.abs(r[ok])), name
    if top:
        assert (got["top_ids"].cpu().numpy() == ref["top_ids"]).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,V,pitch,offset,top", [
    (1, 1, None, 0, 1), (3, 2, None, 1, 2), (5, 7, 9, 3, 7), (2, 33, None, 1, 32),
    (4, 255, 256, 0, 128), (1, 4097, None, 5, 20), (9, 5003, 5003, 0, 128),
    (150, 2049, 2050, 1, 3), (300, 1000, None, 0, 0), (2, 50257, 50304, 0, 5),
    (1, 128256, None, 0, 64), (40, 16391, None, 2, 0), (17, 40000, 40001, 0, 17)])
def test_scores(ctx, dtype, T, V, pitch, offset, top):
    # rows that start at any element of a 16-byte vector, one to eight CTAs a row
    Z = _logits(T, V, dtype, seed=T + V, pitch=pitch, offset=offset)
    tokens = np.random.default_rng(V).integers(0, V, T).astype(np.int32)
    tokens[::4] = -1
    got = ctx.token_logprobs(Z, torch.from_numpy(tokens).cuda(), top=top)
    _check_scores(got, Z, tokens, top)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [300, 9000])
def test_scores_at_the_edges(ctx, dtype, V):
    lowest = torch.finfo(DT[dtype]).min
    Z = _logits(12, V, dtype, seed=5)
    Z[0] = -math.inf                          # a mask that leaves nothing
    Z[1] = -math.inf
    Z[1, 250] = 0.5                           # one token left, of 20 asked for
    Z[2, : V - 3] = -math.inf
    Z[3] = lowest                             # the type's lowest value is a logit
    Z[4, 10:] = lowest
    Z[5, 77] = math.nan
    Z[6, V - 1] = math.inf
    Z[7] = 1.25                               # every logit equal: ids 0, 1, 2, ...
    Z[8] = torch.arange(V).to(Z)              # each better than all before
    Z[9, 5], Z[9, 9] = 0.0, -0.0              # equal, the lower id first
    Z[9, 20:] = -1.0
    Z[10] = torch.finfo(DT[dtype]).max        # exp of differences only
    Z[11] = (torch.arange(V) % 2).to(Z)       # half the row ties for the best
    tokens = np.array([0, 250, V - 1, 3, 4, 5, 6, 7, V - 1, 9, 10, 11], dtype=np.int32)
    got = ctx.token_logprobs(Z, torch.from_numpy(tokens).cuda(), top=20)
    _check_scores(got, Z, tokens, 20)
    assert np.isneginf(np64(got["logp"])[0]) and np64(got["entropy"])[0] == 0.0
    assert got["top_ids"][1].tolist() == [250] + [-1] * 19
    assert got["top_ids"][7].tolist() == list(range(20))


def test_scores_of_hard_rows_for_the_list(ctx):
    # rows that make the list of candidates grow as fast as it can, over
    # eight CTAs, one and unaligned: ascending, all equal, the best ones last
    for T, V, off in ((1, 30011, 1), (160, 30011, 3)):
        Z = _logits(T, V, "f32", seed=T, offset=off)
        Z[0] = torch.linspace(-4, 4, V).cuda()
        if T > 1:
            Z[1] = 0.0
            Z[2, -600:] += 50.0
        tokens = np.zeros(T, dtype=np.int32)
        got = ctx.token_logprobs(Z, torch.from_numpy(tokens).cuda(), top=128)
        _check_scores(got, Z, tokens, 128)


def test_scores_options_and_refusals(ctx):
    Z = _logits(6, 100, "f32")
    tok = torch.zeros(6, dtype=torch.int32, device="cuda")
    assert set(ctx.token_logprobs(Z, top=0)) == {"entropy"}
    assert set(ctx.token_logprobs(Z, tok, want_entropy=False, top=2)) == {
        "logp", "top_ids", "top_logp"}
    out = {"logp": torch.empty(6, device="cuda")}
    assert ctx.token_logprobs(Z, tok, out=out)["logp"] is out["logp"]
    assert ctx.token_logprobs(Z[:0], tok[:0], top=3)["top_ids"].shape == (0, 3)
    for bad in (dict(top=101), dict(top=-1), dict(out={"logp": torch.empty(5, device="cuda")}),
                dict(out={"logp": torch.empty(6)})):
        with pytest.raises(ValueError):
            ctx.token_logprobs(Z, tok, **bad)
    with pytest.raises(ValueError, match="rows"):
        ctx.token_logprobs(Z.t(), torch.zeros(100, dtype=torch.int32, device="cuda"))
    with pytest.raises(TypeError):
        ctx.token_logprobs(Z, tok.long())
    with pytest.raises(TypeError):
        ctx.token_logprobs(Z.half(), tok)
    tok[3] = 100                              # outside [0, V): reported, its logp NaN
    out = {"logp": torch.zeros(6, device="cuda")}
    with pytest.raises(dust.DustError) as e:
        ctx.token_logprobs(Z, tok, out=out)
    assert e.value.status == 4
    assert torch.isnan(out["logp"]).tolist() == [False] * 3 + [True] + [False] * 2
    tok[3] = -2
    ctx.token_logprobs(Z, tok, asynchronous=True)
    with pytest.raises(dust.DustError):
        ctx.check()
    ctx.check()                               # reported once


def _teacher(T, V, k, seed, missing=True):
    r = np.random.default_rng(seed)
    ids = np.stack([r.choice(V, k, replace=V < k) for _ in range(T)]).astype(np.int32)
    vals = (2 * r.normal(size=(T, k))).astype(np.float32)
    if missing and k > 2:
        ids[::3, k - 1] = -1
        vals[1::3, 0] = -np.inf
    return ids, vals


def _check_distill(got, Z, ids, vals, tau, w, dtype):
    ref = oracle.distill(np64(Z), ids, vals, tau, w)
    p = oracle.distill(np64(Z), ids, vals, tau, None)["dZ"] / tau     # p - q
    T, V = ref["dZ"].shape
    q = np.zeros((T, V))
    for t in range(T):
        kept = (ids[t] >= 0) & ~np.isneginf(vals[t])
        if kept.any():
            v = vals[t][kept].astype(np.float64) / tau
            e = np.exp(v - v.max())
            np.add.at(q[t], ids[t][kept], e / e.sum())
    if "loss" in got:
        g, r = np64(got["loss"]), ref["loss"]
        assert (np.isnan(g) == np.isnan(r)).all()
        assert (g[np.isinf(r)] == r[np.isinf(r)]).all()
        ok = np.isfinite(r)
        size = tau ** 2 * (1 + np.abs(r[ok]) / tau ** 2)
        assert np.all(np.abs(g[ok] - r[ok]) <= 2e-5 * size)
    g, r = np64(got["dZ"]), ref["dZ"]
    assert (np.isnan(g) == np.isnan(r)).all()
    ww = np.ones(T) if w is None else np.abs(np.asarray(w, dtype=np.float64))
    ok = ~np.isnan(r)
    # a probability's exponent x = (z - m) / tau, |x| <= -ln p, is rounded three
    # times (z - m, the scale log2(e) / tau, their product): 3 |x| u of p, which
    # the 5e-6 cover only down to p ~ e^-28
    prob = np.abs(np.nan_to_num(p) + q)       # (p is NaN in rows that weight 0 leaves out)
    rel = 5e-6 + 3 * 2.0 ** -24 * -np.log(np.clip(prob, 1e-300, 1.0))
    tol = (ww * tau)[:, None] * (rel * prob + 5e-6 * q) + 1e-37
    tol += torch.finfo(DT[dtype]).eps / 2 * np.abs(r)
    off = np.abs(g - r)[ok] > tol[ok]
    assert not off.any(), off.sum()


def _dev(ids, vals, w=None):
    t = [torch.from_numpy(ids).cuda(), torch.from_numpy(vals).cuda()]
    return t + [None if w is None else torch.from_numpy(np.asarray(w, dtype=np.float32)).cuda()]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,V,pitch,offset,k,tau", [
    (1, 1, None, 0, 1, 1.0), (2, 2, None, 1, 2, 0.7), (5, 9, 11, 1, 4, 2.0),
    (3, 1023, None, 3, 16, 1.0), (150, 515, 516, 0, 7, 1.5), (1, 9001, None, 2, 128, 1.0),
    (4, 50257, 50304, 0, 32, 2.0), (2, 128256, None, 0, 64, 1.0), (160, 8200, None, 1, 50, 0.5),
    (1, 500003, None, 1, 5, 1.0)])
def test_distill(ctx, dtype, T, V, pitch, offset, k, tau):
    # one row and many, one to eight CTAs a row, and a row too long to be resident
    Z = _logits(T, V, dtype, seed=V, pitch=pitch, offset=offset)
    ids, vals = _teacher(T, V, k, V)
    w = np.linspace(0.0, 1.5, T).astype(np.float32) if T > 2 else None
    di, dv, dw = _dev(ids, vals, w)
    got = ctx.distill(Z, di, dv, temperature=tau, weights=dw)
    _check_distill(got, Z, ids, vals, tau, w, dtype)
    only = ctx.distill(Z, di, dv, temperature=tau, weights=dw, want_grad=False)
    torch.testing.assert_close(only["loss"], got["loss"], rtol=2e-5, atol=2e-5 * tau ** 2)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [700, 60001])
def test_distill_gradient_layouts(ctx, dtype, V):
    # in place, into rows of another stride, and into rows of another alignment
    T, k = 6, 9
    ids, vals = _teacher(T, V, k, 3)
    di, dv, _ = _dev(ids, vals)
    Z = _logits(T, V, dtype, seed=1, pitch=V + 3, offset=1)
    ref = ctx.distill(Z, di, dv)["dZ"].clone()
    wide = torch.full((T, V + 16), 7.0, dtype=DT[dtype], device="cuda")
    for first in (0, 1, 2, 8):
        wide.fill_(7.0)
        dst = wide[:, first:first + V]
        ctx.distill(Z, di, dv, out={"dZ": dst})
        assert torch.equal(dst, ref)
        assert (wide[:, :first] == 7).all() and (wide[:, first + V:] == 7).all()
    loss = ctx.distill(Z, di, dv, want_grad=False)["loss"]
    got = ctx.distill(Z, di, dv, out={"dZ": Z})
    assert got["dZ"] is Z and torch.equal(Z, ref)
    torch.testing.assert_close(got["loss"], loss, rtol=2e-5, atol=2e-5)


@pytest.mark.parametrize("V", [64, 9000, 60000])
def test_distill_at_the_edges(ctx, V):
    T, k = 10, 6
    Z = _logits(T, V, "f32", seed=2)
    ids, vals = _teacher(T, V, k, 4, missing=False)
    w = np.ones(T, dtype=np.float32)
    ids[0] = -1                               # no entry: left out, its logits not read
    Z[0] = math.nan
    w[1] = 0.0                                # weight 0: left out
    Z[1, 3] = math.nan
    vals[2] = -np.inf                         # every value masked: no entry
    ids[3, 1:] = ids[3, 0]                    # one token listed six times
    Z[4] = -math.inf                          # the student's mask leaves nothing
    Z[5, ids[5, 2]] = -math.inf               # the student masks what the teacher keeps
    Z[6, 1] = math.nan
    Z[7] = torch.finfo(torch.float32).min
    Z[8, ids[8, 0]] = 60.0                    # a certain student
    vals[9, 0] = 80.0                         # a certain teacher
    di, dv, dw = _dev(ids, vals, w)
    got = ctx.distill(Z, di, dv, weights=dw, temperature=0.9)
    _check_distill(got, Z, ids, vals, 0.9, w, "f32")
    assert got["loss"][:3].tolist() == [0.0] * 3 and not got["dZ"][:3].any()
    assert torch.isinf(got["loss"][4:6]).all()


def test_distill_gradient_against_differences(ctx):
    # central differences of the loss itself: at step h the loss's rounding
    # (about 1e-6) over 2h and the third derivative's h^2 stay below 1e-3
    T, V, k, tau, h = 3, 50, 5, 1.3, 0.05
    Z = _logits(T, V, "f32", seed=8, sd=1.0)
    ids, vals = _teacher(T, V, k, 6)
    di, dv, _ = _dev(ids, vals)
    dZ = ctx.distill(Z, di, dv, temperature=tau)["dZ"].clone()
    for j in (0, 17, 49, int(ids[1, 1])):
        step = torch.zeros_like(Z)
        step[:, j] = h
        f = [ctx.distill(Z + s * step, di, dv, temperature=tau, want_grad=False)["loss"]
             for s in (1, -1)]
        torch.testing.assert_close(dZ[:, j], (f[0] - f[1]) / (2 * h), rtol=0, atol=1e-3)


def test_distill_refusals(ctx):
    Z = _logits(4, 60, "f32")
    ids, vals = _teacher(4, 60, 5, 1)
    di, dv, _ = _dev(ids, vals)
    for bad in (dict(temperature=0.0), dict(temperature=-1.0), dict(temperature=math.nan),
                dict(temperature=math.inf)):
        with pytest.raises(dust.DustError) as e:
            ctx.distill(Z, di, dv, **bad)
        assert e.value.status == 1
    with pytest.raises(dust.DustError, match="apart"):   # overlaps, but not in place
        ctx.distill(Z[:3], di[:3], dv[:3], out={"dZ": Z[1:]})
    with pytest.raises(dust.DustError, match="k must"):
        ctx.distill(Z, di[:, :0].contiguous(), dv[:, :0].contiguous())
    with pytest.raises(ValueError):
        ctx.distill(Z, di, dv[:, :4].contiguous())
    with pytest.raises(TypeError):
        ctx.distill(Z, di.long(), dv)
    with pytest.raises(TypeError):
        ctx.distill(Z, di, dv.double())
    with pytest.raises(ValueError):
        ctx.distill(Z, di, dv, out={"dZ": torch.empty(4, 60, dtype=torch.bfloat16, device="cuda")})
    assert ctx.distill(Z[:0], di[:0], dv[:0])["dZ"].shape == (0, 60)
    di[2, 1] = 60                             # outside [0, V): reported, counts as no entry
    out = {}
    with pytest.raises(dust.DustError) as e:
        out["dZ"] = torch.empty_like(Z)
        ctx.distill(Z, di, dv, out=out)
    assert e.value.status == 4
    ids[2, 1] = -1
    _check_distill({"dZ": out["dZ"]}, Z, ids, vals, 1.0, None, "f32")
    # far outside, in every entry of the last rows: no live row follows
    di[2:] = 1 << 30
    di[3, 0] = -(1 << 30)
    ids[2:] = -1
    for rows in (Z, _logits(4, 60000, "f32")):
        out = {"dZ": torch.empty_like(rows)}
        with pytest.raises(dust.DustError) as e:
            ctx.distill(rows, di, dv, out=out)
        assert e.value.status == 4
        assert not out["dZ"][2:].any() and out["dZ"][0].any()


def test_teacher_scores_feed_the_student(ctx):
    # the two operators as they are used: a teacher's alternatives, masked
    # vocabulary and all, are the student's targets as they are; a student
    # that equals its teacher on the kept tokens and keeps all of them is done
    T, V, k = 64, 3000, 12
    teacher = _logits(T, V, "bf16", seed=11)
    teacher[::2, 100:] = -math.inf
    teacher[3, 5:] = -math.inf                # five tokens left, twelve asked for
    best = ctx.token_logprobs(teacher, top=k, want_entropy=False)
    student = _logits(T, V, "f32", seed=12).requires_grad_(False)
    got = ctx.distill(student, best["top_ids"], best["top_logp"], temperature=2.0)
    _check_distill(got, student, best["top_ids"].cpu().numpy(), best["top_logp"].cpu().numpy(),
                   2.0, None, "f32")
    # gradient steps on the logits lower the loss of every row (KL is convex in
    # z with curvature at most 1/2, and the step is below 2 / (1/2))
    z = student.clone()
    for _ in range(5):
        step = ctx.distill(z, best["top_ids"], best["top_logp"], temperature=1.0)
        z -= step["dZ"]
    after = ctx.distill(z, best["top_ids"], best["top_logp"], temperature=1.0, want_grad=False)
    assert (after["loss"] < step["loss"]).all()


def test_vocab_calls_in_a_graph_and_on_another_stream(ctx):
    T, V, k = 20, 7001, 6
    Z = _logits(T, V, "bf16", seed=3)
    ids, vals = _teacher(T, V, k, 3)
    di, dv, _ = _dev(ids, vals)
    tok = torch.arange(T, dtype=torch.int32, device="cuda")
    want = {**ctx.token_logprobs(Z, tok, top=4), **ctx.distill(Z, di, dv)}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = dust.Context(0, stream=side)
    with torch.cuda.stream(side):
        got = {**other.token_logprobs(Z, tok, top=4), **other.distill(Z, di, dv)}
    for name in want:
        assert torch.equal(want[name], got[name]), name
    static = {name: torch.zeros_like(v) for name, v in want.items()}
    scores = {n: static[n] for n in ("logp", "entropy", "top_ids", "top_logp")}
    grads = {n: static[n] for n in ("loss", "dZ")}
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ctx.token_logprobs(Z, tok, top=4, out=scores, asynchronous=True)
        ctx.distill(Z, di, dv, out=grads, asynchronous=True)
    for _ in range(2):
        for v in static.values():
            v.zero_()
        g.replay()
        torch.cuda.synchronize()
        for name in want:
            assert torch.equal(want[name], static[name]), name
    ctx.check()
    other.close()


def test_vocab_offsets_past_32_bits(ctx):
    # the last rows lie more than 2^31 elements into the logits
    T, V, k = 17000, 128256, 5
    Z = torch.zeros(T, V, dtype=torch.bfloat16, device="cuda")
    last = _logits(6, V, "bf16", seed=4)
    Z[-6:] = last
    ids, vals = _teacher(6, V, k, 4, missing=False)
    di = torch.full((T, k), -1, dtype=torch.int32, device="cuda")
    dv = torch.zeros(T, k, device="cuda")
    di[-6:], dv[-6:] = _dev(ids, vals)[:2]
    got = ctx.token_logprobs(Z, torch.zeros(T, dtype=torch.int32, device="cuda"), top=3)
    want = ctx.token_logprobs(last, torch.zeros(6, dtype=torch.int32, device="cuda"), top=3)
    assert torch.equal(got["top_ids"][-6:], want["top_ids"])
    torch.testing.assert_close(got["logp"][-6:], want["logp"], rtol=1e-5, atol=1e-5)
    assert got["top_ids"][0].tolist() == [0, 1, 2]
    ref = ctx.distill(last, di[-6:].contiguous(), dv[-6:].contiguous())
    got = ctx.distill(Z, di, dv, out={"dZ": Z})
    # one CTA a row here and a cluster there: the row's sum in another order
    torch.testing.assert_close(got["loss"][-6:], ref["loss"], rtol=1e-5, atol=1e-5)
    torch.testing.assert_close(Z[-6:].float(), ref["dZ"].float(), rtol=2.0 ** -7, atol=1e-9)
    assert not got["loss"][:-6].any() and not Z[:64].any()


@pytest.mark.parametrize("every", [2, 3, 10])
def test_distill_with_periodic_padding(ctx, every):
    # more rows than resident CTAs, a mask of every n-th and of the first 700
    T, V, k = 1500, 2003, 4
    Z = _logits(T, V, "bf16", seed=every)
    ids, vals = _teacher(T, V, k, every)
    w = np.ones(T, dtype=np.float32)
    w[::every] = 0.0
    w[:700] = 0.0
    di, dv, dw = _dev(ids, vals, w)
    got = ctx.distill(Z, di, dv, weights=dw)
    _check_distill(got, Z, ids, vals, 1.0, w, "bf16")
    assert not got["dZ"][:700].any() and not got["loss"][:700].any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_distill_of_rows_far_apart(ctx, dtype):
    # the last position of every sequence: rows a whole sequence apart, whose
    # gradient is made without the room between them
    B, L, V, k = 5, 40, 3001, 6
    wide = _logits(B, L * V, dtype, seed=2)
    Z = wide.view(B, L, V)[:, -1]
    ids, vals = _teacher(B, V, k, 5)
    di, dv, _ = _dev(ids, vals)
    got = ctx.distill(Z, di, dv)
    _check_distill(got, Z, ids, vals, 1.0, None, dtype)
    room = got["dZ"].untyped_storage().nbytes()
    assert room <= B * (V + 8) * (4 if dtype == "f32" else 2)


def test_the_bound_stream_is_the_current_one(ctx, monkeypatch):
    # with torch's direct accessor of the stream's handle, and without it
    bound = []

    class Lib:
        def dust_set_stream(self, h, s):
            bound.append(getattr(s, "value", s) or 0)

    monkeypatch.setattr(ctx, "_L", Lib())
    side = torch.cuda.Stream()
    for accessor in (dust._raw_stream, None):
        monkeypatch.setattr(dust, "_raw_stream", accessor)
        ctx._bind_stream()
        with torch.cuda.stream(side):
            ctx._bind_stream()
    here = torch.cuda.current_stream().cuda_stream
    assert bound == [here, side.cuda_stream] * 2


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_distill_clusters_work_through_several_rows(ctx, dtype):
    # rows of two (bf16) and three (fp32) CTAs, about three to five live rows for
    # every cluster that is resident at once: the exchange of the CTAs' sums and
    # the copies of the next row take turns. Every fifth row is padding, and some
    # clusters get a run of it; rows of odd pitch, then the same in place.
    T, V, k = 450, 60001, 9
    Z = _logits(T, V, dtype, seed=7, pitch=V + 2, offset=1)
    ids, vals = _teacher(T, V, k, 8)
    w = np.linspace(0.5, 1.5, T).astype(np.float32)
    w[4::5] = 0.0
    w[60:110] = 0.0
    di, dv, dw = _dev(ids, vals, w)
    for _ in range(2):
        got = ctx.distill(Z, di, dv, weights=dw, temperature=1.3)
    _check_distill(got, Z, ids, vals, 1.3, w, dtype)
    assert not got["dZ"][60:110].any() and not got["loss"][60:110].any()
    again = ctx.distill(Z, di, dv, weights=dw, temperature=1.3, out={"dZ": Z})
    assert torch.equal(again["dZ"], got["dZ"]) and torch.equal(again["loss"], got["loss"])


@pytest.mark.parametrize("how", ["weight", "entry"])
@pytest.mark.parametrize("T,V", [(4000, 2003), (900, 60001)])
def test_distill_writes_zeros_for_every_row_left_out(ctx, T, V, how):
    # many more rows than CTAs, six of them live: the others hold NaN, before the
    # call and in the gradient's memory, and come out as zeros
    k = 5
    Z = torch.full((T, V), math.nan, dtype=torch.bfloat16, device="cuda")
    live = np.array([0, 3, T // 2, T // 2 + 1, T - 100, T - 1])
    Z[torch.from_numpy(live).cuda()] = _logits(6, V, "bf16", seed=4)
    ids, vals = _teacher(T, V, k, 4, missing=False)
    w = np.ones(T, dtype=np.float32)
    out = np.setdiff1d(np.arange(T), live)
    if how == "weight":
        w[out] = 0.0
    else:
        ids[out] = -1
    di, dv, dw = _dev(ids, vals, w)
    for dZ in (torch.full_like(Z, math.nan), Z):
        rows = Z[torch.from_numpy(live).cuda()].clone()
        got = ctx.distill(Z, di, dv, weights=dw, out={
            "dZ": dZ, "loss": torch.full((T,), math.nan, device="cuda")})
        gone = torch.from_numpy(out).cuda()
        assert not got["dZ"][gone].any() and not got["loss"][gone].any()
        kept = torch.from_numpy(live).cuda()
        _check_distill({"dZ": got["dZ"][kept], "loss": got["loss"][kept]}, rows, ids[live],
                       vals[live], 1.0, None, "bf16")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("tau", [0.25, 0.5, 1.0, 3.0])
@pytest.mark.parametrize("V", [300, 60001])
def test_distill_where_the_student_has_the_lowest_value(ctx, dtype, tau, V):
    # a kept token whose logit is the type's lowest value, a mask that is finite:
    # the loss is tau q 3.4e38, which fp32 holds (q is about 1e-6 for one such
    # entry, and 1 for all of them where tau < 1)
    T, k = 4, 5
    Z = _logits(T, V, dtype, seed=9)
    ids, vals = _teacher(T, V, k, 10, missing=False)
    vals[:, 1] = vals.max(1) - 14.0 * tau
    for t in range(T - 1):
        Z[t, ids[t, 1]] = torch.finfo(DT[dtype]).min
    if tau < 1.0:                             # the whole of the teacher's weight
        Z[0, ids[0]] = torch.finfo(DT[dtype]).min
    di, dv, _ = _dev(ids, vals)
    got = ctx.distill(Z, di, dv, temperature=tau)
    assert torch.isfinite(got["loss"]).all()
    _check_distill(got, Z, ids, vals, tau, None, dtype)
    only = ctx.distill(Z, di, dv, temperature=tau, want_grad=False)
    torch.testing.assert_close(only["loss"], got["loss"], rtol=2e-5, atol=2e-5 * tau ** 2)
