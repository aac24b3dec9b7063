"""Cases that measure the LM-head loss operators and the exact attention operators.

Operators: ``token_logprobs`` (log probabilities of given tokens, entropy, top alternatives),
``distill`` (loss and logit gradient against a teacher's top logits), ``attn_forward`` and
``attn_backward`` (causal attention over ragged sequences and its gradients).

``own`` false: plain torch arithmetic in fp32. ``own`` true: the library's calls.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # one decoding step of a few requests that report 20 alternatives: latency counts
        dict(name="logprobs_decode", op="logprobs", T=4, V=128256, pitch=128256, dtype="f32",
             top=20, masked=True),
        # scoring text: an odd vocabulary inside rows padded to the GEMM's width
        dict(name="logprobs_score", op="logprobs", T=8192, V=50257, pitch=50304, dtype="bf16",
             top=0, masked=False),
        # a teacher's pass that keeps its 64 best per token for a student
        dict(name="logprobs_teacher", op="logprobs", T=4096, V=128256, pitch=128256, dtype="f32",
             top=64, masked=False),
        # validation loss of a student, no gradient
        dict(name="distill_eval", op="distill", T=1000, V=50304, pitch=50304, dtype="f32", k=16,
             tau=1.0, grad=False, weighted=False),
        # a student's training step over a padded batch
        dict(name="distill_step", op="distill", T=8192, V=50304, pitch=50304, dtype="bf16", k=32,
             tau=2.0, grad=True, weighted=True),
        # the same with a large vocabulary and fp32 logits
        dict(name="distill_large_vocab", op="distill", T=2048, V=128256, pitch=128256,
             dtype="f32", k=64, tau=1.0, grad=True, weighted=True),
        # the attention-internals workload's own shape and type: 8 sequences of 1024
        dict(name="attn_fwd_f32", op="attn", back=False, lengths="1024," * 7 + "1024", heads=12,
             kv_heads=12, d_h=64, dtype="f32", fused=False),
        # packed sequences, grouped heads, slices of one fused projection
        dict(name="attn_fwd_grouped", op="attn", back=False, lengths="3000,2500,1692,1000",
             heads=16, kv_heads=4, d_h=128, dtype="bf16", fused=True),
        # a handful of short prompts: latency counts
        dict(name="attn_bwd_short", op="attn", back=True, lengths="1,37,200,130", heads=4,
             kv_heads=4, d_h=64, dtype="bf16", fused=False),
        # the exact gradient beside the attention-internals estimator, in its own type
        dict(name="attn_bwd_f32", op="attn", back=True, lengths="1024," * 7 + "1024", heads=12,
             kv_heads=12, d_h=64, dtype="f32", fused=False),
        # the same training shape in bf16
        dict(name="attn_bwd_bf16", op="attn", back=True, lengths="1024," * 7 + "1024", heads=12,
             kv_heads=12, d_h=64, dtype="bf16", fused=False),
        # long packed sequences with shared key/value heads
        dict(name="attn_bwd_grouped", op="attn", back=True, lengths="3000,2500,1692,1000",
             heads=16, kv_heads=4, d_h=128, dtype="bf16", fused=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["logprobs", "distill", "attn", "attn"])
    dtype = rng.choice(["f32", "bf16"])
    if op in ("logprobs", "distill"):
        V = _log_int(rng, 1000, 131072)
        T = _log_int(rng, 1, max(1, min(8192, 200_000_000 // V)))
        case = dict(op=op, T=T, V=V, pitch=V + rng.choice([0, 0, 1, 7, 47]), dtype=dtype)
        if op == "logprobs":
            case.update(top=rng.choice([0, 1, 5, 20, 64, 128]), masked=rng.random() < 0.5)
        else:
            case.update(k=rng.choice([1, 7, 16, 50, 64, 128]), tau=rng.choice([1.0, 0.7, 2.0]),
                        grad=rng.random() < 0.7, weighted=rng.random() < 0.5)
        return case
    d_h = rng.choice([32, 64, 64, 128, 128])
    kv_heads = rng.choice([1, 2, 4])
    heads = kv_heads * rng.choice([1, 1, 2, 4])
    n = rng.randint(1, 6)
    longest = _log_int(rng, 16, 1500 if dtype == "f32" else 3000)
    lengths = [longest] + [rng.randint(1, longest) for _ in range(n - 1)]
    rng.shuffle(lengths)
    return dict(op="attn", back=rng.random() < 0.7, lengths=",".join(map(str, lengths)),
                heads=heads, kv_heads=kv_heads, d_h=d_h, dtype=dtype, fused=rng.random() < 0.5)


# ---- inputs -----------------------------------------------------------------------


def _logits(case, gen):
    """Logits of a head: normal around a per-token offset, a few likely tokens well above the
    rest, in rows of `pitch` of which the first V columns are the vocabulary."""
    T, V, pitch = case["T"], case["V"], case["pitch"]
    z = torch.randn(T, pitch, generator=gen, device="cuda")
    z.mul_(1.5).add_(torch.randn(T, 1, generator=gen, device="cuda"))
    likely = torch.randint(0, V, (T, 12), generator=gen, device="cuda")
    z.scatter_add_(1, likely, 6.0 * torch.rand(T, 12, generator=gen, device="cuda"))
    return z.to(DTYPES[case["dtype"]])


def _prepare_logprobs(case, gen):
    T, V = case["T"], case["V"]
    z = _logits(case, gen)
    tokens = torch.randint(0, V, (T,), generator=gen, device="cuda", dtype=torch.int32)
    if case["masked"]:
        # a vocabulary mask over a third of the tokens, and padding rows without a token
        out = torch.rand(z.shape, generator=gen, device="cuda") < 0.33
        out.scatter_(1, tokens.long()[:, None], False)
        z.masked_fill_(out, -math.inf)
        if T > 8:
            tokens[::9] = -1
    return dict(case=case, Z=z[:, :V], tokens=tokens)


def _prepare_distill(case, gen):
    T, V, k = case["T"], case["V"], case["k"]
    z = _logits(case, gen)
    # the teacher is like the student but not the same, and keeps its best k
    ids, vals = [], []
    step = max(1, 100_000_000 // V)
    for a in range(0, T, step):
        t = z[a:a + step, :V].float()
        t = t + 0.5 * torch.randn(t.shape, generator=gen, device="cuda")
        v, i = torch.topk(t, k, dim=1)
        vals.append(v)
        ids.append(i.to(torch.int32))
    ids, vals = torch.cat(ids), torch.cat(vals)
    if k > 8:  # some rows have kept fewer
        ids[::5, k - 3:] = -1
    w = None
    if case["weighted"]:  # the mean over the tokens that count; every tenth is padding
        w = torch.ones(T, device="cuda")
        w[9::10] = 0.0
        w /= w.sum()
    return dict(case=case, Z=z[:, :V], ids=ids, vals=vals, w=w, tau=case["tau"])


def _prepare_attn(case, gen):
    lens = [int(x) for x in case["lengths"].split(",")]
    H, G, d_h, dt = case["heads"], case["kv_heads"], case["d_h"], DTYPES[case["dtype"]]
    T, L = sum(lens), max(lens)
    if case["fused"]:
        qkv = torch.randn(T, (H + 2 * G) * d_h, generator=gen, device="cuda").to(dt)
        q, k, v = qkv.split([H * d_h, G * d_h, G * d_h], dim=1)
    else:
        q, k, v = (torch.randn(T, n * d_h, generator=gen, device="cuda").to(dt)
                   for n in (H, G, G))
    n = torch.tensor(lens, device="cuda")
    cu = torch.zeros(len(lens) + 1, dtype=torch.int32, device="cuda")
    cu[1:] = torch.cumsum(n, 0)
    # plain form only: the padded batch's row indexes and which of them are tokens
    pos = torch.arange(L, device="cuda")[None, :]
    valid = pos < n[:, None]
    index = (cu[:-1, None].long() + pos).clamp_(max=T - 1)
    state = dict(case=case, Q=q, K=k, V=v, cu=cu, L=L, H=H, G=G, index=index, valid=valid)
    if case["back"]:
        state["E"] = torch.randn(T, H * d_h, generator=gen, device="cuda").to(dt)
        state["O"], state["lse"] = _plain_attn_forward(state)
    return state


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return {"logprobs": _prepare_logprobs, "distill": _prepare_distill,
            "attn": _prepare_attn}[case["op"]](case, gen)


# ---- plain forms ------------------------------------------------------------------


def _plain_logprobs(s):
    z = s["Z"].float()
    V, top = z.shape[1], s["case"]["top"]
    x = z - z.amax(1, keepdim=True)
    e = torch.exp(x)
    total = e.sum(1)
    log_total = torch.log(total)
    tok = s["tokens"].long()
    logp = x.gather(1, tok.clamp(min=0)[:, None])[:, 0] - log_total
    out = {"logp": torch.where(tok >= 0, logp, 0.0),
           "entropy": log_total - torch.where(e > 0, e * x, 0.0).sum(1) / total}
    if top:
        # order by value, then by the lower index: both in one 64-bit key
        bits = (z + 0.0).contiguous().view(torch.int32)
        key = torch.where(bits >= 0, bits, bits ^ 0x7FFFFFFF).long()
        key = key * 2 ** 32 + (2 ** 32 - 1 - torch.arange(V, device=z.device))
        best = torch.topk(key, top, dim=1, sorted=True).values
        ids = 2 ** 32 - 1 - (best & 0xFFFFFFFF)
        out["top_ids"] = ids.to(torch.int32)
        out["top_logp"] = x.gather(1, ids) - log_total[:, None]
    return out


def _plain_distill(s):
    z = s["Z"].float() / s["tau"]
    there = s["ids"] >= 0
    ids = s["ids"].long().clamp(min=0)
    v = torch.where(there, s["vals"].float() / s["tau"], -math.inf)
    v = v - v.amax(1, keepdim=True)
    log_q = v - torch.log(torch.exp(v).sum(1, keepdim=True))
    q = torch.exp(log_q)
    x = z - z.amax(1, keepdim=True)
    e = torch.exp(x)
    total = e.sum(1, keepdim=True)
    log_p = x.gather(1, ids) - torch.log(total)
    out = {"loss": s["tau"] ** 2 * torch.where(q > 0, q * (log_q - log_p), 0.0).sum(1)}
    if s["w"] is not None:  # padding is left out
        out["loss"] = torch.where(s["w"] != 0, out["loss"], 0.0)
    if s["case"]["grad"]:
        g = e / total
        g.scatter_add_(1, ids, -q)
        g *= s["tau"] if s["w"] is None else s["tau"] * s["w"][:, None]
        out["dZ"] = g.to(s["Z"].dtype)
    return out


def _padded(s, t, heads):
    """T x (heads d_h) rows as batch x key/value heads x group x L x d_h, zero past the ends."""
    d_h, G = s["case"]["d_h"], s["G"]
    p = torch.where(s["valid"][..., None], t.float()[s["index"]], 0.0)
    return p.view(*s["index"].shape, G, heads // G, d_h).permute(0, 2, 3, 1, 4)


def _rows(s, p):
    """The way back, rounded to the inputs' type."""
    return p.permute(0, 3, 1, 2, 4).flatten(2)[s["valid"]].to(s["Q"].dtype)


def _plain_probs(s, q, k):
    L = s["L"]
    scores = q @ k.transpose(-1, -2) / math.sqrt(s["case"]["d_h"])
    future = torch.ones(L, L, dtype=torch.bool, device=q.device).triu(1)
    scores.masked_fill_(future, -math.inf)
    m = scores.amax(-1, keepdim=True)
    e = torch.exp(scores - m)
    total = e.sum(-1, keepdim=True)
    return e / total, (m + torch.log(total))[..., 0]


def _plain_attn_forward(s):
    q, k, v = _padded(s, s["Q"], s["H"]), _padded(s, s["K"], s["G"]), _padded(s, s["V"], s["G"])
    p, lse = _plain_probs(s, q, k)
    return _rows(s, p @ v), lse.permute(0, 3, 1, 2).flatten(2)[s["valid"]].contiguous()


def _plain_attn_backward(s):
    q, k, v = _padded(s, s["Q"], s["H"]), _padded(s, s["K"], s["G"]), _padded(s, s["V"], s["G"])
    e = _padded(s, s["E"], s["H"])
    p, _ = _plain_probs(s, q, k)
    dp = e @ v.transpose(-1, -2)
    ds = p * (dp - (p * dp).sum(-1, keepdim=True)) / math.sqrt(s["case"]["d_h"])
    dq = ds @ k
    dk = (ds.transpose(-1, -2) @ q).sum(2, keepdim=True)
    dv = (p.transpose(-1, -2) @ e).sum(2, keepdim=True)
    return {"dQ": _rows(s, dq), "dK": _rows(s, dk), "dV": _rows(s, dv)}


# ---- one pass ---------------------------------------------------------------------


def run(state):
    s, case = state, state["case"]
    if own:
        import zeroth_order_transformer_dust_b200 as dust
        if case["op"] == "logprobs":
            return dust.token_logprobs(s["Z"], s["tokens"], top=case["top"], asynchronous=True)
        if case["op"] == "distill":
            return dust.distill(s["Z"], s["ids"], s["vals"], temperature=s["tau"],
                                weights=s["w"], want_grad=case["grad"], asynchronous=True)
        shape = dict(n_heads=s["H"], n_kv_heads=s["G"], cu_seqlens=s["cu"], max_len=s["L"],
                     asynchronous=True)
        if case["back"]:
            return dust.attn_backward(s["Q"], s["K"], s["V"], s["O"], s["lse"], s["E"], **shape)
        return dust.attn_forward(s["Q"], s["K"], s["V"], **shape)
    if case["op"] == "logprobs":
        return _plain_logprobs(s)
    if case["op"] == "distill":
        return _plain_distill(s)
    if case["back"]:
        return _plain_attn_backward(s)
    o, lse = _plain_attn_forward(s)
    return {"O": o, "lse": lse}


def work(case):
    b = 4 if case["dtype"] == "f32" else 2
    if case["op"] in ("logprobs", "distill"):
        T, n = case["T"], case["T"] * case["V"]
        if case["op"] == "logprobs":
            return {"bytes": n * b + T * (12 + 8 * case["top"]), "flops": 6 * n}
        # padding rows are not read, their gradient is written as zeros
        live = n - (T // 10 * case["V"] if case["weighted"] else 0)
        back = n if case["grad"] else 0
        return {"bytes": (live + back) * b + T * (8 * case["k"] + 8),
                "flops": 4 * live * (2 if back else 1)}
    lens = [int(x) for x in case["lengths"].split(",")]
    T, H, G, d_h = sum(lens), case["heads"], case["kv_heads"], case["d_h"]
    pairs = sum(n * (n + 1) // 2 for n in lens)
    if case["back"]:  # Q, O, E, dQ; K, V, dK, dV; lse; five products over the causal half
        return {"bytes": T * d_h * b * 4 * (H + G) + 4 * T * H, "flops": 10 * pairs * H * d_h}
    return {"bytes": T * d_h * b * 2 * (H + G) + 4 * T * H, "flops": 4 * pairs * H * d_h}


# ---- the definitions in 64 bits -----------------------------------------------------


def _exact_logprobs(s):
    outs = []
    for a in range(0, s["Z"].shape[0], 256):
        z = s["Z"][a:a + 256].double()
        tok = s["tokens"][a:a + 256].long()
        lp = torch.log_softmax(z, dim=1)
        d = {"logp": torch.stack([r[t] if t >= 0 else r.new_zeros(()) for r, t in
                                  zip(lp, tok.tolist())]),
             "entropy": torch.special.entr(lp.exp()).sum(1)}
        if s["case"]["top"]:
            order = torch.sort(z, dim=1, descending=True, stable=True).indices[:, :s["case"]["top"]]
            d["top_ids"] = order.to(torch.int32)
            d["top_logp"] = torch.take_along_dim(lp, order, 1)
        outs.append(d)
    return {name: torch.cat([d[name] for d in outs]) for name in outs[0]}


def _exact_distill(s):
    losses, grads = [], []
    for a in range(0, s["Z"].shape[0], 256):
        z = s["Z"][a:a + 256].double().requires_grad_(s["case"]["grad"])
        ids, vals = s["ids"][a:a + 256].long(), s["vals"][a:a + 256].double()
        q = torch.softmax(torch.where(ids >= 0, vals / s["tau"], -math.inf), dim=1)
        lp = torch.take_along_dim(torch.log_softmax(z / s["tau"], dim=1), ids.clamp(min=0), 1)
        loss = s["tau"] ** 2 * (torch.xlogy(q, q) - q * lp).sum(1)
        if s["case"]["grad"]:
            w = torch.ones_like(loss) if s["w"] is None else s["w"][a:a + 256].double()
            grads.append(torch.autograd.grad((loss * w).sum(), z)[0])
        if s["w"] is not None:
            loss = loss * (s["w"][a:a + 256] != 0)
        losses.append(loss.detach())
    out = {"loss": torch.cat(losses)}
    if grads:
        out["dZ"] = torch.cat(grads)
    return out


def _exact_attn(s):
    H, G, d_h, back = s["H"], s["G"], s["case"]["d_h"], s["case"]["back"]
    cu = s["cu"].tolist()
    parts = []
    for a, b in zip(cu[:-1], cu[1:]):
        q, k, v = (t[a:b].double().requires_grad_(back) for t in (s["Q"], s["K"], s["V"]))
        n = b - a
        qh = q.view(n, H, d_h).transpose(0, 1)
        kh, vh = (t.view(n, G, d_h).transpose(0, 1).repeat_interleave(H // G, 0) for t in (k, v))
        sc = torch.matmul(qh, kh.mT) * d_h ** -0.5
        sc = sc + torch.full((n, n), -math.inf, dtype=sc.dtype, device=sc.device).triu(1)
        o = torch.matmul(torch.softmax(sc, -1), vh).transpose(0, 1).reshape(n, H * d_h)
        if back:
            dq, dk, dv = torch.autograd.grad(o, (q, k, v), s["E"][a:b].double())
            parts.append({"dQ": dq, "dK": dk, "dV": dv})
        else:
            parts.append({"O": o, "lse": torch.logsumexp(sc, -1).T})
    return {name: torch.cat([p[name] for p in parts]) for name in parts[0]}


def exact(case, seed):
    s = prepare(case, seed)
    return {"logprobs": _exact_logprobs, "distill": _exact_distill,
            "attn": _exact_attn}[case["op"]](s)
