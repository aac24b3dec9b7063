"""The binding and the C-ABI refuse bad calls of the exact losses and attention
before anything reaches a kernel (no GPU)."""
import ctypes

import pytest
import torch

import zeroth_order_transformer_dust_b200 as dust
from zeroth_order_transformer_dust_b200 import build

f32, bf16, i32 = torch.float32, torch.bfloat16, torch.int32


def _t(*shape, dtype=f32):
    return torch.zeros(*shape, dtype=dtype)


class _FakeLib:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        if not name.startswith("dust_"):
            raise AttributeError(name)

        def fn(*args):
            self.calls.append((name, args))
            return 0
        return fn


def _fake_context():
    c = dust.Context.__new__(dust.Context)
    c._L = _FakeLib()
    c.device = None                       # outputs live in host memory here
    c._h = ctypes.c_void_p(1)
    c._stream = None
    c._bind_stream = lambda: None
    c._dev = c._cuda = lambda t, name: t  # host tensors stand in for device ones
    return c


def _value(arg):
    return arg.value if isinstance(arg, ctypes.c_void_p) else arg


def test_row_strides():
    assert dust._row_stride(_t(4, 6), "x") == 6
    assert dust._row_stride(_t(4, 9)[:, 2:8], "x") == 9
    assert dust._row_stride(_t(1, 6).expand(1, 6), "x") == 6
    for bad in (_t(6, 4).t(), _t(4, 12)[:, ::2], _t(1, 6).expand(4, 6), _t(24)):
        with pytest.raises(ValueError):
            dust._row_stride(bad, "x")


def test_logprobs_call():
    c = _fake_context()
    Z, tok = _t(5, 40)[:, 3:33], _t(5, dtype=i32)
    out = c.token_logprobs(Z, tok, top=4)
    (name, a), = c._L.calls
    assert name == "dust_token_logprobs"
    assert a[1:4] == (5, 30, dust.DUST_F32) and a[5] == 40 and a[7] == 4 and a[12] == 0
    assert _value(a[4]) == Z.data_ptr() and _value(a[6]) == tok.data_ptr()
    assert [(k, tuple(v.shape), v.dtype) for k, v in out.items()] == [
        ("logp", (5,), f32), ("entropy", (5,), f32), ("top_ids", (5, 4), i32),
        ("top_logp", (5, 4), f32)]
    out = c.token_logprobs(Z.to(bf16), want_entropy=False, top=1, asynchronous=True)
    a = c._L.calls[-1][1]
    assert a[3] == dust.DUST_BF16 and a[6] is None and a[8] is None and a[9] is None
    assert a[12] == dust.FLAG_ASYNC and set(out) == {"top_ids", "top_logp"}
    n = len(c._L.calls)
    for kw in (dict(top=31), dict(top=-1), dict(top=2, out={"top_ids": _t(5, 2)}),
               dict(top=2, out={"top_ids": _t(5, 3, dtype=i32)}), dict(out={"logp": _t(10)[::2]})):
        with pytest.raises(ValueError):
            c.token_logprobs(Z, tok, **kw)
    with pytest.raises(ValueError):
        c.token_logprobs(Z, _t(4, dtype=i32))
    with pytest.raises(TypeError):
        c.token_logprobs(Z.double(), tok)
    assert len(c._L.calls) == n


def test_distill_call():
    c = _fake_context()
    Z, ids, vals = _t(5, 40, dtype=bf16)[:, :30], _t(5, 7, dtype=i32), _t(5, 7)
    out = c.distill(Z, ids, vals, temperature=2.0, weights=_t(5))
    (name, a), = c._L.calls
    assert name == "dust_distill" and a[1:4] == (5, 30, dust.DUST_BF16)
    assert a[5] == 40 and a[8] == 7 and a[9] == 2.0 and a[13] == 40
    assert out["dZ"].stride(0) == 40 and tuple(out["dZ"].shape) == (5, 30)
    assert out["dZ"].dtype == bf16 and tuple(out["loss"].shape) == (5,)
    dst = _t(5, 64, dtype=bf16)[:, 1:31]
    assert c.distill(Z, ids, vals, out={"dZ": dst})["dZ"] is dst
    assert c._L.calls[-1][1][13] == 64
    out = c.distill(Z, ids, vals, want_grad=False)
    assert set(out) == {"loss"} and c._L.calls[-1][1][12] is None
    n = len(c._L.calls)
    for bad in (dict(weights=_t(4)), dict(out={"dZ": _t(5, 30)}), dict(out={"loss": _t(6)}),
                dict(out={"dZ": _t(30, 5, dtype=bf16).t()})):
        with pytest.raises(ValueError):
            c.distill(Z, ids, vals, **bad)
    for args in ((Z, ids, _t(5, 6)), (Z, ids[:4], vals)):
        with pytest.raises(ValueError):
            c.distill(*args)
    for args in ((Z, ids.long(), vals), (Z, ids, vals.double())):
        with pytest.raises(TypeError):
            c.distill(*args)
    assert len(c._L.calls) == n


def test_attention_calls():
    c = _fake_context()
    T, H, G, dh = 12, 4, 2, 64
    qkv = _t(T, (H + 2 * G) * dh, dtype=bf16)
    q, k, v = qkv.split([H * dh, G * dh, G * dh], 1)
    cu = torch.tensor([0, 5, 12], dtype=i32)
    f = c.attn_forward(q, k, v, n_heads=H, n_kv_heads=G, cu_seqlens=cu, max_len=7, scale=0.5)
    name, a = c._L.calls[-1]
    d = a[1]._obj
    assert name == "dust_attn_forward"
    assert (d.T, d.n_seqs, d.max_len, d.n_heads, d.n_kv_heads, d.head_dim, d.dtype, d.scale) == (
        T, 2, 7, H, G, dh, dust.DUST_BF16, 0.5)
    assert (d.ldq, d.ldk, d.ldv, d.ldo) == (512, 512, 512, 256) and d.cu_seqlens == cu.data_ptr()
    assert tuple(f["O"].shape) == (T, H * dh) and tuple(f["lse"].shape) == (T, H)
    g = c.attn_backward(q, k, v, f["O"], f["lse"], _t(T, H * dh, dtype=bf16), n_heads=H,
                        n_kv_heads=G, seq_len=6, asynchronous=True)
    name, a = c._L.calls[-1]
    d = a[1]._obj
    assert name == "dust_attn_backward" and len(a) == 12
    assert (d.n_seqs, d.max_len, d.scale, d.flags, d.cu_seqlens) == (2, 6, 0.0, 2, None)
    assert {n: tuple(x.shape) for n, x in g.items()} == {
        "dQ": (T, 256), "dK": (T, 128), "dV": (T, 128)}
    n = len(c._L.calls)
    for kw in (dict(n_heads=3), dict(n_heads=H), dict(n_heads=H, n_kv_heads=G, seq_len=5),
               dict(n_heads=H, n_kv_heads=G, scale=0.0),
               dict(n_heads=H, n_kv_heads=G, seq_len=6, cu_seqlens=cu),
               dict(n_heads=H, n_kv_heads=G, seq_len=6, max_len=5),
               dict(n_heads=H, n_kv_heads=G, out={"O": _t(T, 256)})):
        with pytest.raises(ValueError):
            c.attn_forward(q, k, v, **kw)
    with pytest.raises(TypeError):
        c.attn_forward(q, k.float(), v, n_heads=H, n_kv_heads=G)
    with pytest.raises(TypeError):
        c.attn_forward(q, k, v, n_heads=H, n_kv_heads=G, cu_seqlens=cu.long())
    assert len(c._L.calls) == n


def test_null_contexts_and_struct_layout():
    build.build()
    L = dust.load_library()
    assert L.dust_token_logprobs(None, 1, 1, 0, None, 1, None, 0, None, None, None, None, 0) == 1
    assert L.dust_distill(None, 1, 1, 0, None, 1, None, None, 1, 1.0, None, None, None, 1, 0) == 1
    d = dust.DustAttnDims()
    assert L.dust_attn_forward(None, ctypes.byref(d), *[None] * 6) == 1
    assert L.dust_attn_backward(None, ctypes.byref(d), *[None] * 10) == 1
    assert L.dust_attn_work_bytes(ctypes.byref(d), 0) == -1
    d = dust.DustAttnDims(T=100, n_seqs=1, max_len=100, n_heads=4, n_kv_heads=2, head_dim=64,
                          dtype=dust.DUST_BF16)
    assert [L.dust_attn_work_bytes(ctypes.byref(d), b) for b in (0, 1)] == [0, 1792]
    d.dtype = dust.DUST_F32       # three bf16 planes of Q, K, V (and E)
    assert [L.dust_attn_work_bytes(ctypes.byref(d), b) for b in (0, 1)] == [
        100 * 64 * 6 * 8, 100 * 64 * 6 * 12 + 1792]
    # int64, pointer, int32 x6, float, uint32, int64 x8
    assert ctypes.sizeof(d) == 112 and dust.DustAttnDims.ldq.offset == 48
    assert dust.DustAttnDims.scale.offset == 40


def test_scale_that_fp32_does_not_hold():
    # the struct's scale is fp32, where 0 stands for the default
    c = _fake_context()
    x = _t(6, 64)
    for scale in (1e-50, 1e-46, 0.0, -1e-50, float("nan")):
        with pytest.raises(ValueError, match="scale"):
            c.attn_forward(x, x, x, n_heads=1, scale=scale)
        with pytest.raises(ValueError, match="scale"):
            c.attn_backward(x, x, x, x, _t(6, 1), x, n_heads=1, scale=scale)
    assert not [name for name, _ in c._L.calls if name != "dust_attn_work_bytes"]
    c.attn_forward(x, x, x, n_heads=1, scale=1e-44)
    assert c._L.calls[-1][1][1]._obj.scale > 0.0


def test_distill_makes_its_gradient_without_the_room_between_rows():
    # rows far apart: V wide, each as far from a 16-byte boundary as Z's
    c = _fake_context()
    ids, vals = _t(3, 4, dtype=i32), _t(3, 4)
    for dtype, step in ((f32, 4), (bf16, 8)):
        for V, ld in ((1001, 50007), (1001, 1001 + 257), (4096, 1 << 20)):
            Z = torch.zeros(3 * ld, dtype=dtype).view(3, ld)[:, :V]
            dZ = c.distill(Z, ids, vals)["dZ"]
            assert tuple(dZ.shape) == (3, V) and dZ.dtype == dtype
            assert dZ.stride(0) < V + step and (dZ.stride(0) - ld) % step == 0
            assert c._L.calls[-1][1][13] == dZ.stride(0)
        Z = torch.zeros(3, 1257, dtype=dtype)[:, :1001]     # a GEMM's padding is kept
        assert c.distill(Z, ids, vals)["dZ"].stride(0) == 1257


def test_streams_without_the_direct_accessor(monkeypatch):
    # torch's accessor of a stream's handle is not part of its documented
    # interface: where it is missing, the documented one is used
    c = _fake_context()
    del c._bind_stream
    c.device = 3
    asked = []

    class Stream:
        cuda_stream = 77

    monkeypatch.setattr(torch.cuda, "current_stream", lambda d: asked.append(d) or Stream())
    monkeypatch.setattr(dust, "_raw_stream", None)
    c._bind_stream()
    assert asked == [3] and _value(c._L.calls[-1][1][1]) == 77
    monkeypatch.setattr(dust, "_raw_stream", lambda d: 10 + d)
    c._bind_stream()
    assert asked == [3] and _value(c._L.calls[-1][1][1]) == 13
    c._stream = Stream()
    c._bind_stream()
    assert _value(c._L.calls[-1][1][1]) == 77


def test_packed_rows_beyond_the_longest_sequence():
    # many packed rows, no max_len: the default stays within what a sequence may have
    c = _fake_context()
    T = (1 << 22) + 5
    x = torch.zeros(1, 64, dtype=bf16).expand(T, 64)
    cu = torch.tensor([0, 9, T], dtype=i32)
    dims = dust._exact_attn_dims(_Rows(x), _Rows(x), _Rows(x), 1, None, None, cu, None, None)
    assert (dims.T, dims.n_seqs, dims.max_len) == (T, 2, 1 << 22)
    dims = dust._exact_attn_dims(_Rows(x), _Rows(x), _Rows(x), 1, None, None, cu, 77, None)
    assert dims.max_len == 77
    small = _t(6, 64)
    c.attn_forward(small, small, small, n_heads=1, cu_seqlens=torch.tensor([0, 6], dtype=i32))
    assert c._L.calls[-1][1][1]._obj.max_len == 6


class _Rows:
    """Stands in for a contiguous 2-D tensor of many rows without its memory."""

    def __init__(self, like):
        self.shape, self.dtype = like.shape, like.dtype

    def dim(self):
        return 2

    def is_contiguous(self):
        return True
