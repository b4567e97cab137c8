"""The 8-bit operators without a GPU: the references' own pins, and every refusal of the C entry
points and of the binding (each before any device work)."""

import ctypes

import pytest
import torch

import q8_ref as R
import qwen2_decode_step_b200 as q2

F = ctypes.c_float


def test_reference_encode_is_torchs_e4m3_cast():
    gen = torch.Generator().manual_seed(1)
    x = torch.cat([torch.randn(20000, generator=gen) * 100, torch.randn(20000, generator=gen) * 0.01,
                   torch.tensor([0.0, -0.0, 448.0, 464.0, -465.0, 2.0 ** -10, 2.0 ** -11, 3 * 2.0 ** -10])])
    want = x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    assert torch.equal(R.encode(x.double()), want)
    codes = torch.arange(256, dtype=torch.uint8)
    assert torch.equal(R.value(codes).nan_to_num(9e9), codes.view(torch.float8_e4m3fn).double().nan_to_num(9e9))


def test_reference_block_scale():
    assert R.block_scale(448.0) == 1.0 and R.block_scale(448.1) == 2.0 and R.block_scale(224.0) == 0.5
    assert R.block_scale(0.0) == 2.0 ** -60 and R.block_scale(3.3e38) == 2.0 ** 119


def test_reference_append_of_a_growing_block_stays_within_half_a_step_twice():
    gen = torch.Generator().manual_seed(2)
    codes, scales = torch.zeros(1, 1, 70, 32, dtype=torch.uint8), torch.zeros(1, 1, 2)
    x = torch.randn(1, 60, 1, 32, generator=gen) * torch.logspace(-2, 2, 60)[None, :, None, None]
    for t in range(60):
        R.append(codes, scales, x[:, t:t + 1], [t])
    y = R.dense(codes, scales)[0, 0, :60]
    s = float(scales[0, 0, 0])
    # one rounding when written (2^-4 of the value), later ones only among the subnormals (half
    # of 2^-9 of the scale each, at most log2 of the growth of them, halving backwards)
    assert ((y - x[0, :, 0].double()).abs() <= 2.0 ** -4 * x[0, :, 0].abs() + 2 * 2.0 ** -10 * s).all()


def _raw(name, *args):
    return getattr(q2.lib(), name)(*args)


def _append(kc=16, vc=16, ks=16, vs=16, k=16, v=16, start=16, batch=1, ntok=1, nkv=2, hd=128, max_seq=64, dtype=1):
    return _raw("q2_kv8_append", kc, vc, ks, vs, k, v, None, None, start, batch, ntok, nkv, hd, max_seq, dtype, None)


def _read(kc=16, vc=16, ks=16, vs=16, k=16, v=16, start=16, batch=1, ntok=1, nkv=2, hd=128, max_seq=64, dtype=1):
    return _raw("q2_kv8_read", k, v, kc, vc, ks, vs, start, batch, ntok, nkv, hd, max_seq, dtype, None)


@pytest.mark.parametrize("call", [_append, _read])
def test_cache_calls_refuse(call):
    assert call(dtype=2) == 2
    assert call(hd=96) == 3 and call(hd=0) == 3
    assert call(nkv=0) == 3 and call(max_seq=0) == 3 and call(batch=40000) == 3
    assert call(max_seq=1 << 31) == 3
    assert call(ntok=65) == 4                                  # past max_seq
    for p in ("kc", "vc", "ks", "vs", "k", "v", "start"):
        assert call(**{p: None}) == 1
    assert call(kc=24) == 1 and call(vc=8) == 1                # codes not on 16 bytes
    assert b"16-byte" in q2.lib().q2_last_error()
    assert call(batch=0, kc=None) == 0 and call(ntok=0, kc=None) == 0


def _attn(out=256, q=256, kc=256, vc=256, ks=256, vs=256, lens=256, batch=1, ntok=1, nh=12, nkv=2, hd=128,
          max_seq=64, dtype=1, ws=256, ws_bytes=1 << 40):
    return _raw("q2_kv8_attention", out, q, None, kc, vc, ks, vs, lens, batch, ntok, nh, nkv, hd, max_seq, F(1.0),
                dtype, ws, ws_bytes, None)


def _self(out=256, q=256, kc=256, vc=256, ks=256, vs=256, seqlen=1, total=1, nh=12, nkv=2, hd=128, max_seq=64,
          dtype=1, ws=256, ws_bytes=1 << 40):
    return _raw("q2_kv8_self_attention", out, q, kc, vc, ks, vs, seqlen, total, nh, nkv, hd, max_seq, F(1.0), dtype,
                ws, ws_bytes, None)


@pytest.mark.parametrize("call", [_attn, _self])
def test_attention_calls_refuse(call):
    assert call(dtype=5) == 2
    assert call(hd=48) == 3 and call(nh=13) == 3 and call(nkv=0) == 3 and call(nh=0) == 3
    assert call(nh=18) == 3                                    # nine query heads per kv head
    assert call(max_seq=0) == 3
    for p in ("out", "q", "kc", "vc", "ks", "vs"):
        assert call(**{p: None}) == 1
    assert call(kc=264) == 1 and call(vc=260) == 1
    assert call(out=264) == 1
    for bad in ({"ws": None}, {"ws": 300}, {"ws_bytes": 100}):
        assert call(max_seq=8192, **bad) == 1


def test_attention_length_refusals():
    assert _attn(ntok=65) == 4 and _attn(lens=None) == 1 and _attn(batch=40000) == 3
    assert _attn(batch=0, out=None) == 0 and _attn(ntok=0, out=None) == 0
    assert _self(seqlen=2, total=1) == 3 and _self(seqlen=1, total=65) == 4
    assert _self(seqlen=0, total=0, out=None) == 0


def test_attention_workspace_refusals():
    n = ctypes.c_size_t(0)
    assert _raw("q2_kv8_attention_workspace", 1, 1, 0, 13, 2, 128, 64, 1, ctypes.byref(n)) == 3
    assert _raw("q2_kv8_attention_workspace", 1, 1, 0, 12, 2, 128, 64, 7, ctypes.byref(n)) == 2
    assert _raw("q2_kv8_attention_workspace", 1, 1, 0, 12, 2, 128, 64, 1, None) == 1
    assert _raw("q2_kv8_attention_workspace", 2, 4, 64, 12, 2, 128, 64, 1, ctypes.byref(n)) == 3  # a total_len is one sequence's
    assert _raw("q2_kv8_attention_workspace", 1, 65, 64, 12, 2, 128, 64, 1, ctypes.byref(n)) == 3
    assert _raw("q2_kv8_attention_workspace", 0, 1, 0, 12, 2, 128, 64, 1, ctypes.byref(n)) == 0 and n.value == 0
    assert _raw("q2_kv8_attention_workspace", 1, 1, 0, 12, 2, 128, 64, 1, ctypes.byref(n)) == 0 and n.value == 0
    assert _raw("q2_kv8_attention_workspace", 1, 1, 0, 12, 2, 128, 4096, 1, ctypes.byref(n)) == 0 and n.value > 0


def test_attention_sizes_past_its_counters_are_refused():
    assert _attn(batch=32767, nkv=2, max_seq=1 << 20) == 3      # batch * nkv * max_seq
    assert _attn(batch=16, ntok=65535, max_seq=1 << 20) == 3    # times the row groups and blocks
    assert _self(seqlen=65536, total=65536, max_seq=1 << 20) == 3


def test_quantize_refuses():
    def call(codes=16, scales=16, x=16, rows=4, cols=256, stride=256, br=1, dtype=0):
        return _raw("q2_quantize_q8", codes, scales, x, rows, cols, stride, br, dtype, None)

    assert call(dtype=3) == 2 and call(br=64) == 1 and call(stride=255) == 3
    assert call(rows=1 << 31) == 3 and call(cols=1 << 23, stride=1 << 23) == 3
    for p in ("codes", "scales", "x"):
        assert call(**{p: None}) == 1
    assert call(rows=0, x=None) == 0 and call(cols=0, x=None) == 0


def test_linear_refuses():
    def call(out=16, xq=16, xs=16, wq=16, ws=16, M=4, N=4, K=128, dtype=1):
        return _raw("q2_linear_q8", out, xq, xs, wq, ws, None, M, N, K, dtype, None)

    assert call(dtype=3) == 2 and call(K=0) == 3 and call(K=120) == 3 and call(K=1 << 24) == 3
    assert call(M=1 << 31) == 3
    for p in ("out", "xq", "xs", "wq", "ws"):
        assert call(**{p: None}) == 1
    assert call(xq=20) == 1 and call(wq=24) == 1
    assert call(M=0, out=None) == 0 and call(N=0, out=None) == 0


def _cache(B=1, nkv=2, S=70, hd=32):
    nb = -(-S // 64)
    return (torch.zeros(B, nkv, S, hd, dtype=torch.uint8), torch.zeros(B, nkv, S, hd, dtype=torch.uint8),
            torch.ones(B, nkv, nb), torch.ones(B, nkv, nb))


def test_binding_refuses_wrong_tensors():
    kc, vc, ks, vs = _cache()
    k = torch.zeros(1, 3, 2, 32)
    start = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):  # CPU tensors
        q2.q2_kv8_append(kc, vc, ks, vs, k, k, start)
    with pytest.raises(ValueError):  # scales of another length
        q2.q2_kv8_append(kc, vc, ks[..., :1].contiguous(), vs, k, k, start)
    with pytest.raises(TypeError):   # start is int32
        q2.q2_kv8_append(kc, vc, ks, vs, k, k, start.long())
    with pytest.raises(TypeError):   # codes are bytes
        q2.q2_kv8_append(kc.float(), vc, ks, vs, k, k, start)
    with pytest.raises(TypeError):   # k and v of one type
        q2.q2_kv8_append(kc, vc, ks, vs, k, k.bfloat16(), start)
    with pytest.raises(ValueError):  # k of other heads
        q2.q2_kv8_read(k[:, :, :1].contiguous(), k, kc, vc, ks, vs, start)
    q = torch.zeros(1, 3, 4, 32)
    with pytest.raises(ValueError):
        q2.q2_kv8_attention(torch.zeros_like(q), q, kc, vc, ks, vs, start, 1.0)
    with pytest.raises(TypeError):
        q2.q2_kv8_attention(q.bfloat16(), q, kc, vc, ks, vs, start, 1.0)
    with pytest.raises(ValueError):
        q2.q2_kv8_self_attention(q[0], q[0], kc[0], vc[0], ks[0], vs[0][:, :1], 3, 1.0)
    with pytest.raises(ValueError):  # transposed rows
        q2.q2_quantize_q8(torch.zeros(4, 6, dtype=torch.uint8), torch.zeros(1, 4), torch.zeros(6, 4).t())
    with pytest.raises(ValueError):  # scales laid out [rows, groups]
        q2.q2_linear_q8(torch.zeros(3, 5), torch.zeros(3, 256, dtype=torch.uint8), torch.zeros(3, 2),
                        torch.zeros(5, 256, dtype=torch.uint8), torch.zeros(1, 2))


def test_token_strides_of_the_packed_projection():
    qkv = torch.zeros(2, 5, 8, 32)
    k = qkv[:, :, 4:6]
    s = q2._tok_strides(k)
    assert list(s) == [5 * 8 * 32, 8 * 32]
    assert q2._tok_strides(k.contiguous()) is None
    with pytest.raises(ValueError):
        q2._tok_strides(qkv[:, :, ::2])
