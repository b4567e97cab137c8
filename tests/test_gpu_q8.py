"""The 8-bit operators (e4m3 KV cache: append, read, attention; e4m3 linear: quantise, product)
against plain 64-bit references (q8_ref), at the sizes, lengths, masks, strides and values where
they can go wrong, and run together as they are used.  Written and quantised codes are compared
bit for bit; the bounds of the others count their roundings (q8_ref)."""

import math
import os
import subprocess
import sys

import pytest
import torch

import q8_ref as R
import qwen2_decode_step_b200 as q2

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(autouse=True)
def _gpu(cuda_ok):
    yield
    torch.cuda.synchronize()
    q2.q2_check_device_error()


def randn(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed))


def i32(v):
    return torch.tensor(v, dtype=torch.int32)


def same_codes(got, want, what):
    """Bit for bit, but for the sign of a NaN."""
    g = got.cpu().view(torch.uint8)
    same = (g == want) | ((g & 127 == 127) & (want & 127 == 127))
    assert bool(same.all()), f"{what}: {int((~same).sum())} codes differ, first at {(~same).nonzero()[0].tolist()}"


def empty_cache(B, nkv, S, hd, seed=0):
    """A cache of random bytes (NaN codes among them) and scales: nothing may lean on it."""
    g = torch.Generator().manual_seed(1000 + seed)
    nb = -(-S // 64)
    c = [torch.randint(0, 256, (B, nkv, S, hd), generator=g, dtype=torch.uint8) for _ in range(2)]
    s = [torch.full((B, nkv, nb), 2.0 ** 30) for _ in range(2)]
    return c[0], c[1], s[0], s[1]


def filled_cache(B, nkv, S, hd, seed, spread=1.0):
    """codes and scales of a full cache (the reference's), blocks of unequal size."""
    k = randn(seed, B, S, nkv, hd) * torch.exp(spread * randn(seed + 1, B, S, 1, 1))
    v = randn(seed + 2, B, S, nkv, hd) * torch.exp(spread * randn(seed + 3, B, S, 1, 1))
    kc, vc, ks, vs = empty_cache(B, nkv, S, hd, seed)
    R.append(kc, ks, k, [0] * B)
    R.append(vc, vs, v, [0] * B)
    return kc, vc, ks, vs


def both(*ts):
    return [t.cuda() for t in ts]


# ----------------------------------------------------------------- append and read

APPENDS = [  # hd, nkv, max_seq, ntok, starts
    (128, 2, 200, 1, [0, 63, 64, 130, 199]),
    (128, 1, 577, 300, [0, 37, 277]),
    (64, 3, 131, 65, [0, 1, 63, 64, 66]),
    (32, 8, 64, 64, [0]),
    (32, 2, 1, 1, [0]),
    (64, 1, 333, 2, [62, 63, 64, -1, 331]),
]


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("hd,nkv,S,T,starts", APPENDS)
def test_append(dt, hd, nkv, S, T, starts):
    B = len(starts)
    kc, vc, ks, vs = empty_cache(B, nkv, S, hd)
    hist = max(starts)
    if hist > 0:  # earlier positions, smaller than the new ones: scales have to grow
        old = 0.3 * randn(5, B, hist, nkv, hd)
        R.append(kc, ks, old, [0] * B)
        R.append(vc, vs, old.flip(0), [0] * B)
    x = randn(6, B, T, 2, nkv, hd).to(DT[dt])
    x[:, -1, 1] *= 7
    dev = both(kc, vc, ks, vs)
    q2.q2_kv8_append(*dev, *both(x[:, :, 0].contiguous(), x[:, :, 1].contiguous()), i32(starts).cuda())
    R.append(kc, ks, x[:, :, 0], starts)
    R.append(vc, vs, x[:, :, 1], starts)
    same_codes(dev[0], kc, "k")
    same_codes(dev[1], vc, "v")
    assert torch.equal(dev[2].cpu(), ks) and torch.equal(dev[3].cpu(), vs)


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("view", ["packed", "odd stride", "broadcast", "one byte off"])
def test_append_strided_rows(dt, view):
    B, T, nkv, hd, S = 3, 70, 2, 64, 150
    t = DT[dt]
    if view == "packed":
        x = randn(7, B, T, 6, hd).to(t).cuda()
        k, v = x[:, :, 2:4], x[:, :, 4:6]
    elif view == "odd stride":
        x = randn(8, B, T, nkv * hd + 1).to(t).cuda()
        k = x[..., 1:].unflatten(2, (nkv, hd))
        v = x[..., :-1].unflatten(2, (nkv, hd))
    elif view == "broadcast":
        k = randn(9, 1, 1, nkv, hd).to(t).cuda().expand(B, T, nkv, hd)
        v = randn(10, B, 1, nkv, hd).to(t).cuda().expand(B, T, nkv, hd)
    else:
        flat = randn(11, 2 * B * T * nkv * hd + 1).to(t).cuda()[1:]
        k, v = flat.view(2, B, T, nkv, hd)
    starts = [0, 5, 80]
    kc, vc, ks, vs = empty_cache(B, nkv, S, hd)
    ks.fill_(2.0 ** -9)  # the scale of the blocks that hold earlier positions
    vs.fill_(2.0 ** -9)
    dev = both(kc, vc, ks, vs)
    q2.q2_kv8_append(*dev, k, v, i32(starts).cuda())
    R.append(kc, ks, k.cpu(), starts)
    R.append(vc, vs, v.cpu(), starts)
    same_codes(dev[0], kc, "k")
    same_codes(dev[1], vc, "v")
    assert torch.equal(dev[2].cpu(), ks) and torch.equal(dev[3].cpu(), vs)


def test_append_of_extreme_values():
    vals = [0.0, -0.0, 1e-30, 2.0 ** -69, -(2.0 ** -70), 448 * 2.0 ** -60, 3.3e38, -3.3e38, math.inf, -math.inf,
            math.nan, 1.75, 448.0, 1e-40, 17.0, 19.0]
    for i, top in enumerate([0.0, 2.0 ** -64, 1.0, 448.0, 449.0, 3.3e38, math.inf, math.nan]):
        x = torch.tensor([v for v in vals if not (abs(v) > abs(top)) or math.isnan(v) or math.isinf(v)] + [top])
        row = x.repeat(40)[:32].reshape(1, 1, 1, 32)
        kc, vc, ks, vs = empty_cache(1, 1, 64, 32, i)
        dev = both(kc, vc, ks, vs)
        q2.q2_kv8_append(*dev, row.cuda(), -row.cuda(), i32([0]).cuda())
        R.append(kc, ks, row, [0])
        R.append(vc, vs, -row, [0])
        same_codes(dev[0], kc, f"k {top}")
        same_codes(dev[1], vc, f"v {top}")
        assert torch.equal(dev[2].cpu(), ks) and torch.equal(dev[3].cpu(), vs)


def test_append_token_by_token_grows_scales_as_the_reference():
    B, nkv, hd, S, n = 2, 2, 128, 100, 90
    kc, vc, ks, vs = empty_cache(B, nkv, S, hd)
    dev = both(kc, vc, ks, vs)
    x = randn(12, B, n, nkv, hd).bfloat16() * torch.logspace(-3, 3, n)[None, :, None, None].bfloat16()
    for t in range(n):
        starts = [t, t if t % 3 else -1]  # the second sequence pauses: an inactive row of the batch
        q2.q2_kv8_append(*dev, x[:, t:t + 1].cuda(), -x[:, t:t + 1].cuda(), i32(starts).cuda())
        R.append(kc, ks, x[:, t:t + 1], starts)
        R.append(vc, vs, -x[:, t:t + 1], starts)
    same_codes(dev[0], kc, "k")
    same_codes(dev[1], vc, "v")
    assert torch.equal(dev[2].cpu(), ks) and torch.equal(dev[3].cpu(), vs)


def test_append_twice_writes_the_same():
    kc, vc, ks, vs = both(*filled_cache(2, 2, 140, 64, 20))
    k, v = randn(24, 2, 30, 2, 64).cuda() * 9, randn(25, 2, 30, 2, 64).cuda() * 9
    start = i32([50, 97]).cuda()
    q2.q2_kv8_append(kc, vc, ks, vs, k, v, start)
    once = [t.clone() for t in (kc, vc, ks, vs)]
    q2.q2_kv8_append(kc, vc, ks, vs, k, v, start)
    for a, b in zip(once, (kc, vc, ks, vs)):
        assert torch.equal(a, b)


def test_length_past_capacity_is_reported_and_writes_nothing():
    kc, vc, ks, vs = both(*filled_cache(2, 1, 70, 32, 30))
    keep = [t.clone() for t in (kc, vc, ks, vs)]
    k = randn(31, 2, 6, 1, 32).cuda()
    q2.q2_kv8_append(kc, vc, ks, vs, k, k, i32([65, 2 ** 31 - 3]).cuda())
    with pytest.raises(q2.Q2Error) as e:
        q2.q2_check_device_error()
    assert e.value.status == "Q2_ERR_CAPACITY"
    for a, b in zip(keep, (kc, vc, ks, vs)):
        assert torch.equal(a, b)
    out = torch.full_like(k, 5.0)
    q2.q2_kv8_read(out, torch.empty_like(k), kc, vc, ks, vs, i32([65, -4]).cuda())
    with pytest.raises(q2.Q2Error):
        q2.q2_check_device_error()
    assert bool((out == 5.0).all())
    q = randn(32, 2, 1, 2, 32).cuda()
    o = torch.full_like(q, 5.0)
    q2.q2_kv8_attention(o, q, kc, vc, ks, vs, i32([71, 2 ** 31 - 1]).cuda(), 1.0)
    with pytest.raises(q2.Q2Error) as e:
        q2.q2_check_device_error()
    assert e.value.status == "Q2_ERR_CAPACITY"
    assert bool((o == 0).all())
    q2.q2_check_device_error()  # cleared


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("hd,nkv,S,T,starts", APPENDS)
def test_read(dt, hd, nkv, S, T, starts):
    B = len(starts)
    kc, vc, ks, vs = filled_cache(B, nkv, S, hd, 40, spread=3.0)
    kc[0, 0, 0, :4] = torch.tensor([127, 255, 128, 1])  # NaN, NaN, -0, the smallest
    k = torch.full((B, T, nkv, hd), 3.0, dtype=DT[dt], device="cuda")
    v = k.clone()
    q2.q2_kv8_read(k, v, *both(kc, vc, ks, vs), i32(starts).cuda())
    for got, c, s in ((k, kc, ks), (v, vc, vs)):
        full = R.dense(c, s)
        want = torch.full((B, T, nkv, hd), 3.0, dtype=torch.float64)
        for b, p in enumerate(starts):
            if p >= 0:
                want[b] = full[b, :, p:p + T].transpose(0, 1)
        # exact: a code times a power of two
        assert torch.equal(got.cpu().double().nan_to_num(1e9), want.nan_to_num(1e9))


def test_read_into_rows_off_16_bytes():
    kc, vc, ks, vs = filled_cache(1, 2, 80, 32, 50)
    flat = torch.zeros(2 * 77 * 64 + 1, device="cuda")[1:]
    k, v = flat.view(2, 1, 77, 2, 32)
    q2.q2_kv8_read(k, v, *both(kc, vc, ks, vs), i32([3]).cuda())
    assert torch.equal(v.cpu()[0].double(), R.dense(vc, vs)[0, :, 3:80].transpose(0, 1))


# -------------------------------------------------------------------- attention

ATTN = [  # hd, nh, nkv, max_seq, ntok, lens
    (128, 12, 2, 200, 1, [1, 64, 65, 200]),
    (128, 12, 2, 700, 1, [513, 0, 700, 640, 129, 1]),
    (128, 12, 2, 300, 5, [5, 3, 64, 66, 300, 0, 261]),
    (128, 2, 2, 130, 3, [130, 2, 67]),
    (128, 8, 1, 1100, 8, [1100, 9]),
    (64, 15, 3, 333, 1, [333, 128, 63]),
    (64, 8, 8, 190, 4, [190, 60, 127]),
    (32, 4, 2, 64, 1, [64, 33]),
    (32, 7, 1, 257, 17, [257, 17, 100]),
    (128, 6, 1, 150, 33, [150, 70]),
    (128, 1, 1, 64, 1, [1]),
    (128, 12, 2, 900, 1, [899, 0, 64, 33, 32, 700]),
    (64, 12, 2, 800, 5, [799, 4, 5, 300, 64]),
    (32, 8, 1, 820, 12, [819, 11, 128]),
    (128, 8, 1, 800, 40, [800, 500]),
]


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("hd,nh,nkv,S,T,lens", ATTN)
def test_attention(dt, hd, nh, nkv, S, T, lens):
    B = len(lens)
    kc, vc, ks, vs = filled_cache(B, nkv, S, hd, 60, spread=0.7)
    for b, n in enumerate(lens):  # what lies past a sequence's end is anything, NaN codes included
        kc[b, :, n:], vc[b, :, n:] = 127, 255
    q = randn(64, B, T, nh, hd).to(DT[dt])
    scale = 1.0 / math.sqrt(hd)
    out = torch.full((B, T, nh, hd), 7.0, dtype=DT[dt], device="cuda")
    q2.q2_kv8_attention(out, q.cuda(), *both(kc, vc, ks, vs), i32(lens).cuda(), scale)
    ref, bound = R.attention(q, kc, vc, ks, vs, lens, scale)
    R.within(out, ref, bound, "attention")


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("hd,nh,nkv,S,T,total", [
    (128, 12, 2, 400, 130, 390), (128, 12, 2, 300, 16, 300), (128, 6, 3, 260, 129, 129), (128, 4, 2, 200, 2, 77),
    (128, 2, 1, 700, 300, 650), (128, 2, 2, 520, 515, 520), (64, 6, 2, 200, 70, 199), (32, 4, 4, 90, 40, 64), (128, 8, 1, 150, 1, 150),
])
def test_self_attention(dt, hd, nh, nkv, S, T, total):
    kc, vc, ks, vs = filled_cache(1, nkv, S, hd, 70, spread=0.7)
    kc[:, :, total:], vc[:, :, total:] = 255, 127
    q = randn(74, 1, T, nh, hd).to(DT[dt])
    scale = 1.0 / math.sqrt(hd)
    out = torch.empty((T, nh, hd), dtype=DT[dt], device="cuda")
    d = both(kc, vc, ks, vs)
    q2.q2_kv8_self_attention(out, q[0].cuda(), *(t[0] for t in d), total, scale)
    ref, bound = R.attention(q, kc, vc, ks, vs, [total], scale)
    R.within(out, ref[0], bound[0], "self attention")


def test_attention_of_a_slot_inside_a_larger_cache():
    """A sequence's slice of the batch's cache, the rows of the packed q/k/v projection."""
    kc, vc, ks, vs = filled_cache(3, 2, 100, 64, 80)
    qkv = randn(81, 2, 3, 8, 64).bfloat16()
    q = qkv[:, :, 1:5]
    d = both(kc, vc, ks, vs)
    out = torch.empty(2, 3, 4, 64, dtype=torch.bfloat16, device="cuda")
    q2.q2_kv8_attention(out, qkv.cuda()[:, :, 1:5], *(t[1:] for t in d), i32([99, 4]).cuda(), 0.2)
    ref, bound = R.attention(q, kc[1:], vc[1:], ks[1:], vs[1:], [99, 4], 0.2)
    R.within(out, ref, bound)


@pytest.mark.parametrize("dt", DT)
def test_attention_of_rows_off_16_bytes(dt):
    """Query tokens an odd number of elements apart, from an odd address."""
    kc, vc, ks, vs = filled_cache(2, 2, 90, 32, 85)
    x = randn(86, 2, 3, 4 * 32 + 1).to(DT[dt]).cuda()
    q = x[..., 1:].unflatten(2, (4, 32))
    out = torch.empty(2, 3, 4, 32, dtype=DT[dt], device="cuda")
    q2.q2_kv8_attention(out, q, *both(kc, vc, ks, vs), i32([90, 41]).cuda(), 0.2)
    ref, bound = R.attention(q.cpu(), kc, vc, ks, vs, [90, 41], 0.2)
    R.within(out, ref, bound)


def test_prompt_rows_off_16_bytes():
    """The prompt path that reads q in 16-byte pieces gives way to the other one."""
    kc, vc, ks, vs = filled_cache(1, 1, 300, 128, 87)
    x = randn(88, 260 * 2 * 128 + 1).bfloat16().cuda()[1:].view(260, 2, 128)
    d = both(kc, vc, ks, vs)
    out = torch.empty_like(x.clone())
    q2.q2_kv8_self_attention(out, x, *(t[0] for t in d), 300, 0.09)
    ref, bound = R.attention(x.cpu()[None], kc, vc, ks, vs, [300], 0.09)
    R.within(out, ref[0], bound[0])


def test_many_short_and_few_long_items_take_the_same_values():
    """One CTA per item (a short cache, or items in plenty) and runs over all items: the same
    sequences in a cache with room for 256 positions and for 4096, and 512 of them."""
    B, nkv, hd, nh, S = 3, 2, 64, 6, 256
    kc, vc, ks, vs = filled_cache(B, nkv, S, hd, 89)
    lens = [256, 77, 0]
    q = randn(89, B, 1, nh, hd).bfloat16()
    ref, bound = R.attention(q, kc, vc, ks, vs, lens, 0.125)
    small = torch.empty(B, 1, nh, hd, dtype=torch.bfloat16, device="cuda")
    q2.q2_kv8_attention(small, q.cuda(), *both(kc, vc, ks, vs), i32(lens).cuda(), 0.125)
    R.within(small, ref, bound, "short cache")
    wide = [torch.cat([t, torch.full((*t.shape[:2], (4096 - S) // (1 if t.dim() == 4 else 64), *t.shape[3:]), 127,
                                     dtype=t.dtype)], 2) for t in (kc, vc, ks, vs)]
    large = torch.empty_like(small)
    q2.q2_kv8_attention(large, q.cuda(), *both(*wide), i32(lens).cuda(), 0.125)
    R.within(large, ref, bound, "long cache")
    many = [t.repeat(171, *[1] * (t.dim() - 1)).contiguous().cuda() for t in (kc, vc, ks, vs)]
    out = torch.empty(B * 171, 1, nh, hd, dtype=torch.bfloat16, device="cuda")
    q2.q2_kv8_attention(out, q.repeat(171, 1, 1, 1).cuda(), *many, i32(lens * 171).cuda(), 0.125)
    assert torch.equal(out.view(171, B, 1, nh, hd), small.expand(171, B, 1, nh, hd))


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("rows", [1, 4, 40, 260])
def test_attention_keeps_nan_to_the_rows_that_see_it(dt, rows):
    """A NaN of K makes every dimension of the rows that see it NaN, a NaN of V only its own
    dimension; rows before it do not see it."""
    S, hd, nh, nkv = 320, 128, 4, 2
    kc, vc, ks, vs = filled_cache(1, nkv, S, hd, 90)
    n = 310
    kc[0, 0, n - 2, 5] = 127
    vc[0, 1, n - 2, 9] = 255
    vc[0, 1, 20, 77] = 127
    q = randn(94, 1, rows, nh, hd).to(DT[dt])
    ref, bound = R.attention(q, kc, vc, ks, vs, [n], 0.09)
    d = both(kc, vc, ks, vs)
    out = torch.empty(1, rows, nh, hd, dtype=DT[dt], device="cuda")
    q2.q2_kv8_attention(out, q.cuda(), *d, i32([n]).cuda(), 0.09)
    R.within(out, ref, bound, "batch")
    q2.q2_kv8_self_attention(out[0], q[0].cuda(), *(t[0] for t in d), n, 0.09)
    R.within(out, ref, bound, "rows")


@pytest.mark.parametrize("dt", DT)
def test_attention_over_blocks_of_very_unequal_scales(dt):
    """Neighbouring blocks' scales 2^-60 .. 2^119 apart, zero blocks among them."""
    S, hd, nh, nkv = 64 * 7, 64, 4, 2
    x = randn(100, 1, S, nkv, hd)
    size = torch.tensor([1.0, 0.0, 1e30, 1e-12, 1.0, 1e-25, 3.0]).repeat_interleave(64)[None, :, None, None]
    kc, vc, ks, vs = empty_cache(1, nkv, S, hd)
    R.append(kc, ks, x, [0])
    for sizes in (size, size.flip(1), torch.clamp(size, max=1e3)):
        R.append(vc, vs, x.flip(3) * sizes, [0])
        q = randn(101, 1, 2, nh, hd).to(DT[dt])
        out = torch.empty(1, 2, nh, hd, dtype=DT[dt], device="cuda")
        for n in (S, 200, 100):
            q2.q2_kv8_attention(out, q.cuda(), *both(kc, vc, ks, vs), i32([n]).cuda(), 0.1)
            ref, bound = R.attention(q, kc, vc, ks, vs, [n], 0.1)
            R.within(out, ref, bound)


@pytest.mark.parametrize("dt", DT)
def test_attention_with_large_small_and_zero_queries(dt):
    S, hd, nh, nkv = 150, 128, 6, 2
    kc, vc, ks, vs = filled_cache(1, nkv, S, hd, 110)
    q = randn(111, 1, 6, nh, hd)
    q[0, 0] *= 1e5      # past fp16's range
    q[0, 1] *= 1e-9     # below it
    q[0, 2] = 0
    q[0, 3, :, 7] *= 3000.0
    q[0, 4] *= 1e-38    # fp32's edge: scores of 0
    q = q.to(DT[dt])
    out = torch.empty(1, 6, nh, hd, dtype=DT[dt], device="cuda")
    for scale in (0.09, 1e-4, -0.05):
        q2.q2_kv8_attention(out, q.cuda(), *both(kc, vc, ks, vs), i32([150]).cuda(), scale)
        ref, bound = R.attention(q, kc, vc, ks, vs, [150], scale)
        R.within(out, ref, bound, f"scale {scale}")


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("rows", [1, 4, 40, 260])
@pytest.mark.parametrize("x", [math.inf, -math.inf, math.nan])
def test_attention_with_queries_that_are_not_finite(dt, rows, x):
    """They make their own rows NaN, also where every score is -inf, and no others."""
    S, hd, nh, nkv = 300, 128, 4, 2
    kc, vc, ks, vs = filled_cache(1, nkv, S, hd, 106)
    kc[..., 3] |= 128   # (q[3] = inf: -inf everywhere)
    kc[..., 3] &= 0xfe  # (no NaN code)
    kc[..., 5] &= 0x7e
    q = randn(109, 1, rows, nh, hd).to(DT[dt])
    q[0, 0, 0, 3], q[0, rows // 2, 2, 5], q[0, rows - 1, 3, 100] = x, x, x
    d = both(kc, vc, ks, vs)
    ref, bound = R.attention(q, kc, vc, ks, vs, [S], 0.09)
    out = torch.empty(1, rows, nh, hd, dtype=DT[dt], device="cuda")
    q2.q2_kv8_attention(out, q.cuda(), *d, i32([S]).cuda(), 0.09)
    R.within(out, ref, bound, "batch")
    q2.q2_kv8_self_attention(out[0], q[0].cuda(), *(t[0] for t in d), S, 0.09)
    R.within(out, ref, bound, "rows")


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("rows", [1, 5, 300])
def test_attention_over_a_stretch_of_nan_keys(dt, rows):
    """Whole key ranges of NaN, as a split of the keys may hand one to a CTA."""
    S, hd, nh, nkv = 2000, 128, 4, 2
    kc, vc, ks, vs = filled_cache(1, nkv, S, hd, 110)
    kc[0, 0, 400:1300] = 127
    q = randn(114, 1, rows, nh, hd).to(DT[dt])
    d = both(kc, vc, ks, vs)
    out = torch.empty(1, rows, nh, hd, dtype=DT[dt], device="cuda")
    for n in (S, 690):  # all rows see them; the first of the 300 do not
        ref, bound = R.attention(q, kc, vc, ks, vs, [n], 0.09)
        q2.q2_kv8_attention(out, q.cuda(), *d, i32([n]).cuda(), 0.09)
        R.within(out, ref, bound, "batch")
        q2.q2_kv8_self_attention(out[0], q[0].cuda(), *(t[0] for t in d), n, 0.09)
        R.within(out, ref, bound, "rows")


def test_attention_is_the_same_every_time_and_beside_other_sequences():
    S, hd, nh, nkv, B = 3000, 128, 12, 2, 5
    g = torch.Generator(device="cuda").manual_seed(3)
    kc = torch.randint(0, 120, (B, nkv, S, hd), generator=g, dtype=torch.uint8, device="cuda")
    vc = torch.randint(0, 120, (B, nkv, S, hd), generator=g, dtype=torch.uint8, device="cuda")
    ks = torch.full((B, nkv, 47), 2.0 ** -8, device="cuda")
    q = torch.randn(B, 1, nh, hd, generator=g, device="cuda").bfloat16()
    lens = i32([3000, 17, 2900, 0, 1555]).cuda()
    outs = [torch.empty_like(q) for _ in range(3)]
    for o in outs:
        q2.q2_kv8_attention(o, q, kc, vc, ks, ks, lens, 0.01)
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


@pytest.mark.parametrize("dt", DT)
def test_long_ragged_decode_against_a_dense_fp64_product(dt):
    """Long caches (checked on the GPU in 64 bits): many splits of each sequence's keys."""
    S, hd, nh, nkv = 20011, 128, 12, 2
    lens = [20011, 1, 9000, 64 * 100]
    B, T = len(lens), 2
    g = torch.Generator(device="cuda").manual_seed(4)
    kc, vc = (torch.randint(0, 256, (B, nkv, S, hd), generator=g, dtype=torch.uint8, device="cuda") for _ in range(2))
    kc[kc & 127 == 127] = 0
    vc[vc & 127 == 127] = 0
    ks, vs = (2.0 ** torch.randint(-9, -6, (B, nkv, 313), generator=g, device="cuda").float() for _ in range(2))
    q = torch.randn(B, T, nh, hd, generator=g, device="cuda").to(DT[dt])
    out = torch.empty_like(q)
    scale = 0.02
    q2.q2_kv8_attention(out, q, kc, vc, ks, vs, i32(lens).cuda(), scale)
    table = R.VALUES.cuda()
    for b, n in enumerate(lens):
        for t in range(T):
            m = n - T + 1 + t
            if m <= 0:
                assert bool((out[b, t] == 0).all())
                continue
            for gk in range(nkv):
                k = table[kc[b, gk, :m].long()] * ks[b, gk].double().repeat_interleave(64)[:m, None]
                v = table[vc[b, gk, :m].long()] * vs[b, gk].double().repeat_interleave(64)[:m, None]
                qq = q[b, t, gk * 6:gk * 6 + 6].double()
                p = torch.softmax(qq @ k.t() * scale, -1)
                ref, A = p @ v, p @ v.abs()
                s1 = (qq.abs() @ k.abs().t()).amax(1, keepdim=True) * scale
                w = 2.0 ** -11 if dt == "bf16" else 0.0
                # as q8_ref.attention; the n additions of a sum count 2 sqrt(n) steps here (their
                # signs vary; n whole steps would allow more than the fp32 output resolves)
                rel = 2 * (hd * 2.0 ** -23 + 2.0 ** -22) * s1 + 2.0 ** -21 + w + 4 * math.sqrt(m) * 2.0 ** -23 + 2.0 ** -21
                bound = R.HALF[DT[dt]] * ref.abs() + (1 + R.HALF[DT[dt]]) * rel * A
                R.within(out[b, t, gk * 6:gk * 6 + 6], ref.cpu(), bound.cpu(), f"sequence {b}")


# ---------------------------------------------------------------- quantise, linear

@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 128), (5, 1536), (33, 200), (129, 257), (70, 64), (3, 130)])
@pytest.mark.parametrize("br", [1, 128])
def test_quantize(dt, rows, cols, br):
    x = (randn(120, rows, cols) * torch.exp(2 * randn(121, rows, 1))).to(DT[dt])
    if rows * cols > 300:
        x[0, :140] = 0
        x[-1, -1], x[-1, 0], x[0, 0] = math.nan, math.inf, -math.inf
    c, s = R.quantise(x, br)
    codes = torch.full((rows, cols), 77, dtype=torch.uint8, device="cuda")
    scales = torch.full(tuple(s.shape), -1.0, device="cuda")
    q2.q2_quantize_q8(codes, scales, x.cuda(), br)
    same_codes(codes, c, "codes")
    assert torch.equal(scales.cpu(), s)


@pytest.mark.parametrize("br", [1, 128])
def test_quantize_strided_rows(br):
    for x in (randn(122, 40, 700)[:, 3:515], randn(123, 40, 704)[:, :512].bfloat16(), randn(124, 512)[None].expand(40, 512)):
        c, s = R.quantise(x, br)
        codes, scales = torch.empty(40, 512, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(tuple(s.shape), device="cuda")
        q2.q2_quantize_q8(codes, scales, x.contiguous().cuda() if x.stride(0) == 0 else _copy_with_strides(x), br)
        same_codes(codes, c, "codes")
        assert torch.equal(scales.cpu(), s)


def _copy_with_strides(x):
    base = torch.zeros(x.shape[0] * x.stride(0) + x.shape[1], dtype=x.dtype, device="cuda")
    v = base.as_strided(x.shape, x.stride(), base.numel() - x.shape[0] * x.stride(0) - x.shape[1])
    v.copy_(x)
    return v


LIN = [(1, 128, 128), (1, 1, 16), (1, 200, 1536), (2, 384, 144), (3, 130, 400), (7, 17, 8960), (16, 256, 256),
       (17, 300, 512), (33, 129, 1536), (64, 64, 272), (61, 1000, 1536), (65, 128, 640), (100, 512, 128),
       (128, 1536, 1536), (130, 257, 1040), (200, 140, 112), (257, 384, 896), (300, 640, 2048), (513, 129, 256)]


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("M,N,K", LIN)
def test_linear(dt, M, N, K):
    x = randn(130, M, K) * torch.exp(randn(131, M, 1))
    w = 0.02 * randn(132, N, K)
    xq, xs = R.quantise(x, 1)
    wq, ws = R.quantise(w, 128)
    bias = randn(133, N).to(DT[dt]) if M % 2 else None
    out = torch.full((M, N), 9.0, dtype=DT[dt], device="cuda")
    q2.q2_linear_q8(out, *both(xq, xs, wq, ws), None if bias is None else bias.cuda())
    ref, bound = R.linear(xq, xs, wq, ws, bias, DT[dt])
    R.within(out, ref, bound, "linear")


def test_linear_carries_nan_and_extreme_scales():
    M, N, K = 5, 140, 256
    xq, xs = R.quantise(randn(140, M, K), 1)
    wq, ws = R.quantise(randn(141, N, K), 128)
    xq[2, 130] = 127
    wq[7, 3] = 255
    xs[0, 0], xs[1, 0], ws[1, 0], ws[0, 1] = 1e-30, 1e20, 1e-12, 0.0
    out = torch.empty(M, N, device="cuda")
    q2.q2_linear_q8(out, *both(xq, xs, wq, ws))
    ref, bound = R.linear(xq, xs, wq, ws, None, torch.float32)
    R.within(out, ref, bound)


def test_linear_of_zero_codes_is_the_bias():
    out = torch.empty(9, 130, dtype=torch.bfloat16, device="cuda")
    bias = randn(142, 130).bfloat16().cuda()
    z = lambda *s: torch.zeros(*s, dtype=torch.uint8, device="cuda")  # noqa: E731
    q2.q2_linear_q8(out, z(9, 48), torch.ones(1, 9, device="cuda"), z(130, 48), torch.ones(2, 1, device="cuda"), bias)
    assert torch.equal(out, bias.expand(9, 130))


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("M,N,K", [(1, 17920, 1536), (4, 1536, 8960), (61, 2048, 1536), (700, 1536, 1536),
                                   (1025, 2100, 8960), (4096, 1536, 256), (4001, 1544, 144), (2300, 4104, 272),
                                   (2500, 3001, 128), (2500, 3000, 4096), (2500, 3001, 4112), (2500, 3000, 8960)])
def test_linear_at_the_layers_sizes(dt, M, N, K):
    """Full-size products, the whole output against a 64-bit product on the GPU."""
    g = torch.Generator(device="cuda").manual_seed(6)
    xq, wq = torch.empty(M, K, dtype=torch.uint8, device="cuda"), torch.empty(N, K, dtype=torch.uint8, device="cuda")
    xs, ws = torch.empty(-(-K // 128), M, device="cuda"), torch.empty(-(-N // 128), -(-K // 128), device="cuda")
    q2.q2_quantize_q8(xq, xs, torch.randn(M, K, generator=g, device="cuda"))
    q2.q2_quantize_q8(wq, ws, 0.02 * torch.randn(N, K, generator=g, device="cuda"), 128)
    out = torch.empty(M, N, dtype=DT[dt], device="cuda")
    q2.q2_linear_q8(out, xq, xs, wq, ws)
    table = R.VALUES.cuda()
    x = table[xq.long()] * xs.double().t().repeat_interleave(128, 1)[:, :K]
    w = table[wq.long()] * ws.double().repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
    ref = x @ w.t()
    bound = R.HALF[DT[dt]] * ref.abs() + 1.01 * (132 + xs.shape[0]) * 2.0 ** -23 * (x.abs() @ w.abs().t())
    R.within(out, ref.cpu(), bound.cpu())


# -------------------------------------------------------------- streams and graphs

def test_calls_on_another_stream():
    kc, vc, ks, vs = filled_cache(2, 2, 300, 64, 150)
    q = randn(151, 2, 1, 4, 64)
    ref, bound = R.attention(q, kc, vc, ks, vs, [300, 77], 0.125)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        d = both(kc, vc, ks, vs, q, i32([300, 77]))
        out = torch.empty(2, 1, 4, 64, device="cuda")
        q2.q2_kv8_attention(out, d[4], *d[:4], d[5], 0.125)
    s.synchronize()
    R.within(out, ref, bound)


def test_two_calls_at_once_have_a_workspace_each():
    S, B = 4000, 3
    g = torch.Generator(device="cuda").manual_seed(8)
    c = [torch.randint(0, 120, (B, 2, S, 128), generator=g, dtype=torch.uint8, device="cuda") for _ in range(4)]
    sc = torch.full((B, 2, 63), 2.0 ** -8, device="cuda")
    q = torch.randn(2, B, 1, 12, 128, generator=g, device="cuda").bfloat16()
    lens = [i32([4000, 3, 999]).cuda(), i32([100, 3500, 2222]).cuda()]
    want = [q2.q2_kv8_attention(torch.empty_like(q[i]), q[i], c[2 * i], c[2 * i + 1], sc, sc, lens[i], 0.01)
            for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [torch.empty_like(q[0]) for _ in range(2)]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                q2.q2_kv8_attention(got[i], q[i], c[2 * i], c[2 * i + 1], sc, sc, lens[i], 0.01)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("T,lens", [(1, [65, 640, 0, 128]), (3, [65, 640, 3, 128]), (300, [700, 300, 0, 449])])
def test_nothing_past_a_sequences_end_is_seen(dt, T, lens):
    """NaN codes and NaN scales of every block behind a sequence's last one."""
    nh, nkv, S, hd = 4, 2, 1000, 128
    kc, vc, ks, vs = filled_cache(4, nkv, S, hd, 170)
    for b, n in enumerate(lens):
        kc[b, :, n:], vc[b, :, n:] = 255, 127
        ks[b, :, -(-n // 64):], vs[b, :, -(-n // 64):] = math.nan, math.nan
    q = randn(174, 4, T, nh, hd).to(DT[dt])
    d = both(kc, vc, ks, vs)
    out = torch.empty(4, T, nh, hd, dtype=DT[dt], device="cuda")
    q2.q2_kv8_attention(out, q.cuda(), *d, i32(lens).cuda(), 0.09)
    ref, bound = R.attention(q, kc, vc, ks, vs, lens, 0.09)
    R.within(out, ref, bound, "batch")
    for b, n in enumerate(lens):
        if n >= T:
            q2.q2_kv8_self_attention(out[b], q[b].cuda(), *(t[b] for t in d), n, 0.09)
            R.within(out[b], ref[b], bound[b], f"rows of {b}")


def test_cache_offsets_past_32_bits():
    """The third sequence's slot of a cache of 2^24 positions starts past 2^32 bytes."""
    B, nkv, S, hd, nh, T = 3, 1, 1 << 24, 128, 2, 3
    kc, vc = (torch.empty(B, nkv, S, hd, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.ones(B, nkv, S // 64, device="cuda") for _ in range(2))
    k, v = randn(180, B, T, nkv, hd).bfloat16(), randn(181, B, T, nkv, hd).bfloat16()
    q = randn(182, B, T, nh, hd).bfloat16()
    small = empty_cache(B, nkv, 64, hd)
    R.append(small[0], small[2], k, [0, 0, 0])
    R.append(small[1], small[3], v, [0, 0, 0])
    for start in ([0, -1, 0], [-1, S - 64, S - 64]):  # both ends of the last slot
        q2.q2_kv8_append(kc, vc, ks, vs, k.cuda(), v.cuda(), i32(start).cuda())
        kr, vr = (torch.zeros(B, T, nkv, hd, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        q2.q2_kv8_read(kr, vr, kc, vc, ks, vs, i32(start).cuda())
        for b in range(B):
            if start[b] >= 0:
                assert torch.equal(kr[b, :, 0].cpu().double(), R.dense(small[0], small[2])[b, 0, :T])
                assert torch.equal(vr[b, :, 0].cpu().double(), R.dense(small[1], small[3])[b, 0, :T])
    out = torch.empty(B, T, nh, hd, dtype=torch.bfloat16, device="cuda")
    lens = [T, 0, T]
    q2.q2_kv8_attention(out, q.cuda(), kc, vc, ks, vs, i32(lens).cuda(), 0.1)
    ref, bound = R.attention(q, *small, lens, 0.1)
    R.within(out, ref, bound)


@pytest.mark.parametrize("N", [151936, 151935])
def test_linear_output_past_32_bits(N):
    """More than 2^31 outputs, in rows on 16 bytes and off them."""
    M, K = 16400, 16
    xq, xs = R.quantise(randn(183, M, K), 1)
    wq, ws = R.quantise(randn(184, N, K), 128)
    out = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    q2.q2_linear_q8(out, *both(xq, xs, wq, ws))
    rows = [0, 2 ** 31 // N, 2 ** 31 // N + 1, M - 1]
    ref, bound = R.linear(xq[rows], xs[:, rows], wq, ws, None, torch.bfloat16)
    R.within(out[rows], ref, bound)


@pytest.mark.parametrize("br", [1, 128])
def test_quantize_past_32_bits(br):
    rows, cols = (1 << 20) + 131, 2064
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(185))
    codes = torch.empty(rows, cols, dtype=torch.uint8, device="cuda")
    G = -(-cols // 128)
    scales = torch.empty((G, rows) if br == 1 else (-(-rows // 128), G), device="cuda")
    q2.q2_quantize_q8(codes, scales, x, br)
    first = rows // 128 * 128 - 128
    c, s = R.quantise(x[first:].cpu(), br)
    same_codes(codes[first:], c, "codes")
    assert torch.equal(scales[:, first:].cpu() if br == 1 else scales[first // 128:].cpu(), s)


FIRST = """
import torch, qwen2_decode_step_b200 as q2
z = lambda *s, dt=torch.float32: torch.zeros(*s, dtype=dt, device="cuda")
u8, bf = torch.uint8, torch.bfloat16
cache = z(2, 2, 700, 128, dt=u8), z(2, 2, 700, 128, dt=u8), z(2, 2, 11), z(2, 2, 11)
k, start, lens = z(2, 300, 2, 128, dt=bf) + 1, z(2, dt=torch.int32), z(2, dt=torch.int32) + 300
o, r, one = z(2, 300, 4, 128, dt=bf), z(2, 300, 2, 128, dt=bf), z(300, 4, 128, dt=bf)
q = z(2, 300, 4, 128, dt=bf)
x, c, s, wc, ws, y = z(70, 256, dt=bf) + 2, z(70, 256, dt=u8), z(2, 70), z(256, 256, dt=u8), z(2, 2), z(70, 256)
y1 = z(1, 256)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    q2.q2_kv8_append(*cache, k, k, start)
    q2.q2_kv8_read(r, torch.empty_like(r), *cache, start)
    q2.q2_kv8_attention(o, q, *cache, lens, 0.1)
    q2.q2_kv8_self_attention(one, q[0], *(t[0] for t in cache), 300, 0.1)
    q2.q2_quantize_q8(c, s, x)
    q2.q2_quantize_q8(wc, ws, torch.cat([x] * 4)[:256], 128)
    q2.q2_linear_q8(y, c, s, wc, ws)
    q2.q2_linear_q8(y1, c[:1], s[:, :1].contiguous(), wc, ws)
g.replay()
torch.cuda.synchronize()
assert bool((r == 1).all()) and bool((o == 1).all()) and bool((one == 1).all())
assert bool(((y - 1024).abs() < 1e-2).all()) and torch.equal(y1, y[:1])
"""


def test_the_first_calls_of_a_process_may_be_captured():
    """Attributes, symbols and occupancies are asked for inside the capture."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def test_workspace_too_small_is_refused():
    kc, vc, ks, vs = both(*empty_cache(1, 2, 3000, 128))
    q = randn(153, 1, 1, 4, 128).cuda()
    with pytest.raises(q2.Q2Error) as e:
        q2.q2_kv8_attention(torch.empty_like(q), q, kc, vc, ks, vs, i32([300]).cuda(), 1.0,
                            workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert e.value.status == "Q2_ERR_INVALID_ARG"


def _layer(x, wts, cache, start, lens, nh, nkv, hd):
    """One attention + MLP block as a serving step runs it: 8-bit linears, 8-bit cache."""
    B, T, H = x.shape
    rows = B * T

    def linear(a, w, dt=torch.bfloat16):
        wq, ws = w
        K, N = a.shape[-1], wq.shape[0]
        aq = torch.empty(rows, K, dtype=torch.float8_e4m3fn, device="cuda")
        as_ = torch.empty(-(-K // 128), rows, device="cuda")
        q2.q2_quantize_q8(aq, as_, a.view(rows, K))
        return q2.q2_linear_q8(torch.empty(rows, N, dtype=dt, device="cuda"), aq, as_, wq, ws)

    h = torch.empty_like(x)
    q2.q2_add_rms_norm(x, None, h, wts["norm"], 1e-6)
    qkv = linear(h, wts["qkv"]).view(B, T, nh + 2 * nkv, hd)
    q, k, v = qkv[:, :, :nh], qkv[:, :, nh:nh + nkv], qkv[:, :, nh + nkv:]
    q2.q2_kv8_append(*cache, k, v, start)
    att = q2.q2_kv8_attention(torch.empty(B, T, nh, hd, dtype=torch.bfloat16, device="cuda"), q, *cache, lens,
                              1 / math.sqrt(hd))
    o = linear(att.view(rows, nh * hd), wts["o"])
    q2.q2_add_rms_norm(x, o.view_as(x), h, wts["norm"], 1e-6)
    gate, up = linear(h, wts["gate"]), linear(h, wts["up"])
    s = torch.empty_like(gate)
    q2.q2_swiglu(s, gate, up)
    y = linear(s, wts["down"])
    q2.q2_add(x, x, y.view_as(x))
    return x


def _layer_case(seed, B, T, nh, nkv, hd, H, inter, S):
    def weight(i, n, k):
        w = (0.05 * randn(seed + i, n, k)).cuda()
        wq = torch.empty(n, k, dtype=torch.float8_e4m3fn, device="cuda")
        ws = torch.empty(-(-n // 128), -(-k // 128), device="cuda")
        return q2.q2_quantize_q8(wq, ws, w, 128)

    wts = {"norm": torch.ones(H, dtype=torch.bfloat16, device="cuda"), "qkv": weight(1, (nh + 2 * nkv) * hd, H),
           "o": weight(2, H, nh * hd), "gate": weight(3, inter, H), "up": weight(4, inter, H),
           "down": weight(5, H, inter)}
    cache = both(*filled_cache(B, nkv, S, hd, seed + 6))
    x = randn(seed + 10, B, T, H).bfloat16().cuda()
    return wts, cache, x


@pytest.mark.parametrize("T", [1, 3])
def test_a_layer_in_8_bits(T):
    """Quantise, linear, append, attention together, against the same chain of references fed
    with the GPU's own inputs at each step's start; the whole within the operators' roundings."""
    B, nh, nkv, hd, H, inter, S = 3, 4, 2, 64, 256, 384, 200
    wts, cache, x = _layer_case(160, B, T, nh, nkv, hd, H, inter, S)
    start, lens = [100, 63, 0], [100 + T, 63 + T, T]
    xc, cc = x.cpu().double(), [t.cpu().clone() for t in cache]

    def lin(a, w):
        aq, as_ = R.quantise(a.bfloat16().float().view(-1, a.shape[-1]), 1)
        return R.linear(aq, as_, w[0].cpu(), w[1].cpu(), None, torch.bfloat16)[0].bfloat16()

    def norm(a):
        return (a / (a.pow(2).mean(-1, keepdim=True) + 1e-6).sqrt()).bfloat16()

    qkv = lin(norm(xc), wts["qkv"]).view(B, T, nh + 2 * nkv, hd)
    R.append(cc[0], cc[2], qkv[:, :, nh:nh + nkv], start)
    R.append(cc[1], cc[3], qkv[:, :, nh + nkv:], start)
    att = R.attention(qkv[:, :, :nh], *cc, lens, 1 / math.sqrt(hd))[0].bfloat16()
    r = (xc + lin(att.reshape(B * T, nh * hd), wts["o"]).view(B, T, H).double()).bfloat16().double()
    h = norm(r)
    gate, up = lin(h, wts["gate"]).double(), lin(h, wts["up"]).double()
    s = (up * gate / (1 + torch.exp(-gate))).bfloat16()
    want = r + lin(s, wts["down"]).view(B, T, H).double()

    got = _layer(x, wts, cache, i32(start).cuda(), i32(lens).cuda(), nh, nkv, hd)
    # the chain's e4m3 roundings may fall on the other side where an input differs by a bf16 step:
    # a code's step is 2^-3 of it at most, on few elements; in norm, each of the chain's four
    # quantised products may then move by a fraction of 2^-4, far below the 2e-2 of two bf16
    # operators in a row held elementwise elsewhere
    err = float((got.cpu().double() - want).norm() / want.norm())
    assert err <= 2e-2, err


def test_a_layer_captured_and_replayed_with_other_lengths():
    B, T, nh, nkv, hd, H, inter, S = 2, 1, 4, 2, 64, 256, 384, 300
    wts, cache, x0 = _layer_case(180, B, T, nh, nkv, hd, H, inter, S)
    keep = [t.clone() for t in cache]
    x, start, lens = x0.clone(), i32([5, 200]).cuda(), i32([6, 201]).cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _layer(x, wts, cache, start, lens, nh, nkv, hd)
    torch.cuda.current_stream().wait_stream(side)
    graphs = []
    for _ in range(2):  # two graphs of the same step, each with workspaces of its own
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = _layer(x, wts, cache, start, lens, nh, nkv, hd)
        graphs.append(g)
    for step, (a, b) in enumerate([(5, 200), (64, 0), (299, 129)]):
        for c, k in zip(cache, keep):
            c.copy_(k)
        x.copy_(x0)
        start.copy_(i32([a, b]))
        lens.copy_(i32([a + 1, b + 1]))
        graphs[step % 2].replay()
        got, got_cache = out.clone(), [c.clone() for c in cache]
        for c, k in zip(cache, keep):
            c.copy_(k)
        want = _layer(x0.clone(), wts, cache, start, lens, nh, nkv, hd)
        assert torch.equal(got, want)
        for c, d in zip(cache, got_cache):
            assert torch.equal(c, d)


def test_prompt_then_decode_equals_the_dense_operators_over_the_read_back_cache():
    """A prompt chunk and a decode step over the 8-bit cache against the framework's dense
    attention over what q2_kv8_read returns (the same values; each side rounds once to bf16)."""
    nh, nkv, hd, S, P = 12, 2, 128, 400, 333
    x = randn(190, 1, P + 1, nh + 2 * nkv, hd).bfloat16().cuda()
    q, k, v = x[:, :, :nh], x[:, :, nh:nh + nkv], x[:, :, nh + nkv:]
    kc, vc, ks, vs = both(*empty_cache(1, nkv, S, hd))
    for lo, hi in ((0, 100), (100, 120), (120, P), (P, P + 1)):
        q2.q2_kv8_append(kc, vc, ks, vs, k[:, lo:hi], v[:, lo:hi], i32([lo]).cuda())
        rows = q[0, lo:hi].contiguous()
        if hi - lo > 1:
            got = q2.q2_kv8_self_attention(torch.empty_like(rows), rows, kc[0], vc[0], ks[0], vs[0], hi, 0.088)
        else:
            got = q2.q2_kv8_attention(torch.empty_like(rows)[None], q[:, lo:hi], kc, vc, ks, vs, i32([hi]).cuda(), 0.088)[0]
        dk, dv = (torch.empty(1, hi, nkv, hd, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        q2.q2_kv8_read(dk, dv, kc, vc, ks, vs, i32([0]).cuda())
        want = q2.q2_self_attention(torch.empty_like(rows), rows, dk[0], dv[0], 0.088)
        scale = torch.maximum(want.abs().float(), want.float().pow(2).mean().sqrt())
        assert float(((got.float() - want.float()).abs() / scale).max()) <= 1e-2
