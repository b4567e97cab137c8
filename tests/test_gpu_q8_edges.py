"""The 8-bit operators where a rare value, size or division of the work decides: against the plain
64-bit references of q8_ref, with its bounds."""

import math

import pytest
import torch

import q8_ref as R
import qwen2_decode_step_b200 as q2
from test_gpu_q8 import DT, both, empty_cache, filled_cache, i32, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu(cuda_ok):
    yield
    torch.cuda.synchronize()
    q2.q2_check_device_error()


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("M,N,K", [(3, 130, 8960), (3, 131, 384), (20, 5, 640), (70, 130, 4096), (129, 333, 2048),
                                   (66, 201, 384)])
def test_linear_split_over_a_cluster_with_remainder_tiles(dt, M, N, K):
    """Lanes of one warp that have an output next to lanes that have none, between two barriers of
    the cluster; many launches behind one another."""
    xq, xs = R.quantise(randn(300, M, K), 1)
    wq, ws = R.quantise(0.02 * randn(301, N, K), 128)
    bias = randn(302, N).to(DT[dt])
    d = both(xq, xs, wq, ws, bias)
    outs = torch.full((40, M, N), 9.0, dtype=DT[dt], device="cuda")
    for o in outs:
        q2.q2_linear_q8(o, *d)
    ref, bound = R.linear(xq, xs, wq, ws, bias, DT[dt])
    R.within(outs[0], ref, bound, "linear")
    assert torch.equal(outs, outs[:1].expand_as(outs))


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("hd,nh,nkv,T", [(128, 7, 1, 1), (128, 6, 2, 5), (64, 5, 1, 3), (32, 3, 3, 9), (128, 5, 1, 14)])
def test_attention_of_odd_rows_and_many_items_a_run(dt, hd, nh, nkv, T):
    """Several items in a CTA's run, rows that fill neither a warp's tiles nor the CTA; many launches
    behind one another."""
    S, lens = 4100, [T, 33, 700, 0, 96, 4100, T + 1, 61, 2047, 350, 31, 64]
    B = len(lens)
    kc, vc, ks, vs = filled_cache(B, nkv, S, hd, 310, spread=0.7)
    q = randn(314, B, T, nh, hd).to(DT[dt])
    scale = 1.0 / math.sqrt(hd)
    d = both(q, kc, vc, ks, vs, i32(lens))
    outs = torch.full((20, B, T, nh, hd), 7.0, dtype=DT[dt], device="cuda")
    for o in outs:
        q2.q2_kv8_attention(o, *d, scale)
    ref, bound = R.attention(q, kc, vc, ks, vs, lens, scale)
    R.within(outs[0], ref, bound, "attention")
    assert torch.equal(outs, outs[:1].expand_as(outs))


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("rows", [6, 200, 260])
@pytest.mark.parametrize("scale", [-0.05, 0.0, -3.0])
def test_self_attention_with_scales_that_are_not_positive(dt, rows, scale):
    """200 rows of two heads stay below the tcgen05 attention's sizes, 260 reach them."""
    kc, vc, ks, vs = filled_cache(1, 1, 300, 128, 320)
    q = randn(324, 1, rows, 2, 128).to(DT[dt])
    d = both(kc, vc, ks, vs)
    out = torch.empty(rows, 2, 128, dtype=DT[dt], device="cuda")
    q2.q2_kv8_self_attention(out, q[0].cuda(), *(t[0] for t in d), 290, scale)
    ref, bound = R.attention(q, kc, vc, ks, vs, [290], scale)
    R.within(out, ref[0], bound[0], "self attention")


@pytest.mark.parametrize("rows", [5, 100, 260])
@pytest.mark.parametrize("scale", [-0.05, 0.0])
def test_dense_self_attention_with_scales_that_are_not_positive(rows, scale):
    """The bf16 attention that shares the tcgen05 kernel, over the values of an 8-bit cache."""
    kc, vc, ks, vs = filled_cache(1, 2, 290, 128, 325)
    k, v = (R.dense(c, s)[0].transpose(0, 1).bfloat16().contiguous().cuda() for c, s in ((kc, ks), (vc, vs)))
    q = randn(329, 1, rows, 4, 128).bfloat16()
    out = torch.empty(rows, 4, 128, dtype=torch.bfloat16, device="cuda")
    q2.q2_self_attention(out, q[0].cuda(), k, v, scale)
    ref, bound = R.attention(q, kc, vc, ks, vs, [290], scale)
    R.within(out, ref[0], bound[0], "dense")


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("S", [500, 3000])  # an item whole, and cut into runs
@pytest.mark.parametrize("nh,T", [(4, 1), (6, 3), (8, 5), (4, 40), (4, 200)])
def test_a_nan_of_v_stays_where_its_weight_is_nothing(dt, S, nh, T):
    """A key whose weight underflows next to another part's is seen all the same."""
    hd, nkv = 128, 1
    k = 0.01 * randn(330, 1, S, nkv, hd)
    k[0, 130] = 8.0                       # its score lies 700 above the others
    kc, vc, ks, vs = empty_cache(1, nkv, S, hd)
    R.append(kc, ks, k, [0])
    R.append(vc, vs, randn(331, 1, S, nkv, hd), [0])
    for i, p in enumerate([2, 37, 69, 100, 129, 140, 163, 200, 230, 260, 290]):
        vc[0, 0, p, 3 + 5 * i] = 127
    q = (0.9 + 0.1 * torch.rand(1, T, nh, hd, generator=torch.Generator().manual_seed(332))).to(DT[dt])
    d = both(kc, vc, ks, vs)
    ref, bound = R.attention(q, kc, vc, ks, vs, [S], 0.7)
    assert int(torch.isnan(ref).sum()) == 11 * T * nh
    out = torch.empty(1, T, nh, hd, dtype=DT[dt], device="cuda")
    q2.q2_kv8_attention(out, q.cuda(), *d, i32([S]).cuda(), 0.7)
    R.within(out, ref, bound, "batch")
    q2.q2_kv8_self_attention(out[0], q[0].cuda(), *(t[0] for t in d), S, 0.7)
    R.within(out, ref, bound, "rows")


@pytest.mark.parametrize("nats", [10.0, 21.0, 22.0, 25.0])
def test_fp32_weights_far_below_a_dominant_key(nats):
    """One key holds nearly all the weight and has a V of 0 or 1, 32767 others share the rest.

    In units of the dominant weight a small one is e^-nats, known to 2^-43 (the fp16 parts' floor,
    2^-37, of probabilities of at least 2^6); the rest as q8_ref.attention counts it, the sums over
    n keys with 2 sqrt(n) steps each."""
    n, hd, nh, T = 32768, 32, 8, 2048
    kc, vc = (torch.zeros(1, n, hd, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.ones(1, n // 64, device="cuda") for _ in range(2))
    one = 7 << 3
    kc[0, 7] = one                        # a score of nats; every other one is 0
    g = torch.Generator(device="cuda").manual_seed(340)
    vc[0, :, :16] = one
    vc[0, :, 16:] = torch.randint(0, 120, (n, 16), generator=g, dtype=torch.uint8, device="cuda")
    vc[0, 7, ::2] = 0
    q = torch.ones(T, nh, hd, device="cuda")
    out = torch.empty_like(q)
    q2.q2_kv8_self_attention(out, q, kc, vc, ks, vs, n, nats / hd)
    v = R.value(vc[0]).cuda()
    w = math.exp(-float(torch.tensor(nats / hd)) * hd)
    seen = torch.arange(n - T + 1, n + 1, device="cuda")
    sums = (v.cumsum(0) - v[7])[seen - 1]
    ref = (v[7] + w * sums) / (1 + w * (seen - 1))[:, None]
    ds = (hd * 2.0 ** -23 + 4 * 2.0 ** -24) * nats
    rel = 2 * ds + 2.0 ** -21 + 4 * math.sqrt(n) * 2.0 ** -23 + 8 * 2.0 ** -24
    bound = rel * ref + 2.0 ** -43 * (sums + ref * seen[:, None])
    for h in range(nh):
        R.within(out[:, h], ref.cpu(), bound.cpu(), f"head {h}")


def test_fp32_query_elements_far_below_the_largest():
    """The row's largest element meets keys of 0; what decides is 2^-34 of it, known to 2^-45."""
    S, hd, nh, nkv = 300, 64, 4, 2
    k = 2.0 ** 14 * randn(345, 1, S, nkv, hd)
    k[..., 0] = 0
    kc, vc, ks, vs = empty_cache(1, nkv, S, hd)
    R.append(kc, ks, k, [0])
    R.append(vc, vs, randn(346, 1, S, nkv, hd), [0])
    for T in (1, 5):
        q = 2.0 ** -14 * randn(347, 1, T, nh, hd)
        q[..., 0] = 2.0 ** 20
        out = torch.empty(1, T, nh, hd, device="cuda")
        q2.q2_kv8_attention(out, q.cuda(), *both(kc, vc, ks, vs), i32([S]).cuda(), 0.2)
        ref, bound = R.attention(q, kc, vc, ks, vs, [S], 0.2)
        # an element's error, 2^-45 of 2^20, moves a score by at most e, and a weight by e^2e
        e = 2.0 ** -25 * float(R.dense(kc, ks).abs().sum(-1).max()) * 0.2
        A = R.attention(q, kc, vc & 127, ks, vs, [S], 0.2)[0]
        R.within(out, ref, bound + math.expm1(2 * e) * A)


def _average_of_rows(out, vc, vs, group, what):
    """Every row lies between the least and the largest of V, but for the roundings of weights (fp16's
    2^-11), their products and sums over S keys (a whole step each, twice) and of the result."""
    v = R.dense(vc, vs)[0].repeat_interleave(group, 0)
    lo, hi, x = v.amin(1), v.amax(1), out.cpu().double()
    tol = hi * (R.HALF[out.dtype] + 2.0 ** -10 + v.shape[1] * 2.0 ** -22)
    assert bool(((x >= lo - tol) & (x <= hi + tol)).all()), what


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("S", [700, 3000])  # an item whole, and cut into runs
@pytest.mark.parametrize("nh,T", [(4, 1), (6, 5), (4, 30), (4, 100)])
@pytest.mark.parametrize("size", [1e5, 1e7, 1e8, 1e10, 1e14])
def test_attention_with_scores_whose_steps_are_large(dt, nh, T, size, S):
    """Scores of 2^20 to 2^50 in powers of two: a step of fp32 there is up to 2^26, and a row is still
    an average of V rows."""
    hd, nkv = 128, 2
    kc, vc, ks, vs = filled_cache(1, nkv, S, hd, 350)
    R.append(vc, vs, 1 + 0.5 * randn(353, 1, S, nkv, hd).clamp(-1, 1), [0])
    q = (size * randn(354, 1, T, nh, hd)).to(DT[dt])
    out = torch.empty(1, T, nh, hd, dtype=DT[dt], device="cuda")
    q2.q2_kv8_attention(out, q.cuda(), *both(kc, vc, ks, vs), i32([S]).cuda(), 0.09)
    ref, bound = R.attention(q, kc, vc, ks, vs, [S], 0.09)
    R.within(out, ref, bound)
    _average_of_rows(out[0], vc, vs, nh // nkv, size)


@pytest.mark.parametrize("S,T", [(700, 300), (4000, 140)])
@pytest.mark.parametrize("size", [1e5, 1e7, 1e8, 1e10, 1e14])
def test_prompt_rows_with_scores_whose_steps_are_large(size, S, T):
    """On the tcgen05 attention a row is an average of V rows up to scores of 2^30, NaN past them."""
    hd, nh, nkv = 128, 8, 2
    kc, vc, ks, vs = filled_cache(1, nkv, S, hd, 355)
    R.append(vc, vs, 1 + 0.5 * randn(358, 1, S, nkv, hd).clamp(-1, 1), [0])
    q = (size * randn(359, 1, T, nh, hd)).bfloat16()
    out = torch.empty(T, nh, hd, dtype=torch.bfloat16, device="cuda")
    q2.q2_kv8_self_attention(out, q[0].cuda(), *(t[0].cuda() for t in (kc, vc, ks, vs)), S, 0.09)
    k = R.dense(kc, ks)[0].repeat_interleave(nh // nkv, 0)
    s = torch.einsum("thd,hsd->ths", q[0].double(), k) * 0.09 * math.log2(math.e)
    hidden = torch.arange(S) > torch.arange(S - T, S)[:, None]
    top = s.masked_fill(hidden[:, None], -math.inf).amax(-1).abs()
    nan = torch.isnan(out.cpu()).all(-1)
    # (a score is off by hd 2^-23 of the sum of its magnitudes at most: far less than the thousandth here)
    assert bool(nan[top > 2.0 ** 30 * 1.001].all()) and not bool(torch.isnan(out.cpu()[top < 2.0 ** 30 / 1.001]).any())
    assert int((top > 2.0 ** 30 * 1.001).sum()) > 0 or size < 1e8
    ref, bound = R.attention(q, kc, vc, ks, vs, [S], 0.09)
    out[nan.cuda()] = ref[0][nan].bfloat16().cuda()
    R.within(out, ref[0], bound[0])
    _average_of_rows(out, vc, vs, nh // nkv, size)


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("nh,T", [(4, 1), (6, 5), (4, 100), (4, 300)])
def test_attention_where_the_scores_factor_leaves_the_range(dt, nh, T):
    """Queries near the type's largest value over keys that are 0 there and large elsewhere; queries
    near its smallest over keys near the largest."""
    S, hd, nkv = 400, 128, 2
    k = torch.zeros(1, S, nkv, hd)
    k[..., 5] = 2.0 ** 30 * (1 + torch.rand(1, S, nkv, generator=torch.Generator().manual_seed(370)))
    k[:, :, :, 9] = randn(371, 1, S, nkv) * 2.0 ** 29
    kc, vc, ks, vs = empty_cache(1, nkv, S, hd)
    R.append(kc, ks, k, [0])
    R.append(vc, vs, randn(372, 1, S, nkv, hd), [0])
    q = torch.zeros(1, T, nh, hd)
    q[..., 0] = 2.0 ** 120                # scores of 0
    q[:, :, 1, 0], q[:, :, 1, 9] = 0.0, 2.0 ** -28
    q = q.to(DT[dt])
    d = both(kc, vc, ks, vs)
    out = torch.empty(1, T, nh, hd, dtype=DT[dt], device="cuda")
    ref, bound = R.attention(q, kc, vc, ks, vs, [S], 0.09)
    q2.q2_kv8_attention(out, q.cuda(), *d, i32([S]).cuda(), 0.09)
    R.within(out, ref, bound, "batch")
    q2.q2_kv8_self_attention(out[0], q[0].cuda(), *(t[0] for t in d), S, 0.09)
    R.within(out, ref, bound, "rows")
    # the other end
    R.append(kc, ks, randn(373, 1, S, nkv, hd) * 2.0 ** 124, [0])
    q = (randn(374, 1, T, nh, hd) * 2.0 ** -122).to(DT[dt])
    ref, bound = R.attention(q, kc, vc, ks, vs, [S], 0.09)
    q2.q2_kv8_attention(out, q.cuda(), *both(kc, vc, ks, vs), i32([S]).cuda(), 0.09)
    R.within(out, ref, bound, "small queries")


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("nh,T", [(4, 1), (6, 5), (2, 40)])
def test_parts_of_values_near_the_largest_are_joined(dt, nh, T):
    S, hd, nkv = 3000, 64, 2
    kc, vc, ks, vs = filled_cache(1, nkv, S, hd, 375, spread=0.5)
    R.append(vc, vs, 2.0 ** 126 * randn(379, 1, S, nkv, hd).clamp(-1.9, 1.9), [0])
    q = randn(379, 1, T, nh, hd).to(DT[dt])
    out = torch.empty(1, T, nh, hd, dtype=DT[dt], device="cuda")
    q2.q2_kv8_attention(out, q.cuda(), *both(kc, vc, ks, vs), i32([S]).cuda(), 0.125)
    ref, bound = R.attention(q, kc, vc, ks, vs, [S], 0.125)
    R.within(out, ref, bound)


@pytest.mark.parametrize("T", [1, 5, 12, 40, 130])
@pytest.mark.parametrize("dt,large,small", [
    ("bf16", 1.0, 2.0 ** -64), ("bf16", 2.0 ** 20, 2.0 ** -57), ("bf16", 2.0 ** 100, 2.0 ** 25),
    ("f32", 1.0, 2.0 ** -64), ("f32", 2.0 ** 110, 2.0 ** -40), ("f32", 2.0 ** 100, 2.0 ** 35),
    ("f32", 2.0 ** 124, 2.0 ** -55)])
def test_attention_to_small_values_beside_large_ones(dt, T, large, small):
    """Every other query row sees, for all its weight is worth, the small blocks alone."""
    S, hd, nh, nkv = 64 * 6, 64, 2, 2
    which = torch.tensor([1, 0, 0, 1, 0, 1]).repeat_interleave(64)   # 1: a block of small values
    k = torch.zeros(1, S, nkv, hd)
    k[0, :, :, 0] = torch.where(which == 1, 4.0, -4.0)[:, None]
    k[..., 1:] = 0.05 * randn(380, 1, S, nkv, hd - 1)
    v = randn(381, 1, S, nkv, hd) * torch.where(which == 1, small, large)[None, :, None, None]
    kc, vc, ks, vs = empty_cache(1, nkv, S, hd)
    R.append(kc, ks, k, [0])
    q = randn(382, 1, T, nh, hd)
    q[0, :, :, 0] = 90.0
    q[0, 1::2, :, 0] = -90.0
    q = q.to(DT[dt])
    for values in (v, v.flip(1)):
        R.append(vc, vs, values, [0])
        out = torch.empty(1, T, nh, hd, dtype=DT[dt], device="cuda")
        for n in (S, 130):
            q2.q2_kv8_attention(out, q.cuda(), *both(kc, vc, ks, vs), i32([n]).cuda(), 1.0)
            ref, bound = R.attention(q, kc, vc, ks, vs, [n], 1.0)
            R.within(out, ref, bound)


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("M,N,K", [(1, 200, 512), (5, 140, 400), (30, 130, 640), (64, 260, 384), (70, 130, 512),
                                   (130, 8200, 400), (2500, 3000, 272), (2500, 3001, 512)])
def test_linear_with_scales_near_the_ends_of_the_range(dt, M, N, K):
    """Scales whose product passes fp32's largest value over a group that sums to 0, and products near
    both ends of the normal range."""
    g = torch.Generator().manual_seed(360)
    xq = torch.randint(0, 127, (M, K), generator=g, dtype=torch.uint8)
    wq = torch.randint(0, 127, (N, K), generator=g, dtype=torch.uint8)
    G, NB = -(-K // 128), -(-N // 128)
    xs, ws = torch.ones(G, M), torch.ones(NB, G)
    # group 0: 1e19 x 1e20, nothing but zeros
    xq[::2, :128], wq[:, :128] = 0, 0
    xs[0], ws[:, 0] = 1e19, 1e20
    xs[0, 2::4], ws[NB - 1, 0] = -1e19, -1e20
    # group 1: 1e18 x 1e19, one product of the smallest codes or none
    xq[:, 128:256], wq[:, 128:256] = 0, 0
    xq[:, 133], wq[::2, 133] = 1, 129
    xs[1], ws[:, 1] = 1e18, 1e19
    # the last group: 1e-19 x 1e-18, all that every third row has
    xs[G - 1], ws[:, G - 1] = 1e-19, 1e-18
    xs[:G - 1, ::3] = 0.0
    out = torch.empty(M, N, dtype=DT[dt], device="cuda")
    q2.q2_linear_q8(out, *both(xq, xs, wq, ws))
    ref, bound = R.linear(xq, xs, wq, ws, None, DT[dt])
    R.within(out, ref, bound)


@pytest.mark.parametrize("M", [3, 130])
def test_linear_scales_that_are_not_finite_reach_their_results(M):
    N, K = 140, 256
    xq, xs = R.quantise(randn(365, M, K), 1)
    wq, ws = R.quantise(randn(366, N, K), 128)
    xs[0, 0], xs[1, 1], ws[1, 1] = math.nan, math.inf, -math.inf
    out = torch.empty(M, N, device="cuda")
    q2.q2_linear_q8(out, *both(xq, xs, wq, ws))
    got = out.cpu()
    assert bool(torch.isnan(got[0]).all())
    assert not bool(torch.isfinite(got[1]).any()) and not bool(torch.isfinite(got[2:, 128:]).any())
    ref, bound = R.linear(xq[2:], xs[:, 2:], wq[:128], ws[:1], None, torch.float32)
    R.within(got[2:, :128], ref, bound)


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("T", [1, 4])
def test_a_sequence_is_the_same_alone_and_beside_others(dt, T):
    """Where its keys are cut depends on its neighbours' lengths; its rows stay within the bound."""
    S, hd, nh, nkv = 3000, 128, 12, 2
    kc, vc, ks, vs = filled_cache(6, nkv, S, hd, 390, spread=0.7)
    q = randn(394, 6, T, nh, hd).to(DT[dt])
    scale = 1.0 / math.sqrt(hd)
    lens = [1555, 3000, 17, T, 2900, 640]
    ref, bound = R.attention(q, kc, vc, ks, vs, lens, scale)
    d = both(q, kc, vc, ks, vs)
    for batch in ([0], [4], [5], [0, 1, 4], [4, 2, 3], [3, 3, 5, 3], [1, 2, 0, 3, 5, 4]):
        at = torch.tensor(batch, device="cuda")
        out = torch.empty(len(batch), T, nh, hd, dtype=DT[dt], device="cuda")
        q2.q2_kv8_attention(out, *(t[at].contiguous() for t in d), i32([lens[b] for b in batch]).cuda(), scale)
        R.within(out, ref[at.cpu()], bound[at.cpu()], batch)


@pytest.mark.parametrize("S,T,nh,nkv", [(300, 140, 8, 2), (900, 130, 8, 2), (1000, 140, 8, 2), (2000, 140, 8, 2),
                                        (3000, 128, 8, 2), (4000, 140, 8, 2), (4000, 129, 6, 3), (4096, 512, 2, 2)])
def test_prompt_rows_cut_into_short_key_ranges(S, T, nh, nkv):
    """Few row blocks over a long cache: a CTA has one to six key tiles, and a row group of it may run
    a tile ahead of the others.  The dense attention shares the kernel."""
    kc, vc, ks, vs = filled_cache(1, nkv, S, 128, 410, spread=0.5)
    R.append(vc, vs, 1 + 0.5 * randn(413, 1, S, nkv, 128).clamp(-1, 1), [0])
    q = randn(414, 1, T, nh, 128).bfloat16()
    ref, bound = R.attention(q, kc, vc, ks, vs, [S], 0.09)
    d = [t[0].cuda() for t in (kc, vc, ks, vs)]
    k, v = (R.dense(c, s)[0].transpose(0, 1).bfloat16().contiguous().cuda() for c, s in ((kc, ks), (vc, vs)))
    qd = q[0].cuda()
    outs = torch.empty(2, 6, T, nh, 128, dtype=torch.bfloat16, device="cuda")
    for i in range(6):
        q2.q2_kv8_self_attention(outs[0, i], qd, *d, S, 0.09)
        q2.q2_self_attention(outs[1, i], qd, k, v, 0.09)
    R.within(outs[0, 0], ref[0], bound[0], "8-bit cache")
    R.within(outs[1, 0], ref[0], bound[0], "dense")
    assert torch.equal(outs, outs[:, :1].expand_as(outs))


@pytest.mark.parametrize("S,T,nh", [(16, 16, 1), (17, 17, 8), (130, 128, 1), (700, 300, 6), (2000, 140, 8)])
def test_dense_self_attention_with_one_kv_head(S, T, nh):
    kc, vc, ks, vs = filled_cache(1, 1, S, 128, 420, spread=0.5)
    q = randn(424, 1, T, nh, 128).bfloat16()
    ref, bound = R.attention(q, kc, vc, ks, vs, [S], 0.09)
    k, v = (R.dense(c, s)[0].transpose(0, 1).bfloat16().contiguous().cuda() for c, s in ((kc, ks), (vc, vs)))
    out = torch.empty(T, nh, 128, dtype=torch.bfloat16, device="cuda")
    q2.q2_self_attention(out, q[0].cuda(), k, v, 0.09)
    R.within(out, ref[0], bound[0])


@pytest.mark.parametrize("S,T", [(700, 300), (4000, 140)])  # whole items, and key ranges that are merged
@pytest.mark.parametrize("size", [2.0 ** 126, 2.0 ** -62])
def test_prompt_rows_over_values_near_the_ends_of_the_range(size, S, T):
    hd, nh, nkv = 128, 8, 2
    kc, vc, ks, vs = filled_cache(1, nkv, S, hd, 400, spread=0.5)
    v = randn(404, 1, S, nkv, hd).clamp(-1.9, 1.9)
    v[..., ::3] = v[..., ::3].abs()
    R.append(vc, vs, size * v, [0])
    vc[0, 1, S - 100, 9] = 127
    q = randn(405, 1, T, nh, hd).bfloat16()
    out = torch.empty(T, nh, hd, dtype=torch.bfloat16, device="cuda")
    q2.q2_kv8_self_attention(out, q[0].cuda(), *(t[0].cuda() for t in (kc, vc, ks, vs)), S, 0.09)
    ref, bound = R.attention(q, kc, vc, ks, vs, [S], 0.09)
    R.within(out, ref[0], bound[0])
