"""Plain 64-bit references of the 8-bit operators (torch CPU, loops where they are clearer), and
the error bounds that the GPU tests hold the kernels to.

Bounds count roundings, each at most half a step: eps / 2 = 2^-24 (fp32), 2^-8 (bf16), 2^-11
(fp16), relative to the rounded value; a tensor-core sum may truncate, so each of its additions
counts a whole fp32 step, 2^-23 of the sum of the magnitudes."""

import math

import torch

BLOCK, GROUP = 64, 128
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def e4m3_values():
    t = []
    for code in range(256):
        e, m = (code >> 3) & 15, code & 7
        x = math.ldexp(m, -9) if e == 0 else math.ldexp(8 + m, e - 10)
        t.append(float("nan") if code & 127 == 127 else -x if code & 128 else x)
    return torch.tensor(t, dtype=torch.float64)


VALUES = e4m3_values()
_POS = VALUES[:127]  # 0 .. 448, ascending


def value(codes):
    return VALUES[codes.cpu().view(torch.uint8).long()]


def encode(y):
    """uint8 codes of the e4m3 values nearest to y (float64), ties to the even code, held to 448."""
    a = y.abs().clamp(max=448.0)
    nan = torch.isnan(y)
    a = torch.where(nan, 0.0, a)
    hi = torch.searchsorted(_POS, a.contiguous()).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    dl, dh = a - _POS[lo], _POS[hi] - a
    pick = torch.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    code = pick + torch.where(torch.signbit(y), 128, 0)
    return torch.where(nan, torch.full_like(code, 127), code).to(torch.uint8)


def block_scale(amax: float) -> float:
    k = -60
    while k < 119 and amax > 448.0 * 2.0 ** k:
        k += 1
    return 2.0 ** k


def finite_amax(x) -> float:
    a = x.double().abs()
    a = a[torch.isfinite(a)]
    return float(a.max()) if a.numel() else 0.0


def append(codes, scales, new, start):
    """codes uint8 [B, nkv, S, hd], scales [B, nkv, nb] fp32 (CPU, changed in place)."""
    B, T, nkv, hd = new.shape
    for b in range(B):
        p0 = int(start[b])
        if p0 < 0 or p0 + T > codes.shape[2]:
            continue
        for g in range(nkv):
            for blk in range(p0 // BLOCK, (p0 + T - 1) // BLOCK + 1):
                lo, end = blk * BLOCK, min((blk + 1) * BLOCK, p0 + T)
                at = max(lo, p0)
                x = new[b, at - p0:end - p0, g].double()
                s = block_scale(finite_amax(x))
                if at > lo:
                    old = float(scales[b, g, blk])
                    s = max(s, old)
                    if s != old:
                        codes[b, g, lo:at] = encode(value(codes[b, g, lo:at]) * (old / s))
                codes[b, g, at:end] = encode(x / s)
                scales[b, g, blk] = s


def dense(codes, scales):
    s = scales.cpu().double().repeat_interleave(BLOCK, -1)[..., :codes.shape[-2], None]
    return value(codes) * s


def attention(q, kc, vc, ks, vs, lens, scale):
    """(out, bound): out [B, T, nh, hd] in 64 bits, and the error allowed at each element.

    With p the softmax weights and A = sum p |v|: a score's error moves p by at most twice its
    size (numerator and denominator); a score sums hd products (each addition 2^-23 of S1 = sum
    |q||k| scale), and four roundings of the scaled score (2^-24 of S1 each) follow; exp2 and the
    weight's own roundings: 2^-21; the weight enters the product as fp16 (bf16 inputs, 2^-11) or
    as two fp16 parts (2^-22, in 2^-21); the sums over n keys: n * 2^-23 of A for the numerator,
    the same for the denominator; merging and dividing: 8 * 2^-24."""
    dt = q.dtype
    q = q.cpu().double()
    B, T, nh, hd = q.shape
    nkv = kc.shape[1]
    k, v = dense(kc, ks), dense(vc, vs)
    out = torch.zeros(B, T, nh, hd, dtype=torch.float64)
    bound = torch.zeros_like(out)
    for b in range(B):
        for t in range(T):
            n = int(lens[b]) - T + 1 + t
            if n <= 0 or int(lens[b]) > kc.shape[2]:
                continue
            for h in range(nh):
                g = h // (nh // nkv)
                s = (k[b, g, :n] @ q[b, t, h]) * scale
                p = torch.softmax(s, 0)
                out[b, t, h] = p @ v[b, g, :n]
                s1 = float((k[b, g, :n].abs() @ q[b, t, h].abs()).max()) * abs(scale)
                A = p @ v[b, g, :n].abs()
                ds = (hd * 2.0 ** -23 + 4 * 2.0 ** -24) * s1
                w = 2.0 ** -11 if dt == torch.bfloat16 else 0.0
                rel = 2 * ds + 2.0 ** -21 + w + 2 * n * 2.0 ** -23 + 8 * 2.0 ** -24
                bound[b, t, h] = HALF[dt] * out[b, t, h].abs() + (1 + HALF[dt]) * rel * A
    return out, bound


def quantise(x, block_rows):
    """codes uint8 and scales of the definition, its fp32 roundings (the scale; the value that is
    converted) included."""
    r, c = x.shape
    G, R = -(-c // GROUP), -(-r // block_rows)
    codes = torch.zeros(r, c, dtype=torch.uint8)
    scales = torch.zeros(R, G)
    for i in range(R):
        for j in range(G):
            rows, cols = slice(i * block_rows, (i + 1) * block_rows), slice(j * GROUP, (j + 1) * GROUP)
            a = torch.tensor(max(finite_amax(x[rows, cols]), 2.0 ** -100), dtype=torch.float32)
            y = x[rows, cols].double() * (448.0 / a.double())
            codes[rows, cols] = encode(y.float().double())
            scales[i, j] = a / 448.0
    return codes, scales.t().contiguous() if block_rows == 1 else scales


def linear(xq, xs, wq, ws, bias, dt):
    """(out, bound).  The tensor core adds 128 products of a group (each addition 2^-23 of the
    sum of magnitudes), then one product with the scales and one fused addition per group, and
    the operands' common scale is itself a rounded product: (128 + groups + 4) * 2^-23 of A."""
    M, K = xq.shape
    N = wq.shape[0]
    x = value(xq) * xs.cpu().double().t().repeat_interleave(GROUP, 1)[:, :K]
    w = value(wq) * ws.cpu().double().repeat_interleave(128, 0)[:N].repeat_interleave(GROUP, 1)[:, :K]
    y, A = x @ w.t(), x.abs() @ w.abs().t()
    if bias is not None:
        y, A = y + bias.cpu().double(), A + bias.cpu().double().abs()
    rel = (128 + xs.shape[0] + 4) * 2.0 ** -23
    return y, HALF[dt] * y.abs() + (1 + HALF[dt]) * rel * A


def within(got, ref, bound, what=""):
    g = got.detach().cpu().double()
    assert g.shape == ref.shape, (what, g.shape, ref.shape)
    same_nan = torch.equal(torch.isnan(g), torch.isnan(ref))
    assert same_nan, f"{what}: NaN in other places"
    ok = ((g - ref).abs() <= bound) | torch.isnan(ref) | (g == ref)
    if not bool(ok.all()):
        bad = (~ok).nonzero()
        i = tuple(bad[0].tolist())
        raise AssertionError(f"{what}: {bad.shape[0]} of {ok.numel()} elements outside; first {i}: "
                             f"{float(g[i]):.6e} against {float(ref[i]):.6e}, allowed {float(bound[i]):.2e}")
