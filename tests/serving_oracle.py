"""Plain 64-bit implementations of the serving operators, and the error bounds of their fp32
kernels (test helper, not product code). CPU tensors throughout."""
import math

import torch

E2M1 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)


# ------------------------------------------------------------------ cache
def pow2_ceil_byte(v: torch.Tensor) -> torch.Tensor:
    """Biased exponent of the smallest power of two >= v (v > 0, float64)."""
    man, ex = torch.frexp(v)  # v = man * 2^ex, man in [0.5, 1)
    return torch.where(man == 0.5, ex - 1, ex).to(torch.int64) + 127


def quantize(x: torch.Tensor):
    """(codes [..., D/2], scale bytes [..., D/32]) uint8 of x [..., D]: byte of the smallest power of
    two >= amax / 6, then the nearest e2m1 value, ties to the even code."""
    g = x.double().unflatten(-1, (-1, 32))
    amax = g.abs().amax(-1, keepdim=True).clamp_min(float(torch.tensor(1e-10, dtype=torch.float32)))
    byte = pow2_ceil_byte(amax / 6)
    # amax / 6 in 64 bits: the quotient can only reach a power of two it does not equal if amax has more
    # than 50 bits, which no fp32 value has
    v = torch.ldexp(g, 127 - byte)
    dist = (v.abs().unsqueeze(-1) - E2M1).abs()
    best = dist.argmin(-1)  # the lower of two equally near ones
    up = (best + 1).clamp_max(7)
    tie = torch.gather(dist, -1, up.unsqueeze(-1)).squeeze(-1) == dist.amin(-1)
    code = torch.where(tie & (best % 2 == 1), up, best)
    code = (code + 8 * torch.signbit(v).long()).flatten(-2)
    return (code[..., 0::2] | (code[..., 1::2] << 4)).to(torch.uint8), byte.squeeze(-1).to(torch.uint8)


def dequantize(codes: torch.Tensor, scales: torch.Tensor) -> torch.Tensor:
    """float64 values of codes [..., D/2] with scale bytes [..., D/32]."""
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).long()
    v = E2M1[c & 7] * torch.where(c >= 8, -1.0, 1.0)
    return torch.ldexp(v.unflatten(-1, (-1, 32)), scales.long().unsqueeze(-1) - 127).flatten(-2)


# ------------------------------------------------------------------ norm
def norm(x, weight, residual, eps):
    """y in float64 (x, weight, residual: tensors of the model's type)."""
    h = x.double() + (0.0 if residual is None else residual.double())
    return h / torch.sqrt(h.square().mean(-1, keepdim=True) + eps) * weight.double()


def norm_bound(K: int) -> float:
    """Relative error of the kernel's fp32 y against the exact one. A lane sums up to 64 squares
    by fma (4 chunks of 16), then 8 additions join at most 64 x 16 lanes' sums in a tree: at most
    64 + 6 + 15 roundings of positive terms; h itself carries one rounding, which counts twice in
    its square. The root halves the sum's relative error; mean, root, division and the two products
    add five roundings and h's own one more."""
    terms = 64 + 6 + 15 + 2
    return (terms / 2 + 7) * 2.0 ** -24


def check_norm_quant(q, s, y, group, ue8m0, tau):
    """q float64 values of the codes [M, K], s float64 scales [M, K/group], y exact. Scales must be
    those of a y within tau; every code must be a nearest one of such a y at the kernel's scale."""
    g = y.unflatten(-1, (-1, group))
    r = g.abs().amax(-1).clamp_min(1e-10) / 448
    if ue8m0:
        lo, hi = pow2_ceil_byte(r * (1 - 2 * tau)), pow2_ceil_byte(r * (1 + 2 * tau))
        byte = pow2_ceil_byte(s)
        assert torch.equal(torch.ldexp(torch.ones_like(s), byte - 127), s), "a scale is no power of two"
        assert bool(((byte >= lo) & (byte <= hi)).all()), "scale byte"
        # where no rounding could decide the byte it is exact
        assert bool((byte == lo)[lo == hi].all())
    else:
        assert float(((s - r) / r).abs().max()) <= tau + 2.0 ** -22, "fp32 scale"
    v = (g / s.unsqueeze(-1)).clamp(-448, 448)
    ulp = torch.ldexp(torch.ones_like(v), (torch.frexp(v.abs().clamp_min(2.0 ** -6))[1] - 1 - 3).to(torch.int64))
    err = (q.unflatten(-1, (-1, group)) - v).abs()
    # 2 tau |v|: y's error and, with fp32 scales, the reciprocal's; a binade's edge is inside it
    assert bool((err <= 0.5 * ulp + 2 * (tau + 2.0 ** -22) * v.abs()).all()), f"code off by {float((err / ulp).max())} steps"


# ------------------------------------------------------------------ attention
def attention(q, k, v, table, kv_lens, q_lens, page, pages, sm_scale, causal):
    """q [T, Hq, D]; k, v float64 [pages, page, Hkv, D]. Returns float64 (out, lse, mass, slack):
    mass [2, T, Hq, D] = sum_j p_j |v_j| and sum_j |v_j|, slack [T, Hq] = the largest
    sm_scale * sum_d |q_d k_jd| of a row."""
    T, Hq, D = q.shape
    Hkv = k.shape[2]
    out = torch.zeros(T, Hq, D, dtype=torch.float64)
    mass = torch.zeros(2, T, Hq, D, dtype=torch.float64)
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64)
    slack = torch.zeros(T, Hq, dtype=torch.float64)
    at = 0
    for b, (n, length) in enumerate(zip(q_lens, kv_lens)):
        toks = torch.arange(length)
        pg = table[b, toks // page].long() if length else toks
        there = (pg >= 0) & (pg < pages)
        kb = k[pg[there], toks[there] % page]
        vb = v[pg[there], toks[there] % page]
        for i in range(n):
            sees = toks[there] < (length - n + 1 + i if causal else length)
            if not bool(sees.any()):
                continue
            for h in range(Hq):
                kk, vv = kb[sees, h * Hkv // Hq], vb[sees, h * Hkv // Hq]
                a = sm_scale * (kk @ q[at + i, h].double())
                s = torch.logsumexp(a, 0)
                p = torch.exp(a - s)
                out[at + i, h], lse[at + i, h] = p @ vv, s
                mass[0, at + i, h], mass[1, at + i, h] = p @ vv.abs(), vv.abs().sum(0)
                slack[at + i, h] = abs(sm_scale) * (kk.abs() @ q[at + i, h].double().abs()).max()
        at += n
    return out, lse, mass, slack


def attention_bounds(out, lse, mass, slack, D, most, dtype):
    """Largest errors of the kernel's (out, lse). Scores: products are exact in fp32 sums of D
    terms, each rounding (or truncation) at most 2^-23 of the sum of magnitudes, then the product
    with the scale and the subtraction of the maximum (4 roundings of at most twice that
    magnitude): delta. A probability moves by 2 delta (it and the sum) and exp2's and log2's last
    places; it is rounded to bf16 (half a unit in the last place: 2^-8 relative at a binade's lower
    end; to two bf16 parts, 2^-16, for fp16); `most` terms are summed in fp32; the output is rounded
    to its type (2^-8, 2^-11). Probabilities under the smallest normal number, and a second part
    that is, may become zero (2^-125 of every |v_j|), and so may such an output."""
    delta = slack * ((D + 8) * 2.0 ** -23) + 2.0 ** -21
    part, unit, least = (2.0 ** -8, 2.0 ** -8, 2.0 ** -126) if dtype == torch.bfloat16 else (2.0 ** -16, 2.0 ** -11, 2.0 ** -25)
    rel = (2 * delta + part + (most + 16) * 2.0 ** -23).unsqueeze(-1)
    lse_bound = delta + (most + 16) * 2.0 ** -23 + 2.0 ** -22 * lse.abs().nan_to_num(posinf=0.0)
    return mass[0] * rel * (1 + unit) + out.abs() * unit + mass[1] * 2.0 ** -125 + least, lse_bound
