"""The 4-bit microscaled quantizer, its way back and the product of such operands against plain 64-bit forms."""
import math

import pytest
import torch

import serving_oracle as ref

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def fq():
    import fp8_group_quant_amd
    return fp8_group_quant_amd


def gen(seed):
    return torch.Generator().manual_seed(seed)


def rows(seed, m, k, dtype):
    g = gen(seed)
    return (torch.randn(m, k, generator=g) * torch.exp(torch.randn(m, 1, generator=g))).to(DT[dtype])


def bytes_of(s):
    """Scale bytes [M, K/32] of uint8 bytes or int32 words."""
    s = s.cpu()
    return s if s.dtype == torch.uint8 else torch.stack([(s >> (8 * i)) & 255 for i in range(4)], -1).flatten(-2).to(torch.uint8)


# ------------------------------------------------------------------ quantizer
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("fmt,layout", [("ue8m0", "row"), ("ue8m0", "col"), ("ue8m0_packed", "row"), ("ue8m0_packed", "col")])
@pytest.mark.parametrize("M,K", [(1, 128), (1, 7168), (3, 256), (5, 1152), (130, 512), (2050, 640), (4099, 2048)])
def test_quant(M, K, fmt, layout, dtype):
    f = fq()
    x = rows(M + K, M, K, dtype)
    x[M // 2] = 0
    q, s = f.mxfp4_quant(x.cuda(), fmt, layout)
    codes, byte = ref.quantize(x)
    assert torch.equal(q.cpu(), codes) and torch.equal(bytes_of(s), byte)
    back = f.mxfp4_dequant(q, s, DT[dtype])
    assert torch.equal(back.cpu(), ref.dequantize(codes, byte).to(DT[dtype]))


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M,K", [(1, 32), (7, 96), (33, 160), (5000, 32), (2049, 1056)])
def test_quant_widths_that_fill_no_word(M, K, dtype):
    f = fq()
    x = rows(K, M, K, dtype)
    for layout in ("row", "col"):
        q, s = f.mxfp4_quant(x.cuda(), "ue8m0", layout)
        codes, byte = ref.quantize(x)
        assert torch.equal(q.cpu(), codes) and torch.equal(bytes_of(s), byte)
        assert torch.equal(f.mxfp4_dequant(q, s, torch.float32).cpu(), ref.dequantize(codes, byte).float())


def test_quant_rounding_edges():
    """Ties, block maxima at and around 6 and 1.5 x powers of two, zeros, tiny and huge values."""
    f = fq()
    blocks = []
    for e in (-30, -3, 0, 1, 100, 125):
        base = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 0.2499, 0.2501, 0.7499, 5.0001, 4.999, 1.2501, 6.0, 0, -0.0])
        blocks.append(torch.cat([base, -base]) * 2.0 ** e)
    for m in (1.0, 1.5, 1.5000001, 1.4999999, 1.9999999, 3.0, 6.0, 6.0000005, 5.9999995):
        r = torch.linspace(-1, 1, 32) * m
        blocks += [r, r * 2.0 ** -20]
    blocks += [torch.zeros(32), torch.full((32,), 1e-12), torch.full((32,), 3e38), torch.full((32,), -1e-38)]
    x = torch.stack(blocks).reshape(-1, 64)
    q, s = f.mxfp4_quant(x.cuda(), "ue8m0", "row")
    codes, byte = ref.quantize(x)
    assert torch.equal(q.cpu(), codes) and torch.equal(s.cpu(), byte)


def test_every_code_and_scale_back():
    """Every byte of codes at every scale byte but 0 and 255, in each type: past its largest finite value, that one."""
    f = fq()
    q = torch.arange(256, dtype=torch.uint8).repeat(254, 1)  # [254, 256]: 512 elements per row
    s = torch.arange(1, 255, dtype=torch.uint8).unsqueeze(1).expand(254, 16).contiguous()
    want = ref.dequantize(q, s)
    for name, dt in DT.items():
        got = f.mxfp4_dequant(q.cuda(), s.cuda(), dt).cpu()
        big = torch.finfo(dt).max
        exp = want.clamp(-big, big).to(dt)
        if name != "f16":  # 2^-127 and half of it: subnormal in fp32 and bf16
            assert torch.equal(got[2:], exp[2:])
        else:
            assert torch.equal(got, exp)


def silu64(x):
    g, u = x.double().chunk(2, -1)
    return g * torch.sigmoid(g) * u


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M,K", [(1, 2048), (7, 96), (130, 640), (4099, 1024)])
def test_silu_quant(M, K, dtype):
    """y in fp32 is within 5 roundings (exp twice 2 ulp, the sum, the quotient, the product) of silu(gate) * up: scales are
    those of such a y, and a code is off only where y lies that near to a border."""
    f = fq()
    x = rows(M * K, M, 2 * K, dtype)
    q, s = f.mxfp4_quant(x.cuda(), "ue8m0", "col", silu=True)
    y = silu64(x)
    tau = 8 * 2.0 ** -23
    codes_lo, lo = ref.quantize((y * (1 - tau)))
    codes_hi, hi = ref.quantize((y * (1 + tau)))
    byte = s.cpu()
    assert bool(((byte == lo) | (byte == hi)).all())
    same = (lo == hi).repeat_interleave(16, 1)
    assert bool(((q.cpu() == codes_lo) | (q.cpu() == codes_hi) | ~same).float().mean() > 0.9999)
    v = ref.dequantize(q.cpu(), byte)
    step = torch.ldexp(torch.ones_like(v), (byte.repeat_interleave(32, 1).long() - 127))
    a = (y.abs() / step)
    half = torch.where(a < 2, 0.25, torch.where(a < 4, 0.5, 1.0)) * step
    assert bool(((v - y).abs() <= half + 2 * tau * y.abs() + step * 2.0 ** -22).all())


@pytest.mark.parametrize("silu", [False, True])
def test_quant_views_and_untouched_bytes(silu):
    """Rows inside wider tensors: what lies between them stays as it was."""
    f = fq()
    M, K = 37, 384
    W = 2 * K if silu else K
    x = rows(3, M, W, "bf16")
    q0, s0 = f.mxfp4_quant(x.cuda(), "ue8m0_packed", "row", silu=silu)
    xp = torch.zeros(M, W + 24, dtype=torch.bfloat16, device="cuda")
    xp[:, 8:W + 8] = x.cuda()
    qp = torch.full((M + 1, K // 2 + 32), 0xA5, dtype=torch.uint8, device="cuda")
    sp = torch.full((K // 128 + 1, M + 5), 0x5A5A5A5A, dtype=torch.int32, device="cuda")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    (f.fp8q_silu_mul_mxfp4_quant if silu else f.fp8q_mxfp4_quant)(xp[:, 8:W + 8], qp[:M, 16:K // 2 + 16], sp[:K // 128, :M].t(), stream=st)
    st.synchronize()
    assert torch.equal(qp[:M, 16:K // 2 + 16], q0) and torch.equal(sp[:K // 128, :M].t(), s0)
    assert bool((qp[:, :16] == 0xA5).all()) and bool((qp[:, K // 2 + 16:] == 0xA5).all()) and bool((qp[M] == 0xA5).all())
    assert bool((sp[K // 128] == 0x5A5A5A5A).all()) and bool((sp[:, M:] == 0x5A5A5A5A).all())


# ------------------------------------------------------------------ product
def operand(seed, n, k, how, spread=4):
    """(codes, scales as a program holds them, the values in 64 bits)."""
    g = gen(seed)
    codes = torch.randint(0, 256, (n, k // 2), generator=g, dtype=torch.uint8)
    byte = torch.randint(127 - spread, 128 + spread, (n, k // 32), generator=g).to(torch.uint8)
    word = byte.view(torch.int32)
    s = {"bytes": byte.cuda(), "row": word.cuda(), "col": word.t().contiguous().cuda().t()}[how]
    return codes.cuda(), s, ref.dequantize(codes, byte)


def product_bound(a, b, exact):
    """The matrix core's sums: a term is exact (6-bit products times a power of two); a sum of K terms in fp32, each addition
    rounding or truncating by at most 2^-23 of the sum of magnitudes, and the partial sums of a split once more; then
    bf16 (2^-8 at a binade's lower end)."""
    mag = a.abs() @ b.abs().t()
    return mag * ((a.shape[1] + 32) * 2.0 ** -23) + exact.abs() * 2.0 ** -8 * (1 + 2.0 ** -7) + 2.0 ** -126


def check_product(M, N, K, sa="col", sb="col", split=True, seed=0, spread=4, ldy=None):
    f = fq()
    a, s_a, a64 = operand(seed, M, K, sa, spread)
    b, s_b, b64 = operand(seed + 1, N, K, sb, spread)
    holder = torch.full((M + 1, ldy or N), 77.0, dtype=torch.bfloat16, device="cuda")
    y = holder[:M, :N]
    ws = None if split else torch.empty(0, dtype=torch.uint8, device="cuda")
    f.fp8q_gemm_mxfp4(a, s_a, b, s_b, y, workspace=ws)
    torch.cuda.synchronize()
    exact = a64 @ b64.t()
    err = (y.cpu().double() - exact).abs() - product_bound(a64, b64, exact)
    assert float(err.max()) <= 0, f"off by {float(err.max())} at {divmod(int(err.argmax()), N)}"
    assert bool((holder[M] == 77).all()) and bool((holder[:, N:] == 77).all())


@pytest.mark.parametrize("sa", ["col", "row", "bytes"])
@pytest.mark.parametrize("sb", ["col", "row", "bytes"])
@pytest.mark.parametrize("M", [1, 16, 100, 300])
def test_product_scale_layouts(M, sa, sb):
    check_product(M, 272, 1024, sa, sb)


@pytest.mark.parametrize("split", [True, False])
@pytest.mark.parametrize("K", [128, 256, 384, 640, 1152, 4224])
@pytest.mark.parametrize("M,N", [(1, 1), (1, 17), (2, 4096), (15, 33), (16, 64), (17, 130), (33, 257), (64, 48), (65, 4096), (100, 1),
                                 (127, 255), (129, 513), (200, 129), (257, 255), (512, 384)])
def test_product_sizes(M, N, K, split):
    check_product(M, N, K, split=split, seed=M + N + K, ldy=N + N % 2 + 4)


@pytest.mark.parametrize("M,N,K", [(1, 4097, 7168), (777, 1031, 2176), (2048, 2305, 512), (1300, 4096, 1280), (4100, 260, 256)])
def test_product_larger(M, N, K):
    check_product(M, N, K, seed=5)
    check_product(M, N, K, "bytes", "row", split=False, seed=6)


@pytest.mark.parametrize("M", [1, 20, 140, 600])
def test_product_scales_far_apart(M):
    """Blocks whose scales differ by up to 2^40: the sums' bound is by their largest terms."""
    check_product(M, 160, 768, spread=20, seed=9)


@pytest.mark.parametrize("M", [3, 40, 260])
def test_product_odd_output_strides(M):
    """Rows of y that begin at every address a bf16 may have."""
    f = fq()
    N, K = 131, 512
    a, s_a, a64 = operand(1, M, K, "col")
    b, s_b, b64 = operand(2, N, K, "col")
    want = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    f.fp8q_gemm_mxfp4(a, s_a, b, s_b, want)
    for pad, first in ((2, 1), (1, 0), (4, 3)):
        holder = torch.full((M, N + pad), 77.0, dtype=torch.bfloat16, device="cuda")
        f.fp8q_gemm_mxfp4(a, s_a, b, s_b, holder[:, first:N + first])
        assert torch.equal(holder[:, first:N + first], want)
        assert bool((holder[:, :first] == 77).all()) and bool((holder[:, N + first:] == 77).all())


def test_product_is_the_same_each_time():
    f = fq()
    for M, N, K in ((1, 4096, 7168), (40, 4096, 7168), (128, 1024, 4096), (700, 1024, 1024)):
        a, s_a, _ = operand(1, M, K, "col")
        b, s_b, _ = operand(2, N, K, "col")
        ys = []
        for _ in range(4):
            ys.append(torch.empty(M, N, dtype=torch.bfloat16, device="cuda"))
            f.fp8q_gemm_mxfp4(a, s_a, b, s_b, ys[-1])
        assert all(torch.equal(ys[0], y) for y in ys[1:])


def test_quantized_layer():
    """x through the quantizer and a product, silu * up through the quantizer and a second product: the same as the
    operators' own 64-bit forms on the codes."""
    f = fq()
    g = gen(3)
    M, D, I = 45, 512, 384
    x = torch.randn(M, D, generator=g).to(torch.bfloat16).cuda()
    w1, w2 = (torch.randn(2 * I, D, generator=g) / D ** 0.5).cuda(), (torch.randn(D, I, generator=g) / I ** 0.5).cuda()
    (b1, t1), (b2, t2) = f.mxfp4_quant(w1), f.mxfp4_quant(w2)
    q, s = f.mxfp4_quant(x)
    h = torch.empty(M, 2 * I, dtype=torch.bfloat16, device="cuda")
    f.fp8q_gemm_mxfp4(q, s, b1, t1, h)
    q2, s2 = f.mxfp4_quant(h, silu=True)
    y = torch.empty(M, D, dtype=torch.bfloat16, device="cuda")
    f.fp8q_gemm_mxfp4(q2, s2, b2, t2, y)
    val = lambda c, t: ref.dequantize(c.cpu(), bytes_of(t))  # noqa: E731
    for got, a, b in ((h, val(q, s), val(b1, t1)), (y, val(q2, s2), val(b2, t2))):
        want = a @ b.t()
        assert bool(((got.cpu().double() - want).abs() <= product_bound(a, b, want)).all())
