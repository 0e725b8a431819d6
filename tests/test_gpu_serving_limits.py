"""The serving operators at the limits of their ranges: sizes, magnitudes and scales that the entry
points accept and that ordinary cases do not come near."""
import pytest
import torch

import serving_oracle as ref

pytestmark = pytest.mark.gpu


def fq():
    import fp8_group_quant_amd
    return fp8_group_quant_amd


def gen(seed):
    return torch.Generator().manual_seed(seed)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("K,group,fmt", [(16400, 16400, "f32"), (16512, 128, "ue8m0"), (32768, 128, "ue8m0_packed"), (32800, 32, "f32"),
                                         (49152, 49152, "ue8m0"), (65520, 65520, "f32"), (65536, 64, "ue8m0")])
def test_long_norm_rows(K, group, fmt, dtype):
    """Rows of two and four passes, with and without a residual, and updated in place."""
    from test_gpu_serving import DT, check_norm, run_norm, values
    x, res = values(K, 3, K, dtype=dtype), values(K + 1, 3, K, dtype=dtype, spread=0.5)
    w = (1 + 0.2 * torch.randn(K, generator=gen(K))).to(DT[dtype])
    check_norm(x, w, res, group, fmt, "row")
    check_norm(x, w, None, group, fmt, "col")
    f = fq()
    q0, s0, h0 = run_norm(x, w, res, group, fmt, "row")
    for into in (0, 1):
        xr = [x.cuda(), res.cuda()]
        q = torch.empty(3, K, dtype=torch.uint8, device="cuda")
        s = f.alloc_scales(None, 3, K // group, fmt, "row", "cuda")
        f.fp8q_rms_norm_group_quant(xr[0], w.cuda(), q, s, group, residual=xr[1], residual_out=xr[into])
        torch.cuda.synchronize()
        assert torch.equal(q.cpu().view(torch.float8_e4m3fn).double(), q0) and torch.equal(xr[into].cpu(), h0)


def saturated(v, dtype):
    """float64 values rounded to dtype, those past its largest finite value as that value."""
    most = torch.finfo(dtype).max
    return v.clamp(-most, most).to(dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_largest_finite_values_read_back_finite(dtype):
    """Codes round up to 4 / 3.5 of a value: the largest finite inputs are held as more than their type
    has, and come back as its largest finite value."""
    f = fq()
    most = torch.finfo(dtype).max
    steps = torch.cat([torch.linspace(0.80, 1.0, 63, dtype=torch.float64), torch.tensor([57344 / 65504], dtype=torch.float64)])
    x = (most * steps).to(dtype).reshape(64, 1, 1) * torch.tensor([1.0, -1.0] * 32, dtype=dtype)
    assert bool(torch.isfinite(x).all())
    n = x.shape[0]
    c = f.alloc_kv4_cache(n, 1, 1, 128)
    x = torch.cat([x, x / 3], -1).cuda()
    slots = torch.arange(n, dtype=torch.int32).cuda()
    f.fp8q_kv4_write(x, -x, slots, c)
    k, v = f.kv4_read(c, slots, dtype)
    torch.cuda.synchronize()
    exp = saturated(ref.dequantize(*ref.quantize(x.cpu())), dtype)
    assert bool(torch.isfinite(k).all()) and bool((k.abs() == most).any())
    assert torch.equal(k.cpu(), exp) and torch.equal(v.cpu(), -exp)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_every_scale_byte_reads_back(dtype):
    """Every code at every scale byte that is a number."""
    f = fq()
    c = f.alloc_kv4_cache(255, 1, 1, 64)
    codes = torch.arange(16).repeat(4)
    packed = (codes[0::2] | (codes[1::2] << 4)).to(torch.uint8)
    for t in (c.k, c.v):
        t.copy_(packed.cuda().expand(t.shape))
    for t in (c.k_scales, c.v_scales):
        t.copy_(torch.arange(255, dtype=torch.uint8).cuda().reshape(-1, 1, 1, 1).expand(t.shape))
    k, v = f.kv4_read(c, torch.arange(255, dtype=torch.int32).cuda(), dtype)
    exp = saturated(ref.dequantize(c.k.cpu(), c.k_scales.cpu())[:, 0], dtype)
    assert torch.equal(k.cpu(), exp) and torch.equal(v.cpu(), exp)


@pytest.mark.parametrize("queries,tokens", [(1, 1), (1, 70), (3, 3000), (40, 100), (40, 2500)])
def test_fp16_outputs_stay_finite(queries, tokens):
    """Values at the top of fp16, all held as 65536 (and half of them negative): averages of one sign are
    the largest finite value, whole units and joined pieces alike."""
    f = fq()
    D, page = 64, 16
    pages = -(-tokens // page)
    c = f.alloc_kv4_cache(pages, page, 1, D)
    sign = torch.tensor([1.0, -1.0] * 32)
    v = (torch.linspace(57344, 65504, tokens)[:, None, None] * sign).to(torch.float16).cuda()
    k = torch.randn(tokens, 1, D, generator=gen(3)).to(torch.float16).cuda()
    f.fp8q_kv4_write(k, v, torch.arange(tokens, dtype=torch.int32).cuda(), c)
    q = torch.randn(queries, 2, D, generator=gen(4)).to(torch.float16).cuda()
    args = (q, c, torch.arange(pages, dtype=torch.int32).cuda()[None], torch.tensor([tokens], dtype=torch.int32).cuda())
    out = f.kv4_attention(*args, 0.125, causal=False, q_indptr=torch.tensor([0, queries], dtype=torch.int32).cuda())
    torch.cuda.synchronize()
    assert torch.equal(out.cpu(), (65504 * sign).to(torch.float16).expand(out.shape))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("queries", [1, 40])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_values_at_every_scale(D, queries, dtype):
    """Caches of one token, whose softmax is 1 up to the roundings of its exponent, of 1 / sum and of their
    product (2^-22 together, which decides fp16's ties below its normal numbers): the outputs are its
    values, those past the type's largest finite value that value."""
    f = fq()
    first, last = 8, 254
    B = last - first + 1
    c = f.alloc_kv4_cache(B, 1, 1, D)
    c.k.copy_(torch.randint(0, 256, c.k.shape, generator=gen(5), dtype=torch.uint8))
    c.k_scales.fill_(125)
    c.v.copy_(torch.randint(0, 256, c.v.shape, generator=gen(6), dtype=torch.uint8))
    byte = torch.randint(first, last + 1, c.v_scales.shape, generator=gen(7), dtype=torch.uint8)
    byte[..., 0] = torch.arange(first, last + 1, dtype=torch.uint8)[:, None, None]
    c.v_scales.copy_(byte)
    q = torch.randn(B * queries, 2, D, generator=gen(8)).to(dtype).cuda()
    out = f.kv4_attention(q, c, torch.arange(B, dtype=torch.int32).cuda()[:, None], torch.ones(B, dtype=torch.int32).cuda(),
                          0.125, causal=False, q_indptr=torch.arange(0, (B + 1) * queries, queries, dtype=torch.int32).cuda())
    torch.cuda.synchronize()
    exact, got = ref.dequantize(c.v.cpu(), byte), out.cpu().view(B, queries, 2, D)  # [B, 1, 1, D]
    assert bool(((got == saturated(exact * (1 - 2.0 ** -22), dtype)) | (got == saturated(exact * (1 + 2.0 ** -22), dtype))).all())


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("queries,tokens", [(1, 200), (1, 5000), (40, 200), (40, 2500)])
def test_keys_at_the_top(queries, tokens, D):
    """Keys up to bf16's largest value, held as up to 2^128, with queries small enough for ordinary scores."""
    f = fq()
    page, big = 16, 2.0 ** 126
    pages = -(-tokens // page)
    c = f.alloc_kv4_cache(pages, page, 1, D)
    most = torch.finfo(torch.bfloat16).max
    k = (torch.randn(tokens, 1, D, generator=gen(9), dtype=torch.float64) * big).clamp(-most, most).to(torch.bfloat16)
    v = torch.randn(tokens, 1, D, generator=gen(10)).to(torch.bfloat16)
    f.fp8q_kv4_write(k.cuda(), v.cuda(), torch.arange(tokens, dtype=torch.int32).cuda(), c)
    assert int(c.k_scales.max()) == 253
    q = (torch.randn(queries, 2, D, generator=gen(11)) * 2.0 ** -110).to(torch.bfloat16)
    table, scale = torch.arange(pages, dtype=torch.int32)[None], 2.0 ** -16 / D ** 0.5
    out, lse = torch.empty_like(q, device="cuda"), torch.empty(queries, 2, device="cuda")
    f.fp8q_kv4_attention(q.cuda(), c, table.cuda(), torch.tensor([tokens], dtype=torch.int32).cuda(), out, scale, True,
                         torch.tensor([0, queries], dtype=torch.int32).cuda(), lse)
    torch.cuda.synchronize()
    k64, v64 = ref.dequantize(c.k.cpu(), c.k_scales.cpu()), ref.dequantize(c.v.cpu(), c.v_scales.cpu())
    o, l, mass, slack = ref.attention(q, k64, v64, table, [tokens], [queries], page, pages, scale, True)
    ob, lb = ref.attention_bounds(o, l, mass, slack, D, tokens, torch.bfloat16)
    assert float(k64.abs().max()) >= 2.0 ** 128 and float(l.min()) < 20
    assert bool(((out.cpu().double() - o).abs() <= ob).all()) and bool(((lse.cpu().double() - l).abs() <= lb).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("scale", [0.0, 1e-36, 2.0 ** -104, -(2.0 ** -104)])
@pytest.mark.parametrize("queries,tokens", [(3, 200), (3, 3000), (40, 200), (40, 2500)])
def test_small_scales_of_large_scores(queries, tokens, scale, dtype):
    """Products of 2^100 and more, scaled to ordinary scores, to almost nothing or to zero, with tokens
    that are masked and a sequence that sees none."""
    f = fq()
    D, page = 128, 16
    pages = -(-tokens // page)
    c = f.alloc_kv4_cache(pages, page, 1, D)
    k = torch.randn(tokens, 1, D, generator=gen(12)) * 2.0 ** 100
    v = torch.randn(tokens, 1, D, generator=gen(13))
    f.fp8q_kv4_write(k.cuda(), v.cuda(), torch.arange(tokens, dtype=torch.int32).cuda(), c)
    q = torch.randn(2 * queries, 2, D, generator=gen(14)).to(dtype)
    table = torch.arange(pages, dtype=torch.int32).expand(2, -1)
    out, lse = torch.empty_like(q, device="cuda"), torch.empty(2 * queries, 2, device="cuda")
    f.fp8q_kv4_attention(q.cuda(), c, table.contiguous().cuda(), torch.tensor([tokens, 0], dtype=torch.int32).cuda(), out, scale,
                         True, torch.tensor([0, queries, 2 * queries], dtype=torch.int32).cuda(), lse)
    torch.cuda.synchronize()
    k64, v64 = ref.dequantize(c.k.cpu(), c.k_scales.cpu()), ref.dequantize(c.v.cpu(), c.v_scales.cpu())
    o, l, mass, slack = ref.attention(q, k64, v64, table, [tokens, 0], [queries, queries], page, pages, scale, True)
    ob, lb = ref.attention_bounds(o, l, mass, slack, D, tokens, dtype)
    got, sums = out.cpu().double(), lse.cpu().double()
    assert bool((got[queries:] == 0).all()) and bool(torch.isinf(sums[queries:]).all())
    assert bool(((got - o).abs() <= ob).all()) and bool(((sums - l).abs() <= lb)[:queries].all())


def test_many_heads_and_sequences():
    """One query of 2^19 heads in one of 4096 sequences: more (sequence, head) pairs than 2^31. A
    cache of one token makes the softmax 1, so the outputs are its values."""
    f = fq()
    B, H, D = 4096, 1 << 19, 64
    assert f.fp8q_kv4_attention_workspace_size(torch.bfloat16, B, 1, H, H, D, 1) == 0
    c = f.alloc_kv4_cache(1, 1, H, D, "token")
    for t, lo, hi in zip(c, (0, 120, 0, 120), (256, 132, 256, 132)):
        t.copy_(torch.randint(lo, hi, t.shape, generator=gen(1), dtype=torch.uint8))
    q = torch.randn(1, H, D, generator=gen(2)).to(torch.bfloat16).cuda()
    indptr = torch.ones(B + 1, dtype=torch.int32)
    indptr[:4001] = 0
    out = f.kv4_attention(q, c, torch.zeros(B, 1, dtype=torch.int32, device="cuda"),
                          torch.ones(B, dtype=torch.int32, device="cuda"), 0.125, q_indptr=indptr.cuda())
    torch.cuda.synchronize()
    assert torch.equal(out.cpu()[0], ref.dequantize(c.v.cpu(), c.v_scales.cpu())[0, 0].to(torch.bfloat16))


@pytest.mark.parametrize("dtype,M,K,residual", [("bf16", 8192, 7168, True), ("f16", 30011, 576, False), ("bf16", 20000, 1024, True),
                                                ("bf16", 20000, 256, False), ("f32", 8192, 2048, True)])
def test_norm_is_rounded_once(dtype, M, K, residual):
    """A row's fp32 scale is its largest |y| / 448, each rounded to fp32, so it shows whether y is the exact value's
    own rounding. That y is another number takes an error before its rounding that reaches the nearest
    boundary, of probability E|error| / unit. Sums of squares whose last additions are in 64 bits are of
    at least four 32-bit parts, each at most 0.58 sqrt(2) = 0.82 units rms off (the unit 2^-24, halves of
    it per addition, their weights halving from the last one on): 0.41 together, of which the root
    takes half; mean, root and products add nothing of that size. E|error| is then 0.8 x 0.2 units: 0.17
    of the scales at most. (A mean or a root rounded to 32 bits alone would be 0.2 and more.)"""
    f = fq()
    g = torch.Generator(device="cuda").manual_seed(K)
    dt = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}[dtype]
    x = torch.randn(M, K, device="cuda", generator=g).to(dt)
    r = torch.randn(M, K, device="cuda", generator=g).to(dt) if residual else None
    w = (1 + 0.1 * torch.randn(K, device="cuda", generator=g)).to(dt)
    s = f.rms_norm_group_quant(x, w, K, "f32", "row", 1e-6, residual=r)[1].double()
    h = x.float() + r.float() if residual else x.float()  # rounded to fp32, as the formula says
    y = h.double() / torch.sqrt(h.double().square().mean(-1, keepdim=True) + float(torch.tensor(1e-6))) * w.double()
    own = y.abs().amax(-1, keepdim=True).float() / torch.tensor(448.0, device="cuda")
    off = float((s.float() != own).double().mean())
    print(f"{dtype} {M} x {K}: {off:.3f}")
    assert off <= 0.17
