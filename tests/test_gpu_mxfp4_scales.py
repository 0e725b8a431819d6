"""Scale bytes at the ends of their range: the way back, and the product."""
import pytest
import torch

import serving_oracle as ref
from test_gpu_mxfp4 import DT, fq, gen, product_bound

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,first", [("f32", 0), ("bf16", 2), ("f16", 0)])
def test_every_code_and_scale_back(dtype, first):
    """Every byte of codes at every scale byte but 255: exact in fp32, subnormal values among them (2^-128 is the least),
    and in bf16 from byte 2 on, the first at which no value is subnormal; in fp16 rounded once (its subnormals too). Past
    the type's largest finite value, that one."""
    q = torch.arange(256, dtype=torch.uint8).repeat(255, 1)
    s = torch.arange(0, 255, dtype=torch.uint8).unsqueeze(1).expand(255, 16).contiguous()
    big = torch.finfo(DT[dtype]).max
    want = ref.dequantize(q, s).clamp(-big, big).to(DT[dtype])
    for scales in (s, s.view(torch.int32)):  # bytes, and words of four
        got = fq().mxfp4_dequant(q.cuda(), scales.cuda(), DT[dtype]).cpu()
        rows = [b for b in range(first, 255) if not torch.equal(got[b], want[b])]
        assert not rows, (rows, got[rows[0]][:16], want[rows[0]][:16])


@pytest.mark.parametrize("M,N,K", [(1, 48, 384), (40, 48, 640), (130, 300, 1152), (1000, 260, 640), (4100, 3731, 256), (300, 300, 8192)])
@pytest.mark.parametrize("lo,hi", [(0, 254), (1, 230), (0, 140), (2, 126)])
def test_product_of_the_least_and_the_largest_scales(M, N, K, lo, hi):
    """Bytes lo on one side and hi on the other, 0 counting as 2^-127 (products are exact before they are added)."""
    codes = [torch.randint(0, 256, (n, K // 2), generator=gen(n + K), dtype=torch.uint8) for n in (M, N)]
    for sa, sb in ((lo, hi), (hi, lo)):
        byte = [torch.full((n, K // 32), s, dtype=torch.uint8) for n, s in ((M, sa), (N, sb))]
        a, b = (ref.dequantize(c, s).cuda() for c, s in zip(codes, byte))
        y = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
        fq().fp8q_gemm_mxfp4(codes[0].cuda(), byte[0].cuda(), codes[1].cuda(), byte[1].cuda(), y)
        exact = a @ b.t()
        err = (y.double() - exact).abs() - product_bound(a, b, exact)
        assert float(err.max()) <= 0 and float(y.double().abs().max()) > 0


@pytest.mark.parametrize("M,N", [(1, 48), (40, 48), (130, 300), (1000, 260), (4100, 3731)])
def test_sums_past_the_range(M, N):
    """A row whose sums pass fp32's largest value is infinite, one whose sums pass bf16's alone too, with its sign; its
    neighbours are as ever. K = 256 codes of 6 and 1: 2^(e + 127 - 254) * 1536 or its negative."""
    K = 256
    six, one = 0x77, 0x22
    a = torch.full((M, K // 2), six, dtype=torch.uint8)
    a[M // 2] = six | 0x88
    b = torch.full((N, K // 2), one, dtype=torch.uint8)
    sa, sb = (torch.full((n, K // 32), 127, dtype=torch.uint8) for n in (M, N))
    sb[N // 3] = 254
    sb[N // 2] = 254 - 11  # 1.5 * 2^126
    y = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    fq().fp8q_gemm_mxfp4(a.cuda(), sa.cuda(), b.cuda(), sb.cuda(), y)
    want = torch.full((M, N), 1536.0)
    want[:, N // 3] = float("inf")
    want[:, N // 2] = 1.5 * 2.0 ** 126
    want[M // 2] *= -1
    assert torch.equal(y.float().cpu(), want)


@pytest.mark.parametrize("dtype", list(DT))
def test_a_scale_byte_of_255_is_nan(dtype):
    """Every code of its 32 elements, zeros too, and no other."""
    q = torch.arange(256, dtype=torch.uint8).repeat(8, 1)
    s = torch.full((8, 16), 127, dtype=torch.uint8)
    s[2, 5] = s[7, 15] = s[3] = 255
    for scales in (s, s.view(torch.int32)):
        got = fq().mxfp4_dequant(q.cuda(), scales.cuda(), DT[dtype]).cpu()
        assert torch.equal(torch.isnan(got), (s == 255).repeat_interleave(32, 1))
