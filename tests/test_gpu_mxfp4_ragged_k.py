"""Rows whose length is a multiple of 32 but not of 128 as operands of the 4-bit product: quantized into wider rows of
zeros, whose codes and scales add nothing."""
import pytest
import torch

import serving_oracle as ref
from test_gpu_mxfp4 import fq, product_bound, rows

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,N,K", [(1, 40, 2080), (20, 130, 32), (70, 300, 2880), (333, 520, 160), (4100, 3731, 416)])
def test_rows_filled_up_with_zeros(M, N, K):
    f, wide = fq(), -(-K // 128) * 128
    held, values = [], []
    for n, seed in ((M, 1), (N, 2)):
        x = rows(seed + K, n, K, "bf16")
        q = torch.zeros(n, wide // 2, dtype=torch.uint8, device="cuda")
        s = torch.zeros(n, wide // 32, dtype=torch.uint8, device="cuda")
        f.fp8q_mxfp4_quant(x.cuda(), q[:, :K // 2], s[:, :K // 32])
        assert bool((q[:, K // 2:] == 0).all()) and bool((s[:, K // 32:] == 0).all())
        codes, byte = ref.quantize(x)
        held += [q, s]
        values.append(ref.dequantize(codes, byte).cuda())
    y = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    f.fp8q_gemm_mxfp4(*held, y)
    exact = values[0] @ values[1].t()
    assert float(((y.double() - exact).abs() - product_bound(*values, exact)).max()) <= 0
