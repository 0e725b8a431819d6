"""Every kernel of the 4-bit product at sizes that its choice sends there (test_mxfp4_shape.py holds the choice to this
list): all outputs against 64-bit products, with unsplit calls where K is split, each layout of the scales, rows of y at
odd places and rows of the operands as far apart as is allowed."""
import pytest
import torch

import serving_oracle as ref
from test_gpu_mxfp4 import fq, gen, product_bound

pytestmark = pytest.mark.gpu

# M, N, K, kernel, ranges of K. Tiles of 256 x 256 with one, two, three and four steps to a tile, in one round of tiles and
# in several, with 5 units of K; 128 x 128 and 64 x 128 likewise, and with an odd number of units in a range.
SHAPES = [
    (16, 300, 640, "few", 1), (32, 300, 640, "few", 1), (64, 300, 640, "few", 1),
    (6574, 10665, 128, "large", 1), (4100, 3731, 256, "large", 1), (6574, 2050, 384, "large", 1), (2576, 10665, 512, "large", 1),
    (4100, 3731, 640, "large", 1),
    (3001, 2050, 128, "deep", 1), (2050, 2050, 384, "deep", 1), (1000, 4100, 1152, "deep", 1),
    (2668, 23, 27008, "deep", 12), (6574, 16, 7168, "deep", 4),
    (130, 515, 1152, "flat", 1), (64, 40000, 384, "flat", 1), (40, 70001, 640, "flat", 1),
    (4100, 64, 13184, "flat", 3), (300, 300, 8192, "flat", 7), (65, 4096, 7168, "flat", 4),
]


def spaced(t, stride):
    """t [R, C] with rows `stride` elements apart."""
    holder = torch.empty((t.shape[0] - 1) * stride + t.shape[1], dtype=t.dtype, device="cuda")
    return holder.as_strided(t.shape, (stride, 1)).copy_(t)


def operand(seed, n, k, how, far=False):
    """(codes, scales as a program holds them, their values in 64 bits), all on the GPU. far: rows as far apart as may be."""
    g = gen(seed)
    codes = torch.randint(0, 256, (n, k // 2), generator=g, dtype=torch.uint8)
    byte = torch.randint(123, 131, (n, k // 32), generator=g).to(torch.uint8)
    v = ref.dequantize(codes, byte).cuda()
    word = byte.view(torch.int32)
    codes = spaced(codes.cuda(), (1 << 24) - 16) if far else codes.cuda()
    if far:
        return codes, spaced(byte.cuda(), (1 << 24) - 4) if how == "bytes" else spaced(word.cuda(), (1 << 22) - 1), v
    return codes, {"bytes": byte.cuda(), "row": word.cuda(), "col": word.t().contiguous().cuda().t()}[how], v


def check(a, s_a, a64, b, s_b, b64, ldy, first, workspaces):
    f = fq()
    M, N = a.shape[0], b.shape[0]
    exact = a64 @ b64.t()
    bound = product_bound(a64, b64, exact)
    holder = torch.empty(M + 1, ldy, dtype=torch.bfloat16, device="cuda")
    for ws in workspaces:
        holder.fill_(77)
        f.fp8q_gemm_mxfp4(a, s_a, b, s_b, holder[:M, first:N + first], workspace=ws)
        err = (holder[:M, first:N + first].double() - exact).abs_() - bound
        assert float(err.max()) <= 0, f"off by {float(err.max())} at {divmod(int(err.argmax()), N)}"
        assert bool((holder[M] == 77).all()) and bool((holder[:, :first] == 77).all()) and bool((holder[:, N + first:] == 77).all())


@pytest.mark.parametrize("sa,sb,pad,first", [("col", "col", 0, 0), ("bytes", "row", 3, 1), ("row", "bytes", 5, 2)])
@pytest.mark.parametrize("M,N,K,kernel,splits", SHAPES)
def test_every_kernel(M, N, K, kernel, splits, sa, sb, pad, first):
    assert (fq().fp8q_gemm_mxfp4_workspace_size(M, N, K) > 0) == (splits > 1)
    none = torch.empty(0, dtype=torch.uint8, device="cuda")
    check(*operand(M + K, M, K, sa), *operand(N + K, N, K, sb), N + pad, first, (None, none) if splits > 1 else (None,))


@pytest.mark.parametrize("M,N,K,far_a", [(6574, 2050, 640, False), (2576, 10665, 640, True), (6574, 16, 7168, False), (65, 4096, 7168, True)])
def test_rows_as_far_apart_as_may_be(M, N, K, far_a):
    """The last of a tile's rows lies just within 32 bits of its first one, the last of all far past 4 GiB."""
    torch.cuda.empty_cache()
    try:
        a, b = operand(1, M, K, "row" if far_a else "col", far_a), operand(2, N, K, "col" if far_a else "bytes", not far_a)
        check(*a, *b, N + 1, 1, (None,))
    finally:
        a = b = None
        torch.cuda.empty_cache()
