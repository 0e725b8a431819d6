"""The 4-bit product over no elements: its sums are zeros."""
import pytest
import torch

import fp8_group_quant_amd as fq
from test_mxfp4_kv4_abi import GEMM
from test_serving_abi import EALIGN, EDEVICE, EINVAL, OK, no_gpu

EMPTY = dict(GEMM, K=0, a=None, sa=None, b=None, sb=None, lda=0, ldb=0)


@no_gpu
@pytest.mark.parametrize("kw,status", [({}, EDEVICE), (dict(y=None), OK), (dict(M=0), OK), (dict(N=0), OK), (dict(ldy=99), EINVAL),
                                       (dict(M=1, ldy=0), EDEVICE), (dict(y=0x50001), EALIGN), (dict(ldy=-1), EINVAL)])
def test_validation(kw, status):
    assert fq.load_library().fp8q_gemm_mxfp4(*{**EMPTY, **kw}.values()) == status, fq.fp8q_last_error()


@pytest.mark.gpu
@pytest.mark.parametrize("M,N", [(1, 1), (3, 77), (70, 4096), (513, 1025)])
def test_sums_of_nothing_are_zeros(M, N):
    y = torch.full((M + 1, N + 3), 77.0, dtype=torch.bfloat16, device="cuda")
    none = dict(dtype=torch.uint8, device="cuda")
    words = dict(dtype=torch.int32, device="cuda")
    for sa, sb in ((torch.empty(M, 0, **none), torch.empty(N, 0, **words)), (torch.empty(M, 0, **words), torch.empty(N, 0, **none))):
        y.fill_(77)
        fq.fp8q_gemm_mxfp4(torch.empty(M, 0, **none), sa, torch.empty(N, 0, **none), sb, y[:M, :N])
        assert bool((y[:M, :N] == 0).all()) and bool((y[M] == 77).all()) and bool((y[:, N:] == 77).all())
