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
