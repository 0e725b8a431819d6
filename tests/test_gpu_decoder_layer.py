"""The layer of examples/decoder_layer.py: norm, FP8 projections, 4-bit cache and attention over it
run together, prompts and single tokens."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def inputs(hidden, lens, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [[torch.randn(n, hidden, device="cuda", generator=g).to(torch.bfloat16) for n in lens] for _ in range(2)]


@pytest.mark.parametrize("hidden,heads,kv_heads,dim,page", [(512, 4, 2, 128, 16), (1024, 16, 4, 64, 64), (768, 2, 1, 256, 1)])
def test_prompt_and_decode_agree(hidden, heads, kv_heads, dim, page):
    """The same tokens as one prompt and as a prompt followed by single tokens. Both quantize the same
    values token by token; the GEMMs sum in another order for few rows, and a bf16 result that falls to
    the other side moves by 2^-8 and may move a 4-bit code, rarely: 1e-2 bounds bf16's own rounding
    (2^-8 per element at most) with as much again for those."""
    from decoder_layer import AttentionLayer, decode_batch
    prompts, steps = [37, 1, 150], 9
    x, res = inputs(hidden, [n + steps for n in prompts])
    layer = AttentionLayer(hidden, heads, kv_heads, dim, len(prompts), max(prompts) + steps, page)
    some = decode_batch(layer, x, res, prompts, steps)
    whole = decode_batch(layer, x, res, [n + steps for n in prompts], 0)
    for a, b in zip(some, whole):
        assert float((a.float() - b.float()).norm() / b.float().norm()) <= 1e-2


def test_layer_is_near_the_fp32_layer():
    """Against fp32 without quantized activations and cache. e2m1 with a power-of-two scale rounds
    by up to a quarter of a value (2 of 8 at a step's end) and at most a sixth of the block's largest
    otherwise: about 0.12 rms on keys and values; e4m3 activations add 0.04 twice. 0.25 is their sum."""
    from decoder_layer import AttentionLayer, decode_batch
    prompts, steps = [200, 65], 3
    x, res = inputs(1024, [n + steps for n in prompts], 2)
    layer = AttentionLayer(1024, 8, 2, 128, len(prompts), max(prompts) + steps)
    out = torch.cat(decode_batch(layer, x, res, prompts, steps)).float()
    ref = layer.reference(torch.cat(x), torch.cat(res), [n + steps for n in prompts])
    assert float((out - ref).norm() / ref.norm()) <= 0.25
