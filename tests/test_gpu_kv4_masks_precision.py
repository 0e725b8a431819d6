"""Windowed and tree attention hold their probabilities in 16 bits or more in both types: outputs are as near to 64 bits
as their own rounding."""
import pytest
import torch

import masked_oracle as masked
import serving_oracle as ref
from test_gpu_kv4_masks import DT, cache_of, ends_of, fq, gen, table_of, trees

pytestmark = pytest.mark.gpu


def bound(o, mass, slack, D, most, dtype):
    """serving_oracle.attention_bounds with the probabilities' 2^-16 for both types: two bf16 parts, each rounded by half
    its last place (2^-8), the second of what the first leaves. The output's own rounding is 2^-8 or 2^-11."""
    unit, least = (2.0 ** -8, 2.0 ** -126) if dtype == torch.bfloat16 else (2.0 ** -11, 2.0 ** -25)
    delta = slack * ((D + 8) * 2.0 ** -23) + 2.0 ** -21
    rel = (2 * delta + 2.0 ** -16 + (most + 16) * 2.0 ** -23).unsqueeze(-1)
    return mass[0] * rel * (1 + unit) + o.abs() * unit + mass[1] * 2.0 ** -125 + least


@pytest.mark.parametrize("split", [True, False])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D,page", [(64, 16), (128, 64), (256, 1)])
@pytest.mark.parametrize("kind,q_lens,kv_lens", [
    ("window", [1, 1, 1], [700, 90, 3]), ("window", [1, 3], [9000, 7000]), ("window", [130, 65, 200], [700, 70, 350]),
    ("tree", [25], [600]), ("tree", [5, 64, 33], [900, 64, 2500]), ("tree", [130, 70], [300, 4500]),
])
def test_probabilities_are_not_rounded_to_eight_bits(kind, q_lens, kv_lens, D, page, dtype, split):
    f = fq()
    T, ends, H, G = sum(q_lens), ends_of(q_lens), 2, 4
    window, sinks, scale = 5000 if max(kv_lens) > 5000 else 100, 5, 0.01  # (small scores: their own errors are small)
    mask = trees(q_lens, D)
    table, pages = table_of(kv_lens, page, D)
    c = cache_of(pages, page, H, D, "head", 3)
    q = torch.randn(T, G * H, D, generator=gen(T + D)).to(DT[dtype])
    ip, kv = (torch.tensor(v, dtype=torch.int32).cuda() for v in (ends, kv_lens))
    out = torch.empty(T, G * H, D, dtype=DT[dtype], device="cuda")
    ws = None if split else torch.empty(0, dtype=torch.uint8, device="cuda")
    if kind == "window":
        f.fp8q_kv4_window_attention(q.cuda(), c, table.cuda(), kv, out, scale, window, sinks, ip, workspace=ws)
    else:
        f.fp8q_kv4_tree_attention(q.cuda(), c, table.cuda(), kv, out, scale, mask.cuda(), ip, workspace=ws)
    k64, v64 = (ref.dequantize(x.cpu(), y.cpu()) for x, y in ((c.k, c.k_scales), (c.v, c.v_scales)))

    def sees(b, n, length, at):
        return masked.window_sees(n, length, window, sinks) if kind == "window" else masked.tree_sees(mask[at:at + n], n, length)

    o, _, mass, slack = masked.attention(q, k64, v64, table, kv_lens, q_lens, page, pages, scale, sees)
    err = (out.cpu().double() - o).abs() - bound(o, mass, slack, D, max(kv_lens), DT[dtype])
    assert float(err.max()) <= 0, f"off by {float(err.max())} at {err.argmax()}"
