"""Windowed and tree attention on a stream that is not the current one: what it reads is made before the stream goes on,
and kept until it is done."""
import pytest
import torch

from test_gpu_kv4_masks import cache_of, ends_of, fq, gen, table_of, trees

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["window", "tree"])
def test_views_and_other_streams(kind):
    """Queries, outputs, masks and tables that are views with strides of their own, and contiguous ones through the
    allocating forms: the same results."""
    f = fq()
    q_lens, lens = [3, 1, 20], [90, 40, 200]
    T = sum(q_lens)
    table, pages = table_of(lens, 16, 3)
    c = cache_of(pages, 16, 2, 64, "token", 4)
    q = torch.randn(T, 2, 8, 64, generator=gen(5)).to(torch.float16).cuda()[:, 1]
    wide_table = torch.full((3, table.shape[1] + 3), -1, dtype=torch.int32)
    wide_table[:, 1:1 + table.shape[1]] = table
    tb = wide_table.cuda()[:, 1:1 + table.shape[1]]
    wide_mask = torch.full((T, 4), -1, dtype=torch.int32)
    wide_mask[:, 1:2] = trees(q_lens, 12)
    mask = wide_mask.cuda()[:, 1:2]
    ip, kv = (torch.tensor(v, dtype=torch.int32).cuda() for v in (ends_of(q_lens), lens))
    holder = torch.full((T, 3, 8, 64), 5.0, dtype=torch.float16, device="cuda")
    whole = [t.contiguous() for t in (q, tb, mask)]  # held to the end of the test
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())  # after the last of them
    if kind == "window":
        f.fp8q_kv4_window_attention(q, c, tb, kv, holder[:, 2], 0.1, 30, 4, ip, stream=st)
        b = f.kv4_window_attention(whole[0], c, whole[1], kv, 0.1, 30, 4, ip, stream=st)
    else:
        f.fp8q_kv4_tree_attention(q, c, tb, kv, holder[:, 2], 0.1, mask, ip, stream=st)
        b = f.kv4_tree_attention(whole[0], c, whole[1], kv, 0.1, whole[2], ip, stream=st)
    st.synchronize()
    assert torch.equal(holder[:, 2], b) and bool((holder[:, :2] == 5).all())
