"""Attention over the 4-bit cache with a window and sinks, and of draft trees, against plain 64-bit forms
(masked_oracle.py; the error bounds are serving_oracle's), at the lengths, masks and layouts where they can go wrong."""
import math

import pytest
import torch

import masked_oracle as masked
import serving_oracle as ref

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16}


def fq():
    import fp8_group_quant_amd
    return fp8_group_quant_amd


def gen(seed):
    return torch.Generator().manual_seed(seed)


def cache_of(pages, page, heads, D, layout, seed):
    c = fq().alloc_kv4_cache(pages, page, heads, D, layout)
    g = gen(seed)
    for t in (c.k, c.v):
        t.copy_(torch.randint(0, 256, t.shape, generator=g, dtype=torch.uint8))
    for t in (c.k_scales, c.v_scales):
        t.copy_(torch.randint(120, 132, t.shape, generator=g, dtype=torch.uint8))
    return c


def table_of(kv_lens, page, seed, extra=2):
    counts = [-(-n // page) for n in kv_lens]
    pages = sum(counts) + extra
    order = torch.randperm(pages, generator=gen(seed)).to(torch.int32)
    table = torch.full((len(kv_lens), max(max(counts), 1)), -1, dtype=torch.int32)
    table[:, 1::2] = 2 ** 30
    at = 0
    for b, n in enumerate(counts):
        table[b, :n] = order[at:at + n]
        at += n
    return table, pages


def poison(c, table, kv_lens, page, seen):
    """Every cached byte of a token that no query sees becomes 0xFF (scale bytes: NaN), and the pages without a seen
    token leave the table."""
    used = torch.zeros(c.k.shape[0], page, dtype=torch.bool)
    out = table.clone()
    for b, n in enumerate(kv_lens):
        t = torch.arange(n)
        pg = table[b, t // page].long()
        keep = seen[b] & (pg >= 0) & (pg < c.k.shape[0])
        used[pg[keep], t[keep] % page] = True
        for j in range(-(-n // page)):
            if not bool(keep[j * page:(j + 1) * page].any()):
                out[b, j] = -9 if j % 2 else 2 ** 31 - 1
    free = ~used.cuda()
    for x in c:
        x[free] = 0xFF
    return out


def ends_of(q_lens):
    ends = [0]
    for n in q_lens:
        ends.append(ends[-1] + n)
    return ends


def trees(q_lens, seed, words=None, density=None):
    """Mask rows of random trees, or of random bits where `density` is given."""
    g = gen(seed)
    words = words or max(1, -(-max(q_lens + [1]) // 32))
    rows = []
    for n in q_lens:
        bits = torch.zeros(n, 32 * words, dtype=torch.bool)
        for i in range(n):
            if density is not None:
                bits[i] = torch.rand(32 * words, generator=g) < density
                continue
            parent = int(torch.randint(-1, i, (1,), generator=g)) if i else -1
            if parent >= 0:
                bits[i] = bits[parent]
            if i < 32 * words:
                bits[i, i] = True
        w = (bits.view(n, words, 32).long() << torch.arange(32)).sum(-1)
        rows.append(torch.where(w >= 2 ** 31, w - 2 ** 32, w).to(torch.int32))
    return torch.cat(rows) if rows else torch.zeros(0, words, dtype=torch.int32)


def check(kind, q_lens, kv_lens, Hq, Hkv, D, page, dtype="bf16", layout="head", window=1, sinks=0, mask=None, split=True,
          seed=0, indptr=True, sm_scale=None, q_scale=1.0, stray=True):
    f = fq()
    sm_scale = 1 / math.sqrt(D) if sm_scale is None else sm_scale
    T, ends = sum(q_lens), ends_of(q_lens)

    def sees(b, n, length, at):
        if kind == "window":
            return masked.window_sees(n, length, window, sinks)
        return masked.tree_sees(mask[at:at + n], n, length)

    table, pages = table_of(kv_lens, page, seed)
    c = cache_of(pages, page, Hkv, D, layout, seed)
    if stray:
        seen = [sees(b, n, length, ends[b]).any(0) if n else torch.zeros(length, dtype=torch.bool)
                for b, (n, length) in enumerate(zip(q_lens, kv_lens))]
        table = poison(c, table, kv_lens, page, seen)
    g = gen(seed + 1)
    q = (torch.randn(max(T, 1), Hq, D, generator=g) * torch.exp(0.3 * torch.randn(max(T, 1), Hq, 1, generator=g)) * q_scale)[:T].to(DT[dtype])
    out = torch.full((T + 1, Hq, D), 77.0, dtype=DT[dtype], device="cuda")
    lse = torch.full((T + 1, Hq), 77.0, device="cuda")
    ip = torch.tensor(ends, dtype=torch.int32).cuda() if indptr else None
    ws = None if split else torch.empty(0, dtype=torch.uint8, device="cuda")
    lens = torch.tensor(kv_lens, dtype=torch.int32).cuda()
    if kind == "window":
        f.fp8q_kv4_window_attention(q.cuda(), c, table.cuda(), lens, out[:T], sm_scale, window, sinks, ip, lse[:T], workspace=ws)
    else:
        f.fp8q_kv4_tree_attention(q.cuda(), c, table.cuda(), lens, out[:T], sm_scale, mask.cuda(), ip, lse[:T], workspace=ws)
    torch.cuda.synchronize()
    assert bool((out[T] == 77).all()) and bool((lse[T] == 77).all())
    k64, v64 = (ref.dequantize(a.cpu(), torch.where(b.cpu() == 255, 127, b.cpu())) for a, b in ((c.k, c.k_scales), (c.v, c.v_scales)))
    o, l, mass, slack = masked.attention(q, k64, v64, table, kv_lens, q_lens, page, pages, sm_scale, sees)
    ob, lb = ref.attention_bounds(o, l, mass, slack, D, max(kv_lens), DT[dtype])
    got_o, got_l = out[:T].cpu().double(), lse[:T].cpu().double()
    empty = torch.isinf(l)
    assert torch.equal(torch.isinf(got_l), empty)
    assert bool((got_o[empty] == 0).all())
    err = ((got_o - o).abs() - ob).max() if T else torch.tensor(-1.0)
    assert float(err) <= 0, f"out exceeds its bound by {float(err)}"
    lerr = ((got_l - l).abs() - lb)[~empty]
    assert lerr.numel() == 0 or float(lerr.max()) <= 0, f"lse exceeds its bound by {float(lerr.max())}"


# ------------------------------------------------------------------ window and sinks
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D,page", [(64, 1), (64, 16), (128, 32), (128, 64), (256, 16), (256, 128)])
def test_window_decode_lengths(D, page, dtype):
    """Single tokens over caches from empty to many windows, one ragged batch; window and sinks inside a step."""
    lens = [0, 1, 2, 15, 40, 63, 64, 65, 66, 100, 128, 129, 193, 300, 0, 1000]
    check("window", [1] * len(lens), lens, 8, 2, D, page, dtype, window=37, sinks=3, indptr=False)


@pytest.mark.parametrize("window", [1, 2, 63, 64, 65, 128, 500, 2 ** 40])
@pytest.mark.parametrize("sinks", [0, 1, 64, 65, 200, 2 ** 40])
def test_window_and_sinks_around_the_steps(window, sinks):
    check("window", [1, 5, 1, 3], [700, 5, 64, 260], 4, 2, 64, 16, window=window, sinks=sinks)


@pytest.mark.parametrize("split", [True, False])
@pytest.mark.parametrize("layout", ["head", "token"])
@pytest.mark.parametrize("window,sinks", [(4000, 4), (9000, 0), (16000, 300)])
def test_window_long(window, sinks, layout, split):
    """Windows that are cut between blocks."""
    check("window", [1, 1], [20000, 777], 8, 2, 128, 64, window=window, sinks=sinks, split=split, layout=layout, indptr=False)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D,Hq,Hkv,page", [(64, 8, 2, 16), (128, 4, 4, 32), (256, 5, 1, 1)])
def test_window_ragged_queries(D, Hq, Hkv, page, dtype):
    """Sequences without queries, without cache, with more queries than cached tokens."""
    check("window", [0, 1, 5, 9, 16, 33, 7], [40, 200, 5, 3, 100, 33, 0], Hq, Hkv, D, page, dtype, window=12, sinks=2)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D,page", [(64, 1), (64, 16), (128, 64), (256, 8), (256, 32)])
@pytest.mark.parametrize("split", [True, False])
def test_window_many_query_rows(D, page, dtype, split):
    """Tiles of 64 and 128 rows, their windows apart from the sinks, next to them, and over the whole cache."""
    check("window", [17, 9, 0, 1, 40], [300, 9, 40, 1000, 900], 8, 2, D, page, dtype, window=100, sinks=5, split=split)
    check("window", [130, 65, 200], [700, 70, 150], 2, 2, D, page, dtype, window=70, sinks=66, split=split, q_scale=0.02)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D,page", [(64, 64), (128, 16), (128, 64), (256, 64)])
def test_window_split_many_rows(D, page, dtype):
    """Many rows whose windows are cut between blocks."""
    check("window", [40, 0, 25, 33], [5000, 10, 3500, 33], 4, 2, D, page, dtype, window=2600, sinks=4)
    check("window", [150, 140, 90, 160], [900, 140, 600, 230], 32, 8, D, page, dtype, window=256, sinks=1, q_scale=0.05)


def assert_both_near(a, b, q, c, table, lens, q_lens):
    """Two results of causal attention. Their bits need not agree: calls with masks have tile sizes of their own, whose
    sums run in another order. Each is off by at most the bound, |a - x| <= e and |b - x| <= e, so |a - b| <= 2 e."""
    k64, v64 = (ref.dequantize(x.cpu(), y.cpu()) for x, y in ((c.k, c.k_scales), (c.v, c.v_scales)))
    o, l, mass, slack = masked.attention(q.cpu(), k64, v64, table, lens, q_lens, c.k.shape[1], c.k.shape[0], 0.1,
                                         lambda b, n, length, at: masked.window_sees(n, length, length, 0))
    bound = ref.attention_bounds(o, l, mass, slack, q.shape[2], max(lens), q.dtype)[0]
    for x in (a, b):
        assert bool(((x.cpu().double() - o).abs() <= bound).all())
    assert bool(((a.cpu().double() - b.cpu().double()).abs() <= 2 * bound).all())


def test_window_that_reaches_everything_is_causal_attention():
    f = fq()
    lens, q_lens = [500, 70, 9, 3000], [3, 70, 1, 20]
    table, pages = table_of(lens, 16, 3)
    c = cache_of(pages, 16, 2, 128, "head", 4)
    q = torch.randn(sum(q_lens), 8, 128, generator=gen(5)).to(torch.bfloat16).cuda()
    ip = torch.tensor(ends_of(q_lens), dtype=torch.int32).cuda()
    kv = torch.tensor(lens, dtype=torch.int32).cuda()
    none = torch.empty(0, dtype=torch.uint8, device="cuda")
    outs = []
    for call in (lambda o: f.fp8q_kv4_attention(q, c, table.cuda(), kv, o, 0.1, True, ip, workspace=none),
                 lambda o: f.fp8q_kv4_window_attention(q, c, table.cuda(), kv, o, 0.1, 3000, 0, ip, workspace=none)):
        outs.append(torch.empty_like(q))
        call(outs[-1])
    assert_both_near(*outs, q, c, table, lens, q_lens)


# ------------------------------------------------------------------ draft trees
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D,page", [(64, 1), (64, 16), (128, 32), (128, 64), (256, 16)])
@pytest.mark.parametrize("q_lens,kv_lens", [
    ([1, 3, 8, 0, 4], [1, 3, 40, 20, 300]),       # drafts that are the whole cache, and short of one step
    ([31, 32, 33, 2], [64, 63, 97, 1000]),        # around a word, and around a step
    ([64, 65, 27], [64, 400, 129]),
])
def test_tree_shapes(q_lens, kv_lens, D, page, dtype):
    check("tree", q_lens, kv_lens, 4, 2, D, page, dtype, mask=trees(q_lens, D + page))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D,page", [(64, 16), (128, 64), (256, 32)])
@pytest.mark.parametrize("split", [True, False])
def test_tree_many_rows(D, page, dtype, split):
    """Trees of more than a step and four words, more rows than a tile, over caches that are cut between blocks."""
    check("tree", [130, 20, 70], [180, 2500, 1500], 8, 2, D, page, dtype, mask=trees([130, 20, 70], 7), split=split)
    check("tree", [200], [200], 2, 2, D, page, dtype, mask=trees([200], 8), split=split)


@pytest.mark.parametrize("density", [0.0, 0.3, 1.0])
def test_tree_masks_of_any_bits(density):
    """Rows that see nothing of the draft, rows that see later tokens, bits past the draft."""
    q_lens, kv_lens = [5, 40, 9, 3], [5, 90, 9, 500]
    check("tree", q_lens, kv_lens, 4, 1, 64, 16, mask=trees(q_lens, 9, words=3, density=density))


def test_tree_words_that_do_not_hold_the_draft():
    """Drafted tokens past the mask's words are not seen; no words at all: only what was before."""
    q_lens, kv_lens = [40, 70], [100, 70]
    check("tree", q_lens, kv_lens, 4, 1, 128, 16, mask=trees(q_lens, 10, words=1))
    check("tree", q_lens, kv_lens, 4, 1, 128, 16, mask=torch.zeros(110, 0, dtype=torch.int32))


def test_tree_of_more_tokens_than_are_cached():
    """kv_len below the number of drafted tokens: the first of them are not held."""
    q_lens, kv_lens = [8, 5, 40], [3, 0, 20]
    check("tree", q_lens, kv_lens, 4, 2, 64, 16, mask=trees(q_lens, 11))


def test_tree_single_tokens_without_indptr():
    check("tree", [1] * 6, [1, 2, 64, 65, 300, 1000], 8, 2, 128, 16, mask=torch.ones(6, 1, dtype=torch.int32), indptr=False)
    check("tree", [1] * 3, [1, 2, 64], 8, 2, 128, 16, mask=torch.zeros(3, 1, dtype=torch.int32), indptr=False)


def test_chain_is_causal_attention():
    """A tree in which every drafted token's parent is the one before it."""
    f = fq()
    q_lens, lens = [9, 33, 70, 2], [500, 70, 90, 3000]
    table, pages = table_of(lens, 16, 3)
    c = cache_of(pages, 16, 2, 128, "head", 4)
    q = torch.randn(sum(q_lens), 8, 128, generator=gen(5)).to(torch.bfloat16).cuda()
    ip = torch.tensor(ends_of(q_lens), dtype=torch.int32).cuda()
    kv = torch.tensor(lens, dtype=torch.int32).cuda()
    bits = torch.cat([torch.tril(torch.ones(n, 96, dtype=torch.int64)) for n in q_lens])
    w = (bits.view(-1, 3, 32) << torch.arange(32)).sum(-1)
    mask = torch.where(w >= 2 ** 31, w - 2 ** 32, w).to(torch.int32).cuda()
    none = torch.empty(0, dtype=torch.uint8, device="cuda")
    a, b = torch.empty_like(q), torch.empty_like(q)
    f.fp8q_kv4_attention(q, c, table.cuda(), kv, a, 0.1, True, ip, workspace=none)
    f.fp8q_kv4_tree_attention(q, c, table.cuda(), kv, b, 0.1, mask, ip, workspace=none)
    assert_both_near(a, b, q, c, table, lens, q_lens)


@pytest.mark.parametrize("kind", ["window", "tree"])
def test_views_and_other_streams(kind):
    """Queries, outputs, masks and tables that are views with strides of their own, on a stream that is not the current
    one, and allocating forms."""
    f = fq()
    q_lens, lens = [3, 1, 20], [90, 40, 200]
    T = sum(q_lens)
    table, pages = table_of(lens, 16, 3)
    c = cache_of(pages, 16, 2, 64, "token", 4)
    base = torch.randn(T, 2, 8, 64, generator=gen(5)).to(torch.float16).cuda()
    q = base[:, 1]
    wide_table = torch.full((3, table.shape[1] + 3), -1, dtype=torch.int32)
    wide_table[:, 1:1 + table.shape[1]] = table
    tb = wide_table.cuda()[:, 1:1 + table.shape[1]]
    mask = torch.full((T, 4), -1, dtype=torch.int32)
    mask[:, 1:2] = trees(q_lens, 12)
    mask = mask.cuda()[:, 1:2]
    ip = torch.tensor(ends_of(q_lens), dtype=torch.int32).cuda()
    kv = torch.tensor(lens, dtype=torch.int32).cuda()
    holder = torch.full((T, 3, 8, 64), 5.0, dtype=torch.float16, device="cuda")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    if kind == "window":
        f.fp8q_kv4_window_attention(q, c, tb, kv, holder[:, 2], 0.1, 30, 4, ip, stream=st)
        b = f.kv4_window_attention(q.contiguous(), c, tb.contiguous(), kv, 0.1, 30, 4, ip, stream=st)
    else:
        f.fp8q_kv4_tree_attention(q, c, tb, kv, holder[:, 2], 0.1, mask, ip, stream=st)
        b = f.kv4_tree_attention(q.contiguous(), c, tb.contiguous(), kv, 0.1, mask.contiguous(), ip, stream=st)
    st.synchronize()
    assert torch.equal(holder[:, 2], b)
    assert bool((holder[:, :2] == 5).all())
