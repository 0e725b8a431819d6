"""The quantizing norm and the 4-bit cache's write, read and attention against plain 64-bit
implementations (serving_oracle.py, which also derives every tolerance), at the sizes, masks
and layouts where they can go wrong."""
import math

import pytest
import torch

import serving_oracle as ref

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def fq():
    import fp8_group_quant_amd
    return fp8_group_quant_amd


def gen(seed):
    return torch.Generator().manual_seed(seed)


def values(seed, *shape, dtype="bf16", spread=1.0):
    """Normal values, each row of the last axis with a magnitude of its own."""
    g = gen(seed)
    x = torch.randn(*shape, generator=g) * torch.exp(spread * torch.randn(*shape[:-1], 1, generator=g))
    return x.to(DT[dtype])


# ------------------------------------------------------------------ norm
def run_norm(x, w, res, group, fmt, layout, eps=1e-6):
    f = fq()
    xd, wd = x.cuda(), w.cuda()
    rd = None if res is None else res.cuda()
    q, s, h = f.rms_norm_group_quant(xd, wd, group, fmt, layout, eps, residual=rd)
    torch.cuda.synchronize()
    M, K = x.shape
    sc = s.cpu()
    if fmt == "ue8m0_packed":
        sc = torch.stack([(sc >> (8 * i)) & 0xFF for i in range(4)], -1).flatten(-2).to(torch.uint8)
    s64 = sc.double() if fmt == "f32" else torch.ldexp(torch.ones(sc.shape, dtype=torch.float64), sc.long() - 127)
    return q.cpu().view(torch.float8_e4m3fn).double(), s64, None if h is None else h.cpu()


def check_norm(x, w, res, group, fmt, layout, eps=1e-6):
    q, s, h = run_norm(x, w, res, group, fmt, layout, eps)
    y = ref.norm(x, w, res, eps)
    ref.check_norm_quant(q, s, y, group, fmt != "f32", ref.norm_bound(x.shape[1]))
    if res is not None:
        assert torch.equal(h, (x.float() + res.float()).to(x.dtype))


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M,K,group,fmt,layout,residual", [
    (1, 7168, 128, "ue8m0", "col", True),
    (1, 16, 16, "f32", "row", True),           # one group of one lane
    (5, 32, 32, "ue8m0", "col", False),
    (33, 576, 64, "f32", "col", False),        # part of a wave's chunk
    (7, 1024, 128, "ue8m0_packed", "row", True),
    (9, 1536, 128, "ue8m0_packed", "col", True),
    (31, 2048, 32, "f32", "row", True),
    (130, 4096, 64, "ue8m0", "row", True),
    (66, 7168, 128, "ue8m0", "col", True),
    (17, 8192, 128, "f32", "row", False),
    (3, 8224, 32, "ue8m0", "col", True),       # one group into the ninth chunk
    (4, 16384, 128, "ue8m0", "row", True),
    (2, 20000, 20000, "f32", "row", True),     # one scale per row
    (3, 7168, 7168, "ue8m0", "col", True),
    (6, 48, 48, "f32", "col", False),
    (2, 65536, 128, "ue8m0", "col", True),     # the longest row
])
def test_norm(M, K, group, fmt, layout, residual, dtype):
    x = values(K + M, M, K, dtype=dtype)
    w = (1 + 0.2 * torch.randn(K, generator=gen(K))).to(DT[dtype])
    res = values(K + M + 1, M, K, dtype=dtype, spread=0.5) if residual else None
    check_norm(x, w, res, group, fmt, layout)


def test_norm_many_rows():
    """More rows than any launch has blocks at once."""
    x = values(5, 70001, 64)
    w = torch.ones(64, dtype=torch.bfloat16)
    check_norm(x, w, None, 32, "ue8m0", "col")


def test_norm_zero_rows_and_outliers():
    x = values(6, 8, 512)
    x[2] = 0
    x[3, 100] = 3e4
    x[4] = 1e-20
    w = torch.randn(512, generator=gen(1)).to(torch.bfloat16)
    w[7] = 0
    for fmt in ("ue8m0", "f32"):
        check_norm(x, w, None, 128, fmt, "row")
    check_norm(x, w, -x, 128, "f32", "row")  # every sum is zero: the amax floor's scale and zero codes


def test_norm_strides_and_aliases():
    """Views with padded rows; the residual updated in place, or into x's own tensor."""
    f = fq()
    M, K = 37, 896
    x, res = values(7, M, K), values(8, M, K, spread=0.3)
    w = torch.ones(K, dtype=torch.bfloat16)
    q0, s0, h0 = run_norm(x, w, res, 64, "ue8m0", "row")
    for into in ("residual", "x"):
        xp = torch.zeros(M, K + 64, dtype=torch.bfloat16, device="cuda")
        rp = torch.zeros(M, K + 128, dtype=torch.bfloat16, device="cuda")
        qp = torch.full((M, K + 32), 0xA5, dtype=torch.uint8, device="cuda")
        xp[:, 8:K + 8] = x.cuda()
        rp[:, :K] = res.cuda()
        s = f.alloc_scales(None, M, K // 64, "ue8m0", "col", "cuda")
        xv, rv = xp[:, 8:K + 8], rp[:, :K]
        f.fp8q_rms_norm_group_quant(xv, w.cuda(), qp[:, :K], s, 64, residual=rv, residual_out=rv if into == "residual" else xv)
        torch.cuda.synchronize()
        assert torch.equal(qp[:, :K].cpu().view(torch.float8_e4m3fn).double(), q0)
        assert bool((qp[:, K:] == 0xA5).all())
        assert torch.equal((rv if into == "residual" else xv).cpu(), h0)
        assert torch.equal((xv if into == "residual" else rv).cpu(), x if into == "residual" else res)
        assert torch.equal(torch.ldexp(torch.ones(s.shape, dtype=torch.float64), s.cpu().long() - 127), s0)
        assert bool((xp[:, :8] == 0).all()) and bool((xp[:, K + 8:] == 0).all()) and bool((rp[:, K:] == 0).all())


# ------------------------------------------------------------------ cache: write and read
def filled_cache(pages, page, heads, D, layout, seed=0):
    """A cache of random bytes (any bytes are codes; the scales stay in the range that is written)."""
    f = fq()
    c = f.alloc_kv4_cache(pages, page, heads, D, layout)
    g = gen(seed)
    for t, hi in ((c.k, 256), (c.v, 256)):
        t.copy_(torch.randint(0, hi, t.shape, generator=g, dtype=torch.uint8))
    for t in (c.k_scales, c.v_scales):
        t.copy_(torch.randint(120, 132, t.shape, generator=g, dtype=torch.uint8))
    return c


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("layout", ["head", "token"])
@pytest.mark.parametrize("T,H,D,page", [(1, 1, 64, 1), (1, 8, 128, 16), (77, 3, 64, 16), (130, 2, 256, 32),
                                        (1000, 8, 128, 64), (33, 5, 128, 1)])
def test_write_then_read(T, H, D, page, layout, dtype):
    f = fq()
    pages = -(-T // page) + 3
    c = filled_cache(pages, page, H, D, layout)
    before = [t.cpu() for t in c]
    kv = values(T + D, T, 2, H, D, dtype=dtype).cuda()
    k, v = kv[:, 0], kv[:, 1]  # views of one tensor
    slots = torch.randperm(pages * page, generator=gen(T))[:T].to(torch.int32)
    slots[T // 2] = -1  # a padding token, except where it is the only one
    if T == 1:
        slots[0] = pages * page - 1
    f.fp8q_kv4_write(k, v, slots.cuda(), c)
    torch.cuda.synchronize()
    want = [t.clone() for t in before]
    live = slots >= 0
    sl = slots[live].long()
    for x, (i, j) in ((k, (0, 1)), (v, (2, 3))):
        codes, scales = ref.quantize(x.cpu()[live])
        want[i][sl // page, sl % page] = codes
        want[j][sl // page, sl % page] = scales
    for got, exp in zip(c, want):
        assert torch.equal(got.cpu(), exp)
    # read back: every slot once more, and slots outside the cache
    back = torch.cat([slots, torch.tensor([pages * page, -5, 2 ** 31 - 1], dtype=torch.int32)])
    ko, vo = f.kv4_read(c, back.cuda(), DT[dtype])
    torch.cuda.synchronize()
    inside = (back >= 0) & (back < pages * page)
    bl = back.clamp(0, pages * page - 1).long()
    for got, (i, j) in ((ko, (0, 1)), (vo, (2, 3))):
        exp = ref.dequantize(want[i], want[j])[bl // page, bl % page]
        exp = torch.where(inside[:, None, None], exp, 0.0).to(DT[dtype])
        assert torch.equal(got.cpu(), exp)


def test_write_rounding_edges():
    """Ties, block maxima at and around 6 and 1.5 x powers of two, zeros, tiny and huge values."""
    f = fq()
    rows = []
    for e in (-30, -3, 0, 1, 100, 125):
        base = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 0.2499, 0.2501, 0.7499, 5.0001, 4.999, 1.2501, 6.0, 0, -0.0])
        rows.append(torch.cat([base, -base]) * 2.0 ** e)
    for m in (1.0, 1.5, 1.5000001, 1.4999999, 1.9999999, 3.0, 6.0, 6.0000005, 5.9999995):
        r = torch.linspace(-1, 1, 32) * m
        rows += [r, r * 2.0 ** -20]
    rows += [torch.zeros(32), torch.full((32,), 1e-12), torch.full((32,), 3e38), torch.full((32,), -1e-38),
             torch.full((32,), 1e-42)]
    x = torch.stack(rows)
    if len(rows) % 2:
        x = torch.cat([x, x[:1]])
    x = x.reshape(-1, 1, 64)
    c = f.alloc_kv4_cache(x.shape[0], 1, 1, 64)
    slots = torch.arange(x.shape[0], dtype=torch.int32)
    f.fp8q_kv4_write(x.cuda(), (-x).cuda(), slots.cuda(), c)
    torch.cuda.synchronize()
    codes, scales = ref.quantize(x)
    assert torch.equal(c.k.cpu()[:, 0], codes) and torch.equal(c.k_scales.cpu()[:, 0], scales)
    codes, scales = ref.quantize(-x)
    assert torch.equal(c.v.cpu()[:, 0], codes) and torch.equal(c.v_scales.cpu()[:, 0], scales)


def test_every_bf16_value():
    """Every finite bf16 value as the largest of a block that also holds two that it scales down."""
    f = fq()
    bits = torch.arange(65536, dtype=torch.int32).to(torch.uint16).view(torch.bfloat16)
    top = bits[torch.isfinite(bits.float())]
    x = torch.zeros(top.numel() // 2, 2, 32, dtype=torch.bfloat16)
    t = top[: top.numel() // 2 * 2].reshape(-1, 2)
    for i in range(16):
        x[:, :, 2 * i] = (t.float() * (1 - i / 16)).to(torch.bfloat16)
        x[:, :, 2 * i + 1] = (t.float() * (i / 37)).to(torch.bfloat16)
    x = x.reshape(-1, 1, 64)
    n = x.shape[0]
    c = f.alloc_kv4_cache(-(-n // 64), 64, 1, 64)
    f.fp8q_kv4_write(x.cuda(), x.cuda(), torch.arange(n, dtype=torch.int32).cuda(), c)
    torch.cuda.synchronize()
    codes, scales = ref.quantize(x)
    assert torch.equal(c.k.cpu().reshape(-1, 1, 32)[:n], codes)
    assert torch.equal(c.v_scales.cpu().reshape(-1, 1, 2)[:n], scales)


def test_broadcast_inputs():
    """Keys and values with stride 0 along heads (one head's rows for all)."""
    f = fq()
    x = values(3, 40, 1, 128).cuda()
    c = f.alloc_kv4_cache(4, 16, 4, 128, "token")
    f.fp8q_kv4_write(x.expand(40, 4, 128), x.expand(40, 4, 128), torch.arange(40, dtype=torch.int32).cuda(), c)
    k, v = f.kv4_read(c, torch.arange(40, dtype=torch.int32).cuda(), torch.float32)
    exp = ref.dequantize(*ref.quantize(x.cpu())).float().expand(40, 4, 128)
    assert torch.equal(k.cpu(), exp) and torch.equal(v.cpu(), exp)


# ------------------------------------------------------------------ attention
def make_table(kv_lens, page, extra_pages, seed, width=None):
    """Random pages; entries past a sequence's pages are out of range or another's."""
    counts = [-(-n // page) for n in kv_lens]
    pages = sum(counts) + extra_pages
    order = torch.randperm(pages, generator=gen(seed)).to(torch.int32)
    width = width or max(max(counts), 1)
    table = torch.full((len(kv_lens), width), -1, dtype=torch.int32)
    table[:, 1::2] = 2 ** 30
    at = 0
    for b, n in enumerate(counts):
        table[b, :n] = order[at:at + n]
        at += n
    return table, pages


def poison_unused(c, table, kv_lens, page):
    """Every cached byte that no sequence holds becomes 0xFF (scale bytes: NaN)."""
    used = torch.zeros(c.k.shape[0], page, dtype=torch.bool)
    for b, n in enumerate(kv_lens):
        t = torch.arange(n)
        pg = table[b, t // page].long()
        ok = (pg >= 0) & (pg < c.k.shape[0])
        used[pg[ok], t[ok] % page] = True
    free = ~used.cuda()
    for t in c:
        t[free] = 0xFF


def check_attention(q_lens, kv_lens, Hq, Hkv, D, page, causal=True, dtype="bf16", layout="head", split=True,
                    sm_scale=None, seed=0, drop_page=False, indptr=True, spread=0.3, q_scale=1.0):
    f = fq()
    sm_scale = 1 / math.sqrt(D) if sm_scale is None else sm_scale
    table, pages = make_table(kv_lens, page, 2, seed)
    c = filled_cache(pages, page, Hkv, D, layout, seed)
    if drop_page:  # pages inside a sequence that the table does not have
        table[0, 0] = pages
        table[-1, (kv_lens[-1] - 1) // page // 2] = -7
    poison_unused(c, table, kv_lens, page)
    T = sum(q_lens)
    q = (values(seed + 1, max(T, 1), Hq, D, dtype=dtype, spread=spread) * q_scale)[:T]
    ends = [0]
    for n in q_lens:
        ends.append(ends[-1] + n)
    ip = torch.tensor(ends, dtype=torch.int32).cuda() if indptr else None
    out = torch.full((T + 1, Hq, D), 77.0, dtype=DT[dtype], device="cuda")
    lse = torch.full((T + 1, Hq), 77.0, device="cuda")
    ws = None if split else torch.empty(0, dtype=torch.uint8, device="cuda")
    f.fp8q_kv4_attention(q.cuda(), c, table.cuda(), torch.tensor(kv_lens, dtype=torch.int32).cuda(), out[:T], sm_scale,
                         causal, ip, lse[:T], workspace=ws)
    torch.cuda.synchronize()
    assert bool((out[T] == 77).all()) and bool((lse[T] == 77).all())
    k64, v64 = (ref.dequantize(a.cpu(), torch.where(b.cpu() == 255, 127, b.cpu())) for a, b in ((c.k, c.k_scales), (c.v, c.v_scales)))
    o, l, mass, slack = ref.attention(q, k64, v64, table, kv_lens, q_lens, page, pages, sm_scale, causal)
    ob, lb = ref.attention_bounds(o, l, mass, slack, D, max(kv_lens), DT[dtype])
    got_o, got_l = out[:T].cpu().double(), lse[:T].cpu().double()
    empty = torch.isinf(l)
    assert torch.equal(torch.isinf(got_l), empty)
    assert bool((got_o[empty] == 0).all())
    err = ((got_o - o).abs() - ob).max() if T else torch.tensor(-1.0)
    assert float(err) <= 0, f"out exceeds its bound by {float(err)}"
    lerr = ((got_l - l).abs() - lb)[~empty]
    assert lerr.numel() == 0 or float(lerr.max()) <= 0, f"lse exceeds its bound by {float(lerr.max())}"


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("page", [1, 16, 64])
def test_decode_lengths(D, page, dtype):
    """Single tokens over caches from empty to several chunks, all in one ragged batch."""
    lens = [0, 1, 2, 15, 16, 17, 31, 32, 33, 127, 128, 129, 300, 0, 1000]
    check_attention([1] * len(lens), lens, 8, 2, D, page, dtype=dtype, indptr=False)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (4, 4), (5, 1), (16, 1), (17, 1), (40, 2), (64, 2)])
def test_decode_head_groups(Hq, Hkv):
    check_attention([1, 1, 1], [77, 260, 5], Hq, Hkv, 128, 16, indptr=False)


@pytest.mark.parametrize("split", [True, False])
@pytest.mark.parametrize("layout", ["head", "token"])
def test_decode_long(split, layout):
    check_attention([1, 1], [20000, 777], 8, 2, 128, 64, split=split, layout=layout, indptr=False)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("D,Hq,Hkv,page", [(64, 8, 2, 16), (128, 4, 4, 32), (256, 5, 1, 1)])
def test_ragged_queries(D, Hq, Hkv, page, causal, dtype):
    """Sequences without queries, without cache, with more queries than cached tokens (their first
    rows see nothing), and with query counts around the tiles' sizes."""
    check_attention([0, 1, 5, 9, 16, 33, 7], [40, 200, 5, 3, 100, 33, 0], Hq, Hkv, D, page, causal, dtype)


@pytest.mark.parametrize("split", [True, False])
def test_chunk_of_a_prompt(split):
    check_attention([70, 129], [513, 129], 8, 2, 128, 64, split=split)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D,page", [(64, 1), (64, 16), (128, 64), (256, 8), (256, 32)])
@pytest.mark.parametrize("q_lens,kv_lens,G", [
    ([17, 9, 0, 1], [300, 9, 40, 1000], 4),       # tiles of 64 rows, most of them part filled
    ([130, 65, 1, 200], [400, 70, 500, 150], 1),  # of 128 (or 64): waves without rows, rows without tokens
])
def test_many_query_rows(q_lens, kv_lens, G, D, page, dtype):
    check_attention(q_lens, kv_lens, 2 * G, 2, D, page, dtype=dtype)
    check_attention(q_lens, kv_lens, 2 * G, 2, D, page, causal=False, dtype=dtype, split=False, q_scale=0.02)


def test_pages_missing_from_the_table():
    check_attention([3, 2], [100, 70], 4, 2, 128, 16, drop_page=True)
    check_attention([1], [9], 4, 2, 64, 16, drop_page=True)  # the only page: nothing is seen
    check_attention([90, 70], [300, 170], 4, 2, 128, 16, drop_page=True)
    check_attention([40, 70], [300, 170], 2, 2, 64, 4, drop_page=True)


def test_scales_of_the_scores():
    """Zero, negative and large scales: a flat softmax, the smallest score first, one token alone."""
    for s in (0.0, -0.2, 4.0):
        check_attention([2, 1], [50, 300], 4, 1, 128, 16, sm_scale=s)
    check_attention([1, 1], [500, 64], 4, 1, 64, 16, sm_scale=0.125, q_scale=40.0)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_flat_softmax(D, dtype):
    """Small scores, so that every token counts and the bound is that of the roundings alone."""
    check_attention([1] * 5, [1, 40, 129, 700, 2500], 8, 2, D, 16, dtype=dtype, indptr=False, q_scale=0.01)
    check_attention([40, 3], [500, 90], 4, 1, D, 32, dtype=dtype, q_scale=0.01)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D,page", [(64, 16), (128, 64), (256, 8)])
@pytest.mark.parametrize("most", [450, 1700, 9000])
def test_ragged_queries_over_longer_caches(most, D, page, dtype):
    """Few queries per sequence, the longest cache of one block's steps, of several, or split."""
    check_attention([1, 3, 0, 6, 2], [most, 40, 300, most * 2 // 3, 1], 8, 2, D, page, dtype=dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D,page", [(64, 16), (128, 64), (256, 32)])
def test_many_queries_over_longer_caches(D, page, dtype):
    """Many queries per sequence over a split cache: pieces of units that are cut between blocks."""
    check_attention([40, 0, 25, 33], [2500, 10, 1500, 33], 4, 2, D, page, dtype=dtype)
    check_attention([70, 21], [2200, 700], 8, 2, D, page, dtype=dtype, causal=False, q_scale=0.02)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D,page", [(64, 2), (64, 64), (128, 16), (128, 64), (256, 64)])
def test_more_units_than_compute_units(D, page, dtype):
    """So many query rows that the widest tiles are taken, and blocks take one unit after another."""
    check_attention([150, 140, 90, 160], [300, 140, 200, 230], 32, 8, D, page, dtype=dtype)
    check_attention([300, 140, 290, 160, 1], [300, 440, 200, 230, 0], 32, 8, D, page, dtype=dtype, causal=False, q_scale=0.05)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D,page", [(64, 1), (64, 64), (128, 16), (128, 64), (256, 16)])
@pytest.mark.parametrize("queries", [3, 12, 90])
def test_tokens_that_a_row_does_not_see(queries, D, page, dtype):
    """Scale bytes of NaN in the last two tokens: the queries before them give the same bits."""
    f = fq()
    n, Hkv, G = 200, 2, 4
    table, pages = make_table([n], page, 1, 5)
    c = filled_cache(pages, page, Hkv, D, "head", 6)
    q = values(7, queries, G * Hkv, D, dtype=dtype).cuda()
    ends = torch.tensor([0, queries], dtype=torch.int32).cuda()
    lens = torch.tensor([n], dtype=torch.int32).cuda()
    runs = []
    for poison in (False, True):
        if poison:
            for t in (n - 2, n - 1):
                for x in c:
                    x[table[0, t // page], t % page] = 0xFF
        out, lse = torch.empty_like(q), torch.empty(queries, G * Hkv, device="cuda")
        f.fp8q_kv4_attention(q, c, table.cuda(), lens, out, D ** -0.5, True, ends, lse)
        torch.cuda.synchronize()
        runs.append((out[:-2], lse[:-2]))
    assert torch.equal(runs[0][0], runs[1][0]) and torch.equal(runs[0][1], runs[1][1])
    assert bool(torch.isfinite(runs[0][0]).all())


@pytest.mark.parametrize("queries", [1, 5, 40])
def test_cache_without_pages(queries):
    """No page in the cache, whatever the lengths and the table say: nothing is seen, read or written."""
    f = fq()
    D, Hkv = 128, 2
    c = f.Kv4Cache(*(torch.empty(0, 16, Hkv, w, dtype=torch.uint8, device="cuda") for w in (D // 2, D // 32) * 2))
    q = values(1, 2 * queries, 4 * Hkv, D).cuda()
    table = torch.arange(8, dtype=torch.int32, device="cuda").reshape(2, 4)
    out, lse = torch.full_like(q, 77.0), torch.full(q.shape[:2], 77.0, device="cuda")
    f.fp8q_kv4_attention(q, c, table, torch.tensor([33, 64], dtype=torch.int32, device="cuda"), out, 0.1,
                         q_indptr=torch.tensor([0, queries, 2 * queries], dtype=torch.int32, device="cuda"), lse=lse)
    slots = torch.tensor([0, 5, -1], dtype=torch.int32, device="cuda")
    rows = values(2, 3, Hkv, D).cuda()
    f.fp8q_kv4_write(rows, rows, slots, c)
    k, v = f.kv4_read(c, slots)
    torch.cuda.synchronize()
    assert bool((out == 0).all()) and bool((lse == -math.inf).all())
    assert bool((k == 0).all()) and bool((v == 0).all())


def test_no_queries_or_sequences():
    f = fq()
    c = f.alloc_kv4_cache(4, 16, 2, 64)
    z = torch.zeros(0, dtype=torch.int32, device="cuda")
    q = torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    f.fp8q_kv4_attention(q, c, torch.zeros(0, 1, dtype=torch.int32, device="cuda"), z, q.clone(), 0.1)
    check_attention([0, 0], [10, 3], 4, 2, 64, 16)


def test_most_sequences():
    """4096 sequences, one of them long: the plan's prefix over all of them."""
    lens = [(7 * i) % 23 for i in range(4096)]
    lens[4000] = 3000
    check_attention([1] * 4096, lens, 2, 1, 256, 16, indptr=False)


def test_lengths_past_the_table_are_cut():
    """kv_lens above the table's width, negative lengths and query ranges outside T are clamped."""
    f = fq()
    D, page = 64, 16
    table = torch.arange(6, dtype=torch.int32).reshape(2, 3)
    c = filled_cache(6, page, 1, D, "head", 4)
    q = values(9, 5, 2, D)
    out = torch.full((5, 2, D), 77.0, dtype=torch.bfloat16, device="cuda")
    f.fp8q_kv4_attention(q.cuda(), c, table.cuda(), torch.tensor([1000, -4], dtype=torch.int32).cuda(), out, 0.125,
                         q_indptr=torch.tensor([-3, 2, 900], dtype=torch.int32).cuda())
    torch.cuda.synchronize()
    k64, v64 = ref.dequantize(c.k.cpu(), c.k_scales.cpu()), ref.dequantize(c.v.cpu(), c.v_scales.cpu())
    o, l, mass, slack = ref.attention(q, k64, v64, table, [48, 0], [2, 3], page, 6, 0.125, True)
    ob, _ = ref.attention_bounds(o, l, mass, slack, D, 48, torch.bfloat16)
    assert bool(((out.cpu().double() - o).abs() <= ob).all())


def test_query_ranges_that_overlap_write_nothing_outside():
    """A q_indptr that does not ascend names more rows than there are: no row outside is touched."""
    f = fq()
    table, pages = make_table([300] * 8, 16, 1, 3)
    c = filled_cache(pages, 16, 1, 64, "head", 5)
    out = torch.full((11, 4, 64), 77.0, dtype=torch.bfloat16, device="cuda")
    f.fp8q_kv4_attention(values(1, 10, 4, 64).cuda(), c, table.cuda(), torch.full((8,), 300, dtype=torch.int32).cuda(),
                         out[:10], 0.1, q_indptr=torch.tensor([0, 10, 0, 10, 0, 10, 0, 10, 0], dtype=torch.int32).cuda())
    torch.cuda.synchronize()
    assert bool((out[10] == 77).all())


def test_strided_queries_outputs_and_table():
    f = fq()
    D, page, Hq = 128, 16, 8
    lens = [100, 37, 250]
    table, pages = make_table(lens, page, 1, 3, width=40)
    c = filled_cache(pages, page, 2, D, "head", 5)
    qkv = values(2, 3, Hq + 4, D).cuda()  # queries, then keys and values, of one projection
    wide = torch.full((3, 40 + 24), -1, dtype=torch.int32)
    wide[:, 8:48] = table
    want = torch.empty(3, Hq, D, dtype=torch.bfloat16, device="cuda")
    f.fp8q_kv4_attention(qkv[:, :Hq].contiguous(), c, table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), want, 0.1)
    out = torch.full((Hq, 3, D + 8), 77.0, dtype=torch.bfloat16, device="cuda")
    f.fp8q_kv4_attention(qkv[:, :Hq], c, wide.cuda()[:, 8:48], torch.tensor(lens, dtype=torch.int32).cuda(),
                         out[:, :, :D].transpose(0, 1), 0.1)
    torch.cuda.synchronize()
    assert torch.equal(out[:, :, :D].transpose(0, 1), want) and bool((out[:, :, D:] == 77).all())


def test_results_do_not_change_from_run_to_run():
    f = fq()
    lens = [5000, 123, 9000]
    table, pages = make_table(lens, 64, 1, 3)
    c = filled_cache(pages, 64, 2, 128, "head", 5)
    q = values(2, 3, 16, 128).cuda()
    args = (q, c, table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda())
    first = f.kv4_attention(*args, 0.09)
    for _ in range(5):
        assert torch.equal(f.kv4_attention(*args, 0.09), first)


def test_offsets_past_32_bits():
    """Pages beyond 4 GiB of codes: written, read back and attended to."""
    f = fq()
    H, D, page = 8, 256, 64
    pages = (5 << 30) // (H * page * D // 2)
    c = f.Kv4Cache(*(torch.empty(pages, H, page, w, dtype=torch.uint8, device="cuda").transpose(1, 2)
                     for w in (D // 2, D // 32, D // 2, D // 32)))
    n = 100
    kv = values(1, n, 2, H, D).cuda()
    table = torch.tensor([[pages - 1, 3, pages // 2]], dtype=torch.int32)
    t = torch.arange(n)
    slots = (table[0, t // page].long() * page + t % page).to(torch.int32).cuda()
    f.fp8q_kv4_write(kv[:, 0], kv[:, 1], slots, c)
    k, v = f.kv4_read(c, slots)
    k64, v64 = (ref.dequantize(*ref.quantize(kv[:, i].cpu())) for i in (0, 1))
    assert torch.equal(k.cpu().double(), k64) and torch.equal(v.cpu().double(), v64)
    q = values(2, 1, 16, D)
    out = f.kv4_attention(q.cuda(), c, table.cuda(), torch.tensor([n], dtype=torch.int32).cuda(), 1 / 16)
    pad = torch.zeros(2 * page - n, H, D, dtype=torch.float64)
    k64, v64 = (torch.cat([x, pad]).reshape(2, page, H, D) for x in (k64, v64))
    o, l, mass, slack = ref.attention(q, k64, v64, torch.tensor([[0, 1]]), [n], [1], page, 2, 1 / 16, True)
    ob, _ = ref.attention_bounds(o, l, mass, slack, D, n, torch.bfloat16)
    assert bool(((out.cpu().double() - o).abs() <= ob).all())


# ------------------------------------------------------------------ streams and graphs
def step(f, x, w, q, s, kv, slots, c, table, lens, out, stream=None):
    f.fp8q_rms_norm_group_quant(x, w, q, s, 128, stream=stream)
    f.fp8q_kv4_write(kv[:, 0], kv[:, 1], slots, c, stream=stream)
    f.fp8q_kv4_attention(x.view(x.shape[0], -1, 128), c, table, lens, out, 0.09, stream=stream)


def operands(seed, B=3, Hq=8, Hkv=2):
    f = fq()
    lens = torch.tensor([4000, 77, 1500], dtype=torch.int32)
    table, pages = make_table(lens.tolist(), 64, 1, seed)
    c = filled_cache(pages, 64, Hkv, 128, "head", seed)
    x = values(seed, B, Hq * 128).cuda()
    kv = values(seed + 1, B, 2, Hkv, 128).cuda()
    last = lens - 1
    slots = (table[torch.arange(B), (last // 64).long()] * 64 + last % 64).to(torch.int32).cuda()
    q = torch.empty(B, Hq * 128, dtype=torch.uint8, device="cuda")
    s = f.alloc_scales(None, B, Hq, "ue8m0", "col", "cuda")
    out = torch.empty(B, Hq, 128, dtype=torch.bfloat16, device="cuda")
    return x, torch.ones(Hq * 128, dtype=torch.bfloat16, device="cuda"), q, s, kv, slots, c, table.cuda(), lens.cuda(), out


@pytest.mark.parametrize("raw", [False, True])
def test_another_stream(raw):
    f = fq()
    a = operands(11)
    step(f, *a)
    torch.cuda.synchronize()
    want = [t.clone() for t in (a[2], a[3], a[-1])]
    b = operands(11)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    step(f, *b, stream=st.cuda_stream if raw else st)
    junk = [torch.full((1 << 22,), 1.0, device="cuda") for _ in range(4)]  # may take memory freed on this stream
    st.synchronize()
    for got, exp in zip((b[2], b[3], b[-1]), want):
        assert torch.equal(got, exp)
    del junk


def test_graph_replays():
    f = fq()
    a = operands(21)
    step(f, *a)  # what a library sets up on first use
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(f, *a)
    for seed in (31, 41, 51):
        new = operands(seed)
        for dst, src in zip(a, new):
            for d, s in zip(dst, src) if isinstance(dst, tuple) else ((dst, src),):
                d.copy_(s)
        step(f, *new)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for i in (2, 3, 9):
            assert torch.equal(a[i], new[i])
        for x, y in zip(a[6], new[6]):
            assert torch.equal(x, y)
