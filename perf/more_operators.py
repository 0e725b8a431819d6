"""Operators of a decoder layer whose products and cache are held in 4 bits, as measured cases.

  quant   rows (or silu(gate) * up of them) as e2m1 codes with one power of two (UE8M0) per 32 elements, and
          the rows that they stand for: the operands of the product.
  product Y = A B^T of two matrices in that form, rounded to bf16.
  plan    one serving step's page bookkeeping from the requests' lengths: new pages into the block table, the
          slot and position of every new token, the prefix of the new tokens and the new lengths.
  window  attention over the paged 4-bit cache in which a query sees the last `window` tokens up to its own
          and the first `sinks` of the sequence.
  tree    attention over that cache for drafted tokens that form a tree: each sees what came before the
          draft and the drafted tokens that its mask names.

`own` False computes them with elementary torch operations, `own` True through the package's entry points.
"""
import math

import torch

own = False

BLOCK = 32  # elements that share one scale
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ------------------------------------------------------------------ cases
def _quant(name, rows, width, dtype="bf16", scales="words", layout="col", silu=False):
    """scales: "bytes", or four of them per 32-bit "words"."""
    return {"name": name, "op": "quant", "rows": rows, "width": width, "dtype": dtype, "scales": scales,
            "layout": layout, "silu": silu}


def _product(name, m, n, k, sa="words", sb="words"):
    """sa, sb: column-major "words" of four scales, or row-major "bytes"."""
    return {"name": name, "op": "product", "m": m, "n": n, "k": k, "sa": sa, "sb": sb}


def _plan(name, seqs, new, held, page, new_ragged=0, held_ragged=0):
    return {"name": name, "op": "plan", "seqs": seqs, "q_len": new, "kv_len": held, "page": page,
            "q_ragged": new_ragged, "kv_ragged": held_ragged}


def _attend(name, op, seqs, q_len, kv_len, heads, kv_heads, dim, page, q_ragged=0, kv_ragged=0, dtype="bf16", window=0,
            sinks=0):
    """q_ragged, kv_ragged: by how many percent the lengths of the sequences fall below the longest."""
    return {"name": name, "op": op, "seqs": seqs, "q_len": q_len, "kv_len": kv_len, "heads": heads,
            "kv_heads": kv_heads, "dim": dim, "page": page, "q_ragged": q_ragged, "kv_ragged": kv_ragged,
            "dtype": dtype, "window": window, "sinks": sinks}


def listed():
    return [
        # one token of one user: latency
        _quant("quant one token", 1, 7168),
        # the dense workload's rows, before its product
        _quant("quant dense rows", 4096, 7168),
        # gate and up of an odd number of tokens on the way to the down projection, fp16, scales as plain bytes
        _quant("quant silu odd rows", 6007, 2080, dtype="f16", scales="bytes", layout="row", silu=True),
        # one token through a projection: the weights are all there is to read
        _product("product one token", 1, 4096, 7168),
        # a decode batch with drafted tokens, an output width that fills no tile
        _product("product odd rows", 333, 4104, 2176, sb="bytes"),
        # a prompt through the largest projection
        _product("product cube", 8192, 8192, 8192),
        # a decode step of 64 users: latency
        _plan("plan decode step", 64, 1, 8192, 16, held_ragged=60),
        # prompts of many users start, most of them after a prefix that is there already
        _plan("plan prompts", 256, 1024, 4096, 16, new_ragged=90, held_ragged=100),
        # a decode step of a full batch in a layer that looks back 4096 tokens, ragged contexts
        _attend("window decode batch", "window", 64, 1, 16384, 64, 8, 128, 64, kv_ragged=60, window=4096, sinks=4),
        # a chunk of a prompt in a layer that looks back 1024 tokens
        _attend("window prompt chunk", "window", 2, 2048, 8192, 32, 8, 128, 64, q_ragged=30, kv_ragged=40,
                window=1024, sinks=4),
        # one user's small draft tree: latency
        _attend("tree one user", "tree", 1, 25, 1000, 32, 8, 128, 16),
        # draft trees of a batch, fp16, narrow heads, small pages
        _attend("tree batch", "tree", 16, 64, 4096, 32, 8, 64, 16, q_ragged=50, kv_ragged=70, dtype="f16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("quant", "product", "product", "plan", "window", "tree"))
    if op == "quant":
        silu, scales = rng.random() < 0.4, rng.choice(("bytes", "words"))
        unit = 128 if scales == "words" else 32
        width = unit * max(1, _log(rng, 64, 16384) // unit)
        rows = _log(rng, 1, min(32768, (1 << 24) // width))
        c = _quant("", rows, width, rng.choice(("bf16", "f16", "f32")), scales, rng.choice(("row", "col")), silu)
    elif op == "product":
        n, k = _log(rng, 48, 8192), 128 * _log(rng, 2, 64)
        m = _log(rng, 1, min(8192, (1 << 36) // (n * k)))
        c = _product("", m, n, k, rng.choice(("words", "bytes")), rng.choice(("words", "bytes")))
    elif op == "plan":
        seqs = _log(rng, 1, 1024)
        new = 1 if rng.random() < 0.4 else _log(rng, 2, max(2, min(4096, (1 << 17) // seqs)))
        c = _plan("", seqs, new, _log(rng, 1, 16384), rng.choice((1, 16, 32, 64, 128)), rng.choice((0, 50, 100)),
                  rng.choice((0, 60, 100)))
    else:
        dim, kv_heads, group = rng.choice((64, 128, 256)), rng.choice((1, 2, 4, 8)), rng.choice((1, 4, 5, 8))
        if op == "tree":
            q_len, window, sinks = _log(rng, 2, 160), 0, 0
            seqs = _log(rng, 1, max(1, min(32, 1024 // q_len)))
        else:
            q_len, window, sinks = 1 if rng.random() < 0.5 else _log(rng, 2, 1024), _log(rng, 16, 8192), rng.choice((0, 1, 4, 100))
            seqs = _log(rng, 1, 64 if q_len == 1 else max(1, min(32, 2048 // q_len)))
        most = min(65536, 2 ** 28 // (seqs * kv_heads * dim), 2 ** 34 // (seqs * kv_heads * group * dim * q_len))
        c = _attend("", op, seqs, q_len, q_len + _log(rng, 16, max(16, most)), kv_heads * group, kv_heads, dim,
                    rng.choice((16, 32, 64)), rng.choice((0, 50)), rng.choice((0, 30, 90)), rng.choice(("bf16", "f16")),
                    window, sinks)
    del c["name"]
    return c


def _lengths(count, longest, ragged, least=1):
    """Lengths of `count` sequences, the first of them the longest."""
    return [max(least, longest - longest * ragged * (b * 619 % 997) // 99700) for b in range(count)]


def _spans(case):
    """(query length, cache length) of each sequence; no sequence has more queries than cached tokens."""
    q = _lengths(case["seqs"], case["q_len"], case["q_ragged"])
    kv = _lengths(case["seqs"], case["kv_len"], case["kv_ragged"])
    return [(min(a, b), b) for a, b in zip(q, kv)]


def _held(case):
    """(new tokens, cached tokens) of each sequence of a plan; a cache may be empty."""
    return list(zip(_lengths(case["seqs"], case["q_len"], case["q_ragged"]),
                    _lengths(case["seqs"], case["kv_len"], case["kv_ragged"], 0)))


def _seen(case, n, length):
    """(cached tokens that some query of a sequence sees, pairs of a query and a token that it sees). A tree's
    pairs among the drafted tokens are not counted: they go by its shape."""
    if case["op"] == "tree":
        return length, n * (length - n)
    w, z = case["window"], case["sinks"]
    first = length - n + 1  # tokens up to the first query's own
    ends = range(first, length + 1)
    pairs = sum(min(e, w) + min(max(e - w, 0), z) for e in ends)
    return length - max(0, first - w) + min(max(0, first - w), z), pairs


def work(case):
    op = case["op"]
    if op == "quant":
        size = torch.empty(0, dtype=TYPES[case["dtype"]]).element_size()
        n = case["rows"] * case["width"]
        held = n // 2 + n // BLOCK
        return {"bytes": (2 if case["silu"] else 1) * n * size + held + held + n * size, "flops": (12 if case["silu"] else 4) * n}
    if op == "product":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": (m + n) * (k // 2 + k // BLOCK) + 2 * m * n, "flops": 2 * m * n * k}
    if op == "plan":
        spans, page = _held(case), case["page"]
        fresh = sum(-(-(a + b) // page) - -(-b // page) for a, b in spans)
        tokens = sum(a for a, _ in spans)
        return {"bytes": 20 * len(spans) + 8 * fresh + 8 * tokens, "flops": 8 * tokens}
    size, d, spans = 2, case["dim"], _spans(case)
    seen = [_seen(case, a, b) for a, b in spans]
    tokens = sum(a for a, _ in spans)
    cached = sum(s for s, _ in seen) * case["kv_heads"] * 2 * (d // 2 + d // BLOCK)
    return {"bytes": cached + tokens * case["heads"] * (2 * d * size + 4), "flops": 4 * sum(p for _, p in seen) * case["heads"] * d}


# ------------------------------------------------------------------ what a program has in hand
def _scales_like(byte, how, layout):
    """Scale bytes [rows, groups] as a program holds them: the bytes, or words of four, in this order."""
    if how == "bytes":
        return byte.contiguous() if layout == "row" else byte.t().contiguous().t()
    word = byte.contiguous().view(torch.int32)
    return word if layout == "row" else word.t().contiguous().t()


def _operand(gen, rows, k, how):
    """Codes [rows, k / 2] and scales of rows whose channels have magnitudes of their own."""
    codes = torch.empty(rows, k // 2, dtype=torch.uint8, device="cuda")
    byte = torch.empty(rows, k // BLOCK, dtype=torch.uint8, device="cuda")
    channel = torch.exp(0.5 * torch.randn(k, device="cuda", generator=gen))
    step = max(1, (1 << 26) // k)
    for r in range(0, rows, step):
        n = min(step, rows - r)
        codes[r:r + n], byte[r:r + n] = _encode(torch.randn(n, k, device="cuda", generator=gen) * channel)
    return codes, _scales_like(byte, how, "col" if how == "words" else "row")


def _cache_of(gen, pages, page, heads, dim):
    """(codes, scales) of one cached tensor, viewed as [page, token, head, ...], each head's tokens adjacent."""
    codes = torch.empty(pages, heads, page, dim // 2, dtype=torch.uint8, device="cuda")
    scales = torch.empty(pages, heads, page, dim // BLOCK, dtype=torch.uint8, device="cuda")
    channel = torch.exp(0.5 * torch.randn(heads, 1, dim, device="cuda", generator=gen))
    step = max(1, (1 << 26) // (heads * page * dim))
    for p in range(0, pages, step):
        n = min(step, pages - p)
        codes[p:p + n], scales[p:p + n] = _encode(torch.randn(n, heads, page, dim, device="cuda", generator=gen) * channel)
    return codes.transpose(1, 2), scales.transpose(1, 2)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _tables(counts, width, order):
    """Rows of the first `counts` pages of each sequence, taken from `order` one after the other."""
    table = torch.full((len(counts), width), -1, dtype=torch.int32)
    held, at = order.cpu(), 0
    for b, n in enumerate(counts):
        table[b, :n] = held[at:at + n]
        at += n
    return table.cuda()


def _trees(gen, lengths):
    """Masks int32 [drafted tokens, words] of random trees: bit j of a token's row is set for itself and each of
    its ancestors j. The parent of a token is an earlier one, or none."""
    longest = max(lengths)
    n = len(lengths)
    parent = (torch.rand(n, longest, device="cuda", generator=gen) * torch.arange(longest + 1, device="cuda")[:longest].add(1)).long() - 1
    parent = torch.minimum(parent, torch.arange(longest, device="cuda") - 1)
    up = torch.zeros(n, longest, longest + 1, device="cuda")
    up.scatter_(2, torch.where(parent < 0, longest, parent).unsqueeze(2), 1.0)
    up = up[:, :, :longest].contiguous()
    reach = torch.eye(longest, device="cuda").expand(n, -1, -1) + up
    for _ in range(max(1, longest.bit_length())):
        reach = torch.matmul(reach, reach.contiguous()).clamp_max(1.0)
    words = -(-longest // 32)
    bits = torch.zeros(n, longest, 32 * words, dtype=torch.int64, device="cuda")
    bits[:, :, :longest] = reach > 0
    word = (bits.unflatten(2, (words, 32)) << torch.arange(32, device="cuda")).sum(-1)
    word = torch.where(word >= 2 ** 31, word - 2 ** 32, word).to(torch.int32)
    there = torch.arange(longest, device="cuda") < _ints(lengths).unsqueeze(1)
    return word[there].contiguous()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case)

    def randn(*shape):
        return torch.randn(*shape, device="cuda", generator=gen)

    if case["op"] == "quant":
        m, k, dt = case["rows"], case["width"], TYPES[case["dtype"]]
        wide = 2 * k if case["silu"] else k
        s["x"] = (randn(m, wide) * torch.exp(0.5 * randn(wide))).to(dt)
        s["q"] = torch.empty(m, k // 2, dtype=torch.uint8, device="cuda")
        s["s"] = _scales_like(torch.zeros(m, k // BLOCK, dtype=torch.uint8, device="cuda"), case["scales"], case["layout"])
        s["back"] = torch.empty(m, k, dtype=dt, device="cuda")
        return s
    if case["op"] == "product":
        s["a"], s["s_a"] = _operand(gen, case["m"], case["k"], case["sa"])
        s["b"], s["s_b"] = _operand(gen, case["n"], case["k"], case["sb"])
        s["y"] = torch.empty(case["m"], case["n"], dtype=torch.bfloat16, device="cuda")
        return s
    if case["op"] == "plan":
        spans, page = _held(case), case["page"]
        before = [-(-b // page) for _, b in spans]
        after = [-(-(a + b) // page) for a, b in spans]
        fresh = sum(after) - sum(before)
        pages = sum(after) + 5
        order = torch.randperm(pages, device="cuda", generator=gen).to(torch.int32)
        s["table"] = _tables(before, max(after) + 2, order)
        s["free"] = order[sum(before):].contiguous()  # five more than are needed
        s["pages"], s["fresh"] = pages, fresh
        s["lens"], s["new"] = _ints([b for _, b in spans]), _ints([a for a, _ in spans])
        tokens = sum(a for a, _ in spans)
        for name, n in (("lens_out", len(spans)), ("indptr", len(spans) + 1), ("slots", tokens), ("positions", tokens), ("taken", 1)):
            s[name] = torch.empty(n, dtype=torch.int32, device="cuda")
        return s
    spans, page, h, d, dt = _spans(case), case["page"], case["kv_heads"], case["dim"], TYPES[case["dtype"]]
    counts = [-(-b // page) for _, b in spans]
    pages = sum(counts) + 3
    s["cache"] = _cache_of(gen, pages, page, h, d) + _cache_of(gen, pages, page, h, d)
    s["table"] = _tables(counts, max(counts), torch.randperm(pages, device="cuda", generator=gen).to(torch.int32))
    ends = [0]
    for a, _ in spans:
        ends.append(ends[-1] + a)
    s["indptr"], s["lens"] = _ints(ends), _ints([b for _, b in spans])
    s["longest"] = max(a for a, _ in spans)
    s["q"] = randn(ends[-1], case["heads"], d).to(dt)
    s["out"] = torch.empty(ends[-1], case["heads"], d, dtype=dt, device="cuda")
    s["lse"] = torch.empty(ends[-1], case["heads"], dtype=torch.float32, device="cuda")
    s["mask"] = _trees(gen, [a for a, _ in spans]) if case["op"] == "tree" else None
    s["sm_scale"] = 1.0 / math.sqrt(d)
    return s


# ------------------------------------------------------------------ the plain forms
def _pow2(byte):
    return (byte.to(torch.int32) << 23).view(torch.float32)


def _encode(x):
    """e2m1 codes (the even element in the low half of a byte) and scale bytes of x [..., width]: the byte is that
    of the smallest power of two that is not below a sixth of the block's largest magnitude."""
    g = x.float().unflatten(-1, (-1, BLOCK))
    bits = (g.abs().amax(-1, keepdim=True).clamp_min(1e-10) / 6).view(torch.int32)
    byte = (bits >> 23) + ((bits & 0x7FFFFF) != 0).to(torch.int32)
    v = g * _pow2(254 - byte)
    a = v.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    r = torch.round(a / step) * step
    code = torch.where(r < 2, r * 2, torch.where(r < 4, r + 2, r / 2 + 4)).to(torch.uint8)
    code = (code | (torch.signbit(v).to(torch.uint8) << 3)).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), byte.squeeze(-1).to(torch.uint8)


def _decode(codes, scales, dtype=torch.float32):
    """The values that e2m1 codes [..., width / 2] with scale bytes [..., width / 32] stand for."""
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=dtype, device=codes.device)
    v = torch.stack((table[(codes & 15).int()], table[(codes >> 4).int()]), -1).flatten(-2)
    return (v.unflatten(-1, (-1, BLOCK)) * _pow2(scales).to(dtype).unsqueeze(-1)).flatten(-2)


def _bytes_of(s):
    """The scale bytes [rows, groups] that a program's scales hold."""
    return s if s.dtype == torch.uint8 else s.contiguous().view(torch.uint8)


def _powers(s):
    """A program's scales as the powers of two that they stand for, word by word."""
    return s.view(torch.float8_e8m0fnu) if s.dtype == torch.uint8 else \
        s.unsqueeze(-1).view(torch.uint8).view(torch.float8_e8m0fnu)


def _fma(a, b, c):
    """a * b + c in 32 bits, rounded once (the product is exact in 64 bits)."""
    return (a.double() * b + c).float()


def _silu_mul(x):
    """silu(gate) * up in fp32, with the exponential that the package's activation defines: 2^n times a
    polynomial of degree 7 in what the multiple n of ln 2 leaves."""
    gate, up = x.float().chunk(2, -1)
    t = (-gate).clamp(-87.0, 88.0)
    n = torch.round(t * float.fromhex("0x1.715476p+0"))
    r = _fma(n, -float.fromhex("0x1.62e430p-1"), t.double())
    r = _fma(n, float.fromhex("0x1.05c610p-29"), r.double())
    p = torch.full_like(r, float.fromhex("0x1.a01a02p-13"))
    p = _fma(p, r.double(), float.fromhex("0x1.6c16c2p-10"))
    p = _fma(p, r.double(), float.fromhex("0x1.111112p-7"))
    p = _fma(p, r.double(), float.fromhex("0x1.555556p-5"))
    p = _fma(p, r.double(), float.fromhex("0x1.555556p-3"))
    p = _fma(p, r.double(), 0.5)
    p = _fma(p, r.double(), 1.0)
    p = _fma(p, r.double(), 1.0)
    return gate / (1.0 + torch.ldexp(p, n.to(torch.int32))) * up


def _quant_plain(s):
    x = _silu_mul(s["x"]) if s["silu"] else s["x"]
    codes, byte = _encode(x)
    return [_decode(codes, byte).to(s["x"].dtype), _powers(_scales_like(byte, s["scales"], s["layout"]))]


def _product_plain(s):
    a, b = _decode(s["a"], _bytes_of(s["s_a"])), _decode(s["b"], _bytes_of(s["s_b"]))
    return [torch.matmul(a, b.t()).to(torch.bfloat16)]


def _plan_plain(s):
    page, lens, new, table = s["page"], s["lens"].long(), s["new"].long(), s["table"]
    total = s["slots"].shape[0]
    ends = new.cumsum(0)
    first = -(-lens // page)
    need = -(-(lens + new) // page) - first
    starts = need.cumsum(0) - need
    fresh = s["fresh"]
    j = torch.arange(fresh, device="cuda")
    b = torch.repeat_interleave(need, output_size=fresh)
    table[b, first[b] + j - starts[b]] = s["free"][:fresh]
    b = torch.repeat_interleave(new, output_size=total)
    at = lens[b] + torch.arange(total, device="cuda") - (ends - new)[b]
    slots = table[b, at // page].long() * page + at % page
    indptr = torch.cat((ends.new_zeros(1), ends)).to(torch.int32)
    return [(lens + new).to(torch.int32), indptr, slots.to(torch.int32), at.to(torch.int32), need.sum().to(torch.int32).view(1), table]


def _padded(s):
    """(row of q for each sequence and place, whether it is there, the cached token at its place)."""
    first, last = s["indptr"][:-1].long(), s["indptr"][1:].long()
    i = torch.arange(s["longest"], device="cuda")
    there = i < (last - first).unsqueeze(1)
    row = (first.unsqueeze(1) + i).clamp_max(s["q"].shape[0] - 1)
    place = s["lens"].unsqueeze(1) - (last - first).unsqueeze(1) + i
    return row, there, place


def _hidden(s, row, there, place, tokens):
    """Whether a query [sequence, place] does not see a cached token."""
    token = torch.arange(tokens, device="cuda")
    beyond = (token >= s["lens"].view(-1, 1, 1)) | ~there.unsqueeze(-1)
    if s["op"] == "window":
        p = place.unsqueeze(-1)
        return beyond | (token > p) | ((token <= p - s["window"]) & (token >= s["sinks"]))
    drafted = token - place[:, :1].unsqueeze(-1)  # which drafted token a cached one is
    word = s["mask"][row].long()  # [sequence, place, words]
    at = (drafted.clamp_min(0) // 32).clamp_max(word.shape[2] - 1).expand(-1, word.shape[1], -1)
    named = (torch.gather(word, 2, at) >> (drafted.clamp_min(0) % 32)) & 1
    return beyond | ((drafted >= 0) & (named == 0))


def _attend_plain(s):
    b, h, d = s["table"].shape[0], s["kv_heads"], s["dim"]
    row, there, place = _padded(s)
    k, ks, v, vs = [c[s["table"].clamp_min(0).long()].flatten(1, 2).transpose(1, 2) for c in s["cache"]]
    k, v = _decode(k, ks), _decode(v, vs)
    q = s["q"][row].float().view(b, -1, h, s["heads"] // h, d).permute(0, 2, 1, 3, 4)
    a = torch.matmul(q.reshape(b, h, -1, d), k.transpose(-1, -2).contiguous()) * s["sm_scale"]
    a = a.view(b, h, row.shape[1], s["heads"] // h, -1)
    a = a.masked_fill_(_hidden(s, row, there, place, a.shape[-1])[:, None, :, None], -math.inf)
    most = a.amax(-1, keepdim=True)
    most = torch.where(most == -math.inf, 0.0, most)
    a = a.sub_(most).exp_()
    total = a.sum(-1, keepdim=True)
    lse = (most + total.log()).squeeze(-1)
    b, h, n, g, _ = a.shape
    o = torch.matmul(a.view(b, h, n * g, -1), v).view(b, h, n, g, -1) / torch.where(total == 0, 1.0, total)
    o = o.permute(0, 2, 1, 3, 4).reshape(b * n, h * g, -1)
    lse = lse.permute(0, 2, 1, 3).reshape(b * n, h * g)
    # rows that are there go to their places; the others to one more row that is cut off
    to = torch.where(there, row, s["q"].shape[0]).flatten()
    out = torch.empty(s["q"].shape[0] + 1, *o.shape[1:], dtype=s["out"].dtype, device="cuda")
    sums = torch.empty(s["q"].shape[0] + 1, h * g, dtype=torch.float32, device="cuda")
    out[to], sums[to] = o.to(out.dtype), lse
    return [out[:-1], sums[:-1]]


def _run_own(s):
    import fp8_group_quant_amd as fq
    if s["op"] == "quant":
        (fq.fp8q_silu_mul_mxfp4_quant if s["silu"] else fq.fp8q_mxfp4_quant)(s["x"], s["q"], s["s"])
        fq.fp8q_mxfp4_dequant(s["q"], s["s"], s["back"])
        return [s["back"], _powers(s["s"])]
    if s["op"] == "product":
        fq.fp8q_gemm_mxfp4(s["a"], s["s_a"], s["b"], s["s_b"], s["y"])
        return [s["y"]]
    if s["op"] == "plan":
        fq.fp8q_kv4_plan(s["lens"], s["new"], s["free"], s["table"], s["pages"], s["page"], s["lens_out"], s["indptr"],
                         s["slots"], s["taken"], positions=s["positions"])
        return [s["lens_out"], s["indptr"], s["slots"], s["positions"], s["taken"], s["table"]]
    cache = fq.Kv4Cache(*s["cache"])
    if s["op"] == "window":
        fq.fp8q_kv4_window_attention(s["q"], cache, s["table"], s["lens"], s["out"], s["sm_scale"], s["window"], s["sinks"],
                                     q_indptr=None if s["longest"] == 1 else s["indptr"], lse=s["lse"])
    else:
        fq.fp8q_kv4_tree_attention(s["q"], cache, s["table"], s["lens"], s["out"], s["sm_scale"], s["mask"], s["indptr"],
                                   lse=s["lse"])
    return [s["out"], s["lse"]]


def run(state):
    if own:
        return _run_own(state)
    return {"quant": _quant_plain, "product": _product_plain, "plan": _plan_plain, "window": _attend_plain,
            "tree": _attend_plain}[state["op"]](state)


# ------------------------------------------------------------------ the definitions in 64 bits
def _decode64(codes, scales):
    """sign * magnitude * 2^(byte - 127), each part taken from its bits."""
    nib = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).to(torch.int64)
    ex, man = (nib >> 1) & 3, (nib & 1).double()
    mag = torch.where(ex == 0, 0.5 * man, torch.ldexp(1 + 0.5 * man, ex - 1))
    mag = torch.where(nib >= 8, -mag, mag).unflatten(-1, (-1, BLOCK))
    return torch.ldexp(mag, scales.to(torch.int64).unsqueeze(-1) - 127).flatten(-2)


def _nearest64(x):
    """(x [..., width] rounded to the e2m1 values times its blocks' scales, those scales), in 64 bits."""
    g = x.unflatten(-1, (-1, BLOCK))
    most = g.abs().amax(-1, keepdim=True).clamp_min(1e-10)
    scale = torch.exp2(torch.ceil(torch.log2(most / 6)))
    scale = torch.where(scale * 6 < most, scale * 2, scale)
    scale = torch.where(scale * 3 >= most, scale / 2, scale)
    grid = torch.tensor(E2M1, dtype=torch.float64, device=x.device)
    v = (g / scale).abs()
    up = torch.bucketize(v, grid).clamp_max(7)
    down = (up - 1).clamp_min(0)
    to_up, to_down = grid[up] - v, v - grid[down]
    pick = torch.where((to_up < to_down) | ((to_up == to_down) & (up % 2 == 0)), up, down)
    return (torch.where(g < 0, -grid[pick], grid[pick]) * scale).flatten(-2), scale.squeeze(-1)


def exact(case, seed):
    if case["op"] == "plan":
        return None  # whole numbers
    s = prepare(case, seed)
    if case["op"] == "quant":
        x = s["x"].double()
        if case["silu"]:
            gate, up = x.chunk(2, -1)
            x = gate * torch.sigmoid(gate) * up
        value, scale = _nearest64(x)
        if case["scales"] == "words":
            scale = scale.unflatten(-1, (-1, 4))
        return [value, scale]
    if case["op"] == "product":
        def words(c):
            w = c if c.dtype == torch.uint8 else torch.stack([(c >> (8 * i)) & 255 for i in range(4)], -1).flatten(-2)
            return w
        return [_decode64(s["a"], words(s["s_a"])) @ _decode64(s["b"], words(s["s_b"])).t().contiguous()]
    d, group, page = case["dim"], case["heads"] // case["kv_heads"], case["page"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device="cuda")
    at = 0
    for b, (n, length) in enumerate(_spans(case)):  # one sequence and cached head after the other
        pages = s["table"][b, :-(-length // page)].long()
        k, ks, v, vs = [c[pages].flatten(0, 1)[:length] for c in s["cache"]]
        k, v = _decode64(k, ks), _decode64(v, vs)
        sees = torch.ones(n, length, dtype=torch.bool, device="cuda")
        if case["op"] == "window":
            back = torch.arange(length - n, length, device="cuda").unsqueeze(1) - torch.arange(length, device="cuda")
            sees = (back >= 0) & ((back < case["window"]) | (torch.arange(length, device="cuda") < case["sinks"]))
        else:
            bits = torch.stack([(s["mask"][at:at + n] >> i) & 1 for i in range(32)], -1).flatten(1)
            sees[:, length - n:] = bits[:, :n] == 1
        sees = sees.repeat_interleave(group, 0)
        for h in range(case["kv_heads"]):
            q = s["q"][at:at + n, h * group:(h + 1) * group].double().reshape(n * group, d)
            a = (q @ k[:, h].t() / math.sqrt(d)).masked_fill(~sees, -math.inf)
            sums = torch.logsumexp(a, -1)
            o = torch.exp(a - sums.unsqueeze(1)) @ v[:, h]
            out[at:at + n, h * group:(h + 1) * group] = o.view(n, group, d)
            lse[at:at + n, h * group:(h + 1) * group] = sums.view(n, group)
        at += n
    return [out, lse]
