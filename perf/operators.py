"""The serving operators around the block-scaled FP8 GEMMs, as measured cases.

Four operators of one decoder layer that keeps its key/value cache in 4 bits:

  norm    h = x (+ residual); y = h / sqrt(mean(h^2) + eps) * weight; y quantized to e4m3 in groups
          of a row, with fp32 or power-of-two (UE8M0) scales: the input of the next FP8 GEMM.
  write   keys and values quantized to e2m1 codes with one UE8M0 scale per 32 elements, at the slots
          of a paged cache, and the same slots read back.
  read    slots of the cache read back as rows of the model's type.
  attend  softmax(scale * q k^T) v over the cached keys and values, grouped query heads, ragged
          query and cache lengths, with the logarithm of each row's softmax sum.

`own` False computes them with elementary torch operations in fp32, `own` True through the
package's entry points.
"""
import math

import torch

own = False

EPS = 1e-6
BLOCK = 32  # cached elements that share one scale
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ------------------------------------------------------------------ cases
def _norm(name, rows, width, dtype="bf16", group=128, scales="ue8m0", layout="col", residual=True):
    return {"name": name, "op": "norm", "rows": rows, "width": width, "dtype": dtype, "group": group,
            "scales": scales, "layout": layout, "residual": residual}


def _write(name, tokens, heads, dim, page, pages, dtype="bf16"):
    return {"name": name, "op": "write", "tokens": tokens, "heads": heads, "dim": dim, "page": page,
            "pages": pages, "dtype": dtype}


def _read(name, tokens, heads, dim, page, pages, dtype="bf16"):
    return {"name": name, "op": "read", "tokens": tokens, "heads": heads, "dim": dim, "page": page,
            "pages": pages, "dtype": dtype}


def _attend(name, seqs, q_len, kv_len, heads, kv_heads, dim, page, q_ragged=0, kv_ragged=0, dtype="bf16"):
    """q_ragged, kv_ragged: by how many percent the lengths of the sequences fall below the longest."""
    return {"name": name, "op": "attend", "seqs": seqs, "q_len": q_len, "kv_len": kv_len, "heads": heads,
            "kv_heads": kv_heads, "dim": dim, "page": page, "q_ragged": q_ragged, "kv_ragged": kv_ragged,
            "dtype": dtype}


def listed():
    return [
        # one token of one user: the launch and its latency are all there is
        _norm("norm one token", 1, 7168),
        # the dense workload's rows, before its GEMM
        _norm("norm dense rows", 4096, 7168),
        # per-head-sized rows of an odd number of tokens, fp16, fp32 row-major scales, no residual
        _norm("norm narrow odd rows", 30011, 576, dtype="f16", group=64, scales="f32", layout="row", residual=False),
        # one decode step of 32 users writes one token each
        _write("write decode step", 32, 8, 128, 16, 4096),
        # a prompt of 16k tokens goes into the cache
        _write("write prompt", 16384, 8, 128, 64, 1024),
        # a prefix of 5003 tokens is taken out of the cache again, fp16, narrow heads
        _read("read prefix", 5003, 4, 64, 16, 1024, dtype="f16"),
        # the whole context of several users is taken out, for a kernel that reads plain rows
        _read("read contexts", 131072, 8, 128, 64, 2304),
        # one user, a short context: latency
        _attend("attend one user", 1, 1, 1000, 32, 8, 128, 16),
        # a decode step of a full batch, ragged contexts
        _attend("attend decode batch", 64, 1, 8192, 64, 8, 128, 64, kv_ragged=60),
        # one user with a very long context: the cache axis is all there is to split
        _attend("attend long context", 1, 1, 262144, 32, 8, 128, 64),
        # several tokens of each user are verified at once, fp16, narrow heads, small pages
        _attend("attend drafted tokens", 17, 5, 3001, 32, 8, 64, 16, q_ragged=80, kv_ragged=90, dtype="f16"),
        # a chunk of a prompt attends to what came before it and to itself
        _attend("attend prompt chunk", 2, 2048, 8192, 32, 8, 128, 64, q_ragged=30, kv_ragged=40),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm", "write", "read", "attend", "attend"))
    if op == "norm":
        group = rng.choice((32, 64, 128))
        width = group * max(1, _log(rng, 256, 8192) // group)
        rows = _log(rng, 1, min(32768, 4096 * 7168 // (2 * width)))
        c = _norm("", rows, width, rng.choice(("bf16", "f16", "f32")), group, rng.choice(("ue8m0", "f32")),
                  rng.choice(("row", "col")), rng.random() < 0.7)
    elif op in ("write", "read"):
        heads, dim, page = rng.choice((1, 2, 4, 8)), rng.choice((64, 128, 256)), rng.choice((1, 16, 32, 64))
        tokens = _log(rng, 1, min(131072, (1 << 26 if op == "read" else 1 << 23) // (heads * dim)))
        pages = -(-tokens // page) + rng.randrange(1, 65)
        c = (_write if op == "write" else _read)("", tokens, heads, dim, page, pages, rng.choice(("bf16", "f16", "f32")))
    else:
        dim, kv_heads, group = rng.choice((64, 128, 256)), rng.choice((1, 2, 4, 8)), rng.choice((1, 4, 5, 8))
        q_len = 1 if rng.random() < 0.5 else _log(rng, 2, 1024)
        seqs = _log(rng, 1, 64 if q_len == 1 else max(1, min(32, 2048 // q_len)))
        most = min(65536, 2 ** 28 // (seqs * kv_heads * dim), 2 ** 34 // (seqs * kv_heads * group * dim * q_len))
        kv_len = q_len + _log(rng, 16, max(16, most))
        c = _attend("", seqs, q_len, kv_len, kv_heads * group, kv_heads, dim, rng.choice((16, 32, 64)),
                    rng.choice((0, 50)), rng.choice((0, 30, 90)), rng.choice(("bf16", "f16")))
    del c["name"]
    return c


def _lengths(count, longest, ragged):
    """Lengths of `count` sequences, the first of them the longest."""
    return [max(1, longest - longest * ragged * (b * 619 % 997) // 99700) for b in range(count)]


def _spans(case):
    """(query length, cache length) of each sequence; no sequence has more queries than cached tokens."""
    q = _lengths(case["seqs"], case["q_len"], case["q_ragged"])
    kv = _lengths(case["seqs"], case["kv_len"], case["kv_ragged"])
    return [(min(a, b), b) for a, b in zip(q, kv)]


def work(case):
    size = torch.empty(0, dtype=TYPES[case["dtype"]]).element_size()
    if case["op"] == "norm":
        n, m, k = case["rows"] * case["width"], case["rows"], case["width"]
        scales = m * (k // case["group"]) * (4 if case["scales"] == "f32" else 1)
        return {"bytes": n * size * (3 if case["residual"] else 1) + k * size + n + scales, "flops": 6 * n}
    if case["op"] in ("write", "read"):
        n = 2 * case["tokens"] * case["heads"] * case["dim"]
        held = n // 2 + n // BLOCK
        passes = 2 if case["op"] == "write" else 1
        return {"bytes": passes * (n * size + held + 4 * case["tokens"]), "flops": 2 * passes * n}
    d, spans = case["dim"], _spans(case)
    pairs = sum(a * b - a * (a - 1) // 2 for a, b in spans)
    tokens = sum(a for a, _ in spans)
    cached = sum(b for _, b in spans) * case["kv_heads"] * 2 * (d // 2 + d // BLOCK)
    return {"bytes": cached + tokens * case["heads"] * (2 * d * size + 4), "flops": 4 * pairs * case["heads"] * d}


# ------------------------------------------------------------------ what a program has in hand
def _cache_of(gen, pages, page, heads, dim):
    """(codes, scales) of one cached tensor, viewed as [page, token, head, ...], each head's tokens adjacent."""
    codes = torch.empty(pages, heads, page, dim // 2, dtype=torch.uint8, device="cuda")
    scales = torch.empty(pages, heads, page, dim // BLOCK, dtype=torch.uint8, device="cuda")
    channel = torch.exp(0.5 * torch.randn(heads, 1, dim, device="cuda", generator=gen))
    step = max(1, (1 << 26) // (heads * page * dim))
    for p in range(0, pages, step):
        n = min(step, pages - p)
        x = torch.randn(n, heads, page, dim, device="cuda", generator=gen) * channel
        codes[p:p + n], scales[p:p + n] = _encode(x)
    return codes.transpose(1, 2), scales.transpose(1, 2)


def _slots_of(gen, case):
    """Distinct slots of a sequence's tokens: its pages lie anywhere in the cache."""
    page, n = case["page"], case["tokens"]
    order = torch.randperm(case["pages"], device="cuda", generator=gen)
    t = torch.arange(n, device="cuda")
    return (order[t // page] * page + t % page).to(torch.int32)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = TYPES[case["dtype"]]

    def randn(*shape):
        return torch.randn(*shape, device="cuda", generator=gen)

    s = dict(case)
    if case["op"] == "norm":
        m, k, g = case["rows"], case["width"], case["group"]
        s["x"] = randn(m, k).to(dt)
        s["res"] = (4 * randn(m, k)).to(dt) if case["residual"] else None
        s["w"] = (1 + 0.1 * randn(k)).to(dt)
        s["q"] = torch.empty(m, k, dtype=torch.uint8, device="cuda")
        held = torch.float32 if case["scales"] == "f32" else torch.uint8
        s["s"] = torch.empty(m, k // g, dtype=held, device="cuda") if case["layout"] == "row" else \
            torch.empty(k // g, m, dtype=held, device="cuda").t()
        s["res_out"] = torch.empty(m, k, dtype=dt, device="cuda") if case["residual"] else None
        return s
    if case["op"] in ("write", "read"):
        t, h, d = case["tokens"], case["heads"], case["dim"]
        s["cache"] = _cache_of(gen, case["pages"], case["page"], h, d) + \
            _cache_of(gen, case["pages"], case["page"], h, d)
        s["slots"] = _slots_of(gen, case)
        if case["op"] == "write":  # views of one projection's output, as a program has them
            kv = (randn(t, 2, h, d) * torch.exp(0.5 * randn(1, 2, h, d))).to(dt)
            s["k"], s["v"] = kv[:, 0], kv[:, 1]
        s["k_out"] = torch.empty(t, h, d, dtype=dt, device="cuda")
        s["v_out"] = torch.empty(t, h, d, dtype=dt, device="cuda")
        return s
    spans, page, h, d = _spans(case), case["page"], case["kv_heads"], case["dim"]
    counts = [-(-b // page) for _, b in spans]
    pages = sum(counts) + 3
    s["cache"] = _cache_of(gen, pages, page, h, d) + _cache_of(gen, pages, page, h, d)
    order = torch.randperm(pages, device="cuda", generator=gen).to(torch.int32)
    table = torch.zeros(len(spans), max(counts), dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(counts):
        table[b, :n] = order[at:at + n]
        at += n
    s["table"] = table
    ends = [0]
    for a, _ in spans:
        ends.append(ends[-1] + a)
    s["indptr"] = torch.tensor(ends, dtype=torch.int32, device="cuda")
    s["lens"] = torch.tensor([b for _, b in spans], dtype=torch.int32, device="cuda")
    s["longest"] = max(a for a, _ in spans)
    s["q"] = randn(ends[-1], case["heads"], d).to(dt)
    s["out"] = torch.empty(ends[-1], case["heads"], d, dtype=dt, device="cuda")
    s["lse"] = torch.empty(ends[-1], case["heads"], dtype=torch.float32, device="cuda")
    s["sm_scale"] = 1.0 / math.sqrt(d)
    return s


# ------------------------------------------------------------------ the plain forms
def _pow2_byte(r):
    """Biased exponent of the smallest power of two that is not below r (fp32, normal)."""
    bits = r.view(torch.int32)
    return (bits >> 23) + ((bits & 0x7FFFFF) != 0).to(torch.int32)


def _pow2(byte):
    return (byte.to(torch.int32) << 23).view(torch.float32)


def _encode(x):
    """e2m1 codes (the even element in the low half of a byte) and scale bytes of x [..., dim]."""
    g = x.float().unflatten(-1, (-1, BLOCK))
    byte = _pow2_byte(g.abs().amax(-1, keepdim=True).clamp_min(1e-10) / 6)
    v = g * _pow2(254 - byte)
    a = v.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    r = torch.round(a / step) * step
    code = torch.where(r < 2, r * 2, torch.where(r < 4, r + 2, r / 2 + 4)).to(torch.uint8)
    code = (code | (torch.signbit(v).to(torch.uint8) << 3)).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), byte.squeeze(-1).to(torch.uint8)


def _decode(codes, scales, dtype=torch.float32):
    """The values that e2m1 codes [..., dim / 2] with scale bytes [..., dim / 32] stand for."""
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=dtype, device=codes.device)
    v = torch.stack((table[(codes & 15).int()], table[(codes >> 4).int()]), -1).flatten(-2)
    return (v.unflatten(-1, (-1, BLOCK)) * _pow2(scales).to(dtype).unsqueeze(-1)).flatten(-2)


def _at(cache, slots, page):
    return [c[slots // page, slots % page] for c in cache]


def _norm_plain(s):
    h = s["x"].float()
    if s["residual"]:
        h = h + s["res"].float()
    y = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS) * s["w"].float()
    g = y.unflatten(-1, (-1, s["group"]))
    r = g.abs().amax(-1, keepdim=True).clamp_min(1e-10) / 448
    if s["scales"] == "f32":
        scale, inv = r.squeeze(-1), 1 / r
    else:
        byte = _pow2_byte(r)
        scale, inv = byte.squeeze(-1).to(torch.uint8).view(torch.float8_e8m0fnu), _pow2(254 - byte)
    q = (g * inv).clamp(-448, 448).flatten(-2).to(torch.float8_e4m3fn)
    return [q, scale] + ([h.to(s["x"].dtype)] if s["residual"] else [])


def _write_plain(s):
    slots, page = s["slots"], s["page"]
    for x, (codes, scales) in ((s["k"], s["cache"][:2]), (s["v"], s["cache"][2:])):
        codes[slots // page, slots % page], scales[slots // page, slots % page] = _encode(x)
    return _read_plain(s)


def _read_plain(s):
    k, ks, v, vs = _at(s["cache"], s["slots"], s["page"])
    dt = s["k_out"].dtype
    return [_decode(k, ks).to(dt), _decode(v, vs).to(dt)]


def _padded(s):
    """(row of q for each sequence and place, whether it is there, the last cached token that it sees)."""
    first, last = s["indptr"][:-1].long(), s["indptr"][1:].long()
    i = torch.arange(s["longest"], device="cuda")
    there = i < (last - first).unsqueeze(1)
    row = (first.unsqueeze(1) + i).clamp_max(s["q"].shape[0] - 1)
    sees = s["lens"].unsqueeze(1) - (last - first).unsqueeze(1) + i
    return row, there, sees


def _scores(s, dtype):
    """Scaled scores [seq, kv head, query, head in group, token] with -inf where none counts, and the values."""
    b, h, d = s["table"].shape[0], s["kv_heads"], s["dim"]
    row, there, sees = _padded(s)
    k, ks, v, vs = [c[s["table"].long()].flatten(1, 2).transpose(1, 2) for c in s["cache"]]
    k, v = _decode(k, ks, dtype), _decode(v, vs, dtype)
    q = s["q"][row].to(dtype).view(b, -1, h, s["heads"] // h, d).permute(0, 2, 1, 3, 4)
    a = torch.matmul(q.reshape(b, h, -1, d), k.transpose(-1, -2).contiguous()) * s["sm_scale"]
    a = a.view(b, h, row.shape[1], s["heads"] // h, -1)
    token = torch.arange(a.shape[-1], device="cuda")
    hidden = (token > sees.unsqueeze(-1)) | (token >= s["lens"].view(-1, 1, 1)) | ~there.unsqueeze(-1)
    return a.masked_fill_(hidden[:, None, :, None], -math.inf), v, row, there


def _attend_plain(s, dtype=torch.float32):
    a, v, row, there = _scores(s, dtype)
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
    out[to], sums[to] = o.to(out.dtype), lse.float()
    return [out[:-1], sums[:-1]]


def _run_own(s):
    import fp8_group_quant_amd as fq
    if s["op"] == "norm":
        fq.fp8q_rms_norm_group_quant(s["x"], s["w"], s["q"], s["s"], s["group"], EPS, residual=s["res"],
                                     residual_out=s["res_out"])
        scale = s["s"] if s["scales"] == "f32" else s["s"].view(torch.float8_e8m0fnu)
        return [s["q"].view(torch.float8_e4m3fn), scale] + ([s["res_out"]] if s["residual"] else [])
    cache = fq.Kv4Cache(*s["cache"])
    if s["op"] == "attend":
        fq.fp8q_kv4_attention(s["q"], cache, s["table"], s["lens"], s["out"], s["sm_scale"],
                              q_indptr=None if s["longest"] == 1 else s["indptr"], lse=s["lse"])
        return [s["out"], s["lse"]]
    if s["op"] == "write":
        fq.fp8q_kv4_write(s["k"], s["v"], s["slots"], cache)
    fq.fp8q_kv4_read(s["k_out"], s["v_out"], s["slots"], cache)
    return [s["k_out"], s["v_out"]]


def run(state):
    if own:
        return _run_own(state)
    return {"norm": _norm_plain, "write": _write_plain, "read": _read_plain, "attend": _attend_plain}[state["op"]](state)


# ------------------------------------------------------------------ the definitions in 64 bits
def _decode64(codes, scales):
    """sign * magnitude * 2^(byte - 127), each part taken from its bits."""
    nib = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).to(torch.int64)
    ex, man = (nib >> 1) & 3, (nib & 1).double()
    mag = torch.where(ex == 0, 0.5 * man, torch.ldexp(1 + 0.5 * man, ex - 1))
    mag = torch.where(nib >= 8, -mag, mag).unflatten(-1, (-1, BLOCK))
    return torch.ldexp(mag, scales.to(torch.int64).unsqueeze(-1) - 127).flatten(-2)


def _nearest64(x):
    """x [..., dim] rounded to the e2m1 values times its blocks' scales, in 64 bits."""
    g = x.double().unflatten(-1, (-1, BLOCK))
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
    return (torch.where(g < 0, -grid[pick], grid[pick]) * scale).flatten(-2)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        h = s["x"].double() + (s["res"].double() if case["residual"] else 0.0)
        y = h / torch.sqrt(h.square().mean(-1, keepdim=True) + EPS) * s["w"].double()
        g = y.unflatten(-1, (-1, case["group"]))
        r = g.abs().amax(-1, keepdim=True).clamp_min(1e-10) / 448
        if case["scales"] == "ue8m0":
            r = torch.exp2(torch.ceil(torch.log2(r)))
        q = (g / r).clamp(-448, 448).flatten(-2).to(torch.float8_e4m3fn).double()
        return [q, r.squeeze(-1)] + ([h] if case["residual"] else [])
    if case["op"] == "write":
        return [_nearest64(s["k"]), _nearest64(s["v"])]
    if case["op"] == "read":
        k, ks, v, vs = _at(s["cache"], s["slots"].long(), case["page"])
        return [_decode64(k, ks), _decode64(v, vs)]
    d, group, page = case["dim"], case["heads"] // case["kv_heads"], case["page"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device="cuda")
    at = 0
    for b, (n, length) in enumerate(_spans(case)):  # one sequence and cached head after the other
        pages = s["table"][b, :-(-length // page)].long()
        k, ks, v, vs = [c[pages].flatten(0, 1)[:length] for c in s["cache"]]
        k, v = _decode64(k, ks), _decode64(v, vs)
        rows = torch.arange(n, device="cuda").repeat_interleave(group)
        late = torch.arange(length, device="cuda") > (length - n + rows).unsqueeze(1)
        for h in range(case["kv_heads"]):
            q = s["q"][at:at + n, h * group:(h + 1) * group].double().reshape(n * group, d)
            a = (q @ k[:, h].t() / math.sqrt(d)).masked_fill(late, -math.inf)
            sums = torch.logsumexp(a, -1)
            o = torch.exp(a - sums.unsqueeze(1)) @ v[:, h]
            out[at:at + n, h * group:(h + 1) * group] = o.view(n, group, d)
            lse[at:at + n, h * group:(h + 1) * group] = sums.view(n, group)
        at += n
    return [out, lse]
