"""Plain 64-bit attention over a paged cache with any mask (test helper, not product code), laid out as
serving_oracle.attention so that its error bounds apply. CPU tensors throughout."""
import math

import torch


def window_sees(n, length, window, sinks):
    """[n, length]: whether the i-th of a sequence's n queries sees cached token j."""
    place = torch.arange(length - n, length).unsqueeze(1)
    j = torch.arange(length)
    return (j <= place) & ((j > place - window) | (j < sinks))


def tree_sees(mask, n, length):
    """[n, length] from the rows mask [n, words] of drafted tokens held at the last n of `length` places."""
    sees = torch.zeros(n, length, dtype=torch.bool)
    for i in range(n):
        for j in range(length):
            d = j - (length - n)
            if d < 0:
                sees[i, j] = True
            elif d < 32 * mask.shape[1]:
                sees[i, j] = bool((int(mask[i, d // 32]) >> (d % 32)) & 1)
    return sees


def attention(q, k, v, table, kv_lens, q_lens, page, pages, sm_scale, sees):
    """q [T, Hq, D]; k, v float64 [pages, page, Hkv, D]; sees(b, n, length, first row) gives [n, length]. Returns float64
    (out, lse, mass, slack) as serving_oracle.attention does."""
    T, Hq, D = q.shape
    Hkv = k.shape[2]
    G = Hq // Hkv
    out = torch.zeros(T, Hq, D, dtype=torch.float64)
    mass = torch.zeros(2, T, Hq, D, dtype=torch.float64)
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64)
    slack = torch.zeros(T, Hq, dtype=torch.float64)
    at = 0
    for b, (n, length) in enumerate(zip(q_lens, kv_lens)):
        if n == 0:
            continue
        toks = torch.arange(length)
        pg = table[b, toks // page].long() if length else toks
        there = (pg >= 0) & (pg < pages)
        sb = sees(b, n, length, at)[:, there]
        kb, vb = k[pg[there], toks[there] % page], v[pg[there], toks[there] % page]
        rows = sb.any(1)
        for h in range(Hq):
            kk, vv, qq = kb[:, h // G], vb[:, h // G], q[at:at + n, h].double()
            a = (sm_scale * (qq @ kk.t())).masked_fill(~sb, -math.inf)
            s = torch.logsumexp(a, 1)
            p = torch.where(rows.unsqueeze(1), torch.exp(a - s.unsqueeze(1)), 0.0)
            p = torch.where(sb, p, 0.0)
            out[at:at + n, h] = p @ vv
            lse[at:at + n, h] = torch.where(rows, s, -math.inf)
            mass[0, at:at + n, h] = p @ vv.abs()
            mass[1, at:at + n, h] = sb.double() @ vv.abs()
            big = torch.where(sb, qq.abs() @ kk.abs().t(), 0.0)
            if big.shape[1]:
                slack[at:at + n, h] = abs(sm_scale) * big.amax(1)
        at += n
    return out, lse, mass, slack
