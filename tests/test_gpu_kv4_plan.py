"""The page plan of a serving step against a plain loop, and the plan, the cache and its attention together."""
import math

import pytest
import torch

import masked_oracle as masked
import serving_oracle as ref

pytestmark = pytest.mark.gpu


def fq():
    import fp8_group_quant_amd
    return fp8_group_quant_amd


def gen(seed):
    return torch.Generator().manual_seed(seed)


def plain_plan(kv_lens, q_lens, free, table, pages, page, tokens):
    """(new lengths, indptr, slots, positions, pages taken, table) by the definition."""
    table = table.clone()
    most = table.shape[1] * page
    new, ends, slots, places, taken = [], [0], [-1] * tokens, [-1] * tokens, 0
    for b, (l, n) in enumerate(zip(kv_lens, q_lens)):
        l = min(max(l, 0), most)
        n = max(n, 0)
        first = ends[-1]
        ends.append(min(first + n, tokens))
        n = ends[-1] - first
        held = min(n, most - l)
        new.append(l + held)
        for j in range(-(-l // page), -(-(l + held) // page)):
            number = free[taken] if taken < len(free) else -1
            table[b, j] = number if 0 <= number < pages else -1
            taken += 1
        for i in range(n):
            places[first + i] = l + i
            if l + i < most:
                number = int(table[b, (l + i) // page])
                if 0 <= number < pages:
                    slots[first + i] = number * page + (l + i) % page
    return new, ends, slots, places, taken, table


def check(kv_lens, q_lens, page, width, tokens=None, spare=3, short=0, seed=0, junk=False):
    f = fq()
    most = width * page
    counts = [-(-min(max(l, 0), most) // page) for l in kv_lens]
    need = sum(max(n, 0) for n in q_lens) // page + 2 * len(q_lens) + spare
    pages = sum(counts) + need
    order = torch.randperm(pages, generator=gen(seed)).to(torch.int32)
    table = torch.full((len(kv_lens), width + 2), -5, dtype=torch.int32)
    at = 0
    for b, n in enumerate(counts):
        table[b, :n] = order[at:at + n]
        at += n
    free = order[at:at + need - short] if not short or need > short else order[:0]
    if junk and free.numel() > 3:
        free = free.clone()
        free[1], free[2] = -4, pages
    tokens = sum(max(n, 0) for n in q_lens) if tokens is None else tokens
    want = plain_plan(kv_lens, q_lens, free.tolist(), table[:, :width], pages, page, tokens)
    td = table.cuda()
    i32 = dict(dtype=torch.int32, device="cuda")
    B = len(kv_lens)
    new, ends, slots, places, taken = (torch.full((n + 1,), 77, **i32) for n in (B, B + 1, tokens, tokens, 1))
    f.fp8q_kv4_plan(torch.tensor(kv_lens, **i32), torch.tensor(q_lens, **i32), free.cuda(), td[:, :width], pages, page, new[:B],
                    ends[:B + 1], slots[:tokens], taken[:1], positions=places[:tokens])
    torch.cuda.synchronize()
    assert new[:B].tolist() == want[0] and ends[:B + 1].tolist() == want[1]
    assert slots[:tokens].tolist() == want[2] and places[:tokens].tolist() == want[3]
    assert int(taken[0]) == want[4]
    assert torch.equal(td[:, :width].cpu(), want[5]) and bool((td[:, width:] == -5).all())
    for t in (new, ends, slots, places, taken):
        assert int(t[-1]) == 77


@pytest.mark.parametrize("page", [1, 4, 16, 64])
def test_plan(page):
    check([0, 1, 15, 16, 17, 63, 64, 65, 0, 200], [1, 1, 1, 1, 0, 3, 70, 16, 0, 40], page, 300 // page + 5)


@pytest.mark.parametrize("B,longest,held", [(1, 1, 0), (1, 5000, 77), (64, 1, 900), (255, 30, 400), (257, 9, 100), (1000, 4, 50), (4096, 3, 40)])
def test_plan_sizes(B, longest, held):
    g = gen(B)
    q = torch.randint(0, longest + 1, (B,), generator=g).tolist()
    kv = torch.randint(0, held + 1, (B,), generator=g).tolist()
    check(kv, q, 16, (longest + held) // 16 + 2)


def test_plan_edges():
    check([5, 9], [0, 0], 16, 4)                                  # no new tokens
    check([], [], 16, 4, tokens=3)                                # no sequences: every slot is -1
    check([30, 0, 7], [10, 20, 5], 16, 4, tokens=60)              # room past the last token
    check([30, 0, 7], [10, 20, 5], 16, 4, tokens=17)              # fewer places than tokens
    check([30, 0, 7], [10, 20, 5], 16, 4, tokens=0)
    check([60, 64, 70, -3], [10, 3, 5, 4], 16, 4)                 # past the table's row, lengths out of range
    check([30, 0, 7], [-4, 20, 5], 16, 4)                         # a negative count
    check([3, 0, 7], [40, 20, 50], 4, 40, short=30)               # too few free pages
    check([3, 0, 7], [40, 20, 50], 4, 40, short=10 ** 6)          # none
    check([3, 0, 7], [40, 20, 50], 4, 40, junk=True)              # pages that the cache does not have
    check([3, 0], [4, 2], 16, 0)                                  # a table without columns


def test_counts_whose_sum_passes_32_bits():
    check_big = [2 ** 31 - 1] * 5
    f = fq()
    i32 = dict(dtype=torch.int32, device="cuda")
    B, width, page, tokens = 5, 40, 64, 2000
    table = torch.full((B, width), -1, **i32)
    free = torch.arange(100, **i32)
    new, ends, slots, taken = torch.empty(B, **i32), torch.empty(B + 1, **i32), torch.empty(tokens, **i32), torch.empty(1, **i32)
    f.fp8q_kv4_plan(torch.zeros(B, **i32), torch.tensor(check_big, **i32), free, table, 100, page, new, ends, slots, taken)
    assert ends.tolist() == [0] + [tokens] * B and new.tolist() == [tokens, 0, 0, 0, 0]
    assert slots.tolist() == list(range(tokens)) and int(taken) == 32


def test_steps_of_two_requests():
    """Prompts, drafted trees and decode steps of two requests, with tables and slots from the plan alone: what attention gives
    is that of the keys and values as they were written. The accepted branch's rows are read and written to the
    places after the prompt."""
    f = fq()
    H, G, D, page, width = 2, 4, 64, 16, 20
    c = f.alloc_kv4_cache(40, page, H, D)
    g = gen(1)
    i32 = dict(dtype=torch.int32, device="cuda")
    table = torch.full((2, width), -1, **i32)
    free = torch.randperm(40, generator=g).to(torch.int32).cuda()
    lens = torch.zeros(2, **i32)
    held = [torch.zeros(0, 2, H, D), torch.zeros(0, 2, H, D)]  # keys and values in order, by request

    def step(new, sees, attend):
        nonlocal lens, free
        T = sum(new)
        plan = f.kv4_plan(c, lens, torch.tensor(new, **i32), free, table, T)
        kv = torch.randn(T, 2, H, D, generator=g).to(torch.bfloat16)
        q = torch.randn(T, G * H, D, generator=g).to(torch.bfloat16)
        f.fp8q_kv4_write(kv[:, 0].cuda(), kv[:, 1].cuda(), plan.slots, c)
        out = attend(q.cuda(), plan)
        at = 0
        for b, n in enumerate(new):
            held[b] = torch.cat([held[b], kv[at:at + n].float()])
            k64, v64 = (ref.dequantize(*ref.quantize(held[b][:, i])) for i in (0, 1))
            m = held[b].shape[0]
            o, l, mass, slack = masked.attention(q[at:at + n], k64.unsqueeze(0), v64.unsqueeze(0), torch.zeros(1, 1, dtype=torch.int32),
                                                 [m], [n], m, 1, D ** -0.5, lambda *_: sees(b, n, m))
            ob, _ = ref.attention_bounds(o, l, mass, slack, D, m, torch.bfloat16)
            assert bool(((out[at:at + n].cpu().double() - o).abs() <= ob).all())
            at += n
        free = free[int(plan.pages_taken):]
        lens = plan.kv_lens
        return plan

    window = lambda b, n, m: masked.window_sees(n, m, 24, 2)  # noqa: E731
    run_window = lambda q, p: f.kv4_window_attention(q, c, table, p.kv_lens, D ** -0.5, 24, 2, p.q_indptr)  # noqa: E731
    step([37, 90], window, run_window)
    step([1, 1], window, run_window)
    # trees of 5 and 3 drafted tokens: 0 <- 1 <- 3, 0 <- 2 <- 4; 0 <- 1, 0 <- 2
    mask = torch.tensor([[0b1], [0b11], [0b101], [0b1011], [0b10101], [0b1], [0b11], [0b101]], dtype=torch.int32)
    plan = step([5, 3], lambda b, n, m: masked.tree_sees(mask[5 * b:5 * b + n], n, m),
                lambda q, p: f.kv4_tree_attention(q, c, table, p.kv_lens, D ** -0.5, mask.cuda(), p.q_indptr))
    # tokens 0, 2, 4 of the first request and 0, 2 of the second are accepted
    taken = torch.tensor([2, 4, 7]).cuda()
    into = torch.tensor([1, 2, 6]).cuda()
    k, v = f.kv4_read(c, plan.slots[taken])
    f.fp8q_kv4_write(k, v, plan.slots[into], c)
    held[0] = torch.cat([held[0][:-5], held[0][-5:][[0, 2, 4]]])
    held[1] = torch.cat([held[1][:-3], held[1][-3:][[0, 2]]])
    lens = lens - torch.tensor([2, 1], **i32)
    step([1, 1], window, run_window)
    causal = lambda b, n, m: masked.window_sees(n, m, m, 0)  # noqa: E731
    step([20, 1], causal, lambda q, p: f.kv4_attention(q, c, table, p.kv_lens, D ** -0.5, True, p.q_indptr))
    assert math.isfinite(float(lens.sum()))
