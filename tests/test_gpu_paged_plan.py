"""usp_page_plan where the new tokens do not fit into slot_map: the plan against the header's definition, written
column by column, and the steps that follow over tables that hold other requests' former pages."""
import random

import pytest
import torch

import sequence_long_context_zigzag_gb300 as usp

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def plan_by_columns(ctx, new, free, head, table, ps, num_pages, max_tokens):
    """(table, slots, cu, kv, counts) as include/usp.h defines them, in Python integers."""
    ctx, new = [max(x, 0) for x in ctx], [max(x, 0) for x in new]
    table, width = [list(row) for row in table], len(table[0])
    slots, cu, lost, at = [-1] * max_tokens, [0], 0, head
    for i, (c, n) in enumerate(zip(ctx, new)):
        old, end = -(-c // ps), -(-(c + n) // ps)
        f = at
        for col in range(old, min(end, width)):
            table[i][col] = free[f + col - old] if f + col - old < len(free) else -1
        at += end - old
        first = sum(new[:i])
        for j in range(n):
            col = (c + j) // ps
            fits = col < width and (col < old or f + col - old < len(free)) and first + j < max_tokens
            lost += not fits
            if first + j < max_tokens and col < width and 0 <= table[i][col] < num_pages:
                slots[first + j] = table[i][col] * ps + (c + j) % ps
        cu.append(min(first + n, max_tokens))
    kv = [c + n for c, n in zip(ctx, new)]
    return table, slots, cu, kv, [sum(new), at, lost, max(kv)]


def run_plan(ctx, new, free, head, table, ps, num_pages, max_tokens):
    t = i32(table)
    outs = usp.usp_page_plan(i32(ctx), i32(new), i32(free), i32([head]), t, ps, num_pages, max_tokens)
    usp.usp_check()
    got = [t.tolist()] + [x.tolist() for x in outs]
    want = plan_by_columns(ctx, new, free, head, table, ps, num_pages, max_tokens)
    for name, g, w in zip(("table", "slots", "cu", "kv", "counts"), got, want):
        assert list(g) == list(w), name
    return want


def lengths(r, nreq, ctx_hi, new_hi):
    return ([r.choice([0, r.randint(0, ctx_hi)]) for _ in range(nreq)],
            [r.choice([0, 1, r.randint(0, new_hi)]) for _ in range(nreq)])


@pytest.mark.parametrize("ps", [16, 256])
@pytest.mark.parametrize("nreq,ctx_hi,new_hi", [(1, 0, 5000), (5, 40, 700), (70, 500, 300), (2500, 60, 90)])
@pytest.mark.parametrize("share", [0.0, 0.3, 0.97])
@pytest.mark.parametrize("spare,width_less", [(9, 0), (-20, 0), (3, 2)])
def test_pages_of_tokens_past_the_slot_map(nreq, ctx_hi, new_hi, ps, share, spare, width_less):
    """max_tokens ends before the new tokens do: these have no slot, but their pages are taken and written."""
    r = random.Random(nreq + ps)
    ctx, new = lengths(r, nreq, ctx_hi, new_hi)
    new[-1] = new_hi   # the tokens without a slot open pages
    old, end = [-(-c // ps) for c in ctx], [-(-(c + n) // ps) for c, n in zip(ctx, new)]
    num = sum(end) + 30
    ids = list(range(num))
    r.shuffle(ids)
    width, at, table = max(max(end) - width_less, 1), 0, []
    for o in old:
        row = ids[at:at + o][:width]
        at += o
        table.append(row + [r.randrange(num) for _ in range(width - len(row))])   # other requests' former pages
    free = ids[at:at + max(sum(end) - sum(old) + spare, 0)]
    run_plan(ctx, new, free, 0, table, ps, num, int(sum(new) * share))


@pytest.mark.parametrize("nreq", [3, 40, 1100])
def test_steps_after_a_plan_that_ran_out_of_slots(nreq):
    """Step after step with too small a slot map, over rows full of stale ids: no page is ever two requests'."""
    r = random.Random(nreq)
    ps, width = 16, 24
    num = nreq * width
    free = list(range(num))
    r.shuffle(free)
    stale = [[r.randrange(num) for _ in range(width)] for _ in range(nreq)]
    ctx, head, table = [0] * nreq, 0, stale
    for _ in range(4):
        new = [r.choice([0, 1, r.randint(0, 90)]) for _ in range(nreq)]
        table, slots, _, ctx, counts = run_plan(ctx, new, free, head, table, ps, num, sum(new) // 2)
        head = counts[1]
        held = [table[i][:-(-c // ps)] for i, c in enumerate(ctx)]
        pages = [x for row in held for x in row]
        assert len(pages) == len(set(pages)) == head
        taken = [s for s in slots if s >= 0]
        assert len(taken) == len(set(taken))
