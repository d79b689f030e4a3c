"""A serving step's maps on MI355X against the same rules request by request on the host: equal whole numbers."""
import random

import pytest
import torch

import gated_deltanet_fwd_amd as G

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def reference(lengths, contexts, table, free, room, block):
    width, free, table = len(table[0]), list(free), [list(r) for r in table]
    cu, pos, slots, keep, granted, sin, sout, ctx = [0], [], [], [], [], [], [], []
    held = False
    for n, (x, c) in enumerate(zip(lengths, contexts)):
        odd = c < 0 or c > width * block
        base = 0 if odd else c
        if odd or x < 0 or base + x > width * block:
            x = 0
        has = -(-base // block)
        need = -(-(base + x) // block) - has
        held = held or len(pos) + x > room or need > len(free)
        if held:
            x, need = 0, 0
        for i in range(need):
            table[n][has + i] = free.pop()
        sin.append(table[n][(base - 1) // block] if base else -1)
        sout.append(table[n][(base + x - 1) // block] if base + x else -1)
        for p in range(base, base + x):
            pos.append(p)
            slots.append(table[n][p // block] * block + p % block)
            keep.append(table[n][p // block] if (p + 1) % block == 0 and p + 1 < base + x else -1)
        cu.append(len(pos))
        granted.append(x)
        ctx.append(c if odd else c + x)
    rest = room - len(pos)
    return dict(cu_seqlens=cu, positions=pos + [0] * rest, token_slots=slots + [-1] * rest, granted=granted, slot_in=sin,
                slot_out=sout, slot_tok=keep + [-1] * rest, contexts=ctx, free_count=[len(free)]), table


def check(lengths, contexts, room, block, width, n_free, seed=0, in_place=True, count=None):
    r = random.Random(seed)
    held = [-(-max(c, 0) // block) if c <= width * block else 0 for c in contexts]
    ids = list(range(sum(held) + n_free))
    r.shuffle(ids)
    table, at = [], 0
    for h in held:
        table.append(ids[at:at + h] + [-1] * (width - h))
        at += h
    free, count = ids[at:], n_free if count is None else count
    p = G.StepMapsProblem(len(lengths), room, block, width, n_free)
    ctx, cnt, tab = i32(contexts), i32([count]), i32(table)
    kw = {} if in_place else dict(contexts_out=torch.empty_like(ctx), free_count_out=torch.empty_like(cnt))
    got = G.gdn_step_maps(p, i32(lengths), ctx, tab, i32(free), cnt, **kw)
    want, wtab = reference(lengths, contexts, table, free[:max(min(count, n_free), 0)], room, block)
    for name, x in want.items():
        assert got[name].tolist() == x, (name, seed)
    assert tab.tolist() == wtab
    if in_place:
        assert ctx.tolist() == want["contexts"] and cnt.tolist() == want["free_count"]
    else:
        assert ctx.tolist() == contexts and cnt.tolist() == [count]


@pytest.mark.parametrize("room", [300, 4096, 4097, 9000])
@pytest.mark.parametrize("block", [1, 16, 100])
def test_random_batches(room, block):
    for seed in range(8):
        r = random.Random(seed * 31 + room)
        n = r.choice([1, 2, 17, 70])
        lengths = [r.choice([0, 1, 1, r.randint(1, max(1, 2 * room // n))]) for _ in range(n)]
        contexts = [r.choice([0, block, 2 * block, r.randint(0, 200)]) for _ in range(n)]
        width = (max(contexts) + max(lengths)) // block + 1
        need = sum(-(-(c + x) // block) - -(-c // block) for c, x in zip(contexts, lengths))
        check(lengths, contexts, room, block, width, max(0, need - r.choice([0, 0, 1, need // 2])), seed, in_place=seed % 2 == 0)


def test_edges():
    check([0], [0], 4, 16, 1, 0)
    check([1], [0], 1, 1, 1, 1)
    check([0, 0, 0], [5, 0, 16], 0, 16, 2, 3)           # no room for tokens
    check([5, 5, 5], [0, 0, 0], 10, 4, 4, 9)            # tokens for two
    check([5, 5, 0, 5], [0, 0, 0, 0], 100, 4, 4, 3)     # blocks for one
    check([-3, 4, 4, 2], [0, -1, 60, 7], 100, 4, 15, 9)  # what no request can have: only that one gets nothing
    check([2, 2], [9, 3], 100, 4, 2, 9)                 # a context past its table
    check([3, 3], [0, 0], 100, 4, 2, 5, count=99)       # a count past the list
    check([3, 3], [0, 0], 100, 4, 2, 5, count=-7)
    check([1] * 4096, [15] * 4096, 4096, 16, 2, 10)
    check([2] * 4096, [15] * 4096, 8192, 16, 2, 4095)
    check([2 ** 31 - 1, 2 ** 31 - 1, 1], [0, 0, 0], 50, 2 ** 20, 2 ** 11, 2)


def test_graph_moves_on():
    """Captured once, replayed: contexts, table and the free list's count move on in place as in eager steps."""
    for room, lengths in ((8, [1, 1, 0, 2]), (6000, [900, 1, 0, 2])):
        p = G.StepMapsProblem(4, room, 4, 5000, 4000)
        new = lambda: [i32(lengths), i32([0, 3, 0, 8]), torch.full((4, 5000), -1, dtype=torch.int32, device=DEV),  # noqa: E731
                       torch.arange(4000, dtype=torch.int32, device=DEV), i32([4000])]
        a, b = new(), new()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = G.gdn_step_maps(p, *a)
        s = torch.cuda.Stream()
        for _ in range(4):
            s.wait_stream(torch.cuda.current_stream())
            want = G.gdn_step_maps(p, *b, stream=s)
            s.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            for name in want:
                assert torch.equal(got[name], want[name]), name
            assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_binding_refusals():
    p = G.StepMapsProblem(2, 4, 4, 3, 5)
    a = [i32([1, 1]), i32([0, 0]), i32([[-1] * 3] * 2), i32([0] * 5), i32([5])]
    for i, bad in ((0, i32([1])), (1, a[1].long()), (2, a[2].t()), (3, i32([0])), (4, i32([5, 5])), (1, a[1].cpu())):
        x = list(a)
        x[i] = bad
        with pytest.raises(G.GdnError):
            G.gdn_step_maps(p, *x)
    with pytest.raises(G.GdnError):
        G.gdn_step_maps(p, *a, outs=dict(token_slots=i32([0] * 4)))
