"""Copying, forking, freeing and compacting the pages of a cache: books and bytes equal to a plain list
form (seq_ref), with repeated and bad requests among them."""
import random

import pytest
import torch

import seq_ref as ref

pytestmark = pytest.mark.gpu


def pool(n_pages, seed, odd=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = [torch.randn(n_pages, 3, 64, 64, device="cuda", generator=g), torch.randn(n_pages, 5, 7, device="cuda", generator=g),
         torch.randn(n_pages, 3, 24, device="cuda", generator=g).bfloat16()]
    if odd:  # pages of odd byte counts, a tensor whose base is 1 byte off
        raw = torch.randint(0, 255, (n_pages * 13 + 1,), device="cuda", generator=g, dtype=torch.uint8)
        t += [raw[1:].view(n_pages, 13), torch.randint(0, 255, (n_pages, 70001), device="cuda", generator=g, dtype=torch.uint8)]
    return t


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def moved(tensors, moves):
    want = [t.clone() for t in tensors]
    for src, dst in moves:
        for w, t in zip(want, tensors):
            w[dst] = t[src] if src >= 0 else 0
    return want


def books(rng, n_rows, n_pages, live):
    table, owner = [-1] * n_rows, [-1] * n_pages
    for r, p in zip(rng.sample(range(n_rows), live), rng.sample(range(n_pages), live)):
        table[r], owner[p] = p, r
    return table, owner


@pytest.mark.parametrize("n_rows,n_pages,live,n", [(4, 4, 2, 3), (40, 16, 9, 12), (10, 300, 8, 5), (3000, 2500, 1100, 1700), (1, 1, 0, 2)])
def test_fork(libttt, n_rows, n_pages, live, n):
    rng = random.Random(n_rows)
    table, owner = books(rng, n_rows, n_pages, live)
    small = n_pages > 1000
    t = [torch.randn(n_pages, 12, device="cuda")] if small else pool(n_pages, 1, odd=True)
    held = [r for r in range(n_rows) if table[r] >= 0] or [0]
    parents = [rng.choice([-1, -1, rng.randrange(n_rows), rng.choice(held), rng.choice(held), n_rows, -7]) for _ in range(n)]
    children = [rng.choice([rng.randrange(n_rows), rng.randrange(n_rows), rng.randrange(n_rows), n_rows + 3, -1]) for _ in range(n)]
    dt, do = i32(table), i32(owner)
    before = [x.clone() for x in t]
    pages = libttt.ttt_cache_fork(t, dt, do, i32(parents), i32(children))
    want, moves = ref.fork(table, owner, parents, children, n_pages)
    assert pages.tolist() == want and dt.tolist() == table and do.tolist() == owner
    for x, y in zip(t, moved(before, moves)):
        assert torch.equal(x, y)


@pytest.mark.parametrize("n_rows,n_pages,live,n", [(4, 4, 3, 2), (40, 16, 16, 12), (300, 257, 200, 150), (3000, 2500, 2400, 2600), (1, 1, 1, 1), (5, 9, 0, 3)])
def test_free_then_compact(libttt, n_rows, n_pages, live, n):
    rng = random.Random(n_pages)
    table, owner = books(rng, n_rows, n_pages, live)
    t = [torch.randn(n_pages, 12, device="cuda")] if n_pages > 1000 else pool(n_pages, 2, odd=True)
    rows = [rng.choice([rng.randrange(n_rows), rng.randrange(n_rows), -1, n_rows]) for _ in range(n)]
    dt, do = i32(table), i32(owner)
    freed = libttt.ttt_cache_free(dt, do, i32(rows))
    count = 0
    for r in rows:
        if 0 <= r < n_rows and table[r] >= 0:
            owner[table[r]], table[r] = -1, -1
            count += 1
    assert int(freed) == count and dt.tolist() == table and do.tolist() == owner
    before = [x.clone() for x in t]
    got, new = libttt.ttt_cache_compact(t, dt, do)
    want, new_want, moves = ref.compact(table, owner)
    assert int(got) == want and new.tolist() == new_want and dt.tolist() == table and do.tolist() == owner
    for x, y in zip(t, moved(before, moves)):
        assert torch.equal(x, y)
    assert all((o >= 0) == (p < want) for p, o in enumerate(owner))


def test_copy_refuses_what_depends_on_order(libttt):
    t = pool(10, 3, odd=True)
    before = [x.clone() for x in t]
    src, dst = [0, 1, 2, 3, 0, 4, 9, -1, 5], [5, 5, 7, 2, 8, 4, 10, 6, 6]
    # 0->5 is refused since 5 is a source, so is 1->5; 3->2 since 2 is a source; 4->4, 9->10, -1->6 too
    copied = libttt.ttt_cache_copy(t, i32(src), i32(dst))
    want = []
    for i, (a, b) in enumerate(zip(src, dst)):
        want.append(int(0 <= a < 10 and 0 <= b < 10 and a != b and b not in src and b not in dst[:i]))
    assert copied.tolist() == want and sum(want) == 2
    for x, y in zip(t, moved(before, [(a, b) for a, b, ok in zip(src, dst, want) if ok])):
        assert torch.equal(x, y)


def test_calls_are_captured(libttt):
    """Fork, free and compact in one graph, replayed on other books."""
    t = [torch.randn(12, 40, device="cuda")]
    dt, do, par, chi, rows = i32([-1] * 6), i32([-1] * 12), i32([-1, -1]), i32([0, 1]), i32([3])
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        libttt.ttt_cache_fork(t, dt, do, par, chi)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        pages = libttt.ttt_cache_fork(t, dt, do, par, chi)
        libttt.ttt_cache_free(dt, do, rows)
        live, _ = libttt.ttt_cache_compact(t, dt, do)
    table, owner = [7, -1, 3, 9, -1, -1], [-1] * 12
    for r, p in enumerate(table):
        if p >= 0:
            owner[p] = r
    for parents, children, gone in (([0, -1], [1, 4], [3]), ([4, 1], [3, 5], [0])):
        dt.copy_(i32(table)), do.copy_(i32(owner)), par.copy_(i32(parents)), chi.copy_(i32(children)), rows.copy_(i32(gone))
        before = t[0].clone()
        g.replay()
        want, moves = ref.fork(table, owner, parents, children, 12)
        after = moved([before], moves)
        for r in gone:
            owner[table[r]], table[r] = -1, -1
        n, _, moves = ref.compact(table, owner)
        after = moved(after, moves)
        assert pages.tolist() == want and int(live) == n and dt.tolist() == table and do.tolist() == owner
        assert torch.equal(t[0], after[0])
