"""GPU tests of the state pool's pages: copy, fork, free, compact and the
reordering of a beam batch, bit for bit against plain loops on the host."""
import pytest
import torch

import kda_chunked_delta_amd as kda

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def say(*a):
    print(*a, flush=True)


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def make_pool(pages, page, layers=0, dtype=torch.float32, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed + pages)
    shape = ((layers,) if layers else ()) + (pages,) + page
    return torch.randn(*shape, generator=g, device=DEV).to(dtype)


def pages_of(pool, layers):
    """[pages][...] on the host, the layers of a page together."""
    p = pool.cpu()
    return (p.movedim(1, 0) if layers else p).clone()


# pages of one state, odd sizes of 16-byte multiples, several layers, other types
POOLS = [((1, 128, 128), 0, torch.float32), ((3, 128, 128), 2, torch.float32), ((4,), 0, torch.float32),
         ((1028,), 3, torch.float32), ((8200,), 0, torch.bfloat16), ((5, 16), 0, torch.uint8)]


@pytest.mark.parametrize("page,layers,dtype", POOLS)
@pytest.mark.parametrize("P,n", [(1, 1), (7, 3), (40, 40), (64, 200)])
def test_copy_reads_before_it_writes(page, layers, dtype, P, n):
    say("case copy", page, layers, dtype, P, n)
    g = torch.Generator().manual_seed(P * n)
    pool = make_pool(P, page, layers, dtype)
    src = torch.randint(-2, P + 2, (n,), generator=g).tolist()
    dst = torch.randint(-2, P + 2, (n,), generator=g).tolist()
    old = pages_of(pool, layers)
    want = old.clone()
    for a, b in zip(src, dst):
        if 0 <= a < P and 0 <= b < P:
            want[b] = old[a]
    got = kda.pool_copy(pool, ints(src), ints(dst), page_dim=1 if layers else 0)
    assert got is pool and torch.equal(pages_of(pool, layers), want)


@pytest.mark.parametrize("n", [2, 31, 33, 100, 257, 1024])
def test_copy_rotation(n):
    """A rotation of n pages: every page is source and destination."""
    say("case rotation", n)
    pool = make_pool(n, (3, 64), seed=1)
    old = pool.clone()
    src = torch.arange(n, dtype=torch.int32, device=DEV)
    kda.pool_copy(pool, src, src.roll(1).contiguous())
    assert torch.equal(pool, old.roll(1, 0).roll(-2, 0))


def plain_fork(used, src):
    used, dst = list(used), []
    before = list(used)
    for a in src:
        d = -1
        if 0 <= a < len(used) and before[a] and False in used:
            d = used.index(False)
            used[d] = True
        dst.append(d)
    return used, dst


@pytest.mark.parametrize("page,layers,dtype", POOLS[:4])
@pytest.mark.parametrize("P,n,share", [(1, 2, 0.5), (9, 5, 0.5), (64, 40, 0.9), (1500, 300, 0.7), (2100, 1300, 0.3)])
def test_fork(page, layers, dtype, P, n, share):
    if P > 100 and len(page) > 1:
        page = (1, 16, 16)
    say("case fork", page, layers, P, n)
    g = torch.Generator().manual_seed(P + n)
    pool = make_pool(P, page, layers, dtype)
    used = (torch.rand(P, generator=g) < share).tolist()
    src = torch.randint(-1, P + 1, (n,), generator=g).tolist()
    old = pages_of(pool, layers)
    used_want, dst_want = plain_fork(used, src)
    u = torch.tensor(used, device=DEV)
    dst = kda.pool_fork(pool, u, ints(src), page_dim=1 if layers else 0)
    assert dst.tolist() == dst_want and u.tolist() == used_want
    for a, b in zip(src, dst_want):
        if b >= 0:
            old[b] = old[a]
    assert torch.equal(pages_of(pool, layers), old)


def test_fork_a_full_and_an_empty_pool():
    pool = make_pool(5, (64,))
    old = pool.clone()
    for value in (True, False):
        used = torch.full((5,), value, device=DEV)
        assert kda.pool_fork(pool, used, ints([0, 1, 2])).tolist() == [-1] * 3
        assert used.tolist() == [value] * 5 and torch.equal(pool, old)
    used = torch.tensor([True, False, True, False, False], device=DEV)
    assert kda.pool_fork(pool, used, ints([])).numel() == 0
    assert kda.pool_fork(pool, used, ints([2, 2, 2, 0])).tolist() == [1, 3, 4, -1]
    assert torch.equal(pool[[1, 3, 4]], old[[2, 2, 2]])


def test_free():
    used = torch.ones(300, dtype=torch.bool, device=DEV)
    pages = ints([5, 5, -1, 299, 300, 1 << 30, 0, -(1 << 31)])
    assert kda.pool_free(used, pages) is used
    assert (~used).nonzero()[:, 0].tolist() == [0, 5, 299]
    kda.pool_free(used, ints([]))


@pytest.mark.parametrize("page,layers,dtype", POOLS[:4])
@pytest.mark.parametrize("P,share", [(1, 0.0), (1, 1.0), (17, 0.4), (64, 0.9), (1025, 0.5), (3000, 0.2), (2048, 0.98)])
def test_compact(page, layers, dtype, P, share):
    if P > 100 and len(page) > 1:
        page = (1, 16, 16)
    say("case compact", page, layers, P, share)
    g = torch.Generator().manual_seed(P)
    pool = make_pool(P, page, layers, dtype)
    used = (torch.rand(P, generator=g) < share).tolist()
    live = sum(used)
    new = [p if used[p] and p < live else -1 for p in range(P)]
    holes = [p for p in range(live) if not used[p]]
    movers = [p for p in range(live, P) if used[p]]
    assert len(holes) == len(movers)
    want = pages_of(pool, layers)
    for a, b in zip(movers, holes):
        new[a] = b
        want[b] = want[a]
    table = torch.randint(-2, P + 3, (50, 2), generator=g).int()
    table_want = [[new[t] if 0 <= t < P else -1 for t in row] for row in table.tolist()]
    u, t = torch.tensor(used, device=DEV), table.to(DEV)
    got, n_live = kda.pool_compact(pool, u, t, page_dim=1 if layers else 0)
    assert n_live.item() == live and got.tolist() == new
    assert u.tolist() == [p < live for p in range(P)] and t.tolist() == table_want
    assert torch.equal(pages_of(pool, layers)[:live], want[:live])
    assert torch.equal(pages_of(pool, layers)[live:], want[live:])  # the rest is left as it was
    again, _ = kda.pool_compact(pool, u, page_dim=1 if layers else 0)
    assert again.tolist() == [p if p < live else -1 for p in range(P)]


@pytest.mark.parametrize("B,W", [(1, 1), (3, 2), (5, 7), (2, 64), (17, 4)])
@pytest.mark.parametrize("layers", [0, 2])
@pytest.mark.parametrize("page", [(1, 128, 128), (1028,)])
def test_reorder(B, W, layers, page):
    say("case reorder", B, W, layers, page)
    g = torch.Generator().manual_seed(B * W)
    P = B * W + 3
    pool = make_pool(P, page, layers)
    old = pages_of(pool, layers)
    slots = torch.randperm(P, generator=g)[:B * W].view(B, W).int()
    parents = torch.randint(0, W, (B, W), generator=g).int()
    new = kda.beam_reorder(pool, slots.to(DEV), parents.to(DEV), page_dim=1 if layers else 0).cpu()
    now = pages_of(pool, layers)
    for b in range(B):
        assert sorted(new[b].tolist()) == sorted(slots[b].tolist())  # the pages are dealt out anew
        seen = set()
        for w in range(W):
            q = parents[b, w].item()
            assert torch.equal(now[new[b, w]], old[slots[b, q]])
            if q not in seen:  # the first child keeps its parent's page
                assert new[b, w] == slots[b, q]
            seen.add(q)
    rest = [p for p in range(P) if p not in slots.flatten().tolist()]
    assert torch.equal(now[rest], old[rest])


def test_reorder_skips_what_is_no_parent_or_page():
    pool = make_pool(8, (64,))
    old = pool.clone()
    slots = ints([[3, -1, 5, 6], [0, 9, 1, 2]])
    parents = ints([[0, 0, -1, 4], [1, 1, 2, 2]])
    new = kda.beam_reorder(pool, slots, parents).tolist()
    # entry 0: beam 1 copies page 3 to the first page without a beam (-1: not copied)
    assert new[0] == [3, -1, 5, 6]
    # entry 1: beam 0 keeps page 9 (outside), beam 1 gets page 0 uncopied, beam 2 keeps 1, beam 3 copies it to 2
    assert new[1] == [9, 0, 1, 2]
    old[2] = old[1]
    assert torch.equal(pool, old)
    assert kda.beam_reorder(pool, ints([]).view(0, 4), ints([]).view(0, 4)).shape == (0, 4)


def test_strided_layers_and_a_view_of_a_larger_pool():
    """Layers further apart than their pages; what lies between them stays."""
    whole = make_pool(12, (256,), layers=3)
    old = whole.clone()
    view = whole[:, 2:9]
    kda.pool_copy(view, ints([0, 1]), ints([1, 0]), page_dim=1)
    old[:, [2, 3]] = old[:, [3, 2]]
    assert torch.equal(whole, old)


def test_large_offsets():
    """Pages beyond 2^32 bytes of a pool."""
    pool = torch.empty(2300, 1 << 19, device=DEV)  # 2 MiB pages, 4.8 GB
    for p in (0, 1, 2298, 2299):
        pool[p] = torch.randn(1 << 19, device=DEV)
    a, b = pool[0].clone(), pool[2299].clone()
    kda.pool_copy(pool, ints([0, 2299]), ints([2299, 0]))
    assert torch.equal(pool[2299], a) and torch.equal(pool[0], b)
    used = torch.zeros(2300, dtype=torch.bool, device=DEV)
    used[2299] = True
    new, live = kda.pool_compact(pool, used)
    assert live.item() == 1 and new[2299].item() == 0 and torch.equal(pool[0], a)
    new = kda.beam_reorder(pool, ints([[2298, 2299]]), ints([[1, 1]]))
    assert new.tolist() == [[2299, 2298]] and torch.equal(pool[2298], a)


def test_refusals():
    pool = make_pool(4, (64,))
    used = torch.ones(4, dtype=torch.bool, device=DEV)
    i = ints([0, 1])
    for call in (lambda: kda.pool_copy(pool, i, ints([0])), lambda: kda.pool_copy(pool, i.long(), i),
                 lambda: kda.pool_copy(pool, i.cpu(), i), lambda: kda.pool_copy(pool[:, :32], i, i),
                 lambda: kda.pool_copy(pool[::2], i, i), lambda: kda.pool_copy(pool.cpu(), i, i),
                 lambda: kda.pool_fork(pool, used[:3], i), lambda: kda.pool_fork(pool, used.int(), i),
                 lambda: kda.pool_free(used.int(), i), lambda: kda.pool_compact(pool, used, i.float()),
                 lambda: kda.beam_reorder(pool, i, i), lambda: kda.beam_reorder(pool, i.view(1, 2), i.view(2, 1)),
                 lambda: kda.pool_copy(pool, i, i, page_dim=2), lambda: kda.pool_copy(pool[:0], i, i)):
        with pytest.raises(ValueError):
            call()
    many = torch.zeros(1025, dtype=torch.int32, device=DEV)
    for call in (lambda: kda.pool_copy(pool, many, many), lambda: kda.pool_copy(pool[:, :3].contiguous(), i, i),
                 lambda: kda.beam_reorder(pool, many[:65].view(1, 65), many[:65].view(1, 65)),
                 lambda: kda.pool_fork(pool, used, pool.view(torch.int32).view(-1)[:4])):
        with pytest.raises(kda.KDAError):
            call()


def test_graph_of_a_serving_step():
    """Free, fork, copy, reorder and compact captured together and replayed with new tables."""
    P = 24
    g = torch.Generator().manual_seed(3)
    pool, used = make_pool(P, (2, 64)), torch.zeros(P, dtype=torch.bool, device=DEV)
    gone, src, a, b = ints([0, 0]), ints([0, 0, 0]), ints([0, 0]), ints([0, 0])
    slots, parents = ints([[0, 1, 2]]), ints([[0, 0, 0]])

    def step(pool, used):
        kda.pool_free(used, gone)
        dst = kda.pool_fork(pool, used, src)
        kda.pool_copy(pool, a, b)
        new = kda.beam_reorder(pool, slots, parents)
        table = torch.cat([dst, new.view(-1)])
        pages, live = kda.pool_compact(pool, used, table)
        return dst, new, table, pages, live

    step(pool.clone(), used.clone())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step(pool, used)
    for it in range(4):
        mask = torch.rand(P, generator=g) < 0.7
        live = mask.nonzero()[:, 0]
        pick = lambda n: live[torch.randint(0, len(live), (n,), generator=g)].int()
        fresh = torch.randn(P, 2, 64, generator=g)
        for t, v in ((pool, fresh), (used, mask), (gone, pick(2)), (src, pick(3)), (a, pick(2)), (b, pick(2)),
                     (slots, live[:3].int().view(1, 3)), (parents, torch.randint(0, 3, (1, 3), generator=g).int())):
            t.copy_(v)
        p2, u2 = pool.clone(), used.clone()
        want = step(p2, u2)
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(outs, want):
            assert torch.equal(x, y)
        assert torch.equal(pool, p2) and torch.equal(used, u2)
