"""moe_cache_fork, moe_cache_compact and moe_cache_copy against the plain
definition (loops over rows and pages on the host). Everything is exact."""
import pytest
import torch

import padded_permute_combine_gb300 as p
from padded_permute_combine_gb300 import _lib

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def needs_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def i32(v, shape=None):
    t = torch.tensor(v, dtype=torch.int32)
    return (t if shape is None else t.reshape(shape)).cuda()


def fork(table, lengths, parents, page, pool, grow, width):
    """What moe_cache_fork says, row by row: (table, lengths, src, dst, status)."""
    rows, lens, status = [], [], 0
    for q in parents:
        if q < -1 or q >= len(table):
            status |= _lib.MOE_STATUS_BAD_INDEX
            q = -1
        n = 0
        if q >= 0:
            n = min(max(lengths[q], 0), len(table[q]) * page)
            if n != lengths[q]:
                status |= _lib.MOE_STATUS_BAD_INDEX
        row = [] if q < 0 else [i if 0 <= i < pool else -1 for i in table[q][:-(-n // page)]]
        if -1 in row:
            status |= _lib.MOE_STATUS_BAD_INDEX
        rows.append(row)
        lens.append(n)
    used = {i for row in rows for i in row}
    free = [i for i in range(pool) if i not in used]
    holders, src, dst, out = set(), [], [], []
    for r, (row, n) in enumerate(zip(rows, lens)):
        src.append(-1)
        dst.append(-1)
        alive = -1 < parents[r] < len(table)
        asked = []
        if alive and grow > 0 and n % page and row[-1] >= 0:
            if row[-1] in holders:
                asked.append(len(row) - 1)
            holders.add(row[-1])
        new = row + [-1] * (width - len(row))
        if alive:
            want = -(-(n + grow) // page)
            if want > width:
                status |= _lib.MOE_STATUS_NO_PAGES
            asked += range(len(row), min(want, width))
        for j in asked:
            got = free.pop(0) if free else -1
            if got < 0:
                status |= _lib.MOE_STATUS_NO_PAGES
            elif j < len(row):
                src[r], dst[r] = row[j], got
            new[j] = got
        out.append(new)
    return out, lens, src, dst, status


def beams(requests, width, page, seed, longest=200, shared=0.7):
    """Rows' tables and lengths in a pool, page numbers scattered; (table, lengths, pages used)."""
    g = torch.Generator().manual_seed(seed)
    r = lambda n: int(torch.randint(0, max(1, n), (1,), generator=g))  # noqa: E731
    table, lengths, used = [], [], 0
    for _ in range(requests):
        n = 1 + r(longest)
        common = int(n * shared) // page
        first = used
        used += common
        for _ in range(width):
            own = -(-n // page) - common
            table.append(list(range(first, first + common)) + list(range(used, used + own)))
            used += own
            lengths.append(n)
    pool = int(used * 1.5) + 3 * len(table)
    ids = torch.randperm(pool, generator=g).tolist()
    most = max(len(t) for t in table) + 2
    return [[ids[i] for i in t] + [-9] * (most - len(t)) for t in table], lengths, pool


def run_fork(table, lengths, parents, page, pool, grow=1, width=None):
    status = i32([0])
    got = p.moe_cache_fork(i32(table, (len(table), -1)), i32(lengths, (-1,)), i32(parents, (-1,)), page, pool, grow, width, status=status)
    want = fork(table, lengths, parents, page, pool, grow, width or len(table[0]))
    for g, w, name in zip(got, want, got._fields):
        assert g.flatten().tolist() == (sum(w, []) if name == "page_table" else w), name
    assert int(status) == want[4]
    return got


@pytest.mark.parametrize("page", [1, 3, 16, 64])
@pytest.mark.parametrize("requests,width", [(1, 1), (1, 8), (5, 4), (40, 5), (300, 2)])
@pytest.mark.parametrize("grow", [0, 1, 37])
def test_fork(requests, width, page, grow):
    table, lengths, pool = beams(requests, width, page, seed=requests * 10 + page)
    g = torch.Generator().manual_seed(page)
    R = len(table)
    parents = [b * width + int(torch.randint(0, width, (1,), generator=g)) for b in range(requests) for _ in range(width)]
    run_fork(table, lengths, parents, page, pool, grow, len(table[0]) + 40)
    run_fork(table, lengths, list(range(R)), page, pool, grow, len(table[0]) + 40)
    parents = [-1 if i % 3 == 0 else q for i, q in enumerate(parents)]  # some end
    run_fork(table, lengths, parents, page, pool, grow, len(table[0]) + 40)
    run_fork(table, lengths, [0] * 50, page, pool, grow, len(table[0]) + 40)  # one parent for all
    run_fork(table, lengths, [-1] * 7, page, pool, grow)


def test_fork_twice_and_free():
    """Rows forked without growth share a page that is not full; the next fork still copies it for all but one."""
    table, lengths, pool = [[5, 2, -1], [7, -1, -1]], [20, 16], 12
    got = run_fork(table, lengths, [0, 0, 1, 0], 16, pool, grow=0)
    again = run_fork(got.page_table.tolist(), got.lengths.tolist(), [1, 0, 2, 3], 16, pool)
    assert again.src.tolist() == [-1, 2, -1, 2] and again.dst.tolist() == [-1, 0, -1, 3]
    run_fork(got.page_table.tolist(), got.lengths.tolist(), [2], 16, pool)


def test_fork_without_enough_pages_or_columns():
    table, lengths = [[0, 1], [2, 3]], [8, 7]
    run_fork(table, lengths, [0, 1, 1], 4, 4)          # nothing is free
    run_fork(table, lengths, [0, 1, 1, 1], 4, 5, width=3)  # one page for three requests
    run_fork(table, lengths, [0, 1, 1, 1], 4, 6, width=3)
    run_fork(table, lengths, [0, 1], 4, 100)           # row 0 needs a third column
    run_fork(table, lengths, [0, 1], 4, 100, grow=1000, width=5)
    run_fork(table, lengths, [0, -7, 2, 1], 4, 100, width=3)  # parents that are none
    run_fork([[0, 55], [-3, 3]], [8, 7], [0, 1, 1], 4, 50, width=3)  # pages that are none
    run_fork(table, [-4, 99], [0, 1], 4, 100, width=4)  # lengths that are none


def test_fork_large_pools():
    for pool in (33, 8 * 1024 * 32 + 5, _lib.MOE_CACHE_MAX_PAGES):
        table = [[pool - 1, 0, pool // 2], [pool - 2, 3, 4]]
        run_fork(table, [44, 40], [0, 1, 0, 1, 0, -1], 16, pool, grow=200, width=16)
    # the lowest pages are all in use
    table = [list(range(i * 1000, (i + 1) * 1000)) for i in range(70)]
    run_fork(table, [15999] * 70, [i // 2 for i in range(140)], 16, 75000, grow=33, width=1003)
    R = _lib.MOE_CACHE_MAX_ROWS
    run_fork([[i, -1] for i in range(R)], [3] * R, [i // 3 for i in range(R)], 16, 2 * R)


def compact(table, lengths, page, pool):
    rows = [t[:-(-n // page)] for t, n in zip(table, lengths)]
    named = {i for row in rows for i in row}
    n = len(named)
    movers, holes = sorted(i for i in named if i >= n), [i for i in range(n) if i not in named]
    now = dict(zip(movers, holes))
    return [[now.get(i, i) for i in row] + [-1] * (len(t) - len(row)) for row, t in zip(rows, table)], movers, holes


@pytest.mark.parametrize("page", [1, 16])
@pytest.mark.parametrize("requests,width", [(1, 1), (3, 4), (60, 2), (500, 1)])
def test_compact(requests, width, page):
    table, lengths, pool = beams(requests, width, page, seed=7 * requests + page)
    lengths = [0 if i % 5 == 2 else n for i, n in enumerate(lengths)]  # some were freed
    for size in (pool, pool + 40000):
        status = i32([0])
        got = p.moe_cache_compact(i32(table), i32(lengths), page, size, status=status)
        want, src, dst = compact(table, lengths, page, size)
        assert got.page_table.tolist() == want and int(got.count) == len(src) and int(status) == 0
        assert got.src.tolist() == src + [-1] * (size // 2 - len(src)) and got.dst.tolist() == dst + [-1] * (size // 2 - len(dst))


def test_compact_edges():
    got = p.moe_cache_compact(i32([], (0, 4)), i32([], (0,)), 16, 9)  # no row: nothing in use
    assert int(got.count) == 0 and got.src.tolist() == [-1] * 4
    got = p.moe_cache_compact(i32([[0]]), i32([5]), 16, 1)  # a pool of one page
    assert int(got.count) == 0 and got.page_table.tolist() == [[0]]
    status = i32([0])
    got = p.moe_cache_compact(i32([[7, 99, 3]]), i32([40]), 16, 8, status=status)  # a bad page stays away
    assert got.page_table.tolist() == [[1, -1, 0]] and int(status) == _lib.MOE_STATUS_BAD_INDEX
    assert got.src.tolist() == [3, 7, -1, -1] and got.dst.tolist() == [0, 1, -1, -1]
    N = _lib.MOE_CACHE_MAX_PAGES
    got = p.moe_cache_compact(i32([[N - 1, 5, N - 7]]), i32([48]), 16, N)
    want, src, dst = compact([[N - 1, 5, N - 7]], [48], 16, N)
    assert got.page_table.tolist() == want and got.src[:4].tolist() == src + [-1] and got.dst[:4].tolist() == dst + [-1]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32, torch.uint8])
@pytest.mark.parametrize("shape", [(16, 8, 128), (7, 33), (1,), (5, 3, 11), (16, 8, 1024), (40000,)])
def test_copy(dtype, shape):
    pool = 40
    g = torch.Generator().manual_seed(1)
    new = lambda *s: torch.randint(0, 200, s, generator=g, dtype=torch.int32).cuda().to(dtype)  # noqa: E731
    both = new(pool, 2, *shape)  # keys and values of a page together
    caches = [new(pool, *shape), both[:, 0], both[:, 1], new(3, pool, *shape)[1]]
    if len(shape) == 3:
        caches.append(new(pool, shape[1], shape[0], shape[2]).transpose(1, 2))
    flat = new(pool * 11 + 1)[1:].view(pool, 11)  # off every alignment
    caches.append(flat)
    src = i32([3, -1, 7, 7, 0, 39, 5, 6])
    dst = i32([10, 11, -1, 12, 13, 14, 40, 15])  # 40: beyond the pool
    want = [t.clone() for t in caches]
    for w in want:
        for a, b in ((3, 10), (7, 12), (0, 13), (39, 14), (6, 15)):
            w[b] = w[a]
    status = i32([0])
    p.moe_cache_copy(caches, src, dst, status=status)
    assert all(torch.equal(t, w) for t, w in zip(caches, want)) and int(status) == _lib.MOE_STATUS_BAD_INDEX
    before = [t.clone() for t in caches]
    p.moe_cache_copy(caches, i32([1, 2]), i32([20, 21]), i32([1]))  # one of the two
    for t, b in zip(caches, before):
        b[20] = b[1]
        assert torch.equal(t, b)
    p.moe_cache_copy(caches, i32([1, 2]), i32([22, 23]), i32([-3]))
    p.moe_cache_copy(caches, i32([], (0,)), i32([], (0,)))
    p.moe_cache_copy([], i32([1]), i32([2]))
    assert all(torch.equal(t, b) for t, b in zip(caches, before))


def test_copy_of_many_caches_and_pairs():
    caches = list(torch.arange(300 * 600 * 5, device="cuda").view(300, 600, 5).unbind(0))
    src, dst = torch.full((200,), -1), torch.full((200,), -1)
    src[::3], dst[::3] = torch.arange(67), torch.arange(67) + 300
    want = [t.clone() for t in caches]
    for w in want:
        w[300:367] = w[:67]
    p.moe_cache_copy(caches, src.int().cuda(), dst.int().cuda())
    assert all(torch.equal(t, w) for t, w in zip(caches, want))


def test_captured_step():
    """Fork and copy in a graph, replayed on other parents."""
    table, lengths, pool = beams(4, 4, 16, seed=2)
    t, n, cache = i32(table), i32(lengths), torch.randn(pool, 16, 32, device="cuda")
    parents = i32(list(range(16)))
    p.moe_cache_fork(t, n, parents, 16, pool)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = p.moe_cache_fork(t, n, parents, 16, pool)
        p.moe_cache_copy([cache], got.src, got.dst)
    for seed in range(3):
        g = torch.Generator().manual_seed(seed)
        now = [b * 4 + int(torch.randint(0, 4, (1,), generator=g)) for b in range(4) for _ in range(4)]
        parents.copy_(torch.tensor(now))
        want = fork(table, lengths, now, 16, pool, 1, len(table[0]))
        before = cache.clone()
        graph.replay()
        assert got.page_table.tolist() == want[0] and got.src.tolist() == want[2] and got.dst.tolist() == want[3]
        for a, b in zip(want[2], want[3]):
            if a >= 0:
                before[b] = before[a]
        assert torch.equal(cache, before)
