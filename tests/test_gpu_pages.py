"""The pages' calls against the same done page by page on the host."""
import random

import pytest
import torch

from sparse_attention_top_idx_gb300 import dsaidx, latent, pages

pytestmark = pytest.mark.gpu

I32 = torch.int32


def dev(x):
    return torch.tensor(x, dtype=I32, device="cuda")


class Host:
    """Counts and tables as lists."""

    def __init__(self, refs, bs):
        self.refs, self.bs = list(refs), bs

    def lowest(self, n):
        got = [i for i, r in enumerate(self.refs) if r == 0][:n]
        return got if len(got) == n else None

    def fork(self, table, lens, parents, width):
        """Rows, lengths, pairs and whether a check failed."""
        bad, starved, rows, out, pairs = False, False, [], [], []
        fresh, taken = iter([i for i, r in enumerate(self.refs) if r == 0]), []
        for p in parents:
            row, n, pair = [], 0, (-1, -1)
            if p != -1:
                if not 0 <= p < len(table) or not 0 <= lens[p] <= min(len(table[p]), width) * self.bs:
                    bad = True
                else:
                    n = lens[p]
                    new = None
                    if n % self.bs:
                        new = next(fresh, None)
                        if new is None:
                            bad, n = True, 0
                    if n:
                        for x in table[p][:n // self.bs]:
                            if 0 <= x < len(self.refs):
                                self.refs[x] += 1
                                row.append(x)
                            else:
                                bad = True
                                row.append(-1)
                        if new is not None:
                            row.append(new)
                            taken.append(new)
                            pair = (table[p][n // self.bs], new)
            rows.append(row + [-1] * (width - len(row)))
            out.append(n)
            pairs.append(pair)
        for x in taken:
            self.refs[x] = 1
        return rows, out, pairs, bad

    def extend(self, table, lens, longer):
        bad, starved = False, False
        fresh = [i for i, r in enumerate(self.refs) if r == 0]
        for i, (n, m) in enumerate(zip(list(lens), longer)):
            if not 0 <= n <= m <= len(table[i]) * self.bs:
                bad = True
                continue
            a, b = -(-n // self.bs), -(-m // self.bs)
            if b > a and (starved or b - a > len(fresh)):
                bad = starved = True
                continue
            for j in range(a, b):
                table[i][j] = fresh.pop(0)
                self.refs[table[i][j]] = 1
            lens[i] = m
        return bad

    def free(self, table, lens, which):
        bad = False
        for r in which:
            if not 0 <= r < len(table):
                bad = True
                continue
            lens[r] = 0
            for j, x in enumerate(table[r]):
                if x >= len(self.refs) or (x >= 0 and self.refs[x] <= 0):
                    bad = True
                elif x >= 0:
                    self.refs[x] -= 1
                if x >= 0:
                    table[r][j] = -1
        return bad

    def compact(self, table):
        n = sum(1 for r in self.refs if r > 0)
        holes = iter([i for i in range(n) if self.refs[i] <= 0])
        new = [(i if i < n else next(holes)) if r > 0 else -1 for i, r in enumerate(self.refs)]
        moved = [(i, k) for i, k in enumerate(new) if k >= 0 and k != i]
        after = [0] * len(new)
        for i, k in enumerate(new):
            if k >= 0:
                after[k] = self.refs[i]
        bad = any(x >= len(new) or (x >= 0 and new[x] < 0) for row in table for x in row)
        rows = [[new[x] if 0 <= x < len(new) else -1 for x in row] for row in table]
        return rows, after, new, moved, bad


def state(seed, rows=6, width=9, bs=8, spare=20, top=None):
    """Host counts and a table of rows with random lengths; pages at random ids."""
    r = random.Random(seed)
    lens = [min(r.choice([0, 1, bs, bs + 1, r.randint(0, width * bs)]), width * bs) for _ in range(rows)]
    if top:
        lens[-1] = top
    nblk = [-(-n // bs) for n in lens]
    nb = sum(nblk) + spare
    ids = list(range(nb))
    r.shuffle(ids)
    h = Host([0] * nb, bs)
    table = []
    for k in nblk:
        row = [ids.pop() for _ in range(k)]
        for x in row:
            h.refs[x] = 1
        table.append(row + [-1] * (width - k))
    return h, table, lens, r


def workspace(nb, rows):
    return dsaidx.new_workspace(pages.workspace_bytes(nb, rows))


def gpu_fork(ps, table, lens, parents, width, ws, stream=None):
    n = len(parents)
    t2 = torch.full((n, width), 77, dtype=I32, device="cuda")
    l2, pairs = torch.full((n,), 77, dtype=I32, device="cuda"), torch.full((n, 2), 77, dtype=I32, device="cuda")
    pages.fork(ps, table, lens, dev(parents), t2, l2, pairs, ws, stream=stream)
    return t2, l2, pairs


@pytest.mark.parametrize("seed,rows,width,bs,spare,n", [(0, 1, 1, 64, 1, 1), (1, 6, 9, 8, 20, 11), (2, 40, 30, 16, 300, 130),
                                                       (3, 3, 700, 4, 50, 7), (4, 200, 5, 1, 9, 300), (5, 9, 70, 64, 5000, 1500),
                                                       (6, 2, 3, 7, 3, 0)])
def test_fork(seed, rows, width, bs, spare, n):
    h, table, lens, r = state(seed, rows, width, bs, max(spare, n))
    parents = [r.choice([-1] + list(range(rows))) for _ in range(n)]
    ps = pages.PageSet(dev(h.refs), bs)
    ws = workspace(len(h.refs), n)
    t, l = dev(table), dev(lens)
    wide = width + r.randint(0, 3)
    got = gpu_fork(ps, t, l, parents, wide, ws)
    want = h.fork(table, lens, parents, wide)
    assert [x.tolist() for x in got] == [want[0], want[1], [list(p) for p in want[2]]]
    assert ps.refs.tolist() == h.refs and dsaidx.read_device_status(ws) == 0
    assert t.tolist() == table and l.tolist() == lens


def test_fork_checks():
    h, table, lens, r = state(7, 8, 6, 4, 3)
    lens[:4] = [5, 9, 21, 22]                          # some pages of rows 2 and 3 are not there
    for i in range(4):
        table[i] = (table[i] + [-1] * 6)[:6]
    table[1][0], table[1][1] = len(h.refs), -9
    lens[5], lens[6] = -1, 25
    parents = [0, 1, 8, -2, 5, 6, 2, 0, 0, 3, 0, -1]   # three free pages: the fourth row that needs one gets none
    ps, ws = pages.PageSet(dev(h.refs), 4), workspace(len(h.refs), len(parents))
    got = gpu_fork(ps, dev(table), dev(lens), parents, 6, ws)
    want = h.fork(table, lens, parents, 6)
    assert want[3] and dsaidx.read_device_status(ws) == 5
    pairs = [p if 0 <= p[0] < len(h.refs) else (-1, -1) for p in want[2]]
    assert [x.tolist() for x in got] == [want[0], want[1], [list(p) for p in pairs]]
    assert ps.refs.tolist() == h.refs
    # a new table that is too narrow for the parent's length
    ws = workspace(len(h.refs), 1)
    t2, l2, _ = gpu_fork(ps, dev([[0, 1, 2]]), dev([12]), [0], 2, ws)
    assert dsaidx.read_device_status(ws) == 5 and t2.tolist() == [[-1, -1]] and l2.tolist() == [0]


@pytest.mark.parametrize("seed,rows,width,bs,spare", [(0, 1, 2, 64, 2), (1, 7, 12, 8, 100), (2, 300, 9, 4, 3000), (3, 2, 900, 2, 2000),
                                                     (4, 1100, 3, 16, 2500), (5, 30, 8, 4, 25)])
def test_extend(seed, rows, width, bs, spare):
    h, table, lens, r = state(seed, rows, width, bs, spare)
    longer = [r.randint(n, width * bs) for n in lens]
    if seed == 5:                                       # too few pages, a length that falls, one past its row
        longer[3], longer[4] = lens[3] - 1, width * bs + 1
    ps, ws, t, l = pages.PageSet(dev(h.refs), bs), workspace(len(h.refs), rows), dev(table), dev(lens)
    pages.extend(ps, t, l, dev(longer), ws)
    bad = h.extend(table, lens, longer)
    assert dsaidx.read_device_status(ws) == (5 if bad else 0) and bad == (seed == 5)
    assert t.tolist() == table and l.tolist() == lens and ps.refs.tolist() == h.refs


@pytest.mark.parametrize("seed,rows,width,which", [(0, 1, 1, None), (1, 6, 9, [2, 0, 2, 2, 5]), (2, 40, 700, None), (3, 5, 3, []),
                                                  (4, 300, 4, list(range(299, -1, -3)))])
def test_free(seed, rows, width, which):
    h, table, lens, r = state(seed, rows, width, 4)
    extra = h.fork(table, lens, [r.randrange(rows) for _ in range(rows)], width)     # shared pages
    table, lens = table + extra[0], lens + extra[1]
    ps, t, l = pages.PageSet(dev(h.refs), 4), dev(table), dev(lens)
    status = torch.zeros(1, dtype=I32, device="cuda")
    pages.free(ps, t, l, None if which is None else dev(which), status=status)
    assert not h.free(table, lens, range(len(table)) if which is None else sorted(set(which)))
    assert t.tolist() == table and l.tolist() == lens and ps.refs.tolist() == h.refs and int(status) == 0
    if which is None:
        assert not any(h.refs)


def test_free_checks():
    h, table, lens, r = state(8, 5, 6, 4)
    table[0][5], table[3][5] = len(h.refs) + 3, h.refs.index(0)
    ps, t, l = pages.PageSet(dev(h.refs), 4), dev(table), dev(lens)
    for which in ([0], [3], [5], [-1], [1]):
        status = torch.zeros(1, dtype=I32, device="cuda")
        pages.free(ps, t, l, dev(which), status=status)
        bad = h.free(table, lens, which)
        assert int(status) == (5 if bad else 0) and bad == (which != [1])
        assert t.tolist() == table and l.tolist() == lens and ps.refs.tolist() == h.refs
    pages.free(ps, t, l, dev([7, 0]))                    # no status word to set


def compact_call(ps, t, in_place=False):
    nb = ps.num_blocks
    refs2, t2 = (ps.refs, t) if in_place else (torch.full_like(ps.refs, 77), torch.full_like(t, 77))
    page_map, pairs = torch.full((nb,), 77, dtype=I32, device="cuda"), torch.full((max(nb // 2, 1), 2), 77, dtype=I32, device="cuda")
    count, ws = torch.full((1,), 77, dtype=I32, device="cuda"), workspace(nb, 0)
    pages.compact(ps, t, refs2, t2, page_map, pairs, count, ws)
    return t2, refs2, page_map, pairs, int(count), dsaidx.read_device_status(ws)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("nb,live", [(1, 1.0), (1, 0.0), (2, 0.5), (3, 0.5), (127, 0.4), (128, 0.9), (129, 0.1), (5000, 0.5),
                                     (40001, 0.3), (300000, 0.6), (777, 0.0), (778, 1.0)])
def test_compact(nb, live, in_place):
    r = random.Random(nb)
    h = Host([r.randint(1, 3) if r.random() < live else 0 for _ in range(nb)], 8)
    used = [i for i, x in enumerate(h.refs) if x]
    table = [[r.choice(used) if used and r.random() < 0.8 else -1 for _ in range(37)] for _ in range(11)]
    ps, t = pages.PageSet(dev(h.refs), 8), dev(table)
    t2, refs2, page_map, pairs, count, status = compact_call(ps, t, in_place)
    rows, after, new, moved, bad = h.compact(table)
    assert status == 0 and not bad and count == len(moved)
    assert t2.tolist() == rows and refs2.tolist() == after and page_map.tolist() == new
    if nb > 1:
        assert pairs.tolist() == [list(p) for p in moved] + [[-1, -1]] * (nb // 2 - len(moved))
    if not in_place:
        assert ps.refs.tolist() == h.refs and t.tolist() == table


def test_compact_checks():
    h = Host([1, 0, 2, 0, 0, 3, 1], 4)
    table = [[0, 2, 5], [1, 7, 6], [-3, 1 << 30, -1]]      # a free page, one past the pool, -3, one far past
    t2, refs2, _, _, count, status = compact_call(pages.PageSet(dev(h.refs), 4), dev(table))
    rows, after, _, moved, bad = h.compact(table)
    assert bad and status == 5 and t2.tolist() == rows and refs2.tolist() == after and count == len(moved) == 2


@pytest.mark.parametrize("n,nb,sizes", [(1, 2, [16]), (5, 40, [16 * 1024, 8448, 41216]), (300, 900, [32, 20608 + 4224]),
                                        (0, 4, [64]), (9, 30, [16 * 1025, 48, 131072 + 16] * 9)])
def test_copy(n, nb, sizes):
    g = torch.Generator(device="cuda").manual_seed(n)
    pools = [torch.randint(0, 256, (nb, b), generator=g, device="cuda", dtype=torch.uint8) for b in sizes]
    order = torch.randperm(nb, generator=g, device="cuda")[:2 * n].view(n, 2).to(I32)
    if n > 3:
        order[2, 0], order[3, 1] = -1, -4
        order[4:7, 0] = int(order[4, 0])                      # one page to several
    pairs = order.contiguous()
    want = [p.clone() for p in pools]
    keep = (pairs >= 0).all(1)
    for w in want:
        w[pairs[keep, 1].long()] = w[pairs[keep, 0].long()]
    ps = pages.PageSet(torch.zeros(nb, dtype=I32, device="cuda"), 64, pools)
    status = torch.zeros(1, dtype=I32, device="cuda")
    pages.copy(ps, pairs, status=status)
    assert int(status) == 0 and all(torch.equal(a, b) for a, b in zip(pools, want))


def test_copy_counts_and_checks():
    pools = [torch.arange(6, dtype=torch.uint8, device="cuda")[:, None].repeat(1, 32)]
    ps = pages.PageSet(torch.zeros(6, dtype=I32, device="cuda"), 64, pools)
    pairs = dev([[0, 3], [6, 1], [1, 6], [1, 4], [2, 5]])
    for count, want, bad in ((0, [0, 1, 2, 3, 4, 5], 0), (-4, [0, 1, 2, 3, 4, 5], 0), (1, [0, 1, 2, 0, 4, 5], 0),
                             (4, [0, 1, 2, 0, 1, 5], 5), (99, [0, 1, 2, 0, 1, 2], 5)):
        status = torch.zeros(1, dtype=I32, device="cuda")
        pages.copy(ps, pairs, count=dev([count]), status=status)
        assert pools[0][:, 0].tolist() == want and torch.equal(pools[0][:, :1].expand(-1, 32), pools[0])
        assert int(status) == bad
    pages.copy(pages.PageSet(ps.refs, 64), pairs)           # no pools: nothing to do


def test_far_pages():
    """A page beyond 2^32 bytes into its pool."""
    b = 41216
    nb = (1 << 32) // b + 20
    pool = torch.empty(nb, b, dtype=torch.uint8, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    pool[-1] = torch.randint(0, 256, (b,), generator=g, device="cuda", dtype=torch.uint8)
    last, first = pool[-1].clone(), torch.randint(0, 256, (b,), generator=g, device="cuda", dtype=torch.uint8)
    pool[0] = first
    ps = pages.PageSet(torch.zeros(nb, dtype=I32, device="cuda"), 64, [pool])
    pages.copy(ps, dev([[nb - 1, 3], [0, nb - 2]]))
    assert torch.equal(pool[3], last) and torch.equal(pool[nb - 2], first) and torch.equal(pool[nb - 1], last)


def test_a_life_of_rows():
    """Forks, growth, ends and compactions in turn, through two tables, against the host."""
    h, table, lens, r = state(11, 12, 10, 4, 60)
    nb = len(h.refs)
    g = torch.Generator(device="cuda").manual_seed(2)
    pool = torch.randint(0, 256, (nb, 64), generator=g, device="cuda", dtype=torch.uint8)
    host = [pool[i].tolist() for i in range(nb)]
    ps, ws, t, l = pages.PageSet(dev(h.refs), 4, [pool]), workspace(nb, 12), dev(table), dev(lens)
    for step in range(25):
        parents = [r.choice([-1, 0, 1, 2, 3, 4, 5, 6, 7, 8, 9, 10, 11]) for _ in range(12)]
        t2, l2, pairs = gpu_fork(ps, t, l, parents, 10, ws)
        t3, lens3, p3, _ = h.fork(table, lens, parents, 10)
        pages.copy(ps, pairs)
        for a, b in p3:
            if a >= 0:
                host[b] = list(host[a])
        pages.free(ps, t, l)                                # the rows before end
        h.free(table, lens, range(12))
        longer = [min(n + r.randint(0, 9), 40) for n in lens3]
        pages.extend(ps, t2, l2, dev(longer), ws)
        h.extend(t3, lens3, longer)
        assert t2.tolist() == t3 and l2.tolist() == lens3 and ps.refs.tolist() == h.refs
        if step % 5 == 4:
            count, page_map = torch.zeros(1, dtype=I32, device="cuda"), torch.empty(nb, dtype=I32, device="cuda")
            moves = torch.empty(nb // 2, 2, dtype=I32, device="cuda")
            pages.compact(ps, t2, ps.refs, t2, page_map, moves, count, ws)
            pages.copy(ps, moves, count=count)
            t3, h.refs, _, moved, _ = h.compact(t3)
            for a, b in moved:
                host[b] = list(host[a])
            assert t2.tolist() == t3 and ps.refs.tolist() == h.refs
            n = sum(1 for x in h.refs if x)
            assert all(h.refs[:n]) and not any(h.refs[n:])
        t, l, table, lens = t2, l2, t3, lens3
        used = [i for i, x in enumerate(h.refs) if x]
        assert pool[used].tolist() == [host[i] for i in used]
    dsaidx.read_device_status(ws)                           # rows that found no page set it; nothing else differs


def test_captured_and_on_another_stream():
    h, table, lens, r = state(12, 6, 8, 4, 40)
    pool = torch.arange(len(h.refs), dtype=torch.uint8, device="cuda")[:, None].repeat(1, 48).contiguous()
    ps, ws, t, l = pages.PageSet(dev(h.refs), 4, [pool]), workspace(len(h.refs), 9), dev(table), dev(lens)
    t2, l2 = torch.full((9, 8), -1, dtype=I32, device="cuda"), torch.zeros(9, dtype=I32, device="cuda")
    pairs, parents, longer = torch.empty(9, 2, dtype=I32, device="cuda"), dev([0] * 9), dev([0] * 9)

    def step(stream=None):
        pages.free(ps, t2, l2, stream=stream)
        pages.fork(ps, t, l, parents, t2, l2, pairs, ws, stream=stream)
        pages.copy(ps, pairs, stream=stream)
        pages.extend(ps, t2, l2, longer, ws, stream=stream)

    def check():
        torch.cuda.synchronize()
        k = Host(h.refs, 4)
        rows, after, _, bad = k.fork(table, lens, parents.tolist(), 8)
        assert not k.extend(rows, after, longer.tolist()) and not bad
        assert t2.tolist() == rows and l2.tolist() == after and ps.refs.tolist() == k.refs
        for a, b in pairs.tolist():
            assert a < 0 or torch.equal(pool[a], pool[b])

    def refill():
        p = [r.randrange(6) for _ in range(9)]
        parents.copy_(dev(p))
        longer.copy_(dev([min(lens[x] + r.randint(0, 5), 32) for x in p]))
        torch.cuda.synchronize()

    side = torch.cuda.Stream()
    refill()
    with torch.cuda.stream(side):
        torch.cuda._sleep(1000000)
    step(stream=side)
    check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        refill()
        graph.replay()
        check()


def test_pools_of_the_caches():
    """An index cache, latent records of both kinds: forked rows read the same keys and records."""
    nb, bs = 12, 32
    index = dsaidx.IndexCache.allocate(nb, bs, dsaidx.FP8)
    a, b = latent.LatentCache.allocate(nb, bs), latent.QuantLatentCache.allocate(nb, bs)
    g = torch.Generator(device="cuda").manual_seed(3)
    n = 70
    table, lens = dev([[7, 2, 9, -1]]), dev([n])
    i = torch.arange(n, device="cuda")
    slots = table[0].long()[i // bs] * bs + i % bs
    kv = torch.randn(n, 576, generator=g, device="cuda").bfloat16()
    dsaidx.store_keys(index, kv[:, :128].contiguous(), slots)
    for c in (a, b):
        latent.latent_append(c, kv[:, :512], kv[:, 512:], None, slots, None)
    ps = pages.PageSet.allocate(nb, bs, [index.pool, a.pool, b.pool])
    ps.refs[[7, 2, 9]] = 1
    ws = workspace(nb, 3)
    t2, l2, pairs = gpu_fork(ps, table, lens, [0, -1, 0], 4, ws)
    pages.copy(ps, pairs)
    assert t2.tolist() == [[7, 2, 0, -1], [-1] * 4, [7, 2, 1, -1]] and l2.tolist() == [70, 0, 70]
    for row in (0, 2):
        s2 = t2[row].long()[i // bs] * bs + i % bs
        assert torch.equal(a.pool.view(-1, 576)[s2], kv)
        one, two = torch.empty(n, 576, dtype=torch.bfloat16, device="cuda"), torch.empty(n, 576, dtype=torch.bfloat16, device="cuda")
        assert torch.equal(latent.latent_read(b, slots, one), latent.latent_read(b, s2, two))
        assert torch.equal(index.pool.view(nb, -1)[t2[row, 2].long()], index.pool.view(nb, -1)[9])
