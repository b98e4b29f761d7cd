"""The pages of the cache: growing, forking, freeing, compacting and copying,
against the definitions carried out one row at a time on the host."""
import random

import pytest
import torch

import diffusion_transformer_mlp_gb300 as fc2
from test_gpu_mxfp4_cache import make_cache

pytestmark = pytest.mark.gpu

NAMES = ("k_codes", "k_scales", "v_codes", "v_scales")


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Host:
    """refs, table and lens as lists, and each operation as it is defined."""

    def __init__(self, pages, page, rows, per_row):
        self.page, self.per_row = page, per_row
        self.refs, self.lens = [0] * pages, [0] * rows
        self.table = [[0] * per_row for _ in range(rows)]

    def held(self, n):
        return -(-n // self.page)

    def select(self, sources):
        old, lens = [r[:] for r in self.table], self.lens[:]
        for b, s in enumerate(sources):
            if s == b:
                continue
            for p in old[b][:self.held(lens[b])]:
                self.refs[p] -= 1
            n = lens[s] if 0 <= s < len(lens) else 0
            for i in range(self.held(n)):
                self.table[b][i] = old[s][i]
                self.refs[old[s][i]] += 1
            self.lens[b] = n

    def extend(self, counts, total):
        counts = [max(c, 0) for c in counts]
        rows = range(len(self.lens))
        into = {b: self.table[b][self.lens[b] // self.page] for b in rows if counts[b] and self.lens[b] % self.page}
        writers = {}
        for b in into:
            writers.setdefault(into[b], []).append(b)
        copies, need = {}, 0
        for b in rows:
            if b in into:
                mine = writers[into[b]]
                if self.refs[into[b]] > 1 and not (len(mine) == self.refs[into[b]] and min(mine) == b):
                    copies[b] = into[b]
            need += self.held(self.lens[b] + counts[b]) - self.held(self.lens[b]) + (b in copies)
        free = [i for i, r in enumerate(self.refs) if r == 0]
        fail = [-1] * total, [[-1, -1] for _ in rows]
        if sum(counts) > total or any(c and self.held(n + c) > self.per_row for n, c in zip(self.lens, counts)):
            return *fail, -1
        if need > len(free):
            return *fail, need - len(free)
        slots, pairs = [], []
        for b in rows:
            pairs.append([-1, -1])
            if b in copies:
                new = free.pop(0)
                pairs[b] = [copies[b], new]
                self.refs[copies[b]] -= 1
                self.refs[new] = 1
                self.table[b][self.lens[b] // self.page] = new
            for i in range(self.held(self.lens[b]), self.held(self.lens[b] + counts[b])):
                self.table[b][i] = free.pop(0)
                self.refs[self.table[b][i]] = 1
            for t in range(self.lens[b], self.lens[b] + counts[b]):
                slots.append(self.table[b][t // self.page] * self.page + t % self.page)
            self.lens[b] += counts[b]
        return slots + [-1] * (total - len(slots)), pairs, 0

    def compact(self):
        used = sum(r > 0 for r in self.refs)
        holes = [i for i in range(used) if self.refs[i] == 0]
        movers = [i for i in range(used, len(self.refs)) if self.refs[i] > 0]
        to = dict(zip(movers, holes))
        for a, b in to.items():
            self.refs[b], self.refs[a] = self.refs[a], 0
        for row, n in zip(self.table, self.lens):
            for i in range(self.held(n)):
                row[i] = to.get(row[i], row[i])
        return [[a, b] for a, b in to.items()] + [[-1, -1]] * (len(self.refs) // 2 - len(to)), used

    def check(self, dev):
        assert dev.refs.tolist() == self.refs
        assert dev.lens.tolist() == self.lens
        assert dev.table.tolist() == self.table
        count = [0] * len(self.refs)
        for row, n in zip(self.table, self.lens):
            for p in row[:self.held(n)]:
                count[p] += 1
        assert count == self.refs


def both(pages, page, rows, per_row):
    return Host(pages, page, rows, per_row), fc2.empty_mxfp4_pages(pages, page, rows, per_row)


def extend(host, dev, counts, total=None):
    total = sum(max(c, 0) for c in counts) if total is None else total
    slots, copies, missing = fc2.mxfp4_pages_extend(dev, i32(counts), total)
    want = host.extend(counts, total)
    assert (slots.tolist(), copies.tolist(), int(missing)) == want
    host.check(dev)
    return want[2], copies


def select(host, dev, sources):
    fc2.mxfp4_pages_select(dev, i32(sources))
    host.select(sources)
    host.check(dev)


@pytest.mark.parametrize("pages,page,rows,per_row", [(1, 16, 1, 1), (7, 16, 3, 2), (300, 16, 40, 12), (260, 64, 1, 300),
                                                     (5000, 256, 70, 90), (20000, 16, 1500, 20), (2000, 32, 9000, 3),
                                                     (6000, 16, 1024, 9), (6000, 16, 1025, 9), (3000, 16, 300, 400)])
def test_random_operations(pages, page, rows, per_row):
    rng = random.Random(pages + rows)
    host, dev = both(pages, page, rows, per_row)
    seen = set()
    for step in range(25 if rows < 1000 else 10):
        what = rng.choice(["grow", "grow", "grow", "one", "select", "free", "compact"])
        if what == "grow":
            room = max(1, pages * page // (2 * rows))
            counts = [rng.choice([0, -3, 1, rng.randint(0, 2 * room), rng.randint(0, page)]) for _ in range(rows)]
            seen.add(extend(host, dev, counts, rng.choice([None, None, 3, sum(max(c, 0) for c in counts) + 5]))[0] > 0)
        elif what == "one":
            extend(host, dev, [rng.choice([1, 1, 0]) for _ in range(rows)])
        elif what == "select":
            select(host, dev, [rng.choice([b, b, rng.randrange(rows), -1, rows + 3]) for b in range(rows)])
        elif what == "free":
            select(host, dev, [b if rng.random() < 0.5 else -1 for b in range(rows)])
        else:
            moves, used = fc2.mxfp4_pages_compact(dev)
            want = host.compact()
            assert moves.tolist() == want[0] and int(used) == want[1]
            host.check(dev)


def test_writers_of_a_shared_page():
    """Of all holders of a page that go on in it the first keeps it; a holder that
    does not makes all others copy."""
    host, dev = both(64, 16, 5, 4)
    extend(host, dev, [20, 0, 0, 0, 0])
    select(host, dev, [0, 0, 0, 3, 0])
    state = [t.clone() for t in (dev.refs, dev.table, dev.lens)]
    _, copies = extend(host, dev, [1, 1, 1, 0, 1])
    assert copies[:, 0].tolist() == [-1, 1, 1, -1, 1]
    host2, dev2 = both(64, 16, 5, 4)
    for t, s in zip((dev2.refs, dev2.table, dev2.lens), state):
        t.copy_(s)
    host2.refs, host2.table, host2.lens = (s.tolist() for s in state)
    _, copies = extend(host2, dev2, [0, 1, 3, 0, 40])
    assert copies[:, 0].tolist() == [-1, 1, 1, -1, 1]
    # a full last page is nobody's to write in
    host3, dev3 = both(64, 16, 2, 4)
    extend(host3, dev3, [32, 0])
    select(host3, dev3, [0, 0])
    _, copies = extend(host3, dev3, [1, 1])
    assert copies[:, 0].tolist() == [-1, -1]


def test_what_does_not_fit_changes_nothing():
    host, dev = both(10, 16, 3, 8)
    extend(host, dev, [30, 17, 0])
    assert extend(host, dev, [100, 16, 1])[0] == -1  # 130 tokens: nine pages in a row of eight
    assert extend(host, dev, [90, 16, 1])[0] == 2    # six, one and one of the six that are left
    assert extend(host, dev, [0, 0, 129])[0] == -1
    assert extend(host, dev, [1, 1, 1], 2)[0] == -1  # three tokens in two slots
    assert extend(host, dev, [0, 0, 96])[0] == 0     # the last six pages
    assert extend(host, dev, [2, 0, 0])[0] == 0      # room in the last page
    assert extend(host, dev, [1, 0, 0])[0] == 1


def test_long_prompts():
    """Slots by the second launch, table rows of many pages."""
    host, dev = both(9000, 16, 3, 4100)
    extend(host, dev, [40000, 0, 65000])
    extend(host, dev, [1, 33000, 600])


@pytest.mark.parametrize("page,heads,dim", [(16, 1, 64), (64, 8, 128), (256, 3, 256), (32, 5, 64)])
def test_copies(page, heads, dim):
    a, b = make_cache(40, page, heads, dim, 1), make_cache(25, page, heads, dim, 2)
    for dst, src, n in ((a, a, 12), (b, a, 24), (a, b, 20)):
        g = torch.Generator(device="cuda").manual_seed(n)
        rows = torch.randperm(len(dst.k_codes), generator=g, device="cuda")
        to = rows[:n]
        others = rows[n:] if dst is src else torch.arange(len(src.k_codes), device="cuda")
        src_at = others[torch.randint(0, len(others), (n,), generator=g, device="cuda")]
        pairs = torch.stack((src_at, to), 1).to(torch.int32)
        pairs[3, 0], pairs[4, 1], pairs[5, 0], pairs[6, 1] = -1, -1, len(src.k_codes), len(dst.k_codes)
        real = torch.ones(n, dtype=torch.bool)
        real[3:7] = False
        want = {}
        for name in NAMES:
            want[name] = getattr(dst, name).clone()
            want[name][to[real]] = getattr(src, name)[src_at[real]]
        fc2.mxfp4_cache_copy(dst, pairs, None if src is dst else src)
        for name in NAMES:
            assert torch.equal(getattr(dst, name), want[name]), name
    fc2.mxfp4_cache_copy(a, pairs[:0])
    many = torch.full((30000, 2), -1, dtype=torch.int32, device="cuda")
    many[29999] = i32([2, 3])
    fc2.mxfp4_cache_copy(a, many)
    assert torch.equal(a.k_codes[3], a.k_codes[2]) and torch.equal(a.v_scales[3], a.v_scales[2])


def test_copies_past_32_bits():
    """Pages behind 4 GB of codes."""
    c = fc2.empty_mxfp4_cache(2300, 256, 64, 256)
    assert c.k_codes.numel() > 1 << 32
    for name in NAMES:
        getattr(c, name)[2298] = torch.randint(0, 256, getattr(c, name)[0].shape, device="cuda", dtype=torch.uint8)
    fc2.mxfp4_cache_copy(c, i32([[2298, 2299], [2298, 0]]))
    for name in NAMES:
        t = getattr(c, name)
        assert torch.equal(t[2299], t[2298]) and torch.equal(t[0], t[2298]), name


def test_captured():
    """A captured step grows with the state it finds."""
    host, dev = both(200, 16, 4, 30)
    extend(host, dev, [20, 33, 0, 16])
    counts = i32([1, 2, 1, 0])
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        fc2.mxfp4_pages_select(dev, i32([0, 1, 2, 3]))
    torch.cuda.current_stream().wait_stream(stream)
    graph, sources = torch.cuda.CUDAGraph(), i32([0, 1, 2, 3])
    with torch.cuda.graph(graph):
        fc2.mxfp4_pages_select(dev, sources)
        slots, copies, missing = fc2.mxfp4_pages_extend(dev, counts, 5)
    for fork in ([0, 1, 2, 3], [0, 0, 2, 1], [0, 1, 2, 3]):
        sources.copy_(i32(fork))
        graph.replay()
        host.select(fork)
        assert (slots.tolist(), copies.tolist(), int(missing)) == host.extend([1, 2, 1, 0], 5)
        host.check(dev)


def test_rows_out_of_range_touch_nothing_else():
    """Lengths and ids outside their ranges: no access outside, the other rows right."""
    dev = fc2.empty_mxfp4_pages(8, 16, 3, 2)
    dev.lens.copy_(i32([-5, 1000, 3]))
    dev.table.copy_(i32([[-7, 99], [99, -1], [2, 0]]))
    dev.refs[2] = 1
    fc2.mxfp4_pages_select(dev, i32([1, 0, 2]))
    assert dev.refs.tolist() == [0, 0, 1, 0, 0, 0, 0, 0]
    fc2.mxfp4_pages_select(dev, i32([-1, -1, 2]))
    slots, copies, missing = fc2.mxfp4_pages_extend(dev, i32([1, 0, 1]), 2)
    assert slots.tolist() == [0, 2 * 16 + 3] and int(missing) == 0
    fc2.mxfp4_pages_compact(dev)


def test_refusals():
    p = fc2.empty_mxfp4_pages(8, 16, 3, 2)
    with pytest.raises(ValueError, match="sources"):
        fc2.mxfp4_pages_select(p, i32([0, 1]))
    with pytest.raises(ValueError, match="sources"):
        fc2.mxfp4_pages_select(p, i32([0, 1, 2]).long())
    with pytest.raises(ValueError, match="counts"):
        fc2.mxfp4_pages_extend(p, i32([0, 1]), 1)
    with pytest.raises(ValueError, match="total"):
        fc2.mxfp4_pages_extend(p, i32([0, 1, 2]), -1)
    for bad, match in ((fc2.MXFP4Pages(p.refs[:0], p.table, p.lens, 16), "must be pages"),
                       (fc2.MXFP4Pages(p.refs, p.table[:2], p.lens, 16), "row for each"),
                       (fc2.MXFP4Pages(p.refs.long(), p.table, p.lens, 16), "refs"),
                       (fc2.MXFP4Pages(p.refs, p.table.T, p.lens, 16), "table"),
                       (fc2.MXFP4Pages(p.refs, p.table.cpu(), p.lens, 16), "device")):
        with pytest.raises(ValueError, match=match):
            fc2.mxfp4_pages_compact(bad)
    with pytest.raises(fc2.NVFP4Error):
        fc2.mxfp4_pages_compact(fc2.MXFP4Pages(p.refs, p.table, p.lens, 24))
    a = make_cache(3, 16, 2, 64, 0)
    with pytest.raises(ValueError, match="pairs"):
        fc2.mxfp4_cache_copy(a, i32([0, 1]))
    with pytest.raises(ValueError, match="pairs"):
        fc2.mxfp4_cache_copy(a, i32([[0, 1, 2]]))
    for other in (make_cache(3, 32, 2, 64, 0), make_cache(3, 16, 1, 64, 0), make_cache(3, 16, 2, 128, 0)):
        with pytest.raises(fc2.NVFP4Error):
            fc2.mxfp4_cache_copy(a, i32([[0, 1]]), other)
