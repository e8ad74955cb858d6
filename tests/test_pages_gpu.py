"""Forking, freeing, copying and compacting the pages of a cache on the GPU,
against the same written with lists."""
import random

import pytest
import torch

from io_aware_exact_02_gb300 import build, fa

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return fa.load()


class Book:
    """Tables of `rows` rows over `pages` pages; rows of lens[r] keys."""

    def __init__(self, lens, rows, pages, page, width, seed, share=True):
        rng = random.Random(seed)
        self.page, self.pages, self.width = page, pages, width
        self.table = [[-5] * width for _ in range(rows)]
        self.lens = list(lens) + [0] * (rows - len(lens))
        self.refs = [0] * pages
        ids = rng.sample(range(pages), sum(-(-n // page) for n in lens))
        for r, n in enumerate(lens):
            for j in range(-(-n // page)):
                self.table[r][j] = ids.pop()
            if share and r % 3 == 2:
                for j in range(min(self.lens[r - 1], n) // page // 2):
                    self.table[r][j] = self.table[r - 1][j]
            for j in range(-(-n // page)):
                self.refs[self.table[r][j]] += 1

    def tensors(self):
        put = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        return put(self.table), put(self.lens), put(self.refs)

    def check(self, table, lens, refs):
        assert lens.tolist() == self.lens
        assert refs.tolist() == self.refs
        assert table.tolist() == self.table

    def fork(self, parents, children, pools):
        free = [p for p in range(self.pages) if self.refs[p] == 0]
        for a, b in zip(parents, children):
            n = self.lens[a]
            for j in range(n // self.page):
                self.table[b][j] = self.table[a][j]
                self.refs[self.table[a][j]] += 1
            if n % self.page:
                new = free.pop(0)
                self.table[b][n // self.page] = new
                self.refs[new] = 1
                for t in pools:
                    t[new] = t[self.table[a][n // self.page]]
            self.lens[b] = n

    def free(self, rows):
        for r in rows:
            for j in range(-(-self.lens[r] // self.page)):
                self.refs[self.table[r][j]] -= 1
            self.lens[r] = 0

    def compact(self, pools):
        live = sum(x != 0 for x in self.refs)
        holes = [p for p in range(live) if self.refs[p] == 0]
        high = [p for p in range(self.pages - 1, live - 1, -1) if self.refs[p]]
        assert len(holes) == len(high)
        to = dict(zip(high, holes))
        for a, b in to.items():
            self.refs[b], self.refs[a] = self.refs[a], 0
            for t in pools:
                t[b] = t[a]
        for r, n in enumerate(self.lens):
            for j in range(-(-n // self.page)):
                self.table[r][j] = to.get(self.table[r][j], self.table[r][j])
        return live


def pools_of(pages, kind, seed):
    g = torch.Generator().manual_seed(seed)
    byte = lambda *s: torch.randint(0, 256, s, generator=g, dtype=torch.uint8)  # noqa: E731
    if kind == "stack":
        t = byte(3, pages, 2, 16, 64)
        return t, list(t.unbind(0))
    if kind == "list":  # of other sizes, one above a chunk
        t = [byte(pages, 16), byte(pages, 2, 16, 144), byte(pages, 40000), byte(pages, 16, 3)]
        return t, t
    return [], []


def to_gpu(p):
    return p.cuda() if isinstance(p, torch.Tensor) else [t.cuda() for t in p]


def same(gpu, host):
    got = gpu if isinstance(gpu, torch.Tensor) else list(gpu)
    for a, b in zip(got, host):
        assert torch.equal(a.cpu(), b)


@pytest.mark.parametrize("kind", ["stack", "list", "none"])
@pytest.mark.parametrize("lens,kids,pages,page", [
    ([1], 1, 4, 16), ([16], 3, 9, 16), ([17, 5, 64, 100], 2, 40, 16),
    ([300, 256, 255, 257, 1, 33, 64], 4, 120, 64)])
def test_fork_and_free(lens, kids, pages, page, kind):
    rows = len(lens) * (kids + 1) + 1
    width = max(-(-n // page) for n in lens) + 1
    b = Book(lens, rows, pages, page, width, seed=1)
    t = b.tensors()
    given, host = pools_of(pages, kind, 2)
    dev = to_gpu(given)
    rng = random.Random(3)
    parents = [r for r in range(len(lens)) for _ in range(kids)]
    children = rng.sample(range(len(lens), rows), len(parents))
    put = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    fa.pages_fork(put(parents), put(children), *t, dev, page)
    fa.check_device_status()
    b.fork(parents, children, host)
    b.check(*t)
    same(dev, host)
    gone = rng.sample(range(rows), rows // 2)
    fa.pages_free(put(gone + gone[:1]), *t, page)  # (one of them twice)
    fa.check_device_status()
    b.free(gone)
    b.check(*t)
    live = fa.pages_compact(*t, dev, page)
    fa.check_device_status()
    assert live.item() == b.compact(host)
    b.check(*t)
    same(dev, host)


@pytest.mark.parametrize("pages", [1, 5, 1023, 4096, 4097, 20000])
@pytest.mark.parametrize("used", [0.0, 0.03, 0.5, 0.97, 1.0])
def test_compact_pools(pages, used):
    n = int(pages * used)
    lens = [16] * n
    b = Book(lens, max(n, 1), pages, 16, 1, seed=pages, share=False)
    t = b.tensors()
    host = [torch.randint(0, 1 << 30, (pages, 4), dtype=torch.int32)]
    dev = to_gpu(host)
    live = fa.pages_compact(*t, dev, 16)
    fa.check_device_status()
    assert live.item() == b.compact(host) == n
    b.check(*t)
    same(dev, host)
    fa.pages_compact(*t, dev, 16)  # nothing to move
    b.check(*t)
    same(dev, host)


def test_fork_many_children_over_many_ranges():
    b = Book([33] * 1500, 4600, 9000, 16, 4, seed=4, share=False)
    t = b.tensors()
    host = [torch.randint(0, 1 << 30, (9000, 4), dtype=torch.int32)]
    dev = to_gpu(host)
    parents, children = [i % 1500 for i in range(3000)], list(range(1500, 4500))
    put = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    fa.pages_fork(put(parents), put(children), *t, dev, 16)
    fa.check_device_status()
    b.fork(parents, children, host)
    b.check(*t)
    same(dev, host)


def test_copy():
    for kind in ("stack", "list"):
        given, host = pools_of(30, kind, 5)
        dev = to_gpu(given)
        src, dst = [0, 3, 29, 3], [5, 6, 7, 28]
        put = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        fa.pages_copy(put(src), put(dst), dev)
        fa.check_device_status()
        for t in host:
            t[dst] = t[src]
        same(dev, host)


def status():
    code, site = fa.device_status()
    return code, site


def test_what_is_left_out():
    put = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    b = Book([20, 40], 6, 8, 16, 4, seed=6, share=False)
    t = b.tensors()
    # no free page for the second and third of three children
    taken = [p for p in range(8) if b.refs[p] == 0][1:]
    t[2][taken] = 1
    for p in taken:
        b.refs[p] = 1
    fa.pages_fork(put([0, 1, 0]), put([2, 3, 4]), *t, [], 16)
    assert status() == (fa.FA_ERR_PAGE, 306)
    b.fork([0], [2], [])
    b.check(*t)
    # a row out of the table, a row as its own child, a child that holds keys
    for a, c in ((9, 3), (0, -1), (0, 0), (1, 2)):
        fa.pages_fork(put([a]), put([c]), *t, [], 16)
        assert status() == (fa.FA_ERR_PAGE, 305)
        b.check(*t)
    fa.pages_free(put([6, -1]), *t, 16)
    assert status() == (fa.FA_ERR_PAGE, 305)
    b.check(*t)
    # a child listed twice is made once
    for p in taken:
        t[2][p] = b.refs[p] = 0
    fa.pages_fork(put([0, 0]), put([5, 5]), *t, [], 16)
    assert status() == (fa.FA_ERR_PAGE, 305)
    assert t[1].tolist() == [20, 40, 20, 0, 0, 20]
    assert t[2].sum().item() == sum(b.refs) + 2
    # a page number outside the pool, and a page that nobody counted
    x = Book([32], 2, 4, 16, 4, seed=7)
    t = x.tensors()
    t[0][0, 0] = 4
    fa.pages_free(put([0]), *t, 16)
    assert status() == (fa.FA_ERR_PAGE, 304)
    y = Book([32], 2, 4, 16, 4, seed=7)
    t = y.tensors()
    t[2].zero_()
    fa.pages_free(put([0]), *t, 16)
    assert status() == (fa.FA_ERR_PAGE, 307)
    assert t[2].tolist() == [0] * 4 and t[1].tolist() == [0, 0]
    fa.pages_copy(put([0, 9]), put([1, 2]), torch.zeros(1, 4, 16, dtype=torch.uint8, device="cuda"))
    assert status() == (fa.FA_ERR_PAGE, 304)


@pytest.mark.parametrize("pages,given", [(60, True), (60, False), (9000, True)])
def test_captured_and_replayed(pages, given):
    # A fork, a release and a compaction in one graph, replayed on other tables.
    width, rows, page = 12, 8, 16
    gpu_pools = torch.zeros((2, pages, 2, 144), dtype=torch.uint8, device="cuda")
    book = Book([33, 16, 100], rows, pages, page, width, 3)
    table, lens, refs = book.tensors()
    parents, children = (torch.tensor(x, dtype=torch.int32, device="cuda")
                         for x in ([0, 2, 0], [3, 4, 5]))
    gone = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    live = torch.zeros(1, dtype=torch.int32, device="cuda")
    need = (fa.pages_fork_workspace_size(pages, 3), fa.pages_compact_workspace_size(pages))
    ws = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") if given else None for n in need]
    graph = torch.cuda.CUDAGraph()
    stream = torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=stream):
        fa.pages_fork(parents, children, table, lens, refs, gpu_pools, page, workspace=ws[0])
        fa.pages_free(gone, table, lens, refs, page)
        fa.pages_compact(table, lens, refs, gpu_pools, page, live=live, workspace=ws[1])
    for seed, start in enumerate(([33, 16, 100], [7, 64, 150], [0, 1, 32], [190, 191, 192])):
        book = Book(start, rows, pages, page, width, seed)
        host = torch.randint(0, 256, gpu_pools.shape, dtype=torch.uint8,
                             generator=torch.Generator().manual_seed(seed))
        gpu_pools.copy_(host)
        for a, b in zip((table, lens, refs), book.tensors()):
            a.copy_(b)
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            graph.replay()
        stream.synchronize()
        fa.check_device_status()
        pools = list(host.unbind(0))
        book.fork([0, 2, 0], [3, 4, 5], pools)
        book.free([0, 1])
        assert live.item() == book.compact(pools)
        book.check(table, lens, refs)
        for t, p in zip(gpu_pools.cpu(), pools):
            held = torch.tensor(book.refs) > 0
            assert torch.equal(t[held], p[held])


@pytest.mark.parametrize("bad", [-1, -(1 << 31), 4 * 16 + 1, (1 << 31) - 1])
def test_a_row_of_bad_length_is_left_as_it_is(bad):
    put = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    b = Book([20, 40, 64, 1], 5, 12, 16, 4, seed=8, share=False)
    t = b.tensors()
    t[1][1] = bad
    fa.pages_free(put([1, 2, 1, 2, 4]), *t, 16)  # (2 twice, 4 empty)
    assert status() == (fa.FA_ERR_PAGE, 302)
    b.free([2])
    b.lens[1] = bad
    b.check(*t)
