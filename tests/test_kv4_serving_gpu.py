"""The 4-bit cache as a server uses it: appends, attention and page operators one
after another, captured, on other streams, with tables that are out of bounds."""
import math

import pytest
import torch

import paged4_common as c4
from io_aware_exact_02_gb300 import build, fa

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return fa.load()


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Server:
    """A layer's cache, its tables and counts; what every row was appended."""

    def __init__(self, rows, pages, page, width, Hq, Hkv, d, seed):
        self.g = torch.Generator().manual_seed(seed)
        self.page, self.Hq, self.Hkv, self.d = page, Hq, Hkv, d
        self.pool = fa.kv4_pages(pages, Hkv, page, d)
        self.pool.fill_(255)
        self.table = torch.full((rows, width), 1 << 30, dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(rows, dtype=torch.int32, device="cuda")
        self.refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
        self.rope = fa.rope_table(width * page, d)
        self.k = [torch.zeros(0, Hkv, d, dtype=torch.float64) for _ in range(rows)]
        self.v = [x.clone() for x in self.k]

    def grow(self, rows, n):
        """n[i] more keys for rows[i], on the lowest free pages."""
        table, lens, refs = self.table.cpu(), self.lens.cpu(), self.refs.cpu()
        free = [p for p in range(len(refs)) if refs[p] == 0]
        for r, m in zip(rows, n):
            have = -(-int(lens[r]) // self.page)
            for j in range(have, -(-(int(lens[r]) + m) // self.page)):
                table[r, j] = free.pop(0)
                refs[table[r, j]] = 1
            lens[r] += m
        self.table.copy_(table)
        self.lens.copy_(lens)
        self.refs.copy_(refs)

    def step(self, rows, n):
        """Appends n[i] tokens to rows[i] and attends from them; checks all."""
        self.grow(rows, n)
        T = sum(n)
        qkv = torch.randn((T, self.Hq + 2 * self.Hkv, self.d), generator=self.g).to(torch.bfloat16)
        x = qkv.cuda()
        q, k, v = x.split([self.Hq, self.Hkv, self.Hkv], 1)
        cu = ints([sum(n[:i]) for i in range(len(n) + 1)])
        tables = self.table[rows].contiguous(), self.lens[rows].contiguous(), cu
        q = fa.kv4_append(k, v, self.pool, *tables, q=q, rope=self.rope)
        k_out = torch.empty((T, self.Hkv, self.d), dtype=torch.bfloat16, device="cuda")
        v_out = torch.empty_like(k_out)
        fa.kv4_read(self.pool, *tables, k_out, v_out)
        o, lse = fa.fwd_paged4(q, self.pool, *tables, max_q=max(n))
        fa.check_device_status()
        at = 0
        for r, m in zip(rows, n):
            self.k[r] = torch.cat([self.k[r], k_out[at:at + m].cpu().double()])
            self.v[r] = torch.cat([self.v[r], v_out[at:at + m].cpu().double()])
            ref = c4.reference(q[at:at + m].cpu(), self.k[r], self.v[r], True, self.d ** -0.5)
            c4.compare(o[at:at + m].cpu(), lse[at:at + m].cpu(), ref, (r, m))
            at += m


@pytest.mark.parametrize("Hq,Hkv,d,page", [(4, 2, 128, 16), (6, 1, 64, 32), (3, 3, 64, 16)])
def test_prompts_tokens_forks_and_compaction(Hq, Hkv, d, page):
    s = Server(7, 40, page, 10, Hq, Hkv, d, seed=2)
    s.step([0, 1], [75, 33])
    s.step([0, 1], [1, 1])
    # Row 2 and 3 continue what row 0 has, which goes on too: each on its own page.
    fa.pages_fork(ints([0, 0, 1]), ints([2, 3, 4]), s.table, s.lens, s.refs, [s.pool], page)
    for a, b in ((0, 2), (0, 3), (1, 4)):
        s.k[b], s.v[b] = s.k[a].clone(), s.v[a].clone()
    s.step([0, 2, 3, 4], [1, 1, 3, 2])
    s.step([2, 0, 1], [20, 1, 70])
    fa.pages_free(ints([0, 1]), s.table, s.lens, s.refs, page)
    for r in (0, 1):
        s.k[r], s.v[r] = s.k[r][:0], s.v[r][:0]
    live = fa.pages_compact(s.table, s.lens, s.refs, [s.pool], page)
    fa.check_device_status()
    n = live.item()
    assert (s.refs[:n] > 0).all() and (s.refs[n:] == 0).all()
    s.step([2, 3, 4], [1, 2, 1])
    s.step([5, 3], [40, 1])


@pytest.mark.parametrize("Hq,Hkv,d,page,lens,nq", [
    (17, 1, 64, 16, [300, 40], [90, 3]),       # whole tokens leave rows of a tile empty
    (128, 1, 128, 32, [140, 33, 7], [40, 1, 7]),
    (100, 1, 64, 16, [90], [60]),
    (14, 2, 128, 64, [1, 200, 130], [1, 150, 130]),
])
@pytest.mark.parametrize("causal", [True, False])
def test_prompts_of_many_heads_to_a_group(Hq, Hkv, d, page, lens, nq, causal):
    x = c4.Batch4(Hq, Hkv, d, page, lens, nq, seed=19)
    o, lse = fa.fwd_paged4(*x.args(), max_q=max(nq), causal=causal, out=x.out, lse=x.lse)
    fa.check_device_status()
    x.check(o, lse, causal, d ** -0.5)


def test_any_max_q_gives_the_results():
    for max_q in (1, 2, 5, 13, 90, 1000):
        x = c4.Batch4(4, 1, 64, 16, [100, 40, 95], [90, 10, 3], seed=3)
        o, lse = fa.fwd_paged4(*x.args(), max_q=max_q, out=x.out, lse=x.lse)
        fa.check_device_status()
        x.check(o, lse, True, 0.125)


@pytest.mark.parametrize("nq", [[1, 1, 1], [60, 2, 1]])
def test_queries_of_every_magnitude(nq):
    x = c4.Batch4(2, 1, 128, 16, [200, 64, 33], nq, seed=4)
    q = x.q_host.clone()
    q[0] *= 1e30
    q[nq[0]] *= 1e-30
    q[-1, 0, 3] = 0.0
    q[-1, 1] = 0.0
    x.q_host, scale = q, 1e-28
    x.q = q.cuda()
    o, lse = fa.fwd_paged4(*x.args(), max_q=max(nq), scale=scale, out=x.out, lse=x.lse)
    fa.check_device_status()
    x.check(o, lse, True, scale)


@pytest.mark.parametrize("nq", [[2, 3], [70, 3]])
def test_a_bad_query_spoils_its_own_row(nq):
    x = c4.Batch4(4, 1, 64, 16, [100, 40], nq, seed=5)
    good, lse_good = fa.fwd_paged4(*x.args(), max_q=max(nq))
    q = x.q.clone()
    q[1, 2, 5] = math.nan
    q[nq[0], 0, 7] = math.inf
    o, lse = fa.fwd_paged4(q, *x.args()[1:], max_q=max(nq))
    fa.check_device_status()
    bad = torch.zeros(x.T, 4, dtype=torch.bool)
    bad[1, 2] = bad[nq[0], 0] = True
    assert torch.isnan(o.cpu().float()[bad]).all() and torch.isnan(lse.cpu()[bad]).all()
    assert torch.equal(o.cpu()[~bad], good.cpu()[~bad])
    assert torch.equal(lse.cpu()[~bad], lse_good.cpu()[~bad])


@pytest.mark.parametrize("rows", [1, 4, 64])
@pytest.mark.parametrize("d", [64, 128])
def test_weak_keys_beside_a_loud_one(rows, d):
    # 127 keys of weight 2^-27 of the first one's, whose value is 0.  They are the
    # result: fp16's step of 2^-24, 7 binary orders lower, is 2^-4 of such a weight.
    k = torch.zeros((128, 1, d), dtype=torch.bfloat16, device="cuda")
    k[0, 0, 0] = 6.0
    v = torch.full_like(k, 6.0)
    v[0] = 0.0
    pool, table = fa.kv4_pages(8, 1, 16, d), torch.arange(8, dtype=torch.int32, device="cuda")[None]
    fa.kv4_append(k, v, pool, table, ints([128]), ints([0, 128]))
    q = torch.zeros((rows, 1, d), dtype=torch.bfloat16, device="cuda")
    q[:, 0, 0] = 1.0
    o, lse = fa.fwd_paged4(q, pool, table, ints([128]), ints([0, rows]), causal=False,
                           scale=27 * math.log(2) / 6)
    fa.check_device_status()
    want = 6 * 127 * 2.0 ** -27 / (1 + 127 * 2.0 ** -27)
    assert ((o.double() - want).abs() <= want * (2.0 ** -5 + 2.0 ** -8)).all(), (o.min(), o.max(), want)
    assert ((lse - 27 * math.log(2)).abs() < 1e-4).all()


def test_results_do_not_change_from_call_to_call():
    for nq in ([1] * 9, [50, 1, 1, 1, 1, 1, 1, 1, 1]):
        x = c4.Batch4(8, 2, 128, 16, [900, 300, 5, 128, 129, 700, 64, 33, 1000], nq, seed=6)
        first = [t.clone() for t in fa.fwd_paged4(*x.args(), max_q=max(nq), out=x.out, lse=x.lse)]
        for _ in range(5):
            again = fa.fwd_paged4(*x.args(), max_q=max(nq), out=x.out, lse=x.lse)
            assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


@pytest.mark.parametrize("Hq,Hkv,d,page,lens,nq", [
    (8, 1, 128, 16, [1000, 100, 333, 129], [129, 1, 300, 140]),
    (6, 2, 64, 32, [2000, 300, 77, 512], [360, 290, 5, 400]),
    (2, 2, 128, 128, [1100] + [5] * 70 + [1200], [1100] + [1] * 70 + [1025]),
])
@pytest.mark.parametrize("causal", [True, False])
def test_room_for_tiles_changes_no_result(Hq, Hkv, d, page, lens, nq, causal):
    x = c4.Batch4(Hq, Hkv, d, page, lens, nq, seed=17)
    sizes = x.T, len(lens), Hq, Hkv, d
    width = x.args()[2].shape[1]
    least = fa.fwd_paged4_workspace_size(*sizes, max(nq))
    best = fa.fwd_paged4_best_workspace_size(*sizes, page, width, max(nq))
    tile, bases = 128 * d * 4 * Hkv, -(-4 * len(lens) // 256) * 256
    assert best > least + bases and (best - least - bases) % tile == 0
    got = []
    for size in (least, best, least + bases + 8 * tile, least + bases - 1, best + 1000):
        ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")  # (NaN, whatever it is read as)
        o, lse = fa.fwd_paged4(*x.args(), max_q=max(nq), causal=causal, out=x.out, lse=x.lse,
                               workspace=ws)
        fa.check_device_status()
        got.append((o.clone(), lse.clone()))
        if size == least:
            x.check(o, lse, causal, d ** -0.5)
        if size == best:  # they were used
            assert not (ws[least + bases:least + bases + tile] == 255).all()
    for o, lse in got[1:]:
        assert torch.equal(o, got[0][0]) and torch.equal(lse, got[0][1])


def test_long_prompts_among_many_sequences():
    # (More sequences than a warp looks at together, the long ones anywhere among them.)
    lens, nq = [9] * 300, [1] * 300
    for b in (0, 3, 127, 128, 200, 299):
        lens[b], nq[b] = 150 + b, 130
    x = c4.Batch4(8, 1, 64, 16, lens, nq, seed=18)
    o, lse = fa.fwd_paged4(*x.args(), max_q=130, out=x.out, lse=x.lse)
    fa.check_device_status()
    x.check(o, lse, True, 0.125)


def test_captured_with_other_lengths_and_pages():
    """One graph of an append and an attention, replayed as the sequences grow."""
    s = Server(3, 30, 16, 8, 4, 2, 64, seed=7)
    s.step([0, 1, 2], [50, 3, 17])
    x = torch.zeros((3, 8, 64), dtype=torch.bfloat16, device="cuda")
    q, k, v = x.split([4, 2, 2], 1)
    table, lens, cu = s.table.clone(), s.lens.clone(), ints([0, 1, 2, 3])
    q_out = torch.zeros((3, 4, 64), dtype=torch.bfloat16, device="cuda")
    o, lse = torch.zeros_like(q_out), torch.zeros((3, 4), device="cuda")
    ws = torch.empty(fa.fwd_paged4_workspace_size(3, 3, 4, 2, 64, 1), dtype=torch.uint8, device="cuda")

    def run():
        fa.kv4_append(k, v, s.pool, table, lens, cu, q=q, q_out=q_out, rope=s.rope)
        fa.fwd_paged4(q_out, s.pool, table, lens, cu, max_q=1, out=o, lse=lse, workspace=ws)

    before = s.pool.clone()
    s.grow([0, 1, 2], [1, 1, 1])
    table.copy_(s.table), lens.copy_(s.lens)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    assert torch.equal(before, s.pool)
    for i in range(3):
        if i:
            s.grow([0, 1, 2], [1, 1, 1])
        table.copy_(s.table), lens.copy_(s.lens)
        x.copy_(torch.randn((3, 8, 64), generator=s.g).to(torch.bfloat16))
        graph.replay()
        fa.check_device_status()
        k_out = torch.empty((3, 2, 64), dtype=torch.bfloat16, device="cuda")
        v_out = torch.empty_like(k_out)
        fa.kv4_read(s.pool, table, lens, cu, k_out, v_out)
        for r in range(3):
            s.k[r] = torch.cat([s.k[r], k_out[r:r + 1].cpu().double()])
            s.v[r] = torch.cat([s.v[r], v_out[r:r + 1].cpu().double()])
            ref = c4.reference(q_out[r:r + 1].cpu(), s.k[r], s.v[r], True, 0.125)
            c4.compare(o[r:r + 1].cpu(), lse[r:r + 1].cpu(), ref, r)


def test_graphs_with_workspaces_of_their_own_run_together():
    xs = [c4.Batch4(8, 2, 128, 16, [700, 300, 900], nq, seed=8 + i)
          for i, nq in enumerate(([1, 1, 1], [60, 1, 5]))]
    graphs, outs = [], []
    for x in xs:
        m = max(x.nq)
        ws = torch.empty(fa.fwd_paged4_workspace_size(x.T, 3, 8, 2, 128, m), dtype=torch.uint8,
                         device="cuda")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(fa.fwd_paged4(*x.args(), max_q=m, out=x.out, lse=x.lse, workspace=ws))
        graphs.append((g, ws))
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    for _ in range(10):
        for (g, _), st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    fa.check_device_status()
    for x, (o, lse) in zip(xs, outs):
        x.check(o, lse, True, 128 ** -0.5)


def test_on_a_stream_of_its_own():
    st = torch.cuda.Stream()
    x = c4.Batch4(8, 2, 64, 32, [700, 300], [3, 100], seed=10)
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        o, lse = fa.fwd_paged4(*x.args(), max_q=100, out=x.out, lse=x.lse)
        code, site = fa.device_status()
    st.synchronize()
    assert (code, site) == (0, 0)
    x.check(o, lse, True, 0.125)


@pytest.mark.parametrize("nq,lens", [([1, 1, 1], [200, 64, 150]), ([100, 1, 80], [200, 64, 150]),
                                     ([600, 550, 5], [700, 600, 150])])
def test_tables_out_of_bounds_are_recorded(nq, lens):

    def call(change, site):
        x = c4.Batch4(4, 2, 64, 16, lens, nq, seed=11)
        change(x)
        o, lse = fa.fwd_paged4(*x.args(), max_q=max(nq), out=x.out, lse=x.lse)
        assert fa.device_status() == (fa.FA_ERR_PAGE, site)
        return x, o, lse

    def page(n):
        def f(x):
            x.table[1, 2] = n
        return f
    for n in (-1, 1 << 30, 10 ** 9):
        x, o, lse = call(page(n), 304)
        x.check(o, lse, True, 0.125, skip=(1,))
    for n in (-3, 10 ** 6):
        x, o, lse = call(lambda x: x.seq_lens.__setitem__(1, n), 302)
        x.check(o, lse, True, 0.125, skip=(1,))
    call(lambda x: x.cu_q.__setitem__(1, 10 ** 6), 301)
    call(lambda x: x.cu_q.__setitem__(2, -4), 301)


def test_append_and_read_tables_out_of_bounds():
    s = Server(2, 8, 16, 3, 2, 1, 64, seed=12)
    s.step([0, 1], [20, 17])
    k = torch.zeros((2, 1, 64), dtype=torch.bfloat16, device="cuda")
    cu = ints([0, 1, 2])
    before = s.pool.clone()
    for table, lens, site in (([[0, 99, 1], [2, 3, 4]], [21, 0], 303),
                              ([[0, 99, 1], [2, 3, 4]], [21, 49], 303),
                              ([[0, 99, 1], [2, -1, 4]], [21, 18], 304)):
        for call in (lambda *t: fa.kv4_append(k, k, s.pool, *t), lambda *t: fa.kv4_read(s.pool, *t, k, k)):
            call(ints(table), ints(lens), cu)
            code, got = fa.device_status()
            assert code == fa.FA_ERR_PAGE and got in (site, 304)
            assert torch.equal(s.pool, before)
    for bad in ([0, 3, 2], [-1, 1, 2], [0, 2, 1]):
        fa.kv4_append(k, k, s.pool, s.table, s.lens, ints(bad))
        assert fa.device_status()[0] == fa.FA_ERR_PAGE
        s.pool.copy_(before)


def test_rope_rows_are_checked():
    s = Server(1, 8, 16, 8, 2, 1, 64, seed=13)
    s.step([0], [20])
    k = torch.zeros((1, 1, 64), dtype=torch.bfloat16, device="cuda")
    before = s.pool.clone()
    fa.kv4_append(k, k, s.pool, s.table, ints([21]), ints([0, 1]), rope=s.rope[:20].contiguous())
    assert fa.device_status() == (fa.FA_ERR_PAGE, 303)
    assert torch.equal(s.pool, before)


def test_a_row_past_the_rotations_table_leaves_its_slot_alone():
    s = Server(1, 8, 16, 8, 2, 1, 64, seed=16)
    s.step([0], [20])
    k = torch.full((2, 1, 64), 6.0, dtype=torch.bfloat16, device="cuda")
    tables = s.table, ints([22]), ints([0, 2])
    s.pool.fill_(0x22)  # codes 1, scales 5/32
    fa.kv4_append(k, k, s.pool, *tables, rope=s.rope[:21].contiguous())
    assert fa.device_status() == (fa.FA_ERR_PAGE, 303)
    k_out, v_out = torch.zeros_like(k), torch.zeros_like(k)
    fa.kv4_read(s.pool, *tables, k_out, v_out)
    fa.check_device_status()
    assert (k_out[1] == 0.15625).all() and (v_out[1] == 0.15625).all()
    assert (v_out[0] == 6.0).all()


def test_pages_behind_four_gigabytes():
    """Block offsets that pass 32 bits, appended, read and attended."""
    Hkv, page, d = 8, 256, 128
    pages = (5 << 30) // (Hkv * page * 9 * d // 8)
    s = Server(1, 4, page, 3, Hkv, Hkv, d, seed=14)
    s.pool = torch.empty((pages, Hkv, page * 9 * d // 8), dtype=torch.uint8, device="cuda")
    s.pool[-3:] = 255
    s.refs = torch.ones(pages, dtype=torch.int32, device="cuda")
    s.refs[-2:] = 0
    s.step([0], [300])
    s.step([0], [1])
    assert s.table[0, :2].tolist() == [pages - 2, pages - 1]
    # ... and copied by the page operators
    fa.pages_copy(ints([pages - 1]), ints([pages - 3]), [s.pool])
    fa.check_device_status()
    assert torch.equal(s.pool[-1], s.pool[-3])


def test_binding_refuses_what_does_not_fit():
    x = c4.Batch4(4, 2, 64, 16, [40], [2], seed=15)
    q, pages, table, lens, cu = x.args()
    for args in ((q.float(), pages, table, lens, cu), (q, pages[:, :, :-1], table, lens, cu),
                 (q, pages.int(), table, lens, cu), (q, pages, table.long(), lens, cu),
                 (q, pages, table, lens[:0], cu), (q, pages, table, lens, cu[:1]),
                 (q[:, :, ::2], pages, table, lens, cu), (q, pages.transpose(0, 1), table, lens, cu),
                 (q.cpu(), pages, table, lens, cu), (q, pages, table, lens.cpu(), cu)):
        with pytest.raises(ValueError):
            fa.fwd_paged4(*args)
    with pytest.raises(ValueError):
        fa.fwd_paged4(*x.args(), out=torch.empty_like(x.out)[:, :1])
    with pytest.raises(ValueError):
        fa.kv4_append(q[:, :2], q[:, :2], pages, table, lens, cu, q_out=q)
    with pytest.raises(ValueError):
        fa.kv4_append(q[:, :1], q[:, :1], pages, table, lens, cu)
    with pytest.raises(fa.FaError):
        fa.fwd_paged4(*x.args(), k_scale=0.0)
    for pools in ([], pages.new_zeros(2, 0, 4), [pages.cpu()], [pages.transpose(0, 2)]):
        with pytest.raises(ValueError):
            fa.pages_copy(lens, lens, pools)
    with pytest.raises(fa.FaError):
        fa.pages_copy(lens, lens, pages.new_zeros(2, 4, 0))
    with pytest.raises(ValueError):
        fa.pages_fork(lens, lens[:0], table, lens, lens, [pages], 16)
    with pytest.raises(ValueError):
        fa.pages_fork(lens, lens, table, lens, torch.zeros(99, dtype=torch.int32, device="cuda"),
                      [pages], 16)


class Refuses:
    """An allocator that has no more than `most` bytes."""

    def __init__(self, alloc, most):
        self.alloc, self.most, self.asked = alloc, most, []

    def __call__(self, size, stream):
        self.asked.append(size)
        if size > self.most:
            raise torch.OutOfMemoryError("no room")
        return self.alloc(size, stream)


def test_without_room_for_tiles_a_call_takes_the_least_workspace(monkeypatch):
    x = c4.Batch4(8, 1, 64, 16, [1000, 70], [300, 1], seed=20)
    sizes = x.T, 2, 8, 1, 64
    least = fa.fwd_paged4_workspace_size(*sizes, 300)
    best = fa.fwd_paged4_best_workspace_size(*sizes, 16, x.table.shape[1], 300)
    assert best > least
    want = [t.clone() for t in fa.fwd_paged4(*x.args(), max_q=300)]
    alloc = torch._C._cuda_cudaCachingAllocator_raw_alloc
    for most in (best - 1, least):
        refuses = Refuses(alloc, most)
        monkeypatch.setattr(torch._C, "_cuda_cudaCachingAllocator_raw_alloc", refuses)
        got = fa.fwd_paged4(*x.args(), max_q=300)
        fa.check_device_status()
        assert refuses.asked == [best, least]
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    monkeypatch.setattr(torch._C, "_cuda_cudaCachingAllocator_raw_alloc", Refuses(alloc, least - 1))
    with pytest.raises(torch.OutOfMemoryError):
        fa.fwd_paged4(*x.args(), max_q=300)


def test_a_full_allocator_still_serves_long_prompts():
    # (Torch's own limit on what a process may hold, in place of a full GPU.)
    x = c4.Batch4(32, 8, 128, 16, [300], [300], seed=21, width=8192)
    sizes = x.T, 1, 32, 8, 128
    least = fa.fwd_paged4_workspace_size(*sizes, 300)
    best = fa.fwd_paged4_best_workspace_size(*sizes, 16, 8192, 300)
    assert best - least > 500 << 20
    want = [t.clone() for t in fa.fwd_paged4(*x.args(), max_q=300, out=x.out, lse=x.lse)]
    x.check(*want, True, 128 ** -0.5)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    total = torch.cuda.get_device_properties(0).total_memory
    limit = torch.cuda.memory_reserved() + least + (128 << 20)
    torch.cuda.set_per_process_memory_fraction(limit / total)
    try:
        got = fa.fwd_paged4(*x.args(), max_q=300, out=x.out, lse=x.lse)
    finally:
        torch.cuda.set_per_process_memory_fraction(1.0)
    fa.check_device_status()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("nq", [60, 330])
@pytest.mark.parametrize("best", [False, True])
def test_appends_and_attentions_back_to_back(nq, best):
    """The same slots written anew and attended, one call after another without a wait:
    what each attention saw is what the append before it wrote."""
    page, L, B, Hq, Hkv, d = 16, 700, 3, 8, 2, 64
    s = Server(B, 150, page, 48, Hq, Hkv, d, seed=22)
    s.grow([0, 1, 2], [L, L - 1, L - 13])
    s.pool.fill_(0x22)
    sizes = B * nq, B, Hq, Hkv, d
    size = (fa.fwd_paged4_best_workspace_size(*sizes, page, 48, nq) if best
            else fa.fwd_paged4_workspace_size(*sizes, nq))
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    cu = ints([b * nq for b in range(B + 1)])
    x = torch.randn((6, B * nq, Hq + 2 * Hkv, d), generator=s.g).to(torch.bfloat16).cuda()
    o = torch.zeros((2, 6, B * nq, Hq, d), dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros((2, 6, B * nq, Hq), device="cuda")
    q_out = torch.empty((B * nq, Hq, d), dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    for waits in (0, 1):
        for i in range(6):
            q, k, v = x[i].split([Hq, Hkv, Hkv], 1)
            fa.kv4_append(k, v, s.pool, s.table, s.lens, cu, q=q, q_out=q_out, rope=s.rope)
            if waits:
                torch.cuda.synchronize()
            fa.fwd_paged4(q_out, s.pool, s.table, s.lens, cu, max_q=nq, out=o[waits, i],
                          lse=lse[waits, i], workspace=ws)
            if waits:
                torch.cuda.synchronize()
    fa.check_device_status()
    assert torch.equal(o[0], o[1]) and torch.equal(lse[0], lse[1])
    assert not torch.equal(o[0, 0], o[0, 1])
