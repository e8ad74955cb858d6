"""The paged key/value cache on the GPU: fa_kv_append, fa_fwd_paged and
fa_fwd_paged_prefix through the binding, against fp64 results with elementwise
rounding bounds.  Every slot outside the sequences holds NaN or infinities."""
import math

import pytest
import torch

from io_aware_exact_02_gb300 import build, fa
from paged_common import BF16, FP32, Batch, compare, reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return fa.load()


def attend(x, causal=True, scale=None, prefix=False, max_q=None):
    scale = 1 / math.sqrt(x.d) if scale is None else scale
    kw = dict(max_q=max(x.nq) if max_q is None else max_q, causal=causal, scale=scale, out=x.out,
              lse=x.lse)
    if prefix:
        o, lse = fa.fwd_paged_prefix(*x.args(), x.prefix_pages, **kw)
    else:
        o, lse = fa.fwd_paged(*x.args(), **kw)
    fa.check_device_status()
    x.check(o, lse, causal, scale)
    return o, lse


CASES = [
    # Hq, Hkv, d, page, lens, nq
    (8, 2, 128, 16, [1], [1]),
    (8, 2, 64, 16, [1, 2, 17], [1, 1, 1]),
    (8, 8, 128, 16, [127, 128, 129, 300], [1, 1, 1, 1]),
    (16, 1, 128, 32, [1000, 5], [1, 1]),
    (6, 2, 128, 64, [700, 64, 65], [1, 3, 2]),
    (10, 2, 64, 128, [513, 130], [4, 1]),
    (14, 2, 64, 256, [300, 900, 256], [1, 2, 5]),
    (8, 2, 128, 16, [0, 40, 0, 33], [0, 1, 0, 1]),
    (8, 2, 128, 16, [40, 50, 60], [0, 1, 0]),
    (4, 2, 128, 16, [3, 2], [5, 4]),               # rows before position 0 see no key
    (4, 4, 64, 16, [200, 77, 300], [200, 77, 129]),  # prompts
    (32, 4, 128, 32, [333, 700], [333, 100]),
    (12, 4, 128, 128, [400, 260, 129], [150, 1, 64]),
    (128, 1, 64, 16, [290, 31], [3, 1]),           # 128 query heads on one key head
    (48, 1, 128, 16, [520], [9]),
    (5, 5, 64, 16, list(range(1, 41)), [1] * 40),  # more sequences than a warp
    (8, 1, 64, 16, [60 + 13 * i for i in range(70)], [1 + i % 3 for i in range(70)]),
    # long and short sequences in one call
    (8, 2, 128, 16, [300, 17, 0, 600, 400] + [90 + i for i in range(9)], [90, 1, 0, 1, 150] + [1] * 9),
    (16, 2, 64, 64, [400] * 20, [1, 2, 3, 40] * 5),
    (40, 1, 64, 32, [333, 100, 40, 9], [1, 30, 2, 1]),
    (96, 1, 128, 16, [333, 100, 40], [1, 30, 1]),
    # more sequences than a CTA has threads
    (2, 1, 64, 16, [1 + (7 * i) % 150 for i in range(900)], [1] * 900),
    (2, 2, 64, 16, [1 + (7 * i) % 150 for i in range(450)], [i % 2 for i in range(450)]),
]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_paged_matches_fp64(case, causal):
    Hq, Hkv, d, page, lens, nq = CASES[case]
    attend(Batch(Hq, Hkv, d, page, lens, nq, seed=case, pad=case % 3), causal)


@pytest.mark.parametrize("max_q", [1, 8, 100])
def test_max_q_is_only_a_hint(max_q):
    x = Batch(8, 2, 128, 32, [300, 90, 200], [40, 1, 9], seed=5)
    attend(x, max_q=max_q)


@pytest.mark.parametrize("nq", [[1, 1], [70, 3]])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("scale", [0.0, -0.2, 1.0])
def test_scales(d, nq, scale):
    attend(Batch(8, 2, d, 16, [150, 333], nq, seed=d + len(nq)), scale=scale)


@pytest.mark.parametrize("nq", [[1, 1, 2], [130, 40, 9]])
def test_growing_scores_move_the_running_maximum(nq):
    # Scores that grow along the keys by far more than the softmax's slack.
    x = Batch(8, 2, 128, 16, [1200, 640, 300], nq, seed=11)
    for b, k in enumerate(x.keys):
        k *= torch.linspace(0.1, 12, k.shape[0])[:, None, None].to(k.dtype)
        for i, pg in enumerate(x.table[b].tolist()[:-(-x.lens[b] // 16)]):
            n = min(16, x.lens[b] - 16 * i)
            x.k_pages[pg, :, :n] = k[16 * i:16 * i + n].transpose(0, 1).to(x.k_pages.device)
    attend(x)


@pytest.mark.parametrize("G,nq", [(4, [1, 1, 1]), (4, [3, 300, 1]), (1, [33, 2, 64])])
def test_fused_projection_slices(G, nq):
    x = Batch(2 * G, 2, 128, 16, [500, 400, 129], nq, seed=3, fused=True, pad=2)
    assert x.q.stride(0) == (2 * G + 4) * 128
    attend(x)


@pytest.mark.parametrize("d,Hq,Hkv,page,nq", [(128, 8, 4, 16, 1), (64, 8, 8, 32, 3), (128, 32, 2, 64, 2),
                                             (128, 12, 1, 16, 5), (64, 4, 4, 16, 30)])
def test_many_ragged_units_per_cta_are_right_and_repeatable(d, Hq, Hkv, page, nq):
    """Hundreds of units of one to a dozen key tiles, so that every CTA goes
    through many: against fp64 once, then bitwise the same every time."""
    lens = [1 + (i * i * 37 + 11 * i) % 1500 for i in range(150)]
    x = Batch(Hq, Hkv, d, page, lens, [min(n, nq) for n in lens], seed=nq)
    o, lse = attend(x)
    o, lse = o.clone(), lse.clone()
    for _ in range(30):
        a, b = fa.fwd_paged(*x.args(), max_q=nq, out=x.out, lse=x.lse)
        assert torch.equal(a, o) and torch.equal(b, lse)
    fa.check_device_status()


def test_long_sequence_decode():
    attend(Batch(8, 2, 128, 64, [20000, 3], [1, 1], seed=1))
    attend(Batch(4, 1, 64, 16, [30001], [2], seed=2))


PREFIX = [
    # Hq, Hkv, d, page, prefix, lens, nq
    (8, 2, 128, 16, 16, [17, 40], [1, 1]),
    (8, 2, 128, 16, 320, [321 + 7 * i for i in range(20)], [1] * 20),
    (6, 2, 64, 64, 640, [700, 641, 900], [2, 1, 3]),
    (4, 4, 64, 256, 256, [300, 300], [1, 44]),
    (8, 1, 128, 32, 1056, [1056 + i for i in range(1, 60)], [1] * 59),
    (4, 1, 128, 16, 2000, [2100, 2001, 2300, 2050], [60, 1, 200, 50]),
    (8, 2, 64, 16, 160, [161, 0, 200], [1, 0, 1]),     # an empty sequence
    (8, 2, 128, 16, 320, [400, 321, 330, 500, 322, 390], [60, 1, 1, 1, 2, 1]),  # long and short
    (8, 2, 128, 16, 160, [161, 100, 160, 30], [1, 4, 1, 2]),  # shorter than the prefix
]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("case", range(len(PREFIX)))
def test_prefix_matches_fp64(case, causal):
    Hq, Hkv, d, page, prefix, lens, nq = PREFIX[case]
    attend(Batch(Hq, Hkv, d, page, lens, nq, seed=case, pad=case % 2, prefix=prefix), causal,
           prefix=True)


def test_prefix_does_not_read_the_tables_part():
    x = Batch(8, 2, 128, 16, [200, 170, 300], [1, 2, 1], seed=9, prefix=160)
    x.table[:, :10] = -5
    attend(x, prefix=True)


# ------------------------------------------------------------------ append

def rotated(x, table, pos, interleaved):
    """fp64 rotation and the bound of a correct kernel's error."""
    x = x.double()
    if table is None:
        return x, torch.zeros_like(x)
    r = table.shape[1]
    c, s = table[pos, :r // 2].double()[:, None], table[pos, r // 2:].double()[:, None]
    i = torch.arange(r // 2) * 2 if interleaved else torch.arange(r // 2)
    j = i + 1 if interleaved else i + r // 2
    y, size = x.clone(), torch.zeros_like(x)
    y[..., i], y[..., j] = x[..., i] * c - x[..., j] * s, x[..., i] * s + x[..., j] * c
    size[..., i] = (x[..., i] * c).abs() + (x[..., j] * s).abs()
    size[..., j] = (x[..., i] * s).abs() + (x[..., j] * c).abs()
    # two products, a sum, and the rounding to bf16
    return y, torch.where(size > 0, BF16 * y.abs() + 4 * FP32 * size, 0.0)


APPEND = [
    # Hq, Hkv, d, page, lens, nq, rope_dim, interleaved, fused
    (8, 2, 128, 16, [1], [1], 128, False, False),
    (32, 8, 128, 16, [1000], [1], 128, False, True),
    (8, 2, 128, 64, [100, 65, 64, 200], [1, 1, 1, 1], 128, True, True),
    (6, 3, 64, 32, [40, 33, 70], [40, 2, 7], 64, False, False),
    (12, 12, 64, 256, [300, 12], [299, 12], 32, True, True),
    (4, 1, 128, 128, [129, 140], [2, 130], 48, False, True),
    (4, 4, 128, 16, [33, 18], [4, 18], 16, True, False),
    (4, 2, 64, 16, [50, 0, 20], [3, 0, 1], 0, False, True),
    (5, 1, 64, 16, [3 + i for i in range(100)], [1 + i % 3 for i in range(100)], 64, False, False),
    (0, 4, 128, 16, [77, 20], [30, 1], 128, False, False),   # keys and values alone
]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("case", range(len(APPEND)))
def test_append_matches_fp64(case, in_place):
    Hq, Hkv, d, page, lens, nq, rd, inter, fused = APPEND[case]
    x = Batch(max(Hq, 1), Hkv, d, page, lens, nq, seed=case)
    g = torch.Generator().manual_seed(case)
    T = x.cu[-1] + 3  # three padding rows
    qkv = torch.randn(T, Hq + 2 * Hkv, d, generator=g).to(torch.bfloat16)
    dev = qkv.cuda()
    q, k, v = dev[:, :Hq], dev[:, Hq:Hq + Hkv], dev[:, Hq + Hkv:]
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    table = fa.rope_table(max(lens), rd).cpu() if rd else None
    q_in = None if Hq == 0 else q
    q_out = None if Hq == 0 else (q if in_place else torch.full((T, Hq, d), 7.0, dtype=q.dtype, device="cuda"))
    kp, vp = x.k_pages.clone(), x.v_pages.clone()
    got = fa.kv_append(k, v, kp, vp, x.table, x.seq_lens, x.cu_q, q=q_in, q_out=q_out,
                       rope=None if table is None else table.cuda(), interleaved=inter)
    fa.check_device_status()
    qh, kh, vh = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    want_k, want_v = x.k_pages.cpu(), x.v_pages.cpu()
    got_k, got_v = kp.cpu(), vp.cpu()
    tab = x.table.cpu()
    for b in range(x.B):
        rows = slice(x.cu[b], x.cu[b + 1])
        pos = torch.arange(lens[b] - nq[b], lens[b])
        if nq[b] == 0:
            continue
        pages, slots = tab[b].long()[pos // page], pos % page
        want, bound = rotated(kh[rows], table, pos, inter)
        have = got_k[pages, :, slots].double()
        assert ((have - want).abs() <= bound).all()
        assert torch.equal(got_v[pages, :, slots], vh[rows])
        want_k[pages, :, slots] = got_k[pages, :, slots]
        want_v[pages, :, slots] = got_v[pages, :, slots]
        if Hq:
            want, bound = rotated(qh[rows], table, pos, inter)
            assert ((got[rows].cpu().double() - want).abs() <= bound).all()
    # every other slot, and the padding rows, as they were
    assert torch.equal(got_k.view(torch.int16), want_k.view(torch.int16))
    assert torch.equal(got_v.view(torch.int16), want_v.view(torch.int16))
    if Hq:
        keep = qh[x.cu[-1]:] if in_place else torch.full((3, Hq, d), 7.0, dtype=q.dtype)
        assert torch.equal(got[x.cu[-1]:].cpu(), keep)


def test_append_positions_far_out():
    # Positions past 2^17 and their pages; the table's rows are what count.
    L, page = 200_001, 256
    width = -(-L // page)
    kp = torch.zeros(width, 1, page, 64, dtype=torch.bfloat16, device="cuda")
    vp = torch.zeros_like(kp)
    k = torch.randn(2, 1, 64, device="cuda").to(torch.bfloat16)
    table = fa.rope_table(L, 64, base=500000.0)
    ids = torch.arange(width, dtype=torch.int32, device="cuda").flip(0)[None].contiguous()
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    fa.kv_append(k, k, kp, vp, ids, i32(L), i32(0, 2), rope=table)
    fa.check_device_status()
    pos = torch.tensor([L - 2, L - 1])
    want, bound = rotated(k.cpu(), table.cpu(), pos, False)
    have = kp[ids[0].cpu().long()[pos // page], :, pos % page].cpu().double()
    assert ((have - want).abs() <= bound).all()


# ------------------------------------------------------ tables out of bounds

def status():
    code, site = fa.device_status()
    return code, site


def test_bad_tables_are_reported_and_nothing_is_written_through_them():
    x = Batch(4, 2, 128, 16, [40, 30, 50], [1, 1, 1], seed=2)
    k = torch.ones(3, 2, 128, dtype=torch.bfloat16, device="cuda")
    before = x.k_pages.view(torch.int16).clone()
    good_rows = lambda kp: kp[int(x.table[0, 39 // 16]), :, 39 % 16]  # noqa: E731

    def run(site, table=x.table, lens=x.seq_lens, cu=x.cu_q, rope=None, attend_site=None):
        kp, vp = x.k_pages.clone(), x.v_pages.clone()
        fa.kv_append(k, k, kp, vp, table, lens, cu, rope=rope)
        if site is None:
            assert status() == (fa.FA_OK, 0)
        else:
            assert status() == (fa.FA_ERR_PAGE, site)
            assert torch.all(good_rows(vp) == 1)  # sequence 0 is sound
            assert (kp.view(torch.int16) != before).sum() <= 2 * 2 * 128
        if attend_site is not None:
            fa.fwd_paged(x.q, x.k_pages, x.v_pages, table, lens, cu, max_q=1)
            assert status() == (fa.FA_ERR_PAGE, attend_site)

    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    for bad in (-1, x.k_pages.shape[0], 1 << 30, -(1 << 31)):
        table = x.table.clone()
        table[1, 1] = bad
        run(304, table=table, attend_site=304)
    run(303, lens=i32(40, 100000, 50), attend_site=302)
    run(303, lens=i32(40, -5, 50), attend_site=302)
    run(303, lens=i32(40, 0, 50))
    run(301, cu=i32(0, 1, 900, 3), attend_site=301)
    run(303, rope=fa.rope_table(45, 128))


def test_bad_prefix_page_is_reported():
    x = Batch(4, 2, 128, 16, [40, 50], [1, 1], seed=2, prefix=32)
    x.prefix_pages[1] = -7
    fa.fwd_paged_prefix(*x.args(), x.prefix_pages, max_q=1)
    assert status() == (fa.FA_ERR_PAGE, 304)


# ------------------------------------------------------- used together

def test_serving_steps_match_dense_attention():
    """A prompt appended and attended, then single tokens, then a batch that
    shares the prompt: equal to the library's dense attention of the same keys."""
    Hq, Hkv, d, page, P = 8, 2, 128, 16, 208
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(1)
    randn = lambda *s: torch.randn(*s, generator=g, device=dev).to(torch.bfloat16)  # noqa: E731
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    kp = torch.full((64, Hkv, page, d), math.nan, dtype=torch.bfloat16, device=dev)
    vp = kp.clone()
    rope = fa.rope_table(512, d)
    ids = torch.randperm(64, generator=g, device=dev).to(torch.int32)
    shared = P // page
    table = torch.stack([torch.cat([ids[:shared], ids[shared + 4 * b:shared + 4 * (b + 1)]])
                         for b in range(3)]).contiguous()
    ks, vs = [[], [], []], [[], [], []]

    def dense(q, kk, vv):  # q (n, Hq, d), the sequence's keys so far
        o, lse = fa.fwd_gqa(q.transpose(0, 1)[None].contiguous(),
                            torch.cat(kk).transpose(0, 1)[None].contiguous(),
                            torch.cat(vv).transpose(0, 1)[None].contiguous(), causal=True)
        return o[0].transpose(0, 1), lse[0].transpose(0, 1)

    def close(a, b):
        # both round P and O to bf16 on their own: two roundings each, values below 4
        assert (a[0].float() - b[0].float()).abs().max().item() <= 4 * 4 * BF16
        assert (a[1] - b[1]).abs().max().item() <= 1e-4

    def rotate_alone(x, pos):
        pages = torch.zeros(1, x.shape[1], 256, d, dtype=torch.bfloat16, device=dev)
        start = torch.zeros(1, 32, dtype=torch.int32, device=dev)
        n = x.shape[0]
        fa.kv_append(x, x, pages, pages.clone(), start, i32(n), i32(0, n),
                     rope=rope[pos:pos + n].contiguous())
        return pages[0, :, :n].transpose(0, 1)

    # the prompt, by sequence 0
    q, k, v = randn(P, Hq, d), randn(P, Hkv, d), randn(P, Hkv, d)
    q1 = fa.kv_append(k, v, kp, vp, table[:1], i32(P), i32(0, P), q=q, rope=rope)
    got = fa.fwd_paged(q1, kp, vp, table[:1], i32(P), i32(0, P), max_q=P)
    kr = rotate_alone(k, 0)
    close(got, dense(q1, [kr], [v]))
    for b in range(3):
        ks[b], vs[b] = [kr], [v]
    # steps of one, two and no tokens; the prefix shared
    lens = [P, P, P]
    for step in ([1, 2, 0], [1, 1, 1], [0, 1, 3], [1, 1, 1]):
        lens = [a + n for a, n in zip(lens, step)]
        T = sum(step)
        cu = [0, step[0], step[0] + step[1], T]
        q, k, v = randn(T, Hq, d), randn(T, Hkv, d), randn(T, Hkv, d)
        args = (table, i32(*lens), i32(*cu))
        qr = fa.kv_append(k, v, kp, vp, *args, q=q, rope=rope)
        a = fa.fwd_paged(qr, kp, vp, *args, max_q=max(step))
        s = fa.fwd_paged_prefix(qr, kp, vp, *args, ids[:shared], max_q=max(step))
        fa.check_device_status()
        for b in range(3):
            if step[b] == 0:
                continue
            rows = slice(cu[b], cu[b + 1])
            ks[b] = ks[b] + [rotate_alone(k[rows], lens[b] - step[b])]
            vs[b] = vs[b] + [v[rows]]
            ref = dense(qr[rows], ks[b], vs[b])
            close((a[0][rows], a[1][rows]), ref)
            close((s[0][rows], s[1][rows]), ref)


def test_graph_replay_with_new_lengths():
    """One captured append + attention step serves the following steps: only
    the tables' contents change."""
    Hq, Hkv, d, page, B = 8, 2, 128, 16, 5
    x = Batch(Hq, Hkv, d, page, [100, 37, 260, 16, 5], [1] * B, seed=6, width=20)
    rope = fa.rope_table(512, d)
    table = torch.arange(B * 20, dtype=torch.int32, device="cuda").reshape(B, 20).contiguous()
    kp = torch.randn(B * 20, Hkv, page, d, device="cuda").to(torch.bfloat16)
    vp = torch.randn(B * 20, Hkv, page, d, device="cuda").to(torch.bfloat16)
    k = torch.randn(B, Hkv, d, device="cuda").to(torch.bfloat16)
    lens = x.seq_lens.clone()
    out, lse, q_out = x.out.clone(), x.lse.clone(), torch.empty_like(x.out)
    ws = torch.empty(max(1, fa.fwd_paged_workspace_size(B, B, Hq, Hkv, d, 1)), dtype=torch.uint8,
                     device="cuda")

    def step():
        fa.kv_append(k, k, kp, vp, table, lens, x.cu_q, q=x.q, q_out=q_out, rope=rope)
        fa.fwd_paged(q_out, kp, vp, table, lens, x.cu_q, max_q=1, out=out, lse=lse, workspace=ws)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step()
    for grow in (1, 30, 3):
        lens += grow
        k.normal_()
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone(), lse.clone()
        step()
        fa.check_device_status()
        assert torch.equal(out, got[0]) and torch.equal(lse, got[1])


def test_two_streams_at_once_give_the_serial_results():
    xs = [Batch(8, 2, 128, 16, [900, 40, 333], [1, 1, 1], seed=1),
          Batch(8, 1, 64, 32, [700, 650], [90, 70], seed=2),
          Batch(8, 2, 128, 16, [700, 641, 800], [1, 2, 1], seed=3, prefix=640)]

    def call(x):
        if x.prefix:
            return fa.fwd_paged_prefix(*x.args(), x.prefix_pages, max_q=max(x.nq))
        return fa.fwd_paged(*x.args(), max_q=max(x.nq))

    serial = [call(x) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    for _ in range(20):
        got = []
        for s, x in zip(streams, xs):
            with torch.cuda.stream(s):
                got.append(call(x))
        torch.cuda.synchronize()
        for a, b in zip(serial, got):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    fa.check_device_status()


def test_cache_past_32_bit_offsets():
    """Pages whose elements lie past 2^31 of the pool."""
    Hkv, page, d = 8, 256, 128
    pages = 9000  # 2.36e9 elements
    kp = torch.empty(pages, Hkv, page, d, dtype=torch.bfloat16, device="cuda")
    vp = torch.empty(pages, Hkv, page, d, dtype=torch.bfloat16, device="cuda")
    x = Batch(16, Hkv, d, page, [400, 300], [1, 3], seed=4)
    far = torch.tensor([8999, 8300, 8990, 8500], dtype=torch.int32, device="cuda")
    tab = x.table.cpu()
    table = torch.zeros_like(x.table)
    for b in range(2):
        for i in range(2):
            f = int(far[2 * b + i])
            kp[f], vp[f] = x.k_pages[int(tab[b, i])], x.v_pages[int(tab[b, i])]
            table[b, i] = f
    o, lse = fa.fwd_paged(x.q, kp, vp, table, x.seq_lens, x.cu_q, max_q=3, out=x.out, lse=x.lse)
    fa.check_device_status()
    x.check(o, lse, True, 1 / math.sqrt(d))
    k = torch.randn(4, Hkv, d, device="cuda").to(torch.bfloat16)
    fa.kv_append(k, k, kp, vp, table, x.seq_lens, x.cu_q)
    fa.check_device_status()
    assert torch.equal(vp[8300, :, 399 - 256], k[0]) and torch.equal(kp[8500, :, 299 - 256], k[3])


# ------------------------------------------------- less usual calls

def test_a_single_row_may_have_any_stride():
    x = Batch(8, 2, 128, 16, [77], [1], seed=8)
    wide = torch.zeros(3, 8 * 128 + 3, dtype=torch.bfloat16, device="cuda")
    q = wide.as_strided((1, 8, 128), (8 * 128 + 3, 128, 1))
    q.copy_(x.q)
    x.q = q
    attend(x)
    k = torch.ones(1, 2, 128 + 8, dtype=torch.bfloat16, device="cuda").as_strided((1, 2, 128), (5, 128, 1))
    got = fa.kv_append(k, k, x.k_pages, x.v_pages, x.table, x.seq_lens, x.cu_q, q=q, q_out=q)
    fa.check_device_status()
    assert got is q and torch.equal(q, x.q_host.cuda())


def test_workspace_is_checked():
    x = Batch(8, 2, 128, 16, [77], [1], seed=8)
    n = fa.fwd_paged_workspace_size(1, 1, 8, 2, 128, 1)
    call = lambda ws: fa.fwd_paged(*x.args(), max_q=1, out=x.out, lse=x.lse, workspace=ws)  # noqa: E731
    with pytest.raises(ValueError, match="workspace"):
        call(torch.empty(n))
    with pytest.raises(ValueError, match="workspace"):
        call(torch.empty(2 * n, dtype=torch.uint8, device="cuda")[::2])
    with pytest.raises(ValueError, match="workspace"):
        call(n)
    with pytest.raises(RuntimeError, match="fa_fwd_paged"):
        call(torch.empty(n - 1, dtype=torch.uint8, device="cuda"))
    o, lse = call(torch.empty(n, dtype=torch.uint8, device="cuda"))
    x.check(o, lse, True, 1 / math.sqrt(128))


def test_captured_graphs_with_their_own_workspaces_replayed_together():
    """Captures that leave the workspace to the allocator: each graph has its
    own, so two of them may run at once, beside eager calls."""
    xs = [Batch(8, 2, 128, 16, [900, 40, 333], [1, 1, 1], seed=1),
          Batch(8, 2, 128, 16, [700, 641, 800], [1, 2, 1], seed=3, prefix=640),
          Batch(8, 1, 64, 32, [700, 650], [90, 70], seed=2)]

    def call(x):
        kw = dict(max_q=max(x.nq), out=x.out, lse=x.lse)
        if x.prefix:
            return fa.fwd_paged_prefix(*x.args(), x.prefix_pages, **kw)
        return fa.fwd_paged(*x.args(), **kw)

    want, graphs, streams = [], [], []
    for x in xs:
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            a, b = call(x)
            want.append((a.clone(), b.clone()))
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            call(x)
        graphs.append(g)
        streams.append(s)
    eager = Batch(8, 2, 128, 16, [500, 600], [1, 30], seed=4)
    first = [t.clone() for t in call(eager)]
    for _ in range(20):
        for x in xs:
            x.out.zero_(), x.lse.zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        again = call(eager)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, again))
        for x, (a, b) in zip(xs, want):
            n = x.cu[-1]
            assert torch.equal(x.out[:n], a[:n]) and torch.equal(x.lse[:n], b[:n])
    fa.check_device_status()


def test_sequences_may_share_pages_in_their_tables():
    """Two sequences whose tables name the same pages, one of them twice."""
    x = Batch(8, 2, 64, 16, [100, 100, 90], [1, 3, 2], seed=12)
    x.table[1] = x.table[0]
    x.keys[1], x.vals[1] = x.keys[0], x.vals[0]
    x.table[2, 1] = x.table[2, 0]
    for y in (x.keys, x.vals):
        y[2] = torch.cat([y[2][:16], y[2][:16], y[2][32:]])
    attend(x)


@pytest.mark.parametrize("Hq,Hkv,d", [(4, 2, 64), (12, 2, 128)])
def test_long_prompt_sampled_rows(Hq, Hkv, d):
    """A prompt of thousands of rows after thousands of keys: a sample of rows
    at the tiles' edges."""
    n, L = 3000, 7001
    x = Batch(Hq, Hkv, d, 64, [L], [n], seed=Hq)
    o, lse = fa.fwd_paged(*x.args(), max_q=n)
    fa.check_device_status()
    for r in (0, 1, 31, 63, 64, 127, 128, 500, 1499, 2047, 2048, 2998, 2999):
        keys = L - n + r + 1
        ref = reference(x.q_host[r:r + 1], x.keys[0][:keys], x.vals[0][:keys], True, 1 / math.sqrt(d))
        compare(o[r:r + 1].cpu(), lse[r:r + 1].cpu(), ref, r)


def test_more_sequences_than_rows_can_fill():
    """A batch whose sequences mostly have no new token, padded to a width."""
    lens = [(i * 53) % 400 for i in range(300)]
    nq = [1 if i % 7 == 3 and lens[i] > 0 else 0 for i in range(300)]
    attend(Batch(16, 4, 128, 16, lens, nq, seed=13, pad=5))


@pytest.mark.parametrize("nq", [[1, 1, 1], [5, 3, 9], [150, 1, 40]])
@pytest.mark.parametrize("prefix", [0, 160])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_a_bad_query_spoils_its_own_row_only(nq, prefix, bad):
    x = Batch(8, 2, 128, 16, [500, 300, 260], nq, seed=14, prefix=prefix)
    want = [t.clone() for t in attend(x, prefix=prefix > 0)]
    row = x.cu[1]
    x.q[row, 3, 7] = bad
    kw = dict(max_q=max(nq), out=x.out, lse=x.lse)
    if prefix:
        o, lse = fa.fwd_paged_prefix(*x.args(), x.prefix_pages, **kw)
    else:
        o, lse = fa.fwd_paged(*x.args(), **kw)
    fa.check_device_status()
    keep = torch.ones(x.T, 8, dtype=torch.bool, device="cuda")
    keep[row, 3] = False
    assert torch.isnan(lse[row, 3]) and torch.isnan(o[row, 3]).all()
    # What shares its tile may rescale at other moments: two roundings of
    # values below 4, and of the probabilities.
    assert (o[keep].float() - want[0][keep].float()).abs().max() <= 8 * BF16
    assert (lse[keep] - want[1][keep]).abs().max() <= 1e-4


WRONG = {  # argument -> what is wrong with it
    "type": lambda t: t.double() if t.is_floating_point() else t.long(),
    "device": lambda t: t.cpu(),
    "shape": lambda t: torch.cat([t, t], t.dim() - 1),
    "rank": lambda t: t[None],
    "none": lambda t: None,
    "list": lambda t: [1, 2],
    "strides": lambda t: torch.stack([t, t], t.dim()).select(t.dim(), 0),
}


@pytest.mark.parametrize("how", sorted(WRONG))
@pytest.mark.parametrize("what", ["k", "v", "k_pages", "v_pages", "page_table", "seq_lens", "cu_q",
                                  "q", "q_out", "rope"])
def test_append_refuses(what, how):
    x = Batch(8, 2, 128, 16, [60, 70], [2, 1], seed=15)
    k = torch.ones(3, 2, 128, dtype=torch.bfloat16, device="cuda")
    kw = dict(k=k, v=k.clone(), k_pages=x.k_pages, v_pages=x.v_pages, page_table=x.table,
              seq_lens=x.seq_lens, cu_q=x.cu_q, q=x.q, q_out=x.q.clone(), rope=fa.rope_table(80, 128))
    fa.kv_append(**kw)
    if how == "none" and what in ("q_out", "rope"):
        pytest.skip("optional")
    before = x.k_pages.view(torch.int16).clone(), kw["q_out"].clone()
    kw[what] = WRONG[how](kw[what])
    if what == "page_table" and how == "shape":
        kw[what] = x.table.repeat(2, 1)  # (a wider one would be right)
    with pytest.raises((ValueError, RuntimeError)) as e:
        fa.kv_append(**kw)
    # (the sizes come from the table, the pages and k: another argument may be
    # the one that does not fit them)
    named = {"k_pages": ("k_pages", "v_pages", "k "), "page_table": ("page_table", "seq_lens")}.get(what, (what,))
    if isinstance(e.value, ValueError):
        assert any(n in str(e.value) for n in named + ("q_out needs q",)), e.value
    fa.check_device_status()
    assert torch.equal(x.k_pages.view(torch.int16), before[0])
    if what != "q_out":
        assert torch.equal(kw["q_out"], before[1])


@pytest.mark.parametrize("how", sorted(WRONG))
@pytest.mark.parametrize("what", ["q", "k_pages", "v_pages", "page_table", "seq_lens", "cu_q",
                                  "prefix_pages", "out", "lse"])
def test_attention_refuses(what, how):
    x = Batch(8, 2, 128, 16, [60, 70], [2, 1], seed=15, prefix=32)
    kw = dict(q=x.q, k_pages=x.k_pages, v_pages=x.v_pages, page_table=x.table,
              seq_lens=x.seq_lens, cu_q=x.cu_q, prefix_pages=x.prefix_pages, out=x.out, lse=x.lse)
    if how == "none" and what in ("out", "lse", "prefix_pages"):
        pytest.skip("optional, or another call")
    kw[what] = WRONG[how](kw[what])
    if what == "prefix_pages" and how == "shape":
        kw[what] = x.prefix_pages.repeat(40)  # more pages than the table is wide
    if what == "page_table" and how == "shape":
        kw[what] = x.table.repeat(2, 1)  # (a wider one would be right)
    with pytest.raises((ValueError, RuntimeError)) as e:
        fa.fwd_paged_prefix(**kw)
    if isinstance(e.value, ValueError):
        assert any(n in str(e.value) for n in (what, "q has shape", "v_pages", "seq_lens")), e.value
    fa.check_device_status()
    assert torch.all(x.out == 7.0) and torch.all(x.lse == 7.0)


def test_the_calls_and_their_words_agree():
    """The C calls, argument by argument, against the binding, which passes
    words."""
    lib = fa.load()
    x = Batch(8, 2, 128, 16, [300, 200, 177], [1, 40, 2], seed=16, prefix=160, fused=True)
    T, B, width = x.T, x.B, x.table.shape[1]
    rope = fa.rope_table(400, 64)
    k = torch.randn(T, 2, 128, device="cuda").to(torch.bfloat16)
    a, b = (x.k_pages.clone(), x.v_pages.clone()), (x.k_pages.clone(), x.v_pages.clone())
    q_out = torch.zeros(T, 8, 128, dtype=torch.bfloat16, device="cuda")
    want = fa.kv_append(k, k, *a, x.table, x.seq_lens, x.cu_q, q=x.q, rope=rope, interleaved=True)
    p = lambda t: t.data_ptr()  # noqa: E731
    stream = torch.cuda.current_stream().cuda_stream
    tables = p(x.table), p(x.seq_lens), p(x.cu_q)
    rc = lib.fa_kv_append(p(x.q), p(k), p(k), p(q_out), p(b[0]), p(b[1]), *tables, p(rope), T, B, 8,
                          2, 128, x.q.stride(0), 256, 256, 1024, x.k_pages.shape[0], 16, width, 64,
                          400, 1, stream)
    assert rc == fa.FA_OK
    fa.check_device_status()
    assert torch.equal(q_out, want)
    for i in range(2):
        assert torch.equal(a[i].view(torch.int16), b[i].view(torch.int16))
    for prefix in (False, True):
        extra = (p(x.prefix_pages), 160) if prefix else ()
        if prefix:
            o, lse = fa.fwd_paged_prefix(*x.args(), x.prefix_pages, max_q=40, scale=0.07)
        else:
            o, lse = fa.fwd_paged(*x.args(), max_q=40, scale=0.07)
        n = fa.fwd_paged_workspace_size(T, B, 8, 2, 128, 40, 160 if prefix else 0)
        ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        fn = lib.fa_fwd_paged_prefix if prefix else lib.fa_fwd_paged
        rc = fn(p(x.q), p(x.k_pages), p(x.v_pages), p(x.out), p(x.lse), *tables, *extra, T, B, 8, 2,
                128, x.q.stride(0), x.k_pages.shape[0], 16, width, 40, 1, 0.07, p(ws), n, stream)
        assert rc == fa.FA_OK
        fa.check_device_status()
        assert torch.equal(o, x.out) and torch.equal(lse, x.lse)
