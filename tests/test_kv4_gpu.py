"""The paged cache in 4 bits on the GPU: appends against the quantisation written
from its definition, bit for bit; reading back; attention against 64 bits."""
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


# ------------------------------------------------------------------ append


def rotated(x, pos, rope, interleaved):
    """x (n, H, d) fp32 turned by the table's rows pos, every operation rounded."""
    rd = rope.shape[1]
    half = rd // 2
    c, s = rope[pos][:, None, :half], rope[pos][:, None, half:]
    y = x.clone()
    a, b = (x[..., 0:rd:2], x[..., 1:rd:2]) if interleaved else (x[..., :half], x[..., half:rd])
    u, v = a * c - b * s, a * s + b * c
    if interleaved:
        y[..., 0:rd:2], y[..., 1:rd:2] = u, v
    else:
        y[..., :half], y[..., half:rd] = u, v
    return y


class Append:
    """New rows of ragged sequences, and the pool the append should leave."""

    def __init__(self, Hq, Hkv, d, page, lens, nq, seed=0, rope=0, interleaved=False, pad=0,
                 k_scale=1.0, v_scale=1.0, fused=False, data=None):
        g = torch.Generator().manual_seed(seed)
        self.Hkv, self.d, self.page, self.interleaved = Hkv, d, page, interleaved
        self.scales = dict(k_scale=k_scale, v_scale=v_scale)
        cu = [0]
        for n in nq:
            cu.append(cu[-1] + n)
        T = cu[-1] + pad
        qkv = torch.randn((T, Hq + 2 * Hkv, d), generator=g) * torch.cat(
            [torch.ones(Hq), torch.full((Hkv,), k_scale), torch.full((Hkv,), v_scale)])[:, None]
        if data is not None:
            qkv = data(qkv)
        qkv = qkv.to(torch.bfloat16)
        self.q, self.k, self.v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        dev = qkv.cuda() if fused else None
        part = (lambda x, lo, hi: dev[:, lo:hi]) if fused else (lambda x, lo, hi: x.cuda().contiguous())
        self.dq, self.dk, self.dv = (part(self.q, 0, Hq), part(self.k, Hq, Hq + Hkv),
                                     part(self.v, Hq + Hkv, Hq + 2 * Hkv))
        counts = [max(1, -(-n // page)) for n in lens]
        order = torch.randperm(sum(counts) + 2, generator=g)
        table = torch.full((len(lens), max(counts)), 1 << 30, dtype=torch.int32)
        pool = torch.randint(0, 256, (sum(counts) + 2, Hkv, page // 16, 18 * d), generator=g,
                             dtype=torch.uint8)
        self.pages = pool.flatten(2).cuda()
        self.rope = None
        if rope:
            half = rope // 2
            ang = torch.arange(max(lens), dtype=torch.float64)[:, None] * 10000.0 ** (
                -torch.arange(half, dtype=torch.float64) / half)
            self.rope = torch.cat([ang.cos(), ang.sin()], 1).float()
        want, at = pool.clone(), 0
        self.rows = []
        self.q_want = self.q.float().clone()
        inv_k, inv_v = (torch.tensor(1.0, dtype=torch.float32) / torch.tensor(x, dtype=torch.float32)
                        for x in (k_scale, v_scale))
        for b, (n, L) in enumerate(zip(nq, lens)):
            ids = order[at:at + counts[b]]
            table[b, :counts[b]] = ids.to(torch.int32)
            at += counts[b]
            if n == 0:
                continue
            rows, pos = slice(cu[b], cu[b + 1]), torch.arange(L - n, L)
            k = self.k[rows].float()
            if rope:
                k = rotated(k, pos, self.rope, interleaved)
                self.q_want[rows] = rotated(self.q[rows].float(), pos, self.rope, interleaved)
            kc, ks = c4.quantize((k * inv_k).double())
            vc, vs = c4.quantize((self.v[rows].float() * inv_v).double())
            self.rows.append((rows, c4.values(kc, ks) * k_scale, c4.values(vc, vs) * v_scale))
            for i in range(n):
                p = int(pos[i])
                blocks = want[ids[p // page], :, p % page // 16]
                for h in range(Hkv):
                    c4.put(blocks[h], p % 16, kc[i, h], ks[i, h], vc[i, h], vs[i, h])
        self.want, self.table, self.lens, self.nq = want.flatten(2), table.cuda(), lens, nq
        self.seq_lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.cu_q = torch.tensor(cu, dtype=torch.int32, device="cuda")
        self.T, self.Hq, self.end = T, Hq, cu[-1]

    def run(self):
        return fa.kv4_append(self.dk, self.dv, self.pages, self.table, self.seq_lens, self.cu_q,
                             q=self.dq, rope=None if self.rope is None else self.rope.cuda(),
                             interleaved=self.interleaved, **self.scales)

    def check_pool(self):
        """Bit for bit, but for what no key owns: the odd half of a V byte (and
        its scale) behind a sequence's last key, when it is even."""
        got, want = self.pages.cpu().clone(), self.want.clone()
        d, page = self.d, self.page
        for b, (n, L) in enumerate(zip(self.nq, self.lens)):
            if n and L % 2 == 1:
                page_id = int(self.table[b, (L - 1) // page])
                r, blk = (L - 1) % 16, (L - 1) % page // 16
                for x in (got, want):
                    v = x[page_id].view(self.Hkv, page // 16, 18 * d)[:, blk]
                    for i in range(8):
                        o = 8 * d + ((r // 8 * 8 + i) * 4 + r % 8 // 2) * (d // 8)
                        v[:, o:o + d // 8] &= 15
        assert torch.equal(got, want), (got != want).nonzero()[:5]


APPENDS = [
    dict(Hq=4, Hkv=2, d=128, page=16, lens=[1, 2, 17, 40], nq=[1, 1, 1, 1], rope=128),
    dict(Hq=4, Hkv=2, d=64, page=16, lens=[5, 6, 33, 48, 9], nq=[5, 3, 17, 48, 0], rope=64, pad=3),
    dict(Hq=3, Hkv=3, d=64, page=32, lens=[31, 64, 65], nq=[7, 8, 9], rope=32, interleaved=True),
    dict(Hq=8, Hkv=1, d=128, page=64, lens=[63, 100], nq=[62, 33], rope=96, fused=True, pad=2),
    dict(Hq=5, Hkv=5, d=128, page=256, lens=[257, 300], nq=[3, 44], rope=16, k_scale=0.7713, v_scale=0.0613),
    dict(Hq=2, Hkv=2, d=64, page=128, lens=[130], nq=[129], k_scale=4.0, v_scale=0.0625),
    dict(Hq=16, Hkv=16, d=128, page=16, lens=[18, 18], nq=[1, 2], rope=128, interleaved=True, fused=True),
    dict(Hq=2, Hkv=1, d=128, page=16, lens=[31], nq=[30], rope=48),
    dict(Hq=2, Hkv=1, d=64, page=16, lens=[31], nq=[30], rope=48, interleaved=True),
]


@pytest.mark.parametrize("case", APPENDS)
def test_append_and_read(case):
    a = Append(seed=11, **case)
    q = a.run()
    fa.check_device_status()
    a.check_pool()
    got = q.cpu().float()
    # (q may be turned with fused products: both roundings of its bf16)
    tol = c4.BF16 * a.q_want.abs() + 4 * c4.FP32 * 2 * a.q_want.abs().amax(-1, keepdim=True)
    assert torch.all((got - a.q_want).abs()[:a.end] <= tol[:a.end]) and torch.all(got[a.end:] == 0)
    k_out = torch.full((a.T, a.Hkv, a.d), 7.0, dtype=torch.bfloat16, device="cuda")
    v_out = torch.full((a.T, a.Hkv + 1, a.d), 7.0, dtype=torch.bfloat16, device="cuda")[:, 1:]
    fa.kv4_read(a.pages, a.table, a.seq_lens, a.cu_q, k_out, v_out, **a.scales)
    fa.check_device_status()
    for rows, k, v in a.rows:
        for x, y in ((k_out, k), (v_out, v)):
            # one rounding of the tensor's scale, of the product, to bf16
            err = (x[rows].cpu().double() - y).abs()
            exact = all(math.log2(s) % 1 == 0 for s in a.scales.values())
            assert torch.all(err <= (0 if exact else c4.BF16 + 3 * c4.FP32) * y.abs())
    assert torch.all(k_out[a.end:] == 7.0) and torch.all(v_out[a.end:] == 7.0)


def test_append_special_numbers():
    def data(x):
        x[0, 2, :16] = 0.0                      # an empty group
        x[1, 2, 16:32] = 1e-5                   # below the smallest scale
        x[2, 2, 0] = math.inf
        x[3, 2, 5] = -math.inf
        x[4, 3, 7] = math.nan
        x[5, 3, 16:32] = 3e4                    # beyond the largest
        x[6, 3] = torch.arange(128) * 0.0625 - 4  # many halfway cases
        x[7, 2, 32:48] = torch.tensor([6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0] * 2)
        return x
    a = Append(2, 1, 128, 16, [8], [8], seed=5, data=data)
    a.run()
    fa.check_device_status()
    k_out = torch.empty((8, 1, 128), dtype=torch.bfloat16, device="cuda")
    v_out = torch.empty_like(k_out)
    fa.kv4_read(a.pages, a.table, a.seq_lens, a.cu_q, k_out, v_out)
    k, v = k_out.cpu().double()[:, 0], v_out.cpu().double()[:, 0]
    assert torch.all(k[0, :16] == 0) and torch.all(k[1, 16:32] == 0)
    assert k[2, 0] == 6 * 448 and k[3, 5] == -6 * 448
    assert torch.all(k[2, 1:16] == 0) and torch.isnan(v[4, :16]).all()
    assert not torch.isnan(v[4, 16:]).any() and torch.all(v[5, 16:32] == 6 * 448)
    assert torch.equal(k[7, 32:48], torch.tensor([6, 0, 1, 1, 2, 2, 4, 4] * 2, dtype=torch.float64))
    (_, kw, vw), = a.rows
    rows = [0, 1, 6, 7]
    assert torch.equal(k[rows], kw[rows, 0]) and torch.equal(v[rows], vw[rows, 0])


def test_append_in_steps_is_the_whole():
    """Token by token, odd and even starts, leaves the same pool as one call."""
    whole = Append(2, 2, 64, 16, [37], [37], seed=3, rope=64)
    whole.run()
    rope = whole.rope.cuda()
    pages = torch.randint(0, 256, whole.pages.shape, dtype=torch.uint8, device="cuda")
    at = 0
    for n in (1, 1, 2, 3, 5, 1, 8, 16):
        rows = slice(at, at + n)
        at += n
        lens = torch.tensor([at], dtype=torch.int32, device="cuda")
        cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        fa.kv4_append(whole.dk[rows], whole.dv[rows], pages, whole.table, lens, cu, rope=rope)
    outs = []
    for p in (whole.pages, pages):
        k = torch.empty((37, 2, 64), dtype=torch.bfloat16, device="cuda")
        v = torch.empty_like(k)
        outs.append(fa.kv4_read(p, whole.table, whole.seq_lens, whole.cu_q, k, v))
    fa.check_device_status()
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])


# --------------------------------------------------------------- attention


def attend(x, causal=True, scale=None, max_q=None, **kw):
    o, lse = fa.fwd_paged4(*x.args(), max_q=max_q, causal=causal, scale=scale, out=x.out, lse=x.lse,
                           **x.scales(), **kw)
    fa.check_device_status()
    x.check(o, lse, causal, x.d ** -0.5 if scale is None else scale)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("case", [
    dict(Hq=4, Hkv=4, d=64, page=16, lens=[1, 2, 15, 16, 17, 33], nq=[1, 1, 1, 1, 1, 1]),
    dict(Hq=8, Hkv=2, d=128, page=16, lens=[1000], nq=[1]),
    dict(Hq=8, Hkv=1, d=128, page=32, lens=[300, 0, 129, 128], nq=[1, 1, 0, 2], pad=3),
    dict(Hq=12, Hkv=2, d=64, page=64, lens=[777, 65], nq=[4, 5], fused=True),
    dict(Hq=16, Hkv=1, d=128, page=128, lens=[260, 500, 1], nq=[1, 1, 1]),
    dict(Hq=24, Hkv=1, d=64, page=16, lens=[100, 31], nq=[1, 3]),
    dict(Hq=17, Hkv=1, d=128, page=16, lens=[50], nq=[2]),
    dict(Hq=4, Hkv=2, d=128, page=256, lens=[513, 90], nq=[60, 90]),
    dict(Hq=4, Hkv=1, d=64, page=16, lens=[400, 70, 40], nq=[100, 1, 1], pad=1),
    dict(Hq=2, Hkv=2, d=128, page=64, lens=[700], nq=[300], k_scale=0.7713, v_scale=0.0613),
    dict(Hq=6, Hkv=2, d=128, page=16, lens=[5, 3], nq=[5, 7]),
])
def test_attention(case, causal):
    attend(c4.Batch4(seed=21, **case), causal, max_q=max(case["nq"]))


@pytest.mark.parametrize("scale", [0.0, -0.125, 1.0])
def test_attention_scales(scale):
    for nq in ([1, 1, 1], [90, 3, 40]):
        attend(c4.Batch4(4, 2, 64, 16, [90, 91, 100], nq, seed=4), True, scale)


@pytest.mark.parametrize("d", [64, 128])
def test_attention_of_loud_keys(d):
    """Scores of some hundred: the running maximum keeps moving."""
    for nq in ([1, 1], [70, 5]):
        attend(c4.Batch4(8, 2, d, 16, [600, 70], nq, seed=6, spread=20.0))


def test_attention_many_sequences():
    lens = [1 + (37 * i) % 200 for i in range(70)]
    attend(c4.Batch4(4, 2, 64, 16, lens, [1] * 70, seed=8), max_q=1)
    nq = [min(n, 1 + (i % 9 == 0) * 40) for i, n in enumerate(lens)]
    attend(c4.Batch4(4, 1, 128, 16, lens, nq, seed=9), max_q=max(nq))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("scale,k_scale", [(-1e-10, 1e-37), (1e-10, 1e-37), (-1e-30, 1e-38),
                                           (-0.0, 1.0), (-1e-20, 1.0)])
def test_attention_of_a_scale_that_vanishes(scale, k_scale, d):
    # (The product with the keys' scale is 0 with a sign, or next to it: every key
    # that is seen counts the same, none that is hidden.)
    for nq in ([1, 1, 1], [90, 3, 40], [600, 2, 300]):
        lens = [max(n, 90 + i) for i, n in enumerate(nq)]
        attend(c4.Batch4(4, 2, d, 16, lens, nq, seed=4, k_scale=k_scale), True, scale, max_q=max(nq))


# More rows than the append's and the read's CTAs have one each of: a CTA's next row
# takes over from its last one.
LONG = [
    dict(Hq=4, Hkv=1, d=128, page=16, lens=[701, 40, 9, 399, 5, 517], nq=[701, 1, 0, 334, 5, 402], rope=64,
         pad=3),
    dict(Hq=2, Hkv=2, d=64, page=64, lens=[3, 1000, 778, 2], nq=[1, 999, 477, 2], rope=64, interleaved=True,
         fused=True),
    dict(Hq=1, Hkv=1, d=64, page=32, lens=[5] * 300 + [77], nq=[5, 4, 3, 5, 5] * 60 + [76], pad=1),
]


def check_rows(a, refused=()):
    """The whole pool, bit for bit, and every row read back; `refused`: (first, end) of
    packed rows that were not to be written or read."""
    skip = torch.zeros(a.T, dtype=torch.bool)
    for lo, hi in refused:
        skip[lo:hi] = True
    assert torch.equal(a.pages.cpu(), a.want), (a.pages.cpu() != a.want).nonzero()[:5]
    k_out = torch.full((a.T, a.Hkv, a.d), 7.0, dtype=torch.bfloat16, device="cuda")
    v_out = torch.full_like(k_out, 7.0)
    fa.kv4_read(a.pages, a.table, a.seq_lens, a.cu_q, k_out, v_out, **a.scales)
    status = fa.device_status()
    want_k = torch.full((a.T, a.Hkv, a.d), 7.0, dtype=torch.float64)
    want_v = want_k.clone()
    for rows, k, v in a.rows:
        want_k[rows], want_v[rows] = k, v
    want_k[skip] = want_v[skip] = 7.0
    assert torch.equal(k_out.cpu().double(), want_k) and torch.equal(v_out.cpu().double(), want_v)
    return status


@pytest.mark.parametrize("case", LONG)
def test_append_and_read_many_rows(case):
    a = Append(seed=13, **case)
    assert a.T > 1216
    a.run()
    fa.check_device_status()
    assert check_rows(a) == (0, 0)


@pytest.mark.parametrize("case", LONG[:2])
@pytest.mark.parametrize("number", [-1, 10 ** 9])
def test_append_and_read_around_a_refused_page(case, number):
    a = Append(seed=14, **case)
    before = a.pages.cpu().clone()
    b = case["nq"].index(max(case["nq"]))
    j = case["lens"][b] // case["page"] // 2
    page = int(a.table[b, j])
    a.table[b, j] = number
    a.want[page] = before[page]
    first = int(a.cu_q[b + 1]) - (case["lens"][b] - j * case["page"])
    a.run()
    assert fa.device_status() == (fa.FA_ERR_PAGE, 304)
    assert check_rows(a, [(first, first + case["page"])]) == (fa.FA_ERR_PAGE, 304)


def test_append_many_rows_past_the_rotations_table():
    a = Append(seed=15, **LONG[0])
    before, page, cut = a.pages.cpu().clone(), 16, 480
    for b, L in enumerate(a.lens):
        for j in range(cut // page, -(-L // page)):
            a.want[a.table[b, j].item()] = before[a.table[b, j].item()]
    a.rope = a.rope[:cut].contiguous()
    a.run()
    assert fa.device_status() == (fa.FA_ERR_PAGE, 303)
    assert torch.equal(a.pages.cpu(), a.want)


@pytest.mark.parametrize("case", APPENDS)
def test_append_leaves_the_other_key_of_a_pair(case):
    """The whole pool bit for bit, the half of a byte that no row owns among it."""
    a = Append(seed=12, **case)
    a.run()
    fa.check_device_status()
    assert torch.equal(a.pages.cpu(), a.want), (a.pages.cpu() != a.want).nonzero()[:5]


def long_batch(Hq, Hkv, d, page, B, length, nq, seed, spread, pool_pages):
    """B sequences of some `length` keys on pages that they share, each in an order of
    its own, some pages more than once: the attention's inputs, and a sequence's keys
    and values in fp64."""
    x = c4.Batch4(Hq, Hkv, d, page, [pool_pages * page], [B * nq], seed=seed, spread=spread)
    g = torch.Generator().manual_seed(seed + 1)
    lens = [length - 37 * b for b in range(B)]
    order = [torch.randint(pool_pages, (-(-n // page),), generator=g) for n in lens]
    table = torch.full((B, -(-length // page)), 1 << 30, dtype=torch.int32)
    base = x.table[0].cpu()
    for b, o in enumerate(order):
        table[b, :len(o)] = base[o]
    x.table, x.lens, x.nq, x.B = table.cuda(), lens, [nq] * B, B
    x.cu = [b * nq for b in range(B + 1)]
    x.seq_lens, x.cu_q = (torch.tensor(t, dtype=torch.int32, device="cuda") for t in (lens, x.cu))

    def sequence(b):
        return [t.unflatten(0, (pool_pages, page))[order[b]].flatten(0, 1)[:lens[b]]
                for t in (x.keys[0], x.vals[0])]
    return x, sequence


# A CTA has a run of some 30 tiles: its warps go round their rings many times, take
# the numbers of their pages again and again, and (spread 20) meet louder keys late.
@pytest.mark.parametrize("spread", [1.0, 20.0])
@pytest.mark.parametrize("Hq,Hkv,d,page,nq", [
    (4, 4, 128, 16, 1),      # 1 row
    (32, 4, 128, 64, 1),     # 8
    (16, 4, 64, 16, 2),      # 8 of two tokens
    (64, 4, 128, 16, 1),     # 16
    (16, 4, 64, 128, 4),     # 16 of four tokens
    (16, 4, 128, 16, 5),     # 16, and 4
])
def test_decode_of_long_segments(Hq, Hkv, d, page, nq, spread):
    x, sequence = long_batch(Hq, Hkv, d, page, 28, 16000, nq, 23, spread, 8192 // page)
    o, lse = fa.fwd_paged4(*x.args(), max_q=nq, out=x.out, lse=x.lse)
    fa.check_device_status()
    o, lse = o.cpu(), lse.cpu()
    for b in range(x.B):
        k, v = sequence(b)
        rows = slice(b * nq, b * nq + nq)
        ref = c4.reference(x.q_host[rows], k, v, True, d ** -0.5)
        c4.compare(o[rows], lse[rows], ref, (b, x.lens[b]))


@pytest.mark.parametrize("size", [1e-24, 1e-28, 1e-32, 1e-36, 1e-38, 3e-40])
@pytest.mark.parametrize("nq", [[1, 2], [90, 3]])
def test_attention_of_tiny_queries(nq, size):
    """Down to the numbers of bf16 that are not normal, under scales that make as much
    of them as of others."""
    x = c4.Batch4(4, 2, 128, 16, [200, 64], nq, seed=24, spread=3.0)
    x.q_host = (x.q_host.double() * size).to(torch.bfloat16)
    x.q = x.q_host.cuda()
    attend(x, True, 128 ** -0.5 * min(1 / size, 2e38), max_q=max(nq))


@pytest.mark.parametrize("rows", [1, 12, 100, 300])
@pytest.mark.parametrize("d", [64, 128])
def test_attention_of_tiny_values(d, rows):
    """Values next to the smallest normal numbers, of keys that all weigh the same: the
    mean of 30,000 equal ones is that one, however large the sum of their weights (many
    sequences on the same pages, so that a CTA adds up most of one)."""
    L, Hkv, v_scale, B = 30000, 4, 4e-39, max(40 * 8 // (rows + 7), 8)
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    v = torch.full((L, Hkv, d), 2688 * v_scale, dtype=torch.bfloat16, device="cuda")
    v[:, :, 1::2] *= -0.5
    n = -(-L // 16)
    pool, table = fa.kv4_pages(n, Hkv, 16, d), torch.arange(n, dtype=torch.int32, device="cuda")[None]
    fa.kv4_append(torch.ones_like(v), v, pool, table, ints([L]), ints([0, L]), v_scale=v_scale)
    q = torch.ones((B * rows, 4 * Hkv, d), dtype=torch.bfloat16, device="cuda")
    o, _ = fa.fwd_paged4(q, pool, table.expand(B, n).contiguous(), ints([L] * B),
                         ints([b * rows for b in range(B + 1)]), max_q=rows, causal=False, v_scale=v_scale)
    fa.check_device_status()
    held = torch.tensor([2688.0, -1344.0], dtype=torch.float64).repeat(d // 2) * v_scale
    # one rounding to bf16, sums of L terms and a few more roundings in fp32, v_scale's
    # own below fp32's normal range
    off = (o.cpu().double() - held).abs() / held.abs()
    assert (off <= c4.BF16 + (L + 64) * c4.FP32 + 2.0 ** -150 / v_scale).all(), off.max().item()
