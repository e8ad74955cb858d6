"""Batches whose kinds of work differ a thousandfold on the GPU: a long prompt
chunk beside a few short decoding sequences, the opposite, and a prefix far
longer than the sequences' own keys.  Every row is written, whatever share of
the call's work it is."""
import math

import pytest
import torch

from io_aware_exact_02_gb300 import build, fa
from paged_common import Batch, compare, reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return fa.load()


def check(x, o, lse, causal=True):
    """Whole sequences against fp64, a sample of the rows of long ones; rows
    outside every sequence as they were."""
    o, lse = o.cpu(), lse.cpu()
    scale = 1 / math.sqrt(x.d)
    assert torch.all(o[x.cu[-1]:] == 7.0) and torch.all(lse[x.cu[-1]:] == 7.0)
    # (no row of the batch has a logsumexp of exactly 7, or 64 channels of 7)
    assert not torch.any(lse[:x.cu[-1]] == 7.0)
    assert not torch.any((o[:x.cu[-1]] == 7.0).all(-1))
    for b in range(x.B):
        t0, n, L = x.cu[b], x.nq[b], x.lens[b]
        if n == 0:
            continue
        if n * L * x.Hq <= 1 << 24:
            runs = [(0, n)]
        else:
            runs = [(r, 1) for r in sorted({0, 1, 31, 32, 63, 64, n // 2, n - 2, n - 1})]
        for r, m in runs:
            keys = L - n + r + m if causal else L
            ref = reference(x.q_host[t0 + r:t0 + r + m], x.keys[b][:keys], x.vals[b][:keys], causal,
                            scale)
            compare(o[t0 + r:t0 + r + m], lse[t0 + r:t0 + r + m], ref, (b, r, L))


MIXED = [
    # Hq, Hkv, d, page, lens, nq: work of the decoding sequences against the
    # chunk's below, at and above one CTA's share
    (4, 1, 128, 16, [32768, 100], [126, 1]),
    (4, 1, 64, 64, [100, 32768, 0], [1, 126, 0]),
    (8, 2, 128, 64, [8192, 64] + [0] * 14, [512, 1] + [0] * 14),
    (4, 1, 128, 256, [65536] + [100] * 8, [512] + [1] * 8),
    (4, 1, 128, 32, [32000] + [1000] * 3 + [0] * 28, [2000] + [1] * 3 + [0] * 28),
    (4, 1, 128, 32, [9000, 100, 100, 90], [126, 1, 1, 1]),
    (4, 1, 128, 32, [20000, 700, 300], [126, 1, 1]),
    (16, 2, 64, 16, [16384] + [30] * 40, [200] + [1] * 40),
    # the opposite: a short chunk beside long decoding sequences
    (4, 1, 128, 16, [100] + [3000 + 7 * i for i in range(40)], [100] + [1] * 40),
    (8, 2, 64, 64, [70, 30000, 20000], [70, 1, 1]),
]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("case", range(len(MIXED)))
def test_mixed_batches_of_very_uneven_work(case, causal):
    Hq, Hkv, d, page, lens, nq = MIXED[case]
    x = Batch(Hq, Hkv, d, page, lens, nq, seed=case, pad=case % 3)
    o, lse = fa.fwd_paged(*x.args(), max_q=max(nq), causal=causal, out=x.out, lse=x.lse)
    fa.check_device_status()
    check(x, o, lse, causal)


@pytest.mark.parametrize("max_q", [1, 16, 64, 126, 1000, 2147483647, None])
@pytest.mark.parametrize("lens,nq", [([9000, 100, 100, 90], [126, 1, 1, 1]),
                                     ([32768, 100], [126, 1]),
                                     ([130] + [4000] * 20, [126] + [1] * 20)])
def test_max_q_is_only_a_hint_for_uneven_work(lens, nq, max_q):
    x = Batch(4, 1, 128, 32, lens, nq, seed=len(lens))
    o, lse = fa.fwd_paged(*x.args(), max_q=max_q, out=x.out, lse=x.lse)
    fa.check_device_status()
    check(x, o, lse)


@pytest.mark.parametrize("Hq,Hkv,d,page,prefix,lens", [
    (8, 2, 128, 16, 16384, [16385 + i % 3 for i in range(20)]),  # all of the work is the prefix's
    (8, 2, 128, 16, 16, [5000 + 31 * i for i in range(20)]),     # nearly none of it is
    (64, 2, 64, 64, 64, [20000] + [65] * 9),
])
def test_prefixes_of_very_uneven_work(Hq, Hkv, d, page, prefix, lens):
    x = Batch(Hq, Hkv, d, page, lens, [1] * len(lens), seed=d, pad=1, prefix=prefix)
    o, lse = fa.fwd_paged_prefix(*x.args(), x.prefix_pages, max_q=1, out=x.out, lse=x.lse)
    fa.check_device_status()
    check(x, o, lse)


@pytest.mark.parametrize("repeat", [20, 30, 60])
def test_a_prefix_of_more_units_than_ctas_beside_one_token(repeat):
    """152 key/value heads, so that the prefix's units are not dealt whole, and
    300 to 1,000 times the work of the one sequence's own key.  The prefix names
    its eight pages over and over."""
    H, d, page, distinct, T = 152, 64, 256, 8, 65
    g = torch.Generator().manual_seed(repeat)
    randn = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16)  # noqa: E731
    kp, vp = randn(distinct + 1, H, page, d), randn(distinct + 1, H, page, d)
    kp[distinct, :, 1:] = math.nan
    vp[distinct, :, 1:] = math.inf
    q, n = randn(T, H, d), distinct * repeat
    pages = torch.arange(distinct, dtype=torch.int32).repeat(repeat)
    table = torch.full((1, n + 1), distinct, dtype=torch.int32)
    L = n * page + 1
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    out = torch.full((T, H, d), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T, H), 7.0, device="cuda")
    fa.fwd_paged_prefix(q.cuda(), kp.cuda(), vp.cuda(), table.cuda(), i32(L), i32(0, 1),
                        pages.cuda(), max_q=1, out=out, lse=lse)
    fa.check_device_status()
    out, lse = out.cpu(), lse.cpu()
    assert torch.all(out[1:] == 7.0) and torch.all(lse[1:] == 7.0)
    assert not torch.any(lse[0] == 7.0) and not torch.any((out[0] == 7.0).all(-1))
    for h in (0, 1, 74, 75, 76, 150, 151):
        one = slice(h, h + 1)
        k, v = (torch.cat([x[:distinct, h].reshape(-1, d).repeat(repeat, 1), x[distinct, h, :1]])
                for x in (kp, vp))
        ref = reference(q[:1, one], k[:, None], v[:, None], True, 1 / math.sqrt(d))
        compare(out[:1, one], lse[:1, one], ref, h)
