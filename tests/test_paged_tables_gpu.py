"""The paged cache's device-side tables on the GPU: entries out of bounds are
recorded, and the other sequences' results stay right."""
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


def sound(x, o, lse, but):
    """The results of all sequences but some."""
    for b in range(x.B):
        rows = slice(x.cu[b], x.cu[b + 1])
        if b in but or x.nq[b] == 0:
            continue
        ref = reference(x.q_host[rows], x.keys[b], x.vals[b], True, 1 / math.sqrt(x.d))
        compare(o[rows].cpu(), lse[rows].cpu(), ref, b)


# Tokens of the sequences: all single, all of four (behind a prefix: both lists
# side by side), chunks, and chunks among single ones.
ROWS = [[1] * 20, [4] * 20, [70] * 20, [90, 150] + [1] * 18]


@pytest.mark.parametrize("prefix", [0, 320])
@pytest.mark.parametrize("nq", ROWS)
@pytest.mark.parametrize("bad", [1 << 20, 2147483647, -1, -(1 << 31)])
def test_a_bad_length_spoils_its_own_sequence_only(nq, prefix, bad):
    x = Batch(8, 2, 128, 16, [500 + 7 * i for i in range(20)], nq, seed=1, prefix=prefix)
    lens = x.seq_lens.clone()
    lens[5] = bad
    args = x.q, x.k_pages, x.v_pages, x.table, lens, x.cu_q
    args += (x.prefix_pages,) if prefix else ()
    o, lse = (fa.fwd_paged_prefix if prefix else fa.fwd_paged)(*args, max_q=max(nq))
    assert fa.device_status() == (fa.FA_ERR_PAGE, 302)
    sound(x, o, lse, (5,))


@pytest.mark.parametrize("fill", [0, 1, 255])
def test_rows_of_no_sequence_behind_a_prefix(fill):
    """Row ranges that leave rows to no sequence, in the form of the call that
    joins a prefix with the sequences' own keys, over a workspace that holds
    anything: an error, and nothing is written to those rows."""
    B, n = 20, 4
    x = Batch(8, 2, 128, 16, [330 + 7 * i for i in range(B)], [n] * B, seed=fill, pad=2, prefix=320)
    cu = x.cu_q.clone()
    cu[7] = 500  # sequences 6 and 7 are none: rows 24 to 31
    ws = torch.full((fa.fwd_paged_workspace_size(x.T, B, 8, 2, 128, n, 320),), fill,
                    dtype=torch.uint8, device="cuda")
    o, lse = fa.fwd_paged_prefix(x.q, x.k_pages, x.v_pages, x.table, x.seq_lens, cu, x.prefix_pages,
                                 max_q=n, out=x.out, lse=x.lse, workspace=ws)
    assert fa.device_status() == (fa.FA_ERR_PAGE, 301)
    for rows in (slice(24, 32), slice(80, 82)):
        assert torch.all(o[rows] == 7.0) and torch.all(lse[rows] == 7.0)


def test_a_prefix_call_without_a_prefix_is_refused():
    x = Batch(8, 2, 128, 16, [60, 70], [2, 1], seed=15)
    with pytest.raises(ValueError, match="prefix_pages"):
        fa.fwd_paged_prefix(*x.args(), None, out=x.out, lse=x.lse)
    with pytest.raises(RuntimeError, match="fa_fwd_paged_prefix"):  # an empty one
        fa.fwd_paged_prefix(*x.args(), x.prefix_pages, out=x.out, lse=x.lse)
    assert torch.all(x.out == 7.0) and torch.all(x.lse == 7.0)
    fa.check_device_status()


def append(T, cu, lens, d=64):
    """Appends T rows of ones; returns the status and how many (row, key/value
    head) pairs were written."""
    B = len(lens)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    kp = torch.zeros(4 * B, 2, 16, d, dtype=torch.bfloat16, device="cuda")
    vp = kp.clone()
    table = torch.arange(4 * B, dtype=torch.int32, device="cuda").reshape(B, 4).contiguous()
    k = torch.ones(T, 2, d, dtype=torch.bfloat16, device="cuda")
    fa.kv_append(k, k, kp, vp, table, i32(lens), i32(cu))
    status = fa.device_status()
    assert torch.equal(kp, vp)
    return status, int(kp[..., 0].sum().item())


@pytest.mark.parametrize("T,cu", [
    (8, (0, 5, 3, 8)),               # descending between two sound ranges
    (3, (-5, 1, 2, 3)),              # beginning before the rows
    (3, (-1, 0, 2, 3)),
    (3, (0, 1, 3, 900)),             # ending past them, in a sequence of no row
    (3, (0, 1, 3, 2)),
    (3, (0, 0, 2147483647, 3)),
    (3, (0, 0, -(1 << 31), 3)),
    (1, (0, 1) + (1,) * 399 + (2,)),  # the last of more sequences than a CTA has threads
    (2, (0,) * 700 + (3, 2)),
])
def test_append_reports_every_bad_row_range(T, cu):
    status, _ = append(T, cu, (20,) * (len(cu) - 1))
    assert status == (fa.FA_ERR_PAGE, 301)


def test_append_writes_no_row_of_a_bad_range():
    # rows 0 of [-5, 1) and 2 of [2, 900) are not written, row 1 of [1, 2) is
    status, written = append(3, (-5, 1, 2, 900), (20, 20, 20))
    assert status == (fa.FA_ERR_PAGE, 301) and written == 2


@pytest.mark.parametrize("T,cu", [
    (3, (0, 1, 2, 3)), (3, (1, 1, 2, 2)), (3, (3, 3, 3, 3)), (3, (0, 0, 0, 3)), (1, (0,) * 700 + (1,)),
    (300, tuple(range(301))),
])
def test_append_reports_no_sound_row_range(T, cu):
    status, written = append(T, cu, (20,) * (len(cu) - 1))
    assert status == (fa.FA_OK, 0) and written == 2 * (cu[-1] - cu[0])
