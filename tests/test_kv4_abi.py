"""The entry points of the 4-bit cache and of a cache's pages without a GPU: every
bad argument is refused with its code before a device is touched."""
import ctypes
import math
import re
import struct

import pytest
import torch

from io_aware_exact_02_gb300 import build, fa

FAKE = 1 << 20  # a 16-byte aligned non-null address; never dereferenced


@pytest.fixture(scope="module")
def lib():
    build.build()
    return fa.load()


def expect_device(call):
    # Valid arguments reach the device check.  Only without a GPU: with one the
    # call would launch kernels on addresses that are none.
    if not torch.cuda.is_available():
        assert call() == fa.FA_ERR_DEVICE


APPEND = dict(q=FAKE, k=FAKE, v=FAKE, q_out=FAKE + 4096, pages=FAKE, table=FAKE, lens=FAKE, cu=FAKE,
              rope=FAKE, T=3, B=2, Hq=4, Hkv=2, d=64, qs=256, ks=128, vs=128, qos=256, n=8, page=16,
              width=4, rd=64, rl=64, inter=0, k_scale=1.0, v_scale=0.5)


def append(lib, **kw):
    a = dict(APPEND, **kw)
    f = ctypes.c_float
    return lib.fa_kv4_append(a["q"], a["k"], a["v"], a["q_out"], a["pages"], a["table"], a["lens"],
                             a["cu"], a["rope"], a["T"], a["B"], a["Hq"], a["Hkv"], a["d"], a["qs"],
                             a["ks"], a["vs"], a["qos"], a["n"], a["page"], a["width"], a["rd"],
                             a["rl"], a["inter"], f(a["k_scale"]), f(a["v_scale"]), None)


BAD_SCALES = [0.0, -1.0, math.nan, math.inf, 1e-45]


@pytest.mark.parametrize("kw", [
    dict(k=None), dict(v=None), dict(pages=None), dict(table=None), dict(lens=None), dict(cu=None),
    dict(q=None), dict(q_out=None), dict(T=0), dict(B=0), dict(Hq=0), dict(Hkv=0), dict(n=0),
    dict(width=0), dict(page=0), dict(page=8), dict(page=48), dict(page=512), dict(rd=24),
    dict(rd=-16), dict(rd=80), dict(rope=None), dict(rd=0), dict(rl=0), dict(inter=2), dict(qs=248),
    dict(ks=120), dict(vs=132), dict(qos=8), dict(qs=260), dict(q_out=FAKE, qos=264),
    dict(n=1 << 30, Hkv=4, ks=256, vs=256), dict(width=1 << 28, page=256), dict(T=1 << 30),
    *[dict(k_scale=x) for x in BAD_SCALES], *[dict(v_scale=x) for x in BAD_SCALES]])
def test_append_argument_errors(lib, kw):
    assert append(lib, **kw) == fa.FA_ERR_ARG


def test_append_other_errors(lib):
    assert append(lib, d=96) == fa.FA_ERR_UNSUPPORTED_D
    for name in ("q", "k", "v", "q_out", "pages", "rope"):
        assert append(lib, **{name: FAKE + 8}) == fa.FA_ERR_ALIGN
    for name in ("table", "lens", "cu"):
        assert append(lib, **{name: FAKE + 2}) == fa.FA_ERR_ALIGN
    expect_device(lambda: append(lib))
    expect_device(lambda: append(lib, q=None, q_out=None, Hq=0, qs=0, qos=0))
    expect_device(lambda: append(lib, rope=None, rd=0, rl=0))


READ = dict(k=FAKE, v=FAKE, pages=FAKE, table=FAKE, lens=FAKE, cu=FAKE, T=3, B=2, Hkv=2, d=64,
            ks=128, vs=128, n=8, page=16, width=4, k_scale=1.0, v_scale=1.0)


def read(lib, **kw):
    a = dict(READ, **kw)
    f = ctypes.c_float
    return lib.fa_kv4_read(a["k"], a["v"], a["pages"], a["table"], a["lens"], a["cu"], a["T"], a["B"],
                           a["Hkv"], a["d"], a["ks"], a["vs"], a["n"], a["page"], a["width"],
                           f(a["k_scale"]), f(a["v_scale"]), None)


@pytest.mark.parametrize("kw", [
    dict(k=None), dict(v=None), dict(pages=None), dict(table=None), dict(lens=None), dict(cu=None),
    dict(T=0), dict(B=0), dict(Hkv=0), dict(n=0), dict(width=0), dict(page=24), dict(ks=120),
    dict(vs=129), dict(n=1 << 30, Hkv=4, ks=256, vs=256), *[dict(k_scale=x) for x in BAD_SCALES]])
def test_read_errors(lib, kw):
    assert read(lib, **kw) == fa.FA_ERR_ARG


def test_read_other_errors(lib):
    assert read(lib, d=48) == fa.FA_ERR_UNSUPPORTED_D
    for name in ("k", "v", "pages"):
        assert read(lib, **{name: FAKE + 8}) == fa.FA_ERR_ALIGN
    for name in ("table", "lens", "cu"):
        assert read(lib, **{name: FAKE + 2}) == fa.FA_ERR_ALIGN
    expect_device(lambda: read(lib))


PAGED = dict(q=FAKE, pages=FAKE, o=FAKE, lse=FAKE, table=FAKE, lens=FAKE, cu=FAKE, T=3, B=2, Hq=4,
             Hkv=2, d=64, qs=256, n=8, page=16, width=4, max_q=2, causal=1, scale=0.125, k_scale=1.0,
             v_scale=1.0, ws=FAKE, wsb=1 << 40)


def paged(lib, **kw):
    a = dict(PAGED, **kw)
    f = ctypes.c_float
    return lib.fa_fwd_paged4(a["q"], a["pages"], a["o"], a["lse"], a["table"], a["lens"], a["cu"],
                             a["T"], a["B"], a["Hq"], a["Hkv"], a["d"], a["qs"], a["n"], a["page"],
                             a["width"], a["max_q"], a["causal"], f(a["scale"]), f(a["k_scale"]),
                             f(a["v_scale"]), a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw", [
    dict(q=None), dict(pages=None), dict(o=None), dict(lse=None), dict(table=None), dict(lens=None),
    dict(cu=None), dict(T=0), dict(B=0), dict(Hq=0), dict(Hkv=0), dict(Hq=3), dict(Hq=258, qs=1 << 16),
    dict(n=0), dict(width=0), dict(page=8), dict(page=100), dict(qs=248), dict(qs=260), dict(max_q=0),
    dict(causal=2), dict(scale=math.nan), dict(scale=math.inf), dict(n=1 << 30, Hkv=4),
    dict(T=1 << 30), dict(scale=1e30, k_scale=1e30), *[dict(k_scale=x) for x in BAD_SCALES],
    *[dict(v_scale=x) for x in BAD_SCALES]])
def test_paged_argument_errors(lib, kw):
    assert paged(lib, **kw) == fa.FA_ERR_ARG


def test_paged_other_errors(lib):
    assert paged(lib, d=32) == fa.FA_ERR_UNSUPPORTED_D
    for name in ("q", "pages", "o", "lse"):
        assert paged(lib, **{name: FAKE + 8}) == fa.FA_ERR_ALIGN
    for name in ("table", "lens", "cu"):
        assert paged(lib, **{name: FAKE + 1}) == fa.FA_ERR_ALIGN
    need = lib.fa_fwd_paged4_workspace_size(3, 2, 4, 2, 64, 2)
    assert need > 0
    assert paged(lib, ws=None) == fa.FA_ERR_WORKSPACE
    assert paged(lib, wsb=need - 1) == fa.FA_ERR_WORKSPACE
    assert paged(lib, ws=FAKE + 16) == fa.FA_ERR_WORKSPACE
    expect_device(lambda: paged(lib, wsb=need))
    assert lib.fa_fwd_paged4_workspace_size(0, 2, 4, 2, 64, 2) == 0
    assert lib.fa_fwd_paged4_workspace_size(3, 2, 4, 2, 72, 2) == 0
    # Room for tiles: only where a sequence may have more than 1,024 rows of a head.
    best = lib.fa_fwd_paged4_best_workspace_size
    assert best(3, 2, 4, 2, 64, 16, 4, 2) == need
    assert best(3, 2, 4, 2, 72, 16, 4, 2) == best(3, 2, 4, 2, 64, 24, 4, 2) == 0
    def room(T, B, max_pages, max_q):
        return best(T, B, 4, 2, 64, 16, max_pages, max_q) - lib.fa_fwd_paged4_workspace_size(
            T, B, 4, 2, 64, max_q)
    assert room(512, 2, 40, 512) == 0
    # All sequences of more than 24 rows,
    assert room(513, 2, 40, 513) == 256 + 10 * 65536
    assert room(49, 9, 40, 49) == 0
    assert room(600, 100, 40, 513) == 512 + 24 * 5 * 65536
    # those of more than 512 where that is beyond the bound, as far as the bound goes.
    assert room(1538, 100, 16 * 256, 513) == 512 + 2 * 512 * 65536
    assert room(1539, 100, 16 * 256, 513) == 512 + 3 * 512 * 65536
    assert room(1539, 100, 1 << 26, 513) == 512 + (512 << 20)


def words(fmt, *args):
    return struct.pack(fmt, *args)


@pytest.mark.parametrize("name,fmt,args,strides", [
    ("fa_kv4_append_words", "=9Q5q4q6q2dQ",
     [FAKE] * 9 + [3, 2, 4, 2, 64, 256, 128, 128, 256, 8, 16, 4, 64, 32, 0, 1.0, 1.0, 0],
     (14, 15, 16, 17)),
    ("fa_kv4_read_words", "=6Q4q2q3q2dQ",
     [FAKE] * 6 + [3, 2, 2, 64, 128, 128, 8, 16, 4, 1.0, 1.0, 0], (10, 11)),
    ("fa_fwd_paged4_words", "=7Q5qq5q3dQQQ",
     [FAKE] * 7 + [3, 2, 4, 2, 64, 256, 8, 16, 4, 2, 1, 0.125, 1.0, 1.0, FAKE, 1 << 40, 0], (12,))])
def test_words(lib, name, fmt, args, strides):
    call = getattr(lib, name)
    n = len(args)
    expect_device(lambda: call(words(fmt, *args), n))
    for wrong in (0, -1, n - 1, n + 1):
        assert call(words(fmt, *args) + bytes(64), wrong) == fa.FA_ERR_ARG
    assert call(None, n) == fa.FA_ERR_ARG
    kinds = "".join(c * int(k or 1) for k, c in re.findall(r"(\d*)([Qqd])", fmt))
    assert len(kinds) == n
    pointers = kinds.index("q")
    for i, kind in enumerate(kinds):
        if kind == "q" and i not in strides:  # an int that only fits 64 bits
            assert call(words(fmt, *args[:i], (1 << 32) + args[i], *args[i + 1:]), n) == fa.FA_ERR_ARG
            assert call(words(fmt, *args[:i], -1, *args[i + 1:]), n) in (
                fa.FA_ERR_ARG, fa.FA_ERR_UNSUPPORTED_D)
        elif kind == "Q" and i < pointers:
            assert call(words(fmt, *args[:i], FAKE + 1, *args[i + 1:]), n) == fa.FA_ERR_ALIGN, i
        elif kind == "d":
            assert call(words(fmt, *args[:i], math.nan, *args[i + 1:]), n) == fa.FA_ERR_ARG


# ------------------------------------------------------------------- pages

PAGES = dict(a=FAKE, b=FAKE, n=3, table=FAKE, lens=FAKE, refs=FAKE, rows=6, width=4, pages=8, page=16,
             pools=[FAKE, FAKE + 4096], sizes=[256, 64], ws=FAKE, wsb=1 << 30)


def pools_of(a):
    if a["pools"] is None:
        return None, None, 2
    n = len(a["pools"])
    return struct.pack("%dQ" % n, *a["pools"]), struct.pack("%dQ" % n, *a["sizes"]), n


def fork(lib, **kw):
    a = dict(PAGES, **kw)
    at, sizes, n = pools_of(a)
    return lib.fa_pages_fork(a["a"], a["b"], a["n"], a["table"], a["lens"], a["refs"], a["rows"],
                             a["width"], a["pages"], a["page"], at, sizes, n, a["ws"], a["wsb"], None)


def free(lib, **kw):
    a = dict(PAGES, **kw)
    return lib.fa_pages_free(a["a"], a["n"], a["table"], a["lens"], a["refs"], a["rows"], a["width"],
                             a["pages"], a["page"], None)


def compact(lib, **kw):
    a = dict(PAGES, **kw)
    at, sizes, n = pools_of(a)
    return lib.fa_pages_compact(a["table"], a["lens"], a["refs"], a["rows"], a["width"], a["pages"],
                                a["page"], at, sizes, n, kw.get("live", FAKE), a["ws"], a["wsb"], None)


def copy(lib, **kw):
    a = dict(PAGES, **kw)
    at, sizes, n = pools_of(a)
    return lib.fa_pages_copy(at, sizes, n, a["a"], a["b"], a["n"], a["pages"], None)


TABLES = [dict(table=None), dict(lens=None), dict(refs=None), dict(rows=0), dict(rows=-1),
          dict(width=0), dict(pages=0), dict(page=0), dict(page=8), dict(page=24), dict(page=512),
          dict(width=1 << 28, page=256)]
POOLS = [dict(pools=None), dict(pools=[FAKE, 0]), dict(sizes=[256, 0]), dict(sizes=[1 << 31, 64]),
         dict(pools=[FAKE] * 257, sizes=[16] * 257)]


@pytest.mark.parametrize("call,bad", [
    (fork, TABLES + POOLS + [dict(a=None), dict(b=None), dict(n=0), dict(n=-1)]),
    (free, TABLES + [dict(a=None), dict(n=0)]), (compact, TABLES + POOLS),
    (copy, POOLS + [dict(a=None), dict(b=None), dict(n=0), dict(pages=0)])])
def test_pages_argument_errors(lib, call, bad):
    for kw in bad:
        assert call(lib, **kw) == fa.FA_ERR_ARG, kw
    expect_device(lambda: call(lib))
    expect_device(lambda: call(lib, pools=[], sizes=[]))
    expect_device(lambda: call(lib, pools=[FAKE] * 256, sizes=[16] * 256))


def test_pages_alignment_and_workspace(lib):
    for call in (fork, compact, copy):
        assert call(lib, pools=[FAKE, FAKE + 8]) == fa.FA_ERR_ALIGN
        assert call(lib, sizes=[256, 40]) == fa.FA_ERR_ALIGN
    for call, names in ((fork, ("a", "b", "table", "lens", "refs")), (copy, ("a", "b")),
                        (free, ("a", "table", "lens", "refs")),
                        (compact, ("table", "lens", "refs", "live"))):
        for name in names:
            assert call(lib, **{name: FAKE + 2}) == fa.FA_ERR_ALIGN
    for call, need in ((fork, lib.fa_pages_fork_workspace_size(8, 3)),
                       (compact, lib.fa_pages_compact_workspace_size(8))):
        assert need > 0
        assert call(lib, ws=None) == fa.FA_ERR_WORKSPACE
        assert call(lib, wsb=need - 1) == fa.FA_ERR_WORKSPACE
        assert call(lib, ws=FAKE + 16) == fa.FA_ERR_WORKSPACE
        expect_device(lambda: call(lib, wsb=need))
    assert lib.fa_pages_fork_workspace_size(0, 3) == 0
    assert lib.fa_pages_fork_workspace_size(8, 0) == 0
    assert lib.fa_pages_compact_workspace_size(0) == 0


def test_binding_refuses_host_tensors_and_shapes():
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    pages = torch.zeros(3, 2, 16 * 72, dtype=torch.uint8)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        fa.kv4_append(x, x, pages, i[None], i, i)
    with pytest.raises(ValueError, match="CUDA"):
        fa.kv4_read(pages, i[None], i, i, x, x)
    with pytest.raises(ValueError, match="CUDA"):
        fa.fwd_paged4(x, pages, i[None], i, i)
    with pytest.raises(ValueError, match="page_table"):
        fa.pages_fork(i, i, i[None], i, i, pages[None], 16)
    with pytest.raises(ValueError, match="page_table"):
        fa.pages_free(i, i[None], i, i, 16)
    with pytest.raises(ValueError, match="page_table"):
        fa.pages_compact(i[None], i, i, pages[None], 16)
    with pytest.raises(ValueError, match="src"):
        fa.pages_copy(i, i, pages[None])


def test_pool_of_a_cache():
    t = fa.kv4_pages(5, 2, 32, 128, device="cpu")
    assert t.shape == (5, 2, 32 * 144) and t.dtype == torch.uint8
