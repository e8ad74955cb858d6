"""The paged-cache entry points without a GPU: every bad argument is refused
with its code before a device is touched, and the binding's own checks."""
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


APPEND = dict(q=FAKE, k=FAKE, v=FAKE, q_out=FAKE + 4096, kp=FAKE, vp=FAKE, table=FAKE, lens=FAKE,
              cu=FAKE, rope=FAKE, T=3, B=2, Hq=4, Hkv=2, d=64, qs=256, ks=128, vs=128, qos=256,
              pages=8, page=16, width=4, rd=64, rl=64, inter=0)


def append(lib, **kw):
    a = dict(APPEND, **kw)
    return lib.fa_kv_append(a["q"], a["k"], a["v"], a["q_out"], a["kp"], a["vp"], a["table"],
                            a["lens"], a["cu"], a["rope"], a["T"], a["B"], a["Hq"], a["Hkv"],
                            a["d"], a["qs"], a["ks"], a["vs"], a["qos"], a["pages"], a["page"],
                            a["width"], a["rd"], a["rl"], a["inter"], None)


@pytest.mark.parametrize("kw", [
    dict(k=None), dict(v=None), dict(kp=None), dict(vp=None), dict(table=None), dict(lens=None),
    dict(cu=None), dict(q=None), dict(q_out=None), dict(T=0), dict(B=0), dict(Hq=0), dict(Hkv=0),
    dict(pages=0), dict(width=0), dict(page=0), dict(page=8), dict(page=48), dict(page=512),
    dict(rd=24), dict(rd=-16), dict(rd=80), dict(rope=None), dict(rd=0), dict(rl=0),
    dict(inter=2), dict(qs=248), dict(ks=120), dict(vs=132), dict(qos=8), dict(qs=260),
    dict(q_out=FAKE, qos=264), dict(pages=1 << 30, Hkv=4, ks=256, vs=256),
    dict(width=1 << 28, page=256), dict(T=1 << 30)])
def test_append_argument_errors(lib, kw):
    assert append(lib, **kw) == fa.FA_ERR_ARG


def test_append_other_errors(lib):
    assert append(lib, d=96) == fa.FA_ERR_UNSUPPORTED_D
    for name in ("q", "k", "v", "q_out", "kp", "vp", "rope"):
        assert append(lib, **{name: FAKE + 8}) == fa.FA_ERR_ALIGN
    for name in ("table", "lens", "cu"):
        assert append(lib, **{name: FAKE + 2}) == fa.FA_ERR_ALIGN
    expect_device(lambda: append(lib))
    expect_device(lambda: append(lib, q=None, q_out=None, Hq=0, qs=0, qos=0))
    expect_device(lambda: append(lib, rope=None, rd=0, rl=0))
    expect_device(lambda: append(lib, q_out=FAKE))


PAGED = dict(q=FAKE, kp=FAKE, vp=FAKE, o=FAKE, lse=FAKE, table=FAKE, lens=FAKE, cu=FAKE, pre=FAKE,
             P=32, T=3, B=2, Hq=4, Hkv=2, d=64, qs=256, pages=8, page=16, width=4, max_q=2,
             causal=1, scale=0.125, ws=FAKE, wsb=1 << 40)


def paged(lib, prefix, **kw):
    a = dict(PAGED, **kw)
    head = [a["q"], a["kp"], a["vp"], a["o"], a["lse"], a["table"], a["lens"], a["cu"]]
    tail = [a["T"], a["B"], a["Hq"], a["Hkv"], a["d"], a["qs"], a["pages"], a["page"], a["width"],
            a["max_q"], a["causal"], ctypes.c_float(a["scale"]), a["ws"], a["wsb"], None]
    if prefix:
        return lib.fa_fwd_paged_prefix(*head, a["pre"], a["P"], *tail)
    return lib.fa_fwd_paged(*head, *tail)


@pytest.mark.parametrize("prefix", [False, True])
@pytest.mark.parametrize("kw", [
    dict(q=None), dict(kp=None), dict(vp=None), dict(o=None), dict(lse=None), dict(table=None),
    dict(lens=None), dict(cu=None), dict(T=0), dict(B=0), dict(Hq=0), dict(Hkv=0), dict(Hq=3),
    dict(Hq=258, qs=1 << 16), dict(pages=0), dict(width=0), dict(page=8), dict(page=100),
    dict(qs=248), dict(qs=260), dict(max_q=0), dict(causal=2), dict(scale=float("nan")),
    dict(scale=float("inf")), dict(pages=1 << 30, Hkv=4), dict(T=1 << 30)])
def test_paged_argument_errors(lib, prefix, kw):
    assert paged(lib, prefix, **kw) == fa.FA_ERR_ARG


@pytest.mark.parametrize("prefix", [False, True])
def test_paged_other_errors(lib, prefix):
    assert paged(lib, prefix, d=32) == fa.FA_ERR_UNSUPPORTED_D
    for name in ("q", "kp", "vp", "o", "lse"):
        assert paged(lib, prefix, **{name: FAKE + 8}) == fa.FA_ERR_ALIGN
    for name in ("table", "lens", "cu"):
        assert paged(lib, prefix, **{name: FAKE + 1}) == fa.FA_ERR_ALIGN
    expect_device(lambda: paged(lib, prefix))


def test_prefix_errors(lib):
    for kw in (dict(pre=None), dict(P=0), dict(P=24), dict(P=-16), dict(P=80)):
        assert paged(lib, True, **kw) == fa.FA_ERR_ARG
    assert paged(lib, True, pre=FAKE + 2) == fa.FA_ERR_ALIGN


def test_paged_workspace_is_checked(lib):
    for prefix, P in ((False, 0), (True, 32)):
        need = lib.fa_fwd_paged_workspace_size(3, 2, 4, 2, 64, 2, P)
        if need:
            assert paged(lib, prefix, ws=None) == fa.FA_ERR_WORKSPACE
            assert paged(lib, prefix, wsb=need - 1) == fa.FA_ERR_WORKSPACE
            assert paged(lib, prefix, ws=FAKE + 16) == fa.FA_ERR_WORKSPACE
        expect_device(lambda: paged(lib, prefix, wsb=need))
    assert lib.fa_fwd_paged_workspace_size(0, 2, 4, 2, 64, 2, 0) == 0
    assert lib.fa_fwd_paged_workspace_size(3, 2, 4, 2, 72, 2, 0) == 0


def test_status_string(lib):
    assert lib.fa_status_string(fa.FA_ERR_PAGE) != b"unknown status"


def test_binding_refuses_host_tensors_and_shapes():
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    pages = torch.zeros(3, 2, 16, 64, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        fa.kv_append(x, x, pages, pages, i[None], i, i)
    with pytest.raises(ValueError):
        fa.fwd_paged(x, pages, pages, i[None], i, i)


def test_rope_table_values():
    t = fa.rope_table(50, 32, base=100.0, device="cpu")
    p, i = 37, 5
    angle = p * 100.0 ** (-2 * i / 32)
    assert t.shape == (50, 32) and t.dtype == torch.float32
    ref = torch.tensor([angle], dtype=torch.float64)
    assert abs(t[p, i].item() - ref.cos().item()) <= 2.0 ** -24
    assert abs(t[p, 16 + i].item() - ref.sin().item()) <= 2.0 ** -24


# The same calls with their arguments as words.

def words(fmt, *args):
    return struct.pack(fmt, *args)


APPEND_ARGS = [FAKE] * 10 + [3, 2, 4, 2, 64] + [4 * 64, 2 * 64, 2 * 64, 4 * 64] + [8, 16, 4, 64, 32, 0] + [0]
PAGED_ARGS = [FAKE] * 8 + [3, 2, 4, 2, 64, 4 * 64, 8, 16, 4, 2, 1, 0.125, FAKE, 1 << 40, 0]
PREFIX_ARGS = [FAKE] * 9 + [32] + PAGED_ARGS[8:]


@pytest.mark.parametrize("name,fmt,args", [
    ("fa_kv_append_words", "=10Q5q4q6qQ", APPEND_ARGS),
    ("fa_fwd_paged_words", "=8Q5qq5qdQQQ", PAGED_ARGS),
    ("fa_fwd_paged_words", "=8QQq5qq5qdQQQ", PREFIX_ARGS)])
def test_words(lib, name, fmt, args):
    call = getattr(lib, name)
    n = len(args)
    expect_device(lambda: call(words(fmt, *args), n))
    for wrong in (0, -1, n - 1, n + 1, n + 2):
        if name == "fa_kv_append_words" or wrong not in (23, 25):
            assert call(words(fmt, *args) + bytes(64), wrong) == fa.FA_ERR_ARG
    assert call(None, n) == fa.FA_ERR_ARG
    kinds = "".join(c * int(k or 1) for k, c in re.findall(r"(\d*)([Qqd])", fmt))
    assert len(kinds) == n
    strides = {"fa_kv_append_words": (15, 16, 17, 18)}.get(name, (13,) if n == 23 else (15,))
    for i, kind in enumerate(kinds):
        if kind == "q" and i not in strides:  # an int that only fits 64 bits
            assert call(words(fmt, *args[:i], (1 << 32) + args[i], *args[i + 1:]), n) == fa.FA_ERR_ARG
            assert call(words(fmt, *args[:i], -1, *args[i + 1:]), n) in (
                fa.FA_ERR_ARG, fa.FA_ERR_UNSUPPORTED_D)
        elif kind == "Q" and i < 8:  # a pointer
            got = call(words(fmt, *args[:i], FAKE + 1, *args[i + 1:]), n)
            assert got == fa.FA_ERR_ALIGN, i
        elif kind == "d":
            assert call(words(fmt, *args[:i], math.nan, *args[i + 1:]), n) == fa.FA_ERR_ARG
