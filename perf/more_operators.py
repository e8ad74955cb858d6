"""Cases of the operators around a paged key/value cache held in 4 bits and of
the operators on a cache's pages: appending to the 4-bit cache (with the
position rotation) and reading rows back, attention over it, forking sequences
copy-on-write and freeing them, and compacting a pool.

Each operator has a plain form in elementary torch operations (``own`` false)
and the framework's call (``own`` true).

The 4-bit cache: uint8 (num_pages, Hkv, page_size * 9 d / 8).  A page's keys
come in blocks of 16, 18 d bytes each: K codes [16 keys][d/2] (a byte holds
channels 2i, low, and 2i+1); V codes [2 halves of 8 keys][8 eighths of the
channels][4 key pairs][d/8 channels] (a byte holds keys 2i, low, and 2i+1); K
scales [16 keys][d/16]; V scales [d/16][16 keys].  A code is an E2M1 number, a
scale an E4M3 number for 16 channels of a key; a value is code * scale * the
tensor's own scale.
"""
import math
import random

import torch

own = False

# ---------------------------------------------------------------- the cases
#
# op       "append4", "attn4", "fork" or "compact"
# B, Hq, Hkv, d, page      batch, query heads, key/value heads, head size, page size
# len      the longest sequence, new tokens included; "even" makes all equal,
#          otherwise lengths are spread over [len/4, len]
# nq       new tokens of a sequence; "few" > 0: only that many sequences have
#          nq of them and the others one (a mixed prefill and decode batch)
# rope     rotated channels, "interleaved" the pairing; fused: q, k and v are
#          slices of one projection's output
# pad      padding rows behind the last sequence's
# ks, vs   the tensors' own scales
# layers   caches of the model (fork, compact), bits: 16 (keys and values
#          apart) or 4 (together); kids: children of a sequence (fork)
# live     per cent of the pages in use (compact)


def _case(name, op, B, Hkv, d, page, len, Hq=1, nq=1, few=0, even=False, causal=True, rope=0,
          interleaved=False, fused=False, pad=0, ks=1.0, vs=1.0, layers=1, bits=4, kids=1, live=50,
          mix=1):
    return dict(name=name, op=op, B=B, Hq=Hq, Hkv=Hkv, d=d, page=page, len=len, nq=nq, few=few,
                even=even, causal=causal, rope=rope, interleaved=interleaved, fused=fused, pad=pad,
                ks=ks, vs=vs, layers=layers, bits=bits, kids=kids, live=live, mix=mix)


def listed():
    return [
        # One user's next token: the smallest append, all latency.
        _case("append4_one", "append4", 1, 8, 128, 16, 1000, Hq=32, rope=128, even=True),
        # A full decode batch's step, q, k and v slices of the fused projection.
        _case("append4_decode_b256", "append4", 256, 8, 128, 16, 300, Hq=32, rope=128, fused=True,
              vs=0.0625),
        # Prompts of a batch going into an empty cache.
        _case("append4_prompts", "append4", 16, 8, 128, 64, 1024, Hq=32, nq=1024, even=True,
              rope=128, fused=True, mix=3),
        # One user's next token over a short context: the smallest attention.
        _case("attn4_b1_1000", "attn4", 1, 8, 128, 16, 1000, Hq=32, even=True),
        # A decode batch of uneven contexts in small pages.
        _case("attn4_b64_4k", "attn4", 64, 8, 128, 16, 4096, Hq=32, mix=5, ks=0.7713, vs=0.0613),
        # The library's decode workload, its keys in 4 bits.
        _case("attn4_b8_32k", "attn4", 8, 8, 128, 64, 32768, Hq=32, even=True),
        # Short heads without groups, four speculated tokens each, odd sizes, padding rows.
        _case("attn4_verify_d64", "attn4", 33, 16, 64, 32, 2049, Hq=16, nq=4, mix=2, pad=3),
        # Chunks of long prompts over what the cache holds already.
        _case("attn4_chunks", "attn4", 4, 8, 128, 128, 4096, Hq=32, nq=1024, even=True),
        # One user's answer in four variants: few children, one page each, all latency.
        _case("fork_answers", "fork", 2, 8, 128, 16, 1000, layers=4, kids=4),
        # A beam step of a decode batch, every layer's keys and values.
        _case("fork_beams", "fork", 64, 8, 128, 16, 700, layers=8, bits=16, kids=4, mix=4),
        # A small pool after a few answers ended.
        _case("compact_small", "compact", 12, 8, 128, 16, 400, layers=4, live=60),
        # A serving pool of which half was freed, to be shrunk.
        _case("compact_pool", "compact", 64, 8, 128, 16, 900, layers=8, bits=16, live=50, mix=6),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append4", "attn4", "attn4", "attn4", "fork", "compact"])
    d = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 3, 4, 8, 16])
    Hq = Hkv * rng.choice([1, 2, 3, 4, 5, 6, 8, 16] if Hkv < 8 else [1, 2, 3, 4, 8])
    page = rng.choice([16, 32, 64, 128, 256])
    mix = rng.randrange(1, 1 << 20)
    ks, vs = rng.choice([1.0, 1.0, 0.7713, 4.0]), rng.choice([1.0, 1.0, 0.0613, 0.5])
    if op in ("fork", "compact"):
        bits, page = rng.choice([4, 16]), min(page, 64)
        layers = _log(rng, 1, 16)
        B, length, kids = _log(rng, 1, 64), _log(rng, 1, 900), rng.choice([1, 2, 4])
        while True:
            case = _case("", op, B, Hkv, d, page, length, layers=layers, bits=bits, kids=kids,
                         live=rng.choice([20, 50, 80]), mix=mix)
            pages = _fork_pages(case) if op == "fork" else _fragments(case)[1]
            if (work(case)["bytes"] < (250e6 if op == "fork" else 1.1e9) and B * kids <= 256
                    and pages * _pool(case)[0] < 2.5e9):
                return case
            B, layers, length = max(1, B * 3 // 4), max(1, layers * 3 // 4), max(1, length * 3 // 4)
    if op == "append4":
        nq = rng.choice([1, 1, 3, _log(rng, 2, 1024)])
        B = min(_log(rng, 1, 256), max(1, 16384 // nq))
        length = max(nq, _log(rng, 1, 1024))
        while B * Hkv * length * d > 16 * 8 * 1024 * 128 or B * nq * Hq * d > 16384 * 32 * 128:
            B, length, nq = max(1, B // 2), max(1, length * 3 // 4), max(1, nq * 3 // 4)
        return _case("", op, B, Hkv, d, page, max(length, nq), Hq=Hq, nq=nq,
                     rope=rng.choice([d, d, d // 2, 16, 0]), interleaved=rng.random() < 0.4,
                     fused=rng.random() < 0.5, pad=rng.choice([0, 0, 7]), ks=ks, vs=vs, mix=mix)
    length = _log(rng, 1, 32768)
    nq = min(length, rng.choice([1, 1, 2, 7, _log(rng, 1, 1024)]))
    B = _log(rng, 1, 128)
    while B * Hkv * length * d > 8 * 8 * 32768 * 128 or B * Hq * nq * length > 4 * 32 * 1024 * 4096:
        B, nq, length = (B * 3 // 4, nq, length) if B > 1 else (B, max(1, nq // 2), length * 3 // 4)
        nq = min(nq, length)
    few = rng.choice([0, 0, 1]) if nq > 1 and B > 2 else 0
    return _case("", op, B, Hkv, d, page, length, Hq=Hq, nq=nq, few=few, even=rng.random() < 0.3,
                 causal=rng.random() < 0.8, fused=rng.random() < 0.3, pad=rng.choice([0, 0, 6]),
                 ks=ks, vs=vs, mix=mix)


def _lengths(case):
    """(new tokens, keys) of every sequence, from the case alone."""
    rng = random.Random(case["mix"])
    B, length, nq = case["B"], case["len"], case["nq"]
    n = [nq] * B
    if case["few"]:
        n = [nq if b < case["few"] else 1 for b in range(B)]
        rng.shuffle(n)
    lens = []
    for b in range(B):
        lo = max(n[b], length // 4)
        lens.append(length if case["even"] else rng.randint(min(lo, length), length))
    lens[0] = length
    return n, lens


def _pool(case):
    """(bytes of a page in all caches, elements of a page in one, caches)."""
    el = case["Hkv"] * case["page"] * case["d"]
    if case["bits"] == 16:
        return 4 * el * case["layers"], el, 2 * case["layers"]
    return el * 9 // 8 * case["layers"], el * 9 // 8, case["layers"]


def _moves(case):
    """Of op compact: (pages in all, those in use, those that move)."""
    used, pages, _, _ = _fragments(case)
    live = len(used)
    return pages, live, sum(x >= live for x in used)


def _fragments(case):
    """A fragmented pool: its pages in use (ascending), their number in all, and
    the sequences' lengths and pages; some pages belong to two sequences."""
    rng = random.Random(case["mix"])
    _, lens = _lengths(case)
    counts = [-(-x // case["page"]) for x in lens]
    total = max(sum(counts) + 1, sum(counts) * 100 // case["live"])
    ids = rng.sample(range(total), sum(counts))
    tables, at = [], 0
    for b, c in enumerate(counts):
        t = ids[at:at + c]
        at += c
        if b % 3 == 2:  # a fork: its first whole pages are the sequence before's
            k = min(c, counts[b - 1], lens[b] // case["page"]) // 2
            t[:k] = tables[b - 1][:k]
        tables.append(t)
    return sorted({x for t in tables for x in t}), total, lens, tables


def work(case):
    n, lens = _lengths(case)
    T, B, Hq, Hkv, d, page = sum(n), case["B"], case["Hq"], case["Hkv"], case["d"], case["page"]
    if case["op"] == "fork":
        # Read and written: each child's last page, the tables' rows, the
        # reference counts (the children's pages' also when they are freed).
        parts = sum(x % page > 0 for x in lens) * case["kids"]
        ids = sum(-(-x // page) for x in lens)
        entries = ids + 5 * case["kids"] * ids + _fork_pages(case)
        return {"bytes": 2 * parts * _pool(case)[0] + 4 * entries, "flops": 0}
    if case["op"] == "compact":
        pages, live, moves = _moves(case)
        ids = sum(-(-x // page) for x in lens)
        return {"bytes": 2 * moves * _pool(case)[0] + 4 * (2 * pages + 2 * ids), "flops": 0}
    if case["op"] == "append4":
        moved = T * d * (4 * Hq + 2 * 2 * Hkv + 2 * 2 * Hkv)  # q in and out, k, v in, read back
        cache = 2 * 2 * T * Hkv * d * 9 // 16                 # written, and read back
        table = 4 * T * case["rope"] + 4 * (T + 2 * B + 1)
        return {"bytes": moved + cache + table,
                "flops": 3 * T * (Hq + Hkv) * case["rope"] + 6 * 2 * T * Hkv * d}
    keys = sum(lens)
    # token i of sequence b sees len - n + i + 1 keys under the causal mask
    seen = sum(m * x - (m * (m - 1) // 2 if case["causal"] else 0) for m, x in zip(n, lens))
    moved = keys * Hkv * d * 9 // 8 + 2 * T * Hq * d * 2 + 4 * T * Hq
    moved += 4 * (-(-keys // page) + 2 * B + 1)
    return {"bytes": moved, "flops": 4 * d * Hq * seen}


def _fork_pages(case):
    _, lens = _lengths(case)
    return (sum(-(-x // case["page"]) for x in lens) + case["B"] * case["kids"]) * 5 // 4 + 8


# ---------------------------------------------------------------- the inputs

_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _quantize(x, scale):
    """Codes (int32) and scales (E4M3) of x (..., d) fp32, groups of 16 channels."""
    y = (x * torch.tensor(1.0 / scale, dtype=torch.float32, device=x.device)).unflatten(-1, (-1, 16))
    top = y.abs().amax(-1)
    # (By a tensor: a division by a number may be a product with its rounded inverse.)
    s = (top / torch.full_like(top, 6.0)).clamp(max=448.0).to(torch.float8_e4m3fn)
    wide = s.float()[..., None]
    m = torch.where(wide > 0, y / wide, torch.zeros_like(y))
    a = m.abs()
    # To the nearest of 0, .5, 1, 1.5, 2, 3, 4, 6; a tie to the even code.
    code = ((a > 0.25).int() + (a >= 0.75).int() + (a > 1.25).int() + (a >= 1.75).int()
            + (a > 2.5).int() + (a >= 3.5).int() + (a > 5.0).int())
    return (code + 8 * (m < 0).int()).flatten(-2), s


def _values(code, s, scale, d):
    """The values of codes (..., d) with their scales (..., d / 16), fp32."""
    lut = torch.tensor(_E2M1 + [-x for x in _E2M1], dtype=torch.float32, device=code.device)
    return (lut[code.int()].unflatten(-1, (-1, 16)) * s.float()[..., None]).flatten(-2) * scale


def _pack(kc, ks, vc, vs, d):
    """Blocks (..., 18 d) of 16 keys' codes (..., 16, d) and scales (..., 16, d / 16)."""
    k = kc[..., 0::2] | kc[..., 1::2] << 4
    v = vc.unflatten(-2, (2, 4, 2)).unflatten(-1, (8, -1))  # half, pair, key; eighth, channel
    v = (v[..., 0, :, :] | v[..., 1, :, :] << 4).transpose(-3, -2)  # half, eighth, pair, channel
    return torch.cat([k.to(torch.uint8).flatten(-2), v.to(torch.uint8).flatten(-4),
                      ks.view(torch.uint8).flatten(-2),
                      vs.view(torch.uint8).transpose(-1, -2).flatten(-2)], -1)


def _unpack(blocks, d):
    """(K codes, K scales, V codes, V scales) of blocks (..., 18 d), by key."""
    k = blocks[..., :8 * d].unflatten(-1, (16, d // 2))
    k = torch.stack([k & 15, k >> 4], -1).flatten(-2)
    v = blocks[..., 8 * d:16 * d].unflatten(-1, (2, 8, 4, d // 8))
    v = torch.stack([v & 15, v >> 4], -1)                    # half, eighth, pair, channel, key
    v = v.permute(*range(v.dim() - 5), -5, -3, -1, -4, -2)   # half, pair, key, eighth, channel
    v = v.flatten(-2).flatten(-4, -2)
    ks = blocks[..., 16 * d:17 * d].unflatten(-1, (16, d // 16)).contiguous().view(torch.float8_e4m3fn)
    vs = blocks[..., 17 * d:].unflatten(-1, (d // 16, 16)).transpose(-1, -2)
    return k, ks, v, vs.contiguous().view(torch.float8_e4m3fn)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    if case["op"] in ("fork", "compact"):
        return _prepare_pool(case, g)
    n, lens = _lengths(case)
    B, Hq, Hkv, d, page = case["B"], case["Hq"], case["Hkv"], case["d"], case["page"]
    cu = [0]
    for m in n:
        cu.append(cu[-1] + m)
    T = cu[-1] + case["pad"]

    def randn(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)

    s = dict(case=case, max_q=max(n), max_len=max(lens),
             cu_q=torch.tensor(cu, dtype=torch.int32, device="cuda"),
             seq_lens=torch.tensor(lens, dtype=torch.int32, device="cuda"))
    # Each sequence's pages, scattered over the pool.
    counts = [-(-x // page) for x in lens]
    pages, width = sum(counts), max(counts)
    perm = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    index, at = [], 0
    for c in counts:
        index.append(list(range(at, at + c)) + [0] * (width - c))
        at += c
    s["page_table"] = perm[torch.tensor(index, device="cuda")].contiguous()
    # The keys held: normal values at the tensors' scales, a few channels larger.
    loud = 1.0 + 3.0 * (torch.rand(Hkv, 1, 1, d, generator=g, device="cuda") < 0.05).float()
    pool = torch.empty((pages, Hkv, page // 16, 18 * d), dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 26) // (Hkv * page * d))
    for i in range(0, pages, step):
        shape = (min(step, pages - i), Hkv, page // 16, 16, d)
        kc, ks = _quantize(randn(*shape) * loud * case["ks"], case["ks"])
        vc, vs = _quantize(randn(*shape) * case["vs"], case["vs"])
        pool[i:i + step] = _pack(kc, ks, vc, vs, d)
    s["pages"] = pool.flatten(2)
    half = lambda *shape: randn(*shape).to(torch.bfloat16)  # noqa: E731
    if case["op"] == "append4":
        scales = torch.cat([torch.ones(Hq), torch.full((Hkv,), case["ks"]), torch.full((Hkv,), case["vs"])])
        qkv = (randn(T, Hq + 2 * Hkv, d) * scales.to("cuda")[:, None]).to(torch.bfloat16)
        s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        if not case["fused"]:
            s["q"], s["k"], s["v"] = (x.contiguous() for x in (s["q"], s["k"], s["v"]))
        s["k_out"] = torch.zeros((T, Hkv, d), dtype=torch.bfloat16, device="cuda")
        s["v_out"] = torch.zeros((T, Hkv, d), dtype=torch.bfloat16, device="cuda")
    else:
        s["q"] = half(T, Hq + 2 * Hkv, d)[:, :Hq] if case["fused"] else half(T, Hq, d)
    # Written by the calls; the padding rows keep what is here.
    s["out"] = torch.zeros((T, Hq, d), dtype=torch.bfloat16, device="cuda")
    s["lse"] = torch.zeros((T, Hq), dtype=torch.float32, device="cuda")
    s["rope"] = None
    if case["rope"]:
        half_dim = case["rope"] // 2
        freq = 10000.0 ** (-torch.arange(half_dim, dtype=torch.float64, device="cuda") / half_dim)
        angle = torch.arange(max(lens), dtype=torch.float64, device="cuda")[:, None] * freq
        s["rope"] = torch.cat([angle.cos(), angle.sin()], 1).to(torch.float32)
    return s


def _prepare_pool(case, g):
    B, kids = case["B"], case["kids"]
    _, el, caches = _pool(case)
    s = dict(case=case)
    if case["op"] == "fork":
        _, lens = _lengths(case)
        counts = [-(-x // case["page"]) for x in lens]
        pages, width = _fork_pages(case), max(counts) + 1
        perm = torch.randperm(pages, generator=g, device="cuda").tolist()
        at, tables = 0, []
        for c in counts:
            tables.append(perm[at:at + c])
            at += c
        lens, tables = lens + [0] * (B * kids), tables + [[]] * (B * kids)
        s["parents"] = torch.arange(B, dtype=torch.int32, device="cuda").repeat_interleave(kids)
        order = torch.randperm(B * kids, generator=g, device="cuda").to(torch.int32)
        s["children"] = B + order
    else:
        _, pages, lens, tables = _fragments(case)
        width = max(len(t) for t in tables)
    refs = [0] * pages
    for t in tables:
        for x in t:
            refs[x] += 1
    # The bookkeeping in one piece: the page table, the lengths, the reference counts.
    rows = len(tables)
    flat = [x for t in tables for x in t + [0] * (width - len(t))] + lens + refs
    s["start"] = torch.tensor(flat, dtype=torch.int32, device="cuda")
    s["book"] = s["start"].clone()
    s["page_table"] = s["book"][:rows * width].view(rows, width)
    s["seq_lens"] = s["book"][rows * width:rows * width + rows]
    s["refs"] = s["book"][rows * width + rows:]
    if case["bits"] == 16:
        shape = (caches, pages, case["Hkv"], case["page"], case["d"])
        s["cache"] = torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)
    else:
        shape = (caches, pages, case["Hkv"], el // case["Hkv"])
        s["cache"] = torch.randint(0, 256, shape, generator=g, device="cuda", dtype=torch.uint8)
    return s


# ---------------------------------------------------------------- one pass


def run(s):
    case = s["case"]
    op = case["op"]
    if op == "compact":
        # The pool as it was: a pass has the same pages to move.
        s["book"].copy_(s["start"])
    if own:
        from io_aware_exact_02_gb300 import fa
        if op == "append4":
            q = fa.kv4_append(s["k"], s["v"], s["pages"], s["page_table"], s["seq_lens"], s["cu_q"],
                              q=s["q"], q_out=s["out"], rope=s["rope"],
                              interleaved=case["interleaved"], k_scale=case["ks"],
                              v_scale=case["vs"])
            k, v = fa.kv4_read(s["pages"], s["page_table"], s["seq_lens"], s["cu_q"],
                               k_out=s["k_out"], v_out=s["v_out"], k_scale=case["ks"],
                               v_scale=case["vs"])
            return {"q": q, "k": k, "v": v}
        if op == "attn4":
            o, lse = fa.fwd_paged4(s["q"], s["pages"], s["page_table"], s["seq_lens"], s["cu_q"],
                                   max_q=s["max_q"], causal=case["causal"], k_scale=case["ks"],
                                   v_scale=case["vs"], out=s["out"], lse=s["lse"])
            return {"o": o, "lse": lse}
        if op == "fork":
            fa.pages_fork(s["parents"], s["children"], s["page_table"], s["seq_lens"], s["refs"],
                          s["cache"], case["page"])
            fa.pages_free(s["children"], s["page_table"], s["seq_lens"], s["refs"], case["page"])
        else:
            fa.pages_compact(s["page_table"], s["seq_lens"], s["refs"], s["cache"], case["page"])
        return {"page_table": s["page_table"], "seq_lens": s["seq_lens"], "refs": s["refs"],
                "cache": s["cache"]}
    return {"append4": _append, "attn4": _attend, "fork": _fork, "compact": _compact}[op](s)


def _tokens(s):
    """Each row's sequence (B for padding rows) and position."""
    cu, lens, B = s["cu_q"].long(), s["seq_lens"].long(), s["case"]["B"]
    t = torch.arange(s["q"].shape[0], device="cuda")
    b = (t[:, None] >= cu[None, 1:]).sum(1)
    bb = b.clamp(max=B - 1)
    return t, b < B, bb, lens[bb] - (cu[bb + 1] - t)


def _rotate(x, cs, rope, interleaved):
    x = x.float()
    half = rope // 2
    c, sn = cs[:, None, :half], cs[:, None, half:]
    if interleaved:
        a, b = x[..., 0:rope:2], x[..., 1:rope:2]
        turned = torch.stack([a * c - b * sn, a * sn + b * c], -1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:rope]
        turned = torch.cat([a * c - b * sn, a * sn + b * c], -1)
    return torch.cat([turned, x[..., rope:]], -1)


def _append(s):
    case = s["case"]
    page, rope, d, Hkv = case["page"], case["rope"], case["d"], case["Hkv"]
    t, valid, b, pos = _tokens(s)
    q, k = s["q"].float(), s["k"].float()
    if rope:
        cs = s["rope"][pos.clamp(0, s["max_len"] - 1)]
        q, k = _rotate(q, cs, rope, case["interleaved"]), _rotate(k, cs, rope, case["interleaved"])
    m = t.numel() - case["pad"]  # the padding rows are not written
    kc, ks = _quantize(k[:m], case["ks"])
    vc, vs = _quantize(s["v"][:m].float(), case["vs"])
    s["k_out"][:m] = _values(kc, ks, case["ks"], d).to(torch.bfloat16)
    s["v_out"][:m] = _values(vc, vs, case["vs"], d).to(torch.bfloat16)
    s["out"][:m] = q[:m].to(torch.bfloat16)
    # Into the blocks of the rows' 16 keys.
    at, slot = s["page_table"].long()[b, pos.clamp(min=0) // page][:m], (pos % page)[:m]
    block = s["pages"].view(-1, Hkv, page // 16, 18 * d)
    blk, r = slot // 16, slot % 16
    i = lambda n: torch.arange(n, device="cuda")  # noqa: E731
    head, where = i(Hkv)[None, :, None], (at[:, None, None], blk[:, None, None], r[:, None, None])
    block[where[0], head, where[1], where[2] * (d // 2) + i(d // 2)] = \
        (kc[..., 0::2] | kc[..., 1::2] << 4).to(torch.uint8)
    block[where[0], head, where[1], 16 * d + where[2] * (d // 16) + i(d // 16)] = ks.view(torch.uint8)
    block[where[0], head, where[1], 17 * d + i(d // 16) * 16 + where[2]] = vs.view(torch.uint8)
    # A byte of V holds two keys: each adds what its own half changes by.
    c, eighth = i(d), d // 8
    byte = 8 * d + ((where[2] // 8 * 8 + c // eighth) * 4 + where[2] % 8 // 2) * eighth + c % eighth
    shift = where[2] % 2 * 4
    old = block[where[0], head, where[1], byte].int() >> shift & 15
    change = ((vc - old) * 2 ** shift).to(torch.uint8)
    place = ((where[0] * Hkv + head) * (page // 16) + where[1]) * (18 * d) + byte
    s["pages"].view(-1).index_put_((place.reshape(-1),), change.reshape(-1), accumulate=True)
    return {"q": s["out"], "k": s["k_out"], "v": s["v_out"]}


def _attend(s):
    case = s["case"]
    B, Hkv, d, L, n = case["B"], case["Hkv"], case["d"], s["max_len"], s["max_q"]
    G = case["Hq"] // Hkv
    t, valid, b, pos = _tokens(s)
    cu, lens, table = s["cu_q"].long(), s["seq_lens"].long(), s["page_table"].long()
    # Every sequence's queries and keys, padded to the longest.
    i = torch.arange(n, device="cuda")
    row = (cu[:B, None] + i).clamp(max=t.numel() - 1)
    q = s["q"].float()[row].view(B, n, Hkv, G, d).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * n, d)
    blocks = s["pages"][table].transpose(1, 2).reshape(B, Hkv, -1, 18 * d)
    kc, ks, vc, vs = _unpack(blocks, d)
    keys = _values(kc, ks, case["ks"], d).flatten(2, 3)[:, :, :L]
    score = q @ keys.transpose(-1, -2) * (1.0 / math.sqrt(d))
    j = torch.arange(L, device="cuda")
    if case["causal"]:
        limit = (lens - (cu[1:] - cu[:B]))[:, None] + i + 1
    else:
        limit = lens[:, None].expand(B, n)
    seen = (j < limit[..., None])[:, None, None].expand(B, 1, G, n, L).reshape(B, 1, G * n, L)
    score = score.masked_fill(~seen, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - top.clamp(min=-1e30))
    total = p.sum(-1, keepdim=True)
    o = (p @ _values(vc, vs, case["vs"], d).flatten(2, 3)[:, :, :L]) / total.clamp(min=1e-30)
    lse = (top + total.log()).squeeze(-1)
    o = o.view(B, Hkv, G, n, d).permute(0, 3, 1, 2, 4).reshape(B, n, Hkv * G, d)
    lse = lse.view(B, Hkv, G, n).permute(0, 3, 1, 2).reshape(B, n, Hkv * G)
    place = (t - cu[b]).clamp(0, n - 1)
    o = torch.where(valid[:, None, None], o[b, place].to(torch.bfloat16), s["out"])
    lse = torch.where(valid[:, None], lse[b, place], s["lse"])
    return {"o": o, "lse": lse}


def _fork(s):
    page, table, lens, refs = s["case"]["page"], s["page_table"], s["seq_lens"], s["refs"]
    parent, child = s["parents"].long(), s["children"].long()
    col = torch.arange(table.shape[1], device="cuda")
    length = lens[parent]
    whole, part = (length // page).long(), length % page > 0
    shared, ids = col < whole[:, None], table[parent]
    # The n-th child that needs a page of its own gets the n-th lowest free one.
    free = (refs == 0).nonzero()[:, 0]
    dst = free[:int(part.sum())]
    src = ids[part, whole[part]].long()
    s["cache"][:, dst] = s["cache"][:, src]
    table[child] = torch.where(shared, ids, table[child])
    table[child[part], whole[part]] = dst.int()
    refs.index_add_(0, ids.long().flatten(), shared.int().flatten())
    refs[dst] = 1
    lens[child] = length
    # Freed again: every page of the children counts one less.
    held = col < ((lens[child] + page - 1) // page)[:, None]
    refs.index_add_(0, table[child].long().flatten(), -held.int().flatten())
    lens[child] = 0
    return {"page_table": table, "seq_lens": lens, "refs": refs, "cache": s["cache"]}


def _compact(s):
    page, table, lens, refs = s["case"]["page"], s["page_table"], s["seq_lens"], s["refs"]
    used = refs != 0
    live = int(used.sum())
    # The k-th highest page in use past the first `live` goes to the k-th lowest hole.
    dst = (~used[:live]).nonzero()[:, 0]
    src = used[live:].nonzero()[:, 0].flip(0) + live
    s["cache"][:, dst] = s["cache"][:, src]
    new = torch.arange(refs.numel(), device="cuda")
    new[src] = dst
    refs[dst] = refs[src]
    refs[live:] = 0
    col = torch.arange(table.shape[1], device="cuda")
    held = col < ((lens + page - 1) // page)[:, None]
    table.copy_(torch.where(held, new[table.long()].int(), table))
    return {"page_table": table, "seq_lens": lens, "refs": refs, "cache": s["cache"]}


# ---------------------------------------------------------------- in 64 bits


def _round_e4m3(x):
    """x (fp64, >= 0) to the nearest E4M3 number: 3 bits behind the leading one,
    steps of 2^-9 below 2^-6, 448 the largest."""
    e = torch.frexp(x.clamp(min=2.0 ** -6, max=500.0)).exponent - 1  # -6 .. 8
    step = torch.tensor([2.0 ** i for i in range(-9, 6)], dtype=x.dtype, device=x.device)[e.long() + 6]
    return (torch.round(x / step) * step).clamp(max=448.0)


def _as_held(x, scale):
    """What the 4-bit cache holds of x (..., d) fp64."""
    y = x.unflatten(-1, (-1, 16)) / torch.full_like(x[..., :1, None], scale)
    top = y.abs().amax(-1, keepdim=True)
    s = _round_e4m3(top / torch.full_like(top, 6.0))
    m = torch.where(s > 0, y / s, torch.zeros_like(y))
    a = m.abs()
    # Steps of 1/2 up to 2, of 1 up to 4, of 2 up to 6.
    step = torch.where(a < 2.0, 0.5, torch.where(a < 4.0, 1.0, 2.0)).to(a.dtype)
    near = (torch.round(a / step) * step).clamp(max=6.0)
    return (torch.copysign(near, m) * s * scale).flatten(-2)


def exact(case, seed):
    if case["op"] in ("fork", "compact"):
        return None
    s = prepare(case, seed)
    n, lens = _lengths(case)
    d, Hkv = case["d"], case["Hkv"]
    if case["op"] == "append4":
        half, rope = case["rope"] // 2, case["rope"]
        q_out, k_out, v_out = s["out"].double(), s["k_out"].double(), s["v_out"].double()
        row = 0
        for b in range(case["B"]):
            rows = slice(row, row + n[b])
            pos = torch.arange(lens[b] - n[b], lens[b], device="cuda")
            new = []
            for x in (s["q"][rows].double(), s["k"][rows].double()):
                y = x.clone()
                if rope:
                    first = torch.arange(half, device="cuda") * (2 if case["interleaved"] else 1)
                    second = first + (1 if case["interleaved"] else half)
                    angle = torch.complex(s["rope"][pos, :half].double(), s["rope"][pos, half:].double())
                    z = torch.complex(x[..., first], x[..., second]) * angle[:, None]
                    y[..., first], y[..., second] = z.real, z.imag
                new.append(y)
            q_out[rows] = new[0]
            k_out[rows] = _as_held(new[1], case["ks"])
            v_out[rows] = _as_held(s["v"][rows].double(), case["vs"])
            row += n[b]
        return {"q": q_out, "k": k_out, "v": v_out}
    if work(case)["flops"] > 4e12:
        return None
    G, page = case["Hq"] // Hkv, case["page"]
    o = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device="cuda")
    magnitude = torch.tensor([0, 1, 2, 3, 4, 6, 8, 12], dtype=torch.float64, device="cuda") / 2

    def number(code):
        return torch.where(code >= 8, -1.0, 1.0) * magnitude[(code % 8).long()]

    def scale(byte):
        e, m = (byte // 8).double(), (byte % 8).double()
        return torch.where(e > 0, (1 + m / 8) * 2.0 ** (e - 7), m / 8 * 2.0 ** -6)

    row = 0
    for b in range(case["B"]):
        ids = s["page_table"][b, :-(-lens[b] // page)].long()
        mask = None
        if case["causal"] and n[b] > 1:
            mask = torch.ones(n[b], lens[b], dtype=torch.bool, device="cuda").tril(lens[b] - n[b])
        for h in range(Hkv):
            blk = s["pages"][ids, h].reshape(-1, 18 * d)
            N = blk.shape[0] * 16
            bytes_ = blk[:, :8 * d].reshape(N, d // 2)
            k = torch.empty(N, d, dtype=torch.float64, device="cuda")
            k[:, 0::2], k[:, 1::2] = number(bytes_ % 16), number(bytes_ // 16)
            k *= scale(blk[:, 16 * d:17 * d].reshape(N, d // 16)).repeat_interleave(16, 1) * case["ks"]
            bytes_ = blk[:, 8 * d:16 * d].reshape(-1, 2, 8, 4, d // 8).permute(0, 1, 3, 2, 4).reshape(N // 2, d)
            v = torch.empty(N, d, dtype=torch.float64, device="cuda")
            v[0::2], v[1::2] = number(bytes_ % 16), number(bytes_ // 16)
            vs = scale(blk[:, 17 * d:].reshape(-1, d // 16, 16)).permute(0, 2, 1).reshape(N, d // 16)
            v *= vs.repeat_interleave(16, 1) * case["vs"]
            k, v = k[:lens[b]], v[:lens[b]]
            heads = slice(h * G, (h + 1) * G)
            q = s["q"][row:row + n[b], heads].double().transpose(0, 1)
            x = torch.matmul(q, k.T) / math.sqrt(d)
            if mask is not None:
                x = torch.where(mask, x, torch.full_like(x, -math.inf))
            lse[row:row + n[b], heads] = torch.logsumexp(x, -1).T
            o[row:row + n[b], heads] = torch.matmul(torch.softmax(x, -1), v).transpose(0, 1)
        row += n[b]
    return {"o": o, "lse": lse}
