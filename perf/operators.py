"""Cases of the paged key/value cache operators: appending to the cache with the
position rotation, attention over the cache, and attention for a batch that
shares a prefix.

Each operator has a plain form in elementary torch operations (``own`` false)
and the framework's call (``own`` true).  All of them work on token-major
packed rows: sequence b's new tokens are rows cu_q[b] .. cu_q[b+1]-1 of q, k
and v; seq_lens[b] counts its keys with the new ones included; page_table[b]
lists its pages, each a (Hkv, page_size, d) block of the cache.  Rows at and
past cu_q[B] are padding and stay as they were.
"""
import math
import random

import torch

own = False

# ---------------------------------------------------------------- the cases
#
# op       "append", "paged" or "prefix"
# B, Hq, Hkv, d, page      batch, query heads, key/value heads, head size, page size
# len      the longest sequence, new tokens included; "even" makes all equal,
#          otherwise lengths are spread over [len/4, len]
# nq       new tokens of a sequence; "few" > 0: only that many sequences have
#          nq of them and the others one (a mixed prefill and decode batch)
# prefix   keys at the start that all sequences share (op "prefix")
# rope     rotated channels, "interleaved" the pairing; fused: q, k and v are
#          slices of one projection's output
# pad      padding rows behind the last sequence's


def _case(name, op, B, Hq, Hkv, d, page, len, nq=1, few=0, even=False, causal=True, prefix=0,
          rope=0, interleaved=False, fused=False, pad=0, mix=1):
    return dict(name=name, op=op, B=B, Hq=Hq, Hkv=Hkv, d=d, page=page, len=len, nq=nq, few=few,
                even=even, causal=causal, prefix=prefix, rope=rope, interleaved=interleaved,
                fused=fused, pad=pad, mix=mix)


def listed():
    return [
        # One user's next token: the smallest append, all latency.
        _case("append_one", "append", 1, 32, 8, 128, 16, 1000, rope=128, even=True),
        # A full decode batch's step, q, k and v slices of the fused projection.
        _case("append_decode_b256", "append", 256, 32, 8, 128, 16, 300, rope=128, fused=True),
        # Prompts of a batch going into an empty cache.
        _case("append_prompts", "append", 16, 32, 8, 128, 64, 1024, nq=1024, even=True, rope=128,
              fused=True, mix=3),
        # Short heads, half of the channels rotated in neighbouring pairs, odd sizes, padding rows.
        _case("append_d64_partial", "append", 7, 12, 12, 64, 32, 777, nq=333, rope=32,
              interleaved=True, pad=5),
        # One user's next token over a short context: the smallest attention.
        _case("decode_b1_1000", "paged", 1, 32, 8, 128, 16, 1000, even=True),
        # A decode batch of uneven contexts in small pages.
        _case("decode_b64_4k", "paged", 64, 32, 8, 128, 16, 4096, mix=5),
        # The library's decode workload, its keys in pages.
        _case("decode_b8_32k", "paged", 8, 32, 8, 128, 64, 32768, even=True),
        # Short heads without groups, four speculated tokens each.
        _case("verify_d64", "paged", 33, 16, 16, 64, 32, 2049, nq=4, mix=2, pad=3),
        # Chunks of long prompts over what the cache holds already.
        _case("prefill_chunks", "paged", 4, 32, 8, 128, 128, 4096, nq=1024, even=True),
        # Two prompt chunks among decoding users, one call.
        _case("mixed_batch", "paged", 32, 32, 8, 128, 16, 2500, nq=500, few=2, mix=7),
        # A serving batch behind one long document.
        _case("prefix_b64_16k", "prefix", 64, 32, 8, 128, 64, 16384 + 500, prefix=16384, mix=4),
        # A batch behind a system prompt, short heads, an odd group.
        _case("prefix_b24_2k", "prefix", 24, 15, 5, 64, 16, 2048 + 200, prefix=2048, mix=9),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "paged", "paged", "prefix"])
    d = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 3, 4, 8, 16])
    Hq = Hkv * rng.choice([1, 2, 3, 4, 5, 6, 8, 16] if Hkv < 8 else [1, 2, 3, 4, 8])
    page = rng.choice([16, 32, 64, 128, 256])
    mix = rng.randrange(1, 1 << 20)
    if op == "append":
        nq = rng.choice([1, 1, 3, _log(rng, 2, 1024)])
        B = min(_log(rng, 1, 256), max(1, 16384 // nq))
        length = max(nq, _log(rng, 1, 1024))
        while B * Hkv * length * d > 16 * 8 * 1024 * 128 or B * nq * Hq * d > 16384 * 32 * 128:
            B, length, nq = max(1, B // 2), max(1, length * 3 // 4), max(1, nq * 3 // 4)
        return _case("", op, B, Hq, Hkv, d, page, max(length, nq), nq=nq, rope=rng.choice([d, d, d // 2, 0]),
                     interleaved=rng.random() < 0.4, fused=rng.random() < 0.5,
                     pad=rng.choice([0, 0, 7]), mix=mix)
    if op == "prefix":
        prefix = max(1, _log(rng, 500, 16384) // page) * page
        suffix = _log(rng, 1, 600)
        B = _log(rng, 2, 64)
        nq = min(rng.choice([1, 1, 1, 2, 5]), suffix)
        while B * Hkv * (prefix + suffix) * d > 64 * 8 * 16884 * 128 or Hq * nq > 256:
            B, nq = max(2, B * 3 // 4), 1
            Hkv, Hq = (Hkv, Hq) if B > 2 else (1, Hq // Hkv)
        return _case("", op, B, Hq, Hkv, d, page, prefix + suffix, nq=nq, prefix=prefix,
                     pad=rng.choice([0, 0, 4]), mix=mix)
    length = _log(rng, 1, 32768)
    nq = min(length, rng.choice([1, 1, 2, 7, _log(rng, 1, 1024)]))
    B = _log(rng, 1, 128)
    while B * Hkv * length * d > 8 * 8 * 32768 * 128 or B * Hq * nq * length > 4 * 32 * 1024 * 4096:
        B, nq, length = (B * 3 // 4, nq, length) if B > 1 else (B, max(1, nq // 2), length * 3 // 4)
        nq = min(nq, length)
    few = rng.choice([0, 0, 1]) if nq > 1 and B > 2 else 0
    return _case("", op, B, Hq, Hkv, d, page, length, nq=nq, few=few,
                 even=rng.random() < 0.3, causal=rng.random() < 0.8, fused=rng.random() < 0.3,
                 pad=rng.choice([0, 0, 6]), mix=mix)


def _lengths(case):
    """(new tokens, keys) of every sequence, from the case alone."""
    rng = random.Random(case["mix"])
    B, length, nq, prefix = case["B"], case["len"], case["nq"], case["prefix"]
    n = [nq] * B
    if case["few"]:
        n = [nq if b < case["few"] else 1 for b in range(B)]
        rng.shuffle(n)
    lens = []
    for b in range(B):
        lo = max(n[b], prefix + n[b], prefix + (length - prefix) // 4)
        lens.append(length if case["even"] else rng.randint(min(lo, length), length))
    lens[0] = length
    return n, lens


def work(case):
    n, lens = _lengths(case)
    T, Hq, Hkv, d = sum(n), case["Hq"], case["Hkv"], case["d"]
    if case["op"] == "append":
        moved = 2 * T * (Hq + 2 * Hkv) * d * 2
        table = 4 * T * case["rope"] + 4 * (T + 2 * case["B"] + 1)
        return {"bytes": moved + table, "flops": 3 * T * (Hq + Hkv) * case["rope"]}
    keys = case["prefix"] + sum(x - case["prefix"] for x in lens)
    # token i of sequence b sees len - n + i + 1 keys under the causal mask
    seen = sum(m * x - (m * (m - 1) // 2 if case["causal"] else 0) for m, x in zip(n, lens))
    moved = 2 * keys * Hkv * d * 2 + 2 * T * Hq * d * 2 + 4 * T * Hq
    moved += 4 * (-(-keys // case["page"]) + 2 * case["B"] + 1)
    return {"bytes": moved, "flops": 4 * d * Hq * seen}


# ---------------------------------------------------------------- the inputs


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    n, lens = _lengths(case)
    B, Hq, Hkv, d, page = case["B"], case["Hq"], case["Hkv"], case["d"], case["page"]
    cu = [0]
    for m in n:
        cu.append(cu[-1] + m)
    T = cu[-1] + case["pad"]

    def randn(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(torch.bfloat16)

    s = dict(case=case, max_q=max(n), max_len=max(lens),
             cu_q=torch.tensor(cu, dtype=torch.int32, device="cuda"),
             seq_lens=torch.tensor(lens, dtype=torch.int32, device="cuda"))
    # The cache: a shared prefix's pages first in every table, then each
    # sequence's own, all of them scattered over the pool.
    shared = case["prefix"] // page
    counts = [-(-(x - case["prefix"]) // page) for x in lens]
    pages = shared + sum(counts)
    perm = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    width = shared + max(counts)
    index, at = [], shared
    for c in counts:
        own_pages = list(range(at, at + c))
        index.append(list(range(shared)) + own_pages + [0] * (width - shared - c))
        at += c
    s["page_table"] = perm[torch.tensor(index, device="cuda")].contiguous()
    s["prefix_pages"] = perm[:shared].contiguous()
    s["k_pages"] = randn(pages, Hkv, page, d)
    s["v_pages"] = randn(pages, Hkv, page, d)
    if case["fused"] or case["op"] == "append":
        qkv = randn(T, Hq + 2 * Hkv, d)
        s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        if not case["fused"]:
            s["q"], s["k"], s["v"] = (x.contiguous() for x in (s["q"], s["k"], s["v"]))
    else:
        s["q"] = randn(T, Hq, d)
    # Written by the calls; the padding rows keep what is here.
    s["out"] = torch.zeros((T, Hq, d), dtype=torch.bfloat16, device="cuda")
    s["lse"] = torch.zeros((T, Hq), dtype=torch.float32, device="cuda")
    s["rope"] = None
    if case["rope"]:
        half = case["rope"] // 2
        freq = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)
        angle = torch.arange(max(lens), dtype=torch.float64, device="cuda")[:, None] * freq
        s["rope"] = torch.cat([angle.cos(), angle.sin()], 1).to(torch.float32)
    return s


# ---------------------------------------------------------------- one pass


def run(s):
    op = s["case"]["op"]
    if own:
        from io_aware_exact_02_gb300 import fa
        if op == "append":
            q = fa.kv_append(s["k"], s["v"], s["k_pages"], s["v_pages"], s["page_table"],
                             s["seq_lens"], s["cu_q"], q=s["q"], q_out=s["out"], rope=s["rope"],
                             interleaved=s["case"]["interleaved"])
            return {"q": q, "k_pages": s["k_pages"], "v_pages": s["v_pages"]}
        if op == "prefix":
            o, lse = fa.fwd_paged_prefix(s["q"], s["k_pages"], s["v_pages"], s["page_table"],
                                         s["seq_lens"], s["cu_q"], s["prefix_pages"],
                                         max_q=s["max_q"], causal=s["case"]["causal"],
                                         out=s["out"], lse=s["lse"])
        else:
            o, lse = fa.fwd_paged(s["q"], s["k_pages"], s["v_pages"], s["page_table"],
                                  s["seq_lens"], s["cu_q"], max_q=s["max_q"],
                                  causal=s["case"]["causal"], out=s["out"], lse=s["lse"])
        return {"o": o, "lse": lse}
    return _append(s) if op == "append" else _attend(s)


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
    return torch.cat([turned, x[..., rope:]], -1).to(torch.bfloat16)


def _append(s):
    case = s["case"]
    page, rope, pad = case["page"], case["rope"], case["pad"]
    t, valid, b, pos = _tokens(s)
    q, k, v = s["q"], s["k"], s["v"]
    if rope:
        cs = s["rope"][pos.clamp(0, s["max_len"] - 1)]
        q, k = _rotate(q, cs, rope, case["interleaved"]), _rotate(k, cs, rope, case["interleaved"])
    m = t.numel() - pad  # the padding rows are not written
    at, slot = s["page_table"].long()[b, pos.clamp(min=0) // page][:m], (pos % page)[:m]
    s["k_pages"][at, :, slot] = k[:m]
    s["v_pages"][at, :, slot] = v[:m]
    s["out"][:m] = q[:m]
    return {"q": s["out"], "k_pages": s["k_pages"], "v_pages": s["v_pages"]}


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
    keys = lambda c: c[table].transpose(1, 2).reshape(B, Hkv, -1, d)[:, :, :L].float()  # noqa: E731
    score = q @ keys(s["k_pages"]).transpose(-1, -2) * (1.0 / math.sqrt(d))
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
    o = (p @ keys(s["v_pages"])) / total.clamp(min=1e-30)
    lse = (top + total.log()).squeeze(-1)
    o = o.view(B, Hkv, G, n, d).permute(0, 3, 1, 2, 4).reshape(B, n, Hkv * G, d)
    lse = lse.view(B, Hkv, G, n).permute(0, 3, 1, 2).reshape(B, n, Hkv * G)
    place = (t - cu[b]).clamp(0, n - 1)
    o = torch.where(valid[:, None, None], o[b, place].to(torch.bfloat16), s["out"])
    lse = torch.where(valid[:, None], lse[b, place], s["lse"])
    return {"o": o, "lse": lse}


# ---------------------------------------------------------------- in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    n, lens = _lengths(case)
    if case["op"] == "append":
        half, rope = case["rope"] // 2, case["rope"]
        q_out, kp, vp = s["out"].double(), s["k_pages"].double(), s["v_pages"].double()
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
            pages = s["page_table"][b].long()[pos // case["page"]]
            q_out[rows] = new[0]
            kp[pages, :, pos % case["page"]] = new[1]
            vp[pages, :, pos % case["page"]] = s["v"][rows].double()
            row += n[b]
        return {"q": q_out, "k_pages": kp, "v_pages": vp}
    if work(case)["flops"] > 4e12:
        return None
    G, d = case["Hq"] // case["Hkv"], case["d"]
    o = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device="cuda")
    row = 0
    for b in range(case["B"]):
        pages = s["page_table"][b, :-(-lens[b] // case["page"])].long()
        mask = None
        if case["causal"] and n[b] > 1:
            mask = torch.ones(n[b], lens[b], dtype=torch.bool, device="cuda").tril(lens[b] - n[b])
        for h in range(case["Hkv"]):
            k = s["k_pages"][pages, h].reshape(-1, d)[:lens[b]].double()
            v = s["v_pages"][pages, h].reshape(-1, d)[:lens[b]].double()
            heads = slice(h * G, (h + 1) * G)
            q = s["q"][row:row + n[b], heads].double().transpose(0, 1)
            x = torch.matmul(q, k.T) / math.sqrt(d)
            if mask is not None:
                x = torch.where(mask, x, torch.full_like(x, -math.inf))
            lse[row:row + n[b], heads] = torch.logsumexp(x, -1).T
            o[row:row + n[b], heads] = torch.matmul(torch.softmax(x, -1), v).transpose(0, 1)
        row += n[b]
    return {"o": o, "lse": lse}
