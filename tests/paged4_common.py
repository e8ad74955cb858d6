"""Ragged batches over a paged cache in 4 bits for the tests: the cache's numbers
and layout restated from their definition, and the attention over them in 64
bits with an elementwise bound on a correct kernel's rounding errors.

Slots that hold no key of a sequence are filled with bytes whose scale is NaN;
table entries past a sequence's last page hold numbers no kernel may follow.
"""
import math

import torch

BF16 = 2.0 ** -8   # half a step, relative
FP16 = 2.0 ** -11
FP32 = 2.0 ** -24

E2M1 = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64)


def e4m3(byte):
    """The numbers of E4M3 bytes, fp64."""
    b = byte.long() & 127
    e, m = b // 8, (b % 8).double()
    pow2 = torch.tensor([2.0 ** (k - 7) for k in range(16)], dtype=torch.float64)
    x = torch.where(e > 0, (1 + m / 8) * pow2[e], m / 8 * 2.0 ** -6)
    x = torch.where(b == 127, torch.full_like(x, math.nan), x)
    return torch.where(byte.long() >= 128, -x, x)


ALL_SCALES = e4m3(torch.arange(127))


def nearest(x, table):
    """Index of the number of the ascending table nearest to x; of two equally
    near ones the even index."""
    hi = torch.searchsorted(table, x.contiguous()).clamp(1, len(table) - 1)
    lo = hi - 1
    dl, dh = x - table[lo], table[hi] - x
    even = torch.where(lo % 2 == 0, lo, hi)
    return torch.where(dl < dh, lo, torch.where(dh < dl, hi, even))


def quantize(y):
    """Codes and scale bytes of y (..., d) fp64 (already divided by the tensor's
    scale), groups of 16."""
    g = y.unflatten(-1, (-1, 16))
    s = nearest((g.abs().amax(-1) / 6).clamp(max=448.0), ALL_SCALES)
    wide = ALL_SCALES[s][..., None]
    q = torch.where(wide > 0, g / wide, torch.zeros_like(g))
    code = nearest(q.abs().clamp(max=6.0), E2M1[:8]) + 8 * (torch.signbit(q)).long()
    return code.flatten(-2).to(torch.uint8), s.to(torch.uint8)


def values(code, scale):
    """(..., d) codes, (..., d / 16) scale bytes -> fp64 numbers."""
    return (E2M1[code.long()].unflatten(-1, (-1, 16)) * e4m3(scale)[..., None]).flatten(-2)


def put(block, r, kc, ks, vc, vs):
    """Writes key r into a block (18 d bytes, numpy-like uint8 tensor): its codes
    kc, vc (d) and scales ks, vs (d / 16)."""
    d = kc.numel()
    block[r * (d // 2):(r + 1) * (d // 2)] = kc[0::2] | kc[1::2] << 4
    e = d // 8
    for i in range(8):
        at = 8 * d + ((r // 8 * 8 + i) * 4 + r % 8 // 2) * e
        old, new = block[at:at + e], vc[i * e:(i + 1) * e]
        block[at:at + e] = (old & 15 | new << 4) if r % 2 else (old & 240 | new)
    block[16 * d + r * (d // 16):16 * d + (r + 1) * (d // 16)] = ks
    block[17 * d + r:18 * d:16] = vs


class Batch4:
    """lens[b] keys, nq[b] new rows of sequence b."""

    def __init__(self, Hq, Hkv, d, page, lens, nq, seed, pad=0, width=None, spread=1.0,
                 k_scale=1.0, v_scale=1.0, device="cuda", fused=False):
        assert len(lens) == len(nq)
        g = torch.Generator().manual_seed(seed)
        self.Hq, self.Hkv, self.d, self.page, self.lens, self.nq = Hq, Hkv, d, page, lens, nq
        self.B, self.k_scale, self.v_scale = len(lens), k_scale, v_scale
        cu = [0]
        for n in nq:
            cu.append(cu[-1] + n)
        self.cu, self.T = cu, max(cu[-1] + pad, 1)

        def randn(*shape):
            return torch.randn(shape, generator=g)

        counts = [-(-n // page) for n in lens]
        pages = sum(counts) + 3
        order = torch.randperm(pages, generator=g)
        table = torch.full((self.B, width or max(1, max(counts))), 1 << 30, dtype=torch.int32)
        pool = torch.full((pages, Hkv, page // 16, 18 * d), 255, dtype=torch.uint8)
        self.keys, self.vals = [], []
        at = 0
        for b, n in enumerate(lens):
            ids = order[at:at + counts[b]]
            at += counts[b]
            table[b, :counts[b]] = ids.to(torch.int32)
            kc, ks = quantize((randn(n, Hkv, d) * spread).double())
            vc, vs = quantize(randn(n, Hkv, d).double())
            self.keys.append(values(kc, ks) * k_scale)
            self.vals.append(values(vc, vs) * v_scale)
            # All keys of a slot of the blocks at once.
            for r in range(min(16, n)):
                j = torch.arange(r, n, 16)
                blk = pool[ids[j // page], :, j % page // 16]  # (keys, Hkv, 18 d), copied
                blk[..., r * (d // 2):(r + 1) * (d // 2)] = kc[j][..., 0::2] | kc[j][..., 1::2] << 4
                e = d // 8
                for i in range(8):
                    o = 8 * d + ((r // 8 * 8 + i) * 4 + r % 8 // 2) * e
                    old, new = blk[..., o:o + e], vc[j][..., i * e:(i + 1) * e]
                    blk[..., o:o + e] = (old & 15 | new << 4) if r % 2 else (old & 240 | new)
                blk[..., 16 * d + r * (d // 16):16 * d + (r + 1) * (d // 16)] = ks[j]
                blk[..., 17 * d + r:18 * d:16] = vs[j]
                pool[ids[j // page], :, j % page // 16] = blk
        q = randn(self.T, Hq + (2 * Hkv if fused else 0), d).to(torch.bfloat16)
        self.q_host = q[:, :Hq]
        self.q = q.to(device)[:, :Hq]
        self.pages = pool.flatten(2).contiguous().to(device)
        self.table = table.to(device)
        self.seq_lens = torch.tensor(lens, dtype=torch.int32, device=device)
        self.cu_q = torch.tensor(cu, dtype=torch.int32, device=device)
        self.out = torch.full((self.T, Hq, d), 7.0, dtype=torch.bfloat16, device=device)
        self.lse = torch.full((self.T, Hq), 7.0, dtype=torch.float32, device=device)

    def args(self):
        return self.q, self.pages, self.table, self.seq_lens, self.cu_q

    def scales(self):
        return dict(k_scale=self.k_scale, v_scale=self.v_scale)

    def check(self, o, lse, causal, scale, skip=()):
        """Compare with the 64-bit reference, element by element."""
        o, lse = o.cpu(), lse.cpu()
        assert torch.all(o[self.cu[-1]:] == 7.0) and torch.all(lse[self.cu[-1]:] == 7.0)
        for b in range(self.B):
            t0, n, L = self.cu[b], self.nq[b], self.lens[b]
            if n == 0 or b in skip:
                continue
            ref = reference(self.q_host[t0:t0 + n], self.keys[b], self.vals[b], causal, scale)
            compare(o[t0:t0 + n], lse[t0:t0 + n], ref, (b, n, L))


def reference(q, k, v, causal, scale):
    """(O, lse, bound on O, bound on lse) of q (n, Hq, d) on k, v (L, Hkv, d)."""
    n, Hq, d = q.shape
    L, Hkv = k.shape[:2]
    G = Hq // Hkv
    q = q.double().transpose(0, 1).reshape(Hkv, G, n, d)
    k, v = k.double().transpose(0, 1)[:, None], v.double().transpose(0, 1)[:, None]
    s = scale * (q @ k.transpose(-1, -2))
    sa = abs(scale) * (q.abs() @ k.abs().transpose(-1, -2))
    if causal:
        s = s.masked_fill(~torch.ones(n, L, dtype=torch.bool).tril(L - n), -math.inf)
    if L == 0:
        top = torch.full((Hkv, G, n, 1), -math.inf, dtype=torch.float64)
    else:
        top = s.amax(-1, keepdim=True)
    p = torch.exp(s - top.clamp(min=-1e300))
    total = p.sum(-1, keepdim=True)
    a = p / total.clamp(min=1e-300)
    o, av = a @ v, a @ v.abs()
    lse = (top + total.log())[..., 0]
    # An fp32 dot product of d terms is off by at most d half steps of its
    # absolute sum, as is the scaled exponent (a few more for scales, maximum
    # and exponential), and the query's channels by 2^-38 of its largest; each
    # probability by that and its fp16 rounding: half a step, or 2^-25 where it is
    # below fp16's normal range (of sums that are at least 1).
    es = ((d + 10) * FP32 * sa).amax(-1) if L else torch.zeros(Hkv, G, n, dtype=torch.float64)
    es = es + 8 * FP32 * (1 + lse.abs().clamp(max=1e4))
    small = 2.0 ** -25 * v.abs().sum(-2, keepdim=True)
    bound_o = ((FP16 + 2 * es[..., None] + (L + 64) * FP32) * av + small
               + (BF16 + 4 * FP32) * o.abs() + 1e-30)
    bound_l = 2 * es + (L + 64) * FP32 + 2.0 ** -20
    back = lambda x: x.reshape(Hq, n, *x.shape[3:]).transpose(0, 1)  # noqa: E731
    return back(o), back(lse), back(bound_o), back(bound_l)


def compare(o, lse, ref, what):
    ro, rl, bo, bl = ref
    none = torch.isneginf(rl)
    assert torch.equal(torch.isneginf(lse), none), what
    assert torch.all(o[none] == 0), what
    assert torch.isfinite(o.float()).all(), what
    do = (o.double() - ro).abs()
    worst = (do / bo).max().item()
    assert worst <= 1.0, (what, "O", worst, do.max().item())
    dl = (lse.double() - rl).abs()[~none]
    if dl.numel():
        worst = (dl / bl[~none]).max().item()
        assert worst <= 1.0, (what, "lse", worst, dl.max().item())
