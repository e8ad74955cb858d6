"""Ragged paged-cache batches for the tests, and their results in 64 bits.

A batch is drawn dense per sequence and scattered into a pool of pages whose
every other slot holds NaN or infinities; table entries past a sequence's last
page hold numbers no kernel may follow.  The reference attends each sequence
on its dense keys in fp64, with an elementwise bound on the rounding errors of
a correct kernel.
"""
import math

import torch

BF16 = 2.0 ** -8   # half a step, relative
FP32 = 2.0 ** -24


class Batch:
    """lens[b] keys, nq[b] new rows of sequence b; prefix: keys all share."""

    def __init__(self, Hq, Hkv, d, page, lens, nq, seed, pad=0, prefix=0, width=None, spread=1.0,
                 device="cuda", fused=False):
        assert prefix % page == 0 and len(lens) == len(nq)
        g = torch.Generator().manual_seed(seed)
        self.Hq, self.Hkv, self.d, self.page, self.lens, self.nq = Hq, Hkv, d, page, lens, nq
        self.prefix, self.B = prefix, len(lens)
        cu = [0]
        for n in nq:
            cu.append(cu[-1] + n)
        self.cu, self.T = cu, max(cu[-1] + pad, 1)

        def randn(*shape):
            return (torch.randn(shape, generator=g) * spread).to(torch.bfloat16)

        pre_k, pre_v = randn(prefix, Hkv, d), randn(prefix, Hkv, d)
        self.keys, self.vals = [], []
        for n in lens:
            own = max(n - prefix, 0)
            m = min(n, prefix)
            self.keys.append(torch.cat([pre_k[:m], randn(own, Hkv, d)]))
            self.vals.append(torch.cat([pre_v[:m], randn(own, Hkv, d)]))
        shared = prefix // page
        counts = [max(-(-n // page) - shared, 0) for n in lens]
        pages = shared + sum(counts) + 3
        order = torch.randperm(pages, generator=g)
        width = width or max(1, shared + max(counts))
        table = torch.full((self.B, width), 1 << 30, dtype=torch.int32)
        bad = torch.tensor([math.nan, math.inf, -math.inf, math.nan]).repeat(page * d // 4)
        kp = bad.reshape(page, d).to(torch.bfloat16).expand(pages, Hkv, page, d).clone()
        vp = kp.clone()
        at = shared
        for b in range(self.B):
            ids = [int(x) for x in order[:shared]] + [int(x) for x in order[at:at + counts[b]]]
            at += counts[b]
            ids = ids[:-(-lens[b] // page)] if lens[b] < prefix else ids
            table[b, :len(ids)] = torch.tensor(ids, dtype=torch.int32)
            for i, pg in enumerate(ids):
                lo, hi = i * page, min((i + 1) * page, lens[b])
                kp[pg, :, :hi - lo] = self.keys[b][lo:hi].transpose(0, 1)
                vp[pg, :, :hi - lo] = self.vals[b][lo:hi].transpose(0, 1)
        for i in range(shared):  # whole, also when every sequence is shorter
            kp[order[i]] = pre_k[i * page:(i + 1) * page].transpose(0, 1)
            vp[order[i]] = pre_v[i * page:(i + 1) * page].transpose(0, 1)
        q = randn(self.T, Hq + (2 * Hkv if fused else 0), d)
        self.q_host = q[:, :Hq]
        self.q = q.to(device)[:, :Hq]
        self.k_pages, self.v_pages = kp.to(device), vp.to(device)
        self.table = table.to(device)
        self.prefix_pages = order[:shared].to(torch.int32).to(device)
        self.seq_lens = torch.tensor(lens, dtype=torch.int32, device=device)
        self.cu_q = torch.tensor(cu, dtype=torch.int32, device=device)
        self.out = torch.full((self.T, Hq, d), 7.0, dtype=torch.bfloat16, device=device)
        self.lse = torch.full((self.T, Hq), 7.0, dtype=torch.float32, device=device)

    def args(self):
        return self.q, self.k_pages, self.v_pages, self.table, self.seq_lens, self.cu_q

    def check(self, o, lse, causal, scale):
        """Compare with the fp64 reference, element by element."""
        o, lse = o.cpu(), lse.cpu()
        assert torch.all(o[self.cu[-1]:] == 7.0) and torch.all(lse[self.cu[-1]:] == 7.0)
        for b in range(self.B):
            t0, n, L = self.cu[b], self.nq[b], self.lens[b]
            if n == 0:
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
    # absolute sum, as is the scaled exponent (a few more for scale, maximum
    # and exponential); each probability by that and its bf16 rounding.
    es = ((d + 8) * FP32 * sa).amax(-1) if L else torch.zeros(Hkv, G, n, dtype=torch.float64)
    es = es + 8 * FP32 * (1 + lse.abs().clamp(max=1e4))
    bound_o = (BF16 + 2 * es[..., None] + (L + 64) * FP32) * av + (BF16 + 4 * FP32) * o.abs() + 1e-30
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
