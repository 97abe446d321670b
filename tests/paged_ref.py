"""float64 references (torch, CPU) of the rotary-position and paged-cache
operators, with the bounds their kernels' roundings allow.

Notation: u = finfo(type).eps / 2, the largest relative error of one rounding
to a 16-bit type."""
import math

import torch

DT = {"bf16": torch.bfloat16, "f16": torch.float16}


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def rope_ref(x, pos, inv_freq, interleaved=False, scale=1.0, sign=1.0):
    """x [..., N, D] float64, pos [..., N] integers, inv_freq [rot/2] float64."""
    r = 2 * inv_freq.numel()
    theta = pos.double()[..., None] * inv_freq.double()
    c, s = scale * torch.cos(theta), scale * sign * torch.sin(theta)
    if interleaved:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        y = torch.stack((a * c - b * s, b * c + a * s), -1).flatten(-2)
    else:
        a, b = x[..., : r // 2], x[..., r // 2:r]
        y = torch.cat((a * c - b * s, b * c + a * s), -1)
    return torch.cat((y, x[..., r:]), -1)


def rope_tol(x, ref, inv_freq, dtype, interleaved=False, scale=1.0):
    """Error allowed to a rotated value: one rounding to the type (u |y|, and half
    a step of the smallest subnormal), and the float32 part: the angle is off by at most
    2^-25 half turns (the rounding of its top 32 bits) and pi times that in
    radians, sine and cosine by 2 units in the last place, the two products and
    the sum by half a unit each, so below 2^-21 (|a| + |b|)."""
    r = 2 * inv_freq.numel()
    m = x.abs()
    if interleaved:
        ab = (m[..., 0:r:2] + m[..., 1:r:2]).repeat_interleave(2, -1)
    else:
        ab = (m[..., : r // 2] + m[..., r // 2:r]).repeat(*([1] * (x.dim() - 1)), 2)
    ab = torch.cat((ab, torch.zeros_like(m[..., r:])), -1)
    return half_step(dtype) * ref.abs() + ab * scale * 2.0 ** -21 + torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps / 2


def paged_attention_ref(q, k_cache, v_cache, table, lens, cu, causal, scale, dtype, max_q=None):
    """(o, lse, o tolerance, lse tolerance) in float64; q [H, T, D], caches
    [P, Hkv, S, D], all CPU; NaN rows are those of no sequence.  Pages outside
    the cache read as zeros.

    Tolerances.  delta bounds the error of a score: D float32 additions and
    the scaling, (D + 4) 2^-24 of the sum of the products' magnitudes; the
    maximum and the exponential add at most 2^-16 relative to a probability.  O
    then differs by twice that (numerator and denominator) and by the rounding
    of P to the type, relative to A = softmax(s) |V|, and by its own rounding.
    With float16, probabilities below 2^-14 round by up to 2^-25 each while the
    row sum is at least 1."""
    H, T, D = q.shape
    P, Hkv, S, _ = k_cache.shape
    G = H // Hkv
    o = torch.full((H, T, D), math.nan, dtype=torch.float64)
    lse = torch.full((H, T), math.nan, dtype=torch.float64)
    to, tl = torch.zeros_like(o), torch.zeros_like(lse)
    u = half_step(dtype)
    for b in range(len(lens)):
        r0, r1 = int(cu[b]), int(cu[b + 1])
        if max_q is not None:
            r1 = min(r1, r0 + max_q)
        n, t = int(lens[b]), r1 - r0
        if t <= 0:
            continue
        j = torch.arange(n)
        page = table[b].long()[j // S]
        ok = (page >= 0) & (page < P)
        page = torch.where(ok, page, 0)
        k = torch.where(ok[:, None, None], k_cache[page, :, j % S].double(), 0.0)     # [n, Hkv, D]
        v = torch.where(ok[:, None, None], v_cache[page, :, j % S].double(), 0.0)
        vis = torch.ones(t, n, dtype=torch.bool)
        if causal:
            vis = j[None] <= torch.arange(t)[:, None] + (n - t)
        for h in range(H):
            qq = q[h, r0:r1].double()
            kk, vv = k[:, h // G], v[:, h // G]
            s = torch.where(vis, qq @ kk.T * scale, -math.inf)
            z = torch.logsumexp(s, -1) if n else torch.full((t,), -math.inf, dtype=torch.float64)
            p = torch.where(vis, torch.exp(s - torch.where(torch.isinf(z), 0.0, z)[:, None]), 0.0)
            delta = (qq.abs() @ kk.abs().T * scale * (D + 4) * 2.0 ** -24)
            delta = torch.where(vis, delta, 0.0).amax(-1) if n else torch.zeros(t, dtype=torch.float64)
            o[h, r0:r1] = p @ vv
            lse[h, r0:r1] = z
            A = p @ vv.abs()
            to[h, r0:r1] = A * (u + 2 * delta + 2.0 ** -15)[:, None] + u * (p @ vv).abs() + 2.0 ** -24
            if dtype == torch.float16 and n:
                to[h, r0:r1] += 2.0 ** -25 * n * vv.abs().amax()
            tl[h, r0:r1] = delta + 2.0 ** -15 + torch.where(torch.isinf(z), 0.0, z).abs() * 2.0 ** -22
    return o, lse, to, tl


def compare(o, lse, ref):
    """Element-wise against paged_attention_ref; rows of no sequence (NaN in the
    reference) must hold the canary NaN still."""
    ro, rl, to, tl = ref
    o, lse = o.double().cpu(), lse.double().cpu()
    none = torch.isnan(rl)
    assert torch.isnan(lse[none]).all() and torch.isnan(o[none]).all(), "a row of no sequence was written"
    live = ~none
    assert not torch.isnan(lse[live]).any() and not torch.isnan(o[live]).any(), "NaN in the result"
    empty = live & torch.isinf(rl)
    assert torch.equal(torch.isinf(lse), torch.isinf(torch.where(none, 0.0, rl))), "empty rows differ"
    assert (lse[empty] < 0).all() and (o[empty] == 0).all()
    full = live & ~empty
    e = ((o - ro).abs() / to)[full]
    assert e.numel() == 0 or float(e.max()) <= 1.0, f"O is off by {float(e.max()):.2f} times the bound"
    e = ((lse - rl).abs() / tl)[full]
    assert e.numel() == 0 or float(e.max()) <= 1.0, f"LSE is off by {float(e.max()):.2f} times the bound"


class Batch:
    """A seeded ragged batch over a paged cache (CPU tensors; .cuda() moves
    it).  Every cache slot that no sequence holds is NaN, table entries past a
    sequence's pages are out of range."""

    def __init__(self, lens, new, H, Hkv, D, page, dtype, seed=0, spare_rows=0, tokens=False, fused=False, gap=0):
        g = torch.Generator().manual_seed(seed)
        dt = DT[dtype]
        self.lens, self.new, self.H, self.Hkv, self.D, self.page, self.dt = lens, new, H, Hkv, D, page, dt
        B = len(lens)
        need = [(n + page - 1) // page for n in lens]
        P, M = sum(need) + 2, max(max(need), 1)
        order = torch.randperm(P, generator=g).tolist()
        self.table = torch.full((B, M), 2 ** 30, dtype=torch.int32)
        self.table[:, 0::2] = -1 - self.table[:, 0::2]
        self.k = torch.full((P, Hkv, page, D), math.nan, dtype=dt)
        self.v = torch.full((P, Hkv, page, D), math.nan, dtype=dt)
        at = 0
        for b in range(B):
            for i in range(need[b]):
                pg = order[at]
                at += 1
                self.table[b, i] = pg
                rows = min(page, lens[b] - i * page)
                self.k[pg, :, :rows] = torch.randn(Hkv, rows, D, generator=g).to(dt)
                self.v[pg, :, :rows] = torch.randn(Hkv, rows, D, generator=g).to(dt)
        cu = [gap]
        for n in new:
            cu.append(cu[-1] + n)
        self.cu = torch.tensor(cu, dtype=torch.int32)
        self.T = cu[-1] + spare_rows
        self.seq_lens = torch.tensor(lens, dtype=torch.int32)
        self.q = torch.randn(H, self.T, D, generator=g).to(dt)
        self.k_new = torch.randn(Hkv, self.T, D, generator=g).to(dt)
        self.v_new = torch.randn(Hkv, self.T, D, generator=g).to(dt)
        self.tokens, self.fused = tokens, fused
        self.max_q = max(max(new), 1)

    def _rows(self, x):
        x = x.cuda()
        return x.transpose(0, 1).contiguous().transpose(0, 1) if self.tokens else x

    def cuda(self):
        import exact_attention_112_b200 as fa
        k, v = self.k.cuda(), self.v.cuda()
        if self.tokens:      # token-major pages
            k, v = (x.transpose(1, 2).contiguous().transpose(1, 2) for x in (k, v))
        if self.fused:       # keys and values of a page side by side in one allocation
            both = torch.stack((k, v), 1).contiguous()
            k, v = both[:, 0], both[:, 1]
        self.dk, self.dv = k, v
        self.dq, self.dkn, self.dvn = self._rows(self.q), self._rows(self.k_new), self._rows(self.v_new)
        self.dcu = self.cu.cuda()
        self.kv = fa.PagedKV(k, v, self.table.cuda(), self.seq_lens.cuda())
        return self

    def attend(self, causal=True, scale=None, max_q=None):
        import exact_attention_112_b200 as fa
        mq = self.max_q if max_q is None else max_q
        o = torch.full_like(self.dq, math.nan)
        lse = torch.full((self.H, self.T), math.nan, device="cuda")
        ws = torch.full((fa.fa_paged_fwd_workspace_bytes(self.kv, self.H, mq),), 0xFF, dtype=torch.uint8, device="cuda")
        fa.fa_paged_fwd(self.kv, self.dq, o, lse, self.dcu, mq, ws, causal=causal, scale=scale)
        torch.cuda.synchronize()
        assert fa.fa_device_status() == fa.FA_OK
        return o, lse

    def ref(self, causal=True, scale=None, max_q=None):
        scale = 1.0 / math.sqrt(self.D) if scale is None else scale
        return paged_attention_ref(self.q, self.k, self.v, self.table, self.lens, self.cu, causal, scale, self.dt, max_q)
