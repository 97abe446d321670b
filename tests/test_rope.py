"""Rotary positions (fa_rope, fa_rope_bwd) against the float64 definition:
layouts, parts of the head, strides, far and negative positions, grouped keys,
in-place calls; the gradient against the formula and against differences."""
import math

import pytest
import torch

import exact_attention_112_b200 as fa
from paged_ref import DT, rope_ref, rope_tol

gpu = pytest.mark.gpu


def _tensor(shape, dtype, g, tokens):
    x = torch.randn(shape, generator=g).to(DT[dtype])
    d = x.cuda()
    return x, (d.transpose(-2, -3).contiguous().transpose(-2, -3) if tokens else d)


def _check(y, x, pos, f, dtype, inter, scale=1.0, sign=1.0):
    xd, yd = x.double(), y.cpu().double()
    ref = rope_ref(xd, pos, f, inter, scale, sign)
    bad = (yd - ref).abs() > rope_tol(xd, ref, f, DT[dtype], inter, scale)
    assert not bad.any(), f"{int(bad.sum())} values beyond the bound"
    r = 2 * f.numel()
    assert torch.equal(yd[..., r:], xd[..., r:])


@gpu
@pytest.mark.parametrize("B,H,Hk,N,D,rot,dtype,inter,tokens", [
    (1, 1, 1, 1, 64, 64, "bf16", False, False),
    (2, 3, 1, 5, 64, 16, "f16", True, False),
    (1, 8, 2, 300, 128, 128, "bf16", False, True),
    (3, 5, 5, 129, 128, 64, "f16", True, True),
    (2, 7, 1, 33, 80, 48, "bf16", True, False),
    (1, 2, 2, 17, 24, 16, "f16", False, False),
    (1, 33, 3, 1000, 64, 32, "bf16", False, False),
    (4, 2, 1, 3, 512, 512, "bf16", True, False),
])
def test_rope_forward_and_gradient(B, H, Hk, N, D, rot, dtype, inter, tokens):
    g = torch.Generator().manual_seed(B * 1000 + N)
    q, dq = _tensor((B, H, N, D), dtype, g, tokens)
    k, dk = _tensor((B, Hk, N, D), dtype, g, tokens)
    f, s = fa.rope_inv_freq(rot, scaling="yarn", factor=4.0)
    rope = fa.Rope(f, s, interleaved=inter)
    f = f.cpu()
    pos = torch.randint(-5000, 1 << 20, (B, N), generator=g, dtype=torch.int32)
    for fwd, sign in ((fa.rope_forward, 1.0), (fa.rope_backward, -1.0)):
        qo, ko = fwd(dq, dk, rope, positions=pos.cuda())
        _check(qo, q, pos[:, None], f, dtype, inter, s, sign)
        _check(ko, k, pos[:, None], f, dtype, inter, s, sign)
    # positions of all batches, an offset instead of a table, q alone
    qo, ko = fa.rope_forward(dq, dk, rope, positions=pos[0].cuda())
    _check(ko, k, pos[0][None, None], f, dtype, inter, s)
    qo, ko = fa.rope_forward(dq, None, rope, offset=70000)
    assert ko is None
    _check(qo, q, 70000 + torch.arange(N), f, dtype, inter, s)


@gpu
def test_far_positions_and_extremes():
    g = torch.Generator().manual_seed(3)
    q, dq = _tensor((1, 2, 6, 64), "f16", g, False)
    pos = torch.tensor([[2 ** 31 - 1, -2 ** 31, 0, -1, 2 ** 24 + 1, 1999999999]], dtype=torch.int32)
    f, _ = fa.rope_inv_freq(64)
    f[0] = 6.5          # more than a turn a position
    f[1] = -0.37
    qo, _ = fa.rope_forward(dq, None, fa.Rope(f), positions=pos.cuda())
    fc, xd = f.cpu(), q.double()
    # the definition's own product needs more than float64 here: whole turns are taken
    # off in integers (Python's), the frequency in turns rounded to 2^-80 as 1/(2 pi) given to 40 digits
    from fractions import Fraction
    inv2pi = Fraction("0.1591549430918953357688837633725143620344596")
    frac = [[float((Fraction(int(p)) * Fraction(float(w)) * inv2pi) % 1) for w in fc] for p in pos[0]]
    theta = 2 * math.pi * torch.tensor(frac, dtype=torch.float64)
    c, s = theta.cos(), theta.sin()
    a, b = xd[..., :32], xd[..., 32:]
    ref = torch.cat((a * c - b * s, b * c + a * s), -1)
    # the frequency in turns is rounded twice in float64: |p| 2^-52 |f| / (2 pi) turns, 2 pi of it in radians
    extra = (a.abs() + b.abs()) * pos[0].abs().double()[:, None] * fc.abs() * 2.0 ** -52
    tol = rope_tol(xd, ref, fc, torch.float16) + torch.cat((extra, extra), -1)
    assert ((qo.cpu().double() - ref).abs() <= tol).all()


@gpu
def test_in_place_and_packed_and_nan_rows():
    g = torch.Generator().manual_seed(4)
    q, dq = _tensor((3, 50, 128), "bf16", g, False)
    k, dk = _tensor((1, 50, 128), "bf16", g, False)
    dq[1, 7] = math.nan                     # a bad row stays its own affair
    f, _ = fa.rope_inv_freq(64, scaling="bands", factor=8.0)
    rope = fa.Rope(f)
    a, b = fa.rope_forward(dq, dk, rope)
    fa.fa_rope(dq, dk, dq, dk, rope)
    assert torch.equal(torch.nan_to_num(a), torch.nan_to_num(dq)) and torch.equal(b, dk)
    assert torch.isnan(dq[1, 7, :64]).all() and not torch.isnan(dq[1, :7]).any() and not torch.isnan(dq[0]).any()
    _check(dk, k, torch.arange(50), f.cpu(), "bf16", False)


@gpu
def test_strided_views_leave_the_rest_alone():
    g = torch.Generator().manual_seed(5)
    big = torch.randn(2, 40, 3, 2, 64, generator=g).to(torch.bfloat16).cuda()
    keep = big.clone()
    x = big[:, :, :, 0].transpose(1, 2)     # [2, 3, 40, 64], rows 128 apart
    f, _ = fa.rope_inv_freq(64)
    fa.fa_rope(x, None, x, None, fa.Rope(f, interleaved=True))
    assert torch.equal(big[:, :, :, 1], keep[:, :, :, 1])
    _check(x, keep[:, :, :, 0].transpose(1, 2).cpu(), torch.arange(40), f.cpu(), "bf16", True)


@gpu
def test_gradient_against_differences():
    """L = sum(w * rope(x)) is linear, so a central difference of the float64
    forward is exact up to float64 rounding; the kernel's gradient rounds once."""
    g = torch.Generator().manual_seed(6)
    f, s = fa.rope_inv_freq(32, scaling="ntk", factor=4.0)
    x = torch.randn(1, 2, 3, 64, generator=g).double()
    w = torch.randn(1, 2, 3, 64, generator=g).to(torch.bfloat16)
    pos = torch.tensor([11, 5000, 131071])
    dx, _ = fa.rope_backward(w.cuda(), None, fa.Rope(f, s), positions=pos.int().cuda())
    L = lambda t: float((w.double() * rope_ref(t, pos, f.cpu(), scale=s)).sum())
    for at in [(0, 0, 0, 0), (0, 1, 2, 31), (0, 0, 1, 16), (0, 1, 1, 7), (0, 1, 0, 63)]:
        e = torch.zeros_like(x)
        e[at] = 0.5
        diff = L(x + e) - L(x - e)
        got = float(dx[at])
        assert abs(got - diff) <= 2.0 ** -8 * abs(diff) + 2.0 ** -20, (at, got, diff)


@gpu
def test_rope_attention_gradients():
    """rope -> attention -> its gradients, as a training step runs them, against
    float64 autograd; the attention's own bound (5e-2 of the largest) covers the
    rotation's roundings."""
    import oracle
    from gpu_util import TOL_GRAD_REL
    g = torch.Generator().manual_seed(7)
    B, H, N, D = 1, 2, 200, 64
    q, k, v, do = (torch.randn(B, H, N, D, generator=g).to(torch.bfloat16) for _ in range(4))
    f, s = fa.rope_inv_freq(64)
    rope = fa.Rope(f, s)
    o, lse, qr, kr = fa.rope_attention_forward(q.cuda(), k.cuda(), v.cuda(), rope, causal=True)
    got = fa.rope_attention_backward(qr, kr, v.cuda(), o, lse, do.cuda(), rope, causal=True)
    ts = [t.double().requires_grad_() for t in (q, k, v)]
    pos = torch.arange(N)
    z = rope_ref(ts[0], pos, f.cpu()) @ rope_ref(ts[1], pos, f.cpu()).transpose(-1, -2) / math.sqrt(D)
    z = z.masked_fill(~torch.ones(N, N, dtype=torch.bool).tril(), -math.inf)
    out = z.softmax(-1) @ ts[2]
    out.backward(do.double())
    assert float((o.cpu().double() - out.detach()).abs().max()) <= 2e-2
    for a, t in zip(got, ts):
        assert float((a.cpu().double() - t.grad).abs().max() / t.grad.abs().max()) <= TOL_GRAD_REL


@gpu
def test_rope_runs_on_a_given_stream_and_in_a_graph():
    g = torch.Generator().manual_seed(8)
    q, dq = _tensor((1, 2, 64, 64), "bf16", g, False)
    f, _ = fa.rope_inv_freq(64)
    rope = fa.Rope(f)
    want, _ = fa.rope_forward(dq, None, rope)
    out = torch.zeros_like(dq)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    fa.fa_rope(dq, None, out, None, rope, stream=side)
    side.synchronize()
    assert torch.equal(out, want)
    pos = torch.arange(64, dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fa.fa_rope(dq, None, out, None, rope, positions=pos)
    pos += 1000
    graph.replay()
    torch.cuda.synchronize()
    _check(out, q, 1000 + torch.arange(64), f.cpu(), "bf16", False)


def test_inv_freq_rules():
    f, s = fa.rope_inv_freq(64, base=500000.0, device="cpu")
    i = torch.arange(32).double()
    want = 500000.0 ** (-i / 32)
    assert s == 1.0 and torch.allclose(f, want, rtol=1e-14, atol=0)
    lin, _ = fa.rope_inv_freq(64, base=500000.0, scaling="linear", factor=4.0, device="cpu")
    assert torch.allclose(lin, want / 4, rtol=1e-14, atol=0)
    ntk, _ = fa.rope_inv_freq(64, scaling="ntk", factor=4.0, device="cpu")
    plain, _ = fa.rope_inv_freq(64, device="cpu")
    assert ntk[0] == 1.0 and math.isclose(float(plain[-1] / ntk[-1]), 4.0, rel_tol=1e-12)
    for rule in ("bands", "yarn"):
        got, s = fa.rope_inv_freq(128, scaling=rule, factor=8.0, original_max_position=8192, device="cpu")
        base, _ = fa.rope_inv_freq(128, device="cpu")
        ratio = base / got
        assert ratio[0] == 1.0 and math.isclose(float(ratio[-1]), 8.0, rel_tol=1e-12)
        assert (ratio[1:] >= ratio[:-1] - 1e-12).all()      # from kept to divided, in order
        assert math.isclose(s, 0.1 * math.log(8.0) + 1.0) if rule == "yarn" else s == 1.0
    # a frequency that turns twice within the original context, between 1 and 4: keeps (2 - 1) / (4 - 1)
    base = (8192 / (2 * math.pi * 2.0)) ** 2.0              # so that inv_freq[8] of 16 turns twice
    got, _ = fa.rope_inv_freq(32, base=base, scaling="bands", factor=8.0, device="cpu")
    plain, _ = fa.rope_inv_freq(32, base=base, device="cpu")
    assert math.isclose(float(got[8] / plain[8]), 1 / 3 + (2 / 3) / 8, rel_tol=1e-9)
    for bad in (dict(rot_dim=24), dict(rot_dim=64, scaling="cubic"), dict(rot_dim=64, factor=0.5),
                dict(rot_dim=64, base=1.0)):
        with pytest.raises(fa.FaError):
            fa.rope_inv_freq(**bad, device="cpu")
