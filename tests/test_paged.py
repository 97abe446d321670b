"""Paged cache: appending (fa_paged_append) and attention (fa_paged_fwd) against
the float64 definition, over ragged batches, head groups, page sizes and
strides; slots that no sequence holds are NaN and must not show."""
import math

import pytest
import torch

import exact_attention_112_b200 as fa
from paged_ref import DT, Batch, compare, rope_ref, rope_tol

pytestmark = pytest.mark.gpu

# lens, new, H, Hkv, D, page, dtype
ATTEND = [
    ([1], [1], 1, 1, 64, 8, "bf16"),
    ([17], [1], 4, 1, 128, 16, "f16"),
    ([1000], [1], 32, 8, 128, 16, "bf16"),
    ([128, 129, 127, 64, 65, 63], [1] * 6, 8, 2, 64, 64, "bf16"),
    ([0, 5, 0, 300], [1, 1, 0, 1], 6, 3, 128, 24, "bf16"),          # empty sequences, odd pages
    ([700, 3, 2049], [5, 3, 2], 8, 8, 64, 128, "f16"),
    ([513, 40, 1100], [4, 7, 1], 20, 4, 128, 48, "bf16"),           # 5 heads a group
    ([260], [260], 3, 1, 128, 32, "bf16"),                          # a prompt
    ([500, 77, 900, 1], [130, 77, 1, 1], 8, 2, 64, 16, "bf16"),     # prompts and tokens
    ([3, 10], [9, 10], 2, 1, 64, 8, "f16"),                         # more rows than keys: empty rows
    ([640], [257], 7, 1, 128, 128, "f16"),                          # 7 heads a group
    ([333, 900], [20, 9], 128, 1, 64, 256, "bf16"),                 # one kv head for 128
    ([2100], [64], 16, 4, 64, 72, "bf16"),
    ([4000, 130], [33, 130], 12, 12, 128, 64, "bf16"),
    ([12000], [1], 8, 1, 128, 64, "bf16"),
    ([9000], [17], 4, 2, 64, 32, "f16"),
]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("case", ATTEND)
def test_attention(case, causal):
    b = Batch(*case, seed=len(case[0]) + sum(case[0])).cuda()
    compare(*b.attend(causal), b.ref(causal))


@pytest.mark.parametrize("new", [[1, 1, 1], [40, 300, 1]])
@pytest.mark.parametrize("kw", [dict(tokens=True), dict(fused=True), dict(spare_rows=5, gap=3)])
def test_strides_and_rows_of_no_sequence(kw, new):
    b = Batch([400, 301, 17], new, 8, 2, 128, 16, "bf16", seed=11, **kw).cuda()
    compare(*b.attend(), b.ref())


@pytest.mark.parametrize("new,max_q", [([5, 2], 3), ([300, 10], 200)])
def test_rows_beyond_the_bound_are_cut(new, max_q):
    b = Batch([320, 70], new, 4, 4, 64, 32, "bf16", seed=12).cuda()
    # rows past the bound belong to no unit of work; the causal edge is that of the cut sequence
    compare(*b.attend(max_q=max_q), b.ref(max_q=max_q))


@pytest.mark.parametrize("new", [[1, 1], [64, 200]])
def test_large_scores_and_infinities(new):
    """Scores in the hundreds (a sharp softmax), and an infinite key value past
    the length."""
    b = Batch([800, 555], new, 8, 2, 64, 32, "bf16", seed=13)
    b.q = (b.q.float() * 8).to(b.dt)
    b.k = (b.k.float() * 8).to(b.dt)
    b.k[torch.isnan(b.k)] = math.inf
    b.v[torch.isnan(b.v)] = -math.inf
    b.cuda()
    compare(*b.attend(), b.ref())


@pytest.mark.parametrize("new", [[1, 1], [90, 257]])
def test_bad_pages_are_not_followed(new):
    b = Batch([300, 280], new, 4, 2, 64, 32, "bf16", seed=14)
    b.table[0, 2] = 10 ** 9
    b.table[1, 0] = -7
    b.cuda()
    compare(*b.attend(), b.ref())
    before = b.dk.clone(), b.dv.clone()
    fa.fa_paged_append(b.kv, b.dkn, b.dvn, b.dcu)
    torch.cuda.synchronize()
    held = {int(p) for p in b.table.flatten() if 0 <= int(p) < b.k.shape[0]}
    for p in range(b.k.shape[0]):
        if p not in held:
            assert torch.equal(torch.nan_to_num(b.dk[p]), torch.nan_to_num(before[0][p]))


@pytest.mark.parametrize("new", [[1, 1, 1], [70, 1, 33]])
def test_lengths_are_clamped(new):
    b = Batch([256, 256, 256], new, 2, 1, 64, 32, "bf16", seed=15)
    b.seq_lens = torch.tensor([10 ** 9, -5, 256], dtype=torch.int32)
    b.cuda()
    b.lens = [256, 0, 256]
    compare(*b.attend(), b.ref())


def _expected_cache(b, f, inter, scale=1.0, positions=None):
    """Caches after the append, in the cache's type where stored as given and
    float64 where rotated; and the slots written."""
    k, v = b.k.double(), b.v.double()
    tol = torch.zeros_like(k)
    qr = b.q.double()
    qt = torch.zeros_like(qr)
    for s in range(len(b.lens)):
        for t in range(int(b.cu[s]), int(b.cu[s + 1])):
            at = b.lens[s] - int(b.cu[s + 1]) + t
            x = b.k_new[:, t].double()[:, None]
            qx = b.q[:, t].double()[:, None]
            if f is None:
                y, ty = x, torch.zeros_like(x)
            else:
                pos = torch.tensor([at if positions is None else int(positions[t])])
                y = rope_ref(x, pos, f, inter, scale)
                ty = rope_tol(x, y, f, b.dt, inter, scale)
                qr[:, t] = rope_ref(qx, pos, f, inter, scale)[:, 0]
                qt[:, t] = rope_tol(qx, qr[:, t][:, None], f, b.dt, inter, scale)[:, 0]
            if at < 0:
                continue
            page = int(b.table[s, at // b.page])
            k[page, :, at % b.page], tol[page, :, at % b.page] = y[:, 0], ty[:, 0]
            v[page, :, at % b.page] = b.v_new[:, t].double()
    return k, v, tol, qr, qt


def _same(got, want, tol):
    got = got.cpu().double()
    assert torch.equal(torch.isnan(got), torch.isnan(want)), "a slot that no row owns was written, or one was not"
    err = torch.nan_to_num(got - want).abs()
    assert (err <= torch.nan_to_num(tol)).all(), f"off by {float((err - tol).max())} beyond the bound"


@pytest.mark.parametrize("lens,new,H,Hkv,D,page,dtype,rot,inter,kw", [
    ([1], [1], 1, 1, 64, 8, "bf16", 64, False, {}),
    ([700, 1, 16], [1, 1, 1], 8, 2, 128, 16, "f16", 128, False, dict(tokens=True)),
    ([40, 0, 333, 9], [40, 0, 100, 3], 5, 1, 64, 24, "bf16", 16, True, dict(fused=True)),
    ([5, 90], [8, 90], 4, 4, 128, 32, "bf16", 64, True, dict(gap=2, spare_rows=4)),   # more new rows than keys
    ([3] * 300, [1] * 300, 2, 2, 64, 8, "f16", 32, False, {}),                        # more sequences than threads
    ([130, 131], [130, 131], 16, 8, 128, 128, "bf16", 128, False, dict(tokens=True)),
])
def test_append(lens, new, H, Hkv, D, page, dtype, rot, inter, kw):
    b = Batch(lens, new, H, Hkv, D, page, dtype, seed=21, **kw)
    b.cuda()
    f, s = fa.rope_inv_freq(rot, scaling="bands", factor=2.0)
    rope = fa.Rope(f, 1.25, interleaved=inter)
    qo = b.dq.clone()
    fa.fa_paged_append(b.kv, b.dkn, b.dvn, b.dcu, rope=rope, q=b.dq, q_out=qo)
    torch.cuda.synchronize()
    k, v, tol, qr, qt = _expected_cache(b, f.cpu(), inter, 1.25)
    _same(b.dk, k, tol)
    _same(b.dv, v, torch.zeros_like(v))
    _same(qo, qr, qt)                       # rows of no sequence as they were


def test_append_positions_and_without_rope():
    b = Batch([50, 64], [7, 20], 4, 2, 64, 16, "bf16", seed=22).cuda()
    f, _ = fa.rope_inv_freq(64)
    pos = torch.randint(0, 100000, (b.T,), dtype=torch.int32, generator=torch.Generator().manual_seed(1))
    fa.fa_paged_append(b.kv, b.dkn, b.dvn, b.dcu, rope=fa.Rope(f), positions=pos.cuda())
    torch.cuda.synchronize()
    k, v, tol, _, _ = _expected_cache(b, f.cpu(), False, positions=pos)
    _same(b.dk, k, tol)
    b = Batch([50, 64], [7, 20], 4, 2, 64, 16, "bf16", seed=23).cuda()
    fa.fa_paged_append(b.kv, b.dkn, b.dvn, b.dcu)
    torch.cuda.synchronize()
    k, v, tol, _, _ = _expected_cache(b, None, False)
    _same(b.dk, k, tol)
    _same(b.dv, v, tol)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_serving_run(dtype):
    """A prompt in two chunks beside a running sequence, then single tokens, each
    step appending (with the rotation) and attending: the last row of every
    step equals the same tokens' rows computed at once in float64."""
    H, Hkv, D, page, total = 8, 2, 64, 16, 150
    g = torch.Generator().manual_seed(31)
    dt = DT[dtype]
    seqs = [total, total - 40]
    q = [torch.randn(H, n, D, generator=g).to(dt) for n in seqs]
    k = [torch.randn(Hkv, n, D, generator=g).to(dt) for n in seqs]
    v = [torch.randn(Hkv, n, D, generator=g).to(dt) for n in seqs]
    P = sum((n + page - 1) // page for n in seqs) + 1
    kc = torch.full((P, Hkv, page, D), math.nan, dtype=dt, device="cuda")
    vc = torch.full_like(kc, math.nan)
    w = (total + page - 1) // page
    table = torch.zeros(2, w, dtype=torch.int32)
    perm = torch.randperm(P, generator=g).tolist()
    table[0, :w] = torch.tensor(perm[:w])
    n1 = (seqs[1] + page - 1) // page
    table[1, :n1] = torch.tensor(perm[w:w + n1])
    lens = torch.zeros(2, dtype=torch.int32, device="cuda")
    kv = fa.PagedKV(kc, vc, table.cuda(), lens)
    f, s = fa.rope_inv_freq(64, scaling="yarn", factor=2.0)
    rope = fa.Rope(f, s)
    done = [0, 0]
    outs = [[], []]
    for step in [(60, 1), (60, 30), (1, 50)] + [(1, 1)] * 29:
        step = tuple(min(n, seqs[i] - done[i]) for i, n in enumerate(step))
        rows = [torch.cat([x[i][:, done[i]:done[i] + step[i]] for i in range(2)], 1).cuda() for x in (q, k, v)]
        cu = torch.tensor([0, step[0], sum(step)], dtype=torch.int32, device="cuda")
        done = [done[i] + step[i] for i in range(2)]
        lens.copy_(torch.tensor(done, dtype=torch.int32))
        o, _ = fa.paged_step(kv, *rows, cu, max(step), rope)
        outs[0].append(o[:, :step[0]].cpu())
        outs[1].append(o[:, step[0]:].cpu())
    assert fa.fa_device_status() == fa.FA_OK and done == seqs
    u = torch.finfo(dt).eps / 2
    for i, n in enumerate(seqs):
        pos = torch.arange(n)
        # the rotated rows as stored: rounded once to the type
        qr = rope_ref(q[i].double(), pos, f.cpu(), scale=s)
        kr = rope_ref(k[i].double(), pos, f.cpu(), scale=s)
        kr, qr = kr.repeat_interleave(H // Hkv, 0), qr
        vv = v[i].double().repeat_interleave(H // Hkv, 0)
        z = (qr @ kr.transpose(-1, -2) / math.sqrt(D)).masked_fill(~torch.ones(n, n, dtype=torch.bool).tril(), -math.inf)
        p = z.softmax(-1)
        ref, A = p @ vv, p @ vv.abs()
        # q and k are rounded once each: a score moves by at most 2.1 u sum |q||k| scale
        dz = 2.1 * u * (qr.abs() @ kr.abs().transpose(-1, -2) / math.sqrt(D)).tril().amax(-1, keepdim=True)
        tol = A * (u + 2 * dz * (1 + dz) + 2.0 ** -14) + u * ref.abs() + 2.0 ** -24 + 2.0 ** -25 * n * vv.abs().amax()
        got = torch.cat(outs[i], 1).double()
        assert ((got - ref).abs() <= tol).all()


@pytest.mark.parametrize("new", [[1, 1, 1], [90, 1, 257]])
def test_same_bits_every_time_and_in_a_graph(new):
    b = Batch([700, 2000, 300], new, 8, 2, 128, 32, "bf16", seed=41).cuda()
    o, lse = b.attend()
    o2, lse2 = b.attend()
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    ws = torch.empty(fa.fa_paged_fwd_workspace_bytes(b.kv, 8, b.max_q), dtype=torch.uint8, device="cuda")
    go, gl = torch.zeros_like(o), torch.zeros_like(lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fa.fa_paged_fwd(b.kv, b.dq, go, gl, b.dcu, b.max_q, ws)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, go) and torch.equal(lse, gl)
    # the captured call reads the tables when it runs: the sequences grow shorter
    b.kv.seq_lens.copy_(torch.tensor([300, 2000, 290], dtype=torch.int32))
    b.lens = [300, 2000, 290]
    graph.replay()
    torch.cuda.synchronize()
    compare(go, gl, b.ref())


def test_two_streams_with_workspaces_of_their_own():
    bs = [Batch([3000, 100 + i], [200, 1], 8, 2, 64, 32, "bf16", seed=50 + i).cuda() for i in range(2)]
    want = [b.attend() for b in bs]
    outs = []
    torch.cuda.synchronize()
    for b in bs:
        s = torch.cuda.Stream()
        o, lse = torch.empty_like(b.dq), torch.empty(b.H, b.T, device="cuda")
        ws = torch.empty(fa.fa_paged_fwd_workspace_bytes(b.kv, b.H, b.max_q), dtype=torch.uint8, device="cuda")
        s.wait_stream(torch.cuda.current_stream())
        for _ in range(5):
            fa.fa_paged_fwd(b.kv, b.dq, o, lse, b.dcu, b.max_q, ws, stream=s)
        outs.append((o, lse, ws))
    torch.cuda.synchronize()
    for (o, lse, _), (wo, wl) in zip(outs, want):
        assert torch.equal(o, wo) and torch.equal(lse, wl)


def test_cache_of_more_than_2_31_elements():
    """Offsets that pass 32 bits: the pages used lie at the end of a 4.3 GB cache."""
    S, Hkv, D = 64, 8, 128
    P = (1 << 31) // (S * Hkv * D) + 8
    kc = torch.zeros((P, Hkv, S, D), dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    b = Batch([200, 300], [1, 100], 16, Hkv, D, S, "bf16", seed=60)
    n = b.k.shape[0]
    kc[P - n:], vc[P - n:] = torch.nan_to_num(b.k).cuda(), torch.nan_to_num(b.v).cuda()
    b.table = torch.where((b.table >= 0) & (b.table < n), b.table + (P - n), b.table)
    ref_table = torch.where(b.table >= P - n, b.table - (P - n), b.table)
    b.cuda()
    b.kv = fa.PagedKV(kc, vc, b.table.cuda(), b.seq_lens.cuda())
    o, lse = b.attend()
    b.table = torch.where(b.table < 2 ** 29, ref_table, b.table)
    compare(o, lse, b.ref())
    fa.fa_paged_append(b.kv, b.dkn, b.dvn, b.dcu)
    torch.cuda.synchronize()
    k, _, tol, _, _ = _expected_cache(b, None, False)
    _same(kc[P - n:], torch.nan_to_num(k), tol)
