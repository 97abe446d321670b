"""Paged attention at the borders of its kernels: the number of query rows of a
unit, head groups, units of many pieces, batches of many sequences, caches with
unusual strides, other streams."""
import math

import pytest
import torch

import exact_attention_112_b200 as fa
from paged_ref import Batch, compare

pytestmark = pytest.mark.gpu


def _check(b, **kw):
    b.cuda()
    compare(*b.attend(**kw), b.ref(**kw))


# rows of a unit: tokens x heads of a group; 16, 32 and 64 are the widths of the
# kernel of few tokens, 128 a tile and 256 a unit of the other
@pytest.mark.parametrize("D,dtype", [(64, "bf16"), (128, "f16")])
@pytest.mark.parametrize("new,G", [(1, 15), (1, 16), (1, 17), (2, 16), (3, 11), (7, 9), (8, 8), (13, 5), (21, 3), (32, 2),
                                   (64, 1), (65, 1), (9, 8), (1, 65), (1, 127), (2, 64), (3, 64), (128, 1), (129, 1),
                                   (51, 5), (52, 5)])
def test_rows_of_a_unit(new, G, D, dtype):
    _check(Batch([300 + new, 129, new], [new, max(1, new // 2), new], 2 * G, 2, D, 16, dtype, seed=new * G))


@pytest.mark.parametrize("lens,new,H,Hkv,D,page", [
    ([2600], [2600], 4, 1, 64, 16),                         # more than 32 units in a sequence
    ([5000, 40], [1400, 1], 16, 2, 128, 64),                # units cut by several CTAs
    ([100, 50, 700], [300, 200, 40], 4, 2, 64, 8),          # more rows than keys, whole units without a key
    ([128 * 150], [1], 2, 2, 64, 128),                      # a token over more tiles than there are CTAs
    ([128 * 37 + 1], [30], 4, 2, 128, 40),
])
@pytest.mark.parametrize("causal", [True, False])
def test_long_units(lens, new, H, Hkv, D, page, causal):
    _check(Batch(lens, new, H, Hkv, D, page, "bf16", seed=sum(lens)), causal=causal)


@pytest.mark.parametrize("most,D", [(1, 64), (3, 128), (90, 64)])
def test_many_sequences(most, D):
    """More sequences than a step of the planning takes, some without new rows, some without keys."""
    g = torch.Generator().manual_seed(most)
    B = 333
    new = [int(x) for x in torch.randint(0, most + 1, (B,), generator=g)]
    lens = [n + int(x) if x > 20 else 0 for n, x in zip(new, torch.randint(0, 260, (B,), generator=g))]
    new[0] = most
    _check(Batch(lens, new, 4, 2, D, 16, "bf16", seed=most))


def _strided(x, shape_strides, offset=0):
    """A copy of x in a buffer of NaN, with the given strides."""
    size = offset + 1 + sum((n - 1) * s for n, s in zip(x.shape, shape_strides))
    buf = torch.full((size,), math.nan, dtype=x.dtype, device="cuda")
    v = torch.as_strided(buf, x.shape, shape_strides, offset)
    v.copy_(x)
    return v


@pytest.mark.parametrize("new", [[1, 1], [6, 300]])
@pytest.mark.parametrize("kind", ["odd pages", "token-major keys", "wide rows", "one head", "one page", "heads outermost"])
def test_cache_strides(kind, new):
    Hkv, S = (1, 16) if kind == "one head" else (3, 16)
    lens = [16, 9] if kind == "one page" else [333, 310]
    if kind == "one page":
        new = [min(n, 9) for n in new]
    D = 64
    b = Batch(lens, new, 4 * Hkv, Hkv, D, S, "bf16", seed=71).cuda()
    k, v, table = b.k.cuda(), b.v.cuda(), b.table.cuda()
    P = k.shape[0]
    if kind == "odd pages":                 # a page stride that no head stride divides
        k = _strided(k, (Hkv * S * D + 8, S * D, D, 1), 8)
        v = _strided(v, (Hkv * S * D + 24, S * D, D, 1))
    elif kind == "token-major keys":        # keys and values laid out differently
        k = _strided(k, (S * Hkv * D, D, Hkv * D, 1))
    elif kind == "wide rows":
        k = _strided(k, (Hkv * S * 2 * D, S * 2 * D, 2 * D, 1), 64)
        v = _strided(v, (Hkv * S * (D + 8), S * (D + 8), D + 8, 1))
    elif kind == "one head":
        k = _strided(k, (S * D + 40, S * D, D, 1))
    elif kind == "heads outermost":
        k, v = (_strided(x, (S * D, P * S * D, D, 1)) for x in (k, v))
    elif kind == "one page":                # both sequences read the same page
        k, v = k[:1].clone(), v[:1].clone()
        table.zero_()
        k.nan_to_num_(0.5)
        v.nan_to_num_(0.25)
        b.k, b.v, b.table = k.cpu(), v.cpu(), table.cpu()
    b.kv = fa.PagedKV(k, v, table, b.seq_lens.cuda())
    compare(*b.attend(), b.ref())
    if kind == "one page":
        return
    fa.fa_paged_append(b.kv, b.dkn, b.dvn, b.dcu)
    torch.cuda.synchronize()
    for s, n in enumerate(lens):
        for i in range(b.new[s]):
            at = n - b.new[s] + i
            row = int(b.cu[s]) + i
            page = int(b.table[s, at // S])
            assert torch.equal(k[page, :, at % S], b.dkn[:, row]) and torch.equal(v[page, :, at % S], b.dvn[:, row])


def test_page_shared_by_sequences():
    """A common prefix: several sequences read the same pages."""
    b = Batch([200, 200, 200], [1, 5, 40], 8, 2, 128, 32, "bf16", seed=72)
    b.table[1, :4] = b.table[0, :4]
    b.table[2, :6] = b.table[0, :6]
    _check(b)


@pytest.mark.parametrize("new", [[1, 1, 1], [50, 1, 200]])
def test_another_stream(new):
    """Every call on a stream of its own, allocations included, while the current
    stream is busy with memory that it frees."""
    b = Batch([700, 80, 300], new, 8, 2, 64, 16, "bf16", seed=73).cuda()
    want, want_lse = b.attend()
    f, _ = fa.rope_inv_freq(64)
    rope = fa.Rope(f)
    s = torch.cuda.Stream()
    for handle in (s, s.cuda_stream):
        torch.cuda.synchronize()
        for _ in range(3):
            junk = torch.randn(b.H, b.T, 64, device="cuda").to(b.dt)
            del junk
            o, lse = fa.paged_attention(b.kv, b.dq, b.dcu, b.max_q, stream=handle)
            qr, _ = fa.rope_forward(b.dq, None, rope, stream=handle)
        torch.cuda.synchronize()
        assert torch.equal(o, want) and torch.equal(lse, want_lse)
        assert torch.equal(qr, fa.rope_forward(b.dq, None, rope)[0])


def test_two_graphs_share_a_workspace():
    """Two captured calls with one workspace, replayed in turn on one stream."""
    bs = [Batch([900, 1000], [1, 1], 8, 2, 64, 32, "bf16", seed=74).cuda(),
          Batch([400, 650], [300, 20], 8, 2, 64, 32, "bf16", seed=75).cuda()]
    want = [b.attend() for b in bs]
    ws = torch.empty(max(fa.fa_paged_fwd_workspace_bytes(b.kv, b.H, b.max_q) for b in bs), dtype=torch.uint8, device="cuda")
    outs, graphs = [], []
    for b in bs:
        o, lse = torch.zeros_like(b.dq), torch.zeros(b.H, b.T, device="cuda")
        fa.fa_paged_fwd(b.kv, b.dq, o, lse, b.dcu, b.max_q, ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            fa.fa_paged_fwd(b.kv, b.dq, o, lse, b.dcu, b.max_q, ws)
        outs.append((o, lse))
        graphs.append(g)
    for o, lse in outs:
        o.zero_()
        lse.zero_()
    for _ in range(4):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for (o, lse), (wo, wl) in zip(outs, want):
        assert torch.equal(o, wo) and torch.equal(lse, wl)


@pytest.mark.parametrize("new", [[4, 3], [40, 130]])
def test_a_row_of_nan_stays_alone(new):
    """A query of NaN and one of infinities: NaN comes out, and the other rows are
    as exact as ever."""
    b = Batch([300, 400], new, 8, 2, 64, 16, "bf16", seed=76)
    ref = b.ref()
    rows = [(1, 2), (3, new[0] + 1)]
    b.q[rows[0]] = math.nan
    b.q[rows[1]] = math.inf
    o, lse = b.cuda().attend()
    for r in rows:
        assert torch.isnan(o[r]).all() and torch.isnan(lse[r])
        for x in ref[:2]:
            x[r] = math.nan
    compare(o, lse, ref)


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("new", [[1, 1], [40, 130]])
def test_waits_for_work_of_two_streams(new, captured):
    """The call may be set up while the kernel before it still runs, so it has to
    wait for it and for an event of another stream: the queries come late on one
    stream, the table on the other."""
    b = Batch([700, 900], new, 8, 2, 64, 16, "bf16", seed=81).cuda()
    want, want_lse = b.attend()
    q, table = b.dq.clone(), b.kv.page_table.clone()
    ws = torch.empty(fa.fa_paged_fwd_workspace_bytes(b.kv, b.H, b.max_q), dtype=torch.uint8, device="cuda")
    o, lse = torch.empty_like(b.dq), torch.empty(b.H, b.T, device="cuda")
    big = torch.randn(4096, 4096, device="cuda")
    zero = torch.zeros((), device="cuda", dtype=torch.bfloat16)
    other = torch.cuda.Stream()

    def work():
        here = torch.cuda.current_stream()
        b.dq.fill_(7.0)
        b.kv.page_table.fill_(-1)
        other.wait_stream(here)
        with torch.cuda.stream(other):
            for _ in range(4):
                big @ big
            b.kv.page_table.copy_(table)
        for _ in range(2):
            big @ big
        torch.add(q, zero, out=b.dq)
        here.wait_stream(other)
        fa.fa_paged_fwd(b.kv, b.dq, o, lse, b.dcu, b.max_q, ws)
        o2 = o.clone()              # and what follows it waits for the merge
        fa.fa_paged_fwd(b.kv, b.dq, o, lse, b.dcu, b.max_q, ws)
        return o2

    o2 = work()
    if captured:
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            o2 = work()
        for _ in range(3):
            o.zero_()
            graph.replay()
    torch.cuda.synchronize()
    assert fa.fa_device_status() == fa.FA_OK
    assert torch.equal(o, want) and torch.equal(lse, want_lse) and torch.equal(o2, want)


@pytest.mark.parametrize("new", [[1, 1, 2], [12, 3, 20], [60, 1, 140]])
@pytest.mark.parametrize("pad,off", [(8, 0), (16, 8), (0, 8), (24, 16)])
def test_strides_of_queries_and_outputs(new, pad, off):
    """Rows of q and o with padding between them and a base that is 16-byte
    aligned only: whatever lies between the rows stays as it was."""
    D = 64
    b = Batch([200, 90, 310], new, 6, 2, D, 16, "bf16", seed=82).cuda()
    want, want_lse = b.attend()
    H, T = b.H, b.T
    strides = (T * (D + pad) + 8 * (pad > 0), D + pad, 1)
    q = _strided(b.q, strides, off)
    buf = torch.full((off + H * strides[0] + 64,), math.nan, dtype=b.dt, device="cuda")
    o = torch.as_strided(buf, (H, T, D), strides, off)
    lse = torch.empty(H, T, device="cuda")
    ws = torch.empty(fa.fa_paged_fwd_workspace_bytes(b.kv, H, b.max_q), dtype=torch.uint8, device="cuda")
    fa.fa_paged_fwd(b.kv, q, o, lse, b.dcu, b.max_q, ws)
    torch.cuda.synchronize()
    assert torch.equal(o, want) and torch.equal(lse, want_lse)
    o.fill_(math.nan)
    assert torch.isnan(buf).all()
