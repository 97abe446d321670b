"""Rotary positions and the paged cache at the edges of what their calls allow:
bounds smaller than a sequence, lengths past the table, table entries outside
the cache, scores near the end of float32, addresses and whole numbers at the
borders of their ranges, calls that are refused."""
import math

import pytest
import torch

import exact_attention_112_b200 as fa
from exact_attention_112_b200 import paged
from paged_ref import Batch, compare, rope_ref, rope_tol

gpu = pytest.mark.gpu


# ------------------------------------------------- a bound below a sequence's rows
@gpu
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens,new,H,Hkv,D,max_q", [
    ([320, 70], [5, 2], 4, 4, 64, 3),                   # few rows
    ([1000, 17, 300], [40, 9, 1], 8, 1, 128, 8),
    ([3, 10], [9, 10], 2, 1, 64, 4),                    # more rows than keys: the first rows see none
    ([320, 70], [300, 10], 4, 4, 64, 200),              # row tiles
    ([2000, 500], [1500, 400], 8, 2, 128, 129),
    ([50, 700], [300, 650], 4, 2, 64, 270),
    ([2600], [2600], 4, 1, 64, 2400),                   # more units than a warp has lanes
])
def test_rows_below_the_bound_are_those_of_the_whole_call(lens, new, H, Hkv, D, max_q, causal):
    """Row i of n new ones sees the keys up to i + length - n, whatever the bound
    leaves of the n: the rows that are computed are the uncut call's."""
    b = Batch(lens, new, H, Hkv, D, 16, "bf16", seed=max_q).cuda()
    ref = b.ref(causal)
    for s, n in enumerate(new):
        for x in ref[:2]:
            x[:, int(b.cu[s]) + min(n, max_q):int(b.cu[s + 1])] = math.nan      # not computed, left as they were
    compare(*b.attend(causal, max_q=max_q), ref)


@gpu
@pytest.mark.parametrize("rows", [4, 90])
def test_a_table_that_ends_past_the_rows(rows):
    """Row t of the packed tensors is key length - cu_seqlens_q[b + 1] + t, also
    where the table's last entry lies past them."""
    whole = Batch([400, 300], [2, 2 * rows], 8, 2, 64, 16, "bf16", seed=5).cuda()
    ref = whole.ref()
    T = 2 + rows
    o, lse = torch.empty_like(whole.dq[:, :T]), torch.empty(8, T, device="cuda")
    ws = torch.empty(fa.fa_paged_fwd_workspace_bytes(whole.kv, 8, 2 * rows), dtype=torch.uint8, device="cuda")
    fa.fa_paged_fwd(whole.kv, whole.dq[:, :T], o, lse, whole.dcu, 2 * rows, ws)
    torch.cuda.synchronize()
    compare(o, lse, [x[:, :T] for x in ref])


# ----------------------------------------------------- lengths past the page table
@gpu
@pytest.mark.parametrize("new", [[1, 2, 2, 1], [5, 64, 2, 3], [40, 64, 2, 30]])
def test_append_and_attention_clamp_lengths_alike(new):
    """Lengths above max_pages * page_size or below 0: the new rows are stored and
    rotated at the clamped length's last positions, and see the keys up to them."""
    from test_paged import _expected_cache, _same
    b = Batch([64, 64, 0, 50], new, 8, 2, 64, 16, "bf16", seed=sum(new)).cuda()
    b.kv.seq_lens.copy_(torch.tensor([64 + 3, 10 ** 9, -5, 50], dtype=torch.int32))
    f, _ = fa.rope_inv_freq(64)
    qo = torch.full_like(b.dq, math.nan)
    fa.fa_paged_append(b.kv, b.dkn, b.dvn, b.dcu, rope=fa.Rope(f), q=b.dq, q_out=qo)
    torch.cuda.synchronize()
    k, v, tol, qr, qt = _expected_cache(b, f.cpu(), False)
    _same(b.dk, k, tol)
    _same(b.dv, v, torch.zeros_like(v))
    _same(qo, qr, qt)
    b.k, b.v = b.dk.cpu(), b.dv.cpu()
    compare(*b.attend(), b.ref())


# ------------------------------------------------------ whole numbers past 32 bits
def _handle(cls, **kw):
    """A handle without its tensors: refusals that come before they are looked at."""
    x = object.__new__(cls)
    x.__dict__.update(kw)
    return x


@pytest.mark.parametrize("offset", [2 ** 31, 2 ** 32, 2 ** 32 + 7, -2 ** 31 - 1, 2 ** 63, -2 ** 40])
def test_offsets_past_32_bits_are_refused(offset):
    q = torch.zeros(1, 2, 8, 64, dtype=torch.bfloat16)
    rope = _handle(fa.Rope, rot_dim=64)
    calls = [lambda: fa.rope_forward(q, q, rope, offset=offset), lambda: fa.rope_backward(q, None, rope, offset=offset),
             lambda: fa.fa_rope(q, None, q, None, rope, offset=offset),
             lambda: fa.fa_rope_bwd(q, q, q, q, rope, offset=offset),
             lambda: fa.rope_attention_forward(q, q, q, rope, offset=offset)]
    for call in calls:
        with pytest.raises(fa.FaError, match="offset"):
            call()


@pytest.mark.parametrize("n", [2 ** 31, 2 ** 32, 2 ** 32 + 4, -2 ** 31 - 1, 2 ** 64 + 1])
def test_sizes_past_32_bits_are_refused(n):
    kv = _handle(fa.PagedKV, num_kv_heads=2, num_seqs=1, D=64)
    for args, name in (((4, n), "max_seqlen_q"), ((n, 1), "Hq")):
        with pytest.raises(fa.FaError, match=name):
            fa.fa_paged_fwd_workspace_bytes(kv, *args)


@gpu
def test_a_bound_past_32_bits_is_refused_by_the_calls():
    b = Batch([40], [3], 4, 2, 64, 16, "bf16", seed=7).cuda()
    o, lse = torch.empty_like(b.dq), torch.empty(4, 3, device="cuda")
    ws = torch.empty(fa.fa_paged_fwd_workspace_bytes(b.kv, 4, 3), dtype=torch.uint8, device="cuda")
    for n in (2 ** 32, 2 ** 32 + 3, -2 ** 32 + 3):
        with pytest.raises(fa.FaError, match="max_seqlen_q"):
            fa.fa_paged_fwd(b.kv, b.dq, o, lse, b.dcu, n, ws)
        with pytest.raises(fa.FaError, match="max_seqlen_q"):
            fa.paged_attention(b.kv, b.dq, b.dcu, n)


# --------------------------------------------------------- scores far below nothing
@gpu
@pytest.mark.parametrize("lens,new", [([1, 100, 128], [1, 1, 2]), ([70, 100, 128], [60, 1, 100])])
@pytest.mark.parametrize("D", [64, 128])
def test_scores_near_the_end_of_float32(lens, new, D):
    """Every score of a row is the same -2^116 scale (operands and scale factors
    are powers of two, so float32 has it exactly): the keys have equal weights.
    The probabilities are 1 and their sum a whole number below 2^8, so O is off by
    one rounding, the quotient's and n float32 additions' 2^-24."""
    b = Batch(lens, new, 4, 2, D, 16, "bf16", seed=D)
    b.q.zero_()
    b.q[..., 5] = -2.0 ** 58
    held = ~torch.isnan(b.k)
    b.k[held] = 0.0
    b.k[..., 5][held[..., 5]] = 2.0 ** 58
    b.cuda()
    scale = 0.125
    o, lse = (x.double().cpu() for x in b.attend(scale=scale))
    for s, n in enumerate(lens):
        j = torch.arange(n)
        v = b.v[b.table[s].long()[j // 16], :, j % 16].double().repeat_interleave(2, 1)        # [n, H, D]
        for t in range(int(b.cu[s]), int(b.cu[s + 1])):
            seen = n - int(b.cu[s + 1]) + t + 1
            want, size = v[:seen].mean(0), v[:seen].abs().mean(0)
            assert ((o[:, t] - want).abs() <= 2.0 ** -8 * want.abs() + (seen + 4) * 2.0 ** -24 * size).all()
            assert ((lse[:, t] + 2.0 ** 116 * scale).abs() <= 2.0 ** 116 * scale * 2.0 ** -22).all()


@gpu
@pytest.mark.parametrize("new", [1, 90])
def test_the_highest_of_very_low_scores_takes_all(new):
    """Over several key tiles and CTAs: one key's score is -2^115 scale, all others
    are -2^116 scale, so O is its value."""
    b = Batch([1000], [new], 4, 2, 64, 16, "bf16", seed=9)
    b.q.zero_()
    b.q[..., 5] = -2.0 ** 58
    held = ~torch.isnan(b.k)
    b.k[held] = 0.0
    b.k[..., 5][held[..., 5]] = 2.0 ** 58
    at = 700
    page = int(b.table[0, at // 16])
    b.k[page, :, at % 16, 5] = 2.0 ** 57
    b.cuda()
    o, _ = b.attend(scale=0.125)
    want = b.v[page, :, at % 16].repeat_interleave(2, 0)[:, None].expand(-1, new, -1)
    assert torch.equal(o.cpu(), want)


# ------------------------------------------------------------------- where LSE lies
@pytest.mark.parametrize("low", [4, 8, 12])
def test_lse_needs_the_alignment_of_a_float(low):
    """16-byte alignment is for rows of O and Q; LSE is single floats.  Without a
    workspace the call ends before anything of it is touched."""
    import ctypes
    from exact_attention_112_b200 import _build
    from test_paged_api import P, _kv
    _build.build()
    call = lambda lse: fa.lib().fa_paged_fwd(_kv(), P(1), None, P(2), None, ctypes.c_void_p(lse), P(4), 4, 1, 4, 1, 0.1,
                                             None, 0, None)
    assert call(48) == fa.FA_ERR_WORKSPACE
    assert call(48 + low) == fa.FA_ERR_WORKSPACE
    assert call(48 + 2) == fa.FA_ERR_INVALID_ARG


@gpu
@pytest.mark.parametrize("off", [1, 2, 3])
@pytest.mark.parametrize("new", [[1, 1, 1], [5, 1, 90]])
def test_lse_in_the_middle_of_a_buffer(new, off):
    b = Batch([300, 17, 1000], new, 6, 2, 64, 16, "bf16", seed=off).cuda()
    want, want_lse = b.attend()
    buf = torch.full((off + b.H * b.T + 5,), 7.0, device="cuda")
    lse = buf[off:off + b.H * b.T].view(b.H, b.T)
    o = torch.empty_like(b.dq)
    ws = torch.empty(fa.fa_paged_fwd_workspace_bytes(b.kv, b.H, b.max_q), dtype=torch.uint8, device="cuda")
    fa.fa_paged_fwd(b.kv, b.dq, o, lse, b.dcu, b.max_q, ws)
    torch.cuda.synchronize()
    assert torch.equal(o, want) and torch.equal(lse, want_lse)
    assert (buf[:off] == 7.0).all() and (buf[off + b.H * b.T:] == 7.0).all()


# ------------------------------------------- what the kernels read is what is set
@pytest.mark.parametrize("struct,source", [("PagedFwdParams", "fa_paged_api.cu"), ("AppendParams", "fa_paged_api.cu"),
                                           ("RopeParams", "fa_paged_api.cu")])
def test_every_parameter_of_the_kernels_is_set(struct, source):
    """A field that a kernel reads and the host never sets leaves one of its paths
    to nobody."""
    import os
    import re
    csrc = os.path.join(os.path.dirname(fa.__file__), "csrc")
    with open(os.path.join(csrc, "fa_paged_internal.h")) as f:
        body = re.search(r"struct %s \{(.*?)\n\};" % struct, f.read(), re.S).group(1)
    with open(os.path.join(csrc, source)) as f:
        text = f.read()
    fields = []
    for line in re.sub(r"//.*", "", body).split(";"):
        names = line.replace("*", " ").split(",")
        fields += [n.split()[-1] for n in names if n.split()]
    unset = [f for f in fields if not re.search(r"\bp\.%s(\.\w+)? = |&p\.%s\b|\(p\.%s, " % (f, f, f), text)]
    assert fields and not unset, f"{struct}: nothing sets {unset}"


# ------------------------------------------------ a step that is refused as a whole
@gpu
def test_a_refused_step_leaves_the_cache_as_it_was():
    """paged_step stores before it attends: what the attention refuses must not
    have been stored, and nothing that was asked for may go unheard."""
    b = Batch([40, 33], [3, 2], 4, 2, 64, 16, "bf16", seed=17).cuda()
    f, _ = fa.rope_inv_freq(64)
    rope = fa.Rope(f)
    before = [x.clone().view(torch.int16) for x in (b.dk, b.dv)]
    pos = torch.arange(b.T, dtype=torch.int32, device="cuda")
    q3 = b.dq[:3].contiguous()
    wide = b.dq[:1].expand(4, -1, -1)                   # heads on top of one another
    same = dict(kv=b.kv, q=b.dq, k=b.dkn, v=b.dvn, cu_seqlens_q=b.dcu, max_seqlen_q=3)
    for match, kw in [("positions", dict(positions=pos)), ("scale", dict(scale=0.0)), ("scale", dict(scale=math.nan)),
                      ("scale", dict(rope=rope, scale=math.inf)), ("max_seqlen_q", dict(max_seqlen_q=-1)),
                      ("max_seqlen_q", dict(rope=rope, max_seqlen_q=2 ** 32)), ("Hq must be", dict(q=q3)),
                      ("Hq must be", dict(q=q3, rope=rope)), ("q must be", dict(q=None)),
                      ("must have shape", dict(q=b.dq[:, :4], rope=rope)), ("strides", dict(q=wide)),
                      ("cu_seqlens_q", dict(cu_seqlens_q=b.dcu[:2])), ("kv must be", dict(kv=None))]:
        with pytest.raises(fa.FaError, match=match):
            fa.paged_step(**dict(same, **kw))
    torch.cuda.synchronize()
    assert all(torch.equal(x.view(torch.int16), y) for x, y in zip((b.dk, b.dv), before))
    o, _ = fa.paged_step(**dict(same, q=wide, rope=rope))      # rotated into rows of their own: fine
    want, _ = fa.paged_step(**dict(same, q=wide.contiguous(), rope=rope))
    assert torch.equal(o, want)


def test_a_cache_without_heads_is_refused():
    k = torch.zeros(3, 0, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(fa.FaError, match="a head"):
        fa.PagedKV(k, k, torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, dtype=torch.int32))


# -------------------------------------------------------- entries outside the cache
@gpu
@pytest.mark.parametrize("rope", [False, True])
@pytest.mark.parametrize("tokens", [False, True])
@pytest.mark.parametrize("new", [[1, 1, 1], [40, 90, 5]])
def test_rows_for_pages_outside_the_cache_are_dropped(new, tokens, rope):
    """New rows whose table entry is -1 or num_pages.  The caches lie between
    canary pages of the same allocation, where such a row would be stored, and
    every other slot is compared bit by bit."""
    S, Hkv, D, pad = 16, 2, 64, 4
    b = Batch([70, 100, 33], new, 4, Hkv, D, S, "bf16", seed=33)
    P = b.k.shape[0]
    bad = [(0, 69 // S, -1), (1, 99 // S, P), (1, 10 // S, -1)]        # the first two hold their sequence's last row
    for s, i, entry in bad:
        b.table[s, i] = entry
    g = torch.Generator().manual_seed(1)
    big = [torch.randint(-2 ** 15, 2 ** 15, (P + 2 * pad, Hkv, S, D), generator=g, dtype=torch.int16) for _ in range(2)]
    for x, c in zip(big, (b.k, b.v)):
        x[pad:pad + P] = c.view(torch.int16)
    if tokens:
        dev = [x.transpose(1, 2).contiguous().cuda().transpose(1, 2) for x in big]
    else:
        dev = [x.cuda() for x in big]
    b.cuda()
    kv = fa.PagedKV(*(x[pad:pad + P].view(torch.bfloat16) for x in dev), b.table.cuda(), b.seq_lens.cuda())
    f, _ = fa.rope_inv_freq(64)
    if rope:
        qo = torch.full_like(b.dq, math.nan)
        fa.fa_paged_append(kv, b.dkn, b.dvn, b.dcu, rope=fa.Rope(f), q=b.dq, q_out=qo)
    else:
        fa.fa_paged_append(kv, b.dkn, b.dvn, b.dcu)
    torch.cuda.synchronize()
    got = [x.cpu() for x in dev]
    dropped = 0
    for s, n in enumerate(b.lens):
        for t in range(int(b.cu[s]), int(b.cu[s + 1])):
            at = n - int(b.cu[s + 1]) + t
            page = int(b.table[s, at // S])
            if not 0 <= page < P:
                dropped += 1
                continue
            if rope:        # within the bound; then as it came, so that the whole buffer can be compared
                x = b.k_new[:, t].double()[:, None]
                y = rope_ref(x, torch.tensor([at]), f.cpu())
                z = got[0][pad + page, :, at % S].view(torch.bfloat16).double()[:, None]
                assert ((z - y).abs() <= rope_tol(x, y, f.cpu(), torch.bfloat16)).all()
                big[0][pad + page, :, at % S] = got[0][pad + page, :, at % S]
            else:
                big[0][pad + page, :, at % S] = b.k_new[:, t].view(torch.int16)
            big[1][pad + page, :, at % S] = b.v_new[:, t].view(torch.int16)
    assert dropped >= 2 and all(torch.equal(x, y) for x, y in zip(got, big))
    if rope:                # the queries of dropped rows are rotated all the same
        assert not torch.isnan(qo).any()
