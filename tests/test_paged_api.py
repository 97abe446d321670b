"""Refusals of the rotary-position and paged-cache entry points, all before any
CUDA call (no GPU needed)."""
import ctypes

import pytest
import torch

import exact_attention_112_b200 as fa
from exact_attention_112_b200 import _build, paged


@pytest.fixture(scope="module")
def L():
    _build.build()
    return fa.lib()


P = lambda x: None if not x else ctypes.c_void_p(16 * x)
S2 = lambda *a: (ctypes.c_longlong * 2)(*a)
S3 = lambda *a: (ctypes.c_longlong * 3)(*a)
BAD, UNSUP = fa.FA_ERR_INVALID_ARG, fa.FA_ERR_UNSUPPORTED


def _spec(inv=1, rot=64, inter=0, scale=1.0):
    return ctypes.byref(paged._RopeSpec(16 * inv if inv else None, rot, inter, scale))


@pytest.mark.parametrize("fn", ["fa_rope", "fa_rope_bwd"])
def test_rope_refusals(L, fn):
    def call(q=1, qo=2, Hq=4, k=3, ko=4, Hk=2, B=1, N=8, D=64, spec=None, qs=None, qos=None, ks=None, pos=0,
             pstride=0, pos0=0, dtype=1):
        return getattr(L, fn)(P(q), qs, P(qo), qos, Hq, P(k), ks, P(ko), None, Hk, B, N, D, spec or _spec(), P(pos),
                              pstride, pos0, dtype, None)

    assert call(N=0) == fa.FA_OK
    assert call(dtype=2) == UNSUP
    assert call(D=12) == UNSUP and call(D=520) == UNSUP
    assert call(B=0) == BAD and call(N=-1) == BAD and call(Hq=0) == BAD and call(pstride=-1) == BAD
    assert call(q=0) == BAD and call(qo=0) == BAD and call(k=0) == BAD and call(ko=0) == BAD
    assert call(Hk=0) == BAD                                   # a k without heads
    for s in (_spec(inv=0), _spec(rot=8), _spec(rot=24), _spec(rot=128), _spec(inter=2), _spec(scale=0.0),
              _spec(scale=float("nan"))):
        assert call(spec=s) == BAD
    assert getattr(L, fn)(P(1), None, P(2), None, 1, None, None, None, None, 0, 1, 8, 64, None, None, 0, 0, 1, None) == BAD
    assert call(qs=S3(512, 64, 4)) == BAD                      # rows on 8-byte boundaries
    assert call(qos=S3(0, 0, 64)) == BAD                       # an output whose heads overlap
    assert call(B=1 << 20, N=1 << 12) == BAD                   # too many rows
    assert call(pos0=2 ** 31 - 4) == BAD                       # the last position passes 31 bits
    q = ctypes.c_void_p(24)
    assert getattr(L, fn)(q, None, P(2), None, 1, None, None, None, None, 0, 1, 8, 64, _spec(), None, 0, 0, 1, None) == BAD


def _kv(k=1, v=2, ks=None, vs=None, table=3, tstride=4, lens=4, seqs=2, max_pages=4, pages=8, heads=2, page=16, D=64,
        dtype=1):
    run = page * D
    ks = ks or (heads * run, run, D)
    vs = vs or (heads * run, run, D)
    a = lambda x: 16 * x if x else None
    return ctypes.byref(paged._PagedSpec(a(k), a(v), S3(*ks), S3(*vs), a(table), tstride, a(lens), seqs, max_pages,
                                         pages, heads, page, D, dtype))


CACHES = [(dict(dtype=3), UNSUP), (dict(D=96), UNSUP), (dict(page=12), BAD), (dict(page=0), BAD), (dict(seqs=0), BAD),
          (dict(page=65544), BAD), (dict(pages=0), BAD), (dict(max_pages=0), BAD), (dict(heads=0), BAD), (dict(k=0), BAD),
          (dict(lens=0), BAD), (dict(table=0), BAD), (dict(tstride=3), BAD), (dict(ks=(2048, 1024, 60)), BAD),
          (dict(vs=(2048, 0, 64)), BAD), (dict(vs=(-2048, 1024, 64)), BAD), (dict(max_pages=1 << 27, tstride=1 << 27), BAD)]


@pytest.mark.parametrize("kw,want", CACHES)
def test_cache_refusals(L, kw, want):
    kv = _kv(**kw)
    assert L.fa_paged_append(kv, P(1), None, P(2), None, P(3), 4, None, None, None, None, None, None, 0, None) == want
    assert L.fa_paged_fwd(kv, P(1), None, P(2), None, P(3), P(4), 4, 1, 4, 1, 0.1, P(5), 1 << 30, None) == want
    assert L.fa_paged_fwd_workspace_bytes(kv, 4, 1) == 0


def test_append_refusals(L):
    def call(kv=None, k=1, v=2, cu=3, T=4, rope=None, q=0, qo=0, H=0, ks=None, qs=None, qos=None):
        return L.fa_paged_append(kv or _kv(), P(k), ks, P(v), None, P(cu), T, rope, None, P(q), qs, P(qo), qos, H, None)

    assert call(T=0) == fa.FA_OK
    assert call(k=0) == BAD and call(v=0) == BAD and call(cu=0) == BAD and call(T=-1) == BAD
    assert call(H=4, rope=_spec()) == BAD                      # no q
    assert call(q=5, qo=6, H=4) == BAD                         # q without a rope
    assert call(q=5, qo=6, H=0, rope=_spec()) == BAD
    assert call(rope=_spec(rot=128)) == BAD                    # more than the head
    assert call(ks=S2(256, 63)) == BAD
    assert call(q=5, qo=6, H=4, rope=_spec(), qos=S2(0, 64)) == BAD
    assert L.fa_paged_append(None, P(1), None, P(2), None, P(3), 4, None, None, None, None, None, None, 0, None) == BAD


def test_attention_refusals(L):
    def call(kv=None, q=1, qs=None, o=2, os_=None, lse=3, cu=4, T=4, mq=1, H=4, causal=1, scale=0.1, ws=5, nbytes=1 << 30):
        return L.fa_paged_fwd(kv or _kv(), P(q), qs, P(o), os_, P(lse), P(cu), T, mq, H, causal, scale, P(ws), nbytes, None)

    assert call(T=0) == fa.FA_OK and call(mq=0) == fa.FA_OK
    assert call(H=3) == BAD and call(H=0) == BAD and call(H=258) == BAD     # not a multiple; more than 128 a group
    assert call(T=-1) == BAD and call(mq=-1) == BAD and call(causal=2) == BAD
    assert call(scale=0.0) == BAD and call(scale=float("inf")) == BAD
    assert call(q=0) == BAD and call(o=0) == BAD and call(lse=0) == BAD and call(cu=0) == BAD
    assert call(qs=S2(256, 32)) == BAD and call(os_=S2(0, 64)) == BAD
    need = L.fa_paged_fwd_workspace_bytes(_kv(), 4, 1)
    assert need > 0
    assert call(ws=0) == fa.FA_ERR_WORKSPACE and call(nbytes=need - 1) == fa.FA_ERR_WORKSPACE
    assert L.fa_paged_fwd_workspace_bytes(_kv(), 3, 1) == 0 and L.fa_paged_fwd_workspace_bytes(_kv(), 4, -1) == 0


def _expect(match, fn, *a, **kw):
    with pytest.raises(fa.FaError, match=match) as e:
        fn(*a, **kw)
    return e.value.status


def test_handles_check_their_tensors(L):
    k = torch.zeros(3, 2, 16, 64, dtype=torch.bfloat16)
    t = torch.zeros(2, 2, dtype=torch.int32)
    n = torch.zeros(2, dtype=torch.int32)
    _expect("CUDA device", fa.PagedKV, k, k, t, n)             # everything right but on the host
    _expect("of one shape", fa.PagedKV, k, k[:, :1], t, n)
    _expect("must be torch.bfloat16", fa.PagedKV, k, k.half(), t, n)
    assert _expect("D must be", fa.PagedKV, k[..., :32], k[..., :32], t, n) == UNSUP
    assert _expect("dtype", fa.PagedKV, k.float(), k.float(), t, n) == UNSUP
    _expect("page_size", fa.PagedKV, k[:, :, :12], k[:, :, :12], t, n)
    _expect("page_table must be", fa.PagedKV, k, k, t.long(), n)
    _expect("seq_lens must be", fa.PagedKV, k, k, t, n[:1])
    _expect("strides", fa.PagedKV, k.expand(3, 2, 16, 64)[:1].expand(3, 2, 16, 64), k, t, n)
    _expect("rows must be contiguous", fa.PagedKV, k.transpose(2, 3).contiguous().transpose(2, 3), k, t, n)
    f = torch.ones(32, dtype=torch.float64)
    _expect("CUDA device", fa.Rope, f)
    _expect("float64", fa.Rope, f.float())
    _expect("multiple of 8", fa.Rope, f[:12])
    _expect("rope must be a Rope", fa.rope_forward, k, k, f)
    _expect("kv must be a PagedKV", fa.paged_attention, None, k[0], n, 1)
    _expect("kv must be a PagedKV", fa.fa_paged_append, None, k[0], k[0], n)
