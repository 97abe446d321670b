// fa_paged_api.cu -- the C ABI of the rotary-position and paged-cache operators
// (declared in include/fa.h): argument validation and launches.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <numeric>

#include "fa.h"
#include "fa_host.h"
#include "fa_internal.h"
#include "fa_paged_internal.h"

namespace {

bool aligned(const void *p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

int check_rope(const fa_rope_spec *r, int D) {
    if (!r || !r->inv_freq || !aligned(r->inv_freq, 8)) return FA_ERR_INVALID_ARG;
    if (r->rot_dim < 16 || r->rot_dim % 16 != 0 || r->rot_dim > D) return FA_ERR_INVALID_ARG;
    if (r->interleaved != 0 && r->interleaved != 1) return FA_ERR_INVALID_ARG;
    if (!std::isfinite(r->scale) || !(r->scale > 0.f)) return FA_ERR_INVALID_ARG;
    return FA_OK;
}

// Strides of a tensor with extents n[] (outermost first) and D contiguous
// values: given or contiguous; extents of 1 need none.  `low` is the least
// stride allowed.
template <int K>
int get_strides(const long long *given, const long long (&n)[K], int D, long long low, long long (&s)[K]) {
    long long run = D;
    for (int i = K - 1; i >= 0; --i) {
        s[i] = given ? given[i] : run;
        run *= n[i];
        if (n[i] <= 1) {
            s[i] = D;
            continue;
        }
        if (s[i] % 8 != 0 || s[i] < low || s[i] > (1LL << 38)) return FA_ERR_INVALID_ARG;
    }
    return FA_OK;
}

int rope_impl(const void *q, const long long *qs, void *qo, const long long *qos, int Hq, const void *k,
              const long long *ks, void *ko, const long long *kos, int Hk, int B, int N, int D,
              const fa_rope_spec *rope, const int *positions, long long pos_stride, int pos0, int dtype, void *stream,
              float sign) {
    if (B < 1 || Hq < 1 || Hk < 0 || N < 0 || pos_stride < 0) return FA_ERR_INVALID_ARG;
    if (dtype != FA_F16 && dtype != FA_BF16) return FA_ERR_UNSUPPORTED;
    if (D < 16 || D > 512 || D % 8 != 0) return FA_ERR_UNSUPPORTED;
    int st = check_rope(rope, D);
    if (st != FA_OK) return st;
    const long long rows = static_cast<long long>(B) * N;
    if (rows > INT32_MAX || rows * ((D + 15) / 16) > INT32_MAX || Hq > 65536 || Hk > 65536) return FA_ERR_INVALID_ARG;
    if (!positions && static_cast<long long>(pos0) + N > INT32_MAX) return FA_ERR_INVALID_ARG;
    if (N == 0) return FA_OK;
    if (!q || !qo || (Hk > 0 && (!k || !ko)) || (Hk == 0 && (k || ko))) return FA_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(qo, 16) || !aligned(k, 16) || !aligned(ko, 16) || !aligned(positions, 4))
        return FA_ERR_INVALID_ARG;
    fa::RopeParams p{};
    long long s[3];
    auto fill = [&](fa::RopeTensor &t, const void *in, const long long *is, void *out, const long long *os, int H) {
        const long long n[3] = {B, H, N};
        int e = get_strides(is, n, D, 0, s);
        if (e != FA_OK) return e;
        t.in = in;
        t.out = out;
        t.H = H;
        t.in_b = s[0]; t.in_h = s[1]; t.in_n = s[2];
        if ((e = get_strides(os, n, D, D, s)) != FA_OK) return e;
        t.out_b = s[0]; t.out_h = s[1]; t.out_n = s[2];
        return static_cast<int>(FA_OK);
    };
    if ((st = fill(p.q, q, qs, qo, qos, Hq)) != FA_OK) return st;
    if (Hk > 0 && (st = fill(p.k, k, ks, ko, kos, Hk)) != FA_OK) return st;
    p.B = B;
    p.N = N;
    p.D = D;
    p.rot = rope->rot_dim;
    p.interleaved = rope->interleaved;
    p.scale = rope->scale;
    p.sign = sign;
    p.inv_freq = rope->inv_freq;
    p.positions = positions;
    p.pos_stride = pos_stride;
    p.pos0 = pos0;
    int *err = nullptr, sms = 1;
    if ((st = fa::host_device(&err, &sms)) != FA_OK) return st;
    return fa::launch_rope(p, dtype == FA_BF16, sms, static_cast<cudaStream_t>(stream)) == cudaSuccess ? FA_OK
                                                                                                       : FA_ERR_CUDA;
}

int check_cache(const fa_paged_kv *kv, fa::PagedCache *c) {
    if (!kv) return FA_ERR_INVALID_ARG;
    if (kv->dtype != FA_F16 && kv->dtype != FA_BF16) return FA_ERR_UNSUPPORTED;
    if (kv->D != 64 && kv->D != 128) return FA_ERR_UNSUPPORTED;
    if (kv->num_seqs < 1 || kv->max_pages < 1 || kv->num_pages < 1 || kv->num_kv_heads < 1) return FA_ERR_INVALID_ARG;
    if (kv->page_size < 8 || kv->page_size % 8 != 0 || kv->page_size > 65536) return FA_ERR_INVALID_ARG;
    if (static_cast<long long>(kv->max_pages) * kv->page_size > (1 << 30)) return FA_ERR_INVALID_ARG;
    if (kv->num_seqs > (1 << 24) || kv->num_kv_heads > 65536) return FA_ERR_INVALID_ARG;
    if (!kv->k_cache || !kv->v_cache || !kv->seq_lens || !kv->page_table) return FA_ERR_INVALID_ARG;
    if (!aligned(kv->k_cache, 16) || !aligned(kv->v_cache, 16) || !aligned(kv->page_table, 4) ||
        !aligned(kv->seq_lens, 4))
        return FA_ERR_INVALID_ARG;
    if (kv->num_seqs > 1 && kv->table_stride < kv->max_pages) return FA_ERR_INVALID_ARG;
    const long long n[3] = {kv->num_pages, kv->num_kv_heads, kv->page_size};
    long long s[3];
    int st;
    if ((st = get_strides(kv->k_strides, n, kv->D, kv->D, s)) != FA_OK) return st;
    c->k_page = s[0]; c->k_head = s[1]; c->k_tok = s[2];
    if ((st = get_strides(kv->v_strides, n, kv->D, kv->D, s)) != FA_OK) return st;
    c->v_page = s[0]; c->v_head = s[1]; c->v_tok = s[2];
    c->k = kv->k_cache;
    c->v = kv->v_cache;
    c->table = kv->page_table;
    c->table_stride = kv->table_stride;
    c->seq_lens = kv->seq_lens;
    c->num_seqs = kv->num_seqs;
    c->max_pages = kv->max_pages;
    c->num_pages = kv->num_pages;
    c->page_size = kv->page_size;
    c->Hkv = kv->num_kv_heads;
    c->D = kv->D;
    return FA_OK;
}

// Shape of the work of a call: how many tokens make a tile of 128 query rows
// (a token has G rows, one per head of the group) and a unit of two tiles.
fa::SchedGeom sched_geom(int G, int max_q) {
    fa::SchedGeom g;
    g.tile_tokens = std::max(1, std::min(128 / G, max_q));
    g.unit_tokens = std::max(1, std::min(2 * (128 / G), max_q));
    // Costs, measured at D = 128: single tokens take 1.5 us a key tile (the memory's
    // rate) and 2 us a unit; in the kernel of row tiles a key tile takes 1.34..1.57 us
    // with one, 1.79..2.02 us with two of them, a unit 3.2 us.  D = 64 goes by the
    // same ones, though its key tiles with one row tile are cheaper (0.90..0.96 us,
    // with two 1.66..1.79): units of both kinds in a batch are shared out less evenly.
    if (max_q * G <= fa::kPagedTokenRows) {
        g.tile_tokens = g.unit_tokens;      // one unit per sequence and kv head
        g.unit_cost = 3;
        g.one_cost = g.two_cost = 2;
    } else {
        g.unit_cost = 20;
        g.one_cost = 9;
        g.two_cost = 12;
    }
    return g;
}

struct PagedWorkspace {
    size_t lse, meta, bytes;    // offsets of the parts after the partial rows
};

PagedWorkspace paged_workspace(const fa::SchedGeom &g, int G, int D) {
    const size_t rows = static_cast<size_t>(2) * fa::kPagedMaxCtas * g.unit_tokens * G;
    PagedWorkspace w;
    w.lse = rows * D * sizeof(float);
    w.meta = w.lse + (rows * sizeof(float) + 15) / 16 * 16;
    w.bytes = w.meta + fa::kPagedMaxCtas * sizeof(fa::MergeMeta);
    return w;
}

// Pages and heads as one dimension: index page * ratio + head, `extent` entries
// (0: not possible) `stride` elements apart.
struct PageFold {
    int ratio;
    long long extent, stride;
};

PageFold page_fold(const fa::PagedCache &c, long long page, long long head) {
    PageFold f{1, 0, 0};
    if (c.Hkv == 1) {
        f.stride = page;
    } else if (c.num_pages == 1 || page % head == 0) {
        const long long r = c.num_pages == 1 ? 0 : page / head;
        if (r > INT32_MAX) return f;
        f.ratio = static_cast<int>(r);
        f.stride = head;
    } else {
        return f;
    }
    const long long n = static_cast<long long>(c.num_pages - 1) * f.ratio + c.Hkv;
    if (n <= INT32_MAX) f.extent = n;
    return f;
}

int encode(CUtensorMap *m, const void *ptr, bool bf16, int rank, const cuuint64_t *dims, const long long *strides,
           const cuuint32_t *box) {
    PFN_cuTensorMapEncodeTiled_v12000 enc;
    const int st = fa::host_encoder(&enc);
    if (st != FA_OK) return st;
    cuuint64_t bytes[4];
    for (int i = 0; i + 1 < rank; ++i) bytes[i] = static_cast<cuuint64_t>(strides[i]) * 2;
    const cuuint32_t one[5] = {1, 1, 1, 1, 1};
    const CUresult r = enc(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, rank,
                           const_cast<void *>(ptr), dims, bytes, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                           CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? FA_OK : FA_ERR_CUDA;
}

}  // namespace

extern "C" {

int fa_rope(const void *q, const long long *q_strides, void *q_out, const long long *q_out_strides, int Hq,
            const void *k, const long long *k_strides, void *k_out, const long long *k_out_strides, int Hk, int B,
            int N, int D, const fa_rope_spec *rope, const int *positions, long long pos_stride, int pos0, int dtype,
            void *stream) {
    return rope_impl(q, q_strides, q_out, q_out_strides, Hq, k, k_strides, k_out, k_out_strides, Hk, B, N, D, rope,
                     positions, pos_stride, pos0, dtype, stream, 1.f);
}

int fa_rope_bwd(const void *dq_out, const long long *dq_out_strides, void *dq, const long long *dq_strides, int Hq,
                const void *dk_out, const long long *dk_out_strides, void *dk, const long long *dk_strides, int Hk,
                int B, int N, int D, const fa_rope_spec *rope, const int *positions, long long pos_stride, int pos0,
                int dtype, void *stream) {
    return rope_impl(dq_out, dq_out_strides, dq, dq_strides, Hq, dk_out, dk_out_strides, dk, dk_strides, Hk, B, N, D,
                     rope, positions, pos_stride, pos0, dtype, stream, -1.f);
}

int fa_paged_append(const fa_paged_kv *kv, const void *k, const long long *k_strides, const void *v,
                    const long long *v_strides, const int *cu_seqlens_q, int total_q, const fa_rope_spec *rope,
                    const int *positions, const void *q, const long long *q_strides, void *q_out,
                    const long long *q_out_strides, int Hq, void *stream) {
    fa::AppendParams p{};
    int st = check_cache(kv, &p.kv);
    if (st != FA_OK) return st;
    if (total_q < 0 || total_q > (1 << 28) || Hq < 0 || Hq > 65536) return FA_ERR_INVALID_ARG;
    if (rope && (st = check_rope(rope, kv->D)) != FA_OK) return st;
    if (Hq == 0 ? (q || q_out) : !rope) return FA_ERR_INVALID_ARG;
    if (!cu_seqlens_q || !aligned(cu_seqlens_q, 4) || !aligned(positions, 4)) return FA_ERR_INVALID_ARG;
    if (total_q == 0) return FA_OK;
    if (!k || !v || (Hq > 0 && (!q || !q_out))) return FA_ERR_INVALID_ARG;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(q, 16) || !aligned(q_out, 16)) return FA_ERR_INVALID_ARG;
    const long long nk[2] = {kv->num_kv_heads, total_q}, nq[2] = {Hq, total_q};
    long long s[2];
    if ((st = get_strides(k_strides, nk, kv->D, 0, s)) != FA_OK) return st;
    p.k_h = s[0]; p.k_n = s[1];
    if ((st = get_strides(v_strides, nk, kv->D, 0, s)) != FA_OK) return st;
    p.v_h = s[0]; p.v_n = s[1];
    if ((st = get_strides(q_strides, nq, kv->D, 0, s)) != FA_OK) return st;
    p.q_h = s[0]; p.q_n = s[1];
    if ((st = get_strides(q_out_strides, nq, kv->D, kv->D, s)) != FA_OK) return st;
    p.qo_h = s[0]; p.qo_n = s[1];
    p.k = k;
    p.v = v;
    p.q = q;
    p.q_out = q_out;
    p.H = Hq;
    p.T = total_q;
    p.cu = cu_seqlens_q;
    if (rope) {
        p.rot = rope->rot_dim;
        p.interleaved = rope->interleaved;
        p.scale = rope->scale;
        p.inv_freq = rope->inv_freq;
        p.positions = positions;
    }
    int *err = nullptr, sms = 1;
    if ((st = fa::host_device(&err, &sms)) != FA_OK) return st;
    return fa::launch_paged_append(p, kv->dtype == FA_BF16, sms, static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? FA_OK : FA_ERR_CUDA;
}

size_t fa_paged_fwd_workspace_bytes(const fa_paged_kv *kv, int Hq, int max_seqlen_q) {
    fa::PagedCache c;
    if (check_cache(kv, &c) != FA_OK || Hq < 1 || Hq % c.Hkv != 0 || Hq / c.Hkv > 128 || max_seqlen_q < 0) return 0;
    return paged_workspace(sched_geom(Hq / c.Hkv, max_seqlen_q), Hq / c.Hkv, c.D).bytes;
}

int fa_paged_fwd(const fa_paged_kv *kv, const void *q, const long long *q_strides, void *o,
                 const long long *o_strides, float *lse, const int *cu_seqlens_q, int total_q, int max_seqlen_q,
                 int Hq, int causal, float scale, void *workspace, size_t workspace_bytes, void *stream) {
    fa::PagedFwdParams p{};
    int st = check_cache(kv, &p.kv);
    if (st != FA_OK) return st;
    if (Hq < 1 || Hq % kv->num_kv_heads != 0 || Hq / kv->num_kv_heads > 128) return FA_ERR_INVALID_ARG;
    if (total_q < 0 || max_seqlen_q < 0 || (causal != 0 && causal != 1)) return FA_ERR_INVALID_ARG;
    if (static_cast<long long>(Hq) * total_q > INT32_MAX || total_q > (1 << 28)) return FA_ERR_INVALID_ARG;
    if (!std::isfinite(scale) || !(scale > 0.f)) return FA_ERR_INVALID_ARG;
    if (!cu_seqlens_q || !aligned(cu_seqlens_q, 4)) return FA_ERR_INVALID_ARG;
    if (total_q == 0 || max_seqlen_q == 0) return FA_OK;
    if (!q || !o || !lse) return FA_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(o, 16) || !aligned(lse, 4) || !aligned(workspace, 16)) return FA_ERR_INVALID_ARG;
    const long long n[2] = {Hq, total_q};
    long long s[2];
    if ((st = get_strides(q_strides, n, kv->D, kv->D, s)) != FA_OK) return st;
    const long long q_h = s[0], q_n = s[1];
    if ((st = get_strides(o_strides, n, kv->D, kv->D, s)) != FA_OK) return st;
    p.o_h = s[0]; p.o_n = s[1];
    if (!workspace || workspace_bytes < fa_paged_fwd_workspace_bytes(kv, Hq, max_seqlen_q)) return FA_ERR_WORKSPACE;
    const int G = Hq / kv->num_kv_heads, D = kv->D;
    const bool bf16 = kv->dtype == FA_BF16;
    p.o = o;
    p.o_v8 = aligned(o, 32) && p.o_h % 16 == 0 && p.o_n % 16 == 0;
    p.lse = lse;
    p.cu = cu_seqlens_q;
    p.T = total_q;
    p.max_q = max_seqlen_q < total_q ? max_seqlen_q : total_q;
    p.H = Hq;
    p.G = G;
    p.causal = causal;
    p.qk_scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634074);
    p.geom = sched_geom(G, p.max_q);
    p.part_rows = p.geom.unit_tokens * G;
    const bool tokens = p.part_rows <= fa::kPagedTokenRows;
    // a key tile at least; two for the kernel of row tiles, which works on two at
    // a time (half a piece holds the first entry of some key tile)
    p.min_piece = tokens ? 2 : 24;
    const PagedWorkspace w = paged_workspace(p.geom, G, D);
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    p.o_part = reinterpret_cast<float *>(ws);
    p.lse_part = reinterpret_cast<float *>(ws + w.lse);
    p.meta = reinterpret_cast<fa::MergeMeta *>(ws + w.meta);
    int sms = 1;
    if ((st = fa::host_device(&p.err, &sms)) != FA_OK) return st;
    p.timeout_ns = fa::host_wait_limit_ns();
    fa::PagedTensorMaps tm;
    {   // rows in the order (token, head of the group): a box is a tile of query rows
        const cuuint64_t dims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(Hq),
                                    static_cast<cuuint64_t>(total_q)};
        const long long str[2] = {q_h, q_n};
        const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(G), static_cast<cuuint32_t>(p.geom.tile_tokens)};
        if ((st = encode(&tm.q, q, bf16, 3, dims, str, box)) != FA_OK) return st;
    }
    // The caches as [.., 8 rows, D / 64, 64]: a box is a run of a page's rows, one
    // head.  With five dimensions there is room for the groups of eight rows or for
    // the head; pages and heads become one dimension where the page stride is a
    // multiple of the head stride (any cache without odd padding), else a box is
    // eight rows.
    const PageFold kf = page_fold(p.kv, p.kv.k_page, p.kv.k_head), vf = page_fold(p.kv, p.kv.v_page, p.kv.v_head);
    p.fold = kf.extent > 0 && vf.extent > 0;
    p.box = p.fold ? std::gcd(kv->page_size, 128) : 8;
    p.k_ratio = kf.ratio;
    p.v_ratio = vf.ratio;
    for (int i = 0; i < 2; ++i) {
        const long long tok = i ? p.kv.v_tok : p.kv.k_tok, head = i ? p.kv.v_head : p.kv.k_head;
        const PageFold &f = i ? vf : kf;
        cuuint64_t dims[5] = {64, 8, static_cast<cuuint64_t>(D / 64)};
        long long str[4] = {tok, 64};
        cuuint32_t box[5] = {64, 8, static_cast<cuuint32_t>(D / 64), 1, 1};
        if (p.fold) {
            dims[3] = kv->page_size / 8;
            str[2] = 8 * tok;
            box[3] = p.box / 8;
            dims[4] = f.extent;
            str[3] = f.stride;
        } else {
            dims[1] = kv->page_size;
            dims[3] = kv->num_kv_heads;
            str[2] = head;
            dims[4] = kv->num_pages;
            str[3] = i ? p.kv.v_page : p.kv.k_page;
        }
        if ((st = encode(i ? &tm.v : &tm.k, i ? p.kv.v : p.kv.k, bf16, 5, dims, str, box)) != FA_OK) return st;
    }
    const auto launch = tokens ? fa::launch_paged_tokens : fa::launch_paged_fwd;
    return launch(tm, p, bf16, sms, static_cast<cudaStream_t>(stream)) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // extern "C"
