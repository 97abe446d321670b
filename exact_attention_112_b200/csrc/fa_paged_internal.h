// fa_paged_internal.h -- structures shared between the C-ABI layer and the
// kernels of the rotary-position and paged-cache operators.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace fa {

// ---------------------------------------------------------------- rotation
// One 16-bit tensor [B, H, N, D] seen through its strides (elements), D
// contiguous.  H == 0: absent.
struct RopeTensor {
    const void *in;
    void *out;
    long long in_b, in_h, in_n;
    long long out_b, out_h, out_n;
    int H;
};

struct RopeParams {
    RopeTensor q, k;
    int B, N, D;
    int rot;                   // rotated values per row, a multiple of 16
    int interleaved;           // pairs (2i, 2i+1) instead of (i, i + rot/2)
    float scale;               // multiplies cos and sin
    float sign;                // +1 forward, -1 transpose (backward)
    const double *inv_freq;    // [rot / 2] radians per position
    const int *positions;      // [B or 1, N] or nullptr
    long long pos_stride;      // between batches (0: shared)
    int pos0;                  // position of row 0 without a table
};

cudaError_t launch_rope(const RopeParams &p, bool bf16, int sms, cudaStream_t stream);

// ------------------------------------------------------------- paged cache
// The cache as the kernels see it: key t of sequence b lies in page
// table[b][t / page_size], row t % page_size.
struct PagedCache {
    void *k, *v;
    long long k_page, k_head, k_tok;    // strides in elements
    long long v_page, v_head, v_tok;
    const int *table;
    long long table_stride;
    const int *seq_lens;
    int num_seqs, max_pages, num_pages, page_size, Hkv, D;
};

struct AppendParams {
    PagedCache kv;
    const void *k, *v;                  // [Hkv, T, D] new rows
    long long k_h, k_n, v_h, v_n;
    const void *q;                      // [H, T, D] or nullptr
    void *q_out;
    long long q_h, q_n, qo_h, qo_n;
    int H;                              // query heads (0: no queries)
    int T;
    const int *cu;                      // [num_seqs + 1]
    int rot, interleaved;               // rot 0: nothing is rotated
    float scale;
    const double *inv_freq;
    const int *positions;               // [T] or nullptr (the cache position)
};

cudaError_t launch_paged_append(const AppendParams &p, bool bf16, int sms, cudaStream_t stream);

// Sequence b of the batch: its first new row in the packed tensors, the new rows
// to be computed and keys, every table entry clamped so that no access can leave
// the tensors.  Row i of them is key i + past of the sequence (the row after the
// last new one being key len_k), however few of the rows max_q leaves.
struct PagedSeq {
    int q0, new_q, len_k, past;
};

__host__ __device__ inline PagedSeq paged_seq(int b, const int *cu, const int *seq_lens, int total_q, int max_q,
                                              long long capacity) {
    PagedSeq s;
    s.q0 = min(max(cu[b], 0), total_q);
    const int end = max(cu[b + 1], s.q0);
    s.new_q = min(end - s.q0, min(max_q, total_q - s.q0));
    const long long len = seq_lens[b];
    s.len_k = static_cast<int>(len < 0 ? 0 : (len < capacity ? len : capacity));    // at most 2^30
    s.past = s.len_k - (end - s.q0);
    return s;
}

// Shape of the work units (fa_paged_sched.cuh).
constexpr int kPagedTile = 128;         // keys per tile

struct SchedGeom {
    int unit_tokens;    // tokens per unit
    int tile_tokens;    // tokens per tile of query rows (a unit past it has two)
    int unit_cost;              // entries that a unit counts by itself,
    int one_cost, two_cost;     // and each of its key tiles, with one or two row tiles
};

// What the merge kernel reads of CTA c: the unit that c begins and does not
// end (last < 0: none).
struct MergeMeta {
    int row0, tokens, h, last;
};

constexpr int kPagedMaxCtas = 148;      // CTAs that share the work (partial results: two each)

struct PagedFwdParams {
    PagedCache kv;
    void *o;                            // [H, T, D]
    long long o_h, o_n;
    float *lse;                         // [H, T]
    const int *cu;
    int T, max_q, H, G;                 // G = H / Hkv
    int causal;
    float qk_scale_log2;
    SchedGeom geom;
    int min_piece;                      // least entries worth a CTA
    int box;                            // keys per TMA box: gcd(page_size, 128), 8 without fold
    int fold;                           // pages and heads are one dimension of the tensor maps
    int k_ratio, v_ratio;               // index (page, head) of that dimension: page * ratio + head
    int o_v8;                           // rows of o start 32-byte aligned
    int part_rows;                      // rows of a partial result: unit_tokens * G
    float *o_part;                      // [2 * kPagedMaxCtas, part_rows, D]
    float *lse_part;                    // [2 * kPagedMaxCtas, part_rows], base-2
    MergeMeta *meta;                    // [kPagedMaxCtas]
    int *err;
    unsigned long long timeout_ns;
};

struct PagedTensorMaps {
    CUtensorMap q, k, v;
};

// Tiles of 128 query rows.
cudaError_t launch_paged_fwd(const PagedTensorMaps &tm, const PagedFwdParams &p, bool bf16, int sms,
                             cudaStream_t stream);
// All new tokens of a sequence in one unit of at most kPagedTokenRows query
// rows (geom.unit_tokens * G).
constexpr int kPagedTokenRows = 64;
cudaError_t launch_paged_tokens(const PagedTensorMaps &tm, const PagedFwdParams &p, bool bf16, int sms,
                                cudaStream_t stream);
// Launches a kernel that may be set up while the grid before it in the stream
// still runs; the kernel waits for that one itself (grid_dependency_wait()).
template <typename... Params, typename... Args>
cudaError_t launch_early(void (*kern)(Params...), dim3 grid, int threads, size_t smem, cudaStream_t stream,
                         const Args &...args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, args...);
    return e != cudaSuccess ? e : cudaGetLastError();
}

// Joins the partial results, after either.
cudaError_t launch_paged_merge(const PagedFwdParams &p, bool bf16, int grid, cudaStream_t stream);

}  // namespace fa
