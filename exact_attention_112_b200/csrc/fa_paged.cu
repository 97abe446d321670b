// fa_paged.cu -- attention of a ragged batch of new tokens over a paged cache.
//
//     o_i = sum_j exp(s_ij - m_i) v_j / l_i,   s_ij = scale * q_i . k_j,
//     l_i = sum_j exp(s_ij - m_i),             lse_i = m_i + ln l_i
// over the keys j < len of row i's sequence, with causal also
// j <= i + len - new; head h reads kv head h / G.
//
// One block per row and head, one thread per key of a 128-key step.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fa_internal.h"
#include "fa_paged_internal.h"

namespace fa {
namespace {

__device__ __forceinline__ float neg_inf() { return __int_as_float(0xff800000); }

template <bool BF16>
__device__ __forceinline__ float to_f(uint16_t x) {
    if constexpr (BF16) return __uint_as_float(static_cast<uint32_t>(x) << 16);
    else return __half2float(__ushort_as_half(x));
}

template <int D, bool BF16>
__global__ void __launch_bounds__(128) fa_paged_rows_kernel(const PagedFwdParams p) {
    __shared__ float sq[D], sp[128], red[4];
    const int t = blockIdx.x, h = blockIdx.y, hk = h / p.G, tid = threadIdx.x;
    int b = 0;
    for (int i = 0; i < p.kv.num_seqs; i += 128)
        b += __syncthreads_count(i + tid < p.kv.num_seqs && p.cu[i + tid + 1] <= t);
    if (b >= p.kv.num_seqs) return;
    const PagedSeq s = paged_seq(b, p.cu, p.kv.seq_lens, p.T, p.max_q,
                                 static_cast<long long>(p.kv.max_pages) * p.kv.page_size);
    const int i = t - s.q0;
    if (i < 0 || i >= s.new_q) return;
    const int n = p.causal ? min(s.len_k, i + s.len_k - s.new_q + 1) : s.len_k;
    const uint16_t *q = static_cast<const uint16_t *>(p.q) + h * p.q_h + t * p.q_n;
    if (tid < D) sq[tid] = to_f<BF16>(q[tid]) * p.qk_scale_log2;
    __syncthreads();
    float m = neg_inf(), l = 0.f, acc = 0.f;
    for (int j0 = 0; j0 < n; j0 += 128) {
        const int j = j0 + tid;
        float x = neg_inf();
        if (j < n) {
            const long long page = p.kv.table[b * p.kv.table_stride + j / p.kv.page_size];
            x = 0.f;
            if (page >= 0 && page < p.kv.num_pages) {
                const uint16_t *k = static_cast<const uint16_t *>(p.kv.k) + page * p.kv.k_page + hk * p.kv.k_head +
                                    (j % p.kv.page_size) * p.kv.k_tok;
                for (int d = 0; d < D; ++d) x = fmaf(sq[d], to_f<BF16>(k[d]), x);
            }
        }
        float mx = x;
        for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        if ((tid & 31) == 0) red[tid >> 5] = mx;
        __syncthreads();
        const float mn = fmaxf(m, fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])));
        const float e = mn == neg_inf() ? 0.f : exp2f(x - mn);
        sp[tid] = e;
        float sum = e;
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        __syncthreads();
        if ((tid & 31) == 0) red[tid >> 5] = sum;
        __syncthreads();
        const float alpha = m == neg_inf() ? 0.f : exp2f(m - mn);
        l = l * alpha + ((red[0] + red[1]) + (red[2] + red[3]));
        m = mn;
        acc *= alpha;
        if (tid < D) {
            for (int jj = 0; jj < min(128, n - j0); ++jj) {
                const long long page = p.kv.table[b * p.kv.table_stride + (j0 + jj) / p.kv.page_size];
                if (page < 0 || page >= p.kv.num_pages) continue;
                acc = fmaf(sp[jj], to_f<BF16>(static_cast<const uint16_t *>(p.kv.v)[page * p.kv.v_page + hk * p.kv.v_head +
                                                                                    ((j0 + jj) % p.kv.page_size) * p.kv.v_tok + tid]), acc);
            }
        }
        __syncthreads();
    }
    if (tid < D) {
        const float r = l > 0.f ? acc / l : 0.f;
        uint16_t *o = static_cast<uint16_t *>(p.o) + h * p.o_h + t * p.o_n;
        if constexpr (BF16) o[tid] = __bfloat16_as_ushort(__float2bfloat16_rn(r));
        else o[tid] = __half_as_ushort(__float2half_rn(r));
    }
    if (tid == 0)
        p.lse[static_cast<long long>(h) * p.T + t] = l > 0.f ? (m + log2f(l)) * 0.69314718055994530942f : neg_inf();
}

}  // namespace

cudaError_t launch_paged_fwd(const PagedFwdParams &p, bool bf16, int sms, cudaStream_t stream) {
    (void)sms;
    const dim3 grid(p.T, p.H);
    auto kern = p.kv.D == 64 ? (bf16 ? fa_paged_rows_kernel<64, true> : fa_paged_rows_kernel<64, false>)
                             : (bf16 ? fa_paged_rows_kernel<128, true> : fa_paged_rows_kernel<128, false>);
    prof_begin(stream, "fa_paged_rows_kernel");
    kern<<<grid, 128, 0, stream>>>(p);
    prof_end(stream);
    note_launch();
    return cudaGetLastError();
}

}  // namespace fa
