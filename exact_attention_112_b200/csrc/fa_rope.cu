// fa_rope.cu -- rotary positions of queries and keys, and the appending of new
// keys and values to a paged cache with the keys rotated on the way.
//
// Rotation of the pair (a, b) of a row at position p by theta = p * f_i:
//     a' = s (a cos theta - b sin theta),   b' = s (b cos theta + a sin theta)
// with pairs (i, i + rot/2) or (2i, 2i + 1), s the attention factor of a
// long-context scaling rule, and the values past rot left as they are.  The
// gradient is the transpose: the same with -theta.
//
// The angle.  In 32 bits p * f_i is off by half a unit in the last place of
// the product, 0.03 rad at p = 2^20.  Here the frequency is held in turns as a
// 64-bit fixed-point fraction F = f / (2 pi) * 2^64 (rounded from float64) and
// p * F is taken modulo 2^64 by the wrap-around of an integer product: the
// fraction of a turn, exact but for F's rounding (p * 2^-55 turns), whatever
// p's sign and size.  Its top 32 bits, as a signed number, are the angle in
// [-1/2, 1/2) turns for sincospif().
//
// Bound by memory: 4 bytes moved per value and about 3 operations.  A thread
// owns eight pairs of one token (two 16-byte vectors), computes their eight
// angles once and applies them to a group of heads, so that the sines cost
// little next to the copies; the groups are as large as leaves the GPU full.
// The first four heads' vectors are asked for before the angles (the append:
// the tables) are looked at, and 80 registers let three blocks share an SM (64
// spill: slower).  Measured: q and k of 32 + 8 heads, N = 8192, D = 128 (168 MB)
// 30.0 us, 5.60 TB/s; four such batches 104 us, 6.4 TB/s; 401 MB of prompt rows
// appended in 68.9 us, 5.83 TB/s; one token's append 3.5 us.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "fa_internal.h"
#include "fa_paged_internal.h"
#include "fa_paged_ptx.cuh"

namespace fa {
namespace {

constexpr int kRopeThreads = 256;

template <bool BF16>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
    if constexpr (BF16) {
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    } else {
        return __half22float2(*reinterpret_cast<__half2 *>(&w));
    }
}

template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    if constexpr (BF16) {
        __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<uint32_t *>(&h);
    } else {
        __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<uint32_t *>(&h);
    }
}

// Radians per position -> turns per position as a fraction of 2^64.
__device__ __forceinline__ unsigned long long turns_fixed(double f) {
    double t = f * 0.15915494309189533577;     // 1 / (2 pi)
    t -= floor(t);
    return __double2ull_rn(t * 18446744073709551616.0);
}

// Cosines and sines of eight pairs at one position.
struct Angles {
    float c[8], s[8];
    __device__ __forceinline__ void set(const double *inv_freq, int pos, float scale, float sign) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const unsigned long long a =
                static_cast<unsigned long long>(static_cast<long long>(pos)) * turns_fixed(__ldg(inv_freq + e));
            // half turns in [-1, 1)
            const float x = static_cast<float>(static_cast<int>(a >> 32)) * 4.656612873077393e-10f;   // 2^-31
            float sn, cs;
            sincospif(x, &sn, &cs);
            c[e] = cs * scale;
            s[e] = sn * scale * sign;
        }
    }
};

// The two vectors of a unit: half layout, a's and b's of eight pairs;
// interleaved, four pairs in each.
template <bool BF16, bool INTER>
__device__ __forceinline__ void rotate(uint4 &u, uint4 &w, const Angles &an) {
    uint32_t *x = reinterpret_cast<uint32_t *>(&u), *y = reinterpret_cast<uint32_t *>(&w);
    if constexpr (INTER) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 p = unpack2<BF16>(x[e]), q = unpack2<BF16>(y[e]);
            x[e] = pack2<BF16>(p.x * an.c[e] - p.y * an.s[e], p.y * an.c[e] + p.x * an.s[e]);
            y[e] = pack2<BF16>(q.x * an.c[e + 4] - q.y * an.s[e + 4], q.y * an.c[e + 4] + q.x * an.s[e + 4]);
        }
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 a = unpack2<BF16>(x[e]), b = unpack2<BF16>(y[e]);
            const float c0 = an.c[2 * e], s0 = an.s[2 * e], c1 = an.c[2 * e + 1], s1 = an.s[2 * e + 1];
            x[e] = pack2<BF16>(a.x * c0 - b.x * s0, a.y * c1 - b.y * s1);
            y[e] = pack2<BF16>(b.x * c0 + a.x * s0, b.y * c1 + a.y * s1);
        }
    }
}

// Offsets of the two vectors of unit u of a row: units below rot / 16 are
// rotated, the others copy 16 values past rot (the last may hold only eight).
template <bool INTER>
__device__ __forceinline__ void unit_offsets(int u, int rot, int D, int &o0, int &o1, bool &turn) {
    turn = u < rot / 16;
    if (turn) {
        o0 = INTER ? 16 * u : 8 * u;
        o1 = INTER ? o0 + 8 : o0 + rot / 2;
    } else {
        o0 = 16 * u;
        o1 = o0 + 8 < D ? o0 + 8 : -1;
    }
}

template <bool BF16, bool INTER>
__global__ void __launch_bounds__(kRopeThreads, 3) fa_rope_kernel(const RopeParams p, int heads_per_group) {
    const int units = (p.D + 15) / 16;
    const long long tokens = static_cast<long long>(p.B) * p.N;
    const long long idx = static_cast<long long>(blockIdx.x) * kRopeThreads + threadIdx.x;
    const long long tok = idx / units;
    if (tok >= tokens) return;
    const int u = static_cast<int>(idx - tok * units);
    const int b = static_cast<int>(tok / p.N), n = static_cast<int>(tok - static_cast<long long>(b) * p.N);
    int o0, o1;
    bool turn;
    unit_offsets<INTER>(u, p.rot, p.D, o0, o1, turn);
    const int all = p.q.H + p.k.H;
    const int h_end = min(static_cast<int>(blockIdx.y + 1) * heads_per_group, all);
    int h0 = blockIdx.y * heads_per_group;
    uint4 x[4], y[4];
    auto load = [&]() {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int h = min(h0 + j, h_end - 1);
            const bool isq = h < p.q.H;
            const RopeTensor &t = isq ? p.q : p.k;
            const uint16_t *src = static_cast<const uint16_t *>(t.in) + b * t.in_b + (isq ? h : h - p.q.H) * t.in_h + n * t.in_n;
            x[j] = *reinterpret_cast<const uint4 *>(src + o0);
            if (o1 >= 0) y[j] = *reinterpret_cast<const uint4 *>(src + o1);
        }
    };
    load();     // on their way while the angles are computed
    Angles an;
    if (turn) {
        const int pos = p.positions ? __ldg(p.positions + b * p.pos_stride + n) : p.pos0 + n;
        an.set(p.inv_freq + 8 * u, pos, p.scale, p.sign);
    }
    for (;;) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int h = h0 + j;
            if (h >= h_end) break;
            const bool isq = h < p.q.H;
            const RopeTensor &t = isq ? p.q : p.k;
            uint16_t *dst = static_cast<uint16_t *>(t.out) + b * t.out_b + (isq ? h : h - p.q.H) * t.out_h + n * t.out_n;
            if (turn) rotate<BF16, INTER>(x[j], y[j], an);
            *reinterpret_cast<uint4 *>(dst + o0) = x[j];
            if (o1 >= 0) *reinterpret_cast<uint4 *>(dst + o1) = y[j];
        }
        h0 += 4;
        if (h0 >= h_end) break;
        load();
    }
}

// New keys (rotated) and values into the cache's pages, and the queries
// rotated into q_out.  A thread owns a unit of one token and a group of the
// H + 2 Hkv rows of that token.  Tokens of no sequence, and positions whose
// page the table does not give, are left alone.
template <bool BF16, bool INTER>
__global__ void __launch_bounds__(kRopeThreads, 3) fa_paged_append_kernel(const AppendParams p, int heads_per_group) {
    grid_launch_dependents();       // the attention after it may be set up; it waits for this grid
    const int D = p.kv.D;
    const int units = D / 16;
    const int per_block = kRopeThreads / units;
    const int t0 = blockIdx.x * per_block;
    const int lt = threadIdx.x / units, u = threadIdx.x - lt * units;
    const int t = t0 + lt;
    const bool live = lt < per_block && t < p.T;
    int o0, o1;
    bool turn;
    unit_offsets<INTER>(u, p.rot, D, o0, o1, turn);
    const int all = p.H + 2 * p.kv.Hkv;
    const int h_end = min(static_cast<int>(blockIdx.y + 1) * heads_per_group, all);
    int h0 = blockIdx.y * heads_per_group;
    uint4 x[4], y[4];
    auto load = [&]() {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int h = min(h0 + j, h_end - 1);
            const uint16_t *src;
            if (h < p.H)
                src = static_cast<const uint16_t *>(p.q) + h * p.q_h + t * p.q_n;
            else if (h < p.H + p.kv.Hkv)
                src = static_cast<const uint16_t *>(p.k) + (h - p.H) * p.k_h + t * p.k_n;
            else
                src = static_cast<const uint16_t *>(p.v) + (h - p.H - p.kv.Hkv) * p.v_h + t * p.v_n;
            x[j] = *reinterpret_cast<const uint4 *>(src + o0);
            y[j] = *reinterpret_cast<const uint4 *>(src + o1);
        }
    };
    // the first rows are on their way while the tables are searched
    if (live) load();
    // the sequence of the block's first token: how many sequences end at or before it
    int b = 0;
    for (int i = 0; i < p.kv.num_seqs; i += kRopeThreads) {
        const int s = i + threadIdx.x;
        b += __syncthreads_count(s < p.kv.num_seqs && __ldg(p.cu + s + 1) <= t0);
    }
    if (!live) return;
    while (b < p.kv.num_seqs && __ldg(p.cu + b + 1) <= t) ++b;
    if (b >= p.kv.num_seqs) return;
    const int first = __ldg(p.cu + b), end = __ldg(p.cu + b + 1);
    if (t < first) return;
    // position in the sequence: its last token sits at length - 1, the length clamped
    // as the attention's
    const int capacity = p.kv.max_pages * p.kv.page_size;       // at most 2^30
    const long long at = static_cast<long long>(min(max(__ldg(p.kv.seq_lens + b), 0), capacity)) - end + t;
    long long page = -1;
    int row = 0;
    if (at >= 0 && at < capacity) {
        const int pi = static_cast<int>(at) / p.kv.page_size;
        row = static_cast<int>(at) - pi * p.kv.page_size;
        page = __ldg(p.kv.table + b * p.kv.table_stride + pi);
        if (page >= p.kv.num_pages) page = -1;
    }
    Angles an;
    if (turn) {
        const int pos = p.positions ? __ldg(p.positions + t) : static_cast<int>(at);
        an.set(p.inv_freq + 8 * u, pos, p.scale, 1.f);
    }
    for (;;) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int h = h0 + j;
            if (h >= h_end) break;
            uint16_t *dst;
            bool rot = turn;
            if (h < p.H) {
                dst = static_cast<uint16_t *>(p.q_out) + h * p.qo_h + t * p.qo_n;
            } else if (page < 0) {
                continue;
            } else if (h < p.H + p.kv.Hkv) {
                dst = static_cast<uint16_t *>(p.kv.k) + page * p.kv.k_page + (h - p.H) * p.kv.k_head + row * p.kv.k_tok;
            } else {
                dst = static_cast<uint16_t *>(p.kv.v) + page * p.kv.v_page + (h - p.H - p.kv.Hkv) * p.kv.v_head +
                      row * p.kv.v_tok;
                rot = false;
            }
            if (rot) rotate<BF16, INTER>(x[j], y[j], an);
            *reinterpret_cast<uint4 *>(dst + o0) = x[j];
            *reinterpret_cast<uint4 *>(dst + o1) = y[j];
        }
        h0 += 4;
        if (h0 >= h_end) break;
        load();
    }
}

// Heads per thread: as many as leaves about two thousand threads per SM, in
// fours (the kernels' unroll).
int heads_per_group(long long threads, int heads, int sms) {
    const long long want = 2048LL * sms;
    long long groups = std::max<long long>(1, std::min<long long>((want + threads - 1) / threads, (heads + 3) / 4));
    const int per = static_cast<int>((heads + groups - 1) / groups);
    return (per + 3) / 4 * 4;
}

}  // namespace

cudaError_t launch_rope(const RopeParams &p, bool bf16, int sms, cudaStream_t stream) {
    const long long threads = static_cast<long long>(p.B) * p.N * ((p.D + 15) / 16);
    const int heads = p.q.H + p.k.H;
    const int per = heads_per_group(threads, heads, sms);
    const dim3 grid(static_cast<unsigned>((threads + kRopeThreads - 1) / kRopeThreads), (heads + per - 1) / per);
    auto kern = bf16 ? (p.interleaved ? fa_rope_kernel<true, true> : fa_rope_kernel<true, false>)
                     : (p.interleaved ? fa_rope_kernel<false, true> : fa_rope_kernel<false, false>);
    prof_begin(stream, "fa_rope_kernel");
    kern<<<grid, kRopeThreads, 0, stream>>>(p, per);
    prof_end(stream);
    note_launch();
    return cudaGetLastError();
}

cudaError_t launch_paged_append(const AppendParams &p, bool bf16, int sms, cudaStream_t stream) {
    const int units = p.kv.D / 16, per_block = kRopeThreads / units;
    const int heads = p.H + 2 * p.kv.Hkv;
    const int per = heads_per_group(static_cast<long long>(p.T) * units, heads, sms);
    const dim3 grid((p.T + per_block - 1) / per_block, (heads + per - 1) / per);
    auto kern = bf16 ? (p.interleaved ? fa_paged_append_kernel<true, true> : fa_paged_append_kernel<true, false>)
                     : (p.interleaved ? fa_paged_append_kernel<false, true> : fa_paged_append_kernel<false, false>);
    prof_begin(stream, "fa_paged_append_kernel");
    kern<<<grid, kRopeThreads, 0, stream>>>(p, per);
    prof_end(stream);
    note_launch();
    return cudaGetLastError();
}

}  // namespace fa
