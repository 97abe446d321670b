// fa_paged_tokens.cu -- attention of a few new tokens per sequence over a paged
// cache: decoding and drafted tokens, at most 64 query rows (tokens x heads of a
// group) per sequence and kv head.  The formulas are those of fa_paged.cu.
//
// Bound by memory: a key and its value are read once, for 4 D operations a row.
// What has to be kept short is the chain from a tile's arrival to its release,
// so that a ring of a few tiles per SM covers the memory's latency.  So the
// products are turned over:
//     S^T = K Q^T   (128 keys x R rows),   O^T += V^T P^T   (D x R),
// with R = 16, 32 or 64: a product costs what its R columns cost instead of 128
// rows, a softmax thread owns one key (a lane of tensor memory) and has only the
// rows that exist to exponentiate, and V is the operand that it is in memory
// (keys outermost).  P^T goes through shared memory as the second operand.
//
// The running maximum is common to the 128 threads but needs no reduction per
// tile: a reference maximum per row is moved only when some score exceeds it by
// more than 2^8, which one vote over the warpgroup finds out; the row sums stay
// spread over the threads until the unit's end.
//
// Measured (D = 128, G = 4): 64 tokens over 512..8192 keys in pages of 16, 1143
// MB, 181..184 us, 6.2..6.3 TB/s; one token over 65536 keys, 8 heads, 54.9 us (41
// at the copy rate); one over 1000 keys 7 us and 2.5 of merging.  With row tiles of 128
// for those rows (fa_paged.cu) the first took 255 us: the softmax of one tile
// held its V for longer than the ring covers.
//
// Warps: one warpgroup of softmax (two for R = 64, half of the rows each), then a
// TMA warp (each lane looks up the page of its box), an MMA warp, and one that
// walks the CTA's share of the work (fa_paged_sched.cuh).
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "fa_internal.h"
#include "fa_paged_internal.h"
#include "fa_paged_sched.cuh"
#include "fa_paged_ptx.cuh"

namespace fa {
namespace {

constexpr int kBN = kPagedTile;     // keys per tile
constexpr int kDescs = 8;           // segment descriptors in the ring
constexpr float kTau = 8.0f;        // a row's reference maximum moves past this (log2 units)
// Reference maximum of a row that has seen no key: every finite score lies above
// it (with -inf the subtraction of a masked score would give NaN).
constexpr float kNone = -3.402823466e38f;
constexpr float kLn2 = 0.69314718055994530942f;

// What the threads share of a row, beside its reference maximum: the factor that
// its O takes next, and where its O goes.
struct alignas(16) RowState {
    float factor;
    int pad;
    long long at;
};

template <int D, int R>
struct TokenLayout {
    static constexpr int kGroups = R == 64 ? 2 : 1;       // softmax warpgroups
    static constexpr int kCols = R / kGroups;             // rows of each
    static constexpr int kProducerWarp = 4 * kGroups;
    static constexpr int kMmaWarp = kProducerWarp + 1;
    static constexpr int kPlanWarp = kProducerWarp + 2;
    static constexpr int kThreads = 32 * (kProducerWarp + 4);
    static constexpr int kChunks = D / 64;                // 128-byte column blocks per row
    static constexpr int kTileBytes = KeyTile<D>::kBytes;
    static constexpr int kQChunk = R * 128;
    static constexpr int kQBytes = kChunks * kQChunk;
    static constexpr int kPBytes = 2 * R * 128;           // R rows of 128 keys, two column blocks
    // Tiles in flight, as many as shared memory holds next to Q and P; V's are
    // held longer (until the softmax is through).
    static constexpr int kKStages = D == 64 ? (R == 64 ? 4 : 6) : (R == 16 ? 3 : 2);
    static constexpr int kVStages = D == 64 ? (R == 64 ? 5 : 6) : 3;
    static constexpr int kQBufs = D == 128 && R == 64 ? 1 : 2;
    static constexpr int kK = 0;
    static constexpr int kV = kK + kKStages * kTileBytes;
    static constexpr int kQ = kV + kVStages * kTileBytes;
    static constexpr int kP = kQ + kQBufs * kQBytes;      // ring of two
    static constexpr int kBar = kP + 2 * kPBytes;
    static constexpr int kQFull = 0;                      // +buffer
    static constexpr int kQEmpty = 2;
    static constexpr int kSFull = 4;                      // +buffer
    static constexpr int kPFull = 6;                      // +buffer
    static constexpr int kPvDone = 8;                     // +tile & 1
    static constexpr int kDrain = 10;
    static constexpr int kDFull = 11;                     // +descriptor
    static constexpr int kDEmpty = kDFull + kDescs;
    static constexpr int kKFull = kDEmpty + kDescs;       // +stage
    static constexpr int kKEmpty = kKFull + kKStages;
    static constexpr int kVFull = kKEmpty + kKStages;
    static constexpr int kVEmpty = kVFull + kVStages;
    static constexpr int kNumBars = kVEmpty + kVStages;
    static constexpr int kMisc = kBar + kNumBars * 8;     // tensor-memory base, abort flag
    static constexpr int kDesc = (kMisc + 8 + 15) / 16 * 16;
    static constexpr int kRed = kDesc + kDescs * static_cast<int>(sizeof(Seg));     // float [warp][kCols]
    static constexpr int kRow = kRed + 4 * R * 4;         // RowState [R]
    static constexpr int kMax = kRow + R * 16;            // float [R]: reference maxima
    static constexpr int kBytes = kMax + R * 4;
    static constexpr int kAlloc = kBytes + 1024;          // room to align the base
    static constexpr uint32_t kTmemCols = 4 * R;          // S twice, O
    static constexpr uint32_t kColS = 0, kColO = 2 * R;
    static_assert(kAlloc <= 231424, "shared memory");
};

template <int C>
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, uint32_t (&r)[C]) {
    if constexpr (C == 16) tmem_ld32dp_x16_wait(taddr, r);
    else tmem_ld32dp_x32_wait(taddr, r);
}

// The warp's maxima (or sums) of N = 16 or 32 values per lane, N - 1 (+ 1)
// shuffles: at every step a lane gives half of its values to the lane across and
// reduces the other half with what it gets.  Value r ends in lane r * (32 / N).
template <int N, bool MAX>
__device__ __forceinline__ float warp_reduce_rows(const float *x, int lane) {
    float v[N];
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = x[i];
#pragma unroll
    for (int o = 16, n = N / 2; o > 0; o >>= 1, n >>= 1) {
        const bool up = lane & o;
        if (n > 0) {
#pragma unroll
            for (int i = 0; i < N / 2; ++i) {
                if (i >= n) break;
                const float give = up ? v[i] : v[i + n], keep = up ? v[i + n] : v[i];
                const float got = __shfl_xor_sync(0xffffffffu, give, o);
                v[i] = MAX ? fmaxf(keep, got) : keep + got;
            }
        } else {
            const float got = __shfl_xor_sync(0xffffffffu, v[0], o);
            v[0] = MAX ? fmaxf(v[0], got) : v[0] + got;
        }
    }
    return v[0];
}

// Per warp and row, into red[row].
template <int C, bool MAX>
__device__ __forceinline__ void reduce_rows(const float (&x)[C], float *red, int lane) {
    const float v = warp_reduce_rows<C, MAX>(x, lane);
    if constexpr (C == 16) {
        if ((lane & 1) == 0) red[lane >> 1] = v;
    } else {
        red[lane] = v;
    }
}

template <bool BF16>
__device__ __forceinline__ uint16_t round16(float x) {
    if constexpr (BF16) return __bfloat16_as_ushort(__float2bfloat16_rn(x));
    else return __half_as_ushort(__float2half_rn(x));
}

template <int D, int R, bool BF16>
__global__ void __launch_bounds__(TokenLayout<D, R>::kThreads, 1)
fa_paged_tokens_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ PagedFwdParams p) {
    using L = TokenLayout<D, R>;
    using KT = KeyTile<D>;
    constexpr int kProducerWarp = L::kProducerWarp, kMmaWarp = L::kMmaWarp, kPlanWarp = L::kPlanWarp;
    constexpr int kThreads = L::kThreads;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const uint32_t sbase = smem_u32(smem);
    auto bar = [&](int i) -> uint32_t { return sbase + L::kBar + 8 * i; };
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L::kMisc);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::kMisc + 4);
    Seg *descs = reinterpret_cast<Seg *>(smem + L::kDesc);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;

    if (warp == kMmaWarp) {
        tmem_alloc(smem_u32(tmem_slot), L::kTmemCols);
        tmem_relinquish();
    }
    if (threadIdx.x == 0) {
        *abort_flag = 0;
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(L::kQFull + i), 1);
            mbar_init(bar(L::kQEmpty + i), 1);
            mbar_init(bar(L::kSFull + i), 1);
            mbar_init(bar(L::kPFull + i), 128 * L::kGroups);
            mbar_init(bar(L::kPvDone + i), 1);
        }
        mbar_init(bar(L::kDrain), 1);
        for (int i = 0; i < kDescs; ++i) {
            mbar_init(bar(L::kDFull + i), 1);
            mbar_init(bar(L::kDEmpty + i), 2 + 4 * L::kGroups);      // producer, MMA, softmax warps
        }
        for (int s = 0; s < L::kKStages; ++s) {
            mbar_init(bar(L::kKFull + s), 1);
            mbar_init(bar(L::kKEmpty + s), 1);
        }
        for (int s = 0; s < L::kVStages; ++s) {
            mbar_init(bar(L::kVFull + s), 1);
            mbar_init(bar(L::kVEmpty + s), 1);
        }
        fence_mbar_init();
    }
    // rows that no box fills hold zeros, not what shared memory held before
    for (int i = threadIdx.x; i < L::kQBufs * L::kQBytes / 16; i += kThreads)
        reinterpret_cast<uint4 *>(smem + L::kQ)[i] = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
    if (warp == kProducerWarp && lane == 0) {
        prefetch_tmap(&tm_q);
        prefetch_tmap(&tm_k);
        prefetch_tmap(&tm_v);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // Nothing above touches what the stream's earlier grids write or read; this
    // grid may have been started while the last of them still ran.
    grid_dependency_wait();
    const uint32_t tmem = *tmem_slot;
    const WaitCtx wctx{p.timeout_ns, p.err, abort_flag};
    auto desc_wait = [&](int u) -> bool {
        return mbar_wait_warp(bar(L::kDFull + u % kDescs), (u / kDescs) & 1, wctx);
    };
    auto desc_release = [&](int u) {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(L::kDEmpty + u % kDescs));
    };
    if (warp == kPlanWarp) {
        // ===================== the CTA's share of the work =====================
        MergeMeta mm{0, 0, 0, -1};
        {
            PlanSeqs seqs;
            plan_load(p, 0, lane, seqs);
            const Piece pc = plan_piece(p, p.geom, p.min_piece, lane, seqs);
            bool ok = true;
            int u = 0;
            auto push = [&](const Seg &s) -> bool {
                const int i = u % kDescs;
                if (u >= kDescs && !mbar_wait_warp(bar(L::kDEmpty + i), ((u / kDescs) - 1) & 1, wctx)) return false;
                if (lane == 0) {
                    descs[i] = s;
                    mbar_arrive(bar(L::kDFull + i));
                }
                ++u;
                return true;
            };
            if (pc.b >= 0) {
                SegWalk w;
                w.first(p, p.geom, pc, lane);
                do {
                    const Seg s = make_seg(w, p.geom);
                    if (w.n == 0) {
                        write_empty<D>(p, s.row0, s.ntok, s.h, lane);
                    } else if (!w.none()) {
                        if (w.t0 == 0 && w.t1 < w.n) mm = MergeMeta{s.row0, s.ntok, s.h, w.last_cta(pc, p.geom)};
                        ok = push(s);
                    }
                } while (ok && w.next(p, p.geom));
            }
            if (ok) push(Seg{});
        }
        if (lane == 0) p.meta[blockIdx.x] = mm;
        grid_launch_dependents();       // the merge may be set up; it waits for this grid
        named_bar_sync(1, kThreads);
    } else if (warp == kProducerWarp) {
        // ===================== TMA producer =====================
        PageBoxes pages;
        pages.init(p, lane);
        const uint32_t q_bytes = static_cast<uint32_t>(L::kChunks * 128 * p.G * p.geom.unit_tokens);
        int t = 0;                      // key tiles begun so far (ring position)
        int k_n = 0, v_n = 0, q_n = 0;  // copies issued
        bool ok = true;
        for (int u = 0; ok; ++u) {
            if (!desc_wait(u)) { ok = false; break; }
            const Seg s = descs[u % kDescs];
            desc_release(u);
            if (s.nt == 0) break;
            pages.segment(p, s);
            pages.look_up(p, s.t0, s.len_k);
            {
                const int bf = q_n % L::kQBufs;
                if (!mbar_wait_warp(bar(L::kQEmpty + bf), ((q_n / L::kQBufs) & 1) ^ 1, wctx)) { ok = false; break; }
                if (lane == 0) {
                    mbar_arrive_expect_tx(bar(L::kQFull + bf), q_bytes);
#pragma unroll
                    for (int c = 0; c < L::kChunks; ++c)
                        tma_load_3d(sbase + L::kQ + bf * L::kQBytes + c * L::kQChunk, &tm_q, bar(L::kQFull + bf), c * 64,
                                    s.h * p.G, s.row0);
                }
                ++q_n;
            }
            for (int j = 0; j < s.nt; ++j, ++t) {
                const int ks = t % L::kKStages, vs = t % L::kVStages;
                const PageBoxes::Box kb = pages.box(p, p.k_ratio), vb = pages.box(p, p.v_ratio);
                if (!mbar_wait_warp(bar(L::kKEmpty + ks), ((t / L::kKStages) & 1) ^ 1, wctx)) { ok = false; break; }
                if (lane == 0) mbar_arrive_expect_tx(bar(L::kKFull + ks), L::kTileBytes);
                __syncwarp();
                pages.copy(p, &tm_k, sbase + L::kK + ks * L::kTileBytes, KT::kGroupBytes, bar(L::kKFull + ks), kb);
                ++k_n;
                if (j + 1 < s.nt) pages.look_up(p, s.t0 + j + 1, s.len_k);
                if (!mbar_wait_warp(bar(L::kVEmpty + vs), ((t / L::kVStages) & 1) ^ 1, wctx)) { ok = false; break; }
                if (lane == 0) mbar_arrive_expect_tx(bar(L::kVFull + vs), L::kTileBytes);
                __syncwarp();
                pages.copy(p, &tm_v, sbase + L::kV + vs * L::kTileBytes, KT::kGroupBytes, bar(L::kVFull + vs), vb);
                ++v_n;
            }
        }
        if (!ok) {
            // bounded chance for the copies in flight to land before the CTA's
            // shared memory goes away
            volatile int zero = 0;
            const WaitCtx drain{wctx.timeout_ns, wctx.err, &zero};
            for (int i = max(0, q_n - L::kQBufs); i < q_n; ++i)
                mbar_wait(bar(L::kQFull + i % L::kQBufs), (i / L::kQBufs) & 1, drain);
            for (int i = max(0, k_n - L::kKStages); i < k_n; ++i)
                mbar_wait(bar(L::kKFull + i % L::kKStages), (i / L::kKStages) & 1, drain);
            for (int i = max(0, v_n - L::kVStages); i < v_n; ++i)
                mbar_wait(bar(L::kVFull + i % L::kVStages), (i / L::kVStages) & 1, drain);
        }
        __syncwarp();
        named_bar_sync(1, kThreads);
    } else if (warp == kMmaWarp) {
        // ============ MMA issuer (whole warp; one elected lane issues) ============
        constexpr uint32_t idesc_s = idesc_f16_f32acc(BF16, 128, R, false, false);
        constexpr uint32_t idesc_o = idesc_f16_f32acc(BF16, 128, R, true, false);
        bool ok = true, any = false;
        int su = 0, sj = 0, sn = 0, st_n = 0;   // the next S: segment, tile of it, its tiles, tiles so far
        int pu = 0, pt = 0;                     // the next P V: segment, tiles so far
        // S^T of the next key tile, whatever segment it is in
        auto step_s = [&]() -> bool {
            if (sj == sn) {
                if (su > 0 && sn == 0) return true;             // the end was seen
                if (!desc_wait(su)) return false;
                sn = descs[su % kDescs].nt;
                sj = 0;
                ++su;
                if (sn == 0) return true;
                if (!mbar_wait_warp(bar(L::kQFull + (su - 1) % L::kQBufs), ((su - 1) / L::kQBufs) & 1, wctx)) return false;
            }
            const int st = st_n % L::kKStages, bf = (su - 1) % L::kQBufs;
            if (!mbar_wait_warp(bar(L::kKFull + st), (st_n / L::kKStages) & 1, wctx)) return false;
            tc_fence_after();
            const uint64_t dk = KT::k_desc(sbase + L::kK + st * L::kTileBytes);
            const uint64_t dq = smem_desc_sw128(sbase + L::kQ + bf * L::kQBytes, 16, 1024);
            const uint32_t d = tmem + L::kColS + (st_n & 1) * R;
            if (elect_one()) {
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
                    umma_f16_ss(d, dk + KT::k_step(kk),
                                dq + (((kk >> 2) * L::kQChunk + (kk & 3) * 32) >> 4), idesc_s, kk > 0);
                umma_commit(bar(L::kSFull + (st_n & 1)));
                umma_commit(bar(L::kKEmpty + st));
                if (sj + 1 == sn) umma_commit(bar(L::kQEmpty + bf));
            }
            __syncwarp();
            any = true;
            ++st_n;
            ++sj;
            return true;
        };
        ok = step_s() && step_s();
        while (ok) {
            if (!desc_wait(pu)) { ok = false; break; }
            const int n = descs[pu % kDescs].nt, tail = descs[pu % kDescs].tail;
            if (n == 0) break;
            for (int j = 0; j < n; ++j, ++pt) {
                const int st = pt % L::kVStages;
                if (!mbar_wait_warp(bar(L::kVFull + st), (pt / L::kVStages) & 1, wctx)) { ok = false; break; }
                if (j + 1 == n && tail < kBN) {
                    // the sequence ends inside this key tile: P is 0 past it, but
                    // the cache may hold anything there (NaN), so V is made 0 too
                    KT::clear(smem + L::kV + st * L::kTileBytes, tail, lane);
                    fence_proxy_async_smem();
                    __syncwarp();
                }
                if (!mbar_wait_warp(bar(L::kPFull + (pt & 1)), (pt >> 1) & 1, wctx)) { ok = false; break; }
                tc_fence_after();
                // the rows of V^T are V's columns, 64 to a block; D = 64 has one
                // block, read twice (the lanes past D are not used)
                const uint64_t dv = KT::v_desc(sbase + L::kV + st * L::kTileBytes, D == 128);
                const uint64_t dp = smem_desc_sw128(sbase + L::kP + (pt & 1) * L::kPBytes, 16, 1024);
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < kBN / 16; ++kk)
                        umma_f16_ss(tmem + L::kColO, dv + KT::v_step(kk),
                                    dp + (((kk >> 2) * L::kQChunk + (kk & 3) * 32) >> 4), idesc_o, j > 0 || kk > 0);
                    umma_commit(bar(L::kPvDone + (pt & 1)));
                    umma_commit(bar(L::kVEmpty + st));
                }
                __syncwarp();
                if (!step_s()) { ok = false; break; }
            }
            if (!ok) break;
            desc_release(pu);
            ++pu;
        }
        if (any) {
            // every issued MMA must finish before tensor memory is released
            if (elect_one()) umma_commit(bar(L::kDrain));
            __syncwarp();
            volatile int zero = 0;
            const WaitCtx drain{wctx.timeout_ns, wctx.err, &zero};
            mbar_wait(bar(L::kDrain), 0, drain);
        }
        __syncwarp();
        named_bar_sync(1, kThreads);
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, L::kTmemCols);
    } else if (warp < kProducerWarp) {
        // ===================== softmax =====================
        constexpr int C = L::kCols;
        const int wg = warp >> 2, wq = warp & 3;    // warpgroup, lane quarter of tensor memory
        const uint32_t wg_bar = 2 + wg;
        const int key = wq * 32 + lane;             // within the tile
        const int row0 = wg * C;                    // first row of the warpgroup's
        const uint32_t tl = tmem + (static_cast<uint32_t>(wq * 32) << 16) + row0;
        float *const red = reinterpret_cast<float *>(smem + L::kRed) + wg * 4 * C;
        RowState *const row_state = reinterpret_cast<RowState *>(smem + L::kRow) + row0;
        float *const m_ref = reinterpret_cast<float *>(smem + L::kMax) + row0;      // log2 units
        const float qk = p.qk_scale_log2;
        // this key's place in row r of P: column block, then 16-byte units swizzled by the row
        uint8_t *const p_key = smem + L::kP + (key >> 6) * L::kQChunk + row0 * 128 + (key & 7) * 2;
        const int p_unit = (key & 63) >> 3;
        // P V of key tile t and all before it.  Its barrier serves every other tile:
        // a wait can tell a phase only from the one before, and S(t), seen before any
        // such wait, covers the products up to t - 2.
        auto wait_pv = [&](int t) { return mbar_wait_warp(bar(L::kPvDone + (t & 1)), (t >> 1) & 1, wctx); };
        int t = 0;                                  // key tiles so far
        bool ok = true;
        for (int u = 0; ok; ++u) {
            if (!desc_wait(u)) ok = false;
            if (key < C) m_ref[key] = kNone;        // row r's state is thread r's to write, everyone's to read
            // one outcome for the four warps: they meet at barriers below
            if (named_bar_or(wg_bar, 128, !ok)) { ok = false; break; }
            const Seg &s = descs[u % kDescs];
            if (s.nt == 0) break;
            const int nt = s.nt, len_k = s.len_k;
            const int edge = p.causal ? min(s.lim0, len_k - 1) : len_k - 1;   // keys up to it are seen by all rows
            // Rows past the segment's compute like the others, from what Q's buffer
            // holds, and are not stored; a product's columns do not mix.
            float l[C];                             // this thread's keys only
#pragma unroll
            for (int r = 0; r < C; ++r) l[r] = 0.f;
            for (int j = 0; j < nt; ++j, ++t) {
                const int kv = (s.t0 + j) * kBN + key;
                const bool got = mbar_wait_warp(bar(L::kSFull + (t & 1)), (t >> 1) & 1, wctx);
                tc_fence_after();
                float x[C];                         // scores, not scaled
                {
                    uint32_t sr[C];
                    tmem_ld_cols<C>(tl + L::kColS + (t & 1) * R, sr);
#pragma unroll
                    for (int r = 0; r < C; ++r) x[r] = __uint_as_float(sr[r]);
                }
                if (kv - key + kBN - 1 > edge) {
                    // row r is the head r % G of token r / G, which sees one key
                    // more than the token before
                    int tok = row0 / p.G, g = row0 - tok * p.G;
                    int lim = p.causal ? min(s.lim0 + tok, len_k - 1) : edge;
#pragma unroll
                    for (int r = 0; r < C; ++r) {
                        if (kv > lim) x[r] = neg_inf();
                        if (++g == p.G) {
                            g = 0;
                            ++tok;
                            lim = p.causal ? min(s.lim0 + tok, len_k - 1) : lim;
                        }
                    }
                }
                // a = log2 of the probability, before l: x * qk - m_ref
                float a[C];
                auto subtract = [&]() {
#pragma unroll
                    for (int r = 0; r < C; r += 4) {
                        const float4 m = *reinterpret_cast<const float4 *>(m_ref + r);
                        a[r] = fmaf(x[r], qk, -m.x);
                        a[r + 1] = fmaf(x[r + 1], qk, -m.y);
                        a[r + 2] = fmaf(x[r + 2], qk, -m.z);
                        a[r + 3] = fmaf(x[r + 3], qk, -m.w);
                    }
                };
                subtract();
                float top = fmaxf(a[0], a[1]), top2 = fmaxf(a[2], a[3]);
#pragma unroll
                for (int r = 4; r < C; r += 4) {
                    top = fmax3(top, a[r], a[r + 1]);
                    top2 = fmax3(top2, a[r + 2], a[r + 3]);
                }
                if (named_bar_or(wg_bar, 128, !got || fmaxf(top, top2) > kTau)) {
                    if (named_bar_or(wg_bar, 128, !got)) { ok = false; break; }
                    reduce_rows<C, true>(x, red + wq * C, lane);
                    named_bar_sync(wg_bar, 128);
                    if (key < C) {
                        const float v =
                            qk * fmaxf(fmaxf(red[key], red[C + key]), fmaxf(red[2 * C + key], red[3 * C + key]));
                        const float m = m_ref[key];
                        const bool move = v > m + kTau;
                        m_ref[key] = move ? v : m;
                        row_state[key].factor = move ? ex2_approx(m - v) : 1.f;     // kNone: 0
                    }
                    named_bar_sync(wg_bar, 128);
#pragma unroll
                    for (int r = 0; r < C; ++r) l[r] *= row_state[r].factor;
                    if (j > 0) {
                        // O's columns too, when the products so far are in it
                        const bool done = wait_pv(t - 1);
                        if (named_bar_or(wg_bar, 128, !done)) { ok = false; break; }
                        tc_fence_after();
#pragma unroll 1
                        for (int c = 0; c < C; c += 16) {
                            uint32_t orr[16];
                            tmem_ld32dp_x16_wait(tl + L::kColO + c, orr);
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                orr[e] = __float_as_uint(__uint_as_float(orr[e]) * row_state[c + e].factor);
                            tmem_st32dp_x16(tl + L::kColO + c, orr);
                        }
                        tmem_wait_st();
                    }
                    subtract();
                }
                // P = 2^a, rounded to the operands' type (the tensor cores take A and B of
                // one type, and V comes as it is); the sums take it unrounded.  Masked
                // keys give 0.
                uint8_t *const pt = p_key + (t & 1) * L::kPBytes;
#pragma unroll
                for (int r = 0; r < C; r += 2) {
                    const float e0 = ex2_approx(a[r]), e1 = ex2_approx(a[r + 1]);
                    l[r] += e0;
                    l[r + 1] += e1;
                    const uint32_t e = pack2<BF16>(e0, e1);
                    *reinterpret_cast<uint16_t *>(pt + r * 128 + ((p_unit ^ (r & 7)) << 4)) = static_cast<uint16_t>(e);
                    *reinterpret_cast<uint16_t *>(pt + (r + 1) * 128 + ((p_unit ^ ((r + 1) & 7)) << 4)) =
                        static_cast<uint16_t>(e >> 16);
                }
                fence_proxy_async_smem();
                tc_fence_before();
                mbar_arrive(bar(L::kPFull + (t & 1)));
            }
            if (!ok) break;

            // ---- the rows' results
            reduce_rows<C, false>(l, red + wq * C, lane);
            const int rows = min(C, s.ntok * p.G - row0);       // this warpgroup's (none: <= 0)
            const bool done = wait_pv(t - 1);
            if (named_bar_or(wg_bar, 128, !done)) { ok = false; break; }
            if (key < rows) {
                const float sum = (red[key] + red[C + key]) + (red[2 * C + key] + red[3 * C + key]);
                const float lse2 = sum == 0.f ? neg_inf() : m_ref[key] + lg2_approx(sum);
                const int r = row0 + key, tok = r / p.G, head = s.h * p.G + r - tok * p.G;
                const size_t part = (2 * blockIdx.x + s.dest) * static_cast<size_t>(p.part_rows) + r;
                row_state[key].factor = sum == 0.f ? 0.f : 1.f / sum;
                row_state[key].at = s.dest < 0 ? head * p.o_h + (s.row0 + tok) * p.o_n : static_cast<long long>(part) * D;
                if (s.dest < 0)
                    p.lse[static_cast<long long>(head) * p.T + s.row0 + tok] = lse2 * kLn2;
                else
                    p.lse_part[part] = lse2;
            }
            named_bar_sync(wg_bar, 128);
            tc_fence_after();
            auto store_rows = [&](auto *out) {
#pragma unroll 1
                for (int c = 0; c < rows; c += 8) {
                    uint32_t orr[8];
                    tmem_ld32dp_x8_wait(tl + L::kColO + c, orr);
                    RowState rs[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) rs[e] = row_state[c + e];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float y = __uint_as_float(orr[e]) * rs[e].factor;
                        if (key < D && c + e < rows) {
                            if constexpr (sizeof(*out) == 2) out[rs[e].at + key] = round16<BF16>(y);
                            else out[rs[e].at + key] = y;
                        }
                    }
                    __syncwarp();
                }
            };
            if (s.dest < 0)
                store_rows(static_cast<uint16_t *>(p.o));
            else
                store_rows(p.o_part);
            tc_fence_before();
            named_bar_sync(wg_bar, 128);     // the rows' state is read, the next segment may replace it
            desc_release(u);
        }
        __syncwarp();
        named_bar_sync(1, kThreads);
    } else {
        named_bar_sync(1, kThreads);    // the last warp
    }
}

template <int D, int R, bool BF16>
cudaError_t launch_t(const PagedTensorMaps &tm, const PagedFwdParams &p, int grid, cudaStream_t stream) {
    auto kern = fa_paged_tokens_kernel<D, R, BF16>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, TokenLayout<D, R>::kAlloc);
    if (e != cudaSuccess) return e;
    prof_begin(stream, "fa_paged_tokens_kernel");
    e = launch_early(kern, dim3(grid), TokenLayout<D, R>::kThreads, TokenLayout<D, R>::kAlloc, stream, tm.q, tm.k, tm.v,
                     p);
    prof_end(stream);
    note_launch();
    if (e != cudaSuccess) return e;
    return launch_paged_merge(p, BF16, grid, stream);
}

template <int D, bool BF16>
cudaError_t launch_d(const PagedTensorMaps &tm, const PagedFwdParams &p, int grid, cudaStream_t stream) {
    if (p.part_rows <= 16) return launch_t<D, 16, BF16>(tm, p, grid, stream);
    if (p.part_rows <= 32) return launch_t<D, 32, BF16>(tm, p, grid, stream);
    return launch_t<D, 64, BF16>(tm, p, grid, stream);
}

}  // namespace

cudaError_t launch_paged_tokens(const PagedTensorMaps &tm, const PagedFwdParams &p, bool bf16, int sms,
                                cudaStream_t stream) {
    const int grid = sms < kPagedMaxCtas ? sms : kPagedMaxCtas;
    if (p.kv.D == 64) return bf16 ? launch_d<64, true>(tm, p, grid, stream) : launch_d<64, false>(tm, p, grid, stream);
    return bf16 ? launch_d<128, true>(tm, p, grid, stream) : launch_d<128, false>(tm, p, grid, stream);
}

}  // namespace fa
