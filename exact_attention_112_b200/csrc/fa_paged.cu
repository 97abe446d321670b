// fa_paged.cu -- attention of a ragged batch of new tokens over a paged cache.
//
//     o_i = sum_j exp(s_ij - m_i) v_j / l_i,   s_ij = scale * q_i . k_j,
//     l_i = sum_j exp(s_ij - m_i),             lse_i = m_i + ln l_i
// over the keys j < len of row i's sequence, with causal also
// j <= i + len - new; head h reads kv head h / G.
//
// One pass over the keys with the running maximum and sum, on the tensor cores:
// S = Q K^T and O += P V are tcgen05 products of 128 x 128 tiles with their
// accumulators in tensor memory, K and V stream in by TMA, box by box as the
// page table says.
//
// Rows.  The query heads of a group read the same keys, so a tile of 128 query
// rows holds floor(128 / G) tokens times the G heads of one kv head (row =
// token * G + head): a single token still shares its keys among its heads.  A
// unit of work is up to two such tiles; how the units are shared out over the
// CTAs is in fa_paged_sched.cuh.
//
// Jobs.  A job is one S product, its softmax and its P V product.  A unit of two
// row tiles makes two jobs of each key tile; a unit of one row tile, one.  Jobs
// alternate between two slots (S and O columns of tensor memory and a softmax
// warpgroup each), so a unit of one row tile sends its even and odd key tiles
// through different slots and adds the two results at its end: single tokens
// keep both warpgroups and the tensor pipe busy too.  The tensor pipe runs
// PV(q), S(q + 2) for job after job, across units.
//
// Bound by the chain softmax -> P V -> next S of a slot and the hand-overs to
// the MMA warp: some 1800 cycles a job for 1024 of tensor work.  2 x 2048 tokens
// over 12001..16384 keys (940 GFLOP, H = 32, Hkv = 8, D = 128): 719..736 us alone
// (1280..1310 TFLOP/s), 902..926 in a long run under the power cap.  The chain is
// no shorter at D = 64, where the products are half: the same tokens 660..670 us
// (470 GFLOP, 288 us at the tensor cores' rate).  A segment of one row tile takes
// 1.34..1.57 us a key tile, at the memory's rate when all CTAs have such.
//
// Warps: 0-3 and 4-7 softmax of slot 0 and 1 (a thread per row), 8 TMA (its
// lanes look up a box's page each), 9 MMA, 10 walks the CTA's share of the work
// and hands descriptors of its segments to the others through a ring.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "fa_internal.h"
#include "fa_paged_internal.h"
#include "fa_paged_sched.cuh"
#include "fa_paged_ptx.cuh"

namespace fa {
namespace {

constexpr int kBM = 128;            // query rows per tile
constexpr int kBN = kPagedTile;     // keys per tile
constexpr int kThreads = 384;       // three warpgroups
constexpr int kProducerWarp = 8;
constexpr int kMmaWarp = 9;
constexpr int kPlanWarp = 10;
// Register split (launch pool 168 x 384 = 64512 = 256 * 192 + 128 * 120).
constexpr uint32_t kRegsSoftmax = 192;
constexpr uint32_t kRegsOther = 120;
constexpr int kDescs = 8;           // segment descriptors in the ring
constexpr float kTau = 8.0f;        // lazy-rescale threshold (log2 units)
constexpr float kLn2 = 0.69314718055994530942f;

template <int D>
struct PagedLayout {
    static constexpr int kStages = D == 64 ? 4 : 2;       // K and V tiles in flight each
    static constexpr int kChunks = D / 64;                // 128-byte column blocks per row
    static constexpr int kChunkBytes = kBN * 128;
    static constexpr int kTileBytes = kChunks * kChunkBytes;
    static constexpr int kQ = 0;                          // ring of two row tiles
    static constexpr int kK = kQ + 2 * kTileBytes;
    static constexpr int kV = kK + kStages * kTileBytes;
    static constexpr int kBar = kV + kStages * kTileBytes;
    static constexpr int kQFull = 0;                      // +buffer
    static constexpr int kQEmpty = 2;
    static constexpr int kSFull = 4;                      // +slot
    static constexpr int kPHalf = 6;                      // +2 * slot + half
    static constexpr int kOFull = 10;                     // +slot
    static constexpr int kStat = 12;                      // statistics of both slots written
    static constexpr int kRead = 13;                      // O of both slots read
    static constexpr int kDrain = 14;
    static constexpr int kDFull = 15;                     // +descriptor
    static constexpr int kDEmpty = kDFull + kDescs;
    static constexpr int kKFull = kDEmpty + kDescs;       // +stage
    static constexpr int kKEmpty = kKFull + kStages;
    static constexpr int kVFull = kKEmpty + kStages;
    static constexpr int kVEmpty = kVFull + kStages;
    static constexpr int kNumBars = kVEmpty + kStages;
    static constexpr int kMisc = kBar + kNumBars * 8;     // tensor-memory base, abort flag
    static constexpr int kDesc = (kMisc + 8 + 15) / 16 * 16;
    static constexpr int kStats = kDesc + kDescs * static_cast<int>(sizeof(Seg));   // float2 [2][128]
    static constexpr int kBytes = kStats + 2 * kBM * 8;
    static constexpr int kAlloc = kBytes + 1024;          // room to align the base
    static constexpr uint32_t kTmemCols = 512;
    static constexpr uint32_t kColS = 0, kColO = 256;     // S of slot s at 128 s, O at 256 + D s
    static_assert(kAlloc <= 232448, "shared memory");
    static_assert(sizeof(Seg) % 16 == 0, "descriptors are copied as int4");
};

// Rows of O in 32-byte stores, whole sectors, where their alignment allows it (a
// first prompt of 8192 tokens 526 us with 16-byte stores, 501 with these; 1 prompt
// among 63 single tokens 233 and 228).
__device__ __forceinline__ void st_global_v8(void *p, const uint32_t *a) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(a[0]), "r"(a[1]),
                 "r"(a[2]), "r"(a[3]), "r"(a[4]), "r"(a[5]), "r"(a[6]), "r"(a[7])
                 : "memory");
}

template <int D, bool BF16>
__global__ void __launch_bounds__(kThreads, 1)
fa_paged_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ PagedFwdParams p) {
    using L = PagedLayout<D>;
    using KT = KeyTile<D>;
    constexpr int kStages = L::kStages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const uint32_t sbase = smem_u32(smem);
    auto bar = [&](int i) -> uint32_t { return sbase + L::kBar + 8 * i; };
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L::kMisc);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::kMisc + 4);
    Seg *descs = reinterpret_cast<Seg *>(smem + L::kDesc);
    float2 *stats = reinterpret_cast<float2 *>(smem + L::kStats);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;

    // This grid may have been started while the one before it in the stream still
    // ran: nothing is read or written before that has ended.
    grid_dependency_wait();
    PlanSeqs seqs;
    if (warp == kPlanWarp) plan_load(p, 0, lane, seqs);     // the tables arrive during the set-up
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
            mbar_init(bar(L::kPHalf + 2 * i), 4 * 32);
            mbar_init(bar(L::kPHalf + 2 * i + 1), 4 * 32);
            mbar_init(bar(L::kOFull + i), 1);
        }
        mbar_init(bar(L::kStat), 8 * 32);
        mbar_init(bar(L::kRead), 8 * 32);
        mbar_init(bar(L::kDrain), 1);
        for (int i = 0; i < kDescs; ++i) {
            mbar_init(bar(L::kDFull + i), 1);
            mbar_init(bar(L::kDEmpty + i), 10);      // producer, MMA and eight softmax warps
        }
        for (int s = 0; s < kStages; ++s) {
            mbar_init(bar(L::kKFull + s), 1);
            mbar_init(bar(L::kKEmpty + s), 1);
            mbar_init(bar(L::kVFull + s), 1);
            mbar_init(bar(L::kVEmpty + s), 1);
        }
        fence_mbar_init();
    }
    if (warp == kProducerWarp && lane == 0) {
        prefetch_tmap(&tm_q);
        prefetch_tmap(&tm_k);
        prefetch_tmap(&tm_v);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const WaitCtx wctx{p.timeout_ns, p.err, abort_flag};
    // Descriptor u, by a whole warp; each warp arrives on its "empty" barrier
    // when it has taken what it needs.
    auto desc_wait = [&](int u) -> bool {
        return mbar_wait_warp(bar(L::kDFull + u % kDescs), (u / kDescs) & 1, wctx);
    };
    auto desc_release = [&](int u) {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(L::kDEmpty + u % kDescs));
    };
    // Nobody asks for registers again after the split, so it cannot deadlock;
    // every role ends at the CTA barrier 1, and the MMA warp frees tensor memory
    // after it.
    if (warp >= 8) regs_release<kRegsOther>();
    if (warp == kPlanWarp) {
        // ===================== the CTA's share of the work =====================
        MergeMeta mm{0, 0, 0, -1};
        {
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
        const uint32_t q_bytes = static_cast<uint32_t>(L::kChunks * 128 * p.G * p.geom.tile_tokens);
        int t = 0;          // key tiles begun so far (ring position)
        int k_n = 0, v_n = 0, q_n = 0;      // copies issued
        bool ok = true;
        for (int u = 0; ok; ++u) {
            if (!desc_wait(u)) { ok = false; break; }
            const Seg s = descs[u % kDescs];
            desc_release(u);
            if (s.nt == 0) break;
            pages.segment(p, s);
            pages.look_up(p, s.t0, s.len_k);
            for (int i = 0; i <= s.two && ok; ++i, ++q_n) {
                const int bf = q_n & 1;
                if (!mbar_wait_warp(bar(L::kQEmpty + bf), ((q_n >> 1) & 1) ^ 1, wctx)) { ok = false; break; }
                if (lane == 0) {
                    mbar_arrive_expect_tx(bar(L::kQFull + bf), q_bytes);
#pragma unroll
                    for (int c = 0; c < L::kChunks; ++c)
                        tma_load_3d(sbase + L::kQ + bf * L::kTileBytes + c * L::kChunkBytes, &tm_q,
                                    bar(L::kQFull + bf), c * 64, s.h * p.G, s.row0 + i * p.geom.tile_tokens);
                }
            }
            for (int j = 0; j < s.nt && ok; ++j, ++t) {
                const int st = t % kStages;
                const uint32_t ph = (t / kStages) & 1;
                const PageBoxes::Box kb = pages.box(p, p.k_ratio), vb = pages.box(p, p.v_ratio);
                if (!mbar_wait_warp(bar(L::kKEmpty + st), ph ^ 1, wctx)) { ok = false; break; }
                if (lane == 0) mbar_arrive_expect_tx(bar(L::kKFull + st), L::kTileBytes);
                __syncwarp();
                pages.copy(p, &tm_k, sbase + L::kK + st * L::kTileBytes, KT::kGroupBytes, bar(L::kKFull + st), kb);
                ++k_n;
                if (j + 1 < s.nt) pages.look_up(p, s.t0 + j + 1, s.len_k);
                if (!mbar_wait_warp(bar(L::kVEmpty + st), ph ^ 1, wctx)) { ok = false; break; }
                if (lane == 0) mbar_arrive_expect_tx(bar(L::kVFull + st), L::kTileBytes);
                __syncwarp();
                pages.copy(p, &tm_v, sbase + L::kV + st * L::kTileBytes, KT::kGroupBytes, bar(L::kVFull + st), vb);
                ++v_n;
            }
        }
        if (!ok) {
            // bounded chance for the copies in flight to land before the CTA's
            // shared memory goes away
            volatile int zero = 0;
            const WaitCtx drain{wctx.timeout_ns, wctx.err, &zero};
            for (int i = max(0, q_n - 2); i < q_n; ++i) mbar_wait(bar(L::kQFull + (i & 1)), (i >> 1) & 1, drain);
            for (int i = max(0, k_n - kStages); i < k_n; ++i)
                mbar_wait(bar(L::kKFull + i % kStages), (i / kStages) & 1, drain);
            for (int i = max(0, v_n - kStages); i < v_n; ++i)
                mbar_wait(bar(L::kVFull + i % kStages), (i / kStages) & 1, drain);
        }
        __syncwarp();
        named_bar_sync(1, kThreads);
    } else if (warp == kMmaWarp) {
        // ============ MMA issuer (whole warp; one elected lane issues) ============
        constexpr uint32_t idesc_qk = idesc_f16_f32acc(BF16, kBM, kBN, false, false);
        constexpr uint32_t idesc_pv = idesc_f16_f32acc(BF16, kBM, D, false, true);
        struct Cursor {
            int u = 0, j = 0, g = 0, t = 0;     // segment, its next job, jobs and key tiles so far
            int jobs = 0, two = 0, tail = kBN;
        };
        bool ok = true, any = false;
        auto enter = [&](Cursor &c) -> bool {   // the cursor's segment; jobs == 0: the end
            if (!desc_wait(c.u)) return false;
            const Seg &s = descs[c.u % kDescs];
            c.two = s.two;
            c.jobs = s.two ? 2 * s.nt : s.nt;
            c.tail = s.tail;
            c.j = 0;
            return true;
        };
        Cursor cs, cp;
        int q_n = 0;            // row tiles taken so far
        const bool lead = elect_one();      // the lane that issues, commits included
        __syncwarp();
        // S of a job, into the S columns of the slot
        auto issue_s = [&](int slot, int bf, int st, bool k_done, bool q_done) {
            const uint64_t dq = smem_desc_sw128(sbase + L::kQ + bf * L::kTileBytes, 16, 1024);
            const uint64_t dk = KT::k_desc(sbase + L::kK + st * L::kTileBytes);
            const uint32_t d = tmem + L::kColS + slot * 128;
            if (lead) {
#pragma unroll 2
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t off = ((kk >> 2) * L::kChunkBytes + (kk & 3) * 32) >> 4;
                    umma_f16_ss(d, dq + off, dk + KT::k_step(kk), idesc_qk, kk > 0);
                }
                umma_commit(bar(L::kSFull + slot));
                if (k_done) umma_commit(bar(L::kKEmpty + st));
                if (q_done) umma_commit(bar(L::kQEmpty + bf));
            }
            __syncwarp();
        };
        auto wait_k = [&](int t) { return mbar_wait_warp(bar(L::kKFull + t % kStages), (t / kStages) & 1, wctx); };
        // the next job's S, whatever segment it is in
        auto step_s = [&]() -> bool {
            if (cs.jobs == 0) return true;
            const int qi = cs.two ? (cs.j & 1) : 0;
            const int bf = (q_n + qi) & 1;
            const bool tile_done = !cs.two || (cs.j & 1);
            if (cs.j <= cs.two && !mbar_wait_warp(bar(L::kQFull + bf), ((q_n + qi) >> 1) & 1, wctx)) return false;
            if (!wait_k(cs.t)) return false;
            tc_fence_after();
            issue_s(cs.g & 1, bf, cs.t % kStages, tile_done, cs.j + 1 + cs.two >= cs.jobs);
            any = true;
            if (tile_done) ++cs.t;
            ++cs.g;
            if (++cs.j == cs.jobs) {
                q_n += 1 + cs.two;
                ++cs.u;
                return enter(cs);
            }
            return true;
        };
        // P V of a job, half by half as the softmax hands P over
        auto issue_pv = [&](int slot, uint32_t ph, int st, bool acc, bool v_done, bool o_done) -> bool {
            const uint64_t dv = KT::v_desc(sbase + L::kV + st * L::kTileBytes, true);
            const uint32_t pa = tmem + L::kColS + slot * 128;
            const uint32_t d = tmem + L::kColO + slot * D;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (!mbar_wait_warp(bar(L::kPHalf + 2 * slot + h), ph, wctx)) return false;
                tc_fence_after();
                if (lead) {
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        umma_f16_ts(d, pa + (4 * h + kk) * 8, dv + KT::v_step(4 * h + kk), idesc_pv, acc || h + kk > 0);
                    if (h == 1) {
                        if (v_done) umma_commit(bar(L::kVEmpty + st));
                        if (o_done) umma_commit(bar(L::kOFull + slot));
                    }
                }
                __syncwarp();
            }
            return true;
        };
        // V of key tile t; where the sequence ends inside it P is 0 past the end,
        // but the cache may hold anything there (NaN), so V is made 0 too
        auto wait_v = [&](int t, int valid) -> bool {
            const int st = t % kStages;
            if (!mbar_wait_warp(bar(L::kVFull + st), (t / kStages) & 1, wctx)) return false;
            if (valid < kBN) {
                KT::clear(smem + L::kV + st * L::kTileBytes, valid, lane);
                fence_proxy_async_smem();
                __syncwarp();
            }
            return true;
        };
        ok = enter(cs);
        cp = cs;
        for (int i = 0; i < 2 && ok; ++i) ok = step_s();
        // PV(q), S(q + 2) for every job q.  The MMA warp paces the kernel, and what it
        // costs is instructions fetched past those of eight softmax warps: the loop
        // over a segment's tiles is kept free of what only its last tile needs, its
        // waits for K and V stand where it waits for P anyway, and the products of S
        // are rolled by two (2 x 2048 tokens over 16384 keys: 807 us with one general
        // loop and a second variant of the softmax, 739 so; rolled by four 749,
        // unrolled 748, P V rolled too 770; P handed over whole 761 for 737).
        while (ok && cp.jobs > 0) {
            if (cp.two) {
                const int nt = cp.jobs >> 1, sa = cp.g & 1, sb = sa ^ 1;
                const int qa = (cs.u == cp.u ? q_n : 0) & 1, qb = qa ^ 1;     // used while S of this segment are left
                for (int j = 0; j + 1 < nt; ++j) {
                    const int st = cp.t % kStages, st1 = (cp.t + 1) % kStages;
                    const bool ends = j + 2 == nt;          // S of the segment's last tile
                    if (!(ok = wait_v(cp.t, kBN) && wait_k(cp.t + 1))) break;
                    if (!(ok = issue_pv(sa, (cp.g >> 1) & 1, st, j > 0, false, false))) break;
                    issue_s(sa, qa, st1, false, ends);
                    if (!(ok = issue_pv(sb, ((cp.g + 1) >> 1) & 1, st, j > 0, true, false))) break;
                    issue_s(sb, qb, st1, true, ends);
                    cp.g += 2;
                    ++cp.t;
                }
                if (!ok) break;
                if (nt > 1) {
                    cs.g = cp.g + 2;
                    cs.t = cp.t + 1;
                    q_n += 2;
                    ++cs.u;
                    if (!(ok = enter(cs))) break;
                }
                const int st = cp.t % kStages;
                if (!(ok = wait_v(cp.t, cp.tail))) break;
                if (!(ok = issue_pv(sa, (cp.g >> 1) & 1, st, nt > 1, false, true))) break;
                if (!(ok = step_s())) break;
                if (!(ok = issue_pv(sb, ((cp.g + 1) >> 1) & 1, st, nt > 1, true, true))) break;
                if (!(ok = step_s())) break;
                cp.g += 2;
                ++cp.t;
            } else {
                for (int j = 0; j < cp.jobs; ++j) {
                    if (!(ok = wait_v(cp.t, j + 1 == cp.jobs ? cp.tail : kBN))) break;
                    if (!(ok = issue_pv(cp.g & 1, (cp.g >> 1) & 1, cp.t % kStages, j >= 2, true, j + 2 >= cp.jobs))) break;
                    if (!(ok = step_s())) break;
                    ++cp.g;
                    ++cp.t;
                }
            }
            if (!ok) break;
            desc_release(cp.u);
            ++cp.u;
            ok = enter(cp);
        }
        if (any) {
            // every issued MMA must finish before tensor memory is released
            if (lead) umma_commit(bar(L::kDrain));
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
    } else if (warp < 8) {
        // ===================== softmax warpgroups =====================
        regs_alloc<kRegsSoftmax>();
        const int slot = warp >> 2;
        const int wq = warp & 3;            // lane quarter of tensor memory
        const int row = wq * 32 + lane;     // row within the tile
        const uint32_t tl = tmem + (static_cast<uint32_t>(wq * 32) << 16);
        const uint32_t tS = tl + L::kColS + slot * 128;
        const float qk = p.qk_scale_log2;
        bool ok = true;
        int g0 = 0;                         // jobs before this segment
        uint32_t ph = 0;                    // parities: bit s the O of slot s, bit 2 the merges
        for (int u = 0;; ++u) {
            if (!desc_wait(u)) break;
            const Seg &s = descs[u % kDescs];               // held until its results are written
            if (s.nt == 0) break;
            const int jobs = s.two ? 2 * s.nt : s.nt;
            const int first = (slot ^ g0) & 1;              // this slot's first job
            const uint32_t uses = jobs > 1 ? 3u : 1u << (g0 & 1);   // slots of this segment
            if (first >= jobs) {                            // a single job, the other slot's
                g0 += jobs;
                ph ^= uses;
                desc_release(u);
                continue;
            }
            bool active;                                    // the warp has rows
            int lim;                                        // last key that the row sees
            float m_ref;                                    // log2 units
            {
                const int tok = (s.two ? first * p.geom.tile_tokens : 0) + row / p.G;
                const bool valid = row < p.geom.tile_tokens * p.G && tok < s.ntok;
                active = __any_sync(0xffffffffu, valid);
                lim = p.causal ? min(s.lim0 + tok, s.len_k - 1) : s.len_k - 1;
                // rows of nothing: a reference maximum that no score exceeds, P = 0
                m_ref = valid ? neg_inf() : 1e30f;
            }
            float l = 0.f;
            const int kv_step = s.two ? kBN : 2 * kBN;
            int kv0 = (s.t0 + (s.two ? 0 : first)) * kBN;
            uint32_t s_ph = ((g0 + first) >> 1) & 1;
            bool later = false;                             // not the segment's first job here
            for (int n = (jobs - first + 1) >> 1; n > 0; --n, kv0 += kv_step, s_ph ^= 1, later = true) {
                {
                    const bool got = mbar_wait(bar(L::kSFull + slot), s_ph, wctx);
                    if (!__all_sync(0xffffffffu, got)) { ok = false; break; }
                }
                tc_fence_after();
                if (!active) {
                    tc_fence_before();
                    mbar_arrive(bar(L::kPHalf + 2 * slot));
                    mbar_arrive(bar(L::kPHalf + 2 * slot + 1));
                    continue;
                }
                uint32_t sr[128];
                tmem_ld32dp_x128_wait(tS, sr);
                float x[128];
#pragma unroll
                for (int c = 0; c < 128; ++c) x[c] = __uint_as_float(sr[c]);
                if (kv0 + kBN - 1 > lim) {
#pragma unroll
                    for (int c = 0; c < 128; ++c)
                        if (kv0 + c > lim) x[c] = neg_inf();
                }
                float mx0 = x[0], mx1 = x[1], mx2 = x[2], mx3 = x[3];
#pragma unroll
                for (int c = 4; c < 124; c += 8) {
                    mx0 = fmax3(mx0, x[c], x[c + 1]);
                    mx1 = fmax3(mx1, x[c + 2], x[c + 3]);
                    mx2 = fmax3(mx2, x[c + 4], x[c + 5]);
                    mx3 = fmax3(mx3, x[c + 6], x[c + 7]);
                }
                const float m_tile =
                    qk * fmax3(fmax3(mx0, mx1, x[124]), fmax3(mx2, mx3, x[125]), fmaxf(x[126], x[127]));
                const bool need = m_tile > m_ref + kTau;
                const bool rescale = __any_sync(0xffffffffu, need);     // warp-uniform
                float alpha = 1.f;
                if (rescale) {
                    const float m_new = need ? m_tile : m_ref;
                    alpha = (m_ref == neg_inf()) ? 0.f : ex2_approx(m_ref - m_new);
                    l *= alpha;
                    m_ref = m_new;
                }
                const float m_use = (m_ref == neg_inf()) ? 0.f : m_ref;
                // p = 2^(x - m) in two halves of 64 keys, each handed to the MMA warp on
                // its own barrier, rounded to the operands' type: the tensor cores take A
                // and B of one type, and P in two pieces (high and low) would double the
                // product.  The sum l takes p unrounded.  All on the MUFU: a quarter of
                // the pairs on the FMA pipe, as the other forward has it, gains in a burst
                // (2 x 2048 tokens over 12001..16384 keys: D = 128 719 -> 707 us, D = 64
                // 663 -> 614) and loses in long runs (D = 128 904 -> 912, with single
                // tokens 353 -> 360), and a quartic's error is in LSE.
                float2 lsum = make_float2(0.f, 0.f), lsum2 = make_float2(0.f, 0.f);
                const float2 neg_m2 = make_float2(-m_use, -m_use);
                const float2 qk2 = make_float2(qk, qk);
                auto half = [&](int h) {
                    uint32_t pk[32];
#pragma unroll
                    for (int c2 = 0; c2 < 32; ++c2) {
                        const int c = 64 * h + 2 * c2;
                        const float2 a = __ffma2_rn(make_float2(x[c], x[c + 1]), qk2, neg_m2);
                        const float2 pp = make_float2(ex2_approx(a.x), ex2_approx(a.y));
                        if (c2 & 1)
                            lsum2 = __fadd2_rn(lsum2, pp);
                        else
                            lsum = __fadd2_rn(lsum, pp);
                        pk[c2] = pack2<BF16>(pp.x, pp.y);
                    }
                    tmem_st32dp_x32(tS + 32 * h, pk);
                };
                half(0);
                if (rescale && later) {
                    // O row *= alpha.  O is stable: this S tile's MMA was issued
                    // after the slot's previous P V and its commit covers it.
                    const uint32_t tO = tl + L::kColO + slot * D;
#pragma unroll 1
                    for (int cc = 0; cc < D / 32; ++cc) {
                        uint32_t orr[32];
                        tmem_ld32dp_x32_wait(tO + cc * 32, orr);
#pragma unroll
                        for (int e = 0; e < 32; ++e) orr[e] = __float_as_uint(__uint_as_float(orr[e]) * alpha);
                        tmem_st32dp_x32(tO + cc * 32, orr);
                    }
                }
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(bar(L::kPHalf + 2 * slot));
                half(1);
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(bar(L::kPHalf + 2 * slot + 1));
                l += (lsum.x + lsum.y) + (lsum2.x + lsum2.y);
            }
            if (!ok) break;

            // ---- the rows' results: O = o / l, LSE = (m_ref + log2 l) ln 2
            const int r_tok = row / p.G, r_head = row - r_tok * p.G;
            const int tok = (s.two ? first * p.geom.tile_tokens : 0) + r_tok;
            const bool valid = r_tok < p.geom.tile_tokens && tok < s.ntok;
            const int ur = tok * p.G + r_head;              // row of the unit
            const int t = s.row0 + tok, head = s.h * p.G + r_head;
            uint16_t *o_row = nullptr;
            float *part = nullptr;
            if (s.dest < 0)
                o_row = static_cast<uint16_t *>(p.o) + head * p.o_h + t * p.o_n;
            else
                part = p.o_part + ((2 * blockIdx.x + s.dest) * static_cast<size_t>(p.part_rows) + ur) * D;
            auto store = [&](int col, const float (&y)[32]) {
                if (!valid) return;
                if (s.dest < 0) {
                    uint32_t pk[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) pk[e] = pack2<BF16>(y[2 * e], y[2 * e + 1]);
                    if (p.o_v8) {
                        st_global_v8(o_row + col, pk);
                        st_global_v8(o_row + col + 16, pk + 8);
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            reinterpret_cast<uint4 *>(o_row + col)[e] =
                                make_uint4(pk[4 * e], pk[4 * e + 1], pk[4 * e + 2], pk[4 * e + 3]);
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        reinterpret_cast<float4 *>(part + col)[e] =
                            make_float4(y[4 * e], y[4 * e + 1], y[4 * e + 2], y[4 * e + 3]);
                }
            };
            auto store_lse = [&](float m, float sum) {
                if (!valid) return;
                const float lse2 = sum == 0.f ? neg_inf() : m + lg2_approx(sum);
                if (s.dest < 0)
                    p.lse[static_cast<long long>(head) * p.T + t] = lse2 * kLn2;
                else
                    p.lse_part[(2 * blockIdx.x + s.dest) * static_cast<size_t>(p.part_rows) + ur] = lse2;
            };
            if (s.two || jobs == 1) {
                const bool got = mbar_wait(bar(L::kOFull + slot), (ph >> slot) & 1, wctx);
                if (!__all_sync(0xffffffffu, got)) { ok = false; break; }
                tc_fence_after();
                if (active) {
                    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
                    for (int cc = 0; cc < D / 32; ++cc) {
                        uint32_t r[32];
                        tmem_ld32dp_x32_wait(tl + L::kColO + slot * D + cc * 32, r);
                        float y[32];
#pragma unroll
                        for (int e = 0; e < 32; ++e) y[e] = __uint_as_float(r[e]) * inv;
                        store(32 * cc, y);
                    }
                    store_lse(m_ref, l);
                }
                tc_fence_before();
            } else {
                // the two slots hold the sums over the even and odd key tiles of
                // the same rows; each warpgroup adds up half of the columns
                stats[slot * kBM + row] = make_float2(m_ref, l);
                mbar_arrive(bar(L::kStat));
                bool got = mbar_wait(bar(L::kStat), (ph >> 2) & 1, wctx) && mbar_wait(bar(L::kOFull + 0), ph & 1, wctx) &&
                           mbar_wait(bar(L::kOFull + 1), (ph >> 1) & 1, wctx);
                if (!__all_sync(0xffffffffu, got)) { ok = false; break; }
                tc_fence_after();
                if (active) {
                    const float2 other = stats[(slot ^ 1) * kBM + row];
                    const float m = fmaxf(m_ref, other.x);
                    const float a = m_ref == neg_inf() ? 0.f : ex2_approx(m_ref - m);
                    const float b = other.x == neg_inf() ? 0.f : ex2_approx(other.x - m);
                    const float sum = l * a + other.y * b;
                    const float inv = sum == 0.f ? 0.f : 1.f / sum;
                    const float w_own = a * inv, w_oth = b * inv;
#pragma unroll
                    for (int cc = 0; cc < D / 64; ++cc) {
                        const int col = slot * (D / 2) + 32 * cc;
                        uint32_t r[32], q[32];
                        tmem_ld32dp_x32_wait(tl + L::kColO + slot * D + col, r);
                        tmem_ld32dp_x32_wait(tl + L::kColO + (slot ^ 1) * D + col, q);
                        float y[32];
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            y[e] = fmaf(__uint_as_float(r[e]), w_own, __uint_as_float(q[e]) * w_oth);
                        store(col, y);
                    }
                    if (slot == 0) store_lse(m, sum);
                }
                // both read the other's O and statistics before either is replaced
                tc_fence_before();
                mbar_arrive(bar(L::kRead));
                got = mbar_wait(bar(L::kRead), (ph >> 2) & 1, wctx);
                if (!__all_sync(0xffffffffu, got)) { ok = false; break; }
                ph ^= 4;
            }
            ph ^= uses;
            g0 += jobs;
            desc_release(u);
        }
        __syncwarp();
        named_bar_sync(1, kThreads);
    } else {
        named_bar_sync(1, kThreads);    // warp 11
    }
}

// Joins the partial results of the units that were cut: CTA c begins such a
// unit (its partial result 1), CTAs c + 1 .. last continue it (their partial
// results 0); added in that order.  One warp per row.
template <int D, bool BF16>
__global__ void __launch_bounds__(256, 6) fa_paged_merge_kernel(const __grid_constant__ PagedFwdParams p) {
    constexpr int kPer = D / 32;
    const int c = blockIdx.x, lane = threadIdx.x & 31;
    const int ur = blockIdx.y * 8 + (threadIdx.x >> 5);
    grid_launch_dependents();           // the next call may be set up; it waits for this grid
    grid_dependency_wait();             // the partial results are complete and visible
    const MergeMeta mm = p.meta[c];
    if (mm.last < 0 || ur >= mm.tokens * p.G) return;
    auto index = [&](int i) -> size_t {
        return static_cast<size_t>(i == c ? 2 * c + 1 : 2 * i) * p.part_rows + ur;
    };
    float m = neg_inf();
    bool nan = false;                   // of a row of NaN: it stays one
    for (int i = c + lane; i <= mm.last; i += 32) {
        const float x = __ldcg(p.lse_part + index(i));
        nan |= x != x;
        m = fmaxf(m, x);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    float acc[kPer], sum = 0.f;
#pragma unroll
    for (int e = 0; e < kPer; ++e) acc[e] = 0.f;
    if (__any_sync(0xffffffffu, nan)) m = 0.f;
    if (m != neg_inf()) {
        for (int i0 = c; i0 <= mm.last; i0 += 32) {
            // lane k has the weight of part i0 + k
            const int cnt = min(32, mm.last + 1 - i0);
            const float wl = lane < cnt ? ex2_approx(__ldcg(p.lse_part + index(i0 + lane)) - m) : 0.f;     // -inf: 0
            // the parts' rows, U loads in flight (more cost the occupancy that many
            // rows of two parts need)
            auto add = [&](auto n, int k) {
                constexpr int U = decltype(n)::value;
                float w[U], v[U][kPer];
#pragma unroll
                for (int q = 0; q < U; ++q) {
                    w[q] = __shfl_sync(0xffffffffu, wl, (k + q) & 31);
                    const float *src = p.o_part + index(i0 + min(k + q, cnt - 1)) * D + lane * kPer;
                    if constexpr (kPer == 4) {
                        const float4 f = __ldcg(reinterpret_cast<const float4 *>(src));
                        v[q][0] = f.x; v[q][1] = f.y; v[q][2] = f.z; v[q][3] = f.w;
                    } else {
                        const float2 f = __ldcg(reinterpret_cast<const float2 *>(src));
                        v[q][0] = f.x; v[q][1] = f.y;
                    }
                }
#pragma unroll
                for (int q = 0; q < U; ++q) {
                    if (k + q >= cnt) break;
                    sum += w[q];
#pragma unroll
                    for (int e = 0; e < kPer; ++e) acc[e] = fmaf(w[q], v[q][e], acc[e]);
                }
            };
            int k = 0;
            for (; k + 2 < cnt; k += 4) add(std::integral_constant<int, 4>{}, k);
            for (; k < cnt; k += 2) add(std::integral_constant<int, 2>{}, k);
        }
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const int t = mm.row0 + ur / p.G, head = mm.h * p.G + ur % p.G;
    uint32_t *dst = reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(p.o) + head * p.o_h + t * p.o_n + lane * kPer);
#pragma unroll
    for (int e = 0; e < kPer / 2; ++e) dst[e] = pack2<BF16>(acc[2 * e] * inv, acc[2 * e + 1] * inv);
    if (lane == 0)
        p.lse[static_cast<long long>(head) * p.T + t] = sum == 0.f ? neg_inf() : (m + lg2_approx(sum)) * kLn2;
}

template <int D, bool BF16>
cudaError_t launch_t(const PagedTensorMaps &tm, const PagedFwdParams &p, int grid, cudaStream_t stream) {
    auto kern = fa_paged_kernel<D, BF16>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, PagedLayout<D>::kAlloc);
    if (e != cudaSuccess) return e;
    prof_begin(stream, "fa_paged_kernel");
    e = launch_early(kern, dim3(grid), kThreads, PagedLayout<D>::kAlloc, stream, tm.q, tm.k, tm.v, p);
    prof_end(stream);
    note_launch();
    if (e != cudaSuccess) return e;
    return launch_paged_merge(p, BF16, grid, stream);
}

template <int D, bool BF16>
cudaError_t launch_merge_t(const PagedFwdParams &p, int grid, cudaStream_t stream) {
    prof_begin(stream, "fa_paged_merge_kernel");
    const cudaError_t e =
        launch_early(fa_paged_merge_kernel<D, BF16>, dim3(grid, (p.part_rows + 7) / 8), 256, 0, stream, p);
    prof_end(stream);
    note_launch();
    return e;
}

}  // namespace

cudaError_t launch_paged_fwd(const PagedTensorMaps &tm, const PagedFwdParams &p, bool bf16, int sms,
                             cudaStream_t stream) {
    const int grid = sms < kPagedMaxCtas ? sms : kPagedMaxCtas;
    if (p.kv.D == 64) return bf16 ? launch_t<64, true>(tm, p, grid, stream) : launch_t<64, false>(tm, p, grid, stream);
    return bf16 ? launch_t<128, true>(tm, p, grid, stream) : launch_t<128, false>(tm, p, grid, stream);
}

cudaError_t launch_paged_merge(const PagedFwdParams &p, bool bf16, int grid, cudaStream_t stream) {
    if (p.kv.D == 64) return bf16 ? launch_merge_t<64, true>(p, grid, stream) : launch_merge_t<64, false>(p, grid, stream);
    return bf16 ? launch_merge_t<128, true>(p, grid, stream) : launch_merge_t<128, false>(p, grid, stream);
}

}  // namespace fa
