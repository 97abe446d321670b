// fa_paged_sched.cuh -- how the paged-attention kernels share out their work.
//
// A unit is a block of new tokens of one sequence for one kv head (all the
// query heads of its group); its work is the key tiles that the block's last
// token sees.  The units of the batch, in the order (sequence, kv head, token
// block), laid end to end make one line of work, and CTA c of C takes the
// piece [c W / C, (c + 1) W / C) of its W entries: whatever the lengths, no CTA
// has more than its share by one tile, and nothing is planned on the host, so
// the tables may change under a captured graph.  A unit cut by a boundary gives
// partial results (O / l, m + log2 l in fp32), at most two per CTA -- slot 0 for
// a unit that began before the CTA's piece, slot 1 for one that ends after it --
// which a second kernel merges in the order of the CTAs, so the result does not
// depend on timing.
//
// A unit counts `unit_cost` entries, for what its beginning and end take, and then
// for each of its key tiles `one_cost`, or `two_cost` where it has two tiles of
// query rows.  A unit without a visible key counts as one tile: its rows have to
// be written.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fa_paged_internal.h"
#include "fa_paged_ptx.cuh"

namespace fa {

// Key tiles of the unit whose tokens start at tok0.
__device__ __forceinline__ int unit_tiles(const PagedSeq &s, int tok0, const SchedGeom &g, int causal) {
    int vis = s.len_k;
    if (causal) {
        const int last = min(tok0 + g.unit_tokens, s.new_q) - 1;
        vis = min(vis, last + 1 + s.past);
    }
    return vis <= 0 ? 0 : (vis + kPagedTile - 1) / kPagedTile;
}

__device__ __forceinline__ long long unit_cost(const PagedSeq &s, int tok0, const SchedGeom &g, int causal) {
    const long long n = max(1, unit_tiles(s, tok0, g, causal));
    return g.unit_cost + n * (tok0 + g.tile_tokens < s.new_q ? g.two_cost : g.one_cost);
}

// Work of one kv head of each lane's sequence.  A sequence of many units is
// summed up by the whole warp.
__device__ __forceinline__ long long head_cost(const PagedSeq &s, const SchedGeom &g, int causal, int lane) {
    const bool many = s.new_q > 2 * g.unit_tokens;
    long long c = 0;
    if (!many && s.new_q > 0) {
        c = unit_cost(s, 0, g, causal);
        if (s.new_q > g.unit_tokens) c += unit_cost(s, g.unit_tokens, g, causal);
    }
    for (unsigned todo = __ballot_sync(0xffffffffu, many); todo != 0; todo &= todo - 1) {
        const int l = __ffs(todo) - 1;
        PagedSeq w;
        w.q0 = 0;
        w.new_q = __shfl_sync(0xffffffffu, s.new_q, l);
        w.len_k = __shfl_sync(0xffffffffu, s.len_k, l);
        w.past = __shfl_sync(0xffffffffu, s.past, l);
        long long sum = 0;
        for (int t = lane * g.unit_tokens; t < w.new_q; t += 32 * g.unit_tokens) sum += unit_cost(w, t, g, causal);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (lane == l) c = sum;
    }
    return c;
}

// Inclusive sums over the warp; narrow: every sum fits 31 bits.
__device__ __forceinline__ long long warp_scan(long long x, int lane, bool narrow) {
    if (narrow) {
        int v = static_cast<int>(x);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += y;
        }
        return v;
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    return x;
}

__device__ __forceinline__ PagedSeq load_seq(const PagedFwdParams &p, int b) {
    return paged_seq(b, p.cu, p.kv.seq_lens, p.T, p.max_q, static_cast<long long>(p.kv.max_pages) * p.kv.page_size);
}

// a / b for a >= 0, b > 0.  Several quotients in a row stand at the beginning of
// every call: below 2^24 a float32 reciprocal gives one that is off by one at
// most (100 cycles less than the 32-bit division, 500 less than the 64-bit one).
__device__ __forceinline__ long long div_wide(long long a, long long b) {
    if (((a | b) >> 24) == 0) {
        const int x = static_cast<int>(a), y = static_cast<int>(b);
        int q = static_cast<int>(__int2float_rn(x) * __frcp_rn(__int2float_rn(y)));
        const int r = x - q * y;
        q += r >= y ? 1 : r < 0 ? -1 : 0;
        return q;
    }
    if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
    return a / b;
}

// One CTA's piece of the line, and where its first unit starts.
struct Piece {
    long long lo, hi;       // entries [lo, hi)
    long long total;        // W
    int ctas;               // C
    long long quot;         // W / C
    int rem;                // W % C: the first `rem` pieces have one more
    long long start;        // first entry of sequence b
    int b;                  // sequence that holds entry lo (-1: no work)
    PagedSeq s;             // its rows and keys
    long long per_head;     // its work for one kv head
};

// The CTA's piece, computed by one warp (every lane gets the same) in steps of
// 128 sequences, four to a lane; a batch of that size costs one latency of the
// tables.  min_piece: the least entries worth a CTA of its own.
constexpr int kPlanRounds = 4;
constexpr int kPlanStep = 32 * kPlanRounds;

struct PlanSeqs {
    PagedSeq s[kPlanRounds];
};

__device__ __forceinline__ void plan_load(const PagedFwdParams &p, int b0, int lane, PlanSeqs &q) {
#pragma unroll
    for (int i = 0; i < kPlanRounds; ++i) {
        const int b = b0 + 32 * i + lane;
        q.s[i] = b < p.kv.num_seqs ? load_seq(p, b) : PagedSeq{0, 0, 0, 0};
    }
}

// q: sequences 0 .. kPlanStep - 1, asked for by the caller ahead of other set-up.
__device__ __forceinline__ Piece plan_piece(const PagedFwdParams &p, const SchedGeom &g, int min_piece, int lane,
                                            PlanSeqs &q) {
    const int B = p.kv.num_seqs;
    Piece pc;
    long long head[kPlanRounds], v = 0;     // work of one kv head of this lane's sequences
    auto costs = [&](int b0) {
#pragma unroll
        for (int i = 0; i < kPlanRounds; ++i) {
            head[i] = b0 + 32 * i < B ? head_cost(q.s[i], g, p.causal, lane) : 0;
            v += p.kv.Hkv * head[i];
        }
    };
#pragma unroll 1
    for (int b0 = 0; b0 < B; b0 += kPlanStep) {
        if (b0 > 0) plan_load(p, b0, lane, q);
        costs(b0);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    pc.total = v;
    pc.ctas = pc.total >= static_cast<long long>(min_piece) * gridDim.x
                  ? static_cast<int>(gridDim.x) : static_cast<int>(div_wide(pc.total + min_piece - 1, min_piece));
    pc.quot = pc.ctas > 0 ? div_wide(pc.total, pc.ctas) : 0;
    pc.rem = static_cast<int>(pc.total - pc.quot * pc.ctas);
    const int c = blockIdx.x;
    pc.b = -1;
    pc.lo = pc.hi = pc.start = 0;
    if (c >= pc.ctas) return pc;
    pc.lo = c * pc.quot + min(c, pc.rem);
    pc.hi = pc.lo + pc.quot + (c < pc.rem ? 1 : 0);
    const bool narrow = (pc.total >> 31) == 0;
    long long base = 0;     // entries before the round's sequences
#pragma unroll 1
    for (int b0 = 0; b0 < B; b0 += kPlanStep) {
        if (B > kPlanStep) {
            plan_load(p, b0, lane, q);
            costs(b0);
        }
#pragma unroll
        for (int i = 0; i < kPlanRounds; ++i) {
            if (b0 + 32 * i >= B) break;
            const long long mine = p.kv.Hkv * head[i];
            const long long inc = warp_scan(mine, lane, narrow);
            const long long at = base + inc - mine;
            const unsigned hit = __ballot_sync(0xffffffffu, mine > 0 && at <= pc.lo && pc.lo < at + mine);
            base += __shfl_sync(0xffffffffu, inc, 31);
            if (hit == 0) continue;
            const int l = __ffs(hit) - 1;
            pc.b = b0 + 32 * i + l;
            pc.start = __shfl_sync(0xffffffffu, at, l);
            pc.s.q0 = __shfl_sync(0xffffffffu, q.s[i].q0, l);
            pc.s.new_q = __shfl_sync(0xffffffffu, q.s[i].new_q, l);
            pc.s.len_k = __shfl_sync(0xffffffffu, q.s[i].len_k, l);
            pc.s.past = __shfl_sync(0xffffffffu, q.s[i].past, l);
            pc.per_head = __shfl_sync(0xffffffffu, head[i], l);
            return pc;
        }
    }
    return pc;
}

// Walks a CTA's segments: (unit, range of its key tiles).
struct SegWalk {
    // the current unit
    PagedSeq s;
    int b, h, tok0;
    int n;                  // key tiles of the unit
    int t0, t1;             // those of this segment
    bool two;               // two tiles of query rows
    int w;                  // entries of a key tile
    long long base;         // the unit's first entry
    long long cost;
    // the piece
    long long lo, hi;

    __device__ __forceinline__ void unit(const PagedFwdParams &p, const SchedGeom &g) {
        n = unit_tiles(s, tok0, g, p.causal);
        two = tok0 + g.tile_tokens < s.new_q;
        w = two ? g.two_cost : g.one_cost;
        cost = g.unit_cost + static_cast<long long>(w) * max(1, n);
    }

    // By a whole warp: the unit that holds entry lo.
    __device__ __forceinline__ void first(const PagedFwdParams &p, const SchedGeom &g, const Piece &pc, int lane) {
        lo = pc.lo;
        hi = pc.hi;
        b = pc.b;
        h = 0;
        tok0 = 0;
        base = pc.start;
        s = pc.s;
        h = static_cast<int>(div_wide(lo - base, pc.per_head));
        base += h * pc.per_head;
        // 32 units at a time
        for (; s.new_q > g.unit_tokens; tok0 += 32 * g.unit_tokens) {
            const int t = tok0 + lane * g.unit_tokens;
            const long long c = t < s.new_q ? unit_cost(s, t, g, p.causal) : 0;
            const long long inc = warp_scan(c, lane, (pc.per_head >> 31) == 0);
            const unsigned hit = __ballot_sync(0xffffffffu, c > 0 && lo < base + inc);
            if (hit != 0) {
                const int l = __ffs(hit) - 1;
                base += __shfl_sync(0xffffffffu, inc - c, l);
                tok0 += l * g.unit_tokens;
                break;
            }
            base += __shfl_sync(0xffffffffu, inc, 31);
        }
        unit(p, g);
        range(g);
    }

    // Key tile j is the CTA's that holds the unit's entry unit_cost + w * j.
    __device__ __forceinline__ void range(const SchedGeom &g) {
        const long long a = lo - base - g.unit_cost, z = hi - base - g.unit_cost;
        t0 = a <= 0 ? 0 : static_cast<int>(min(static_cast<long long>(n), div_wide(a + w - 1, w)));
        t1 = z <= 0 ? 0 : base + cost <= hi ? n : static_cast<int>(min(static_cast<long long>(n), div_wide(z + w - 1, w)));
    }

    // The next unit of the piece; false when there is none.
    __device__ __forceinline__ bool next(const PagedFwdParams &p, const SchedGeom &g) {
        base += cost;
        if (base >= hi) return false;
        tok0 += g.unit_tokens;
        if (tok0 >= s.new_q) {
            tok0 = 0;
            if (++h == p.kv.Hkv) {
                h = 0;
                do {
                    if (++b >= p.kv.num_seqs) return false;
                    s = load_seq(p, b);
                } while (s.new_q == 0);
            }
        }
        unit(p, g);
        range(g);
        return true;
    }

    // Does this segment write the unit's rows itself?
    __device__ __forceinline__ bool whole() const { return t0 == 0 && t1 == n; }

    // Nothing of the unit falls to this CTA (a boundary inside its beginning, or a tile's entries).
    __device__ __forceinline__ bool none() const { return n > 0 && t0 >= t1; }

    // CTA that holds the unit's last key tile.
    __device__ __forceinline__ int last_cta(const Piece &pc, const SchedGeom &g) const {
        const long long at = base + g.unit_cost + static_cast<long long>(w) * (n - 1), wide = pc.rem * (pc.quot + 1);
        return static_cast<int>(at < wide ? div_wide(at, pc.quot + 1) : pc.rem + div_wide(at - wide, pc.quot));
    }
};

// A segment as the kernels' roles hand it on: key tiles [t0, t0 + nt) of a unit
// (nt == 0: the end of the work).
struct Seg {
    int row0, ntok;     // first row of the packed tensors, tokens
    int h, b;           // kv head, sequence
    int len_k, lim0;    // keys of the sequence; last key the first token sees
    int t0, nt;
    int two;            // two tiles of query rows
    int tail;           // keys below len_k in the last key tile
    int dest;           // -1: the rows' results, else partial result `dest` of this CTA
    int pad;
};

__device__ __forceinline__ Seg make_seg(const SegWalk &w, const SchedGeom &g) {
    Seg s;
    s.row0 = w.s.q0 + w.tok0;
    s.ntok = min(g.unit_tokens, w.s.new_q - w.tok0);
    s.h = w.h;
    s.b = w.b;
    s.len_k = w.s.len_k;
    s.lim0 = w.tok0 + w.s.past;
    s.t0 = w.t0;
    s.nt = w.t1 - w.t0;
    s.two = w.two;
    s.tail = min(kPagedTile, w.s.len_k - (w.t1 - 1) * kPagedTile);
    s.dest = w.whole() ? -1 : (w.t0 == 0 ? 1 : 0);
    s.pad = 0;
    return s;
}

__device__ __forceinline__ float neg_inf() { return __int_as_float(0xff800000); }

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

// Where key tiles lie in shared memory: groups of eight rows, in each the row's
// 64-value column blocks one after the other, in each of those eight rows of 128
// bytes, swizzled.  So a box of any multiple of eight rows and the whole head is
// one piece, and one TMA copy: a copy costs the issuing warp some 75 cycles
// whatever its size, and 16-row pages in copies of half a head were bound by that.
template <int D>
struct KeyTile {
    static constexpr int kChunks = D / 64;
    static constexpr int kGroupBytes = kChunks * 1024;      // eight rows
    static constexpr int kBytes = 16 * kGroupBytes;         // 128 rows
    // K (or V^T's columns): 16 values (32 bytes) per step along the row
    __device__ static __forceinline__ uint64_t k_desc(uint32_t addr) { return smem_desc_sw128(addr, 16, kGroupBytes); }
    __device__ static constexpr uint32_t k_step(int kk) { return ((kk >> 2) * 1024 + (kk & 3) * 32) >> 4; }
    // V: 16 keys per step; column blocks of 64 are 1024 bytes apart (`blocks` false:
    // the one block again and again)
    __device__ static __forceinline__ uint64_t v_desc(uint32_t addr, bool blocks) {
        return smem_desc_sw128(addr, blocks ? 1024 : 0, kGroupBytes);
    }
    __device__ static constexpr uint32_t v_step(int kk) { return (kk * 2 * kGroupBytes) >> 4; }
    // Rows [from, 128) = 0, by one warp.
    __device__ static __forceinline__ void clear(uint8_t *tile, int from, int lane) {
        for (int e = lane; e < (128 - from) * kChunks * 8; e += 32) {
            const int r = from + e / (kChunks * 8), c = e % (kChunks * 8);
            *reinterpret_cast<uint4 *>(tile + (r >> 3) * kGroupBytes + (c >> 3) * 1024 + (r & 7) * 128 + (c & 7) * 16) =
                make_uint4(0, 0, 0, 0);
        }
    }
};

// A lane's part of the copies of a key tile: box `lane` of it.  The table's entry
// is asked for a tile ahead.
struct PageBoxes {
    const int *table;
    int h, key_off;
    bool copies;
    int entry, row;

    __device__ __forceinline__ void init(const PagedFwdParams &p, int lane) {
        key_off = lane * p.box;
        copies = key_off < 128;
    }
    __device__ __forceinline__ void segment(const PagedFwdParams &p, const Seg &s) {
        table = p.kv.table + s.b * p.kv.table_stride;
        h = s.h;
    }
    __device__ __forceinline__ void look_up(const PagedFwdParams &p, int kt, int len_k) {
        const int key = kt * 128 + key_off;
        entry = -1;
        row = 0;
        if (copies && key < len_k) {
            const int pi = key / p.kv.page_size;
            row = key - pi * p.kv.page_size;
            entry = __ldg(table + pi);
        }
    }
    // Coordinates of the box (dimensions: 64 values, 8 rows, column blocks, and
    // either groups of eight rows and (page, head), or head and page).  A page that
    // is not to be read is one past the last: TMA fills its box with zeros.
    struct Box {
        int y, z, w;
    };
    __device__ __forceinline__ Box box(const PagedFwdParams &p, int ratio) const {
        const bool ok = entry >= 0 && entry < p.kv.num_pages;
        if (p.fold) return Box{0, row >> 3, ok ? entry * ratio + h : (p.kv.num_pages - 1) * ratio + p.kv.Hkv};
        return Box{row, h, ok ? entry : p.kv.num_pages};
    }
    __device__ __forceinline__ void copy(const PagedFwdParams &p, const CUtensorMap *m, uint32_t tile, int group_bytes,
                                         uint32_t bar, const Box &b) const {
        if (copies) tma_load_5d(tile + (key_off >> 3) * group_bytes, m, bar, 0, b.y, 0, b.z, b.w);
    }
};

// Rows without a visible key: O = 0, LSE = -inf.  By one warp.
template <int D>
__device__ __forceinline__ void write_empty(const PagedFwdParams &p, int row0, int ntok, int h, int lane) {
    const int n = ntok * p.G;
    for (int r = lane; r < n; r += 32) {
        const int t = row0 + r / p.G, head = h * p.G + r % p.G;
        uint4 *o = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.o) + head * p.o_h + t * p.o_n);
        for (int c = 0; c < D / 8; ++c) o[c] = make_uint4(0, 0, 0, 0);
        p.lse[static_cast<long long>(head) * p.T + t] = neg_inf();
    }
}

}  // namespace fa
