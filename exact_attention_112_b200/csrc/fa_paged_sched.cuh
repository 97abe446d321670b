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
// An entry is one key tile of a unit with one tile of query rows, a unit with
// two counts each key tile twice.  A unit without a visible key counts as one
// entry: its rows have to be written.
#pragma once

#include "fa_paged_internal.h"

namespace fa {

// Key tiles of the unit whose tokens start at tok0.
__device__ __forceinline__ int unit_tiles(const PagedSeq &s, int tok0, const SchedGeom &g, int causal) {
    int vis = s.len_k;
    if (causal) {
        const int last = min(tok0 + g.unit_tokens, s.new_q) - 1;
        vis = min(vis, last + 1 + s.len_k - s.new_q);
    }
    return vis <= 0 ? 0 : (vis + g.tile - 1) / g.tile;
}

__device__ __forceinline__ long long unit_cost(const PagedSeq &s, int tok0, const SchedGeom &g, int causal) {
    const int n = max(1, unit_tiles(s, tok0, g, causal));
    return tok0 + g.tile_tokens < s.new_q ? 2ll * n : n;
}

// Work of one kv head of a sequence.
__device__ __forceinline__ long long head_cost(const PagedSeq &s, const SchedGeom &g, int causal) {
    long long c = 0;
    for (int t = 0; t < s.new_q; t += g.unit_tokens) c += unit_cost(s, t, g, causal);
    return c;
}

__device__ __forceinline__ PagedSeq load_seq(const PagedFwdParams &p, int b) {
    return paged_seq(b, p.cu, p.kv.seq_lens, p.T, p.max_q, static_cast<long long>(p.kv.max_pages) * p.kv.page_size);
}

// One CTA's piece of the line, and where its first unit starts.
struct Piece {
    long long lo, hi;       // entries [lo, hi)
    long long total;        // W
    int ctas;               // C
    long long start;        // first entry of sequence b
    int b;                  // sequence that holds entry lo (-1: no work)
};

// Shared memory of plan_piece().
struct PlanSmem {
    long long warp_sum[32];
    long long start;
    int b;
};

// Computed by all NT threads of the CTA together; the result is the same for
// every thread.  min_piece: the least entries worth a CTA of its own.
template <int NT>
__device__ __forceinline__ Piece plan_piece(const PagedFwdParams &p, const SchedGeom &g, int min_piece, PlanSmem &sm) {
    constexpr int kWarps = NT / 32;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int B = p.kv.num_seqs;
    if (tid == 0) sm.b = -1;
    Piece pc;
    pc.total = 0;
    long long mine = 0;         // work of sequence tid of the (last) round of NT sequences
    for (int b0 = 0; b0 < B; b0 += NT) {
        mine = b0 + tid < B ? p.kv.Hkv * head_cost(load_seq(p, b0 + tid), g, p.causal) : 0;
        pc.total += mine;
    }
    long long v = pc.total;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (lane == 0) sm.warp_sum[warp] = v;
    __syncthreads();
    pc.total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) pc.total += sm.warp_sum[w];
    const long long most = (pc.total + min_piece - 1) / min_piece;
    pc.ctas = static_cast<int>(most < gridDim.x ? most : gridDim.x);
    const int c = blockIdx.x;
    if (c >= pc.ctas) {
        pc.b = -1;
        pc.lo = pc.hi = pc.start = 0;
        return pc;              // the same branch for every thread
    }
    pc.lo = c * pc.total / pc.ctas;
    pc.hi = (c + 1) * pc.total / pc.ctas;
    long long base = 0;
    for (int b0 = 0; b0 < B; b0 += NT) {
        if (B > NT) mine = b0 + tid < B ? p.kv.Hkv * head_cost(load_seq(p, b0 + tid), g, p.causal) : 0;
        long long inc = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long x = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += x;
        }
        __syncthreads();        // the sums of the round before have been read
        if (lane == 31) sm.warp_sum[warp] = inc;
        __syncthreads();
        long long before = base;
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) before += sm.warp_sum[w];
            base += sm.warp_sum[w];
        }
        const long long at = before + inc - mine;
        if (mine > 0 && at <= pc.lo && pc.lo < at + mine) {
            sm.start = at;
            sm.b = b0 + tid;
        }
    }
    __syncthreads();
    pc.b = sm.b;
    pc.start = sm.start;
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
    long long base;         // the unit's first entry
    long long cost;
    // the piece
    long long lo, hi;

    __device__ __forceinline__ void unit(const PagedFwdParams &p, const SchedGeom &g) {
        n = unit_tiles(s, tok0, g, p.causal);
        two = tok0 + g.tile_tokens < s.new_q;
        cost = two ? 2ll * max(1, n) : max(1, n);
    }

    __device__ __forceinline__ void first(const PagedFwdParams &p, const SchedGeom &g, const Piece &pc) {
        lo = pc.lo;
        hi = pc.hi;
        b = pc.b;
        h = 0;
        tok0 = 0;
        base = pc.start;
        s = load_seq(p, b);
        const long long per_head = head_cost(s, g, p.causal);
        h = static_cast<int>((lo - base) / per_head);
        base += h * per_head;
        unit(p, g);
        while (base + cost <= lo) {
            base += cost;
            tok0 += g.unit_tokens;
            unit(p, g);
        }
        range();
    }

    __device__ __forceinline__ void range() {
        const int w = two ? 2 : 1;
        const long long a = lo - base, z = hi - base;
        t0 = a <= 0 ? 0 : static_cast<int>(min(static_cast<long long>(n), (a + w - 1) / w));
        t1 = static_cast<int>(min(static_cast<long long>(n), (z + w - 1) / w));
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
        range();
        return true;
    }

    // Does this segment write the unit's rows itself?
    __device__ __forceinline__ bool whole() const { return t0 == 0 && t1 == n; }

    // Nothing of the unit falls to this CTA (a boundary inside a doubled entry).
    __device__ __forceinline__ bool none() const { return n > 0 && t0 >= t1; }

    // CTA that holds the unit's last key tile.
    __device__ __forceinline__ int last_cta(const Piece &pc) const {
        const long long at = base + (two ? 2ll : 1ll) * (n - 1);
        return static_cast<int>(((at + 1) * pc.ctas - 1) / pc.total);
    }
};

}  // namespace fa
