// What the kernels of wh_prefix_attention share: the work's description, how blocks find their group, and
// how a row of a work item names its query.
#pragma once
#include "common.cuh"
#include "internal.h"

namespace wh {

// Weights are 2^((s - m) log2(e) / sqrt(64)) of the raw products s = q . k and their maximum m: the difference
// comes first, so that it is exact near the maximum however large the scores are.
constexpr float PA_SCALE = 0.125f * 1.4426950408889634f;

struct PaSet {
    const __nv_bfloat16 *k, *v;
    long long row_stride, set_stride;   // elements
    const int *n_keys;                  // device [n_set] or null (max_keys for all)
    float *weight;                      // device [n_set][n_kv][max_keys] or null
    int n_set, max_keys;
    int splits, chunk;                  // key ranges of one set and keys of a range
    Divisor by_splits, by_chunk;
};

struct PaArgs {
    PaSet pre, own;
    const __nv_bfloat16 *q;
    long long q_stride;
    const int *group_start;   // device [pre.n_set + 1] or null: gsize sequences each
    int gsize, batch, nq, n_head, n_kv, rep;
    Divisor by_per, by_rep, by_seq;   // nq rep (rows of a sequence), rep, nq n_head
    Divisor by_gsize, by_group_tiles, by_slots, by_pre_tiles, by_own_tiles, by_kv;
    int tile, tile_shift;     // prefix: rows of a row tile, a power of two
    int group_tiles;          // row tiles of a group, without group_start
    int slots;                // prefix: row-tile slots of a key head over all groups
    int own_tiles;            // row tiles of a sequence
    int own_wpi;              // own keys: warps of a work item
    long long own_items;      // own keys: (sequence, key head, row tile, range)
    // How the key ranges of a row come together.  Without own keys, and for own keys alone, the blocks of one
    // item's ranges form a thread-block cluster (its size; 1: a single range) and finish their rows themselves.
    // With both, the prefix blocks leave partial results and the sequences' own blocks, one range each, finish
    // the rows.  Otherwise (0) all leave partial results and k_prefix_merge joins them.
    int pre_cluster, own_cluster;
    int n_part;               // partial results of a row: of the prefix's ranges, then of the own keys'
    int after_pre;            // own keys' blocks: the prefix's may still be running until pdl_wait
    int score_floats;         // own keys: scores that an item keeps in shared memory for the weights, or 0
    float *part_o;            // [row][n_part][64], row = (b nq + i) n_head + h
    float2 *part_ml;          // [row][n_part]: running maximum and sum
    float2 *stats;            // [row]: maximum and 1 / sum (weights only)
    __nv_bfloat16 *out;       // [batch * nq][64 n_head]
    DevCtl ctl;
};

__device__ __forceinline__ int clamp_count(const PaSet &s, int set) {
    return s.n_keys ? min(max(ld_live(s.n_keys + set), 0), s.max_keys) : s.max_keys;
}

// Largest g in [0, n) with start[g] * mul / 2^shift + g * add <= x, by the whole warp, 32 probes at a time.
__device__ __forceinline__ int warp_search(const int *start, int n, int mul, int shift, int add, long long x) {
    int lo = 0, len = n;
    const int lane = threadIdx.x & 31;
    while (len > 1) {
        const int step = (len + 31) / 32, i = lane * step;
        bool le = false;
        if (i < len) {
            const int g = lo + i;
            le = ((long long)ld_live(start + g) * mul >> shift) + (long long)g * add <= x;
        }
        const uint32_t m = __ballot_sync(0xffffffffu, le) | 1u;
        const int top = (31 - __clz(m)) * step;
        lo += top;
        len = min(step, len - top);
    }
    return lo;
}

// Sequences [s, e) of group g, cut to 0 .. batch.
__device__ __forceinline__ void group_range(const PaArgs &p, int g, int &s, int &e) {
    if (p.group_start) {
        s = min(max(ld_live(p.group_start + g), 0), p.batch);
        e = min(max(ld_live(p.group_start + g + 1), s), p.batch);
    } else {
        s = g * p.gsize;
        e = s + p.gsize;
    }
}

// The rows of one work item: queries of sequences first .. (rows / (nq rep)), row r =
// ((sequence, query), query head of the key head).
struct Rows {
    int seq0, n, hk;
    __device__ __forceinline__ void locate(const PaArgs &p, int r, int &qrow, int &head, int &qi) const {
        const int s = p.by_per.of(r), w = r - s * p.nq * p.rep;
        qi = p.by_rep.of(w);
        qrow = (seq0 + s) * p.nq + qi;
        head = hk * p.rep + (w - qi * p.rep);
    }
};

// The prefix set of sequence b, or -1.  Whole warp, one b.
__device__ __forceinline__ int group_of(const PaArgs &p, int b) {
    if (p.pre.n_set <= 0) return -1;
    if (!p.group_start) return p.by_gsize.of(b);
    const int g = warp_search(p.group_start, p.pre.n_set, 1, 0, 0, b);
    int s, e;
    group_range(p, g, s, e);
    return b >= s && b < e ? g : -1;
}
// Partial results that the prefix blocks leave for a sequence of set g.
__device__ __forceinline__ int parts_of(const PaSet &s, int set) { return s.by_chunk.of(clamp_count(s, set) + s.chunk - 1); }
__device__ __forceinline__ int pre_parts_of(const PaArgs &p, int g) {
    return g < 0 ? 0 : parts_of(p.pre, g);
}

// Prefix work of one block: its group, the rows r0 .. of that group's tile, the group's key count (clamped), false
// if the slot is empty.  With group_start, group g's tiles take the slots from start[g] (nq rep) / tile + g on,
// which end before group g + 1's, so no block needs to know the other groups' sizes.  `report`: one block per
// group reports a bad range or count (with group_start the block of slot g, since a group may have no rows).  Whole warps.
__device__ __forceinline__ bool find_tile(const PaArgs &p, int slot, bool report, int &set, int &r0, Rows &rw, int &nk) {
    const int per = p.nq * p.rep, lane = threadIdx.x & 31;
    int s, e, count;
    if (p.group_start && p.pre.n_set <= 32) {
        // a lane a group: bounds and counts arrive together, after one load's latency
        const int g = min(lane, p.pre.n_set - 1);
        const int a = ld_live(p.group_start + g), b = ld_live(p.group_start + g + 1);
        const int c = p.pre.n_keys ? ld_live(p.pre.n_keys + g) : p.pre.max_keys;
        const bool le = lane < p.pre.n_set && ((long long)a * per >> p.tile_shift) + g <= slot;
        set = 31 - __clz(__ballot_sync(0xffffffffu, le) | 1u);
        const bool bad = __any_sync(0xffffffffu, lane == slot && lane < p.pre.n_set &&
                                                     (a < 0 || b < a || b > p.batch || c < 0 || c > p.pre.max_keys));
        if (report && bad && threadIdx.x == 0) set_status(p.ctl, WH_EBOUNDS);
        s = min(max(__shfl_sync(0xffffffffu, a, set), 0), p.batch);
        e = min(max(__shfl_sync(0xffffffffu, b, set), s), p.batch);
        count = __shfl_sync(0xffffffffu, c, set);
    } else {
        if (p.group_start) {
            if (report && slot < p.pre.n_set && threadIdx.x == 0) {
                const int a = ld_live(p.group_start + slot), b = ld_live(p.group_start + slot + 1);
                const int c = p.pre.n_keys ? ld_live(p.pre.n_keys + slot) : 0;
                if (a < 0 || b < a || b > p.batch || c < 0 || c > p.pre.max_keys) set_status(p.ctl, WH_EBOUNDS);
            }
            set = warp_search(p.group_start, p.pre.n_set, per, p.tile_shift, 1, slot);
        } else {
            set = p.by_group_tiles.of(slot);
        }
        count = p.pre.n_keys ? ld_live(p.pre.n_keys + set) : p.pre.max_keys;
        group_range(p, set, s, e);
    }
    r0 = (slot - (p.group_start ? (int)((long long)s * per >> p.tile_shift) + set : set * p.group_tiles)) * p.tile;
    rw.seq0 = s;
    rw.n = (e - s) * per;
    nk = min(max(count, 0), p.pre.max_keys);
    const bool there = r0 >= 0 && r0 < rw.n;
    if (!p.group_start && report && r0 == 0 && count != nk && threadIdx.x == 0) set_status(p.ctl, WH_EBOUNDS);
    return there;
}

// Partial result `part` of row r of a block: dims d0 .. d0 + 7, relative to the maximum mt, with sum lt.
__device__ __forceinline__ void leave_part(const PaArgs &p, const Rows &rw, int r, int part, int d0, float mt, float lt,
                                           const float (&v)[8]) {
    int qrow, head, qi;
    rw.locate(p, r, qrow, head, qi);
    const long long at = ((long long)qrow * p.n_head + head) * p.n_part + part;
    float4 *d = reinterpret_cast<float4 *>(p.part_o + at * 64 + d0);
    d[0] = make_float4(v[0], v[1], v[2], v[3]);
    d[1] = make_float4(v[4], v[5], v[6], v[7]);
    if (d0 == 0) p.part_ml[at] = make_float2(mt, lt);
}

// The finished row, together with the first pre_parts partial results of the row.  Returns the row's maximum
// and 1 / sum.
__device__ __forceinline__ float2 finish_row(const PaArgs &p, const Rows &rw, int r, int d0, float mt, float lt,
                                             float (&v)[8], int pre_parts) {
    int qrow, head, qi;
    rw.locate(p, r, qrow, head, qi);
    const long long row = (long long)qrow * p.n_head + head;
    constexpr int BATCH = 4;   // partial results whose loads are under way together
    for (int i0 = 0; i0 < pre_parts; i0 += BATCH) {
        float2 ml[BATCH];
        float4 x[BATCH], y[BATCH];
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            ml[i] = make_float2(-INFINITY, 0.0f);
            x[i] = y[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (i0 + i < pre_parts) {
                const long long at = row * p.n_part + i0 + i;
                ml[i] = __ldcg(p.part_ml + at);
                x[i] = __ldcg(reinterpret_cast<const float4 *>(p.part_o + at * 64 + d0));
                y[i] = __ldcg(reinterpret_cast<const float4 *>(p.part_o + at * 64 + d0 + 4));
            }
        }
        float mn = mt;
#pragma unroll
        for (int i = 0; i < BATCH; ++i) mn = fmaxf(mn, ml[i].x);
        const float f = mt == -INFINITY ? 0.0f : ex2_approx((mt - mn) * PA_SCALE);
        lt *= f;
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] *= f;
        mt = mn;
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            const float e = ml[i].x == -INFINITY ? 0.0f : ex2_approx((ml[i].x - mt) * PA_SCALE);
            const float u[8] = {x[i].x, x[i].y, x[i].z, x[i].w, y[i].x, y[i].y, y[i].z, y[i].w};
            lt = fmaf(ml[i].y, e, lt);
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = fmaf(u[k], e, v[k]);
        }
    }
    const float2 st = make_float2(mt == -INFINITY ? 0.0f : mt, lt == 0.0f ? 0.0f : 1.0f / lt);   // no key: zeros
    *reinterpret_cast<uint4 *>(p.out + row * 64 + d0) =
        make_uint4(pack_bf16(v[0] * st.y, v[1] * st.y), pack_bf16(v[2] * st.y, v[3] * st.y),
                   pack_bf16(v[4] * st.y, v[5] * st.y), pack_bf16(v[6] * st.y, v[7] * st.y));
    if (p.stats && d0 == 0) p.stats[row] = st;
    return st;
}

// Finishes the rows of a cluster whose blocks hold one key range each: row r's 64 values at `so` (so_row floats
// a row) and its maximum and sum at `sml`, at the same places in every block's shared memory.  Between two
// cluster barriers; the blocks share the rows, each thread takes 8 dims and adds the ranges in order.
template <int THREADS>
__device__ __forceinline__ void finish_cluster(const PaArgs &p, const Rows &rw, int r0, int rows, const void *so, int so_row,
                                               const void *sml, int ranks, int tid) {
    const int rank = (int)cluster_ctarank();
    for (int i = rank * THREADS + tid; i < rows * 8; i += ranks * THREADS) {
        const int r = i >> 3, d0 = 8 * (i & 7);
        const uint8_t *la = static_cast<const uint8_t *>(sml) + r * 8, *oa = static_cast<const uint8_t *>(so) + (r * so_row + d0) * 4;
        float mt = -INFINITY, lt = 0.0f, v[8] = {};
        for (int c = 0; c < ranks; ++c) {
            float m, l;
            const uint32_t ra = mapa_shared(la, c), rb = mapa_shared(oa, c);
            asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(m), "=f"(l) : "r"(ra) : "memory");
            float u[8];
            asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                         : "=f"(u[0]), "=f"(u[1]), "=f"(u[2]), "=f"(u[3])
                         : "r"(rb)
                         : "memory");
            asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                         : "=f"(u[4]), "=f"(u[5]), "=f"(u[6]), "=f"(u[7])
                         : "r"(rb + 16)
                         : "memory");
            const float mn = fmaxf(mt, m);
            const float f = mt == -INFINITY ? 0.0f : ex2_approx((mt - mn) * PA_SCALE), e = m == -INFINITY ? 0.0f : ex2_approx((m - mn) * PA_SCALE);
            lt = lt * f + l * e;
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = v[k] * f + u[k] * e;
            mt = mn;
        }
        finish_row(p, rw, r0 + r, d0, mt, lt, v, 0);
    }
}

// Sequences outside every group have no prefix: the blocks of the first and the last slot finish their rows.
// Whole block.
__device__ __forceinline__ void finish_outside(const PaArgs &p, int slot, int hk) {
    if (!p.group_start || (slot != 0 && slot != p.slots - 1)) return;
    for (int end = 0; end < 2; ++end) {
        if (slot != (end ? p.slots - 1 : 0)) continue;
        Rows rw;
        rw.hk = hk;
        rw.seq0 = end ? min(max(ld_live(p.group_start + p.pre.n_set), 0), p.batch) : 0;
        rw.n = ((end ? p.batch : min(max(ld_live(p.group_start), 0), p.batch)) - rw.seq0) * p.nq * p.rep;
        for (long long i = threadIdx.x; i < 8LL * rw.n; i += blockDim.x) {
            float none[8] = {};
            finish_row(p, rw, (int)(i >> 3), 8 * (int)(i & 7), -INFINITY, 0.0f, none, 0);
        }
    }
}

// prefix_attention_tc.cu: the prefix part on the tcgen05 tensor cores, p.tile = 32, 64 or 128 rows a block.
constexpr int PT_KEYS = 128;   // keys of one step: key ranges are multiples of it
struct PtMaps {
    CUtensorMap k, v;
    int one_set;   // every set is the same one (set_stride 0)
};
int prefix_tc_maps(const PaArgs &a, PtMaps *m);
int prefix_tc_launch(const PaArgs &a, const PtMaps &m, cudaStream_t s);
int prefix_tc_prepare();

}  // namespace wh
