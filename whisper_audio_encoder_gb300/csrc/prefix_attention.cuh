// What the kernels of wh_prefix_attention share: the work's description, how blocks find their group, and
// how a row of a work item names its query.
#pragma once
#include "common.cuh"
#include "internal.h"

namespace wh {

constexpr float PA_SCALE = 0.125f * 1.4426950408889634f;   // log2(e) / sqrt(64): scores in the exp2 domain

struct PaSet {
    const __nv_bfloat16 *k, *v;
    long long row_stride, set_stride;   // elements
    const int *n_keys;                  // device [n_set] or null (max_keys for all)
    float *weight;                      // device [n_set][n_kv][max_keys] or null
    int n_set, max_keys;
    int splits, chunk;                  // key ranges of one set and keys of a range
};

struct PaArgs {
    PaSet pre, own;
    const __nv_bfloat16 *q;
    long long q_stride;
    const int *group_start;   // device [pre.n_set + 1] or null: gsize sequences each
    int gsize, batch, nq, n_head, n_kv, rep;
    int tile;                 // prefix: rows of a row tile
    int slots;                // prefix: row-tile slots of a key head over all groups
    int own_tiles;            // row tiles of a sequence
    int own_wpi;              // own keys: warps of a work item
    long long own_items;      // own keys: (sequence, range, key head, row tile)
    long long pre_blocks;     // blocks [0, pre_blocks) take prefix work, the rest own keys
    float *part_o;            // [row][pre.splits + own.splits][64], row = (b nq + i) n_head + h
    float2 *part_ml;          // [row][pre.splits + own.splits]: running maximum and sum
    float2 *stats;            // [row]: maximum and 1 / sum (weights only)
    __nv_bfloat16 *out;       // [batch * nq][64 n_head]
    int direct;               // one range covers everything a row sees: write out, no merge
    int beside_tc;            // k_prefix_attention runs beside k_prefix_tc: it waits for it at its end
    DevCtl ctl;
};

__device__ __forceinline__ int clamp_count(const PaSet &s, int set) {
    return s.n_keys ? min(max(__ldg(s.n_keys + set), 0), s.max_keys) : s.max_keys;
}

// Largest g in [0, n) with start[g] * mul / div + g * add <= x, by the whole warp, 32 probes at a time.
__device__ __forceinline__ int warp_search(const int *start, int n, int mul, int div, int add, long long x) {
    int lo = 0, len = n;
    const int lane = threadIdx.x & 31;
    while (len > 1) {
        const int step = (len + 31) / 32, i = lane * step;
        bool le = false;
        if (i < len) {
            const int g = lo + i;
            le = (long long)__ldg(start + g) * mul / div + (long long)g * add <= x;
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
        s = min(max(__ldg(p.group_start + g), 0), p.batch);
        e = min(max(__ldg(p.group_start + g + 1), s), p.batch);
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
        const int per = p.nq * p.rep, s = r / per, w = r - s * per;
        qi = w / p.rep;
        qrow = (seq0 + s) * p.nq + qi;
        head = hk * p.rep + (w - qi * p.rep);
    }
};

// Prefix work of one block: its group, the rows r0 .. of that group's tile, false if the slot is empty.  With
// group_start, group g's tiles take the slots from start[g] (nq rep) / tile + g on, which end before group
// g + 1's, so no block needs to know the other groups' sizes.  One block per group reports a bad range.
__device__ __forceinline__ bool find_tile(const PaArgs &p, int slot, bool report, int &set, int &r0, Rows &rw) {
    const int per = p.nq * p.rep;
    int s, e;
    if (p.group_start) {
        if (report && slot < p.pre.n_set && threadIdx.x == 0) {
            const int a = __ldg(p.group_start + slot), b = __ldg(p.group_start + slot + 1);
            if (a < 0 || b < a || b > p.batch) set_status(p.ctl, WH_EBOUNDS);
        }
        set = warp_search(p.group_start, p.pre.n_set, per, p.tile, 1, slot);
        group_range(p, set, s, e);
        r0 = (slot - (int)((long long)s * per / p.tile) - set) * p.tile;
    } else {
        const int tiles = (p.gsize * per + p.tile - 1) / p.tile;
        set = slot / tiles;
        group_range(p, set, s, e);
        r0 = (slot - set * tiles) * p.tile;
    }
    rw.seq0 = s;
    rw.n = (e - s) * per;
    return r0 >= 0 && r0 < rw.n;
}

// Dims d0 .. d0 + 7 of row r of a block's result (v relative to the maximum mt, with sum lt): the output
// itself, or partial result number `part` for the merge.
__device__ __forceinline__ void finish_row(const PaArgs &p, const Rows &rw, int r, int part, int d0, float mt, float lt,
                                           const float (&v)[8]) {
    int qrow, head, qi;
    rw.locate(p, r, qrow, head, qi);
    const long long row = (long long)qrow * p.n_head + head;
    if (p.direct) {
        const float inv = lt == 0.0f ? 0.0f : 1.0f / lt;   // a query that sees no key: zeros
        *reinterpret_cast<uint4 *>(p.out + row * 64 + d0) =
            make_uint4(pack_bf16(v[0] * inv, v[1] * inv), pack_bf16(v[2] * inv, v[3] * inv),
                       pack_bf16(v[4] * inv, v[5] * inv), pack_bf16(v[6] * inv, v[7] * inv));
        if (p.stats && d0 == 0) p.stats[row] = make_float2(mt == -INFINITY ? 0.0f : mt, inv);
    } else {
        const long long at = row * (p.pre.splits + p.own.splits) + part;
        float4 *d = reinterpret_cast<float4 *>(p.part_o + at * 64 + d0);
        d[0] = make_float4(v[0], v[1], v[2], v[3]);
        d[1] = make_float4(v[4], v[5], v[6], v[7]);
        if (d0 == 0) p.part_ml[at] = make_float2(mt, lt);
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
