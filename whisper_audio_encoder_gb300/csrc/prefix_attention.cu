// Attention of a batch whose sequences share long prefixes, and the weight every key receives.
//
// Sequence b of group g has n_query queries a head.  Query i attends over the group's prefix keys
// 0 .. n_g - 1 and over the sequence's own keys 0 .. n_b - (n_query - i), i.e. no key behind its own:
//   s_t = q . k_t / 8,   p = softmax(s),   o = sum_t p_t v_t,   weight[t] += sum over the queries of p_t
// A prefix key and value are read once for all the queries of the group (all sequences, queries and
// query heads of its key head are the rows of one matrix product), not once per sequence.
//
// k_prefix_attention  16 rows a block: prefixes of few rows, and every sequence's own keys; below
// k_prefix_tc         32, 64 or 128 rows a block on tcgen05 (prefix_attention_tc.cu): prefixes of many rows
// k_prefix_merge      joins key ranges where no cluster or own block does
// k_prefix_weight     the keys' weights, where the scores were not kept
// Floors: 256 bytes a key and head once, 4 * 64 flops a (query, key) pair.  The device's copy rate is 6.8 TB/s,
// but one cold read of 153 MB by TMA, with no arithmetic, takes 26 us (5.9 TB/s): short passes pay for the start.
#include "prefix_attention.cuh"

namespace wh {
namespace {

constexpr int PA_WARPS = 4;
constexpr int PA_THREADS = 32 * PA_WARPS;
constexpr int PA_TILE = 16;        // rows of a block
constexpr int PA_KEYS = 32;        // keys of one warp step
constexpr int PA_SLOT_KEYS = 16;   // of one slot of a warp's ring
constexpr int PA_SLOT = 2 * PA_SLOT_KEYS * 128;   // bytes: keys, then values
constexpr int PA_RING = 4 * PA_SLOT;
constexpr int PA_SMEM = PA_WARPS * PA_RING;
constexpr int SO_ROW = 68;         // floats a row of the warps' staged results
constexpr int PM_BATCH = 8;        // partial results that a merging thread loads at once
constexpr int PM_TEAMS = 8;        // teams of 16 threads in a merging block
constexpr int PW_WARPS = 4;        // weight kernel: warps of a block
constexpr int PW_KEYS = 32;        // weight kernel: keys of one warp step
constexpr int PW_BLOCKS = 8 * 152; // weight kernel: blocks, twice what is resident (four an SM: 35.4 us, eight: 33.6)

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Four 8 x 8 matrices of bf16 from shared memory, transposed: lane l gives the address of row l % 8 of matrix
// l / 8 and gets elements (2c, g) and (2c + 1, g) of each.
__device__ __forceinline__ void ldmatrix_trans(uint32_t a, uint32_t &r0, uint32_t &r1, uint32_t &r2, uint32_t &r3) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
                 : "r"(a)
                 : "memory");
}

// 16 bytes global -> shared, the last 16 - bytes of them zeros.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
}

// Query fragments of rows r0 + g and r0 + g + 8 (g = lane / 4).  The 64 dims of a head are spread over the
// four lanes of a row as 8c .. 8c+7 and 32+8c .. 32+8c+7 (c = lane % 4), so that a lane's 16-byte loads of a
// key are its part of four MMA steps; the sum over dims does not mind the order.
__device__ __forceinline__ void load_q(const PaArgs &p, const Rows &rw, int r0, uint32_t (&a)[4][4]) {
    const int g = (threadIdx.x & 31) >> 2, c = threadIdx.x & 3;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        const int r = r0 + g + 8 * half;
        uint4 u0 = make_uint4(0, 0, 0, 0), u1 = u0;
        if (r < rw.n) {
            int qrow, head, qi;
            rw.locate(p, r, qrow, head, qi);
            const uint4 *s = reinterpret_cast<const uint4 *>(p.q + (long long)qrow * p.q_stride + head * 64) + c;
            u0 = ld_live(s);
            u1 = ld_live(s + 4);
        }
        a[0][half] = u0.x, a[0][half + 2] = u0.y, a[1][half] = u0.z, a[1][half + 2] = u0.w;
        a[2][half] = u1.x, a[2][half + 2] = u1.y, a[3][half] = u1.z, a[3][half + 2] = u1.w;
    }
}

__device__ __forceinline__ float min_nan(float a, float b) {
    float d;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}
// Scores of 16 rows x 8 keys: lane (g, c) gives keys 2c, 2c+1 of rows g (0, 1) and g + 8 (2, 3).
__device__ __forceinline__ void score8(const uint32_t (&a)[4][4], const uint4 &k0, const uint4 &k1, float (&s)[4]) {
    s[0] = s[1] = s[2] = s[3] = 0.0f;
    mma_bf16(s, a[0][0], a[0][1], a[0][2], a[0][3], k0.x, k0.y);
    mma_bf16(s, a[1][0], a[1][1], a[1][2], a[1][3], k0.z, k0.w);
    mma_bf16(s, a[2][0], a[2][1], a[2][2], a[2][3], k1.x, k1.y);
    mma_bf16(s, a[3][0], a[3][1], a[3][2], a[3][3], k1.z, k1.w);
}

// OWN = false: the prefixes; true: the sequences' own keys.
// One pass over the keys with a running maximum and sum per row.  Bound by HBM: a warp keeps 4 to 8 KB of keys
// and values in flight by cp.async (96 KB an SM with three blocks of four warps), and the products run on
// mma.sync because 16 rows would leave 7/8 of a tcgen05 tile empty, while 606 TFLOP/s of mma.sync are four times
// what 16 rows need at the full HBM rate.  Steps of 32 keys: the maximum's shuffles and the rescaling vote are
// paid once for two products.  16 prefixes x 5 rows x 20 heads x 1500 keys: 23 us, 123 MB, 5.3 TB/s, 79 % of
// the copy rate; 256 sequences' 448 own keys x 20 heads: 87 us a call, 587 MB, 99 %.
template <bool OWN>
__global__ void __launch_bounds__(PA_THREADS, 3) k_prefix_attention(const PaArgs p) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    // What runs after this kernel's trigger may count on its inputs (the prefix blocks waited for them).
    if (!OWN || !p.after_pre) pdl_wait();
    pdl_launch_dependents();
    // ---- which rows, which keys ----
    // A work item is done by `wpi` neighbouring warps: all four for a prefix, p.own_wpi for own keys.
    const PaSet &ks = OWN ? p.own : p.pre;
    const int cluster = OWN ? p.own_cluster : p.pre_cluster;
    const int wpi = OWN ? p.own_wpi : PA_WARPS, iw = warp & (wpi - 1), wlog = 31 - __clz(wpi), team = OWN ? warp >> wlog : 0;
    Rows rw;
    int set, split, r0, nk;
    if (OWN) {
        int x = blockIdx.x * (PA_WARPS >> wlog) + team;
        if (x >= p.own_items) {
            pdl_wait();   // on every path: the kernel after this one counts on the one before it too
            return;
        }
        split = remainder(ks.by_splits, ks.splits, x);
        const int tile = remainder(p.by_own_tiles, p.own_tiles, x);
        rw.hk = remainder(p.by_kv, p.n_kv, x);
        set = x;
        rw.seq0 = set;
        rw.n = p.nq * p.rep;
        r0 = tile * PA_TILE;
        const int count = ks.n_keys ? ld_live(ks.n_keys + set) : ks.max_keys;
        nk = min(max(count, 0), ks.max_keys);
        if (count != nk && rw.hk == 0 && split == 0 && r0 == 0 && iw == 0 && lane == 0) set_status(p.ctl, WH_EBOUNDS);
    } else {
        int x = blockIdx.x;
        split = remainder(ks.by_splits, ks.splits, x);
        const int slot = remainder(p.by_slots, p.slots, x);
        rw.hk = x;
        if (cluster && split == 0) finish_outside(p, slot, rw.hk);
        if (!find_tile(p, slot, rw.hk == 0 && split == 0, set, r0, rw, nk)) return;
    }
    const int k0 = split * ks.chunk, k1 = min(nk, k0 + ks.chunk);
    if (k0 >= k1 && !cluster) {   // nothing here: the merge knows
        if (OWN) pdl_wait();
        return;
    }
    // Each warp copies its keys and values into a ring of its own, 16 at a time: four rows of 128 bytes an
    // instruction, zeros past the range.  The 16-byte pieces of a row are permuted (keys: by the row's lowest
    // bit, values: by the lowest three) so that the fragment reads below meet no bank twice.  A step takes two
    // slots of the four while the next two are on their way.
    extern __shared__ __align__(128) uint8_t ring_all[];
    const uint32_t ring = smem_u32(ring_all) + warp * PA_RING;
    const int crow = lane >> 3, piece = lane & 7;
    const __nv_bfloat16 *kb = ks.k + (long long)set * ks.set_stride + rw.hk * 64 + 8 * piece;
    const __nv_bfloat16 *vb = ks.v + (long long)set * ks.set_stride + rw.hk * 64 + 8 * piece;
    const long long step4 = 4 * ks.row_stride;   // four rows on
    const uint32_t ck = ring + crow * 128 + ((piece ^ ((crow & 1) << 2)) << 4);
    const uint32_t cv = ring + PA_SLOT_KEYS * 128 + crow * 128 + ((piece ^ crow) << 4);
    auto fetch = [&](int t, int slot) {   // keys t .. t + 15
        if (t >= k1) return;
        const uint32_t dk = ck + slot * PA_SLOT, dv = cv + slot * PA_SLOT;
        const long long at = (long long)(t + crow) * ks.row_stride;
        const __nv_bfloat16 *k = kb + at, *v = vb + at;
        if (t + PA_SLOT_KEYS <= k1) {
#pragma unroll
            for (int i = 0; i < 4; ++i, k += step4, v += step4) {
                cp_async16(dk + i * 512, k, 16u);
                cp_async16((dv + i * 512) ^ ((i & 1) << 6), v, 16u);   // rows 4i + crow: the third bit is i's lowest
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i, k += step4, v += step4) {
                const bool in = t + 4 * i + crow < k1;
                cp_async16(dk + i * 512, in ? k : kb, in ? 16u : 0u);
                cp_async16((dv + i * 512) ^ ((i & 1) << 6), in ? v : vb, in ? 16u : 0u);
            }
        }
    };
    float *scores = reinterpret_cast<float *>(ring_all + PA_SMEM) + team * p.score_floats;
    const int stride = wpi * PA_KEYS;
    int t0 = k0 + iw * PA_KEYS, half_ring = 0;
    fetch(t0, 0);
    fetch(t0 + PA_SLOT_KEYS, 1);
    cp_async_commit();

    uint32_t qa[4][4];
    int lim[2];   // own keys: the first key that a row does not see
    load_q(p, rw, r0, qa);
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        lim[half] = nk;
        if (OWN) {
            int qrow, head, qi;
            rw.locate(p, min(r0 + g + 8 * half, rw.n - 1), qrow, head, qi);
            lim[half] = nk - (p.nq - 1 - qi);
        }
    }
    const int before = OWN && cluster && p.after_pre ? pre_parts_of(p, group_of(p, set)) : 0;   // partial results
    const int full = OWN ? nk - (p.nq - 1) : nk;   // every row sees the keys before this one

    float m[2] = {-INFINITY, -INFINITY}, l[2] = {}, o[8][4] = {};
    for (; t0 < k1; t0 += stride) {
        fetch(t0 + stride, 2 - half_ring);
        fetch(t0 + stride + PA_SLOT_KEYS, 3 - half_ring);
        cp_async_commit();
        cp_async_wait<1>();
        __syncwarp();   // every lane's copies of this step have landed
        const uint32_t base = ring + half_ring * PA_SLOT;
        const int slots = t0 + PA_SLOT_KEYS < k1 ? 2 : 1;   // the second may hold nothing at all
        // scores of keys 8j + 2c, 8j + 2c + 1 for rows g (0, 1) and g + 8 (2, 3)
        float s[4][4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (j < 2 * slots) {
                const uint32_t kk = base + (j >> 1) * PA_SLOT + (8 * (j & 1) + g) * 128;
                const uint4 x = lds128(kk + ((c ^ ((g & 1) << 2)) << 4)), y = lds128(kk + (((c + 4) ^ ((g & 1) << 2)) << 4));
                score8(qa, x, y, s[j]);
            } else {
                s[j][0] = s[j][1] = s[j][2] = s[j][3] = -INFINITY;
            }
        }
        if (t0 + PA_KEYS > min(k1, full)) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (t0 + 8 * j + 2 * c + (i & 1) >= min(k1, lim[i >> 1])) s[j][i] = -INFINITY;
        }
        if (OWN && p.score_floats) {   // for the weights, once the row's sum is known
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int half = 0; half < 2; ++half)
                    if (g + 8 * half < rw.n)
                        *reinterpret_cast<float2 *>(scores + (g + 8 * half) * ks.chunk + t0 - k0 + 8 * j + 2 * c) =
                            make_float2(s[j][2 * half], s[j][2 * half + 1]);
        }
        float mn[2];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int i = 2 * half;
            float mx = fmaxf(fmaxf(fmaxf(s[0][i], s[0][i + 1]), fmaxf(s[1][i], s[1][i + 1])),
                             fmaxf(fmaxf(s[2][i], s[2][i + 1]), fmaxf(s[3][i], s[3][i + 1])));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            mn[half] = fmaxf(m[half], mx);
        }
        if (__any_sync(0xffffffffu, mn[0] > m[0] || mn[1] > m[1])) {   // some row's maximum moved
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const float f = m[half] == -INFINITY ? 0.0f : ex2_approx((m[half] - mn[half]) * PA_SCALE);
                l[half] *= f;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    o[j][2 * half] *= f;
                    o[j][2 * half + 1] *= f;
                }
                m[half] = mn[half];
            }
        }
        const float ms[2] = {m[0] == -INFINITY ? 0.0f : m[0], m[1] == -INFINITY ? 0.0f : m[1]};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (h == 1 && slots == 1) break;
            // the weights as a sum of two bf16 each: 16 bits of mantissa in two products of 8
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) {   // rows g, g + 8 of keys 2c, 2c + 1, then of keys 8 + 2c, 9 + 2c
                const float *sx = s[2 * h + (x >> 1)] + 2 * (x & 1);
                const float e0 = ex2_approx((sx[0] - ms[x & 1]) * PA_SCALE);
                const float e1 = ex2_approx((sx[1] - ms[x & 1]) * PA_SCALE);
                l[x & 1] += e0 + e1;
                hi[x] = pack_bf16(e0, e1);
                lo[x] = pack_bf16(e0 - __uint_as_float(hi[x] << 16), e1 - __uint_as_float(hi[x] & 0xffff0000u));
            }
            const uint32_t vrow = base + h * PA_SLOT + PA_SLOT_KEYS * 128 + (lane & 15) * 128;
#pragma unroll
            for (int w = 0; w < 4; ++w) {   // dims 16w .. 16w + 15
                uint32_t b0, b1, b2, b3;
                ldmatrix_trans(vrow + (((2 * w + (lane >> 4)) ^ (lane & 7)) << 4), b0, b1, b2, b3);
                mma_bf16(o[2 * w], hi[0], hi[1], hi[2], hi[3], b0, b1);
                mma_bf16(o[2 * w + 1], hi[0], hi[1], hi[2], hi[3], b2, b3);
                mma_bf16(o[2 * w], lo[0], lo[1], lo[2], lo[3], b0, b1);
                mma_bf16(o[2 * w + 1], lo[0], lo[1], lo[2], lo[3], b2, b3);
            }
        }
        half_ring = 2 - half_ring;
        __syncwarp();   // every lane is done with the slots before they are filled again
    }

    // ---- merge the item's warps ----
    // (each writes over its own ring; no copy is in flight, the last groups were empty)
    __shared__ float2 sml[PA_WARPS][PA_TILE];
    auto so = [&](int w, int r) { return reinterpret_cast<float *>(ring_all + w * PA_RING) + r * SO_ROW; };
    static_assert(sizeof(float) * PA_TILE * SO_ROW <= PA_RING, "a warp's rows fit in its ring");
    __syncwarp();
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        float ls = l[half];
        ls += __shfl_xor_sync(0xffffffffu, ls, 1);
        ls += __shfl_xor_sync(0xffffffffu, ls, 2);
        const int r = g + 8 * half;
        if (r0 + r >= rw.n) continue;
        if (c == 0) sml[warp][r] = make_float2(m[half], ls);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            *reinterpret_cast<float2 *>(so(warp, r) + 8 * j + 2 * c) = make_float2(o[j][2 * half], o[j][2 * half + 1]);
    }
    auto item_bar = [&] { asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "r"(32 * wpi) : "memory"); };
    item_bar();
    if (OWN && p.after_pre) pdl_wait();   // the prefix's partial results are complete
    __shared__ float2 fin[PA_WARPS][PA_TILE];   // the block's maximum and sum; own weights: the row's maximum, 1 / sum
    const int w0 = warp - iw, rows = min(PA_TILE, rw.n - r0);
    for (int i = 32 * iw + lane; i < 8 * rows; i += 32 * wpi) {
        const int r = i >> 3, d0 = 8 * (i & 7);
        float mt = -INFINITY;
        for (int w = 0; w < wpi; ++w) mt = fmaxf(mt, sml[w0 + w][r].x);
        float lt = 0.0f, v[8] = {};
        for (int w = 0; w < wpi; ++w) {
            const float2 ml = sml[w0 + w][r];
            const float f = ml.x == -INFINITY ? 0.0f : ex2_approx((ml.x - mt) * PA_SCALE);
            lt = fmaf(ml.y, f, lt);
            const float4 x = *reinterpret_cast<const float4 *>(so(w0 + w, r) + d0);
            const float4 y = *reinterpret_cast<const float4 *>(so(w0 + w, r) + d0 + 4);
            v[0] = fmaf(x.x, f, v[0]), v[1] = fmaf(x.y, f, v[1]), v[2] = fmaf(x.z, f, v[2]), v[3] = fmaf(x.w, f, v[3]);
            v[4] = fmaf(y.x, f, v[4]), v[5] = fmaf(y.y, f, v[5]), v[6] = fmaf(y.z, f, v[6]), v[7] = fmaf(y.w, f, v[7]);
        }
        if (cluster == 0) {
            leave_part(p, rw, r0 + r, OWN ? p.pre.splits + split : split, d0, mt, lt, v);
        } else if (cluster == 1) {
            const float2 st = finish_row(p, rw, r0 + r, d0, mt, lt, v, before);
            if (d0 == 0) fin[w0][r] = st;
        } else {
            float *d = so(w0, r) + d0;   // (only this thread reads or writes these dims)
            *reinterpret_cast<float4 *>(d) = make_float4(v[0], v[1], v[2], v[3]);
            *reinterpret_cast<float4 *>(d + 4) = make_float4(v[4], v[5], v[6], v[7]);
            if (d0 == 0) fin[w0][r] = make_float2(mt, lt);
        }
    }
    if (cluster > 1) {   // whole blocks: wpi = 4
        __syncwarp();
        cluster_sync();
        finish_cluster<PA_THREADS>(p, rw, r0, rows, so(0, 0), SO_ROW, fin[0], cluster, threadIdx.x);
        __syncwarp();
        cluster_sync();   // no block leaves while another may still read its rows
    }
    if (OWN && p.score_floats) {
        item_bar();
        float *w = ks.weight + ((long long)set * p.n_kv + rw.hk) * ks.max_keys;
        constexpr int U = 4;   // keys of a thread at a time: their accumulators are read together
        for (int t = 32 * iw + lane; t < k1; t += U * 32 * wpi) {
            float before[U], add[U] = {};   // (the rows' sum first: the accumulator is rounded once, not by every row)
#pragma unroll
            for (int u = 0; u < U; ++u) before[u] = t + u * 32 * wpi < k1 ? __ldcg(w + t + u * 32 * wpi) : 0.0f;
            for (int r = 0; r < rows; ++r) {
                const float2 st = fin[w0][r];
                const float *sr = scores + r * ks.chunk + t;
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (t + u * 32 * wpi < k1) add[u] = fmaf(ex2_approx((sr[u * 32 * wpi] - st.x) * PA_SCALE), st.y, add[u]);
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (t + u * 32 * wpi < k1) w[t + u * 32 * wpi] = before[u] + add[u];
        }
    }
}

// o = sum_s 2^(m_s - m) o_s / sum_s 2^(m_s - m) l_s over the ranges of a row that hold keys.  16 threads hold a
// row's dims; TEAMS such teams share a row's ranges (team k takes ranges k PM_BATCH .. and so on, PM_BATCH at a
// time, all of their loads before any arithmetic) and are joined in order at the end.
template <int TEAMS>
__global__ void __launch_bounds__(16 * PM_TEAMS) k_prefix_merge(const PaArgs p) {
    constexpr int ROWS = PM_TEAMS / TEAMS;
    pdl_launch_dependents();
    const long long rows = (long long)p.batch * p.nq * p.n_head;
    const int lane = threadIdx.x & 15, in_block = (threadIdx.x >> 4) % ROWS, team = (threadIdx.x >> 4) / ROWS;
    const long long mine = (long long)blockIdx.x * ROWS + in_block, row = min(mine, rows - 1);
    const int b = p.by_seq.of((int)row);
    // (the two teams of a warp may have rows of different sequences: one after the other)
    const int b0 = __shfl_sync(0xffffffffu, b, 0), b1 = __shfl_sync(0xffffffffu, b, 16);
    const int np0 = pre_parts_of(p, group_of(p, b0)), np1 = b1 == b0 ? np0 : pre_parts_of(p, group_of(p, b1));
    const int np = (threadIdx.x & 16) ? np1 : np0;
    const int n = np + (p.own.n_set > 0 ? parts_of(p.own, b) : 0);
    const float2 *ml = p.part_ml + row * p.n_part;
    const float4 *po = reinterpret_cast<const float4 *>(p.part_o + row * p.n_part * 64) + lane;
    pdl_wait();   // the partial results; what came before only reads the call's inputs
    float m = -INFINITY, l = 0.0f;
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    auto add = [&](const float2 *x, const float4 *v, int count) {
        float mn = m;
#pragma unroll
        for (int i = 0; i < PM_BATCH; ++i)
            if (i < count) mn = fmaxf(mn, x[i].x);
        const float f = m == -INFINITY ? 0.0f : ex2_approx((m - mn) * PA_SCALE);
        l *= f, o.x *= f, o.y *= f, o.z *= f, o.w *= f;
        m = mn;
#pragma unroll
        for (int i = 0; i < PM_BATCH; ++i) {
            if (i >= count) continue;
            const float e = x[i].x == -INFINITY ? 0.0f : ex2_approx((x[i].x - m) * PA_SCALE);
            l = fmaf(x[i].y, e, l);
            o.x = fmaf(v[i].x, e, o.x), o.y = fmaf(v[i].y, e, o.y), o.z = fmaf(v[i].z, e, o.z), o.w = fmaf(v[i].w, e, o.w);
        }
    };
    float2 x[PM_BATCH];
    float4 v[PM_BATCH];
    for (int i0 = team * PM_BATCH; i0 < n; i0 += TEAMS * PM_BATCH) {
#pragma unroll
        for (int i = 0; i < PM_BATCH; ++i) {
            x[i] = make_float2(-INFINITY, 0.0f);
            v[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (i0 + i < n) {
                const int s = i0 + i < np ? i0 + i : p.pre.splits + i0 + i - np;
                x[i] = __ldcg(ml + s);
                v[i] = __ldcg(po + s * 16);
            }
        }
        add(x, v, PM_BATCH);
    }
    if (TEAMS > 1) {
        __shared__ float4 so[PM_TEAMS][16];
        __shared__ float2 sml[PM_TEAMS];
        so[threadIdx.x >> 4][lane] = o;
        if (lane == 0) sml[threadIdx.x >> 4] = make_float2(m, l);
        __syncthreads();
        if (team > 0) return;
        for (int k = 1; k < TEAMS; ++k) {
            x[0] = sml[k * ROWS + in_block];
            v[0] = so[k * ROWS + in_block][lane];
            add(x, v, 1);
        }
    }
    if (mine >= rows) return;
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    *reinterpret_cast<uint2 *>(p.out + row * 64 + 4 * lane) =
        make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
    if (p.stats && lane == 0) p.stats[row] = make_float2(m == -INFINITY ? 0.0f : m, inv);
}

// weight[t] += sum over the set's queries of 2^(s_t - m) / l: the scores again, with every row's final
// maximum and sum.  A warp takes 32 keys at a time from a ring of two such steps and goes through the rows
// 16 at a time, the next 16 on their way meanwhile; each sum has one fixed order.  Bound by the keys' bytes for few
// rows, by instructions for many (packed pairs; 102 rows x 4874 keys x 40 heads: 47 us with the attention, 66 with
// single values and rows fetched when needed).  Reading the keys again costs half of what the attention reads; keeping
// the scores would cost 8 bytes a (row, key) pair.  16 prefixes of 211 .. 1500 keys, 83 rows, 20 heads: 6 us behind
// the attention for 34 MB of keys, most of them still in L2.
template <bool OWN>
__global__ void __launch_bounds__(32 * PW_WARPS, 4) k_prefix_weight(const PaArgs p) {
    __shared__ __align__(128) uint8_t rings[PW_WARPS][2 * PW_KEYS * 128];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    const PaSet &ks = OWN ? p.own : p.pre;
    Rows rw;
    rw.hk = blockIdx.y;
    const int set = blockIdx.z;
    const int nk = clamp_count(ks, set), stride = gridDim.x * PW_WARPS * PW_KEYS;
    int t0 = (blockIdx.x * PW_WARPS + warp) * PW_KEYS;
    if (t0 >= nk) {
        pdl_wait();   // on every path: a kernel after this one counts on what came before too
        return;
    }
    int s0 = set, e0 = set + 1;
    if (!OWN) group_range(p, set, s0, e0);
    rw.seq0 = s0;
    rw.n = (e0 - s0) * p.nq * p.rep;
    const int crow = lane >> 3, piece = lane & 7;
    const uint32_t ring = smem_u32(rings[warp]);
    const __nv_bfloat16 *kb = ks.k + (long long)set * ks.set_stride + rw.hk * 64 + 8 * piece;
    auto fetch = [&](int t, int slot) {   // keys t .. t + 31, permuted as in k_prefix_attention
        if (t < nk) {
            const uint32_t dst = ring + slot * PW_KEYS * 128 + crow * 128 + ((piece ^ ((crow & 1) << 2)) << 4);
#pragma unroll
            for (int i = 0; i < PW_KEYS / 4; ++i) {
                const bool in = t + 4 * i + crow < nk;
                cp_async16(dst + i * 512, in ? kb + (long long)(t + 4 * i + crow) * ks.row_stride : kb, in ? 16u : 0u);
            }
        }
        cp_async_commit();
    };
    fetch(t0, 0);
    pdl_wait();
    struct Queries {   // of rows r0 + g, r0 + g + 8
        uint32_t a[4][4];
        float2 st[2];   // their maximum and 1 / sum; rows past the last: zeros, and their scores are zero
        int lim[2];     // own keys: the first key that the row does not see
    };
    auto load_rows = [&](int r0, Queries &x) {
        load_q(p, rw, r0, x.a);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            x.st[half] = make_float2(0.0f, 0.0f);
            x.lim[half] = 0;
            if (r0 + g + 8 * half < rw.n) {
                int qrow, head, qi;
                rw.locate(p, r0 + g + 8 * half, qrow, head, qi);
                x.st[half] = __ldcg(p.stats + (long long)qrow * p.n_head + head);
                x.lim[half] = nk - (p.nq - 1 - qi);
            }
        }
    };
    Queries now;
    load_rows(0, now);
    // the key whose sum this lane ends up with
    const int mine = ((lane & 16) ? 16 : 0) + ((lane & 8) ? 8 : 0) + 2 * c + ((lane & 4) ? 1 : 0);
    float *w = ks.weight + ((long long)set * p.n_kv + rw.hk) * ks.max_keys + mine;
    for (int slot = 0; t0 < nk; t0 += stride, slot ^= 1) {
        fetch(t0 + stride, slot ^ 1);
        const float before = t0 + mine < nk ? __ldcg(w + t0) : 0.0f;
        cp_async_wait<1>();
        __syncwarp();
        uint4 kr[4][2];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t kk = ring + slot * PW_KEYS * 128 + (8 * j + g) * 128;
            kr[j][0] = lds128(kk + ((c ^ ((g & 1) << 2)) << 4));
            kr[j][1] = lds128(kk + (((c + 4) ^ ((g & 1) << 2)) << 4));
        }
        __syncwarp();
        uint64_t sum2[4] = {};   // of keys 8j + 2c, 8j + 2c + 1
        for (int r0 = 0; r0 < rw.n; r0 += 16) {
            Queries next;   // on their way while these are worked on (after the last the first: the next step's)
            if (rw.n > 16) load_rows(r0 + 16 < rw.n ? r0 + 16 : 0, next);
            float s[4][4];
#pragma unroll
            for (int j = 0; j < 4; ++j) score8(now.a, kr[j][0], kr[j][1], s[j]);
            const uint64_t scale = f2_pack(PA_SCALE, PA_SCALE);
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const uint64_t less = f2_pack(-now.st[half].x, -now.st[half].x), inv = f2_pack(now.st[half].y, now.st[half].y);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float e0, e1;
                    f2_unpack(mul_f2(add_f2(f2_pack(s[j][2 * half], s[j][2 * half + 1]), less), scale), e0, e1);
                    f2_unpack(mul_f2(f2_pack(ex2_approx(e0), ex2_approx(e1)), inv), e0, e1);
                    // (no weight is above 1: where scores are so large that another kernel's rounding of the same
                    // score is far off this one's, the difference must not run away; NaN stays NaN)
                    e0 = min_nan(e0, 1.0f), e1 = min_nan(e1, 1.0f);
                    if (OWN) {
                        const int key = t0 + 8 * j + 2 * c;
                        e0 = key < now.lim[half] ? e0 : 0.0f;
                        e1 = key + 1 < now.lim[half] ? e1 : 0.0f;
                    }
                    sum2[j] = add_f2(sum2[j], f2_pack(e0, e1));
                }
            }
            if (rw.n > 16) now = next;
        }
        float acc[4][2];
#pragma unroll
        for (int j = 0; j < 4; ++j) f2_unpack(sum2[j], acc[j][0], acc[j][1]);
        // the eight row lanes' sums, each lane keeping half of its keys at every exchange
        float x[2][2], y[2];
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const bool up = lane & 16;
                x[j][i] = (up ? acc[2 + j][i] : acc[j][i]) + __shfl_xor_sync(0xffffffffu, up ? acc[j][i] : acc[2 + j][i], 16);
            }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const bool up = lane & 8;
            y[i] = (up ? x[1][i] : x[0][i]) + __shfl_xor_sync(0xffffffffu, up ? x[0][i] : x[1][i], 8);
        }
        const bool up = lane & 4;
        const float sum = (up ? y[1] : y[0]) + __shfl_xor_sync(0xffffffffu, up ? y[0] : y[1], 4);
        if (t0 + mine < nk) w[t0] = before + sum;
    }
}

constexpr long long PA_BLOCKS = 3 * 152;   // k_prefix_attention: 3 blocks on each of GB300's 152 SMs
constexpr long long PT_BLOCKS = 2 * 152;   // k_prefix_tc: 2 on each
// The prefix part goes to k_prefix_tc when its sets have more than PT_MIN_ROWS rows on average and there are at
// least PT_MIN_WORK products of a 16-row tile with a key (k_prefix_attention's units) to do: below that its
// blocks' longer set-up (TMEM, tensor maps) does not pay.  Measured, us a replayed call, 20 key heads:
//   rows x keys x sets   products   k_prefix_attention   k_prefix_tc
//    40 x  400 x  1         24 k           9.4              12.2
//   128 x 1500 x  1        240 k          16.4              19.0
//    40 x 1500 x  4        360 k          18.4              18.5
//    64 x 1500 x  4        480 k          20.6              18.5
//    40 x 8000 x  1        480 k          22.6              21.0
//   128 x 1500 x 16        3.8 M          94                49
// Beside own keys, whose blocks hide the set-up, more than twice PT_MIN_ROWS rows are taken: 200 rows x 400 keys, 8
// heads, with up to 224 own keys 20.5 and 18.5; 64 rows x 1200 keys, 20 heads 20.4 and 16.5; 40 rows x 400 keys, 8 heads
// 10.2 and 14.3, the same for the host, whose two launches take longer.
constexpr int PT_MIN_ROWS = 16;
constexpr long long PT_MIN_WORK = 300000;
// Ranges of at least PT_LEAST keys (rounded down): a shorter block does not make up for joining one range more.
// 128 rows x 800 keys x 4 sets: 17.8 us with one range, 19.9 with the three that would fill the device;
// 40 rows x 8000 keys: 20.3 with 15, 63.4 with one.  Beside own keys, whose blocks join them anyway, PT_LEAST_BESIDE: 256
// rows x 900 keys, 8 heads, 26.6 us with 512, 22.2 with 384, 20.8 with 256; 8 groups of 45 queries x 2 heads x 1000 keys,
// 6 key heads, 22.5, 20.4 and 18.5; with 128 the same as with 256.
constexpr int PT_LEAST = 512, PT_LEAST_BESIDE = 256;
constexpr int PA_CLUSTER = 16, PT_CLUSTER = 2;   // ranges that a cluster's blocks join by themselves
// Up to this many keys a block, one cluster instead of more ranges and the merge kernel: 5 rows x 2 heads x
// 30000 keys 17.8 us in clusters of 16, 30 us in 228 ranges; 5 x 6 x 1500: 8.2 in 16, 11.7 in 24.
constexpr int PA_CLUSTER_KEYS = 2048;
// Clusters of k_prefix_attention's blocks, by size, that GB300 holds at once (cudaOccupancyMaxActiveClusters)
constexpr int PA_CLUSTERS[PA_CLUSTER + 1] = {0, 456, 228, 148, 110, 87, 74, 59, 51, 46, 43, 36, 36, 28, 26, 26, 21};
constexpr int PA_SCORE_BYTES = 8192;   // own keys' scores kept by a block; three blocks still fit an SM
// Beside a prefix, own keys are cut into ranges of at least this many: one range needs no merge kernel.  2
// sequences x 6 heads x 900 keys: 12.4 us, 10.3 with ranges of 64 keys, but 4 us more of the host's time.
constexpr int OWN_LEAST = 512;
// The prefix's own ranges then, which the own keys' blocks join: 8 rows x 6 heads x 447 keys, up to 200 own keys 10.3 us
// with ranges of 64 keys, 8.2 with 256; 2 sequences x 3 queries x 1500 keys, 8 heads, up to 400 12.0 and 10.3.
constexpr int PA_LEAST_BESIDE = 256;

// Key ranges of a set: as many as are resident at once, in whole steps of a block, `most` at most.
void split_keys(PaSet &s, long long items, long long blocks, int step, long long most) {
    s.splits = s.chunk = 0;
    if (s.n_set <= 0) return;
    long long n = blocks / items;
    n = n > most ? most : n;
    n = n < 1 ? 1 : n;
    if (blocks != PT_BLOCKS) {
        if (n > PA_CLUSTER && (long long)PA_CLUSTER * PA_CLUSTER_KEYS >= s.max_keys) n = PA_CLUSTER;
        if (n <= PA_CLUSTER)
            while (n > 1 && items > PA_CLUSTERS[n]) --n;   // all clusters at once
    }
    s.chunk = (int)(((s.max_keys + n - 1) / n + step - 1) / step * step);
    s.splits = (s.max_keys + s.chunk - 1) / s.chunk;
    s.by_splits = divisor(s.splits);
    s.by_chunk = divisor(s.chunk);
}

struct PaPlan {
    bool tc;      // the prefix part runs on the tcgen05 kernel
    bool merge;   // partial results are joined by k_prefix_merge
    size_t part_o, part_ml, stats, total;
};

// Row tiles, key ranges and the workspace's layout, from host-known sizes only.
PaPlan plan(PaArgs &a, bool may_tc, bool pre_weight, bool own_weight) {
    PaPlan pl;
    const long long per = (long long)a.nq * a.rep, all = a.batch * per;
    a.by_per = divisor((int)per);
    a.by_rep = divisor(a.rep);
    a.by_seq = divisor(a.nq * a.n_head);
    a.by_gsize = divisor(a.gsize);
    a.by_kv = divisor(a.n_kv);
    const long long rows_a_set = a.pre.n_set > 0 ? (all + a.pre.n_set - 1) / a.pre.n_set : 0;
    const bool has_pre = a.pre.n_set > 0, has_own = a.own.n_set > 0;
    const auto slots = [&](int tile) {   // row tiles of a key head over all sets, with ragged groups at most
        return a.gsize == 0 ? a.pre.n_set + all / tile : a.pre.n_set * ((a.gsize * per + tile - 1) / tile);
    };
    const bool much = slots(PA_TILE) * a.n_kv * a.pre.max_keys >= PT_MIN_WORK;
    pl.tc = may_tc && rows_a_set > PT_MIN_ROWS && (much || (has_own && rows_a_set > 2 * PT_MIN_ROWS));
    // the smallest tile that holds an average group (us a call with tiles of 32, 64, 128 rows, 4 prefixes of 1500
    // keys: 20 rows 16.4, 16.5, 16.5; 40 rows 21.1, 18.5, 20.5; 100 rows 33.6, 23.9, 22.6)
    a.tile = !pl.tc ? PA_TILE : rows_a_set > 64 ? 128 : rows_a_set > 32 ? 64 : 32;
    a.slots = has_pre ? (int)slots(a.tile) : 0;
    a.own_tiles = (int)((per + PA_TILE - 1) / PA_TILE);
    a.tile_shift = a.tile == 128 ? 7 : a.tile == 64 ? 6 : a.tile == 32 ? 5 : 4;
    a.group_tiles = (int)((a.gsize * per + a.tile - 1) / a.tile);
    a.by_group_tiles = divisor(a.group_tiles);
    a.by_slots = divisor(a.slots);
    a.by_own_tiles = divisor(a.own_tiles);
    const auto ranges = [](const PaSet &s, int least) { return ((long long)s.max_keys + least - 1) / least; };
    constexpr int STEP = PA_WARPS * PA_SLOT_KEYS;
    // (with ragged groups the slots are more than the tiles that there will be, by half a tile a set on average)
    const long long tiles = a.slots - (a.gsize == 0 && has_own ? a.pre.n_set / 2 : 0);
    if (pl.tc)
        split_keys(a.pre, tiles * a.n_kv, PT_BLOCKS, PT_KEYS, a.pre.max_keys / (has_own ? PT_LEAST_BESIDE : PT_LEAST));
    else
        split_keys(a.pre, (long long)a.slots * a.n_kv, PA_BLOCKS, STEP, ranges(a.pre, has_own ? PA_LEAST_BESIDE : STEP));
    // own keys: one warp an item when that fills the device, more warps, then key ranges, when it does not (us a
    // call with one, two, four warps: 16 sequences x 20 heads x 448 keys 16.5, 13.0, 12.3; 80 sequences 33.8,
    // 34.9, 39.0; 256 sequences x 64 keys 23.2, 28.2, 41.0)
    // (warps without keys still finish rows beside a prefix: 2 sequences x 16 queries x 1500 keys and 17 own, 20 heads 12.0
    // us with four warps, 16.4 with one)
    const long long items = (long long)a.own.n_set * a.n_kv * a.own_tiles;
    const long long pieces = has_pre ? 8 * (per < PA_TILE ? per : PA_TILE) : 0;   // of 16 bytes that an item finishes
    a.own_wpi = PA_WARPS;
    while (a.own_wpi > 1 &&
           (items * a.own_wpi > PA_BLOCKS * PA_WARPS ||
            ((a.own_wpi - 1) * PA_KEYS >= a.own.max_keys && 32 * (a.own_wpi - 1) >= pieces)))
        a.own_wpi /= 2;
    // (with fewer than four warps the items fill the device or are short: one range, which needs no joining)
    split_keys(a.own, items, PA_BLOCKS * (PA_WARPS / a.own_wpi), a.own_wpi * PA_KEYS,
               a.own_wpi < PA_WARPS ? 1 : ranges(a.own, has_pre ? OWN_LEAST : STEP));
    a.own_items = items * a.own.splits;
    const bool one_launch = a.own_wpi == PA_WARPS && a.own.splits <= PA_CLUSTER && !has_pre;
    a.own_cluster = has_own && (a.own.splits == 1 || one_launch) ? a.own.splits : 0;
    a.pre_cluster = has_pre && !has_own && a.pre.splits <= (pl.tc ? PT_CLUSTER : PA_CLUSTER) ? a.pre.splits : 0;
    pl.merge = has_own ? a.own_cluster == 0 : a.pre_cluster == 0;
    a.after_pre = has_pre && has_own;
    a.n_part = pl.merge || a.after_pre ? a.pre.splits + (a.own_cluster ? 0 : a.own.splits) : 0;
    // the weights of own keys without a second pass, when an item sees all its keys and has room for the scores
    const long long scores = (per < PA_TILE ? per : PA_TILE) * (long long)a.own.chunk;
    const bool room = scores * (PA_WARPS / a.own_wpi) * 4 <= PA_SCORE_BYTES;
    a.score_floats = own_weight && a.own_cluster == 1 && a.own_tiles == 1 && room ? (int)scores : 0;
    const size_t rows = (size_t)a.batch * a.nq * a.n_head;
    size_t off = 0;
    pl.part_o = off;  off += up256(rows * a.n_part * 64 * 4);
    pl.part_ml = off; off += up256(rows * a.n_part * 8);
    pl.stats = off;   off += pre_weight || (own_weight && !a.score_floats) ? up256(rows * 8) : 0;
    pl.total = off;
    return pl;
}

int check_keys(const wh_keys *s, int n_kv, PaSet *o) {
    *o = PaSet{};
    if (!s) return WH_OK;
    if (s->n_set < 1 || s->n_set > 65535 || s->max_keys < 1 || s->max_keys > (1 << 30)) return WH_EINVAL;
    if (s->row_stride < 64LL * n_kv || s->row_stride % 8 != 0 || s->set_stride < 0 || s->set_stride % 8 != 0)
        return WH_EINVAL;
    if (!fits(s->k, 16) || !fits(s->v, 16) || (s->n_keys && !fits(s->n_keys, 4)) || (s->weight && !fits(s->weight, 4)))
        return WH_EINVAL;
    o->k = reinterpret_cast<const __nv_bfloat16 *>(s->k);
    o->v = reinterpret_cast<const __nv_bfloat16 *>(s->v);
    o->row_stride = s->row_stride;
    o->set_stride = s->set_stride;
    o->n_keys = s->n_keys;
    o->weight = s->weight;
    o->n_set = s->n_set;
    o->max_keys = s->max_keys;
    return WH_OK;
}

bool shape_ok(int batch, int n_query, int n_head, int n_kv) {
    return batch >= 0 && batch <= 65535 && n_query >= 1 && n_query <= 1024 && n_head >= 1 && n_head <= 1024 &&
           n_kv >= 1 && n_head % n_kv == 0 && (long long)batch * n_query * n_head <= 0x7fffffffLL;
}

int launch(PaArgs &a, const PaPlan &pl, const PtMaps &maps, uint8_t *ws, cudaStream_t s) {
    a.by_pre_tiles = divisor((int)((long long)a.slots * a.n_kv > 0x7fffffffLL ? 1 : a.slots * a.n_kv));
    a.part_o = reinterpret_cast<float *>(ws + pl.part_o);
    a.part_ml = reinterpret_cast<float2 *>(ws + pl.part_ml);
    a.stats = pl.total > pl.stats ? reinterpret_cast<float2 *>(ws + pl.stats) : nullptr;
    const long long pre_blocks = (long long)a.slots * a.n_kv * a.pre.splits;
    const long long own_blocks = (a.own_items * a.own_wpi + PA_WARPS - 1) / PA_WARPS;
    const long long rows = (long long)a.batch * a.nq * a.n_head;
    if (pre_blocks > 0x7fffffffLL || a.own_items > 0x7ffffff0LL) return WH_EINVAL;
    if (pre_blocks > 0) {
        if (int rc = pl.tc ? prefix_tc_launch(a, maps, s)
                           : launch_ex(k_prefix_attention<false>, dim3((unsigned)pre_blocks), PA_THREADS, PA_SMEM,
                                       a.pre_cluster, true, s, a))
            return rc;
    }
    if (own_blocks > 0) {
        const int smem = PA_SMEM + (a.score_floats ? PA_SCORE_BYTES : 0);
        if (int rc = launch_ex(k_prefix_attention<true>, dim3((unsigned)own_blocks), PA_THREADS, smem, a.own_cluster, true, s, a))
            return rc;
    }
    if (pl.merge)
        if (int rc = a.n_part <= 4 * PM_BATCH
                         ? launch_ex(k_prefix_merge<2>, dim3((unsigned)((rows + PM_TEAMS / 2 - 1) / (PM_TEAMS / 2))), 16 * PM_TEAMS, 0, 1, true, s, a)
                         : launch_ex(k_prefix_merge<PM_TEAMS>, dim3((unsigned)rows), 16 * PM_TEAMS, 0, 1, true, s, a))
            return rc;
    for (int own = 0; own < 2; ++own) {
        const PaSet &ks = own ? a.own : a.pre;
        if (!ks.weight || (own && a.score_floats)) continue;
        const int most = (ks.max_keys + PW_WARPS * PW_KEYS - 1) / (PW_WARPS * PW_KEYS);
        const long long fill = (PW_BLOCKS + (long long)a.n_kv * ks.n_set - 1) / ((long long)a.n_kv * ks.n_set);
        if (int rc = launch_ex(own ? k_prefix_weight<true> : k_prefix_weight<false>, dim3(fill < most ? (unsigned)fill : most, a.n_kv, ks.n_set),
                               32 * PW_WARPS, 0, 1, true, s, a))
            return rc;
    }
    return cudaGetLastError() == cudaSuccess ? WH_OK : WH_ECUDA;
}

}  // namespace

int prefix_attention_prepare() {
    const void *const kernels[2] = {reinterpret_cast<const void *>(k_prefix_attention<false>),
                                    reinterpret_cast<const void *>(k_prefix_attention<true>)};
    for (const void *k : kernels)
        if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, PA_SMEM + PA_SCORE_BYTES) != cudaSuccess ||
            cudaFuncSetAttribute(k, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
            return WH_ECUDA;
    return prefix_tc_prepare();
}

}  // namespace wh

using namespace wh;

// The sizes of a call as plan() takes them; false: no such call.
static bool sizes_of(int batch, int n_query, int n_head, int n_kv_head, int n_prefix, int max_prefix, int max_own, int needs,
                     PaArgs &a) {
    if (!shape_ok(batch, n_query, n_head, n_kv_head) || batch == 0 || n_prefix < 0 || n_prefix > 65535 ||
        max_prefix < 0 || max_prefix > (1 << 30) || max_own < 0 || max_own > (1 << 30) || (needs & ~7))
        return false;
    a.batch = batch;
    a.nq = n_query;
    a.n_head = n_head;
    a.n_kv = n_kv_head;
    a.rep = n_head / n_kv_head;
    a.pre.n_set = max_prefix > 0 ? n_prefix : 0;
    a.pre.max_keys = max_prefix;
    a.own.n_set = max_own > 0 ? batch : 0;
    a.own.max_keys = max_own;
    if (a.pre.n_set > 0 && !(needs & WH_GROUP_TABLE)) {
        if (batch % a.pre.n_set != 0) return false;
        a.gsize = batch / a.pre.n_set;
    }
    return true;
}

extern "C" size_t wh_prefix_attention_workspace(int batch, int n_query, int n_head, int n_kv_head, int n_prefix,
                                                int max_prefix, int max_own, int needs) {
    PaArgs a = {};
    if (!sizes_of(batch, n_query, n_head, n_kv_head, n_prefix, max_prefix, max_own, needs, a)) return 0;
    size_t most = 0;   // the prefix part may run on either kernel
    for (int tc = 0; tc < 2; ++tc) {
        const size_t t = plan(a, tc, needs & WH_PREFIX_WEIGHT, needs & WH_OWN_WEIGHT).total;
        most = t > most ? t : most;
    }
    return most;
}

extern "C" int wh_prefix_attention_plan(int batch, int n_query, int n_head, int n_kv_head, int n_prefix, int max_prefix,
                                        int max_own, int needs, wh_prefix_plan *out) {
    PaArgs a = {};
    if (!out || !sizes_of(batch, n_query, n_head, n_kv_head, n_prefix, max_prefix, max_own, needs, a)) return WH_EINVAL;
    const bool has_pre = a.pre.n_set > 0, has_own = a.own.n_set > 0;
    const bool pre_weight = has_pre && (needs & WH_PREFIX_WEIGHT), own_weight = has_own && (needs & WH_OWN_WEIGHT);
    if (!has_pre && !has_own) return WH_EINVAL;
    const PaPlan pl = plan(a, true, pre_weight, own_weight);
    *out = {};
    if (has_pre) {
        out->prefix_rows = a.tile;
        out->prefix_ranges = a.pre.splits;
        out->prefix_cluster = a.pre_cluster;
    }
    if (has_own) {
        out->own_warps = a.own_wpi;
        out->own_ranges = a.own.splits;
        out->own_cluster = a.own_cluster;
        out->own_scores_kept = a.score_floats > 0;
    }
    out->merge = pl.merge;
    out->launches = has_pre + has_own + pl.merge + pre_weight + (own_weight && !a.score_floats);
    return WH_OK;
}

extern "C" int wh_prefix_attention(const wh_bf16 *q, int64_t q_stride, int batch, int n_query, int n_head,
                                   int n_kv_head, const wh_keys *prefix, const int *group_start, const wh_keys *own,
                                   wh_bf16 *out, void *workspace, size_t ws_bytes, void *stream) {
    if (!shape_ok(batch, n_query, n_head, n_kv_head) || q_stride < 64LL * n_head || q_stride % 8 != 0) return WH_EINVAL;
    if (!prefix && !own) return WH_EINVAL;
    if (batch == 0) return WH_OK;
    PaArgs a = {};
    if (int rc = check_keys(prefix, n_kv_head, &a.pre)) return rc;
    if (int rc = check_keys(own, n_kv_head, &a.own)) return rc;
    if (own && own->n_set != batch) return WH_EINVAL;
    if (group_start && (!prefix || !fits(group_start, 4))) return WH_EINVAL;
    if (prefix && !group_start && batch % prefix->n_set != 0) return WH_EINVAL;
    if (!fits(q, 16) || !fits(out, 16) || (workspace && !fits(workspace, 256))) return WH_EINVAL;
    a.q = reinterpret_cast<const __nv_bfloat16 *>(q);
    a.q_stride = q_stride;
    a.group_start = group_start;
    a.gsize = prefix && !group_start ? batch / prefix->n_set : 0;
    a.batch = batch;
    a.nq = n_query;
    a.n_head = n_head;
    a.n_kv = n_kv_head;
    a.rep = n_head / n_kv_head;
    a.out = reinterpret_cast<__nv_bfloat16 *>(out);
    PaPlan pl = plan(a, true, a.pre.weight, a.own.weight);
    const size_t have = workspace ? ws_bytes : 0;
    if (have < pl.total) return WH_ENOSPC;
    DevCtl ctl;
    int num_sms = 0;
    if (int rc = device_ctl(&ctl, &num_sms)) return rc;
    a.ctl = ctl;
    PtMaps maps;
    if (pl.tc && prefix_tc_maps(a, &maps) != WH_OK) {   // strides that a tensor map cannot hold
        pl = plan(a, false, a.pre.weight, a.own.weight);
        if (have < pl.total) return WH_ENOSPC;
    }
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    trace_begin(TR_DEC_ATTN, s);
    const int rc = launch(a, pl, maps, static_cast<uint8_t *>(workspace), s);
    const double pairs = (a.pre.n_set > 0 ? (double)batch * a.pre.max_keys : 0.0) +
                         (a.own.n_set > 0 ? (double)batch * a.own.max_keys : 0.0);
    trace_end(TR_DEC_ATTN, s, pairs * n_query * n_head * 256.0,
              256.0 * n_kv_head * ((double)a.pre.n_set * a.pre.max_keys + (double)a.own.n_set * a.own.max_keys));
    return rc;
}
