// The shared-prefix part of wh_prefix_attention on the tcgen05 tensor cores, for groups of many rows.
//
// A block takes up to 128 rows (queries of a group's sequences and of a key head's query heads) and a range
// of the prefix's keys, in steps of 128 keys:
//   S = Q K^T      tcgen05.mma M = 128, N = 128, K = 64 into TMEM, Q and the TMA-loaded K in shared memory
//   P = 2^(S - m)  one row a thread: read from TMEM, running maximum and sum, back into TMEM
//   O += P V       tcgen05.mma M = 128, N = 64, K = 64 twice, P from TMEM, V as loaded (MN-major), O in TMEM
// With 32 or 64 rows the matrix product's 128 lanes hold 4 or 2 copies of them, each taking a quarter or
// half of the keys' columns (its P is zero elsewhere): the exponentials, not the padded products, are what
// takes time, and so none is spent on padding.  The copies are merged at the end like key ranges.
// O is rescaled only when a row's maximum has grown by more than 2^8.
// Both operands of the product have one type, bf16, whose half step is up to 2^-8 of a weight.  So P goes in as the
// sum of two bf16, 16 bits of mantissa (half a step: 2^-16), like k_prefix_attention's: a query's precision does not
// depend on how many share its keys.  The two take the columns of 128 keys, so a step's keys go in two halves: the
// second half's exponentials run beside the first half's products.
//
// Warp 0 loads (TMA), warp 1 issues the products (2 and 3 idle), warps 4 .. 7 are the rows' (warp w reads the
// TMEM lanes 32 (w % 4) and up).  Two blocks are resident on an SM, so one's softmax runs beside the other's products.
// What bounds it, in cycles of a step with two blocks on the SM: 32 rows wait for keys and values, 1200 of 2500 (exponentials
// 310); with 256 rows the rows' warps are busy, 2250 of 2970 (exponentials and their two parts 1300, maximum 400, TMEM reads
// and writes 365, rescaling 190), and the products' warp issues for 710.
//   32 rows, 20 heads, 30000 keys: 33 us, 154 MB, 4.7 TB/s (a TMA read alone takes 26)
//   256 rows, 20 heads, 15000 keys: 39 us, 19.7 GFLOP, 505 TFLOP/s; both tiles read every key
// Not kept (these and the comparisons below with one bf16 a weight): rings of keys and values with their own barriers, 38 ->
// 40 us at 32 rows; pairs of blocks that load for each other by multicast, 51.5 -> 55 us at 256 rows; two stages instead of
// three, 38 -> 44.  With two: P's low parts in S's columns, read by then, and the next scores after the products, 59.1 ->
// 62.8 us (256 rows beside own keys); the next scores between the halves, 61.5.
// Every wait is bounded; when one runs out the block records WH_ETIMEOUT and winds down.
#include "prefix_attention.cuh"

namespace wh {
namespace {

constexpr int PT_THREADS = 256, PT_STAGES = 3;
// Register split (setmaxnreg): two blocks of 256 threads launch at 128 a thread; the first warpgroup (loads,
// products) drops to 40, the rows' rises to 208 and holds a row's 128 scores: 128 x (40 + 208) <= 256 x 128.
constexpr int REG_LOW = 40, REG_HIGH = 208;
static_assert(128 * (REG_LOW + REG_HIGH) <= PT_THREADS * 128, "register split exceeds the launch total");
constexpr int TILE_BYTES = 128 * 128;                       // 128 rows of 64 bf16
constexpr int OFF_RING = TILE_BYTES;                        // Q first
constexpr int OFF_BARS = OFF_RING + PT_STAGES * 2 * TILE_BYTES;
constexpr int PT_SMEM = OFF_BARS + 1024;                    // two blocks fill an SM's shared memory
constexpr uint32_t PT_COLS = 256;   // S [0, 128), O [128, 192), P of 64 keys: high parts [192, 224), low parts [224, 256)
constexpr int SO_ROW = 68;                                  // floats a row of the epilogue's staging

// (by the array's size, for the columns of a thread)
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[32]) { tmem_ld32(taddr, r); }
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[16]) { tmem_ld16(taddr, r); }
__device__ __forceinline__ void tmem_st(uint32_t taddr, const uint32_t (&r)[16]) { tmem_st16(taddr, r); }
__device__ __forceinline__ void tmem_st(uint32_t taddr, const uint32_t (&r)[8]) { tmem_st8(taddr, r); }
__device__ __forceinline__ void rows_bar() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

template <int COPIES>
__global__ void __launch_bounds__(PT_THREADS, 2) k_prefix_tc(const __grid_constant__ PtMaps tm, const PaArgs p) {
    constexpr int TILE = 128 / COPIES;          // rows of the block
    constexpr int HALF = 64 / COPIES;           // columns that a thread takes of each 64 keys
    constexpr int W = HALF < 32 ? HALF : 32;    // columns of one TMEM access
    constexpr int BLOCKS = HALF / W;            // and accesses of a half
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t *sQ = smem, *sKV = smem + OFF_RING;   // stage s: K at s * 32 KB, V 16 KB behind it
    uint64_t *kv_full = reinterpret_cast<uint64_t *>(smem + OFF_BARS);
    uint64_t *kv_empty = kv_full + PT_STAGES;
    uint64_t *s_full = kv_empty + PT_STAGES;
    uint64_t *s_free = s_full + 1;
    uint64_t *p_full = s_free + 1;
    uint64_t *o_full = p_full + 1;
    uint64_t *drain = o_full + 1;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    Rows rw;
    int set, r0, nk;
    // a cluster's blocks are the ranges of one item; else neighbours are tiles and heads, which read the same
    // rows or the same DRAM pages at about the same time
    const int cluster = p.pre_cluster;
    int x = blockIdx.x, item, split;
    if (cluster > 1) {
        split = remainder(p.pre.by_splits, p.pre.splits, x);
        item = x;
    } else {
        item = remainder(p.by_pre_tiles, p.slots * p.n_kv, x);
        split = x;
    }
    const int slot = remainder(p.by_slots, p.slots, item);
    rw.hk = item;
    if (!p.group_start) {
        // the first step's rows (below max_keys: the cache's own, what they hold is not looked at) are on their way
        // to L2 before the inputs may be read: 1 us of 35 at 32 rows x 20 heads x 30000 keys
        set = p.by_group_tiles.of(slot);
        const int t = split * p.pre.chunk + (threadIdx.x & 127);
        if (t < p.pre.max_keys)
            prefetch_l2((threadIdx.x >= 128 ? p.pre.v : p.pre.k) + (long long)set * p.pre.set_stride +
                        (long long)t * p.pre.row_stride + rw.hk * 64);
    }
    pdl_wait();   // what runs after this kernel's trigger may count on its inputs
    pdl_launch_dependents();
    if (cluster && split == 0) finish_outside(p, slot, rw.hk);
    if (!find_tile(p, slot, rw.hk == 0 && split == 0, set, r0, rw, nk)) return;
    const int k0 = split * p.pre.chunk, k1 = min(nk, k0 + p.pre.chunk);
    const int a = threadIdx.x - 128;   // the rows' threads: TMEM lane and matrix row
    float *so = reinterpret_cast<float *>(sKV);   // the epilogue's rows, then their maxima and sums
    float2 *sml = reinterpret_cast<float2 *>(sKV + 128 * SO_ROW * 4);
    const int rows = min(TILE, rw.n - r0);
    if (k0 >= k1) {                   // no keys here
        // An SM takes no second block before the first has given up its right to allocate TMEM, and this one may
        // stay for its cluster: 24 sets of 300 .. 1500 keys x 80 rows x 6 heads 18.7 us, 28.3 without this.
        if (warp == 1) tmem_relinquish();
        if (cluster) {
            for (int i = threadIdx.x; i < rows * SO_ROW; i += PT_THREADS) so[i] = 0.0f;
            for (int i = threadIdx.x; i < rows; i += PT_THREADS) sml[i] = make_float2(-INFINITY, 0.0f);
            if (cluster > 1) {
                __syncwarp();
                cluster_sync();
                if (warp >= 4) finish_cluster<128>(p, rw, r0, rows, so, SO_ROW, sml, cluster, a);
                __syncwarp();
                cluster_sync();
            } else {
                for (int i = threadIdx.x; i < rows * 8; i += PT_THREADS) {
                    float none[8] = {};
                    finish_row(p, rw, r0 + (i >> 3), 8 * (i & 7), -INFINITY, 0.0f, none, 0);
                }
            }
        }
        return;
    }
    if ((smem_u32(smem) & 1023u) != 0) {   // the swizzled tiles must lie on 1024-byte boundaries
        if (threadIdx.x == 0) set_status(p.ctl, WH_EBOUNDS);
        return;                            // (every block of a cluster alike)
    }
    const int nt = (k1 - k0 + PT_KEYS - 1) / PT_KEYS;
    const int z = tm.one_set ? 0 : set;
    auto load_step = [&](int j) {   // one thread
        uint8_t *kb = sKV + (j % PT_STAGES) * 2 * TILE_BYTES;
        uint64_t *bar = kv_full + j % PT_STAGES;
        mbar_arrive_expect_tx(bar, 2 * TILE_BYTES);
        tma_load_3d(kb, &tm.k, bar, rw.hk * 64, k0 + j * PT_KEYS, z);
        tma_load_3d(kb + TILE_BYTES, &tm.v, bar, rw.hk * 64, k0 + j * PT_KEYS, z);
    };

    if (threadIdx.x == 0) {
        for (int s = 0; s < PT_STAGES; ++s) {
            mbar_init(kv_full + s, 1);
            mbar_init(kv_empty + s, 1);
        }
        mbar_init(s_full, 1);
        mbar_init(s_free, 4);
        mbar_init(p_full, 4);
        mbar_init(o_full, 1);
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
        // the first steps' keys and values are on their way while the block sets up
        for (int j = 0; j < nt && j < PT_STAGES; ++j) load_step(j);
    }
    if (warp == 1) {
        // (not first of all: an SM's second block starts after this, and two that start together, both loading,
        // then both computing, take longer: 35.4 us against 33.3 at 32 rows x 20 heads x 30000 keys)
        tmem_alloc(tmem_slot, PT_COLS);
        tmem_relinquish();
    }
    if (warp >= 4) {
        // matrix row a holds row a % TILE, 128-byte swizzled as the products read it
        const int r = r0 + (a % TILE);
        uint4 u[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) u[i] = make_uint4(0, 0, 0, 0);
        if (r < rw.n) {
            int qrow, head, qi;
            rw.locate(p, r, qrow, head, qi);
            const uint4 *src = reinterpret_cast<const uint4 *>(p.q + (long long)qrow * p.q_stride + head * 64);
#pragma unroll
            for (int i = 0; i < 8; ++i) u[i] = ld_live(src + i);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) *reinterpret_cast<uint4 *>(sQ + a * 128 + ((i ^ (a & 7)) << 4)) = u[i];
        fence_proxy_async_smem();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    if (warp < 4) {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REG_LOW));
      if (warp == 0) {
        if (lane == 0) {
            int j = nt < PT_STAGES ? nt : PT_STAGES;   // the steps so far
            for (; j < nt; ++j) {
                if (*abort_flag || !mbar_wait(kv_empty + j % PT_STAGES, (j / PT_STAGES - 1) & 1u, p.ctl)) {
                    *abort_flag = 1;
                    break;
                }
                load_step(j);
            }
            // no copy of this block may still be in flight when it exits
            for (int i = j > PT_STAGES ? j - PT_STAGES : 0; i < j; ++i)
                mbar_wait(kv_full + i % PT_STAGES, (i / PT_STAGES) & 1u, p.ctl);
        }
      } else if (warp == 1) {
        // The whole warp waits and one elected lane issues: with everything in one lane's branch, the instructions that
        // bring each product's operands together took 2225 of a step's 3400 cycles, now 640 (256 rows x 15000 keys beside
        // own keys 57.9 us, 54.7 so).
        const bool one = elect_one();
        constexpr uint32_t IDESC_S = idesc_bf16_f32(128, PT_KEYS);
        constexpr uint32_t IDESC_O = idesc_bf16_f32(128, 64) | (1u << 16);   // V is MN-major
        // one descriptor of each kind, the others by what their addresses differ (in 16-byte units)
        constexpr uint64_t STAGE = 2 * TILE_BYTES / 16;
        const uint64_t qd = sdesc_sw128(smem_u32(sQ)), kd0 = sdesc_sw128(smem_u32(sKV));
        const uint64_t vd0 = sdesc_sw128_mn(smem_u32(sKV) + TILE_BYTES);
        auto issue_s = [&](int s) {
            const uint64_t kd = kd0 + s * STAGE;
            tc_fence_after();
            if (one) {
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    umma_bf16(tmem, qd + (uint64_t)(2 * kk), kd + (uint64_t)(2 * kk), IDESC_S, kk != 0);
                umma_commit(s_full);
            }
            __syncwarp();
        };
        bool ok = __all_sync(0xffffffffu, !*abort_flag && mbar_wait(kv_full, 0, p.ctl));
        if (ok) issue_s(0);
        int stage = 0;             // of step j
        uint32_t next_phase = 0;   // of the barrier of step j + 1's stage
        for (int j = 0; ok && j < nt; ++j) {
            const int next = stage + 1 == PT_STAGES ? 0 : stage + 1;
            next_phase ^= next == 0;
            if (j + 1 < nt) {   // the next scores as soon as this step's have been read
                ok = __all_sync(0xffffffffu, !*abort_flag && mbar_wait(kv_full + next, next_phase, p.ctl) &&
                                                 mbar_wait(s_free, j & 1u, p.ctl));
                if (!ok) break;
                issue_s(next);
            }
            const uint64_t vd = vd0 + stage * STAGE;
#pragma unroll
            for (int h = 0; h < 2; ++h) {   // the halves are phases 2j and 2j + 1 of p_full and o_full
                ok = __all_sync(0xffffffffu, !*abort_flag && mbar_wait(p_full, h, p.ctl));
                if (!ok) break;
                tc_fence_after();
                if (one) {
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) {
                        const uint64_t v = vd + (uint64_t)((4 * h + kk) * 2048 / 16);
                        umma_bf16_tmem_a(tmem + 128u, tmem + 192u + 8u * kk, v, IDESC_O, h + kk > 0 ? 1u : j != 0);
                        umma_bf16_tmem_a(tmem + 128u, tmem + 224u + 8u * kk, v, IDESC_O, 1u);
                    }
                    umma_commit(o_full);
                    if (h == 1) umma_commit(kv_empty + stage);
                }
                __syncwarp();
            }
            if (!ok) break;
            stage = next;
        }
        if (!ok) *abort_flag = 1;
        if (one) umma_commit(drain);
        __syncwarp();
        mbar_wait(drain, 0, p.ctl);
      }
      __syncwarp();
      if (cluster > 1) {   // the row warps' two barriers
          cluster_sync();
          cluster_sync();
      }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REG_HIGH));
        const int col0 = (a / TILE) * HALF;   // the columns of this copy in every 64
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        const uint32_t tS = tmem + lanes + (uint32_t)col0, tO = tmem + lanes + 128u, tP = tmem + lanes + 192u;
        if (COPIES > 1) {   // the other copies' columns of P stay zero
            const uint32_t zero[32] = {};
            tmem_st32(tP, zero);
            tmem_st32(tP + 32u, zero);
            tmem_wait_st();
        }
        float m = -INFINITY, l = 0.0f;
        bool ok = true;
        for (int j = 0; j < nt; ++j) {
            ok = __all_sync(0xffffffffu, !*abort_flag && mbar_wait(s_full, j & 1u, p.ctl));
            if (!ok) break;
            tc_fence_after();
            uint32_t sv[2][BLOCKS][W];   // scores of keys 64 h + col0 + W i + k of the step
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < BLOCKS; ++i) tmem_ld(tS + 64u * h + (uint32_t)(W * i), sv[h][i]);
            tmem_wait_ld();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(s_free);   // S may now be overwritten
            const int valid = k1 - k0 - j * PT_KEYS;   // keys of this step inside the range
            if (valid < PT_KEYS) {
#pragma unroll
                for (int i = 0; i < 2 * BLOCKS; ++i)
#pragma unroll
                    for (int k = 0; k < W; ++k)
                        if (64 * (i / BLOCKS) + col0 + W * (i % BLOCKS) + k >= valid)
                            sv[i / BLOCKS][i % BLOCKS][k] = 0xff800000u;   // -inf
                // values past the range may be anything, NaN too, and 0 * NaN is NaN: clear them
                ok = __all_sync(0xffffffffu, mbar_wait(kv_full + j % PT_STAGES, (j / PT_STAGES) & 1u, p.ctl));
                if (!ok) break;
                if (a >= valid) {
                    uint4 *row = reinterpret_cast<uint4 *>(sKV + (j % PT_STAGES) * 2 * TILE_BYTES + TILE_BYTES + a * 128);
#pragma unroll
                    for (int i = 0; i < 8; ++i) row[i] = make_uint4(0, 0, 0, 0);
                }
                fence_proxy_async_smem();
            }
            float pm[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) pm[k] = -INFINITY;
#pragma unroll
            for (int i = 0; i < 2 * BLOCKS; ++i)
#pragma unroll
                for (int k = 0; k < W; k += 2) {
                    const uint32_t *x = sv[i / BLOCKS][i % BLOCKS] + k;
                    pm[(k >> 1) & 3] = max3(pm[(k >> 1) & 3], __uint_as_float(x[0]), __uint_as_float(x[1]));
                }
            const float m_new = fmaxf(m, fmaxf(fmaxf(pm[0], pm[1]), fmaxf(pm[2], pm[3])));
            if (j == 0) {
                m = m_new;
            } else {
                // the products of the step before are done: O is stable and P may be overwritten
                ok = __all_sync(0xffffffffu, mbar_wait(o_full, 1u, p.ctl));
                if (!ok) break;
                tc_fence_after();
                const bool need = (m_new - m) * PA_SCALE > 8.0f;
                if (__any_sync(0xffffffffu, need)) {
                    float f = 1.0f;
                    if (need) {
                        f = ex2_approx((m - m_new) * PA_SCALE);
                        l *= f;
                        m = m_new;
                    }
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        uint32_t v[32];
                        tmem_ld32(tO + 32u * half, v);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * f);
                        tmem_st32(tO + 32u * half, v);
                    }
                    tmem_wait_st();
                }
            }
            const float ms = m == -INFINITY ? 0.0f : m;
            const uint64_t scale2 = f2_pack(PA_SCALE, PA_SCALE), minus2 = f2_pack(-ms, -ms);
            uint64_t sum2[2] = {0ull, 0ull};
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t hi[BLOCKS][W / 2], lo[BLOCKS][W / 2];   // the weights as a sum of two bf16 each
#pragma unroll
                for (int i = 0; i < BLOCKS; ++i)
#pragma unroll
                    for (int k = 0; k < W / 2; ++k) {
                        const uint32_t *x = sv[h][i] + 2 * k;
                        float x0, x1;
                        f2_unpack(mul_f2(add_f2(f2_pack(__uint_as_float(x[0]), __uint_as_float(x[1])), minus2), scale2), x0, x1);
                        const float e0 = ex2_approx(x0), e1 = ex2_approx(x1);
                        const uint64_t e = f2_pack(e0, e1);
                        sum2[k & 1] = add_f2(sum2[k & 1], e);
                        const uint32_t top = pack_bf16(e0, e1);
                        hi[i][k] = top;
                        f2_unpack(add_f2(e, f2_pack(__uint_as_float((top << 16) ^ 0x80000000u), __uint_as_float((top & 0xffff0000u) ^ 0x80000000u))), x0, x1);
                        lo[i][k] = pack_bf16(x0, x1);
                    }
                if (h == 1) {   // the first half's products are done with P
                    ok = __all_sync(0xffffffffu, mbar_wait(o_full, 0u, p.ctl));
                    if (!ok) break;
                    tc_fence_after();
                }
#pragma unroll
                for (int i = 0; i < BLOCKS; ++i) {
                    tmem_st(tP + (uint32_t)(col0 / 2 + W / 2 * i), hi[i]);
                    tmem_st(tP + 32u + (uint32_t)(col0 / 2 + W / 2 * i), lo[i]);
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full);
            }
            if (!ok) break;
            float x0, x1;
            f2_unpack(add_f2(sum2[0], sum2[1]), x0, x1);
            l += x0 + x1;
        }
        if (ok) ok = __all_sync(0xffffffffu, mbar_wait(o_full, 1u, p.ctl));
        if (!ok) *abort_flag = 1;
        tc_fence_after();
        // every product is done, so the ring is free: stage O, merge the copies, then the ranges
        float2 *sml_copy = sml + 128;
        if (ok) {
            sml_copy[a] = make_float2(m, l);
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                uint32_t v[32];
                tmem_ld32(tO + 32u * half, v);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    *reinterpret_cast<uint4 *>(so + a * SO_ROW + 32 * half + 4 * i) =
                        make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
            }
        }
        rows_bar();
        if (!*abort_flag) {
            for (int i = a; i < rows * 8; i += 128) {
                const int r = i >> 3, d0 = 8 * (i & 7);
                float mt = -INFINITY, lt = 0.0f, v[8] = {};
#pragma unroll
                for (int c = 0; c < COPIES; ++c) mt = fmaxf(mt, sml_copy[r + TILE * c].x);
#pragma unroll
                for (int c = 0; c < COPIES; ++c) {
                    const float2 ml = sml_copy[r + TILE * c];
                    const float f = COPIES == 1 ? 1.0f : ml.x == -INFINITY ? 0.0f : ex2_approx((ml.x - mt) * PA_SCALE);
                    lt = fmaf(ml.y, f, lt);
#pragma unroll
                    for (int k = 0; k < 8; k += 4) {
                        const float4 x = *reinterpret_cast<const float4 *>(so + (r + TILE * c) * SO_ROW + d0 + k);
                        v[k] = fmaf(x.x, f, v[k]), v[k + 1] = fmaf(x.y, f, v[k + 1]);
                        v[k + 2] = fmaf(x.z, f, v[k + 2]), v[k + 3] = fmaf(x.w, f, v[k + 3]);
                    }
                }
                if (cluster == 0) {
                    leave_part(p, rw, r0 + r, split, d0, mt, lt, v);
                } else if (cluster == 1) {
                    finish_row(p, rw, r0 + r, d0, mt, lt, v, 0);
                } else {
                    float *d = so + r * SO_ROW + d0;   // (only this thread reads or writes these dims)
                    *reinterpret_cast<float4 *>(d) = make_float4(v[0], v[1], v[2], v[3]);
                    *reinterpret_cast<float4 *>(d + 4) = make_float4(v[4], v[5], v[6], v[7]);
                    if (d0 == 0) sml[r] = make_float2(mt, lt);
                }
            }
        }
        if (cluster > 1) {
            __syncwarp();
            cluster_sync();
            if (!*abort_flag) finish_cluster<128>(p, rw, r0, rows, so, SO_ROW, sml, cluster, a);
            __syncwarp();
            cluster_sync();   // no block leaves while another may still read its rows
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, PT_COLS);
    }
}

template <int COPIES>
int set_attr() {
    return cudaFuncSetAttribute(k_prefix_tc<COPIES>, cudaFuncAttributeMaxDynamicSharedMemorySize, PT_SMEM) == cudaSuccess &&
                   cudaFuncSetAttribute(k_prefix_tc<COPIES>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess
               ? WH_OK
               : WH_ECUDA;
}

}  // namespace

int prefix_tc_prepare() { return set_attr<1>() | set_attr<2>() | set_attr<4>(); }

int prefix_tc_maps(const PaArgs &a, PtMaps *m) {
    m->one_set = a.pre.n_set == 1 || a.pre.set_stride == 0;
    const long long sets = m->one_set ? 1 : a.pre.n_set;
    const long long set_ld = m->one_set ? a.pre.row_stride : a.pre.set_stride;   // (not used with one set)
    if (int rc = make_tmap_bf16_sets(&m->k, a.pre.k, 64 * a.n_kv, a.pre.max_keys, a.pre.row_stride, sets, set_ld, PT_KEYS))
        return rc;
    return make_tmap_bf16_sets(&m->v, a.pre.v, 64 * a.n_kv, a.pre.max_keys, a.pre.row_stride, sets, set_ld, PT_KEYS);
}

int prefix_tc_launch(const PaArgs &a, const PtMaps &m, cudaStream_t s) {
    const dim3 grid((unsigned)((long long)a.slots * a.n_kv * a.pre.splits));
    auto *kernel = a.tile == 128 ? k_prefix_tc<1> : a.tile == 64 ? k_prefix_tc<2> : k_prefix_tc<4>;
    return launch_ex(kernel, grid, PT_THREADS, PT_SMEM, a.pre_cluster, true, s, m, a);
}

}  // namespace wh
