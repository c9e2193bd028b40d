// Eviction from key/value caches by accumulated attention weight.
//
// Each head of each set keeps, of its n keys, the last `recent` and of the others the budget - recent
// with the largest weight (ties: the lowest index), in their order, moved together at the front.
//
// Choosing: the weight W below which no older key stays is found by a binary search over the 32 bits of an
// order-preserving integer image of the weights, which the choosing threads hold in registers, counting how
// many are at least the candidate.  Then the keys that stay are numbered in order: those above W, the first
// few equal to W, the recent ones.
// Moving is a copy of 128-byte rows, 16 bytes a thread, bound by HBM: within the cache every key moves towards
// the front, so going up the rows with each step's reads before its writes is safe.
// 512 sets x 20 heads of 301 .. 448 keys to 224: 189 us, 1.21 GB, 94 % of the copy rate (choosing takes 15 us of
// it, mostly instructions: 1600 a warp of 448 keys); 20 heads x 30000 keys to 4001: 24 us for 44 MB, of which
// choosing takes 15 (a search of four or five steps of 3100 cycles, numbering 5500).
//   k_evict_small   up to 2048 keys: a block chooses and moves one head of one set
//   k_evict_select, then k_evict_move (other buffers: rows spread over the device) or k_evict_shift (within
//   the cache: a cluster per head and keys or values), for long caches and where few heads move many rows
#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace wh {
namespace {

constexpr int SM_THREADS = 256;      // k_evict_small
constexpr int SM_MOST = 2048;        // its longest cache
// It is taken for up to SM_HEADS heads (what is resident at once) that move up to SM_ROWS rows, and within the cache for
// at least half as many heads that move more; us a replayed call in one kernel and in two, keys -> budget:
//    12 heads  448 ->  224    8.2  10.3      480 heads  448 -> 224    16.7  18.5
//   320 heads  448 ->  224   13.4  16.4      800 heads  448 -> 224    24.7  25.4
//    12 heads 2000 ->  600   12.4  11.0   (the second kernel costs the host 4 us more)
//    12 heads 2000 -> 1500   16.7  11.6      320 heads 2000 -> 1500   53.0  49.2
//   within the cache, the copy of it that the caller makes included: 320 heads 1500 -> 1200 84.1 and 94.3
constexpr int SM_ROWS = 1024;
constexpr int SM_HEADS = 4 * 152;
constexpr int SEL_THREADS = 1024;    // k_evict_select: the most threads of one block a head
// Up to 16 keys a thread where that many threads can hold them (up to 4096 keys a block of 256: 1000 heads x 3000 keys
// 62 us, 99 with 1024 threads of 8 keys; up to 8192 one of 512; up to 16384 one of 1024: 200 heads x 9000 keys 62 us,
// 80 with 32 keys a thread).  Clusters of SEL_CTAS blocks of 256 threads choose instead for as many heads of long
// caches as are resident at once, and for the longest: 20 heads x 9000 keys 16.3 us, 19.7 with a block each; 60 heads
// 27.8 and 28.3; 60 x 30000 46.2 and 50.5; 20 x 60000 35 and 155.
constexpr int SEL_CTAS = 8;
constexpr int SEL_SPREAD = 72;
constexpr int MV_THREADS = 256;
constexpr int MV_PIECES = 1024;      // 16-byte pieces (of keys, and of values) of a block of k_evict_move
// k_evict_shift.  20 heads 30000 keys -> 15000, the caller's copy of the cache (about 80 us) included: 241 us with one
// block of 512 threads and 4 rows a thread for each head, 144 with clusters of eight, 123 with four blocks of 256
// threads an SM, 118 with six rows a thread, 141 with eight (registers).
constexpr int SH_THREADS = 256;
constexpr int SH_ROWS = 6;           // rows of a thread that are under way together
constexpr int SH_RESIDENT = 4;       // blocks of an SM

struct EvArgs {
    const __nv_bfloat16 *k, *v;
    __nv_bfloat16 *k_out, *v_out;
    long long row_stride, set_stride, out_row_stride, out_set_stride;
    const float *weight;
    float *weight_out;
    const int *n_keys;
    int *n_out;
    int *kept;                 // [n_set][n_head][kept_stride]: source index of every key that stays
    long long kept_stride;     // the caller's: budget; the workspace's: what can stay
    int *count;                // [n_set]: keys before, as clamped
    int max_keys, out_keys, n_set, n_head, budget, recent, in_place;
    Divisor by_row;            // 16-byte pieces of a row
    int *status;
};

// Larger weight, larger image; -0 as 0; NaN below everything.
__device__ __forceinline__ uint32_t weight_key(float w) {
    if (w != w) return 0u;
    const uint32_t u = __float_as_uint(w + 0.0f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Threads that choose together: one warp, a block, or the blocks of a cluster.
template <int THREADS, int CTAS = 1>
struct Team {
    static constexpr int WARPS = THREADS / 32, BLOCKS = CTAS, ALL = THREADS * CTAS;
    int *buf;    // [2 * WARPS]
    int *peers;  // CTAS > 1: [2][CTAS], one number of every block, in turns
    int turn;
    uint32_t *bins;   // CTAS > 1: [2][warp][8] and [2][block][8]
    __device__ __forceinline__ static int rank() { return CTAS == 1 ? 0 : (int)cluster_ctarank(); }
    __device__ __forceinline__ static int thread() {   // of the team
        return THREADS == 32 ? threadIdx.x & 31 : rank() * THREADS + threadIdx.x;
    }
    // Everything written so far is visible to the whole team.
    __device__ __forceinline__ static void sync() {
        if (CTAS > 1)
            cluster_sync();
        else if (WARPS == 1)
            __syncwarp();
        else
            __syncthreads();
    }
    // Every block's x (the same in all of its threads), in every thread of the team: lane c holds block c's.
    // The two turns' places alternate: a place is filled again only behind the barrier after its reads.
    __device__ __forceinline__ int gather(int x) {
        const int lane = threadIdx.x & 31;
        int *mine = peers + turn * CTAS;
        turn ^= 1;
        if (threadIdx.x < CTAS)
            asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(mapa_shared(mine + rank(), threadIdx.x)), "r"(x) : "memory");
        cluster_sync();
        return lane < CTAS ? mine[lane] : 0;
    }
    __device__ __forceinline__ int block_sum(int x) const {
        x = __reduce_add_sync(0xffffffffu, x);
        if (WARPS == 1) return x;
        if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = x;
        __syncthreads();
        const int s = __reduce_add_sync(0xffffffffu, (threadIdx.x & 31) < WARPS ? buf[threadIdx.x & 31] : 0);
        __syncthreads();
        return s;
    }
    // Sum over the team, the same in every thread.
    __device__ __forceinline__ int sum(int x) {
        x = block_sum(x);
        return CTAS == 1 ? x : __reduce_add_sync(0xffffffffu, gather(x));
    }
    __device__ __forceinline__ uint32_t largest(uint32_t x) {
        x = __reduce_max_sync(0xffffffffu, x);
        if (WARPS > 1) {
            if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = (int)x;
            __syncthreads();
            x = __reduce_max_sync(0xffffffffu, (threadIdx.x & 31) < WARPS ? (uint32_t)buf[threadIdx.x & 31] : 0u);
            __syncthreads();
        }
        return CTAS == 1 ? x : __reduce_max_sync(0xffffffffu, (uint32_t)gather((int)x));
    }
    // Exclusive sums over the team's warps of two per-warp numbers.
    __device__ __forceinline__ void before(int x, int y, int &bx, int &by) {
        bx = by = 0;
        if (WARPS == 1) return;
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        if (lane == 0) buf[warp] = x, buf[WARPS + warp] = y;
        __syncthreads();
        const int vx = lane < WARPS ? buf[lane] : 0, vy = lane < WARPS ? buf[WARPS + lane] : 0;
        bx = __reduce_add_sync(0xffffffffu, lane < warp ? vx : 0);
        by = __reduce_add_sync(0xffffffffu, lane < warp ? vy : 0);
        const int tx = __reduce_add_sync(0xffffffffu, vx), ty = __reduce_add_sync(0xffffffffu, vy);
        __syncthreads();
        if (CTAS > 1) {
            const int both = gather(tx | ty << 16);   // (a block holds fewer than 65536 in all)
            bx += __reduce_add_sync(0xffffffffu, lane < rank() ? both & 0xffff : 0);
            by += __reduce_add_sync(0xffffffffu, lane < rank() ? (int)((uint32_t)both >> 16) : 0);
        }
    }
};

// The weights' image W and how many keys equal to it stay: the keys above W, `above` many, all do.  `count`
// gives the number of the older keys whose image is at least a candidate; `most` is the largest image and
// `differ` has a bit set wherever any two images differ, so that their common leading bits cost no counting.
// Stops early when exactly `need` keys are at least the candidate: then none equal to W has to be told apart.
template <class Count>
__device__ __forceinline__ void find_threshold(int need, uint32_t most, uint32_t differ, Count count, uint32_t &W, int &ties) {
    int bit = 31 - __clz(differ | 1u);
    W = bit == 31 ? 0u : most >> (bit + 1) << (bit + 1);
    for (; bit >= 0; --bit) {
        const uint32_t cand = W | (1u << bit);
        const int c = count(cand);
        if (c >= need) W = cand;
        if (c == need) {
            W = cand - 1;   // the need-th largest is at least cand, the next one less
            ties = 0;
            return;
        }
    }
    ties = need - (W == 0xffffffffu ? 0 : count(W + 1));
}

// The same for a cluster, four bits at a time: every thread counts its images under the decided bits in 16 bins of
// 8 bits, the warps, blocks and the cluster add them in bins of 16 (fewer than 65536 older keys: the `pads` zero images
// of a thread that stand for none are not counted).  A step takes 3100 cycles with 16 images a thread: counting 1100,
// adding in the warps 630, the cluster barrier 570.  (Bins counted by ballots: 24.2 -> 25.3 us for 20 heads x 30000.)
// The first step guesses that the threshold lies in 2^-19 .. 512, where weights of long caches mostly do, and then
// knows eight bits of it; else the steps begin anew.
template <int E, class T>
__device__ __forceinline__ void find_threshold_radix(T &team, int need, const uint32_t (&key)[E], int pads, uint32_t &W, int &ties) {
    static_assert(E < 256 && T::WARPS == 8 && T::BLOCKS == 8, "the bins' widths, the lanes' shares");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, word = lane & 7, part = lane >> 3;
    constexpr int GUESS = 0xb5;   // images' first byte: 0xb6 .. 0xc3 (2^-19 .. 512) get bins 1 .. 14, the rest bins 0 and 15
    uint32_t prefix = 0;
    bool guess = true;
    for (int shift = 24, turn = 0; shift >= 0; turn ^= 1) {
        unsigned long long c[2] = {0, 0};
        const auto count = [&](uint32_t x) {
            const unsigned long long one = x < 16u ? 1ull << (8 * (x & 7u)) : 0ull;
            c[0] += x & 8u ? 0ull : one;
            c[1] += x & 8u ? one : 0ull;
        };
        if (guess) {
#pragma unroll
            for (int j = 0; j < E; ++j) count((uint32_t)min(max((int)(key[j] >> 24) - GUESS, 0), 15));
        } else {
#pragma unroll
            for (int j = 0; j < E; ++j) count((key[j] ^ prefix) >> shift);   // below 16: the decided bits agree, these are the next
        }
        if (prefix == 0) c[0] -= pads;   // they are in bin 0 as long as nothing is decided
        // bins 4i and 4i + 2 in word 2i, 4i + 1 and 4i + 3 in word 2i + 1
        uint32_t *mine = team.bins + turn * 64;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t x = (uint32_t)(c[i >> 1] >> (32 * (i & 1)));
            const uint32_t even = __reduce_add_sync(0xffffffffu, x & 0x00ff00ffu);
            const uint32_t odd = __reduce_add_sync(0xffffffffu, (x >> 8) & 0x00ff00ffu);
            if (lane == 0) {
                mine[warp * 8 + 2 * i] = even;
                mine[warp * 8 + 2 * i + 1] = odd;
            }
        }
        __syncthreads();
        uint32_t *all = team.bins + 128 + turn * 64;   // [block][word]
        if (warp == 0) {   // lane (part, word): the block's word, to blocks part and part + 4
            uint32_t v = mine[part * 8 + word] + mine[(part + 4) * 8 + word];
            v += __shfl_xor_sync(0xffffffffu, v, 8);
            v += __shfl_xor_sync(0xffffffffu, v, 16);
#pragma unroll
            for (int i = 0; i < 2; ++i)
                asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(mapa_shared(all + T::rank() * 8 + word, part + 4 * i)), "r"(v)
                             : "memory");
        }
        cluster_sync();
        uint32_t v = all[part * 8 + word] + all[(part + 4) * 8 + word];
        v += __shfl_xor_sync(0xffffffffu, v, 8);
        v += __shfl_xor_sync(0xffffffffu, v, 16);
        // lane b: bin b's count, then how many images lie in bins b .. 15
        const int b = lane & 15;
        const int held = (int)((__shfl_sync(0xffffffffu, v, 2 * (b >> 2) + (b & 1)) >> (16 * ((b >> 1) & 1))) & 0xffffu);
        int upward = held;
#pragma unroll
        for (int o = 1; o < 16; o <<= 1) {
            const int up = __shfl_down_sync(0xffffffffu, upward, o, 16);
            if (b + o < 16) upward += up;
        }
        const uint32_t reach = __ballot_sync(0xffffffffu, upward >= need) & 0xffffu;
        const int digit = 31 - __clz(reach | 1u);
        const int in_bin = __shfl_sync(0xffffffffu, held, digit);
        const int above = __shfl_sync(0xffffffffu, upward, digit) - in_bin;
        if (guess) {
            guess = false;
            if (digit == 0 || digit == 15) {   // somewhere else
                shift = 28;
                continue;
            }
            prefix = (uint32_t)(GUESS + digit) << 24;
        } else {
            prefix |= (uint32_t)digit << shift;
        }
        shift -= 4;
        need -= above;
        if (in_bin == need && prefix != 0) {   // all of them stay: the next smaller image is below prefix
            W = prefix - 1;
            ties = 0;
            return;
        }
    }
    W = prefix;
    ties = need;
}

// The weights of the keys that stay, to wo (which may be w: then a step's reads are before its writes, and a
// key's place is never behind it).
template <class T>
__device__ __forceinline__ void move_weights(T &team, const float *w, const int *src, int rows, float *wo) {
    const int tid = team.thread();
    constexpr int U = 4;
    for (int base = 0; base < rows; base += U * T::ALL) {
        float x[U];
#pragma unroll
        for (int u = 0; u < U; ++u) x[u] = base + u * T::ALL + tid < rows ? w[src[base + u * T::ALL + tid]] : 0.0f;
        if (wo == w) team.sync();
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (base + u * T::ALL + tid < rows) wo[base + u * T::ALL + tid] = x[u];
    }
}

// Chooses among n > budget weights w, at most E a thread: writes the source index of every key that stays to
// src (and kept, if not null) and its weight to wo (which may be w).  Warp k of the team holds the 32 E weights
// from 32 E k on, lane by lane.
template <int E, class T>
__device__ __forceinline__ void choose(T &team, const float *w, int n, int budget, int recent, int *src, int *kept,
                                       float *wo) {
    const int lane = threadIdx.x & 31, first = (team.thread() >> 5) * 32 * E + lane;
    const int old = n - recent, need = budget - recent;   // 0 <= need < old
    // Up to 16 a thread: the weights stay in registers too and go to another buffer from there (20 heads x 9000 keys
    // 21.1 us, 20.1 so; 60 heads with 32 a thread 38.3, 40.4 so).
    constexpr bool DIRECT = E <= 16;
    uint32_t key[E];   // past the older keys: 0, which no candidate reaches
    float raw[E];
#pragma unroll
    for (int j = 0; j < E; ++j) raw[j] = first + 32 * j < (DIRECT ? n : old) ? w[first + 32 * j] : 0.0f;
    uint32_t hi = 0, lo = 0;
#pragma unroll
    for (int j = 0; j < E; ++j) {
        const bool in = first + 32 * j < old;
        key[j] = in ? weight_key(raw[j]) : 0u;
        hi = max(hi, key[j]);
        lo = max(lo, in ? ~key[j] : 0u);
    }
    uint32_t W = 0xffffffffu;
    int ties = 0;
    if constexpr (T::BLOCKS > 1) {
        const int held = (old - first + 31) / 32;   // this thread's older keys
        if (need > 0) find_threshold_radix<E>(team, need, key, E - min(max(held, 0), E), W, ties);
    } else if (need > 0) {
        hi = team.largest(hi);
        lo = ~team.largest(lo);
        find_threshold(need, hi, hi ^ lo, [&](uint32_t cand) {
            int c[4] = {};
#pragma unroll
            for (int j = 0; j < E; ++j) c[j & 3] += key[j] >= cand;
            return team.sum((c[0] + c[1]) + (c[2] + c[3]));
        }, W, ties);
    }
    // number what stays: those above W, the first `ties` equal to W, the recent ones
    int g = 0, e = 0;
    if (T::ALL > 32) {
        int ng = 0, ne = 0;
#pragma unroll
        for (int j = 0; j < E; ++j) {
            const bool in = need > 0 && first + 32 * j < old;
            ng += __popc(__ballot_sync(0xffffffffu, in && key[j] > W));
            if (ties > 0) ne += __popc(__ballot_sync(0xffffffffu, in && key[j] == W));
        }
        team.before(ng, ne, g, e);
    }
    const uint32_t below = (1u << lane) - 1u;
    const int steps = (n - (first - lane) + 31) / 32;   // of this warp that hold keys at all
#pragma unroll
    for (int j = 0; j < E; ++j) {
        if (j >= steps) break;
        const int i = first + 32 * j;
        const bool in = need > 0 && i < old;
        bool stays = in && key[j] > W;
        int at = g;
        const uint32_t mg = __ballot_sync(0xffffffffu, stays);
        at += __popc(mg & below);
        g += __popc(mg);
        if (ties > 0) {
            const bool eq = in && key[j] == W;
            const uint32_t me = __ballot_sync(0xffffffffu, eq);
            const int rank = e + __popc(me & below);   // among the keys equal to W
            stays = stays || (eq && rank < ties);
            at += min(rank, ties);
            e += __popc(me);
        }
        if (i >= old) {
            stays = i < n;
            at = need + i - old;
        }
        if (stays) {
            src[at] = i;
            if (kept) kept[at] = i;
            if (DIRECT && wo != w) wo[at] = raw[j];
        }
    }
    if (DIRECT && wo != w) return;
    team.sync();
    move_weights(team, w, src, budget, wo);
}

// The same for any n, reading the weights again for every bit.
__device__ void choose_long(Team<SEL_THREADS> &team, const float *w, int n, int budget, int recent, int *src, float *wo) {
    const int tid = threadIdx.x, lane = tid & 31;
    const int old = n - recent, need = budget - recent;
    uint32_t W = 0xffffffffu;
    int ties = 0;
    if (need > 0)
        find_threshold(need, 0u, 0xffffffffu, [&](uint32_t cand) {
            int c = 0;
            for (int i = tid; i < old; i += SEL_THREADS) c += weight_key(w[i]) >= cand;
            return team.sum(c);
        }, W, ties);
    int g0 = 0, e0 = 0;
    const uint32_t below = (1u << lane) - 1u;
    for (int base = 0; base < n; base += SEL_THREADS) {
        const int i = base + tid;
        const uint32_t key = i < old ? weight_key(w[i]) : 0u;
        const bool in = need > 0 && i < old, gt = in && key > W, eq = in && key == W;
        const uint32_t mg = __ballot_sync(0xffffffffu, gt), me = __ballot_sync(0xffffffffu, eq);
        int g, e;
        team.before(__popc(mg), __popc(me), g, e);
        g += g0 + __popc(mg & below);
        e += e0 + __popc(me & below);
        int at = -1;
        if (gt || (eq && e < ties)) at = g + min(e, ties);
        if (i >= old && i < n) at = need + i - old;
        if (at >= 0) src[at] = i;
        g0 += team.sum(lane == 0 ? __popc(mg) : 0);
        e0 += team.sum(lane == 0 ? __popc(me) : 0);
    }
    team.sync();
    move_weights(team, w, src, budget, wo);
}

__device__ __forceinline__ int count_of(const EvArgs &p, int set, bool report) {
    int n = p.max_keys;
    if (p.n_keys) {
        const int want = __ldcg(p.n_keys + set);
        n = min(max(want, 0), p.max_keys);
        if (want != n && report) atomicCAS(p.status, 0, WH_EBOUNDS);
    }
    return n;
}

// One head of one set: the block chooses, E keys a thread, then moves.  (A warp that chose among 900 keys took 14.4 us
// for 12 heads, the block 10.3; among 448 9.0 and 8.2.)
template <int E>
__global__ void __launch_bounds__(SM_THREADS) k_evict_small(const EvArgs p) {
    extern __shared__ int src[];   // [budget]
    __shared__ int buf[2 * SM_THREADS / 32];
    pdl_wait();
    pdl_launch_dependents();
    const int h = blockIdx.x, set = blockIdx.y, tid = threadIdx.x;
    const int n = count_of(p, set, h == 0 && tid == 0), rows = min(n, p.budget);
    if (p.n_out && h == 0 && tid == 0) p.n_out[set] = rows;
    const long long sh = (long long)set * p.n_head + h;
    const float *w = p.weight + sh * p.max_keys;
    float *wo = p.weight_out + sh * p.out_keys;
    int *kept = p.kept ? p.kept + sh * p.kept_stride : nullptr;
    const bool all = n <= p.budget;   // everything stays
    if (all) {
        for (int i = tid; i < n; i += SM_THREADS) {
            src[i] = i;
            if (kept) kept[i] = i;
            if (!p.in_place) wo[i] = w[i];
        }
    } else {
        Team<SM_THREADS> team{buf, nullptr, 0, nullptr};
        choose<E>(team, w, n, p.budget, p.recent, src, kept, wo);
    }
    if (all && p.in_place) return;
    __syncthreads();
    // rows in steps of U * SM_THREADS / 8; thread x takes piece x % 8 of keys and values
    constexpr int U = 4, STEP = SM_THREADS / 8;
    const long long in0 = (long long)set * p.set_stride + h * 64 + 8 * (tid & 7);
    const long long to0 = (long long)set * p.out_set_stride + h * 64 + 8 * (tid & 7);
    for (int base = tid >> 3; base < (rows + U * STEP - 1) / (U * STEP) * (U * STEP); base += U * STEP) {
        uint4 a[U], b[U];
        int t[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int j = base + u * STEP;
            t[u] = j < rows ? src[j] : -1;
            if (p.in_place && t[u] == j) t[u] = -1;   // where it was
            if (t[u] >= 0) {
                a[u] = __ldcg(reinterpret_cast<const uint4 *>(p.k + in0 + t[u] * p.row_stride));
                b[u] = __ldcg(reinterpret_cast<const uint4 *>(p.v + in0 + t[u] * p.row_stride));
            }
        }
        if (p.in_place) __syncthreads();   // (the trip count is the block's)
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (t[u] >= 0) {
                const long long to = to0 + (long long)(base + u * STEP) * p.out_row_stride;
                *reinterpret_cast<uint4 *>(p.k_out + to) = a[u];
                *reinterpret_cast<uint4 *>(p.v_out + to) = b[u];
            }
    }
}

// Chooses only: a warp (of four), a block or a cluster of CTAS blocks per head and set.
// (Four blocks of a cluster to an SM with up to 16 weights a thread, 72 clusters at once instead of 36: 40 heads x
// 30000 keys 40.3 us -> 35.8; two with 32 a thread.)
template <int CHOOSERS, int E, int CTAS = 1>
__global__ void __launch_bounds__(CHOOSERS == 32 ? 128 : CHOOSERS, CTAS == 1 ? 0 : E <= 16 ? 4 : 2) k_evict_select(const EvArgs p) {
    __shared__ int buf[2 * SEL_THREADS / 32], peers[2 * CTAS];
    __shared__ uint32_t bins[CTAS > 1 ? 256 : 1];
    pdl_wait();
    pdl_launch_dependents();
    Team<CHOOSERS, CTAS> team{buf, peers, 0, bins};
    const int tid = team.thread();
    const long long sh = CHOOSERS == 32 ? blockIdx.x * 4LL + (threadIdx.x >> 5) : blockIdx.x / CTAS;
    if (sh >= (long long)p.n_set * p.n_head) return;
    const int set = (int)sh / p.n_head, h = (int)sh - set * p.n_head;
    const int n = count_of(p, set, h == 0 && tid == 0);
    if (h == 0 && tid == 0) p.count[set] = n;
    const float *w = p.weight + sh * p.max_keys;
    float *wo = p.weight_out + sh * p.out_keys;
    int *src = p.kept + sh * p.kept_stride;
    if (n <= p.budget) {   // everything stays
        for (int i = tid; i < n; i += team.ALL) {
            src[i] = i;
            if (!p.in_place) wo[i] = w[i];
        }
    } else if constexpr (E > 0) {
        if (CTAS > 1) team.sync();   // every block of the cluster is there before its memory is written
        choose<E>(team, w, n, p.budget, p.recent, src, nullptr, wo);
        if (CTAS > 1) team.sync();   // and none leaves before the last number was read
    } else {
        choose_long(team, w, n, p.budget, p.recent, src, wo);
    }
}

// Row j of head h of a set <- row kept[j] of the cache, for keys and values; other buffers.  I counts 16-byte pieces.
template <class I>
__global__ void __launch_bounds__(MV_THREADS) k_evict_move(const EvArgs p) {
    pdl_wait();
    const int set = blockIdx.y, n = min(__ldcg(p.count + set), p.budget);
    if (blockIdx.x == 0 && threadIdx.x == 0) p.n_out[set] = n;
    const int per_row = p.n_head * 8;   // 16-byte pieces of a row
    const I todo = (I)n * per_row, base = (I)blockIdx.x * MV_PIECES + threadIdx.x;
    constexpr int U = MV_PIECES / MV_THREADS;
    int x[U], j[U], t[U];
    uint4 a[U], b[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const I i = base + u * MV_THREADS;
        t[u] = -1;
        if (i < todo) {
            j[u] = sizeof(I) == 4 ? p.by_row.of((int)i) : (int)(i / per_row);
            x[u] = (int)(i - (I)j[u] * per_row);
            t[u] = __ldcg(p.kept + ((long long)set * p.n_head + (x[u] >> 3)) * p.kept_stride + j[u]);
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
        if (t[u] >= 0) {
            const long long from = (long long)set * p.set_stride + (long long)t[u] * p.row_stride + 8 * x[u];
            a[u] = __ldcg(reinterpret_cast<const uint4 *>(p.k + from));
            b[u] = __ldcg(reinterpret_cast<const uint4 *>(p.v + from));
        }
#pragma unroll
    for (int u = 0; u < U; ++u)
        if (t[u] >= 0) {
            const long long to = (long long)set * p.out_set_stride + (long long)j[u] * p.out_row_stride + 8 * x[u];
            *reinterpret_cast<uint4 *>(p.k_out + to) = a[u];
            *reinterpret_cast<uint4 *>(p.v_out + to) = b[u];
        }
}

// The same within the cache: the blocks of a cluster per (head, set, keys or values).  A step's rows are all read
// before any is written, and no later row comes from where it writes.
template <int CTAS>
__global__ void __launch_bounds__(SH_THREADS, SH_RESIDENT) k_evict_shift(const EvArgs p) {
    pdl_wait();
    const int item = blockIdx.x / CTAS, h = item % p.n_head, set = item / p.n_head, rank = blockIdx.x % CTAS;
    const int n0 = __ldcg(p.count + set), n = min(n0, p.budget), place = rank * SH_THREADS + threadIdx.x;
    if (h == 0 && blockIdx.y == 0 && place == 0) p.n_out[set] = n;
    if (n0 <= p.budget) return;
    __nv_bfloat16 *x = (blockIdx.y ? p.v_out : p.k_out) + (long long)set * p.set_stride + h * 64 + 8 * (threadIdx.x & 7);
    const int *src = p.kept + ((long long)set * p.n_head + h) * p.kept_stride;
    constexpr int U = SH_ROWS, STEP = CTAS * SH_THREADS / 8;
    for (int base = place >> 3; base < (n + U * STEP - 1) / (U * STEP) * (U * STEP); base += U * STEP) {
        int t[U];
        uint4 a[U];
#pragma unroll
        for (int u = 0; u < U; ++u) t[u] = base + u * STEP < n ? __ldcg(src + base + u * STEP) : -1;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (t[u] == base + u * STEP) t[u] = -1;   // where it was
            if (t[u] >= 0) a[u] = __ldcg(reinterpret_cast<const uint4 *>(x + (long long)t[u] * p.row_stride));
        }
        if (CTAS > 1) {
            __syncwarp();
            cluster_sync();
        } else {
            __syncthreads();
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (t[u] >= 0) *reinterpret_cast<uint4 *>(x + (long long)(base + u * STEP) * p.row_stride) = a[u];
    }
}

// The new counts, where they overwrite the old ones that k_evict_small's blocks read.
__global__ void k_evict_counts(const EvArgs p, int *n_out) {
    pdl_wait();
    for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < p.n_set; i += gridDim.x * blockDim.x)
        n_out[i] = min(count_of(p, i, false), p.budget);
}

// The largest clusters that are resident at once and have rows for all their blocks (200 heads 9000 keys -> 3000: 234 us,
// copy included, 245 with clusters twice as large).
int launch_shift(const EvArgs &a, int most, long long items, cudaStream_t s) {
    const int steps = (most + SH_ROWS * SH_THREADS / 8 - 1) / (SH_ROWS * SH_THREADS / 8);
    int ctas = 8;
    while (ctas > 1 && (2 * items * ctas > SH_RESIDENT * 152 || ctas / 2 >= steps)) ctas /= 2;
    auto *kernel = ctas == 8 ? k_evict_shift<8> : ctas == 4 ? k_evict_shift<4> : ctas == 2 ? k_evict_shift<2> : k_evict_shift<1>;
    return launch_ex(kernel, dim3((unsigned)(items * ctas), 2), SH_THREADS, 0, ctas, true, s, a);
}

bool one_kernel(int n_set, int n_head, int max_keys, int budget, bool in_place) {
    const long long items = (long long)n_set * n_head;
    return max_keys <= SM_MOST && items <= SM_HEADS &&
           (budget <= SM_ROWS || max_keys <= SM_ROWS || (in_place && 2 * items >= SM_HEADS));
}

// Whether no row of one set's keys (row t at t * row) meets a row of another's (at d + t * row).
bool rows_apart(int64_t d, int64_t row, int64_t width, int64_t span) {
    const int64_t at = (d % row + row) % row;
    return d >= span || d <= -span || (at >= width && at <= row - width);
}

// What a caller may pass as the cache or as where it goes: no two sets, and no key and value, share memory.
bool keys_ok(const wh_keys *s, int n_kv) {
    if (!s || s->n_set < 1 || s->n_set > 65535 || s->max_keys < 1 || s->max_keys > (1 << 30)) return false;
    const int64_t row = s->row_stride, set = s->set_stride, width = 64LL * n_kv;
    if (row < width || row % 8 != 0 || set < 0 || set % 8 != 0) return false;
    if (!fits(s->k, 16) || !fits(s->v, 16) || !fits(s->weight, 4) || (s->n_keys && !fits(s->n_keys, 4))) return false;
    const int64_t span = (s->max_keys - 1) * row + width, last = s->n_set - 1;
    if (last > 0 && set == 0) return false;
    for (int64_t i = 1; i <= last && i * set < span; ++i)   // (sets one after the other: none to look at)
        if (!rows_apart(i * set, row, width, span)) return false;
    const int64_t gap = s->v - s->k;
    int64_t from = -last, to = last;   // value sets against a key set, by how many sets they are on
    if (last > 0) {
        from = std::max(from, (-span - gap) / set - 1);
        to = std::min(to, (span - gap) / set + 1);
    }
    for (int64_t i = from; i <= to; ++i)
        if (!rows_apart(gap + i * set, row, width, span)) return false;
    return true;
}

struct Span {
    uintptr_t a, b;
};
Span span_of(const void *p, long long elements, int size) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    return {a, a + (uintptr_t)elements * size};
}
bool meet(Span x, Span y) { return x.a < y.b && y.a < x.b; }

}  // namespace
}  // namespace wh

using namespace wh;

extern "C" size_t wh_cache_evict_workspace(int n_set, int n_kv_head, int max_keys, int budget) {
    if (n_set < 1 || n_set > 65535 || n_kv_head < 1 || n_kv_head > 1024 || max_keys < 1 || max_keys > (1 << 30) ||
        budget < 1 || budget > (1 << 30) || one_kernel(n_set, n_kv_head, max_keys, budget, false))
        return 0;
    return up256((size_t)n_set * 4) + up256((size_t)n_set * n_kv_head * std::min(budget, max_keys) * 4);
}

extern "C" int wh_cache_evict(const wh_keys *cache, int n_kv_head, int budget, int recent, const wh_keys *out, int *n_out,
                              int *kept, void *workspace, size_t ws_bytes, void *stream) {
    if (n_kv_head < 1 || n_kv_head > 1024 || budget < 1 || budget > (1 << 30) || recent < 0 || recent > budget)
        return WH_EINVAL;
    if (!keys_ok(cache, n_kv_head) || !fits(n_out, 4) || (kept && !fits(kept, 4)) ||
        (workspace && !fits(workspace, 256)))
        return WH_EINVAL;
    if (out) {
        if (!keys_ok(out, n_kv_head) || out->n_set != cache->n_set) return WH_EINVAL;
        if (out->max_keys < (budget < cache->max_keys ? budget : cache->max_keys)) return WH_EINVAL;
        // other buffers, or the cache itself (out NULL): nothing between
        const auto rows = [&](const wh_keys *s, const wh_bf16 *x) {
            return span_of(x, (s->n_set - 1) * s->set_stride + (s->max_keys - 1) * s->row_stride + 64LL * n_kv_head, 2);
        };
        const auto weights = [&](const wh_keys *s) {
            return span_of(s->weight, (long long)s->n_set * n_kv_head * s->max_keys, 4);
        };
        if (meet(weights(cache), weights(out))) return WH_EINVAL;
        // (k and v of one wh_keys may share rows, as [K | V] do, and so may the two of out; but no row of
        // out may be a row of the cache)
        const Span in[2] = {rows(cache, cache->k), rows(cache, cache->v)}, to[2] = {rows(out, out->k), rows(out, out->v)};
        for (const Span &x : in)
            for (const Span &y : to)
                if (meet(x, y)) return WH_EINVAL;
    }
    if (cache->n_keys && n_out != cache->n_keys && meet(span_of(n_out, cache->n_set, 4), span_of(cache->n_keys, cache->n_set, 4)))
        return WH_EINVAL;
    size_t need = wh_cache_evict_workspace(cache->n_set, n_kv_head, cache->max_keys, budget);
    if (kept && need) need = up256((size_t)cache->n_set * 4);   // the indices go there
    if ((workspace ? ws_bytes : 0) < need) return WH_ENOSPC;
    DevCtl ctl;
    int num_sms = 0;
    if (int rc = device_ctl(&ctl, &num_sms)) return rc;
    const wh_keys *o = out ? out : cache;
    EvArgs a = {};
    a.k = reinterpret_cast<const __nv_bfloat16 *>(cache->k);
    a.v = reinterpret_cast<const __nv_bfloat16 *>(cache->v);
    a.k_out = reinterpret_cast<__nv_bfloat16 *>(const_cast<wh_bf16 *>(o->k));
    a.v_out = reinterpret_cast<__nv_bfloat16 *>(const_cast<wh_bf16 *>(o->v));
    a.row_stride = cache->row_stride;
    a.set_stride = cache->set_stride;
    a.out_row_stride = o->row_stride;
    a.out_set_stride = o->set_stride;
    a.weight = cache->weight;
    a.weight_out = o->weight;
    a.n_keys = cache->n_keys;
    a.n_out = n_out;
    a.count = static_cast<int *>(workspace);
    a.kept_stride = kept ? budget : std::min(budget, cache->max_keys);
    a.max_keys = cache->max_keys;
    a.out_keys = o->max_keys;
    a.n_set = cache->n_set;
    a.n_head = n_kv_head;
    a.budget = budget;
    a.recent = recent;
    a.in_place = out == nullptr;
    a.by_row = divisor(n_kv_head * 8);
    a.status = ctl.status;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int most = budget < a.max_keys ? budget : a.max_keys;
    const dim3 heads(n_kv_head, a.n_set);
    int rc;
    trace_begin(TR_DEC_OTHER, s);
    const long long items = (long long)n_kv_head * a.n_set;
    if (one_kernel(a.n_set, n_kv_head, a.max_keys, budget, a.in_place)) {
        const bool same = n_out == a.n_keys;
        a.kept = kept;
        a.n_out = same ? nullptr : n_out;
        auto *kernel = a.max_keys <= 512 ? k_evict_small<2> : a.max_keys <= 1024 ? k_evict_small<4> : k_evict_small<8>;
        rc = launch_ex(kernel, heads, SM_THREADS, most * (int)sizeof(int), 1, true, s, a);
        if (!rc && same) rc = launch_ex(k_evict_counts, dim3((a.n_set + 255) / 256), 256, 0, 1, true, s, a, n_out);
    } else {
        a.kept = kept ? kept : reinterpret_cast<int *>(static_cast<uint8_t *>(workspace) + up256((size_t)cache->n_set * 4));
        const dim3 warps((unsigned)((items + 3) / 4)), blocks((unsigned)items);
        if (a.max_keys <= 512)
            rc = launch_ex(k_evict_select<32, 16>, warps, 128, 0, 1, true, s, a);
        else if (a.max_keys <= 1024)
            rc = launch_ex(k_evict_select<32, 32>, warps, 128, 0, 1, true, s, a);
        else if (a.max_keys <= 2048)
            rc = launch_ex(k_evict_select<256, 8>, blocks, 256, 0, 1, true, s, a);
        else if (a.max_keys <= 4096)
            rc = launch_ex(k_evict_select<256, 16>, blocks, 256, 0, 1, true, s, a);
        else if (a.max_keys <= 8192)
            rc = launch_ex(k_evict_select<512, 16>, blocks, 512, 0, 1, true, s, a);
        else if (a.max_keys <= 16384 && items <= SEL_SPREAD)
            rc = launch_ex(k_evict_select<256, 8, SEL_CTAS>, dim3((unsigned)(items * SEL_CTAS)), 256, 0, SEL_CTAS, true, s, a);
        else if (a.max_keys <= 16384)
            rc = launch_ex(k_evict_select<SEL_THREADS, 16>, blocks, SEL_THREADS, 0, 1, true, s, a);
        else if (a.max_keys <= 32768 && items <= SEL_SPREAD)
            rc = launch_ex(k_evict_select<256, 16, SEL_CTAS>, dim3((unsigned)(items * SEL_CTAS)), 256, 0, SEL_CTAS, true, s, a);
        else if (a.max_keys <= 32768)
            rc = launch_ex(k_evict_select<SEL_THREADS, 32>, blocks, SEL_THREADS, 0, 1, true, s, a);
        else if (a.max_keys < 65536)
            rc = launch_ex(k_evict_select<256, 32, SEL_CTAS>, dim3((unsigned)(items * SEL_CTAS)), 256, 0, SEL_CTAS, true, s, a);
        else
            rc = launch_ex(k_evict_select<SEL_THREADS, 0>, blocks, SEL_THREADS, 0, 1, true, s, a);
        if (!rc && a.in_place) {
            rc = launch_shift(a, most, items, s);
        } else if (!rc) {
            const long long pieces = (long long)most * n_kv_head * 8;
            rc = launch_ex(pieces > 0x7fff0000LL ? k_evict_move<long long> : k_evict_move<int>,
                           dim3((unsigned)((pieces + MV_PIECES - 1) / MV_PIECES), a.n_set), MV_THREADS, 0, 1, true, s, a);
        }
    }
    const double held = (double)a.n_set * n_kv_head;
    trace_end(TR_DEC_OTHER, s, 0.0, held * (4.0 * a.max_keys + 520.0 * most));
    return rc ? rc : cudaGetLastError() == cudaSuccess ? WH_OK : WH_ECUDA;
}
