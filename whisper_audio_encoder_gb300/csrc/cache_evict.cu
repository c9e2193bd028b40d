// Eviction from key/value caches by accumulated attention weight.
//
// Each head of each set keeps, of its n keys, the last `recent` and of the others the budget - recent
// with the largest weight (ties: the lowest index), in their order, moved together at the front.
//
// k_evict_select: one block per (head, set) finds the weight W below which no older key stays -- a
// binary search over the bits of an order-preserving integer image of the weights, counting how many
// are at least the candidate -- then numbers the keys that stay in order: those above W, the first few
// equal to W, the recent ones.  It writes the source index of each and its weight.
// k_evict_move / k_evict_shift: copy the rows, 16 bytes a thread, to other buffers or within the cache.
#include "common.cuh"
#include "internal.h"

namespace wh {
namespace {

constexpr int EV_THREADS = 256;
constexpr int EV_WARPS = EV_THREADS / 32;
constexpr int MV_THREADS = 256;
constexpr int MV_ROWS = 16;      // rows of one head that a block of k_evict_move copies at a time
constexpr int SH_THREADS = 256;
constexpr int SH_ROWS = SH_THREADS / 8;

struct EvArgs {
    const __nv_bfloat16 *k, *v;
    __nv_bfloat16 *k_out, *v_out;
    long long row_stride, set_stride, out_row_stride, out_set_stride;
    const float *weight;
    float *weight_out;
    const int *n_keys;
    int *n_out;
    int *kept;                 // [n_set][n_head][budget]: source index of every key that stays
    int *count;                // [n_set]: keys before, as clamped
    int max_keys, out_keys, n_set, n_head, budget, recent, in_place;
    int *status;
};

// Larger weight, larger image; -0 as 0; NaN below everything.
__device__ __forceinline__ uint32_t weight_key(float w) {
    if (w != w) return 0u;
    const uint32_t u = __float_as_uint(w + 0.0f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Sum over the block, the same in every thread (two barriers).
__device__ __forceinline__ int block_sum(int x, int *buf) {
    x = __reduce_add_sync(0xffffffffu, x);
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = x;
    __syncthreads();
    int s = 0;
#pragma unroll
    for (int w = 0; w < EV_WARPS; ++w) s += buf[w];
    __syncthreads();
    return s;
}

__global__ void __launch_bounds__(EV_THREADS) k_evict_select(const EvArgs p) {
    __shared__ int buf[EV_WARPS], wgt[EV_WARPS], weq[EV_WARPS];
    pdl_wait();
    pdl_launch_dependents();
    const int h = blockIdx.x, set = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int n = p.max_keys;
    if (p.n_keys) {
        const int want = __ldg(p.n_keys + set);
        n = min(max(want, 0), p.max_keys);
        if (want != n && h == 0 && tid == 0) atomicCAS(p.status, 0, WH_EBOUNDS);
    }
    if (h == 0 && tid == 0) p.count[set] = n;
    const long long sh = (long long)set * p.n_head + h;
    const float *w = p.weight + sh * p.max_keys;
    float *wo = p.weight_out + sh * p.out_keys;
    int *src = p.kept + sh * p.budget;
    if (n <= p.budget) {   // everything stays
        for (int i = tid; i < n; i += EV_THREADS) {
            src[i] = i;
            if (!p.in_place) wo[i] = __ldg(w + i);
        }
        return;
    }
    const int old = n - p.recent, need = p.budget - p.recent;   // 0 <= need < old
    // the need-th largest image of the older keys: the largest W with at least need images >= W
    uint32_t W = 0;
    if (need > 0) {
        for (int bit = 31; bit >= 0; --bit) {
            const uint32_t cand = W | (1u << bit);
            int c = 0;
            for (int i = tid; i < old; i += EV_THREADS) c += weight_key(w[i]) >= cand;
            if (block_sum(c, buf) >= need) W = cand;
        }
    } else {
        W = 0xffffffffu;
    }
    int above = 0;
    for (int i = tid; i < old; i += EV_THREADS) above += weight_key(w[i]) > W;
    above = need > 0 ? block_sum(above, buf) : 0;
    const int ties = need - above;   // how many of the keys with image W stay
    // number what stays, EV_THREADS keys at a time; within the cache every key moves towards the front, so
    // writing behind the reads is safe
    int gt0 = 0, eq0 = 0;
    for (int base = 0; base < old; base += EV_THREADS) {
        const int i = base + tid;
        const float x = i < old ? w[i] : 0.0f;
        const uint32_t key = weight_key(x);
        const bool gt = i < old && need > 0 && key > W, eq = i < old && need > 0 && key == W;
        const uint32_t mg = __ballot_sync(0xffffffffu, gt), me = __ballot_sync(0xffffffffu, eq);
        if (lane == 0) {
            wgt[warp] = __popc(mg);
            weq[warp] = __popc(me);
        }
        __syncthreads();
        int g = gt0, e = eq0;
        for (int j = 0; j < EV_WARPS; ++j) {
            if (j < warp) {
                g += wgt[j];
                e += weq[j];
            }
            gt0 += wgt[j];
            eq0 += weq[j];
        }
        const uint32_t below = (1u << lane) - 1u;
        g += __popc(mg & below);
        e += __popc(me & below);
        if (gt || (eq && e < ties)) {
            const int at = g + min(e, ties);
            src[at] = i;
            wo[at] = x;
        }
        __syncthreads();
    }
    for (int base = 0; base < p.recent; base += EV_THREADS) {
        const int i = base + tid;
        const float x = i < p.recent ? w[old + i] : 0.0f;
        __syncthreads();
        if (i < p.recent) {
            src[need + i] = old + i;
            wo[need + i] = x;
        }
    }
}

// Row j of head h of a set <- row kept[j] of the cache, for keys and values; other buffers.
__global__ void __launch_bounds__(MV_THREADS) k_evict_move(const EvArgs p) {
    pdl_wait();
    const int set = blockIdx.y, n = min(__ldcg(p.count + set), p.budget);
    if (blockIdx.x == 0 && threadIdx.x == 0) p.n_out[set] = n;
    const int j0 = blockIdx.x * MV_ROWS, rows = min(MV_ROWS, n - j0);
    if (rows <= 0) return;
    const int per_row = p.n_head * 8;   // 16-byte pieces of a row
    for (int i = threadIdx.x; i < rows * per_row; i += MV_THREADS) {
        const int j = j0 + i / per_row, x = i % per_row, h = x >> 3;
        const int t = __ldcg(p.kept + ((long long)set * p.n_head + h) * p.budget + j);
        const long long from = (long long)set * p.set_stride + (long long)t * p.row_stride + 8 * x;
        const long long to = (long long)set * p.out_set_stride + (long long)j * p.out_row_stride + 8 * x;
        const uint4 a = __ldg(reinterpret_cast<const uint4 *>(p.k + from));
        const uint4 b = __ldg(reinterpret_cast<const uint4 *>(p.v + from));
        *reinterpret_cast<uint4 *>(p.k_out + to) = a;
        *reinterpret_cast<uint4 *>(p.v_out + to) = b;
    }
}

// The same within the cache: one block per (head, set, keys or values) goes up the rows.  A row's source
// lies at or behind it, so what later rows read is never overwritten; the barrier holds back the writes of
// a step until its reads are done.
__global__ void __launch_bounds__(SH_THREADS) k_evict_shift(const EvArgs p) {
    pdl_wait();
    const int h = blockIdx.x, set = blockIdx.y, n0 = __ldcg(p.count + set), n = min(n0, p.budget);
    if (h == 0 && blockIdx.z == 0 && threadIdx.x == 0) p.n_out[set] = n;
    if (n0 <= p.budget) return;
    __nv_bfloat16 *x = (blockIdx.z ? p.v_out : p.k_out) + (long long)set * p.set_stride + h * 64 + 8 * (threadIdx.x & 7);
    const int *src = p.kept + ((long long)set * p.n_head + h) * p.budget;
    for (int base = 0; base < n; base += SH_ROWS) {
        const int j = base + (threadIdx.x >> 3);
        int t = j;
        uint4 a = make_uint4(0, 0, 0, 0);
        if (j < n) {
            t = __ldcg(src + j);
            if (t != j) a = *reinterpret_cast<const uint4 *>(x + (long long)t * p.row_stride);
        }
        __syncthreads();
        if (t != j) *reinterpret_cast<uint4 *>(x + (long long)j * p.row_stride) = a;
    }
}

size_t up256e(size_t x) { return (x + 255) & ~(size_t)255; }

bool fits(const void *p, size_t a) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// What a caller may pass as the cache or as where it goes: no two sets, and no key and value, share memory.
bool keys_ok(const wh_keys *s, int n_kv) {
    if (!s || s->n_set < 1 || s->n_set > 65535 || s->max_keys < 1 || s->max_keys > (1 << 30)) return false;
    const int64_t row = s->row_stride, width = 64LL * n_kv;
    if (row < width || row % 8 != 0 || s->set_stride < 0 || s->set_stride % 8 != 0) return false;
    const bool apart = s->set_stride >= (s->max_keys - 1) * row + width;                            // [set][key]
    const bool beside = s->set_stride >= width && (s->n_set - 1) * s->set_stride + width <= row;    // [key][set]
    if (s->n_set > 1 && !apart && !beside) return false;
    if (!fits(s->k, 16) || !fits(s->v, 16) || !fits(s->weight, 4) || (s->n_keys && !fits(s->n_keys, 4))) return false;
    const int64_t end = (s->n_set - 1) * s->set_stride + (s->max_keys - 1) * row + width;
    const int64_t gap = s->v > s->k ? s->v - s->k : s->k - s->v;
    return gap >= end || (gap % row >= width && gap % row <= row - width);                          // [K | V] rows
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

extern "C" size_t wh_cache_evict_workspace(int n_set, int n_kv_head, int budget) {
    if (n_set < 1 || n_set > 65535 || n_kv_head < 1 || n_kv_head > 1024 || budget < 1 || budget > (1 << 30)) return 0;
    return up256e((size_t)n_set * 4) + up256e((size_t)n_set * n_kv_head * budget * 4);
}

extern "C" int wh_cache_evict(const wh_keys *cache, int n_kv_head, int budget, int recent, const wh_keys *out, int *n_out,
                              int *kept, void *workspace, size_t ws_bytes, void *stream) {
    if (n_kv_head < 1 || n_kv_head > 1024 || budget < 1 || budget > (1 << 30) || recent < 0 || recent > budget)
        return WH_EINVAL;
    if (!keys_ok(cache, n_kv_head) || !fits(n_out, 4) || (kept && !fits(kept, 4)) || !fits(workspace, 256)) return WH_EINVAL;
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
    if (ws_bytes < wh_cache_evict_workspace(cache->n_set, n_kv_head, budget)) return WH_ENOSPC;
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
    a.kept = kept ? kept : reinterpret_cast<int *>(static_cast<uint8_t *>(workspace) + up256e((size_t)cache->n_set * 4));
    a.max_keys = cache->max_keys;
    a.out_keys = o->max_keys;
    a.n_set = cache->n_set;
    a.n_head = n_kv_head;
    a.budget = budget;
    a.recent = recent;
    a.in_place = out == nullptr;
    a.status = ctl.status;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    trace_begin(TR_DEC_OTHER, s);
    k_evict_select<<<dim3(n_kv_head, a.n_set), EV_THREADS, 0, s>>>(a);
    count_launch();
    cudaLaunchConfig_t lc = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    lc.attrs = attr;
    lc.numAttrs = 1;
    lc.stream = s;
    cudaError_t e;
    if (a.in_place) {
        lc.gridDim = dim3(n_kv_head, a.n_set, 2);
        lc.blockDim = dim3(SH_THREADS);
        e = cudaLaunchKernelEx(&lc, k_evict_shift, a);
    } else {
        const int most = budget < a.max_keys ? budget : a.max_keys;
        lc.gridDim = dim3((most + MV_ROWS - 1) / MV_ROWS, a.n_set);
        lc.blockDim = dim3(MV_THREADS);
        e = cudaLaunchKernelEx(&lc, k_evict_move, a);
    }
    count_launch();
    const double held = (double)a.n_set * n_kv_head;
    trace_end(TR_DEC_OTHER, s, 0.0, held * (4.0 * a.max_keys + 520.0 * (budget < a.max_keys ? budget : a.max_keys)));
    return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? WH_OK : WH_ECUDA;
}
