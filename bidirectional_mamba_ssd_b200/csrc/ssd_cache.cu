// Pages of a pool of cached states, (layers, nslots, page): copies, forks and
// clearings in the order they are listed, and the compaction of a pool with the
// fewest moves. Both only move bytes (two pages' worth a pair, one where a page
// is cleared), so the floor is the copy bandwidth.
//
// Work items are (layer, kChunk bytes of the page, kGroup pairs). A thread owns
// the same 16 bytes of the page in every pair of a group and holds the group's
// loads in flight together. Pairs that stand apart (no page written twice, none
// both read and written) spread over the groups; otherwise one thread applies
// the whole list to its 16 bytes in order, which is the order's meaning and
// needs no synchronisation.
#include <stdint.h>

#include "ssd_causal.h"
#include "ssd_kernels.h"

namespace ssd {
namespace {

constexpr int kThreads = 256;
constexpr int kGroup = 8;

__device__ __forceinline__ uint4 zero_of(uint4) { return make_uint4(0, 0, 0, 0); }
__device__ __forceinline__ uint32_t zero_of(uint32_t) { return 0u; }
__device__ __forceinline__ uint8_t zero_of(uint8_t) { return 0; }

// The pairs i in [0, m) of a group (m <= kGroup) on element e of one layer's
// pages: src[i] < 0 clears dst[i], dst[i] < 0 leaves the pair out. `apart`: the
// loads may all go ahead of the stores.
template <typename V>
__device__ __forceinline__ void move_group(V *layer, long long elems, long long e, const int *src, const int *dst,
                                           int m, bool apart) {
    if (apart) {
        V v[kGroup];
#pragma unroll
        for (int i = 0; i < kGroup; ++i) {
            if (i < m && dst[i] >= 0) {
                if (src[i] < 0) v[i] = zero_of(V());
                else if (i > 0 && dst[i - 1] >= 0 && src[i] == src[i - 1]) v[i] = v[i > 0 ? i - 1 : 0];   // a fork reads its source once
                else v[i] = layer[src[i] * elems + e];
            }
        }
#pragma unroll
        for (int i = 0; i < kGroup; ++i)
            if (i < m && dst[i] >= 0) layer[dst[i] * elems + e] = v[i];
    } else {
        for (int i = 0; i < m; ++i)
            if (dst[i] >= 0) layer[dst[i] * elems + e] = src[i] < 0 ? zero_of(V()) : layer[src[i] * elems + e];
    }
}

// A pair of the caller's list: out-of-range indices leave it out (and are
// reported), so do -1 destinations and copies of a page onto itself.
__device__ __forceinline__ void read_pair(const CacheArgs &a, int i, int &s, int &d, bool &bad) {
    s = a.src[i];
    d = a.dst[i];
    bad = s < -1 || s >= a.nslots || d < -1 || d >= a.nslots;
    if (bad || s == d) d = -1;
}

template <typename V>
__global__ void __launch_bounds__(kThreads)
cache_copy_kernel(const CacheArgs a) {
    extern __shared__ uint32_t map[];      // written pages, one bit each
    __shared__ int ps[kGroup], pd[kGroup];
    const int tid = threadIdx.x;
    const long long elems = a.page_bytes / (long long)sizeof(V);
    const long long chunks = (elems + kThreads - 1) / kThreads;
    // do the pairs stand apart?
    for (int w = tid; w < (a.nslots + 31) / 32; w += kThreads) map[w] = 0u;
    __syncthreads();
    bool clash = false;
    for (int i = tid; i < a.n; i += kThreads) {
        int s, d;
        bool bad;
        read_pair(a, i, s, d, bad);
        if (bad && blockIdx.x == 0) atomicOr(&a.status->flags, kFlagIndex);
        if (d >= 0) clash |= (atomicOr(&map[d >> 5], 1u << (d & 31)) >> (d & 31)) & 1u;
    }
    __syncthreads();
    for (int i = tid; i < a.n; i += kThreads) {
        int s, d;
        bool bad;
        read_pair(a, i, s, d, bad);
        if (d >= 0 && s >= 0) clash |= (map[s >> 5] >> (s & 31)) & 1u;
    }
    clash = __syncthreads_or(clash);
    const int groups = clash ? 1 : (a.n + kGroup - 1) / kGroup;
    const long long items = (long long)a.layers * chunks * groups;
    for (long long it = blockIdx.x; it < items; it += gridDim.x) {
        // the chunks of a page run fastest: neighbouring CTAs stream one page
        const long long c = it % chunks;
        const int grp = (int)((it / chunks) % groups);
        const int layer = (int)(it / chunks / groups);
        V *base = static_cast<V *>(a.pool) + (long long)layer * a.nslots * elems;
        const long long e = c * kThreads + tid;
        for (int i0 = grp * kGroup; i0 < (clash ? a.n : min(a.n, (grp + 1) * kGroup)); i0 += kGroup) {
            const int m = min(kGroup, a.n - i0);
            __syncthreads();
            if (tid < m) {
                bool bad;
                read_pair(a, i0 + tid, ps[tid], pd[tid], bad);
            }
            __syncthreads();
            if (e < elems) move_group(base, elems, e, ps, pd, m, !clash);
        }
    }
}

// k-th (from 0) set bit (ONES) or clear bit of the map, `before[w]` the set
// bits ahead of word w.
template <bool ONES>
__device__ __forceinline__ int select_bit(const uint32_t *map, const int *before, int words, int k) {
    int lo = 0, hi = words - 1;            // last word with fewer than k + 1 such bits ahead
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        const int ahead = ONES ? before[mid] : 32 * mid - before[mid];
        if (ahead <= k) lo = mid;
        else hi = mid - 1;
    }
    int r = k - (ONES ? before[lo] : 32 * lo - before[lo]);
    uint32_t bits = ONES ? map[lo] : ~map[lo];
    for (; r > 0; --r) bits &= bits - 1;
    return lo * 32 + __ffs(bits) - 1;
}

// Every CTA finds the moves by itself (a map of the live pages and its word
// sums in shared memory): the k-th page from `live` on that is in use goes to
// the k-th free page below `live`. No page is both read and written.
template <typename V>
__global__ void __launch_bounds__(kThreads)
cache_compact_kernel(const CacheArgs a) {
    extern __shared__ uint32_t map[];
    __shared__ int ps[kGroup], pd[kGroup], part[kThreads], sum_live, sum_moves;
    const int tid = threadIdx.x;
    const int words = (a.nslots + 31) / 32;
    int *before = reinterpret_cast<int *>(map + words);
    for (int w = tid; w < words; w += kThreads) map[w] = 0u;
    __syncthreads();
    for (int i = tid; i < a.rows; i += kThreads) {
        const int s = a.table[i];
        if (s >= 0 && s < a.nslots) atomicOr(&map[s >> 5], 1u << (s & 31));
        else if (s != -1 && blockIdx.x == 0) atomicOr(&a.status->flags, kFlagIndex);
    }
    __syncthreads();
    // exclusive sums of the words' set bits: a run of words per thread, then the runs
    const int run = (words + kThreads - 1) / kThreads, w0 = min(words, tid * run), w1 = min(words, w0 + run);
    int mine = 0;
    for (int w = w0; w < w1; ++w) mine += __popc(map[w]);
    part[tid] = mine;
    __syncthreads();
    if (tid < 32) {
        int v[kThreads / 32], t = 0;
#pragma unroll
        for (int q = 0; q < kThreads / 32; ++q) {
            v[q] = t;
            t += part[tid * (kThreads / 32) + q];
        }
        int up = t;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int n = __shfl_up_sync(0xffffffffu, up, o);
            if (tid >= o) up += n;
        }
#pragma unroll
        for (int q = 0; q < kThreads / 32; ++q) part[tid * (kThreads / 32) + q] = v[q] + up - t;
        if (tid == 31) sum_live = up;
    }
    __syncthreads();
    int acc = part[tid];
    for (int w = w0; w < w1; ++w) {
        before[w] = acc;
        acc += __popc(map[w]);
    }
    __syncthreads();
    const int live = sum_live;
    // set bits ahead of page s
    auto rank = [&](int s) { return before[s >> 5] + __popc(map[s >> 5] & ((1u << (s & 31)) - 1u)); };
    if (tid == 0) sum_moves = live == 0 || live >= a.nslots ? 0 : live - rank(live);
    __syncthreads();
    const int moves = sum_moves, stay = live - moves;
    auto target = [&](int k) { return select_bit<false>(map, before, words, k); };
    if (blockIdx.x == 0) {
        if (tid == 0) *a.live_out = live;
        for (int i = tid; i < a.rows; i += kThreads) {
            const int s = a.table[i];
            const bool in = s >= 0 && s < a.nslots;
            a.table_out[i] = in && s >= live ? target(rank(s) - stay) : in ? s : -1;
        }
    }
    const long long elems = a.page_bytes / (long long)sizeof(V);
    const long long chunks = (elems + kThreads - 1) / kThreads;
    const int groups = (moves + kGroup - 1) / kGroup;
    const long long items = (long long)a.layers * chunks * groups;
    for (long long it = blockIdx.x; it < items; it += gridDim.x) {
        const long long c = it % chunks;
        const int grp = (int)((it / chunks) % groups);
        const int layer = (int)(it / chunks / groups);
        const int m = min(kGroup, moves - grp * kGroup);
        __syncthreads();
        if (tid < m) pd[tid] = target(grp * kGroup + tid);
        else if (tid >= 32 && tid < 32 + m) ps[tid - 32] = select_bit<true>(map, before, words, stay + grp * kGroup + tid - 32);
        __syncthreads();
        const long long e = c * kThreads + tid;
        V *base = static_cast<V *>(a.pool) + (long long)layer * a.nslots * elems;
        if (e < elems) move_group(base, elems, e, ps, pd, m, true);
    }
}

template <typename V>
cudaError_t copy_v(const CacheArgs &a, cudaStream_t stream) {
    const size_t smem = (size_t)((a.nslots + 31) / 32) * 4;
    cudaError_t e;
    if (smem > 48 * 1024 &&
        (e = cudaFuncSetAttribute(cache_copy_kernel<V>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem)) != cudaSuccess)
        return e;
    const long long chunks = (a.page_bytes / (long long)sizeof(V) + kThreads - 1) / kThreads;
    const long long items = chunks * a.layers * ((a.n + kGroup - 1) / kGroup);
    const long long most = 8LL * device_sms();
    cache_copy_kernel<V><<<(unsigned)(items < most ? items : most), kThreads, smem, stream>>>(a);
    return cudaGetLastError();
}

template <typename V>
cudaError_t compact_v(const CacheArgs &a, cudaStream_t stream) {
    const size_t smem = (size_t)((a.nslots + 31) / 32) * 8;
    cudaError_t e;
    if (smem > 40 * 1024 &&
        (e = cudaFuncSetAttribute(cache_compact_kernel<V>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem)) != cudaSuccess)
        return e;
    const long long chunks = (a.page_bytes / (long long)sizeof(V) + kThreads - 1) / kThreads;
    // no more moves than half the pages or than rows of the table
    const long long moves = a.rows < a.nslots / 2 ? a.rows : a.nslots / 2;
    const long long items = chunks * a.layers * ((moves + kGroup - 1) / kGroup);
    const long long most = 8LL * device_sms();
    cache_compact_kernel<V><<<(unsigned)(items < 1 ? 1 : items < most ? items : most), kThreads, smem, stream>>>(a);
    return cudaGetLastError();
}

int width(const CacheArgs &a) {
    const uintptr_t bits = reinterpret_cast<uintptr_t>(a.pool) | (uintptr_t)a.page_bytes;
    return (bits & 15) == 0 ? 16 : (bits & 3) == 0 ? 4 : 1;
}

}  // namespace

// 16 bytes a thread where the pages allow it, else 4 or 1 (pages of odd sizes)
cudaError_t launch_cache_copy(const CacheArgs &a, cudaStream_t stream) {
    if (device_sms() < 1) return cudaErrorNotSupported;
    const int w = width(a);
    return w == 16 ? copy_v<uint4>(a, stream) : w == 4 ? copy_v<uint32_t>(a, stream) : copy_v<uint8_t>(a, stream);
}

cudaError_t launch_cache_compact(const CacheArgs &a, cudaStream_t stream) {
    if (device_sms() < 1) return cudaErrorNotSupported;
    const int w = width(a);
    return w == 16 ? compact_v<uint4>(a, stream) : w == 4 ? compact_v<uint32_t>(a, stream) : compact_v<uint8_t>(a, stream);
}

}  // namespace ssd
