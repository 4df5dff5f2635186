// Pages of a pool of cached states, (layers, nslots, page): copies, forks and
// clearings in the order they are listed, and the compaction of a pool with the
// fewest moves. Both only move bytes (two pages' worth a pair, one where a page
// is cleared), so the floor is the copy bandwidth.
//
// Pairs that stand apart (no page written twice, none both read and written) are
// moved in any order, by the bulk copy engine: kMovers threads of a CTA (one per SM)
// each keep kAhead loads of up to 16 KB on their way into shared memory and about as
// many stores on their way out, with no data in registers. A page that is forked is loaded once for all
// pairs in a row that name it; a page that is cleared is stored from a buffer of
// zeros. Otherwise (and for pages that are not whole 16-byte pieces) threads own the
// same element of the page in every pair; where pairs do not stand apart one
// thread applies the whole list to its element in order, which is the order's
// meaning and needs no synchronisation.
// Measured on 24 layers with pages of 786 KB: 16 pages to two others each and 8
// cleared (1.06 GB) 189 us, 5.6 TB/s, where a copy through registers (8 loads of 16 bytes
// a thread in flight) took 238 us; compaction of 12 layers with 30 moves (566 MB) 97.8 us,
// 5.8 TB/s (registers: 153 us). In the list's order, 16 pairs: a chain 101 us (apart 103), one
// destination for all 300 us.
#include <stdint.h>

#include "sm100.cuh"
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

// ------------------------------------------------------------------ bulk copies
constexpr int kPiece = 16384;     // bytes of a page moved at a time
constexpr int kMovers = 2;        // threads of a CTA that move pieces, each its own
constexpr int kStages = 4;        // pieces of a mover in shared memory (the maps of the largest pool fit beside them)
constexpr int kAhead = 2;         // loads of a mover on their way; the other stages are for stores
constexpr int kListed = 1024;     // pairs kept in shared memory; a longer list is read where it is

__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ void bulk_store(void *dst, uint32_t src, uint32_t bytes) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(src), "r"(bytes) : "memory");
}

struct BulkSmem {
    alignas(128) uint8_t piece[kMovers][kStages][kPiece];
    alignas(128) uint8_t zero[kPiece];
    uint64_t bars[kMovers][kStages];
    struct Move {
        int pair, dst, bytes;
        long long at;              // byte offset of the piece in a page of the layer
        char *layer;
    } moves[kMovers][kStages];
    int2 list[kListed];
};

// One thread (mover w of its CTA) moves its share of (pair, layer, piece), pieces
// fastest. source(i, dst): the source of the i-th pair (-1: cleared; < -1: leave the
// pair out) and its first destination; dest(i, dst, store): store(d, cleared) for
// every page d that the piece goes to.
template <typename Source, typename Dest>
__device__ void bulk_move(BulkSmem &sm, const CacheArgs &a, int w, int n, int abort_where, Source source, Dest dest) {
    using namespace sm100;
    // Where the mover is in (pair, layer, piece), and its stride: all movers, written in
    // the same digits, so that a step is additions only (divisions of 64 bits a piece cost
    // more than the piece).
    const long long pieces = (a.page_bytes + kPiece - 1) / kPiece;
    const long long all = (long long)gridDim.x * kMovers, me = (long long)w * gridDim.x + blockIdx.x;
    const long long dpiece = all % pieces, dlayer = all / pieces % a.layers, dpair = all / pieces / a.layers;
    long long piece = me % pieces, layer = me / pieces % a.layers, pair = me / pieces / a.layers;
    const long long layer_bytes = (long long)a.nslots * a.page_bytes;
    auto bar = [&](int s) { return smem_u32(&sm.bars[w][s]); };
    int at = -1, src = -2, dst = -1;             // the pair that src belongs to
    uint32_t k = 0;
    bool more = true;
    for (uint32_t done = 0; more || done < k;) {
        // the next piece with something to move
        if (more) {
            more = false;
            while (pair < n && !more) {
                const int i = (int)pair;
                if (i != at) {
                    at = i;
                    src = source(i, dst);
                }
                if (src >= -1) {
                    const int s = (int)(k % kStages);
                    BulkSmem::Move &m = sm.moves[w][s];
                    m.pair = i;
                    m.dst = dst;
                    m.at = piece * kPiece;
                    m.layer = static_cast<char *>(a.pool) + layer * layer_bytes;
                    const long long left = a.page_bytes - m.at;
                    m.bytes = (int)(left < kPiece ? left : kPiece);
                    // the stores of the piece kStages ago have read its stage: of those made
                    // since, kStages - kAhead - 1 may still be on their way
                    asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(kStages - kAhead - 1) : "memory");
                    if (src >= 0) {
                        mbar_arrive_expect_tx(bar(s), m.bytes);
                        bulk_load(smem_u32(sm.piece[w][s]), m.layer + src * a.page_bytes + m.at, m.bytes, bar(s));
                    } else {
                        mbar_arrive(bar(s));
                    }
                    ++k;
                    more = true;
                }
                piece += dpiece;
                layer += dlayer;
                pair += dpair;
                if (piece >= pieces) {
                    piece -= pieces;
                    ++layer;
                }
                if (layer >= a.layers) {
                    layer -= a.layers;
                    ++pair;
                }
            }
        }
        // the oldest piece on its way, once there are enough behind it
        if (done < k && (!more || k - done > kAhead)) {
            const int s = (int)(done % kStages);
            const BulkSmem::Move m = sm.moves[w][s];
            bool here = mbar_try_wait(bar(s), (done / kStages) & 1);
            if (!here) {
                WaitClock clock;
                while (!here && !clock.expired(1000000000ull)) here = mbar_try_wait(bar(s), (done / kStages) & 1);
            }
            if (!here) {
                more = false;
                report_timeout(a.status, abort_where);
                for (; done < k; ++done) mbar_drain(bar((int)(done % kStages)), (done / kStages) & 1);
                break;
            }
            dest(m.pair, m.dst, [&](int d, bool cleared) {
                bulk_store(m.layer + d * a.page_bytes + m.at, smem_u32(cleared ? sm.zero : sm.piece[w][s]), m.bytes);
            });
            tma_store_commit();
            ++done;
        }
    }
    tma_store_wait_all();
}

__device__ __forceinline__ void bulk_init(BulkSmem &sm) {
    using namespace sm100;
    for (int i = threadIdx.x; i < kPiece / 16; i += kThreads) reinterpret_cast<uint4 *>(sm.zero)[i] = make_uint4(0, 0, 0, 0);
    if (threadIdx.x < kMovers * kStages) mbar_init(smem_u32(&sm.bars[0][0] + threadIdx.x), 1);
    fence_mbar_init();
    fence_proxy_async_smem();
    __syncthreads();
}

template <typename V>
__global__ void __launch_bounds__(kThreads)
cache_copy_kernel(const CacheArgs a) {
    extern __shared__ __align__(128) uint8_t shared[];
    // written pages, one bit each; where bulk copies may run their stages come first
    uint32_t *map = reinterpret_cast<uint32_t *>(shared + (sizeof(V) == 16 ? sizeof(BulkSmem) : 0));
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
        if (bad && blockIdx.x == 0) report(a.status, kFlagIndex);
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
    if constexpr (sizeof(V) == 16) {
        if (!clash) {
            BulkSmem &sm = *reinterpret_cast<BulkSmem *>(shared);
            // (source, destination) of a pair; a source of -2 leaves it out
            auto fetch = [&](int i) {
                int s, d;
                bool bad;
                read_pair(a, i, s, d, bad);
                return make_int2(bad ? -2 : s, d);
            };
            for (int i = tid; i < min(a.n, kListed); i += kThreads) sm.list[i] = fetch(i);
            bulk_init(sm);
            auto pair = [&](int i) { return i < kListed ? sm.list[i] : fetch(i); };
            if (tid % 32 == 0 && tid < 32 * kMovers)
                bulk_move(
                    sm, a, tid / 32, a.n, 950,
                    [&](int i, int &dst) {
                        const int2 p = pair(i);
                        dst = p.y;
                        if (p.x < 0) return p.y < 0 ? -2 : p.x;
                        // the first of the pairs in a row with this source loads for all
                        return i > 0 && pair(i - 1).x == p.x ? -2 : p.x;
                    },
                    [&](int i, int dst, auto store) {
                        const int src = pair(i).x;
                        if (src < 0) return store(dst, true);
                        for (int q = i; q < a.n; ++q) {
                            const int2 p = pair(q);
                            if (p.x != src) break;
                            if (p.y >= 0) store(p.y, false);
                        }
                    });
            return;
        }
    }
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
    extern __shared__ __align__(128) uint8_t shared[];
    uint32_t *map = reinterpret_cast<uint32_t *>(shared + (sizeof(V) == 16 ? sizeof(BulkSmem) : 0));
    __shared__ int ps[kGroup], pd[kGroup], part[kThreads], sum_live, sum_moves;
    const int tid = threadIdx.x;
    const int words = (a.nslots + 31) / 32;
    int *before = reinterpret_cast<int *>(map + words);
    for (int w = tid; w < words; w += kThreads) map[w] = 0u;
    __syncthreads();
    for (int i = tid; i < a.rows; i += kThreads) {
        const int s = a.table[i];
        if (s >= 0 && s < a.nslots) atomicOr(&map[s >> 5], 1u << (s & 31));
        else if (s != -1 && blockIdx.x == 0) report(a.status, kFlagIndex);
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
    // nothing to move in a pool of no layers or of empty pages: its table alone counts
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
    if constexpr (sizeof(V) == 16) {
        BulkSmem &sm = *reinterpret_cast<BulkSmem *>(shared);
        bulk_init(sm);
        if (tid % 32 == 0 && tid < 32 * kMovers && a.layers > 0 && a.page_bytes > 0)
            bulk_move(
                sm, a, tid / 32, moves, 951,
                [&](int i, int &dst) {
                    dst = target(i);
                    return select_bit<true>(map, before, words, stay + i);
                },
                [&](int, int dst, auto store) { store(dst, false); });
        return;
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

// Shared memory (MAPS maps of a word for 32 slots) and grid: with bulk copies one CTA per SM, else eight.
template <typename V, int MAPS, typename K>
cudaError_t launch(K kernel, const CacheArgs &a, long long pairs, cudaStream_t stream) {
    constexpr bool kBulk = sizeof(V) == 16;
    constexpr size_t kStaged = kBulk ? sizeof(BulkSmem) : 0, kMost = kStaged + kCacheMaxSlots / 32 * 4 * MAPS;
    static_assert(kMost <= 232448 - 2048, "stages and maps in shared memory");
    const size_t smem = kStaged + (size_t)((a.nslots + 31) / 32) * 4 * MAPS;
    // the limit belongs to the kernel, not to the launch: always the largest pool's, or another
    // thread's call on a smaller pool could lower it ahead of this launch
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMost);
    if (e != cudaSuccess) return e;
    const long long per = kBulk ? (a.page_bytes + kPiece - 1) / kPiece * pairs
                                : (a.page_bytes / (long long)sizeof(V) + kThreads - 1) / kThreads * ((pairs + kGroup - 1) / kGroup);
    const long long items = per * a.layers, most = (kBulk ? 1LL : 8LL) * device_sms();
    kernel<<<(unsigned)(items < 1 ? 1 : items < most ? items : most), kThreads, smem, stream>>>(a);
    return cudaGetLastError();
}
template <typename V>
cudaError_t copy_v(const CacheArgs &a, cudaStream_t stream) {
    return launch<V, 1>(cache_copy_kernel<V>, a, a.n, stream);
}
template <typename V>
cudaError_t compact_v(const CacheArgs &a, cudaStream_t stream) {
    // no more moves than half the pages or than rows of the table
    const long long moves = a.rows < a.nslots / 2 ? a.rows : a.nslots / 2;
    return launch<V, 2>(cache_compact_kernel<V>, a, moves, stream);
}

int width(const CacheArgs &a) {
    const uintptr_t bits = reinterpret_cast<uintptr_t>(a.pool) | (uintptr_t)a.page_bytes;
    return (bits & 15) == 0 ? 16 : (bits & 3) == 0 ? 4 : 1;
}

}  // namespace

// Bulk copies where the pages are whole 16-byte pieces, else 4 or 1 bytes a thread.
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
