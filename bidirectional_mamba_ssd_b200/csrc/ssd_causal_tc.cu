// The causal scan over prompts on the tensor cores (bf16 I/O), one persistent
// CTA per SM.
//
// Mathematics, per (batch row, 64 columns of a head) = unit and tile of 128
// tokens, with a_t = A * (dt_1 + .. + dt_t) inside the tile and H the state
// entering it:
//   y_t = sum_{s <= t} (C_t . B_s) exp(a_t - a_s) dt_s x_s + exp(a_t) C_t H + D x_t
//   H  <- exp(a_T) H + sum_s exp(a_T - a_s) dt_s B_s x_s^T
// Four products a tile: G = C B^T, Y = M X with M = G c_s under the causal mask,
// Yo = C H, S = B^T diag(w) X.
//
// The decay between two tokens is split at a reference a_r:
//   exp(a_t - a_s) = exp(a_t - a_r) * exp(a_r - a_s)
// so that M needs one factor per column, c_s = exp(a_r - a_s) dt_s, and the row's
// factor exp(a_t - a_r) is applied to the fp32 result. With a_r half the tile's decay
// both stay within e^+-40 while that is at most 80; C H is taken of exp(a_r) H and
// adds up with M X in one accumulator. Past that (a test on the tile) the rows of each
// half of the tile have a reference of their own, half way through their half, and the
// columns a factor for each, up to a decay of 80 in a half; past that each entry takes
// its own exponential. In both C H has an accumulator of its own.
// The span is a choice about range: M, exp(a_r) H and the sums of M X carry a factor of up
// to e^+-40 = 2.4e+-17 inside bf16's and fp32's 1.2e-38 .. 3.4e38, which leaves the terms
// G dt x and C H that enter an output 1e-20 .. 1e20 (e^+-75 would leave 4e-6 .. 9e5, which
// activations do reach). With a reference a half, terms that have decayed by more than e^-47 =
// 4e-21 may come out as zero. 32 x 1024 tokens, 24 heads of 64, every tile decaying by 20, 100, 200,
// 320: 132, 131, 143, 155 us (one factor, two, an exponential an entry for the last two).
//
// Roundings to bf16: M and the copy of H that enters C H, both operands of
// products whose result is rounded to bf16 (relative 2^-9 a term, random). A token's
// own term G_tt dt_t x_t is kept out of M and joins D x in fp32: with few terms in a row
// (short prompts, strong decay) it may be as large as D x and of the other sign, and its
// rounding then stood at up to 1.6 % of the outputs (130M shape 158 to 160 us for it, 16 x
// 1000 ragged 60.2 to 60.7). The state is a result in fp32, so diag(w) X enters S as
// three bf16 terms (24 bits), and H stays in fp32 registers.
//
// What bounds it: on paper HBM (x, B, C and y once); as measured the work of a tile
// within an SM. 32 x 1024 tokens, 24 heads of 64, N = 128 (631 MB, 96 us at the rate of
// a copy): 132 us in a short run at 1.96 GHz, 160 us in a long one, where the
// power limit holds the clock near 1.55 GHz. A tile takes an SM about 5500 cycles:
// nearly 3000 of shared-memory traffic (the MMAs' operands and the terms of diag(w) X),
// around which mask, state and output have to fit. One sequence of 65536 tokens (1.21
// GB, 185 us): 437 us, of which the pass for the states takes a third.
//
// Work is cut so that every CTA has
// the same number of tiles: the tiles of all units in order, divided evenly. A
// unit that a cut falls into is shared by two neighbouring CTAs. With a unit or
// more per CTA the first part of a shared unit is its CTA's first work and the
// second part its CTA's last, so the state crosses through global memory long
// before it is wanted. With fewer units (long sequences) a pass over x and B gives
// every part's own end state, a small kernel chains them, and the outputs follow.
//
// Roles (640 threads): warp 0 TMA producer; warp 1 MMA issuer, which polls what
// is ready (S, then Y and Yo, then G) instead of waiting in a fixed order; warps 2
// and 3 the decays of the coming even and odd tiles (up to four ahead) and what else
// is to be known of them; warps 4..11 group C: diag(w) X by halves of a tile, and the state,
// rows n of it a thread, 32 columns each; warps 12..15 and 16..19 groups A and B:
// mask and output of the even and the odd tiles, so that one tile's mask overlaps
// the other's products and output; thread r owns tile row r.
// TMEM (512 columns): two of {G 128: M packed over its first half once read, Y over
// its second}, S 192 (the three terms of diag(w) X side by side: an MMA with N = 192
// reads B^T once for all of them), Yo 64 for tiles past the one-factor mask. Shared
// memory: C and B two tiles deep, x three, H once, the three terms of half a tile of
// diag(w) X.
// Every wait is bounded; one that expires sets the workspace's timeout flag and
// the CTA runs to its end without storing.
#include <cuda.h>
#include <stddef.h>
#include <stdint.h>

#include "sm100.cuh"
#include "ssd_causal.h"
#include "ssd_fused_util.cuh"
#include "ssd_kernels.h"
#include "ssd_tmap.h"

namespace ssd {
namespace {

using namespace sm100;
using namespace fused;

constexpr int kTile = 128;
constexpr uint32_t kSlab = 16384;     // 128 rows x 128 bytes
constexpr int kThreads = 640;
constexpr int kStateThreads = 384;    // without the output groups
constexpr int kVec = 4;               // tiles whose decays are kept
constexpr uint32_t kHalf = 8192;      // 64 rows x 128 bytes
constexpr float kMaxSpan = 80.f;      // decay up to which a tile's, or a half tile's, mask has one factor per column

// A run of work of one CTA: n units from u0 on, of each the tiles [k0, k1) (k1 < 0:
// all). from_cut: the state entering comes from the CTA before; to_cut: the state
// left goes to the CTA behind (else to the unit's end state).
struct Stage {
    int u0, n, k0, k1;
    int from_cut, to_cut;
};

// The part of a unit ahead of the cut behind a CTA: there is none (the cut falls
// between units), it begins with the unit, it goes on from the cut before.
enum { kLinkNone = -1, kLinkFirst = 0, kLinkNext = 1 };

enum { kOrderHandoff = 0, kOrderNatural = 1, kOrderWhole = 2, kOrderState = 3 };

struct TcParams {
    const __nv_bfloat16 *dt;
    long long dt_sb, dt_st;
    const float *A, *D;
    StepSize step;
    const int *lens, *rows;          // (batch) lengths (-1: skipped row) and pages, or nullptr
    const float *init;
    float *state_out;
    __nv_bfloat16 *out;
    float *cut;                      // (CTAs, 64, N): the state at the cut behind CTA c
    float *start;                    // (CTAs, 64, N): start state of the unit that the cut falls into, where its
                                     // end state may be written before the CTA reads it
    float *cut_decay;                // (CTAs) with kOrderState: decay of the part ahead of the cut
    int2 *link;                      // (CTAs) with kOrderState: (kLink*, unit) of the part ahead of the cut
    unsigned int *flags;             // (CTAs) with kOrderHandoff: cut[c] is there
    DeviceStatus *status;
    int batch, L, H, HU, heads_per_group, halves;   // HU = H P / 64 units a row, halves = P / 64
    int order;
};

__device__ __forceinline__ int tiles_of(const TcParams &p, int b) {
    const int len = p.lens ? p.lens[b] : p.L;
    return len < 0 ? 0 : len == 0 ? 1 : (len + kTile - 1) / kTile;   // an empty sequence still passes its state on
}

// Where global tile g lies: unit u and tile k of it.
struct Place {
    int u, k;
};

// The stages of CTA c of nc and the number of its tiles; every thread of the block
// calls it (`scratch`: blockDim.x + 8 entries of shared memory). With fewer tiles
// than CTAs the last CTAs have none, so no share between two cuts is empty.
__device__ void make_stages(const TcParams &p, int c, int nc, Stage *stages, int *nsteps, long long *scratch) {
    const int tid = threadIdx.x, nth = blockDim.x;
    long long *part = scratch;            // nth entries
    Place *at = reinterpret_cast<Place *>(scratch + nth);      // 2
    long long *total = scratch + nth + 2;
    long long T;
    if (p.order == kOrderWhole) {
        if (tid == 0) {
            const int nt = tiles_of(p, c / p.HU);
            stages[0] = Stage{c, nt > 0 ? 1 : 0, 0, -1, 0, 0};
            stages[1].n = stages[2].n = 0;
            *nsteps = nt;
        }
        __syncthreads();
        return;
    }
    long long lo, hi;
    if (!p.lens) {
        const int nt = tiles_of(p, 0);
        T = (long long)p.batch * p.HU * nt;
        if (nc > T) nc = (int)T;
        lo = c < nc ? T * c / nc : T;
        hi = c < nc ? T * (c + 1) / nc : T;
        if (tid == 0) {
            at[0] = Place{(int)(lo / nt), (int)(lo % nt)};
            at[1] = Place{(int)(hi / nt), (int)(hi % nt)};
        }
    } else {
        // sums of the rows' tiles: a run of rows per thread, then the runs
        const int run = (p.batch + nth - 1) / nth, b0 = min(p.batch, tid * run), b1 = min(p.batch, b0 + run);
        long long mine = 0;
        for (int b = b0; b < b1; ++b) mine += tiles_of(p, b);
        part[tid] = mine;
        __syncthreads();
        if (tid < 32) {
            const int each = nth / 32;         // blocks are whole warps
            long long own = 0;
            for (int i = 0; i < each; ++i) own += part[tid * each + i];
            long long acc = own;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long up = __shfl_up_sync(0xffffffffu, acc, o);
                if (tid >= o) acc += up;
            }
            if (tid == 31) {
                *total = acc * p.HU;
                at[0] = at[1] = Place{p.batch * p.HU, 0};
            }
            acc -= own;
            for (int i = 0; i < each; ++i) {
                const long long v = part[tid * each + i];
                part[tid * each + i] = acc;
                acc += v;
            }
        }
        __syncthreads();
        T = *total;
        if (nc > T) nc = (int)T;
        lo = c < nc ? T * c / nc : T;
        hi = c < nc ? T * (c + 1) / nc : T;
        long long acc = part[tid] * p.HU;
        for (int b = b0; b < b1; ++b) {
            const int nt = tiles_of(p, b);
            const long long next = acc + (long long)nt * p.HU;
            for (int q = 0; q < 2; ++q) {
                const long long g = q ? hi : lo;
                if (g >= acc && g < next) at[q] = Place{b * p.HU + (int)((g - acc) / nt), (int)((g - acc) % nt)};
            }
            acc = next;
        }
    }
    __syncthreads();
    if (tid == 0) {
        const Place s = at[0], e = at[1];
        Stage left{}, whole{}, right{};
        if (lo < hi) {
            if (s.u == e.u) {
                right = Stage{s.u, 1, s.k, e.k, s.k > 0, 1};       // inside one unit, which goes on behind
            } else {
                if (s.k > 0) left = Stage{s.u, 1, s.k, -1, 1, 0};
                const int first = s.u + (s.k > 0);
                if (e.u > first) whole = Stage{first, e.u - first, 0, -1, 0, 0};
                if (e.k > 0) right = Stage{e.u, 1, 0, e.k, 0, 1};
            }
        }
        int n = (int)(hi - lo);
        if (p.order == kOrderState) {
            left.n = whole.n = 0;
            right.from_cut = 0;
            n = right.n ? right.k1 - right.k0 : 0;
        }
        const bool hand = p.order == kOrderHandoff;
        stages[0] = hand ? right : left;
        stages[1] = whole;
        stages[2] = hand ? left : right;
        *nsteps = n;
    }
    __syncthreads();
}

// A thread's walk over the tiles of its CTA.
struct Walk {
    const TcParams &p;
    const Stage *st;
    int s = 0, j = -1;
    int b = 0, hu = 0, h = 0, len = 0, k = 0, k1 = 0;
    bool first = false;            // the tile is the first of its unit's here
    __device__ __forceinline__ Walk(const TcParams &p_, const Stage *st_) : p(p_), st(st_) {}
    // the next tile; false behind the last (one call site a role keeps the code small)
    __device__ __forceinline__ bool next() {
        first = false;
        if (++k < k1) return true;
        while (true) {
            ++j;
            while (s < 3 && j >= st[s].n) {
                ++s;
                j = 0;
            }
            if (s == 3) return false;
            if (j == 0) {
                b = st[s].u0 / p.HU;
                hu = st[s].u0 % p.HU;
            } else if (++hu == p.HU) {
                hu = 0;
                ++b;
            }
            h = hu / p.halves;
            len = p.lens ? p.lens[b] : p.L;
            const int nt = len < 0 ? 0 : len == 0 ? 1 : (len + kTile - 1) / kTile;
            if (nt == 0) continue;
            k = st[s].k0;
            k1 = st[s].k1 < 0 ? nt : st[s].k1;
            first = true;
            return true;
        }
    }
};

template <int N, bool STATE>
struct Layout {
    static constexpr int kX = 3;                           // x slots
    static constexpr int kRing = STATE ? 3 : 4;            // B (and C) slots of 32 KB
    static constexpr uint32_t kBC = N * 256;               // bytes of a B or C tile
    static constexpr uint32_t ring = 0;
    static constexpr uint32_t x0 = kRing * 2 * kSlab;
    static constexpr uint32_t h = x0 + kX * kSlab;         // bf16 (N, 64) state
    static constexpr uint32_t xw = h + (STATE ? 0 : kSlab);   // the three terms of half a tile of diag(w) X; STATE: of both
    static constexpr uint32_t small = xw + (STATE ? 2 : 1) * 3 * kHalf;
};

enum {
    B_RING_FULL = 0, B_RING_EMPTY = 4, B_X_FULL = 8, B_X_EMPTY = 12,
    B_G_READY = 16,      // 2: MMA -> output groups: G of the tile
    B_M_READY = 18,      // 2: output groups -> MMA: M of the tile
    B_Y_READY = 20,      // 2: MMA -> output groups and C: Y and Yo of the tile
    B_G_FREE = 22,       // 2: output groups -> MMA: the tile's TMEM buffers are read
    B_VEC_READY = 24,    // kVec: warps 2, 3 -> C and the output groups
    B_VEC_FREE = 28,     // kVec: C and the output groups -> warps 2, 3
    B_XW_READY = 32,     // 2: C -> MMA: a half of diag(w) X of the tile
    B_S_READY = 34,      // 2: MMA -> C: S of that half (and all before it)
    B_H_READY = 36,      // C -> MMA
    B_DONE,
    B_COUNT
};

// What is known of a tile, from warps 2 and 3 to the others: a_s, the column
// factors of M (dt_s times the decay from the token to the reference, if there is
// one), the weights in the state.
enum { kZeroStart = 1, kFirst = 2, kLast = 4, kFromCut = 8, kToCut = 16, kOneFactor = 32, kPartial = 64, kHalves = 128 };
struct alignas(16) TileInfo {
    float a[kTile], col[2][kTile], w[kTile];     // col: for the rows of either half
    int b, h, hu, t0, len, flags;
    float ref[2];           // a_r of either half's rows
    float decay, half, D;   // exp(a_T); the factor of H in C H: exp(a_r), or 1; the head's skip factor
};

static_assert(sizeof(TileInfo) % 16 == 0 && offsetof(TileInfo, col) % 16 == 0, "read 16 bytes at a time");

struct Small {
    uint64_t bars[B_COUNT];
    uint32_t tmem;
    int abort_flag;
    int nsteps;
    int pad;
    Stage stages[3];
    TileInfo info[kVec];
};

__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok));
    return ok != 0;
}
// 8 columns of this thread's TMEM lane.
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&v)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
                 : "r"(taddr));
}

// Two fp32 values to an instruction.
typedef unsigned long long pair_t;
__device__ __forceinline__ pair_t pair_of(uint32_t a, uint32_t b) {
    pair_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ pair_t pair_of(float a, float b) { return pair_of(__float_as_uint(a), __float_as_uint(b)); }
__device__ __forceinline__ void halves_of(pair_t v, uint32_t &a, uint32_t &b) {
    asm("mov.b64 {%0, %1}, %2;" : "=r"(a), "=r"(b) : "l"(v));
}
__device__ __forceinline__ pair_t mul2(pair_t a, pair_t b) {
    pair_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ pair_t add2(pair_t a, pair_t b) {
    pair_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ pair_t fma2(pair_t a, pair_t b, pair_t c) {
    pair_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
// the pair rounded to bf16
__device__ __forceinline__ uint32_t bf16_of(pair_t v) {
    uint32_t a, b;
    halves_of(v, a, b);
    return pack_bf16x2(__uint_as_float(a), __uint_as_float(b));
}
// two bf16 values as a pair
__device__ __forceinline__ pair_t wide_of(uint32_t v) { return pair_of(v << 16, v & 0xffff0000u); }

// 32 bytes of one row of the output, in one store where the output is aligned to them.
__device__ __forceinline__ void store32(void *p, const uint32_t (&v)[8], bool whole) {
    if (!whole) {
        reinterpret_cast<uint4 *>(p)[0] = make_uint4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<uint4 *>(p)[1] = make_uint4(v[4], v[5], v[6], v[7]);
        return;
    }
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                 "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

// 16 bytes (8 values) of a row of diag(w) X as three bf16 terms. Each takes the
// upper 8 bits of what is left, cut off rather than rounded, so that together they
// hold all 24 bits of the fp32 product.
__device__ __forceinline__ void split3(uint4 x, float w, uint4 (&t)[3]) {
    const uint32_t *q = reinterpret_cast<const uint32_t *>(&x);
    const pair_t ww = pair_of(w, w), minus = pair_of(-1.f, -1.f);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        pair_t a = mul2(wide_of(q[j]), ww);
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            uint32_t lo, hi;
            halves_of(a, lo, hi);
            reinterpret_cast<uint32_t *>(&t[k])[j] = __byte_perm(lo, hi, 0x7632);
            if (k < 2) a = fma2(pair_of(lo & 0xffff0000u, hi & 0xffff0000u), minus, a);
        }
    }
}
// v[i] of registers, by halves
__device__ __forceinline__ uint32_t pick(const uint32_t (&v)[16], int i) {
    uint32_t a[8], b[4];
#pragma unroll
    for (int k = 0; k < 8; ++k) a[k] = i & 8 ? v[k + 8] : v[k];
#pragma unroll
    for (int k = 0; k < 4; ++k) b[k] = i & 4 ? a[k + 4] : a[k];
    const uint32_t c = i & 2 ? b[2] : b[0], d = i & 2 ? b[3] : b[1];
    return i & 1 ? d : c;
}
__device__ __forceinline__ void sync_state() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

template <int N, bool STATE>
__global__ void __launch_bounds__(STATE ? kStateThreads : kThreads, 1)
causal_tc_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_b,
                 const __grid_constant__ CUtensorMap tm_c, const TcParams p) {
    using S = Layout<N, STATE>;
    constexpr int NSLAB = N / 64;
    constexpr int kX = S::kX;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    uint8_t *g = smem_raw + (base - smem_u32(smem_raw));
    Small &sm = *reinterpret_cast<Small *>(g + S::small);
    volatile int *abort_flag = &sm.abort_flag;
    // the warp's index as the compiler can see it to be: one value for all its lanes
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    auto bar = [&](int i) { return smem_u32(&sm.bars[i]); };

    if (tid == 0) {
        sm.abort_flag = 0;
        for (int i = 0; i < B_COUNT; ++i)
            mbar_init(bar(i), !STATE && ((i >= B_VEC_FREE && i < B_VEC_FREE + kVec) || (i >= B_X_EMPTY && i < B_X_EMPTY + kX)) ? 2 : 1);
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(&sm.tmem), 512);
        tmem_relinquish();
    }
    grid_dependency_wait();
    // (the ring is not in use yet)
    make_stages(p, blockIdx.x, gridDim.x, sm.stages, &sm.nsteps, reinterpret_cast<long long *>(g));
    if (STATE && tid == 0) {
        const Stage r = sm.stages[2];
        p.link[blockIdx.x] = r.n ? make_int2(r.k0 ? kLinkNext : kLinkFirst, r.u0) : make_int2(kLinkNone, 0);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, sm.tmem, 0);
    const uint32_t nsteps = __shfl_sync(0xffffffffu, (uint32_t)sm.nsteps, 0);
    auto tG = [&](uint32_t n) { return tmem + 128 * (n & 1); };
    auto tY = [&](uint32_t n) { return tG(n) + 64; };
    const uint32_t tYo = tmem + 448;
    // with no G and Y there is room for two S: the one is read while the other fills
    auto tS = [&](uint32_t n) { return STATE ? tmem + 192 * (n & 1) : tmem + 256; };
    auto xwbuf = [&](uint32_t hf) { return S::xw + (STATE ? hf * 3 * kHalf : 0); };
    // ring slots and their use counts
    auto slot_c = [](uint32_t n) { return (2 * n) & 3; };
    auto slot_b = [](uint32_t n) { return STATE ? n % (uint32_t)S::kRing : (2 * n + 1) & 3; };
    auto use_bc = [](uint32_t n) { return STATE ? n / (uint32_t)S::kRing : n >> 1; };
    auto slot_x = [](uint32_t n) { return n % (uint32_t)kX; };
    auto use_x = [](uint32_t n) { return n / (uint32_t)kX; };
    auto ring = [&](uint32_t s) { return base + S::ring + s * 2 * kSlab; };
    auto xslot = [&](uint32_t n) { return S::x0 + slot_x(n) * kSlab; };

    if (warp == 0) {
        // ------------------------------------------------------------ producer
        if (elect_one()) {
            prefetch_tmap(&tm_x);
            prefetch_tmap(&tm_b);
            if (!STATE) prefetch_tmap(&tm_c);
            Walk w(p, sm.stages);
            uint32_t n = 0;
            for (; w.next() && !*abort_flag; ++n) {
                const int grp = w.h / p.heads_per_group, t0 = w.k * kTile;
                const uint32_t xs = slot_x(n);
                if (use_x(n) >= 1 && !mbar_wait_ool(bar(B_X_EMPTY + xs), (use_x(n) - 1) & 1, abort_flag, p.status, 903)) break;
                mbar_arrive_expect_tx(bar(B_X_FULL + xs), kSlab);
                tma_load_4d(base + xslot(n), &tm_x, bar(B_X_FULL + xs), 0, w.hu, t0, w.b);
                if (!STATE) {
                    const uint32_t s = slot_c(n);
                    if (n >= 2 && !mbar_wait_ool(bar(B_RING_EMPTY + s), (use_bc(n) - 1) & 1, abort_flag, p.status, 901)) break;
                    mbar_arrive_expect_tx(bar(B_RING_FULL + s), S::kBC);
                    for (int sl = 0; sl < NSLAB; ++sl)
                        tma_load_4d(ring(s) + sl * kSlab, &tm_c, bar(B_RING_FULL + s), 64 * sl, grp, t0, w.b);
                }
                const uint32_t s = slot_b(n);
                if (use_bc(n) >= 1 && !mbar_wait_ool(bar(B_RING_EMPTY + s), (use_bc(n) - 1) & 1, abort_flag, p.status, 902)) break;
                mbar_arrive_expect_tx(bar(B_RING_FULL + s), S::kBC);
                for (int sl = 0; sl < NSLAB; ++sl)
                    tma_load_4d(ring(s) + sl * kSlab, &tm_b, bar(B_RING_FULL + s), 64 * sl, grp, t0, w.b);
            }
            // every load issued has landed before the CTA may exit: the last use of each slot
            constexpr uint32_t kDeep = STATE ? S::kRing : 2;
            for (uint32_t q = n > kDeep ? n - kDeep : 0; q < n; ++q) {
                if (!STATE) mbar_drain(bar(B_RING_FULL + slot_c(q)), use_bc(q) & 1);
                mbar_drain(bar(B_RING_FULL + slot_b(q)), use_bc(q) & 1);
            }
            for (uint32_t q = n > kX ? n - kX : 0; q < n; ++q) mbar_drain(bar(B_X_FULL + slot_x(q)), use_x(q) & 1);
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer
        if (elect_one()) {
            constexpr uint32_t id_s = idesc_bf16_f32(128, 192, true, true);      // B^T (MN) x the terms of diag(w) X (MN)
            constexpr uint32_t id_g = idesc_bf16_f32(128, 128, false, false);    // C (K) x B (K)
            constexpr uint32_t id_o = idesc_bf16_f32(128, 64, false, true);      // C (K) x H (MN); M (K) x X (MN)
            // descriptors of the fixed buffers and of ring and x slot 0: another slot,
            // and a K step, only add to the start address (in 16-byte units)
            const uint64_t mn = sdesc_sw128(base, kSlab, 1024), kmaj = sdesc_sw128(base, 0, 1024);
            const uint64_t d_xw = sdesc_sw128(base, kHalf, 1024), d_h = mn + (S::h >> 4);
            auto step_mn = [](int q) { return (uint64_t)(q * 128); };                             // 16 rows of 128 bytes
            auto step_k = [](int q) { return (uint64_t)((q >> 2) * (kSlab >> 4) + (q & 3) * 2); };   // 32 bytes; the next slab
            uint32_t nG = 0, mS = 0, nY = 0;     // mS: halves of tiles
            WaitClock clock;
            uint32_t idle = 0;
            while (mS < 2 * nsteps || (!STATE && nY < nsteps)) {
                bool moved = false;
                // S(n), half by half: B^T times the three terms of diag(w) X
                const uint32_t nS = mS >> 1, hf = mS & 1;
                if (nS < nsteps && mbar_test(bar(B_XW_READY + hf), nS & 1) &&
                    (hf || mbar_test(bar(B_RING_FULL + slot_b(nS)), use_bc(nS) & 1))) {
                    tc_fence_after();
                    const uint64_t dB = mn + ((S::ring + slot_b(nS) * 2 * kSlab + hf * kHalf) >> 4);
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        mma_bf16_ss(tS(nS), dB + step_mn(q), d_xw + (xwbuf(hf) >> 4) + step_mn(q), id_s, q ? 1u : hf);
                    mma_commit(bar(B_S_READY + hf));
                    // B goes free with the second of its two readers, S and G
                    if (hf && (STATE || nG > nS)) mma_commit(bar(B_RING_EMPTY + slot_b(nS)));
                    ++mS;
                    moved = true;
                } else if (!STATE) {
                    // Y(n) = M X + C (half H); the copy of H follows both halves of diag(w) X, so what
                    // is behind the sequence's end in x is zero by now; past the one-factor mask C H
                    // goes to Yo, once that of the tile before is read
                    if (nY < nG && mbar_test(bar(B_M_READY + (nY & 1)), (nY >> 1) & 1) && mbar_test(bar(B_H_READY), nY & 1) &&
                        (nY == 0 || (sm.info[nY % kVec].flags & kOneFactor) ||
                         mbar_test(bar(B_G_FREE + ((nY - 1) & 1)), ((nY - 1) >> 1) & 1))) {
                        tc_fence_after();
                        const uint64_t dX = mn + (xslot(nY) >> 4), dC = kmaj + ((S::ring + slot_c(nY) * 2 * kSlab) >> 4);
                        const uint32_t dm = tG(nY), dy = tY(nY);
#pragma unroll
                        for (int q = 0; q < kTile / 16; ++q) mma_bf16_ts(dy, dm + 8 * q, dX + step_mn(q), id_o, q > 0);
                        const int flags = sm.info[nY % kVec].flags;
                        if (!(flags & kZeroStart)) {
                            const uint32_t d = flags & kOneFactor ? dy : tYo, add = flags & kOneFactor ? 1u : 0u;
#pragma unroll
                            for (int q = 0; q < N / 16; ++q)
                                mma_bf16_ss(d, dC + step_k(q), d_h + step_mn(q), id_o, q ? 1u : add);
                        }
                        mma_commit(bar(B_Y_READY + (nY & 1)));
                        mma_commit(bar(B_RING_EMPTY + slot_c(nY)));
                        ++nY;
                        moved = true;
                    } else
                    // G(n) = C B^T: the operands have landed and tile n - 2's buffers are read
                    if (nG < nsteps && mbar_test(bar(B_RING_FULL + slot_c(nG)), use_bc(nG) & 1) &&
                        mbar_test(bar(B_RING_FULL + slot_b(nG)), use_bc(nG) & 1) &&
                        (nG < 2 || mbar_test(bar(B_G_FREE + (nG & 1)), ((nG >> 1) - 1) & 1))) {
                        tc_fence_after();
                        const uint64_t dC = kmaj + ((S::ring + slot_c(nG) * 2 * kSlab) >> 4);
                        const uint64_t dB = kmaj + ((S::ring + slot_b(nG) * 2 * kSlab) >> 4);
                        const uint32_t d = tG(nG);
#pragma unroll
                        for (int q = 0; q < N / 16; ++q) mma_bf16_ss(d, dC + step_k(q), dB + step_k(q), id_g, q > 0);
                        mma_commit(bar(B_G_READY + (nG & 1)));
                        if (mS > 2 * nG + 1) mma_commit(bar(B_RING_EMPTY + slot_b(nG)));
                        ++nG;
                        moved = true;
                    }
                }
                if (moved) {
                    idle = 0;
                    clock = WaitClock();
                } else if ((++idle & 63u) == 0) {
                    if (*abort_flag) break;
                    if (clock.expired(1000000000ull)) {
                        *abort_flag = 1;
                        report_timeout(p.status, 910);
                        break;
                    }
                }
            }
            // all MMAs complete before TMEM is released
            mma_commit(bar(B_DONE));
            mbar_drain(bar(B_DONE), 0);
        }
    } else if (warp < 4) {
        // ------------------------------------------------------------ decays of the coming tiles
        // (lane l: tokens 4 l .. 4 l + 3 of the tile)
        Walk w(p, sm.stages);
        uint32_t raw[4] = {0u, 0u, 0u, 0u};
        float A = 0.f, D = 0.f, bias = 0.f;
        auto load = [&](bool there) {
            if (there) {
                A = p.A[w.h];
                D = !STATE && p.D ? p.D[w.h] : 0.f;
                bias = p.step.bias ? p.step.bias[w.h] : 0.f;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int t = w.k * kTile + 4 * lane + i;
                raw[i] = 0;
                if (there && t < w.len) {
                    const __nv_bfloat16 *q = p.dt + (long long)w.b * p.dt_sb + (long long)t * p.dt_st + w.h;
                    asm volatile("ld.global.nc.u16 %0, [%1];" : "=r"(raw[i]) : "l"(q));
                }
            }
        };
        int b = 0, h = 0, hu = 0, t0 = 0, len = 0, flags = 0;     // the tile whose step sizes have been asked for
        float A_ = 0.f, D_ = 0.f, bias_ = 0.f;
        bool there = false;
#pragma unroll 1
        for (uint32_t n = warp & 1;;) {
            float v[4], up[4], down[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = t0 + 4 * lane + i < len ? p.step.with(bf2f(raw[i]), bias_) : 0.f;
            const int b0 = b, h0 = h, hu0 = hu, t00 = t0, len0 = len;
            int flags0 = flags;
            const float A0 = A_, D0 = D_;
            const bool had = there;
            // the next tile's step sizes are on their way meanwhile
            there = true;
            for (int i = had || (warp & 1) ? 2 : 1; there && i > 0; --i) there = w.next();
            load(there);
            if (there) {
                const Stage &st = sm.stages[w.s];
                const bool zero = w.first && !st.from_cut && (STATE || p.init == nullptr);
                b = w.b; h = w.h; hu = w.hu; t0 = w.k * kTile; len = w.len;
                flags = (zero ? kZeroStart : 0) | (w.first ? kFirst : 0) | (w.k + 1 == w.k1 ? kLast : 0) |
                        (st.from_cut ? kFromCut : 0) | (st.to_cut ? kToCut : 0) | (t0 + kTile > len ? kPartial : 0);
                A_ = A; D_ = D; bias_ = bias;
                // a unit's start state comes to L2 ahead of the state's warps
                if (!STATE && p.init && (flags & kFirst) && !(flags & kFromCut)) {
                    const float *page = p.init + ((size_t)(p.rows ? p.rows[b] : b) * p.HU + hu) * 64 * N;
#pragma unroll
                    for (int i = 0; i < 64 * N; i += 32 * 32) asm volatile("prefetch.global.L2 [%0];" ::"l"(page + i + 32 * lane));
                }
            }
            if (!had) {
                if (!there) break;
                continue;
            }
            up[0] = v[0];
            down[3] = 0.f;
#pragma unroll
            for (int i = 1; i < 4; ++i) up[i] = up[i - 1] + v[i];
#pragma unroll
            for (int i = 2; i >= 0; --i) down[i] = down[i + 1] + v[i + 1];
            const float mine = up[3];
            float pre = mine, suf = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const float x = __shfl_up_sync(0xffffffffu, pre, o), y = __shfl_down_sync(0xffffffffu, suf, o);
                if (lane >= o) pre += x;
                if (lane + o < 32) suf += y;
            }
            const float all = A0 * __shfl_sync(0xffffffffu, pre, 31);
            // a row's weight in the state: the sum behind it, added up from the end
            const float ahead = __shfl_up_sync(0xffffffffu, pre, 1), behind = __shfl_down_sync(0xffffffffu, suf, 1);
            const bool one = all > -kMaxSpan;
            if (one) flags0 |= kOneFactor;
            float a4[4], c4[4], w4[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) a4[i] = A0 * ((lane ? ahead : 0.f) + up[i]);
            const float mid = __shfl_sync(0xffffffffu, a4[3], 15);
            const bool halves = !one && mid > -kMaxSpan && all - mid > -kMaxSpan, factor = one || halves;
            if (halves) flags0 |= kHalves;
            const float ref0 = one ? 0.5f * all : 0.5f * mid, ref1 = one ? ref0 : 0.5f * (mid + all);
            float d4[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                c4[i] = factor ? __expf(ref0 - a4[i]) * v[i] : v[i];
                d4[i] = one ? c4[i] : factor ? __expf(ref1 - a4[i]) * v[i] : v[i];
                w4[i] = expf(A0 * ((lane < 31 ? behind : 0.f) + down[i])) * v[i];
            }
            const uint32_t vb = n % kVec;
            if (n >= kVec) mbar_wait_ool(bar(B_VEC_FREE + vb), ((n / kVec) - 1) & 1, abort_flag, p.status, 920);
            TileInfo &I = sm.info[vb];
            reinterpret_cast<float4 *>(I.a)[lane] = make_float4(a4[0], a4[1], a4[2], a4[3]);
            reinterpret_cast<float4 *>(I.col[0])[lane] = make_float4(c4[0], c4[1], c4[2], c4[3]);
            reinterpret_cast<float4 *>(I.col[1])[lane] = make_float4(d4[0], d4[1], d4[2], d4[3]);
            reinterpret_cast<float4 *>(I.w)[lane] = make_float4(w4[0], w4[1], w4[2], w4[3]);
            if (lane == 0) {
                I.b = b0; I.h = h0; I.hu = hu0; I.t0 = t00; I.len = len0; I.flags = flags0;
                I.decay = expf(all);
                I.half = one ? __expf(ref0) : 1.f;
                I.ref[0] = ref0;
                I.ref[1] = ref1;
                I.D = D0;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(B_VEC_READY + vb));
            n += 2;
            if (!there) break;
        }
    } else if (warp >= 4 && warp < 12) {
        // ------------------------------------------------------------ group C
        const int row = ((warp & 3) << 5) | lane;                 // row n of the state
        const int ph = warp >= 8;                                 // its columns [32 ph, 32 ph + 32)
        const uint32_t lane_off = ((uint32_t)((warp & 3) << 5) << 16) + 32 * ph;
        const int cid = tid - 128, br = cid >> 2, bq = cid & 3;   // diag(w) X: row br of the half tile, 16 columns
        pair_t H[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) H[j] = 0ull;
        float decay = 0.f, all = 1.f;     // of the previous tile; of the part so far
        int pb = 0, phu = 0, pflags = 0;  // of the previous tile
        // an aborted CTA walks on to its end (its waits return at once): a group's
        // threads never part ways ahead of their barriers. The step behind the last
        // tile only takes its state.
#pragma unroll 1
        for (uint32_t n = 0; n <= nsteps; ++n) {
            const TileInfo &I = sm.info[n % kVec];
            const bool tile = n < nsteps;
            int t0 = 0, len = 0, b = 0, hu = 0, flags = 0;
            float this_decay = 0.f, half = 1.f;
            if (tile) {
                mbar_wait_ool(bar(B_VEC_READY + n % kVec), (n / kVec) & 1, abort_flag, p.status, 921);
                mbar_wait_ool(bar(B_X_FULL + slot_x(n)), use_x(n) & 1, abort_flag, p.status, 922);
                t0 = I.t0; len = I.len; b = I.b; hu = I.hu; flags = I.flags;
                this_decay = I.decay; half = I.half;
            }
            // half of diag(w) X in three terms
            auto build = [&](int hf) {
                const int r = hf * 64 + br;
                uint8_t *xt = g + xslot(n) + r * 128;
                uint8_t *dst = g + xwbuf(hf) + br * 128;
                if (t0 + r < len) {
                    const float wt = I.w[r];
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const int at = ((2 * bq + c) ^ (r & 7)) << 4;
                        uint4 t[3];
                        split3(*reinterpret_cast<const uint4 *>(xt + at), wt, t);
#pragma unroll
                        for (int k = 0; k < 3; ++k) *reinterpret_cast<uint4 *>(dst + k * kHalf + at) = t[k];
                    }
                } else {
                    // what lies behind the sequence may be anything: zero it wherever a product
                    // sums over it (x, diag(w) X, B)
                    const uint4 z = make_uint4(0, 0, 0, 0);
                    for (int c = 0; c < 2; ++c) {
                        const int at = ((2 * bq + c) ^ (r & 7)) << 4;
                        *reinterpret_cast<uint4 *>(xt + at) = z;
                        for (int k = 0; k < 3; ++k) *reinterpret_cast<uint4 *>(dst + k * kHalf + at) = z;
                    }
                    mbar_wait_ool(bar(B_RING_FULL + slot_b(n)), use_bc(n) & 1, abort_flag, p.status, 923);
                    uint4 *bt = reinterpret_cast<uint4 *>(g + S::ring + slot_b(n) * 2 * kSlab + r * 128);
                    for (int c = 0; c < 2 * NSLAB; ++c) bt[(c >> 1) * (kSlab / 16) + 2 * bq + (c & 1)] = z;
                }
                fence_proxy_async_smem();
                sync_state();
                if (cid == 0) mbar_arrive(bar(B_XW_READY + hf));
            };
            // H <- exp(a_T) H + S of the tile before
            auto advance = [&]() {
                tc_fence_after();
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    uint32_t sv[3][8];
#pragma unroll
                    for (int k = 0; k < 3; ++k) tmem_ld8(tS(n - 1) + 64 * k + lane_off + q * 8, sv[k]);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        H[q * 4 + j] = fma2(pair_of(decay, decay), H[q * 4 + j],
                                            add2(pair_of(sv[0][2 * j], sv[0][2 * j + 1]),
                                                 add2(pair_of(sv[1][2 * j], sv[1][2 * j + 1]), pair_of(sv[2][2 * j], sv[2][2 * j + 1]))));
                }
                tc_fence_before();
            };
            // the state behind the tile before goes where it is wanted; the one entering this
            // tile, where a part begins with it, comes in
            auto settle = [&]() {
                if (pflags & kLast) {
                    // the state behind the unit or the part of it: the end state, or to the CTA
                    // behind (with kOrderNatural the chain has put it there)
                    const bool cut = pflags & kToCut;
                    float *d = nullptr;
                    if (!cut) {
                        if (p.state_out) d = p.state_out + ((size_t)(p.rows ? p.rows[pb] : pb) * p.HU + phu) * 64 * N;
                    } else if (p.order != kOrderNatural) {
                        d = p.cut + (size_t)blockIdx.x * 64 * N;
                    }
                    if (d && row < N && !*abort_flag) {
                        d += 32 * ph * N + row;
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            uint32_t v0, v1;
                            halves_of(H[j], v0, v1);
                            d[(2 * j) * N] = __uint_as_float(v0);
                            d[(2 * j + 1) * N] = __uint_as_float(v1);
                        }
                    }
                    if (cut && p.order != kOrderNatural) {
                        sync_state();
                        if (cid == 0) {
                            if (STATE) p.cut_decay[blockIdx.x] = all;
                            else if (!*abort_flag) flag_release(p.flags + blockIdx.x, 1u);
                        }
                    }
                }
                if (flags & kFirst) {
                    all = 1.f;
                    const float *from = nullptr;
                    if (!STATE) {
                        if (flags & kFromCut) {
                            from = p.cut + (size_t)(blockIdx.x - 1) * 64 * N;
                            if (p.order == kOrderHandoff) {
                                if (cid == 0) flag_wait(p.flags + blockIdx.x - 1, 1u, abort_flag, p.status, 925);
                                sync_state();
                            }
                        } else if (p.init && p.order == kOrderNatural && (flags & kToCut)) {
                            from = p.start + (size_t)blockIdx.x * 64 * N;
                        } else if (p.init) {
                            from = p.init + ((size_t)(p.rows ? p.rows[b] : b) * p.HU + hu) * 64 * N;
                        }
                    }
                    if (from && row < N) {
                        // another CTA of this launch may have written it: past L1
                        from += 32 * ph * N + row;
#pragma unroll
                        for (int j = 0; j < 16; ++j) H[j] = pair_of(__ldcg(from + (2 * j) * N), __ldcg(from + (2 * j + 1) * N));
                    } else {
#pragma unroll
                        for (int j = 0; j < 16; ++j) H[j] = 0ull;
                    }
                }
                decay = this_decay;
                all *= decay;
                pflags = flags;
                pb = b;
                phu = hu;
            };
            // one buffer for diag(w) X and one S: a half waits for the half before, and S is
            // read ahead of the first. Two of each: a half waits for its like of the tile before.
            // (One call site for each piece: the loop has to stay in the instruction cache.)
#pragma unroll 1
            for (int hf = 0; hf < 2; ++hf) {
                if (n >= 1 && (STATE || hf == 0))
                    mbar_wait_ool(bar(B_S_READY + (STATE ? hf : 1)), (n - 1) & 1, abort_flag, p.status, 924);
                if (!STATE && hf == 0 && n >= 1) advance();
                if (!STATE && hf == 1) {
                    settle();
                    if (!tile) break;
                    mbar_wait_ool(bar(B_S_READY), n & 1, abort_flag, p.status, 927);
                }
                if (tile) build(hf);
            }
            if (STATE) {
                if (n >= 1) advance();
                settle();
            }
            if (!tile) break;
            if (!STATE) {
                // C H of the tile before has read the buffer
                if (n >= 1) mbar_wait_ool(bar(B_Y_READY + ((n - 1) & 1)), ((n - 1) >> 1) & 1, abort_flag, p.status, 926);
                if (row < N && !(flags & kZeroStart)) {
                    const pair_t f = pair_of(half, half);
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        *reinterpret_cast<uint4 *>(g + S::h + sw128_offset(row, 4 * ph + c)) =
                            make_uint4(bf16_of(mul2(f, H[4 * c])), bf16_of(mul2(f, H[4 * c + 1])),
                                       bf16_of(mul2(f, H[4 * c + 2])), bf16_of(mul2(f, H[4 * c + 3])));
                }
                fence_proxy_async_smem();
                tc_fence_before();
                sync_state();
                if (cid == 0) mbar_arrive(bar(B_H_READY));
            }
            if (cid == 0) {
                mbar_arrive(bar(B_VEC_FREE + n % kVec));
                mbar_arrive(bar(B_X_EMPTY + slot_x(n)));
            }
        }
    } else if (!STATE && warp >= 12) {
        // ------------------------------------------------------------ groups A and B
        const bool is_b = warp >= 16;
        const int row = ((warp & 3) << 5) | lane;
        const uint32_t lane_off = (uint32_t)((warp & 3) << 5) << 16;
        const int wq = warp & 3;
        auto sync_g = [&]() { if (is_b) sync_b(); else sync_a(); };
        const bool whole = (reinterpret_cast<uintptr_t>(p.out) & 31u) == 0;
        // zeros in the output rows that no tile covers, while the first tiles are on their
        // way: a batch row's by several CTAs (w: batch row and part), or some rows' by one
        if (p.lens) {
            const int parts = max(1, (int)gridDim.x / p.batch);
            const size_t row16 = (size_t)p.HU * 8;       // 16-byte pieces of a token
            for (long long w = blockIdx.x; w < (long long)p.batch * parts; w += gridDim.x) {
                const int b = (int)(w / parts), len = p.lens[b];
                const int covered = len < 0 ? 0 : len == 0 ? kTile : (len + kTile - 1) / kTile * kTile;
                if (covered >= p.L) continue;
                uint4 *out = reinterpret_cast<uint4 *>(p.out) + ((size_t)b * p.L + covered) * row16;
                const size_t n = (size_t)(p.L - covered) * row16, step = (size_t)parts * 256;
                for (size_t i = (size_t)(w % parts) * 256 + tid - 384; i < n; i += step) out[i] = make_uint4(0, 0, 0, 0);
            }
        }
#pragma unroll 1
        for (uint32_t n = is_b; n < nsteps; n += 2) {
            const uint32_t par = (n >> 1) & 1, nb = n & 1;
            // ---------------- the mask: 16 columns at a time, the next ones on their way from
            // TMEM meanwhile; columns [16 c, 16 c + 16) of M are 8 words over G columns already read
            mbar_wait_ool(bar(B_VEC_READY + n % kVec), (n / kVec) & 1, abort_flag, p.status, 930);
            const TileInfo &I = sm.info[n % kVec];
            const float my_a = I.a[row], *col = I.col[wq >> 1];
            const bool one = I.flags & kOneFactor, factor = I.flags & (kOneFactor | kHalves);
            mbar_wait_ool(bar(B_G_READY + nb), par, abort_flag, p.status, 931);
            tc_fence_after();
            const uint32_t tg = tG(n) + lane_off;
            const int chunks = 2 * wq + 2;             // up to and with the diagonal
            // the row's own G, for the output (two loads of its own: taken out of the chunks as the
            // mask passes them the 130M shape takes 161 to 163 us, out of the last two kept 166)
            float g_own;
            {
                uint32_t lo[16], hi[16];
                tmem_ld16(tg + 32 * wq, lo);
                tmem_ld16(tg + 32 * wq + 16, hi);
                tmem_wait_ld();
#pragma unroll
                for (int q = 0; q < 16; ++q) lo[q] = lane & 16 ? hi[q] : lo[q];
                g_own = __uint_as_float(pick(lo, lane & 15));
            }
            // the row's own entry and those behind it are dropped, never multiplied
            auto put = [&](int c, uint32_t (&m)[8]) {
                if (c >= 2 * wq) {
                    const int own = row - 16 * c;
#pragma unroll
                    for (int q = 0; q < 8; ++q) m[q] = 2 * q + 1 < own ? m[q] : 2 * q < own ? (m[q] & 0xffffu) : 0u;
                }
                tmem_st8(tg + 8 * c, m);
            };
            uint32_t ga[16], gb[16], m[8];
            if (factor) {
                auto mask = [&](int c, const uint32_t (&gv)[16]) {
#pragma unroll
                    for (int q = 0; q < 16; q += 4) {
                        const float4 f = *reinterpret_cast<const float4 *>(col + 16 * c + q);
                        m[q / 2] = bf16_of(mul2(pair_of(gv[q], gv[q + 1]), pair_of(f.x, f.y)));
                        m[q / 2 + 1] = bf16_of(mul2(pair_of(gv[q + 2], gv[q + 3]), pair_of(f.z, f.w)));
                    }
                    put(c, m);
                };
                tmem_ld16(tg, ga);
                tmem_wait_ld();
#pragma unroll 1
                for (int c = 0; c < chunks; c += 2) {
                    tmem_ld16(tg + 16 * c + 16, gb);
                    mask(c, ga);
                    tmem_wait_ld();
                    if (c + 2 < chunks) tmem_ld16(tg + 16 * c + 32, ga);
                    mask(c + 1, gb);
                    tmem_wait_ld();
                }
            } else {
#pragma unroll 1
                for (int c = 0; c < chunks; ++c) {
                    tmem_ld16(tg + 16 * c, ga);
                    tmem_wait_ld();
#pragma unroll
                    for (int q = 0; q < 16; q += 2) {
                        const float e0 = __expf(fminf(my_a - I.a[16 * c + q], 0.f)) * col[16 * c + q];
                        const float e1 = __expf(fminf(my_a - I.a[16 * c + q + 1], 0.f)) * col[16 * c + q + 1];
                        m[q / 2] = bf16_of(mul2(pair_of(ga[q], ga[q + 1]), pair_of(e0, e1)));
                    }
                    put(c, m);
                }
            }
#pragma unroll 1
            for (int c = chunks; c < 8; c += 2) {
                uint32_t z[16];
#pragma unroll
                for (int q = 0; q < 16; ++q) z[q] = 0u;
                tmem_st16(tg + 8 * c, z);
            }
            tmem_wait_st();
            tc_fence_before();
            sync_g();
            if (row == 0) mbar_arrive(bar(B_M_READY + nb));
            // ---------------- the output
            const int t = I.t0 + row;
            const bool own = !one && !(I.flags & kZeroStart);       // C H comes by itself, with the row's decay
            const float rf = factor ? __expf(my_a - I.ref[wq >> 1]) : 1.f, e = __expf(my_a);
            const float D = I.D + rf * (g_own * col[row]);       // of the row's own x
            __nv_bfloat16 *dst = p.out + (((size_t)I.b * p.L + t) * p.HU + I.hu) * 64;
            const bool keep = t < I.len, inside = t < p.L, partial = I.flags & kPartial;
            const pair_t rf2 = pair_of(rf, rf), D2 = pair_of(D, D);
            const uint8_t *xt = g + xslot(n);
            mbar_wait_ool(bar(B_Y_READY + nb), par, abort_flag, p.status, 932);
            tc_fence_after();
            const bool store = inside && !*abort_flag;
            // y = rf Y + D x (+ more), 16 columns
            auto emit = [&](int q, const uint32_t (&yv)[16], const pair_t *more) {
                uint32_t o8[8];
                uint4 xv[2];
#pragma unroll
                for (int c = 0; c < 2; ++c) xv[c] = *reinterpret_cast<const uint4 *>(xt + sw128_offset(row, q * 2 + c));
                const uint32_t *xu = reinterpret_cast<const uint32_t *>(xv);
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    pair_t v = mul2(D2, wide_of(xu[c]));
                    if (more) v = add2(v, more[c]);
                    o8[c] = bf16_of(fma2(rf2, pair_of(yv[2 * c], yv[2 * c + 1]), v));
                }
                if (partial && !keep) {
#pragma unroll
                    for (int c = 0; c < 8; ++c) o8[c] = 0u;
                }
                if (store) store32(dst + q * 16, o8, whole);
            };
            uint32_t ya[16], yb[16];
            if (!own) {
                tmem_ld16(tY(n) + lane_off, ya);
                tmem_wait_ld();
#pragma unroll 1
                for (int q = 0; q < 4; q += 2) {
                    tmem_ld16(tY(n) + lane_off + q * 16 + 16, yb);
                    emit(q, ya, nullptr);
                    tmem_wait_ld();
                    if (q == 0) tmem_ld16(tY(n) + lane_off + 32, ya);
                    emit(q + 1, yb, nullptr);
                    tmem_wait_ld();
                }
            } else {
                const pair_t e2 = pair_of(e, e);
#pragma unroll 1
                for (int q = 0; q < 4; ++q) {
                    pair_t more[8];
                    tmem_ld16(tY(n) + lane_off + q * 16, ya);
                    tmem_ld16(tYo + lane_off + q * 16, yb);
                    tmem_wait_ld();
#pragma unroll
                    for (int c = 0; c < 8; ++c) more[c] = mul2(e2, pair_of(yb[2 * c], yb[2 * c + 1]));
                    emit(q, ya, more);
                }
            }
            tc_fence_before();
            sync_g();
            if (row == 0) {
                mbar_arrive(bar(B_VEC_FREE + n % kVec));
                mbar_arrive(bar(B_G_FREE + nb));
                mbar_arrive(bar(B_X_EMPTY + slot_x(n)));
            }
        }
    }

    // ------------------------------------------------------------ teardown
    tc_fence_before();
    __syncthreads();
    if (warp == 1) tmem_dealloc(tmem, 512);
}

// The chain of states across the cuts: cut[c] holds the own end state (from zero)
// of the part ahead of the cut behind CTA c, cut_decay[c] its decay; they become
// the states at the cuts, in place. A block takes 256 x 4 elements of the chain
// that begins with CTA c.
template <int N>
__global__ void __launch_bounds__(256) causal_chain_kernel(const TcParams p, int nc) {
    constexpr int kParts = 64 * N / 1024;
    constexpr size_t kState = 64 * N / 4;
    const int c0 = blockIdx.x / kParts, e = (blockIdx.x % kParts) * 256 + threadIdx.x;
    grid_launch_dependents();
    const int2 first = p.link[c0];
    if (first.x != kLinkFirst) return;
    const int u = first.y, b = u / p.HU;
    // the CTAs that go on from here
    int end = c0 + 1;
    for (bool more = true; more;) {
        const int c = end + (threadIdx.x & 31);
        const unsigned go = __ballot_sync(0xffffffffu, c < nc && p.link[c < nc ? c : 0].x == kLinkNext);
        const int run = go == 0xffffffffu ? 32 : __ffs(~go) - 1;
        end += run;
        more = run == 32;
    }
    float4 h = make_float4(0.f, 0.f, 0.f, 0.f);
    if (p.init) h = reinterpret_cast<const float4 *>(p.init + ((size_t)(p.rows ? p.rows[b] : b) * p.HU + u % p.HU) * 64 * N)[e];
    // the unit's last part may end, in place, before its first part begins
    if (p.init) reinterpret_cast<float4 *>(p.start)[c0 * kState + e] = h;
    float4 *cut = reinterpret_cast<float4 *>(p.cut) + e;
    constexpr int kAhead = 8;              // loads in flight
    for (int c = c0; c < end; c += kAhead) {
        float4 own[kAhead];
        float d[kAhead];
#pragma unroll
        for (int q = 0; q < kAhead; ++q)
            if (c + q < end) {
                own[q] = cut[(size_t)(c + q) * kState];
                d[q] = p.cut_decay[c + q];
            }
#pragma unroll
        for (int q = 0; q < kAhead; ++q)
            if (c + q < end) {
                h = make_float4(fmaf(d[q], h.x, own[q].x), fmaf(d[q], h.y, own[q].y), fmaf(d[q], h.z, own[q].z),
                                fmaf(d[q], h.w, own[q].w));
                cut[(size_t)(c + q) * kState] = h;
            }
    }
}

// What the scan needs ahead of it: its flags cleared and, for a ragged or paged batch
// (rows not nullptr), resolved pages and effective lengths (-1: skipped). Block b.
__global__ void __launch_bounds__(128) causal_rows_kernel(const CausalArgs a, int *rows, int *lens, unsigned int *flags, int nflags) {
    const int b = blockIdx.x;
    grid_launch_dependents();
    if (b == 0)
        for (int i = threadIdx.x; i < nflags; i += 128) flags[i] = 0u;
    if (!rows) return;
    int row = b;
    bool bad = false;
    if (a.slots) {
        row = a.slots[b];
        bad = row < -1 || row >= a.nslots;
        bool again = false;
        if (row >= 0)
            for (int i = threadIdx.x; i < b; i += 128) again |= a.slots[i] == row;
        bad |= (bool)__syncthreads_or(again);
        if (bad) row = -1;
    }
    if (threadIdx.x == 0) {
        rows[b] = row;
        lens[b] = row < 0 ? -1 : a.len(b);
        if (bad) report(a.status, kFlagIndex);
    }
}

// Scratch of the path behind the status header.
struct TcScratch {
    size_t rows, lens, flags, link, decay, cut, start, total;
};
TcScratch tc_scratch(int batch, int sms, int N) {
    TcScratch s{};
    size_t o = 0;
    auto take = [&](size_t bytes) {
        const size_t at = o;
        o += (bytes + 255) & ~(size_t)255;
        return at;
    };
    s.rows = take(sizeof(int) * (size_t)batch);
    s.lens = take(sizeof(int) * (size_t)batch);
    s.flags = take(sizeof(int) * (size_t)sms);
    s.link = take(sizeof(int2) * (size_t)sms);
    s.decay = take(sizeof(float) * (size_t)sms);
    s.cut = take(sizeof(float) * (size_t)sms * 64 * N);
    s.start = take(sizeof(float) * (size_t)sms * 64 * N);
    s.total = o;
    return s;
}

bool map_rows(CUtensorMap *m, const void *base, int inner, int count, int L, int batch, long long token, long long row) {
    uint64_t dims[4] = {(uint64_t)inner, (uint64_t)count, (uint64_t)L, (uint64_t)batch};
    uint64_t str[3] = {(uint64_t)inner * 2, (uint64_t)token * 2, (uint64_t)row * 2};
    uint32_t box[4] = {64, 1, kTile, 1};
    return tmap::make_map(m, base, 4, dims, str, box);
}

template <int N, bool STATE>
cudaError_t launch_tc(const CUtensorMap &x, const CUtensorMap &b, const CUtensorMap &c, const TcParams &p, int ctas,
                      bool follows, cudaStream_t stream) {
    auto k = causal_tc_kernel<N, STATE>;
    const size_t smem = Layout<N, STATE>::small + sizeof(Small) + 1024;
    static_assert(Layout<N, STATE>::small + sizeof(Small) + 1024 <= 232448, "shared memory of a CTA");
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(STATE ? kStateThreads : kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    // behind a kernel of this call the prologue overlaps that kernel's end
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = follows ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, k, x, b, c, p);
}

template <int N>
cudaError_t run_tc(const CausalArgs &a, void *scratch, cudaStream_t stream) {
    const int sms = device_sms();
    if (sms < 1 || !tmap::encode_fn()) return cudaErrorNotSupported;
    const TcScratch t = tc_scratch(a.batch, sms, N);
    char *ws = static_cast<char *>(scratch);
    cudaError_t e;
    TcParams p{};
    p.dt = static_cast<const __nv_bfloat16 *>(a.dt);
    p.dt_sb = a.dt_sb; p.dt_st = a.dt_st;
    p.A = a.A; p.D = a.D; p.step = a.step;
    p.init = a.init; p.state_out = a.state_out; p.out = static_cast<__nv_bfloat16 *>(a.out);
    p.cut = reinterpret_cast<float *>(ws + t.cut);
    p.start = reinterpret_cast<float *>(ws + t.start);
    p.cut_decay = reinterpret_cast<float *>(ws + t.decay);
    p.link = reinterpret_cast<int2 *>(ws + t.link);
    p.flags = reinterpret_cast<unsigned int *>(ws + t.flags);
    p.status = a.status;
    p.batch = a.batch; p.L = a.L; p.H = a.H;
    p.halves = a.P / 64; p.HU = a.H * p.halves; p.heads_per_group = a.H / a.G;
    CUtensorMap tx, tb, tc;
    if (!map_rows(&tx, a.x, 64, p.HU, a.L, a.batch, a.x_st, a.x_sb) ||
        !map_rows(&tb, a.B, N, a.G, a.L, a.batch, a.b_st, a.b_sb) || !map_rows(&tc, a.C, N, a.G, a.L, a.batch, a.c_st, a.c_sb))
        return cudaErrorInvalidValue;
    const long long units = (long long)a.batch * p.HU, nt = (a.L + kTile - 1) / kTile;
    // fewer units than SMs: the cut work costs a second pass over x and B and two
    // more launches, but spreads over every SM. Whole units take about 2.4 us a tile, cut
    // ones 4 us a tile of the largest share and 10 us. Whole and cut, 24 units: 768 tokens
    // 19.7 and 19.7 us, 1024 24.5 and 23.1, 4096 83 and 39; 48 units: 1024 24.9 and 27.5,
    // 1536 34.7 and 31.8; 96 units: 4096 84 and 100
    const long long share = (units * nt + sms - 1) / sms;
    p.order = units >= sms ? kOrderHandoff : 10 * nt > 16 * share + 40 ? kOrderNatural : kOrderWhole;
    const bool ragged = a.seqlens || a.slots, first = ragged || p.order == kOrderHandoff;
    if (first) {
        int *rows = reinterpret_cast<int *>(ws + t.rows), *lens = reinterpret_cast<int *>(ws + t.lens);
        if (ragged) {
            p.rows = rows;
            p.lens = lens;
        }
        causal_rows_kernel<<<ragged ? a.batch : 1, 128, 0, stream>>>(a, ragged ? rows : nullptr, lens, p.flags,
                                                     p.order == kOrderHandoff ? sms : 0);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    if (p.order == kOrderNatural) {
        TcParams st = p;
        st.order = kOrderState;
        if ((e = launch_tc<N, true>(tx, tb, tc, st, sms, first, stream)) != cudaSuccess) return e;
        causal_chain_kernel<N><<<sms * (64 * N / 1024), 256, 0, stream>>>(p, sms);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
        return launch_tc<N, false>(tx, tb, tc, p, sms, true, stream);
    }
    return launch_tc<N, false>(tx, tb, tc, p, p.order == kOrderWhole ? (int)units : sms, first, stream);
}

}  // namespace

size_t causal_tc_scratch_bytes(int batch, int N) {
    const int sms = device_sms();
    return tc_scratch(batch, sms > 0 ? sms : 148, N).total;
}

cudaError_t launch_causal_tc(const CausalArgs &a, void *scratch, cudaStream_t stream) {
    return a.N == 128 ? run_tc<128>(a, scratch, stream) : run_tc<64>(a, scratch, stream);
}

}  // namespace ssd
