// Single tokens of the causal scan: for every row b of a batch and head h
//   H <- exp(dt A_h) H + dt x B^T,   y = H C + D x
// with the (P, N) fp32 state H read from and written to the row's page of a
// pool. 5 N P operations on 8 N P bytes: the state's traffic is all that
// counts (24 heads x 64 x 128: 1.57 MB a row in and out, the other operands
// 25 KB at most).
//
// A warp takes whole rows p of a state, 16 bytes (four n) a lane, so every
// load and store covers full 128-byte lines, and each lane keeps its four
// values of B and C in registers for all of its warp's rows. All loads of a
// thread (one for each of its rows) are in flight before the first use. The
// rows' dot products with C meet in one butterfly that halves the number of
// rows a lane carries at each step.
//
// Measured, N = 128: fp32, 512 rows of a pool x 32 heads of 64 (1.09 GB) 167 us, 6.5
// TB/s, the rate of a plain copy; bf16, 244 rows and 6 of padding x 24 heads of 64 (385
// MB) 64.5 us, 6.0 TB/s; one row 4.7 us from cold memory. Eight loads a
// thread: 64 rows in L2 take 10.5 us (16 loads 11.3, 4 loads 12.4), 12 rows 3.4 us
// (3.5, 3.8); CTAs of 8 warps are slower at every size (12.9, 3.9).
#include <stdint.h>

#include "ssd_causal.h"
#include "ssd_kernels.h"

namespace ssd {
namespace {

constexpr int kWarps = 4;
constexpr int kRows = 8;      // loads of a thread in flight

__device__ __forceinline__ float4 load4(const float *p) { return __ldg(reinterpret_cast<const float4 *>(p)); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16 *p) {
    const uint2 v = __ldg(reinterpret_cast<const uint2 *>(p));
    return make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u), __uint_as_float(v.y << 16),
                       __uint_as_float(v.y & 0xffff0000u));
}

// One CTA: kWarps warps x ROWS x PER state rows of one (row b, head h). For N =
// 64 a warp's two halves take a row each.
template <typename T, int N, int ROWS>
__global__ void __launch_bounds__(32 * kWarps)
causal_step_kernel(const CausalArgs a) {
    constexpr int LANES = N / 4;                    // lanes of a state row
    constexpr int PER = 32 / LANES;                 // rows a warp loads at once
    constexpr int CTA_ROWS = kWarps * PER * ROWS;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int parts = a.P / CTA_ROWS;
    const int unit = blockIdx.x / parts;
    const int b = unit / a.H, h = unit % a.H;
    const int p0 = (blockIdx.x % parts) * CTA_ROWS + warp * PER * ROWS + lane / LANES;   // + PER * r
    const int n0 = (lane % LANES) * 4;

    int row = b;
    bool skip = false;
    if (a.rows) {
        row = a.rows[b];
        skip = row < 0;
    } else if (a.slots) {
        row = a.slots[b];
        skip = row < 0 || row >= a.nslots;
    }
    const size_t page = ((size_t)(skip ? 0 : row) * a.H + h) * a.P;
    float4 s[ROWS];
    if (!skip) {
        const float *src = a.init + (page + p0) * N + n0;
#pragma unroll
        for (int r = 0; r < ROWS; ++r) s[r] = *reinterpret_cast<const float4 *>(src + (size_t)r * PER * N);
    }
    if (a.slots && !a.rows) {
        // a page belongs to the first row that names it: a later one is skipped
        const int tag = row;
        bool again = false;
        if (!skip)
            for (int i = threadIdx.x; i < b; i += 32 * kWarps) again |= a.slots[i] == tag;
        again = __syncthreads_or(again);
        if ((again || (skip && row != -1)) && threadIdx.x == 0) report(a.status, kFlagIndex);
        skip |= again;
    }
    T *out = static_cast<T *>(a.out) + ((size_t)b * a.H + h) * a.P;
    if (skip) {
        for (int i = threadIdx.x; i < CTA_ROWS; i += 32 * kWarps)
            IO<T>::store(out + (blockIdx.x % parts) * CTA_ROWS + i, 0.f);
        return;
    }
    const int g = h / (a.H / a.G);
    const T *xp = static_cast<const T *>(a.x) + (size_t)b * a.x_sb + (size_t)h * a.P;
    const float4 Bv = load4(static_cast<const T *>(a.B) + (size_t)b * a.b_sb + (size_t)g * N + n0);
    const float4 Cv = load4(static_cast<const T *>(a.C) + (size_t)b * a.c_sb + (size_t)g * N + n0);
    const float dt = a.step(IO<T>::load(static_cast<const T *>(a.dt) + (size_t)b * a.dt_sb + h), h);
    float x[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) x[r] = IO<T>::load(xp + p0 + r * PER);
    const float decay = expf(dt * a.A[h]), D = a.D ? a.D[h] : 0.f;

    float y[ROWS];
    float *dst = a.state_out + (page + p0) * N + n0;
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        const float u = dt * x[r];
        s[r].x = fmaf(decay, s[r].x, u * Bv.x);
        s[r].y = fmaf(decay, s[r].y, u * Bv.y);
        s[r].z = fmaf(decay, s[r].z, u * Bv.z);
        s[r].w = fmaf(decay, s[r].w, u * Bv.w);
        *reinterpret_cast<float4 *>(dst + (size_t)r * PER * N) = s[r];
        y[r] = fmaf(s[r].x, Cv.x, s[r].y * Cv.y) + fmaf(s[r].z, Cv.z, s[r].w * Cv.w);
    }
    // halve the rows a lane carries while lanes remain, then plain sums: a lane
    // ends with row `keep` of its ROWS
    int keep = 0, o = LANES / 2;
#pragma unroll
    for (int m = ROWS / 2; m >= 1; m >>= 1, o >>= 1) {
        const bool up = lane & o;
#pragma unroll
        for (int r = 0; r < m; ++r) {
            const float send = up ? y[r] : y[r + m];
            const float mine = up ? y[r + m] : y[r];
            y[r] = mine + __shfl_xor_sync(0xffffffffu, send, o);
        }
        keep += up ? m : 0;
    }
    for (; o >= 1; o >>= 1) y[0] += __shfl_xor_sync(0xffffffffu, y[0], o);
    if ((lane & (LANES / ROWS - 1)) == 0) {
        const int p = p0 + keep * PER;
        IO<T>::store(out + p, a.D ? fmaf(D, IO<T>::load(xp + p), y[0]) : y[0]);
    }
}

template <typename T, int N>
cudaError_t run(const CausalArgs &a, cudaStream_t stream) {
    constexpr int PER = 32 / (N / 4);
    const long long grid = (long long)a.batch * a.H * (a.P / (kWarps * PER * kRows));
    if (grid > 0x7fffffffLL) return cudaErrorNotSupported;
    causal_step_kernel<T, N, kRows><<<(unsigned)grid, 32 * kWarps, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_causal_step(const CausalArgs &a, cudaStream_t stream) {
    if (a.bf16) return a.N == 128 ? run<__nv_bfloat16, 128>(a, stream) : run<__nv_bfloat16, 64>(a, stream);
    return a.N == 128 ? run<float, 128>(a, stream) : run<float, 64>(a, stream);
}

}  // namespace ssd
