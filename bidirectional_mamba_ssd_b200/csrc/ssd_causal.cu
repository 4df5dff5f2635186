// The causal scan over prompts on CUDA cores, in fp32 whatever the I/O type,
// token by token:
//   H <- exp(dt_t A_h) H + dt_t x_t B_t^T,   y_t = H C_t + D x_t
// and the pieces that every path of the prompts shares: the resolving of pool
// slots and the carry of states across segments.
//
// The state's columns p do not depend on one another, so a CTA takes COLS of a
// head's P columns and walks its tokens with that part of the state in
// registers: a thread owns 4 p x 8 n and works on four tokens at a step, with
// arithmetic packed two to an instruction (f32x2); the 16 outputs of a step meet the other
// n in one butterfly that halves the values a lane carries. The four tokens share one
// rescaling of the state: with d_s the decay behind token s among the four,
//   H <- exp(all) H ahead of the first, H <- H + exp(d_s) dt_s x_s B_s^T, y_t = exp(-d_t) H C_t
// leaves the state itself behind the fourth (d = 0). Where the four decay by more than
// e^-8 they go one by one, by the same code with the others' terms left out. Tokens arrive
// in chunks of kTok through cp.async, two chunks deep.
// What bounds it: with many units instruction issue and shared memory together (fp32, 64
// sequences of even lengths up to 500 tokens, 24 heads of 64, N = 128: 477 us; token by token
// with a butterfly each 543, with a rescaling each as well 581; 64 columns a CTA 557, 16 517; 64
// full sequences 837, and 2877 where four tokens decay by more than e^-8), with few a warp's own
// time per token; there the sequence is cut into segments (own end states, a carry, then
// the outputs), which costs a second pass over x and B.
#include <stdint.h>

#include "ssd_causal.h"
#include "ssd_kernels.h"

namespace ssd {
namespace {

constexpr int kTok = 16;
constexpr int KP = 4;       // columns of a thread

typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 pack2(float lo, float hi) {
    f32x2 d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
    return d;
}
__device__ __forceinline__ float2 unpack2(f32x2 v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
    f32x2 d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
    f32x2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}

// 16 bytes, zeros where `there` is false (the address is not read)
__device__ __forceinline__ void cp_async16(void *dst, const void *src, bool there) {
    const uint32_t d = static_cast<uint32_t>(__cvta_generic_to_shared(dst));
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group 0;" ::: "memory"); }

// four consecutive elements of shared memory
__device__ __forceinline__ float4 lds4(const float *p) { return *reinterpret_cast<const float4 *>(p); }
__device__ __forceinline__ float4 lds4(const __nv_bfloat16 *p) {
    const uint2 v = *reinterpret_cast<const uint2 *>(p);
    return make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u), __uint_as_float(v.y << 16),
                       __uint_as_float(v.y & 0xffff0000u));
}

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void store_row(float *p, const float (&v)[1]) { p[0] = v[0]; }
__device__ __forceinline__ void store_row(float *p, const float (&v)[2]) { *reinterpret_cast<float2 *>(p) = make_float2(v[0], v[1]); }
__device__ __forceinline__ void store_row(__nv_bfloat16 *p, const float (&v)[1]) { p[0] = __float2bfloat16_rn(v[0]); }
__device__ __forceinline__ void store_row(__nv_bfloat16 *p, const float (&v)[2]) {
    *reinterpret_cast<__nv_bfloat162 *>(p) = __floats2bfloat162_rn(v[0], v[1]);
}

template <typename T, int N, int COLS>
struct SimtSmem {
    T B[2][kTok][N], C[2][kTok][N], x[2][kTok][COLS];
    float4 f[2][kTok];    // a token's factors: of the state ahead of it, of x B^T, of the output; 1 if its four go one by one
};

// Decay of four tokens up to which they share one rescaling of the state: e^d carries
// the rounding of d, 2^-24 of it, to the terms of the same four.
constexpr float kMaxQuad = 8.f;

template <typename T, int N, int COLS, int MODE>
__global__ void __launch_bounds__(COLS *N / (8 * KP), 1)
causal_simt_kernel(const CausalArgs a, const CausalSegments sg) {
    constexpr int THREADS = COLS * N / (8 * KP);
    constexpr int NG = N / 8;                 // lanes that share a column
    constexpr bool OUT = MODE == kCausalOutput;
    using S = SimtSmem<T, N, COLS>;
    extern __shared__ __align__(16) uint8_t raw[];
    S &sm = *reinterpret_cast<S *>(raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int gn = lane % NG, cg = (warp * 32 + lane) / NG;   // n group, column group (KP columns)
    const int parts = a.P / COLS;
    const int part = blockIdx.x % parts;
    const int seg = (blockIdx.x / parts) % sg.count;
    const int bh = blockIdx.x / parts / sg.count;
    const int b = bh / a.H, h = bh % a.H;
    const int len = a.len(b), first = seg * sg.tokens;
    const int stop = sg.count == 1 ? a.L : min(a.L, first + sg.tokens);   // rows of this segment
    const int end = max(first, min(len, stop));                           // the ones that hold tokens
    const int row = a.rows ? a.rows[b] : b;
    T *out = static_cast<T *>(a.out) + ((size_t)b * a.L * a.H + h) * a.P + part * COLS;   // + t H P
    // zero rows [t, stop): behind the sequence, or the whole row of a skipped one
    auto blank = [&](int t) {
        constexpr int PIECES = COLS * (int)sizeof(T) / 16;
        static_assert(THREADS % PIECES == 0, "whole rows at a step");
        for (int r = t + tid / PIECES; r < stop; r += THREADS / PIECES)
            reinterpret_cast<uint4 *>(out + (size_t)r * a.H * a.P)[tid % PIECES] = make_uint4(0, 0, 0, 0);
    };
    if (row < 0) {
        if (OUT) blank(first);
        return;
    }
    if (!OUT && first + sg.tokens >= len) return;   // no segment behind this one reads its state
    const T *xp = static_cast<const T *>(a.x) + (long long)b * a.x_sb + (size_t)h * a.P + part * COLS;
    const int g = h / (a.H / a.G);
    const T *Bp = static_cast<const T *>(a.B) + (long long)b * a.b_sb + (size_t)g * N;
    const T *Cp = static_cast<const T *>(a.C) + (long long)b * a.c_sb + (size_t)g * N;
    const T *dtp = static_cast<const T *>(a.dt) + (long long)b * a.dt_sb + h;
    const float A = a.A[h], D = OUT && a.D ? a.D[h] : 0.f;

    // state: element (KP cg + k, n) with n = 4 gn + i (i < 4) and N / 2 + 4 gn + i
    f32x2 H[KP][4];
    const size_t col = (size_t)part * COLS + KP * cg;
    const float *start = nullptr;
    if (OUT && sg.count > 1) start = sg.state + (((size_t)bh * sg.count + seg) * a.P + col) * N;
    else if (OUT && a.init) start = a.init + (((size_t)row * a.H + h) * a.P + col) * N;
#pragma unroll
    for (int k = 0; k < KP; ++k)
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            if (start) v = *reinterpret_cast<const float4 *>(start + (size_t)k * N + q * (N / 2) + 4 * gn);
            H[k][2 * q] = pack2(v.x, v.y);
            H[k][2 * q + 1] = pack2(v.z, v.w);
        }

    float raw_dt = 0.f;
    auto fetch = [&](int t0, int buf) {
        const int m = min(kTok, end - t0);
        constexpr int EPC = 16 / (int)sizeof(T);
#pragma unroll
        for (int i = tid; i < kTok * (N / EPC); i += THREADS) {
            const int t = i / (N / EPC), c = (i % (N / EPC)) * EPC;
            const long long at = t0 + (t < m ? t : 0);
            cp_async16(&sm.B[buf][t][c], Bp + at * a.b_st + c, t < m);
            if (OUT) cp_async16(&sm.C[buf][t][c], Cp + at * a.c_st + c, t < m);
        }
#pragma unroll
        for (int i = tid; i < kTok * (COLS / EPC); i += THREADS) {
            const int t = i / (COLS / EPC), c = (i % (COLS / EPC)) * EPC;
            cp_async16(&sm.x[buf][t][c], xp + (t0 + (t < m ? t : 0)) * a.x_st + c, t < m);
        }
        cp_commit();
        if (tid < m) raw_dt = IO<T>::load(dtp + (long long)(t0 + tid) * a.dt_st);
    };
    float sum = 0.f;          // sum of the step sizes (thread t < kTok: its tokens' share)
    int buf = 0;
    if (first < end) fetch(first, 0);
    for (int t0 = first; t0 < end; t0 += kTok, buf ^= 1) {
        const int m = min(kTok, end - t0);
        if (warp == 0) {
            const float v = tid < m ? a.step(raw_dt, h) : 0.f;
            const float v1 = __shfl_down_sync(0xffffffffu, v, 1), v2 = __shfl_down_sync(0xffffffffu, v, 2),
                        v3 = __shfl_down_sync(0xffffffffu, v, 3);
            const int q = lane & 3;
            const float after = (q < 3 ? v1 : 0.f) + (q < 2 ? v2 : 0.f) + (q < 1 ? v3 : 0.f);
            const float all = A * __shfl_sync(0xffffffffu, v + after, lane & ~3), d = A * after;
            const bool quad = fabsf(all) <= kMaxQuad;
            if (tid < kTok)
                sm.f[buf][tid] = quad ? make_float4(expf(all), expf(d) * v, expf(-d), 0.f) : make_float4(expf(v * A), v, 1.f, 1.f);
            sum += v;
        }
        cp_wait();
        __syncthreads();      // chunk here; the other buffer is read by nobody
        if (t0 + kTok < end) fetch(t0 + kTok, buf ^ 1);
        // four tokens at a time (the last chunk's are filled up with zeros), or, where they
        // go one by one, one of the four at a time
#pragma unroll 1
        for (int j = 0; j < m;) {
            const bool single = sm.f[buf][j].w != 0.f;
            const int t4 = j & ~3;
            const f32x2 G = pack2(sm.f[buf][j].x, sm.f[buf][j].x);
#pragma unroll
            for (int k = 0; k < KP; ++k)
#pragma unroll
                for (int q = 0; q < 4; ++q) H[k][q] = mul2(H[k][q], G);
            float y[4 * KP];      // of token i and column k: y[KP * i + k]
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int t = t4 + i;
                const float fy = !single || t == j ? sm.f[buf][t].y : 0.f;
                const float4 x = lds4(&sm.x[buf][t][KP * cg]);
                const float xs[KP] = {x.x, x.y, x.z, x.w};
                const float4 b0 = lds4(&sm.B[buf][t][4 * gn]), b1 = lds4(&sm.B[buf][t][N / 2 + 4 * gn]);
                const f32x2 Bv[4] = {pack2(b0.x, b0.y), pack2(b0.z, b0.w), pack2(b1.x, b1.y), pack2(b1.z, b1.w)};
#pragma unroll
                for (int k = 0; k < KP; ++k) {
                    const float u = fy * xs[k];
                    const f32x2 U = pack2(u, u);
#pragma unroll
                    for (int q = 0; q < 4; ++q) H[k][q] = fma2(U, Bv[q], H[k][q]);
                }
                if (OUT) {
                    const float4 c0 = lds4(&sm.C[buf][t][4 * gn]), c1 = lds4(&sm.C[buf][t][N / 2 + 4 * gn]);
                    const f32x2 Cv[4] = {pack2(c0.x, c0.y), pack2(c0.z, c0.w), pack2(c1.x, c1.y), pack2(c1.z, c1.w)};
#pragma unroll
                    for (int k = 0; k < KP; ++k) {
                        const f32x2 s = fma2(H[k][3], Cv[3], fma2(H[k][2], Cv[2], fma2(H[k][1], Cv[1], mul2(H[k][0], Cv[0]))));
                        const float2 v = unpack2(s);
                        y[KP * i + k] = v.x + v.y;
                    }
                }
            }
            if (OUT) {
                // butterfly over the NG lanes of a column group: each step halves the values a
                // lane carries, until it has one column (NG = 16) or two (8) of one token
                constexpr int LEFT = 4 * KP / NG;
#pragma unroll
                for (int n = 2 * KP, o = NG / 2; o >= 1; n >>= 1, o >>= 1) {
                    const bool up = gn & o;
#pragma unroll
                    for (int k = 0; k < n; ++k) {
                        const float send = up ? y[k] : y[k + n], mine = up ? y[k + n] : y[k];
                        y[k] = mine + __shfl_xor_sync(0xffffffffu, send, o);
                    }
                }
                const int first_of = gn * LEFT, t = t4 + first_of / KP, k = KP * cg + first_of % KP;
                if (t < m && (!single || t == j)) {
                    const float fz = sm.f[buf][t].z;
                    T *dst = out + (size_t)(t0 + t) * a.H * a.P + k;
                    float v[LEFT];
#pragma unroll
                    for (int q = 0; q < LEFT; ++q) {
                        v[q] = fz * y[q];
                        if (a.D) v[q] = fmaf(D, to_float(sm.x[buf][t][k + q]), v[q]);
                    }
                    store_row(dst, v);
                }
            }
            j = single ? j + 1 : t4 + 4;
        }
    }
    if (OUT) blank(end);
    // the state behind the last token: the sequence's own, or the segment's
    float *last = nullptr;
    if (!OUT) {
        last = sg.state + (((size_t)bh * sg.count + seg) * a.P + col) * N;
        // decay over the segment: thread t holds the step sizes of tokens t mod kTok
        if (warp == 0) {
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            if (lane == 0 && part == 0) sg.decay[(size_t)bh * sg.count + seg] = expf(sum * A);
        }
    } else if (a.state_out && (sg.count == 1 || (end > first && end == len) || (len == 0 && seg == 0))) {
        last = a.state_out + (((size_t)row * a.H + h) * a.P + col) * N;
    }
    if (last) {
#pragma unroll
        for (int k = 0; k < KP; ++k)
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const float2 u = unpack2(H[k][2 * q]), v = unpack2(H[k][2 * q + 1]);
                *reinterpret_cast<float4 *>(last + (size_t)k * N + q * (N / 2) + 4 * gn) = make_float4(u.x, u.y, v.x, v.y);
            }
    }
}

// One CTA per row: a row is padding (-1), out of range, named by an earlier
// row, or its own slot.
__global__ void __launch_bounds__(128) resolve_slots_kernel(const int *slots, int nslots, int *rows, DeviceStatus *st) {
    const int b = blockIdx.x, s = slots[b];
    bool bad = s < -1 || s >= nslots;
    bool again = false;
    if (s >= 0)
        for (int i = threadIdx.x; i < b; i += 128) again |= slots[i] == s;
    bad |= (bool)__syncthreads_or(again);
    if (threadIdx.x == 0) {
        rows[b] = bad ? -1 : s;
        if (bad) report(st, kFlagIndex);
    }
}

// Own end states of the segments -> the states entering them, in place: thread
// by thread over a state's elements, in the order of the segments.
__global__ void __launch_bounds__(256) causal_carry_kernel(const CausalArgs a, const CausalSegments sg) {
    const int per = a.P * a.N / 4;
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
    if (i >= (long long)a.batch * a.H * per) return;
    const long long bh = i / per;
    const int e = (int)(i % per);
    const int b = (int)(bh / a.H), h = (int)(bh % a.H);
    const int row = a.rows ? a.rows[b] : b;
    if (row < 0) return;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (a.init) s = reinterpret_cast<const float4 *>(a.init)[((size_t)row * a.H + h) * per + e];
    float4 *st = reinterpret_cast<float4 *>(sg.state) + bh * sg.count * per + e;
    const float *dc = sg.decay + bh * sg.count;
    // segments that start behind the sequence are never read
    const int n = max(1, min(sg.count, (a.len(b) + sg.tokens - 1) / sg.tokens));
    constexpr int kAhead = 8;              // loads in flight
    for (int g = 0; g < n; g += kAhead) {
        float4 own[kAhead];
        float d[kAhead];
#pragma unroll
        for (int q = 0; q < kAhead; ++q)
            if (g + q + 1 < n) {
                own[q] = st[(size_t)(g + q) * per];
                d[q] = dc[g + q];
            }
#pragma unroll
        for (int q = 0; q < kAhead; ++q)
            if (g + q < n) {
                st[(size_t)(g + q) * per] = s;
                if (g + q + 1 < n)
                    s = make_float4(fmaf(d[q], s.x, own[q].x), fmaf(d[q], s.y, own[q].y), fmaf(d[q], s.z, own[q].z),
                                    fmaf(d[q], s.w, own[q].w));
            }
    }
}

// Columns of a CTA: 128 threads. fp32, even lengths up to the one given, 32 and 64 columns: 4 x
// 777 tokens, 8 heads of 128, N = 64 49.5 and 46.6 us, 100 x 300 tokens 184 and 176; N = 128, 64 x
// 500 tokens, 24 heads of 64 477 and 557. (With the registers that a kernel without a bound on its CTAs
// gets, 32 columns of N = 128 and 64 of N = 64 take 483, 50.2 and 165.)
constexpr int cols_of(int N) { return 4096 / N; }

template <typename T, int N>
cudaError_t run_simt(const CausalArgs &a, const CausalSegments &s, int mode, cudaStream_t stream) {
    constexpr int COLS = cols_of(N);
    const long long grid = (long long)a.batch * a.H * s.count * (a.P / COLS);
    if (grid > 0x7fffffffLL) return cudaErrorNotSupported;
    const int threads = COLS * N / (8 * KP);
    const size_t smem = sizeof(SimtSmem<T, N, COLS>);
    static_assert(sizeof(SimtSmem<T, N, COLS>) <= 48 * 1024, "shared memory within the default limit");
    if (mode == kCausalOutput) causal_simt_kernel<T, N, COLS, kCausalOutput><<<(unsigned)grid, threads, smem, stream>>>(a, s);
    else causal_simt_kernel<T, N, COLS, kCausalState><<<(unsigned)grid, threads, smem, stream>>>(a, s);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_resolve_slots(const int *slots, int batch, int nslots, int *rows, DeviceStatus *st,
                                 cudaStream_t stream) {
    resolve_slots_kernel<<<batch, 128, 0, stream>>>(slots, nslots, rows, st);
    return cudaGetLastError();
}

// Segments of at least 64 tokens, as many as it takes to give every SM 16 warps of
// work (4 x 777 tokens, 8 heads of 128, N = 64, at 32 columns: 49.5 us; with 24 warps 52,
// 12 warps 50; segments of at least 48 tokens 47, but one sequence of 100 tokens is then cut in two
// and takes 12.6 us instead of 7.0).
void causal_simt_segments(int batch, int L, int H, int P, int N, int sms, int *count, int *tokens) {
    const int cols = cols_of(N);
    const long long ctas = (long long)batch * H * (P / cols);
    const long long want = 16LL * sms / (cols * N / 1024);
    long long n = ctas > 0 ? want / ctas : 1;
    const long long most = L / 64;
    n = n < most ? n : most;
    if (n < 2) {
        *count = 1;
        *tokens = L;
        return;
    }
    *tokens = (int)((L + n - 1) / n);
    *count = (L + *tokens - 1) / *tokens;
}

cudaError_t launch_causal_simt(const CausalArgs &a, const CausalSegments &s, int mode, cudaStream_t stream) {
    if (a.bf16) return a.N == 128 ? run_simt<__nv_bfloat16, 128>(a, s, mode, stream) : run_simt<__nv_bfloat16, 64>(a, s, mode, stream);
    return a.N == 128 ? run_simt<float, 128>(a, s, mode, stream) : run_simt<float, 64>(a, s, mode, stream);
}

cudaError_t launch_causal_carry(const CausalArgs &a, const CausalSegments &s, cudaStream_t stream) {
    const long long threads = (long long)a.batch * a.H * a.P * a.N / 4;
    causal_carry_kernel<<<(unsigned)((threads + 255) / 256), 256, 0, stream>>>(a, s);
    return cudaGetLastError();
}

}  // namespace ssd
