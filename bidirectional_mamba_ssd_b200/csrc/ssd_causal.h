// Internal interface of the causal (forward-only) serving operators: prompts
// (ssd_causal.cu), single tokens (ssd_causal_step.cu) and the pages of a pool
// of states (ssd_cache.cu). The C ABI is in ssd_causal_api.cu.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>

#include "ssd_common.cuh"

namespace ssd {

// Step size of one token and head: as given, or from the raw projection as
// min(max(softplus(raw + bias), lo), hi). Past u = 20 softplus(u) - u is below
// e^-20 = 2^-28.9, less than half an ulp of u in fp32.
static __device__ __noinline__ float softplus(float u) { return u > 20.f ? u : log1pf(expf(u)); }
struct StepSize {
    const float *bias;   // (H) or nullptr: the step size is used as given
    float lo, hi;
    __device__ __forceinline__ float operator()(float v, int h) const {
        return with(v, bias ? bias[h] : 0.f);
    }
    // the same with the head's bias at hand
    __device__ __forceinline__ float with(float v, float b) const {
        if (!bias) return v;
        const float s = softplus(v + b);
        return s < lo ? lo : s > hi ? hi : s;      // (fminf and fmaxf would make a limit of a NaN)
    }
};

// Arguments of the causal kernels. Strides are in elements; (H, P) and (G, N)
// are contiguous in every tensor.
struct CausalArgs {
    const void *x, *dt, *B, *C;   // io
    const float *A, *D;           // (H); D nullptr: no skip term
    StepSize step;
    const int *seqlens;           // (batch) or nullptr: every sequence has L tokens
    const int *slots;             // (batch) as the caller gave them, or nullptr
    const int *rows;              // (batch) resolved slots, -1 = skip the row; nullptr = row b
    const float *init;            // start states, row rows[b] (or b), nullptr = zero
    float *state_out;             // end states, or nullptr
    void *out;                    // (batch, L, H, P) io, contiguous
    long long x_sb, x_st, dt_sb, dt_st, b_sb, b_st, c_sb, c_st;
    DeviceStatus *status;
    int batch, L, H, P, G, N, nslots;
    bool bf16;

    __device__ __forceinline__ int len(int b) const {
        if (!seqlens) return L;
        const int v = seqlens[b];
        return v < 0 ? 0 : v > L ? L : v;
    }
};

// Sequences cut into segments of whole tiles where the units alone do not fill
// the GPU: the segments' own end states and decays, then each segment's start.
struct CausalSegments {
    int count = 1;        // segments per sequence; 1 = not cut
    int tokens = 0;       // tokens of a segment (the last one may be shorter)
    float *state = nullptr;   // (batch, H, count, P, N): own end states, then the states entering
    float *decay = nullptr;   // (batch, H, count)
};

enum { kCausalOutput = 0, kCausalState = 1 };

// rows[b] = slots[b], or -1 where the row is padding (-1), out of range or named
// by an earlier row (the last two set kFlagIndex).
cudaError_t launch_resolve_slots(const int *slots, int batch, int nslots, int *rows, DeviceStatus *st,
                                 cudaStream_t stream);

// CUDA-core scan, fp32 arithmetic, either I/O dtype (ssd_causal.cu).
void causal_simt_segments(int batch, int L, int H, int P, int N, int sms, int *count, int *tokens);
cudaError_t launch_causal_simt(const CausalArgs &a, const CausalSegments &s, int mode, cudaStream_t stream);
// Own end states -> states entering every segment (the start state included).
cudaError_t launch_causal_carry(const CausalArgs &a, const CausalSegments &s, cudaStream_t stream);

// Tensor-core scan (ssd_causal_tc.cu), bf16 I/O, L >= 1: resolves slots and lengths
// by itself; `scratch` is behind the workspace's status header.
size_t causal_tc_scratch_bytes(int batch, int N);
cudaError_t launch_causal_tc(const CausalArgs &a, void *scratch, cudaStream_t stream);

cudaError_t launch_causal_step(const CausalArgs &a, cudaStream_t stream);

// ssd_workspace_bytes of the causal operators (0: sizes they reject).
size_t causal_workspace_bytes(int op, int batch, int seqlen, int nheads, int headdim, int dstate, int ngroups, int dtype);

struct CacheArgs {
    void *pool;
    long long page_bytes;
    int layers, nslots;
    const int *src, *dst;   // copy
    int n;
    const int *table;       // compact
    int rows;
    int *table_out, *live_out;
    DeviceStatus *status;
};
constexpr int kCacheMaxSlots = 1 << 18;   // two 32 KB maps in shared memory
cudaError_t launch_cache_copy(const CacheArgs &a, cudaStream_t stream);
cudaError_t launch_cache_compact(const CacheArgs &a, cudaStream_t stream);

}  // namespace ssd
