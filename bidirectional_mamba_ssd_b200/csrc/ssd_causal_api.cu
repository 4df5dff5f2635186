// C ABI of the causal serving operators: argument checks, workspace layout and
// dispatch. Declarations and documentation: include/ssd_bidir.h.
#include <stdint.h>

#include "ssd_bidir.h"
#include "ssd_causal.h"
#include "ssd_kernels.h"

using ssd::CausalArgs;
using ssd::CausalSegments;

namespace {

bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
size_t round256(size_t v) { return (v + 255) & ~(size_t)255; }

int to_status(cudaError_t e) {
    if (e == cudaSuccess) return SSD_OK;
    return e == cudaErrorNotSupported ? SSD_ERR_UNSUPPORTED : SSD_ERR_CUDA;
}

int check_sizes(int batch, int seqlen, int nheads, int headdim, int dstate, int ngroups, int dtype) {
    if (batch < 0 || seqlen < 0 || nheads <= 0 || headdim <= 0 || dstate <= 0 || ngroups <= 0) return SSD_ERR_INVALID_ARG;
    if (nheads % ngroups != 0) return SSD_ERR_INVALID_ARG;
    if (dtype != SSD_F32 && dtype != SSD_BF16) return SSD_ERR_UNSUPPORTED;
    if (headdim % 64 != 0 || headdim > 256) return SSD_ERR_UNSUPPORTED;
    if (dstate != 64 && dstate != 128) return SSD_ERR_UNSUPPORTED;
    if ((long long)batch * seqlen > (1ll << 31) - 1) return SSD_ERR_UNSUPPORTED;
    // every kernel's grid and unit counts stay in int
    if ((long long)batch * nheads * (headdim / 16) > (1ll << 31) - 1) return SSD_ERR_UNSUPPORTED;
    if ((long long)nheads * headdim > (1 << 24) || (long long)ngroups * dstate > (1 << 24)) return SSD_ERR_UNSUPPORTED;
    return SSD_OK;
}

// Rows of `inner` contiguous elements, `stride` elements apart (ignored for a
// single row): at least a row apart, whole 16-byte steps where `vec`, within the
// range of a tensor map.
bool stride_ok(long long &stride, long long n, long long inner, int elem, bool vec) {
    if (n <= 1) stride = inner;
    if (stride < inner || stride >= (1ll << 36)) return false;
    return !vec || stride * elem % 16 == 0;
}

int sm_count() {
    const int n = ssd::device_sms();
    return n > 0 ? n : 148;
}

// Workspace of the CUDA-core scan: status header, resolved rows, segment states.
struct Plan {
    CausalSegments seg;
    size_t rows, state, decay, total;
};
Plan plan(int batch, int seqlen, int nheads, int headdim, int dstate) {
    Plan p{};
    ssd::causal_simt_segments(batch, seqlen, nheads, headdim, dstate, sm_count(), &p.seg.count, &p.seg.tokens);
    size_t o = ssd::kStatusBytes;
    p.rows = o;
    o += round256(sizeof(int) * (size_t)batch);
    if (p.seg.count > 1) {
        const size_t units = (size_t)batch * nheads * p.seg.count;
        p.state = o;
        o += round256(sizeof(float) * units * headdim * dstate);
        p.decay = o;
        o += round256(sizeof(float) * units);
    }
    p.total = o;
    return p;
}

// SSD_PATH_AUTO: bf16 on the tensor cores, fp32 (and an empty sequence, whose end
// state is its start state) on the CUDA cores.
int causal_path(int path, int seqlen, int dtype) {
    if (path == SSD_PATH_AUTO) path = dtype == SSD_BF16 ? SSD_PATH_FUSED : SSD_PATH_SIMT;
    return seqlen == 0 ? SSD_PATH_SIMT : path;
}

size_t fwd_bytes(int path, int batch, int seqlen, int nheads, int headdim, int dstate) {
    return path == SSD_PATH_FUSED ? ssd::kStatusBytes + ssd::causal_tc_scratch_bytes(batch, dstate)
                                  : plan(batch, seqlen, nheads, headdim, dstate).total;
}

// Rows from which the single-token kernel's CTAs no longer look for repeated
// slots by themselves (each reads the slots ahead of its row) and a kernel ahead of it
// does. Four heads of 64 x 64, the search in the CTAs and ahead of them: 256 rows 5.4
// and 6.6 us, 1024 15.8 and 16.2, 4096 88.3 and 89.2, 8192 181 and 177.
constexpr int kScanRows = 2048;

}  // namespace

namespace ssd {
size_t causal_workspace_bytes(int op, int batch, int seqlen, int nheads, int headdim, int dstate, int ngroups, int dtype) {
    if (check_sizes(batch, seqlen, nheads, headdim, dstate, ngroups, dtype) != SSD_OK) return 0;
    if (op == SSD_OP_CAUSAL_STEP) return kStatusBytes + (batch > kScanRows ? round256(sizeof(int) * (size_t)batch) : 0);
    // whichever path is asked for
    const size_t s = fwd_bytes(SSD_PATH_SIMT, batch, seqlen, nheads, headdim, dstate);
    const size_t t = dtype == SSD_BF16 ? fwd_bytes(SSD_PATH_FUSED, batch, seqlen, nheads, headdim, dstate) : 0;
    return s > t ? s : t;
}
}  // namespace ssd

extern "C" {

int ssd_causal_fwd(const void *x, const void *dt, const float *A, const void *B, const void *C, const float *D,
                   const float *dt_bias, float dt_min, float dt_max, const int *seqlens, const int *slots,
                   const float *init_state, float *state_out, void *out, long long x_batch, long long x_token,
                   long long dt_batch, long long dt_token, long long B_batch, long long B_token, long long C_batch,
                   long long C_token, int nslots, int batch, int seqlen, int nheads, int headdim, int dstate,
                   int ngroups, int dtype, int path, void *workspace, size_t ws_bytes, void *stream) {
    const int rc = check_sizes(batch, seqlen, nheads, headdim, dstate, ngroups, dtype);
    if (rc != SSD_OK) return rc;
    if (path != SSD_PATH_AUTO && path != SSD_PATH_SIMT && path != SSD_PATH_FUSED) return SSD_ERR_INVALID_ARG;
    if (path == SSD_PATH_FUSED && dtype != SSD_BF16) return SSD_ERR_UNSUPPORTED;
    if (!workspace) return SSD_ERR_WORKSPACE;
    if (!aligned(workspace, 16)) return SSD_ERR_INVALID_ARG;
    path = causal_path(path, seqlen, dtype);
    if (ws_bytes < fwd_bytes(path, batch, seqlen, nheads, headdim, dstate)) return SSD_ERR_WORKSPACE;
    if (dt_bias && (!(dt_min >= 0.f) || !(dt_max >= dt_min))) return SSD_ERR_INVALID_ARG;
    if (slots && nslots < 0) return SSD_ERR_INVALID_ARG;
    if (batch == 0) return SSD_OK;
    if (!aligned(init_state, 16) || !aligned(state_out, 16) || !aligned(D, 4) || !aligned(dt_bias, 4) ||
        !aligned(seqlens, 4) || !aligned(slots, 4))
        return SSD_ERR_INVALID_ARG;
    const int e = dtype == SSD_BF16 ? 2 : 4;
    if (seqlen > 0) {
        if (!x || !dt || !A || !B || !C || !out) return SSD_ERR_INVALID_ARG;
        if (!aligned(x, 16) || !aligned(dt, e) || !aligned(A, 4) || !aligned(B, 16) || !aligned(C, 16) || !aligned(out, 16))
            return SSD_ERR_INVALID_ARG;
        const long long hp = (long long)nheads * headdim, gn = (long long)ngroups * dstate;
        if (!stride_ok(x_batch, batch, hp, e, true) || !stride_ok(x_token, seqlen, hp, e, true) ||
            !stride_ok(dt_batch, batch, nheads, e, false) || !stride_ok(dt_token, seqlen, nheads, e, false) ||
            !stride_ok(B_batch, batch, gn, e, true) || !stride_ok(B_token, seqlen, gn, e, true) ||
            !stride_ok(C_batch, batch, gn, e, true) || !stride_ok(C_token, seqlen, gn, e, true))
            return SSD_ERR_INVALID_ARG;
    } else if (!A || !aligned(A, 4)) {
        return SSD_ERR_INVALID_ARG;
    }
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    char *ws = static_cast<char *>(workspace);
    CausalArgs a{};
    a.x = x; a.dt = dt; a.B = B; a.C = C; a.A = A; a.D = D;
    a.step = ssd::StepSize{dt_bias, dt_min, dt_max};
    a.seqlens = seqlens; a.slots = slots; a.nslots = nslots;
    a.init = init_state; a.state_out = state_out; a.out = out;
    a.x_sb = x_batch; a.x_st = x_token; a.dt_sb = dt_batch; a.dt_st = dt_token;
    a.b_sb = B_batch; a.b_st = B_token; a.c_sb = C_batch; a.c_st = C_token;
    a.status = reinterpret_cast<ssd::DeviceStatus *>(ws);
    a.batch = batch; a.L = seqlen; a.H = nheads; a.P = headdim; a.G = ngroups; a.N = dstate;
    a.bf16 = dtype == SSD_BF16;
    if (path == SSD_PATH_FUSED) return to_status(ssd::launch_causal_tc(a, ws + ssd::kStatusBytes, s));
    const Plan p = plan(batch, seqlen, nheads, headdim, dstate);
    if (slots) {
        int *rows = reinterpret_cast<int *>(ws + p.rows);
        const cudaError_t err = ssd::launch_resolve_slots(slots, batch, nslots, rows, a.status, s);
        if (err != cudaSuccess) return to_status(err);
        a.rows = rows;
    }
    CausalSegments seg = p.seg;
    if (seg.count > 1) {
        seg.state = reinterpret_cast<float *>(ws + p.state);
        seg.decay = reinterpret_cast<float *>(ws + p.decay);
        cudaError_t err = ssd::launch_causal_simt(a, seg, ssd::kCausalState, s);
        if (err == cudaSuccess) err = ssd::launch_causal_carry(a, seg, s);
        if (err != cudaSuccess) return to_status(err);
    }
    return to_status(ssd::launch_causal_simt(a, seg, ssd::kCausalOutput, s));
}

int ssd_causal_step(const void *x, const void *dt, const float *A, const void *B, const void *C, const float *D,
                    const float *dt_bias, float dt_min, float dt_max, const int *slots, const float *state,
                    float *state_out, void *out, long long x_batch, long long dt_batch, long long B_batch,
                    long long C_batch, int nslots, int batch, int nheads, int headdim, int dstate, int ngroups,
                    int dtype, void *workspace, size_t ws_bytes, void *stream) {
    const int rc = check_sizes(batch, 1, nheads, headdim, dstate, ngroups, dtype);
    if (rc != SSD_OK) return rc;
    if (slots) {
        if (!workspace) return SSD_ERR_WORKSPACE;
        if (!aligned(workspace, 16)) return SSD_ERR_INVALID_ARG;
        if (ws_bytes < ssd::causal_workspace_bytes(SSD_OP_CAUSAL_STEP, batch, 1, nheads, headdim, dstate, ngroups, dtype))
            return SSD_ERR_WORKSPACE;
    }
    if (dt_bias && (!(dt_min >= 0.f) || !(dt_max >= dt_min))) return SSD_ERR_INVALID_ARG;
    if (slots && nslots < 0) return SSD_ERR_INVALID_ARG;
    if (batch == 0) return SSD_OK;
    if (!x || !dt || !A || !B || !C || !state || !state_out || !out) return SSD_ERR_INVALID_ARG;
    const int e = dtype == SSD_BF16 ? 2 : 4;
    if (!aligned(x, 16) || !aligned(dt, e) || !aligned(A, 4) || !aligned(B, 16) || !aligned(C, 16) || !aligned(D, 4) ||
        !aligned(dt_bias, 4) || !aligned(slots, 4) || !aligned(state, 16) || !aligned(state_out, 16) || !aligned(out, 16))
        return SSD_ERR_INVALID_ARG;
    const long long hp = (long long)nheads * headdim, gn = (long long)ngroups * dstate;
    if (!stride_ok(x_batch, batch, hp, e, true) || !stride_ok(dt_batch, batch, nheads, e, false) ||
        !stride_ok(B_batch, batch, gn, e, true) || !stride_ok(C_batch, batch, gn, e, true))
        return SSD_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    CausalArgs a{};
    a.x = x; a.dt = dt; a.B = B; a.C = C; a.A = A; a.D = D;
    a.step = ssd::StepSize{dt_bias, dt_min, dt_max};
    a.slots = slots; a.nslots = nslots;
    a.init = state; a.state_out = state_out; a.out = out;
    a.x_sb = x_batch; a.dt_sb = dt_batch; a.b_sb = B_batch; a.c_sb = C_batch;
    a.status = static_cast<ssd::DeviceStatus *>(workspace);
    a.batch = batch; a.L = 1; a.H = nheads; a.P = headdim; a.G = ngroups; a.N = dstate;
    a.bf16 = dtype == SSD_BF16;
    if (slots && batch > kScanRows) {
        int *rows = reinterpret_cast<int *>(static_cast<char *>(workspace) + ssd::kStatusBytes);
        const cudaError_t err = ssd::launch_resolve_slots(slots, batch, nslots, rows, a.status, s);
        if (err != cudaSuccess) return to_status(err);
        a.rows = rows;
    }
    return to_status(ssd::launch_causal_step(a, s));
}

int ssd_cache_copy(void *pool, long long page_bytes, int layers, int nslots, const int *src, const int *dst, int n,
                   void *workspace, size_t ws_bytes, void *stream) {
    if (page_bytes < 0 || layers < 0 || nslots < 0 || n < 0) return SSD_ERR_INVALID_ARG;
    if (nslots > ssd::kCacheMaxSlots || page_bytes > (1ll << 40)) return SSD_ERR_UNSUPPORTED;
    if (!workspace || ws_bytes < ssd::kStatusBytes) return SSD_ERR_WORKSPACE;
    if (!aligned(workspace, 16)) return SSD_ERR_INVALID_ARG;
    if (page_bytes == 0 || layers == 0 || nslots == 0 || n == 0) return SSD_OK;
    if (!pool || !src || !dst || !aligned(src, 4) || !aligned(dst, 4)) return SSD_ERR_INVALID_ARG;
    ssd::CacheArgs a{};
    a.pool = pool; a.page_bytes = page_bytes; a.layers = layers; a.nslots = nslots;
    a.src = src; a.dst = dst; a.n = n;
    a.status = static_cast<ssd::DeviceStatus *>(workspace);
    return to_status(ssd::launch_cache_copy(a, static_cast<cudaStream_t>(stream)));
}

int ssd_cache_compact(void *pool, long long page_bytes, int layers, int nslots, const int *table, int rows,
                      int *table_out, int *live_out, void *workspace, size_t ws_bytes, void *stream) {
    if (page_bytes < 0 || layers < 0 || nslots < 0 || rows < 0) return SSD_ERR_INVALID_ARG;
    if (nslots > ssd::kCacheMaxSlots || page_bytes > (1ll << 40)) return SSD_ERR_UNSUPPORTED;
    if (!workspace || ws_bytes < ssd::kStatusBytes) return SSD_ERR_WORKSPACE;
    if (!aligned(workspace, 16) || !live_out || !aligned(live_out, 4)) return SSD_ERR_INVALID_ARG;
    if (rows > 0 && (!table || !table_out || !aligned(table, 4) || !aligned(table_out, 4))) return SSD_ERR_INVALID_ARG;
    // every CTA reads the table while the first one writes the new one
    if (rows > 0 && table < table_out + rows && table_out < table + rows) return SSD_ERR_INVALID_ARG;
    if (!pool && page_bytes > 0 && layers > 0 && nslots > 0) return SSD_ERR_INVALID_ARG;
    ssd::CacheArgs a{};
    a.pool = pool; a.page_bytes = page_bytes; a.layers = layers; a.nslots = nslots;
    a.table = table; a.rows = rows; a.table_out = table_out; a.live_out = live_out;
    a.status = static_cast<ssd::DeviceStatus *>(workspace);
    return to_status(ssd::launch_cache_compact(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
