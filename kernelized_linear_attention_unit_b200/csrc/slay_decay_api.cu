// slay_decay_api.cu -- entry points of decayed linear attention and of the state pool:
// argument checks, workspace sizes and dispatch.  See include/slay.h for the contracts.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "slay.h"
#include "slay_decay.h"
#include "slay_internal.h"

namespace slay {
namespace {

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// required: not null, 16-byte aligned
inline bool tensor_ok(const void* p) { return p && aligned(p, 16); }

// a state pair: S null or aligned; z beside S exactly when the form is normalized
bool pair_ok(const float* S, const float* z, bool norm)
{
    if (!S) return !z;
    if (!aligned(S, 16)) return false;
    return norm ? z && aligned(z, 16) : !z;
}

// grid limits of the launches: (b, h), up to three times, indexes grid y / z
bool grid_ok(int B, int H, int L)
{
    return static_cast<int64_t>(B) * H <= 65535 / 3 && (static_cast<int64_t>(L) + 63) / 64 <= 65535;
}

slay_status check_sizes(int B, int H, int L, int F, int Dv, slay_dtype dt, bool norm, float eps)
{
    if (B < 0 || H < 0 || L < 0 || F <= 0 || Dv <= 0) return SLAY_ERR_INVALID_ARG;
    if (Dv != kD || F > kMaxF) return SLAY_ERR_UNSUPPORTED;
    if (!dtype_ok(dt) || (norm && !eps_ok(eps))) return SLAY_ERR_INVALID_ARG;
    return grid_ok(B, H, L) ? SLAY_OK : SLAY_ERR_UNSUPPORTED;
}

DecayArgs sizes(int B, int H, int L, int F, slay_dtype dt, bool norm)
{
    DecayArgs a{};
    a.B = B;
    a.H = H;
    a.L = L;
    a.F = F;
    a.dt = dt;
    a.norm = norm;
    return a;
}

}  // namespace

size_t decay_ws(slay_op op, slay_dtype dt, int B, int H, int L, int F)
{
    if (!grid_ok(B, H, L)) return SIZE_MAX;
    if (static_cast<int64_t>(B) * H * L == 0) return 0;
    const DecayArgs a = sizes(B, H, L, F, dt, true);
    const bool bwd = op == SLAY_OP_DECAY_BWD;
    return kWsHeader + (decay_tc_supported(a) ? decay_tc_ws(a, bwd) : decay_simt_ws(a, bwd));
}

int decay_path(slay_op, slay_dtype dt, int B, int H, int L, int F)
{
    if (!grid_ok(B, H, L)) return -1;
    return static_cast<int64_t>(B) * H > 0 && decay_tc_supported(sizes(B, H, L, F, dt, true)) ? SLAY_PATH_TC_CONTRACTION : 0;
}

}  // namespace slay

using namespace slay;

extern "C" {

slay_status slay_decay_attn_fwd(const void* phq, const void* phk, const void* v, const float* log_decay,
                                const int32_t* lengths, const float* S_in, const float* z_in, void* out, float* den,
                                float* S_out, float* z_out, int B, int H, int L, int F, int Dv, slay_dtype dt,
                                int normalize, float eps, void* workspace, size_t ws_bytes, void* stream)
{
    const bool norm = normalize != 0;
    const slay_status s = check_sizes(B, H, L, F, Dv, dt, norm, eps);
    if (s != SLAY_OK) return s;
    const int64_t BH = static_cast<int64_t>(B) * H;
    if (BH == 0 || (L == 0 && !S_out)) return SLAY_OK;
    if (!log_decay || !aligned(log_decay, 4) || (lengths && !aligned(lengths, 4))) return SLAY_ERR_INVALID_ARG;
    if (!pair_ok(S_in, z_in, norm) || !pair_ok(S_out, z_out, norm)) return SLAY_ERR_INVALID_ARG;
    if (den && (!norm || !aligned(den, 4))) return SLAY_ERR_INVALID_ARG;
    if (L > 0 && (!tensor_ok(phq) || !tensor_ok(phk) || !tensor_ok(v) || !tensor_ok(out))) return SLAY_ERR_INVALID_ARG;
    const size_t need = decay_ws(SLAY_OP_DECAY_FWD, dt, B, H, L, F);
    if (need > 0 && (!workspace || ws_bytes < need || !aligned(workspace, 256))) return SLAY_ERR_INVALID_ARG;
    DecayArgs a = sizes(B, H, L, F, dt, norm);
    a.phq = phq;
    a.phk = phk;
    a.v = v;
    a.log_decay = log_decay;
    a.lengths = lengths;
    a.S_in = S_in;
    a.z_in = z_in;
    a.eps = eps;
    a.out_w = out;
    a.den_w = den;
    a.S_out = S_out;
    a.z_out = z_out;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e = need ? cudaMemsetAsync(workspace, 0, sizeof(int), st) : cudaSuccess;
    void* scratch = static_cast<char*>(workspace) + kWsHeader;
    if (e == cudaSuccess)
        e = decay_tc_supported(a) ? decay_tc_fwd(a, scratch, static_cast<int*>(workspace), st) : decay_simt_fwd(a, scratch, st);
    return e == cudaSuccess ? SLAY_OK : report_cuda(e);
}

slay_status slay_decay_attn_bwd(const void* phq, const void* phk, const void* v, const float* log_decay,
                                const int32_t* lengths, const float* S_in, const float* z_in, const void* out,
                                const float* den, const void* dout, const float* dS_out, const float* dz_out,
                                void* dphq, void* dphk, void* dv, float* dS_in, float* dz_in, int B, int H, int L,
                                int F, int Dv, slay_dtype dt, int normalize, float eps, void* workspace,
                                size_t ws_bytes, void* stream)
{
    const bool norm = normalize != 0;
    const slay_status s = check_sizes(B, H, L, F, Dv, dt, norm, eps);
    if (s != SLAY_OK) return s;
    const int64_t BH = static_cast<int64_t>(B) * H;
    if (BH == 0 || (L == 0 && !dS_in)) return SLAY_OK;
    if (!log_decay || !aligned(log_decay, 4) || (lengths && !aligned(lengths, 4))) return SLAY_ERR_INVALID_ARG;
    if (!pair_ok(S_in, z_in, norm) || !pair_ok(dS_out, dz_out, norm) || !pair_ok(dS_in, dz_in, norm))
        return SLAY_ERR_INVALID_ARG;
    if (L > 0 && (!tensor_ok(phq) || !tensor_ok(phk) || !tensor_ok(v) || !tensor_ok(dout) || !tensor_ok(dphq) ||
                  !tensor_ok(dphk) || !tensor_ok(dv)))
        return SLAY_ERR_INVALID_ARG;
    if (L > 0 && norm && (!tensor_ok(out) || !den || !aligned(den, 4))) return SLAY_ERR_INVALID_ARG;
    const size_t need = decay_ws(SLAY_OP_DECAY_BWD, dt, B, H, L, F);
    if (need > 0 && (!workspace || ws_bytes < need || !aligned(workspace, 256))) return SLAY_ERR_INVALID_ARG;
    DecayArgs a = sizes(B, H, L, F, dt, norm);
    a.phq = phq;
    a.phk = phk;
    a.v = v;
    a.log_decay = log_decay;
    a.lengths = lengths;
    a.S_in = S_in;
    a.z_in = z_in;
    a.eps = eps;
    a.out = out;
    a.den = den;
    a.dout = dout;
    a.dS_out = dS_out;
    a.dz_out = dz_out;
    a.dphq = dphq;
    a.dphk = dphk;
    a.dv = dv;
    a.dS_in = dS_in;
    a.dz_in = dz_in;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e = need ? cudaMemsetAsync(workspace, 0, sizeof(int), st) : cudaSuccess;
    void* scratch = static_cast<char*>(workspace) + kWsHeader;
    if (e == cudaSuccess)
        e = decay_tc_supported(a) ? decay_tc_bwd(a, scratch, static_cast<int*>(workspace), st) : decay_simt_bwd(a, scratch, st);
    return e == cudaSuccess ? SLAY_OK : report_cuda(e);
}

slay_status slay_decay_decode_step(const void* phq, const void* phk, const void* v, const float* log_decay, float* S,
                                   float* z, const int32_t* slots, void* out, int Bt, int H, int F, int Dv,
                                   int n_slots, slay_dtype dt, int normalize, float eps, void* stream)
{
    const bool norm = normalize != 0;
    if (Bt < 0 || H < 0 || F <= 0 || Dv <= 0 || n_slots < 0) return SLAY_ERR_INVALID_ARG;
    if (Dv != kD || F > kMaxF) return SLAY_ERR_UNSUPPORTED;
    if (!dtype_ok(dt) || (norm && !eps_ok(eps))) return SLAY_ERR_INVALID_ARG;
    if (static_cast<int64_t>(Bt) * H == 0) return SLAY_OK;
    if (static_cast<int64_t>(Bt) * H > (int64_t(1) << 27)) return SLAY_ERR_UNSUPPORTED;
    if (!slots && Bt > n_slots) return SLAY_ERR_INVALID_ARG;
    if (!log_decay || !aligned(log_decay, 4) || (slots && !aligned(slots, 4))) return SLAY_ERR_INVALID_ARG;
    if (!tensor_ok(phq) || !tensor_ok(phk) || !tensor_ok(v) || !tensor_ok(out)) return SLAY_ERR_INVALID_ARG;
    if (n_slots > 0 && (!S || !pair_ok(S, z, norm))) return SLAY_ERR_INVALID_ARG;
    DecodeArgs a{};
    a.phq = phq;
    a.phk = phk;
    a.v = v;
    a.log_decay = log_decay;
    a.S = S;
    a.z = z;
    a.slots = slots;
    a.out = out;
    a.B = Bt;
    a.H = H;
    a.F = F;
    a.n_slots = n_slots;
    a.dt = dt;
    a.norm = norm;
    a.eps = eps;
    const cudaError_t e = decay_decode(a, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? SLAY_OK : report_cuda(e);
}

slay_status slay_state_copy(const float* S_src, const float* z_src, const int32_t* src, int n_src, float* S_dst,
                            float* z_dst, const int32_t* dst, int n_dst, int n, int H, int F, int Dv, void* stream)
{
    if (n < 0 || H <= 0 || F <= 0 || Dv <= 0 || n_src < 0 || n_dst < 0) return SLAY_ERR_INVALID_ARG;
    if (Dv != kD || F > kMaxF || n > kMaxCopies || static_cast<int64_t>(H) * F > (int64_t(1) << 24))
        return SLAY_ERR_UNSUPPORTED;
    if (n == 0 || n_dst == 0) return SLAY_OK;
    if (!src || !dst || !aligned(src, 4) || !aligned(dst, 4)) return SLAY_ERR_INVALID_ARG;
    if (!tensor_ok(S_dst) || (z_dst && !aligned(z_dst, 16))) return SLAY_ERR_INVALID_ARG;
    // (a source pool of no slots has no memory: the call only clears)
    if (n_src > 0 && (!tensor_ok(S_src) || (z_src == nullptr) != (z_dst == nullptr) || (z_src && !aligned(z_src, 16))))
        return SLAY_ERR_INVALID_ARG;
    const int64_t hf = static_cast<int64_t>(H) * F;
    // one pool, or two that share no byte
    auto overlap = [&](const float* p, const float* q, int64_t w) {
        return p != q && p < q + n_dst * w && q < p + n_src * w;
    };
    if (overlap(S_src, S_dst, hf * Dv) || (z_src && overlap(z_src, z_dst, hf))) return SLAY_ERR_INVALID_ARG;
    CopyArgs a{};
    a.S_src = S_src;
    a.z_src = z_src;
    a.src = src;
    a.S_dst = S_dst;
    a.z_dst = z_dst;
    a.dst = dst;
    a.n = n;
    a.n_src = n_src;
    a.n_dst = n_dst;
    a.hf = hf;
    const cudaError_t e = state_copy(a, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? SLAY_OK : report_cuda(e);
}

}  // extern "C"
