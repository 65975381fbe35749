// slay_decay.h -- linear attention with a decay for each head: declarations shared by the
// CUDA-core sweeps (slay_decay_simt.cu), the tensor-core sweeps (slay_decay_tc.cu) and the
// entry points (slay_decay_api.cu).
//
// The forward contraction and its three gradients are one recurrence with its operands
// permuted.  With a query row x_i, a key row y_j and a value row u_j,
//   o_i = sum_{j <= i} lambda^(i-j) score(x_i, y_j) u_j + lambda^(i+1) x_i M,
// M the decayed sum of y u^T over the tokens before the chunk (a "sweep"):
//   out  : x = phq, y = phk, u = v           walked forward,  M = S
//   dphq : x = do', y = v,   u = phk         walked forward,  M = S^T
//   dphk : x = v,   y = do', u = phq         walked backward, M = G^T
//   dv   : x = phk, y = phq, u = do'         walked backward, M = G
// where S = sum lambda^. phk v^T (tokens before), G = sum lambda^. phq do'^T (tokens after).
// Walked backward, query i meets keys j >= i with lambda^(j-i), the state enters with
// lambda^(n-1-i) and token j adds to it with lambda^(j+1) (n tokens in the chunk): G is the
// gradient of the state that leaves the chunk.
// In the normalized form do'_i = rz_i do_i with rz_i = 1 / (den_i + eps), and the value row
// carries a last column of ones whose gradient is -rz_i r_i, r_i = out_i . do_i; both enter
// as row scalars: score(do', v) = rz_i (do_i . v_j - r_i).
//
// "F side" is the F-wide tensor that enters the state (phk or phq), "E side" the 64-wide one
// (v or do).  States are [F][64] fp32 with a column z [F] for the ones column.
#pragma once

#include <cstddef>
#include <cstdint>

#include <cuda_runtime.h>

#include "slay.h"
#include "slay_internal.h"

namespace slay {

// lambda^k from log2(lambda) <= 0 (-inf: lambda = 0); lambda^0 = 1.
__device__ __forceinline__ float decay_pow(float log2_lam, int k)
{
    return k == 0 ? 1.0f : exp2f(static_cast<float>(k) * log2_lam);
}

// lambda^n of one whole chunk of n tokens after another, for a state that is carried through many.
// One rounded factor, multiplied k times, is off by up to k 2^-25 where it is near 1; here what a
// factor's rounding leaves goes into the next one, so that their product keeps to lambda^(k n):
// the fp32 state of 10^6 tokens at log_decay -3.1e-6 is 1.4e-6 off, 1.9e-4 with a fixed factor.
struct ChunkDecay {
    float drop, fixed, rest = 0.0f;   // lambda^n - 1; lambda^n
    __device__ __forceinline__ ChunkDecay(float log_lam, float log2_lam, int n)
        : drop(expm1f(static_cast<float>(n) * log_lam)), fixed(decay_pow(log2_lam, n))
    {
    }
    __device__ __forceinline__ float next()
    {
        if (drop < -0.5f) return fixed;   // no state lives through many chunks
        const float want = drop + rest, lam = 1.0f + want;
        rest = want - (lam - 1.0f);
        return lam;
    }
};

// The kernels of one call follow one another on the call's stream.  Each but the first is
// launched while the one before it still runs (programmatic stream serialization): its blocks
// set themselves up and then wait here until everything before them is complete and visible.
__device__ __forceinline__ void after_previous_kernel()
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

template <typename... Params, typename... Args>
cudaError_t launch_in_chain(bool first, void (*kernel)(Params...), dim3 grid, int threads, size_t smem, cudaStream_t st,
                            Args... args)
{
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = first ? 0 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
}

constexpr float kLog2e = 1.4426950408889634f;

// Arguments of the decayed forward and backward, as the entry points take them.
struct DecayArgs {
    const void *phq, *phk, *v;
    const float* log_decay;        // [H]
    const int32_t* lengths;        // [B] or null: all L
    const float *S_in, *z_in;      // [B,H,F,64], [B,H,F] or null: zero
    int B, H, L, F;
    slay_dtype dt;
    bool norm;
    float eps;
    // forward
    void* out_w;
    float *den_w, *S_out, *z_out;  // null: not wanted
    // backward
    const void *out, *dout;
    const float* den;
    const float *dS_out, *dz_out;  // null: zero
    void *dphq, *dphk, *dv;
    float *dS_in, *dz_in;          // null: not wanted
};

// Row statistics of the normalized backward: rz = 1 / (den + eps), r = out . dout, [B,H,L].
// (the first kernel of its call)
cudaError_t decay_row_stats(const DecayArgs& a, float* rz, float* r, cudaStream_t st);

// CUDA cores: any F up to kMaxF, fp32 or bf16 operands, fp32 arithmetic.
size_t decay_simt_ws(const DecayArgs& a, bool bwd);
cudaError_t decay_simt_fwd(const DecayArgs& a, void* ws, cudaStream_t st);
cudaError_t decay_simt_bwd(const DecayArgs& a, void* ws, cudaStream_t st);

// Tensor cores: bf16, F % 8 == 0, F <= 512 (feature blocks of at most 256).  err: the status
// word a bounded wait that ran out is reported in.
bool decay_tc_supported(const DecayArgs& a);
size_t decay_tc_ws(const DecayArgs& a, bool bwd);
cudaError_t decay_tc_fwd(const DecayArgs& a, void* ws, int* err, cudaStream_t st);
cudaError_t decay_tc_bwd(const DecayArgs& a, void* ws, int* err, cudaStream_t st);

// Single-token step on pooled states; pool copies.
struct DecodeArgs {
    const void *phq, *phk, *v;
    const float* log_decay;
    float *S, *z;
    const int32_t* slots;   // null: row b uses slot b
    void* out;
    int B, H, F, n_slots;
    slay_dtype dt;
    bool norm;
    float eps;
};
cudaError_t decay_decode(const DecodeArgs& a, cudaStream_t st);

struct CopyArgs {
    const float *S_src, *z_src;
    const int32_t* src;
    float *S_dst, *z_dst;
    const int32_t* dst;
    int n, n_src, n_dst;
    int64_t hf;             // heads x features of a slot
};
constexpr int kMaxCopies = 4096;
cudaError_t state_copy(const CopyArgs& a, cudaStream_t st);

}  // namespace slay
