// slay_decay_simt.cu -- CUDA-core sweeps of linear attention with a decay for each head (fp32
// mode, and the bf16 sizes the tensor-core sweeps do not take).  The recurrence and its roles
// are described in slay_decay.h.
//
// Three kernels over 64-token chunks, every product a 64 x 64 block of a 256-thread CTA held
// as 4 x 4 fp32 accumulators per thread, operands in shared memory as fp32:
//   k_dec_state : each chunk's own state  T = sum_j w_j y_j u_j^T  (a CTA per 64 features)
//   k_dec_scan  : the states entering each chunk, M <- lambda^n M + T, one thread per element
//   k_dec_fwd, k_dec_grads : the outputs, per chunk out_f (queries on the F side: out, dv;
//                 64 wide) or out_e (queries on the E side: dphq, dphk; F wide, 64 at a time)
// fp32 FMA bounds them (per token and head about 2 (3 * 64 F + 64 * 64) operations per sweep
// against 8 F + 512 bytes); 64-token chunks keep the quadratic part below the state part for
// every F >= 64.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "slay_decay.h"

namespace slay {
namespace {

constexpr int kC = 64;          // tokens per chunk
constexpr int kNT = 256;
constexpr int kPitch = 68;      // floats per shared-memory row of 64: float4 reads of 16
                                // rows (one per thread column) hit distinct banks

__device__ __forceinline__ float ldf(const float* p) { return *p; }
__device__ __forceinline__ float ldf(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void stf(float* p, float x) { *p = x; }
__device__ __forceinline__ void stf(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

__device__ __forceinline__ float4 ld4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 ld4(const __nv_bfloat16* p)
{
    const uint2 w = *reinterpret_cast<const uint2*>(p);
    return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u),
                       __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xFFFF0000u));
}
__device__ __forceinline__ void st4(float* p, float4 x) { *reinterpret_cast<float4*>(p) = x; }
__device__ __forceinline__ void st4(__nv_bfloat16* p, float4 x)
{
    const __nv_bfloat162 a = __floats2bfloat162_rn(x.x, x.y), b = __floats2bfloat162_rn(x.z, x.w);
    uint2 w;
    w.x = *reinterpret_cast<const uint32_t*>(&a);
    w.y = *reinterpret_cast<const uint32_t*>(&b);
    *reinterpret_cast<uint2*>(p) = w;
}

// A sweep's operands (see slay_decay.h); null scalars stand for 1 (mul) and 0 (off).
struct Sweep {
    const float *first, *first_z;   // the state entering the walk (null: zero)
    float *last, *last_z;           // the one leaving it (null: not wanted)
    const void* fs;       // F side of the state [BH][L][F]
    const void* es;       // E side of the state [BH][L][64]
    const void* fq;       // query, F side (out, dv)
    const void* eq;       // query, E side (dphq, dphk)
    const float* s_mul;   // per state token: scales its score and its term of the state
    const float* s_off;   // per state token: taken off its raw score
    const float* q_mul;   // per query token, likewise
    const float* q_off;
    bool z_delta;         // the z weight of a state token is -s_mul s_off (else 1)
    bool rev;
    const float* log_decay;
    const int32_t* lengths;
    int H, L, F, nc;
    float* st;            // [BH][nc][F][64] chunk states
    float* sz;            // [BH][nc][F], null without a z column
};

__device__ __forceinline__ int seq_len(const int32_t* lengths, int b, int L)
{
    return lengths ? min(max(lengths[b], 0), L) : L;
}

// rows [t0, t0 + n) x columns [c0, c0 + 64) of x [.., W] -> dst [64][kPitch] fp32, times
// mul[row] when given; everything else zero
template <typename T>
__device__ __forceinline__ void load_block(float* dst, const T* x, int n, int W, int c0, const float* mul)
{
    const int wc = min(64, W - c0);
    if ((W & 3) == 0) {
        for (int i = threadIdx.x; i < 64 * 16; i += kNT) {
            const int r = i >> 4, c = (i & 15) * 4;
            float4 w = make_float4(0.f, 0.f, 0.f, 0.f);
            if (r < n && c < wc) {
                w = ld4(x + static_cast<int64_t>(r) * W + c0 + c);
                if (mul) { const float m = mul[r]; w.x *= m; w.y *= m; w.z *= m; w.w *= m; }
            }
            *reinterpret_cast<float4*>(dst + r * kPitch + c) = w;
        }
    } else {
        for (int i = threadIdx.x; i < 64 * 64; i += kNT) {
            const int r = i >> 6, c = i & 63;
            float w = 0.0f;
            if (r < n && c < wc) {
                w = ldf(x + static_cast<int64_t>(r) * W + c0 + c);
                if (mul) w *= mul[r];
            }
            dst[r * kPitch + c] = w;
        }
    }
}

// acc[a][b] += sum_k A[ty + 16 a][k] B[tx + 16 b][k], k < 64
__device__ __forceinline__ void mma_nt(float (&acc)[4][4], const float* A, const float* B, int ty, int tx)
{
#pragma unroll 4
    for (int k = 0; k < 64; k += 4) {
        float4 a[4], b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            a[i] = *reinterpret_cast<const float4*>(A + (ty + 16 * i) * kPitch + k);
            b[i] = *reinterpret_cast<const float4*>(B + (tx + 16 * i) * kPitch + k);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                acc[i][j] = fmaf(a[i].x, b[j].x, acc[i][j]);
                acc[i][j] = fmaf(a[i].y, b[j].y, acc[i][j]);
                acc[i][j] = fmaf(a[i].z, b[j].z, acc[i][j]);
                acc[i][j] = fmaf(a[i].w, b[j].w, acc[i][j]);
            }
    }
}

// acc[a][b] += sum_k A[ty + 16 a][k] B[k][4 tx + b], k < 64
__device__ __forceinline__ void mma_nn(float (&acc)[4][4], const float* A, const float* B, int ty, int tx)
{
#pragma unroll 4
    for (int k = 0; k < 64; k += 4) {
        float4 a[4], b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            a[i] = *reinterpret_cast<const float4*>(A + (ty + 16 * i) * kPitch + k);
            b[i] = *reinterpret_cast<const float4*>(B + (k + i) * kPitch + 4 * tx);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float av[4] = {a[i].x, a[i].y, a[i].z, a[i].w};
#pragma unroll
            for (int k2 = 0; k2 < 4; ++k2) {
                acc[i][0] = fmaf(av[k2], b[k2].x, acc[i][0]);
                acc[i][1] = fmaf(av[k2], b[k2].y, acc[i][1]);
                acc[i][2] = fmaf(av[k2], b[k2].z, acc[i][2]);
                acc[i][3] = fmaf(av[k2], b[k2].w, acc[i][3]);
            }
        }
    }
}

// Weight of state token j of a chunk of n in the state that leaves the chunk.
__device__ __forceinline__ float state_weight(float g2, int j, int n, bool rev)
{
    return decay_pow(g2, rev ? j + 1 : n - 1 - j);
}

// ------------------------------------------------------------------ chunk states
// grid (nc, ceil(F / 64), BH, or 2 BH with a second sweep)
template <typename T>
__global__ void __launch_bounds__(kNT) k_dec_state(Sweep s0, Sweep s1, int BH)
{
    const Sweep& s = static_cast<int>(blockIdx.z) < BH ? s0 : s1;
    extern __shared__ __align__(16) float sm[];
    float* fsm = sm;                    // [64 j][f]
    float* esm = sm + 64 * kPitch;      // [64 j][e], weighted
    __shared__ float w[kC], wz[kC];
    const int c = blockIdx.x, f0 = blockIdx.y * 64;
    const int64_t bh = static_cast<int>(blockIdx.z) % BH;
    const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
    const int t0 = c * kC, n = min(kC, seq_len(s.lengths, static_cast<int>(bh / s.H), s.L) - t0);
    const float g2 = s.log_decay[bh % s.H] * kLog2e;
    float* st = s.st + ((bh * s.nc + c) * s.F + f0) * 64;
    const int64_t row0 = bh * s.L + t0;
    after_previous_kernel();
    if (tid < kC) {
        float a = 0.0f, b = 0.0f;
        if (tid < n) {
            a = state_weight(g2, tid, n, s.rev);
            b = a;
            if (s.s_mul) a *= s.s_mul[row0 + tid];
            if (s.z_delta) b = -a * s.s_off[row0 + tid];
        }
        w[tid] = a;
        wz[tid] = b;
    }
    __syncthreads();
    load_block(fsm, static_cast<const T*>(s.fs) + row0 * s.F, n, s.F, f0, nullptr);
    load_block(esm, static_cast<const T*>(s.es) + row0 * 64, n, 64, 0, w);
    __syncthreads();
    float acc[4][4] = {};
#pragma unroll 8
    for (int j = 0; j < kC; ++j) {
        const float4 a = *reinterpret_cast<const float4*>(fsm + j * kPitch + 4 * ty);
        const float4 b = *reinterpret_cast<const float4*>(esm + j * kPitch + 4 * tx);
        const float av[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            acc[i][0] = fmaf(av[i], b.x, acc[i][0]);
            acc[i][1] = fmaf(av[i], b.y, acc[i][1]);
            acc[i][2] = fmaf(av[i], b.z, acc[i][2]);
            acc[i][3] = fmaf(av[i], b.w, acc[i][3]);
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (f0 + 4 * ty + i < s.F)
            *reinterpret_cast<float4*>(st + (4 * ty + i) * 64 + 4 * tx) =
                make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
    if (s.sz && tid < 64 && f0 + tid < s.F) {
        float z = 0.0f;
        for (int j = 0; j < kC; ++j) z = fmaf(wz[j], fsm[j * kPitch + tid], z);
        s.sz[(bh * s.nc + c) * s.F + f0 + tid] = z;
    }
}

// Chunk states -> the state entering each chunk (in place), S and z in one launch; first: the
// state entering the walk (null: zero), last: the one leaving it (null: not wanted; may be
// `first` itself, each element is read before it is written).  Loads run eight chunks ahead.
// grid (ceil(64 F / 4 kNT) + ceil(F / kNT), BH, or 2 BH with a second sweep): a thread has four elements of S or one of z
// (whose rows need not be whole float4s).
__global__ void __launch_bounds__(kNT) k_dec_scan(Sweep s0, Sweep s1, int BH, int s_blocks)
{
    after_previous_kernel();
    const Sweep& s = static_cast<int>(blockIdx.y) < BH ? s0 : s1;
    const int64_t bh = static_cast<int>(blockIdx.y) % BH;
    const int n = seq_len(s.lengths, static_cast<int>(bh / s.H), s.L);
    const float g2 = s.log_decay[bh % s.H] * kLog2e;
    const float lam_c = decay_pow(g2, kC);
    constexpr int kAhead = 8;
    auto walk = [&](auto* p, const auto* from, auto* to, int64_t w, int64_t x, auto zero, auto step) {
        auto run = from ? from[bh * w + x] : zero;
        p += bh * s.nc * w + x;
        for (int i0 = 0; i0 < s.nc; i0 += kAhead) {
            decltype(run) t[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; ++i)
                if (i0 + i < s.nc) t[i] = p[(s.rev ? s.nc - 1 - i0 - i : i0 + i) * w];
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                if (i0 + i >= s.nc) break;
                const int c = s.rev ? s.nc - 1 - i0 - i : i0 + i;
                p[c * w] = run;
                const int nn = min(max(n - c * kC, 0), kC);
                run = step(nn == kC ? lam_c : decay_pow(g2, nn), run, t[i]);
            }
        }
        if (to) to[bh * w + x] = run;
    };
    if (static_cast<int>(blockIdx.x) < s_blocks) {
        const int64_t x = static_cast<int64_t>(blockIdx.x) * kNT + threadIdx.x, w = static_cast<int64_t>(s.F) * 16;
        if (x < w)
            walk(reinterpret_cast<float4*>(s.st), reinterpret_cast<const float4*>(s.first), reinterpret_cast<float4*>(s.last), w, x,
                 make_float4(0.f, 0.f, 0.f, 0.f), [](float l, float4 a, float4 b) {
                     return make_float4(fmaf(l, a.x, b.x), fmaf(l, a.y, b.y), fmaf(l, a.z, b.z), fmaf(l, a.w, b.w));
                 });
    } else {
        const int64_t x = static_cast<int64_t>(blockIdx.x - s_blocks) * kNT + threadIdx.x;
        if (x < s.F) walk(s.sz, s.first_z, s.last_z, s.F, x, 0.0f, [](float l, float a, float b) { return fmaf(l, a, b); });
    }
}

// Masked, decayed scores: query row i, state token j of a chunk of n.
__device__ __forceinline__ float score(float raw, int i, int j, int n, bool rev, float qo, float so, float qm,
                                       const float* sm_mul, const float* pw)
{
    const int d = rev ? j - i : i - j;
    return d >= 0 && i < n && j < n ? (raw - qo - so) * (qm * sm_mul[j]) * pw[d] : 0.0f;
}

// ----------------------------------------------------- outputs 64 wide (out, dv)
template <typename T>
__device__ __forceinline__ void out_f(const Sweep& s, float* sm, int64_t bh, T* o, float* den, bool norm, float eps)
{
    float* fqs = sm;                        // [64 i][64 f]
    float* fss = fqs + 64 * kPitch;         // [64 j][64 f]; then the scores [64 i][64 j]
    float* ms = fss + 64 * kPitch;          // [64 f][64 e]; then the E side [64 j][64 e]
    __shared__ float pw[kC], smul[kC], zs[64], dsum[kC];
    const int c = blockIdx.x;
    const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
    const int t0 = c * kC, n = min(kC, seq_len(s.lengths, static_cast<int>(bh / s.H), s.L) - t0);
    after_previous_kernel();
    if (n <= 0) return;
    const float g2 = s.log_decay[bh % s.H] * kLog2e;
    const int64_t row0 = bh * s.L + t0;
    if (tid < kC) {
        pw[tid] = decay_pow(g2, tid);
        smul[tid] = tid < n && s.s_mul ? s.s_mul[row0 + tid] : 1.0f;
        dsum[tid] = 0.0f;
    }
    float p[4][4] = {}, acc[4][4] = {}, dz = 0.0f;
    for (int f0 = 0; f0 < s.F; f0 += 64) {
        __syncthreads();
        load_block(fqs, static_cast<const T*>(s.fq) + row0 * s.F, n, s.F, f0, nullptr);
        load_block(fss, static_cast<const T*>(s.fs) + row0 * s.F, n, s.F, f0, nullptr);
        load_block(ms, s.st + ((bh * s.nc + c) * s.F + f0) * 64, min(64, s.F - f0), 64, 0, nullptr);
        if (norm && tid < 64) zs[tid] = f0 + tid < s.F ? s.sz[(bh * s.nc + c) * s.F + f0 + tid] : 0.0f;
        __syncthreads();
        mma_nt(p, fqs, fss, ty, tx);
        mma_nn(acc, fqs, ms, ty, tx);
        if (norm) {   // four threads a row, 16 features each
            const int i = tid >> 2, k0 = (tid & 3) * 16;
#pragma unroll
            for (int k = 0; k < 16; ++k) dz = fmaf(fqs[i * kPitch + k0 + k], zs[k0 + k], dz);
        }
    }
    __syncthreads();
    float rs[4] = {};
#pragma unroll
    for (int a = 0; a < 4; ++a)
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const int i = ty + 16 * a, j = tx + 16 * b;
            const float w = score(p[a][b], i, j, n, s.rev, 0.0f, 0.0f, 1.0f, smul, pw);
            fss[i * kPitch + j] = w;
            rs[a] += w;
        }
    if (norm) {
#pragma unroll
        for (int a = 0; a < 4; ++a) {
            for (int x = 8; x > 0; x >>= 1) rs[a] += __shfl_xor_sync(0xffffffffu, rs[a], x);
            if (tx == 0) dsum[ty + 16 * a] = rs[a];
        }
        dz += __shfl_xor_sync(0xffffffffu, dz, 1);
        dz += __shfl_xor_sync(0xffffffffu, dz, 2);
    }
    load_block(ms, static_cast<const T*>(s.es) + row0 * 64, n, 64, 0, nullptr);
    __syncthreads();
    if (norm && (tid & 3) == 0) {
        const int i = tid >> 2;
        const float d = fmaf(decay_pow(g2, s.rev ? max(n - 1 - i, 0) : i + 1), dz, dsum[i]);
        dsum[i] = d;
        if (den && i < n) den[row0 + i] = d;
    }
#pragma unroll
    for (int a = 0; a < 4; ++a) {
        const int i = ty + 16 * a;
        const float fac = decay_pow(g2, s.rev ? max(n - 1 - i, 0) : i + 1);
#pragma unroll
        for (int b = 0; b < 4; ++b) acc[a][b] *= fac;
    }
    mma_nn(acc, fss, ms, ty, tx);
    if (norm) __syncthreads();
#pragma unroll
    for (int a = 0; a < 4; ++a) {
        const int i = ty + 16 * a;
        if (i >= n) continue;
        const float rden = norm ? dsum[i] + eps : 1.0f;
        float4 w = make_float4(acc[a][0], acc[a][1], acc[a][2], acc[a][3]);
        if (norm) { w.x /= rden; w.y /= rden; w.z /= rden; w.w /= rden; }
        st4(o + (row0 + i) * 64 + 4 * tx, w);
    }
}

// ----------------------------------------------------- outputs F wide (dphq, dphk)
template <typename T>
__device__ __forceinline__ void out_e(const Sweep& s, float* sm, int64_t bh, T* o, bool norm)
{
    float* eqs = sm;                        // [64 i][64 e]
    float* ps = eqs + 64 * kPitch;          // E side of the state, then the scores [64 i][64 j]
    float* fss = ps + 64 * kPitch;          // [64 j][64 f]
    float* ms = fss + 64 * kPitch;          // [64 f][64 e]
    __shared__ float pw[kC], smul[kC], soff[kC], zs[64];
    const int c = blockIdx.x;
    const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
    const int t0 = c * kC, n = min(kC, seq_len(s.lengths, static_cast<int>(bh / s.H), s.L) - t0);
    after_previous_kernel();
    if (n <= 0) return;
    const float g2 = s.log_decay[bh % s.H] * kLog2e;
    const int64_t row0 = bh * s.L + t0;
    if (tid < kC) {
        const bool in = tid < n;
        pw[tid] = decay_pow(g2, tid);
        smul[tid] = in && s.s_mul ? s.s_mul[row0 + tid] : 1.0f;
        soff[tid] = in && s.s_off ? s.s_off[row0 + tid] : 0.0f;
    }
    load_block(eqs, static_cast<const T*>(s.eq) + row0 * 64, n, 64, 0, nullptr);
    load_block(ps, static_cast<const T*>(s.es) + row0 * 64, n, 64, 0, nullptr);
    __syncthreads();
    float p[4][4] = {};
    mma_nt(p, eqs, ps, ty, tx);
    __syncthreads();
    // per query row: the score's scalars, the state's factor and the weight of its z column
    float fac[4], zc[4];
#pragma unroll
    for (int a = 0; a < 4; ++a) {
        const int i = ty + 16 * a;
        const bool in = i < n;
        const float qm = in && s.q_mul ? s.q_mul[row0 + i] : 1.0f;
        const float qo = in && s.q_off ? s.q_off[row0 + i] : 0.0f;
        fac[a] = qm * decay_pow(g2, s.rev ? max(n - 1 - i, 0) : i + 1);
        zc[a] = s.q_off ? -qo : 1.0f;
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const int j = tx + 16 * b;
            ps[i * kPitch + j] = score(p[a][b], i, j, n, s.rev, qo, soff[j], qm, smul, pw);
        }
    }
    const bool vec = (s.F & 3) == 0;
    for (int f0 = blockIdx.z * 64; f0 < s.F; f0 += gridDim.z * 64) {
        __syncthreads();
        load_block(fss, static_cast<const T*>(s.fs) + row0 * s.F, n, s.F, f0, nullptr);
        load_block(ms, s.st + ((bh * s.nc + c) * s.F + f0) * 64, min(64, s.F - f0), 64, 0, nullptr);
        if (tid < 64) zs[tid] = norm && f0 + tid < s.F ? s.sz[(bh * s.nc + c) * s.F + f0 + tid] : 0.0f;
        __syncthreads();
        // inter-chunk part with columns tx + 16 b; through shared memory to columns 4 tx + b
        float t[4][4] = {}, acc[4][4] = {};
        mma_nt(t, eqs, ms, ty, tx);
        __syncthreads();
#pragma unroll
        for (int a = 0; a < 4; ++a)
#pragma unroll
            for (int b = 0; b < 4; ++b)
                ms[(ty + 16 * a) * kPitch + tx + 16 * b] = fac[a] * fmaf(zc[a], zs[tx + 16 * b], t[a][b]);
        __syncthreads();
        mma_nn(acc, ps, fss, ty, tx);
#pragma unroll
        for (int a = 0; a < 4; ++a) {
            const int i = ty + 16 * a, f = f0 + 4 * tx;
            if (i >= n) continue;
            const float4 m = *reinterpret_cast<const float4*>(ms + i * kPitch + 4 * tx);
            const float4 w = make_float4(acc[a][0] + m.x, acc[a][1] + m.y, acc[a][2] + m.z, acc[a][3] + m.w);
            T* dst = o + (row0 + i) * s.F + f;
            if (vec) {
                if (f < s.F) st4(dst, w);
            } else {
                if (f < s.F) stf(dst, w.x);
                if (f + 1 < s.F) stf(dst + 1, w.y);
                if (f + 2 < s.F) stf(dst + 2, w.z);
                if (f + 3 < s.F) stf(dst + 3, w.w);
            }
        }
    }
}

// grid (nc, BH)
template <typename T>
__global__ void __launch_bounds__(kNT) k_dec_fwd(Sweep s, T* o, float* den, bool norm, float eps)
{
    extern __shared__ __align__(16) float sm[];
    out_f(s, sm, blockIdx.y, o, den, norm, eps);
}

// The three gradients side by side: grid (nc, 3 BH, column groups of the F-wide ones)
template <typename T>
__global__ void __launch_bounds__(kNT) k_dec_grads(Sweep s, Sweep g, T* dphq, T* dphk, T* dv, int BH, bool norm)
{
    extern __shared__ __align__(16) float sm[];
    const int role = blockIdx.y / BH, bh = blockIdx.y % BH;
    if (role < 2) out_e(role ? g : s, sm, bh, role ? dphk : dphq, norm);
    else if (blockIdx.z == 0) out_f<T>(g, sm, bh, dv, nullptr, false, 0.0f);
}

// Row statistics of the normalized backward: 16 bytes a lane, so 8 (bf16) or 16 (fp32) lanes a
// row; bound by the reads of out and dout.
template <typename T>
__global__ void __launch_bounds__(256) k_dec_row_stats(const T* out, const T* dout, const float* den, float* rz,
                                                       float* r, int64_t rows, float eps, const int32_t* lengths,
                                                       int64_t HL, int L)
{
    constexpr int kE = 16 / sizeof(T), kLanes = 64 / kE;
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x, row = i / kLanes;
    // rows behind a sequence are never read by the sweeps, whatever comes out for them
    const bool in = row < rows && !(lengths && row % L >= lengths[row / HL]);
    float d = 0.0f;
    if (in) {
#pragma unroll
        for (int e = 0; e < kE; e += 4) {
            const float4 a = ld4(out + i * kE + e), b = ld4(dout + i * kE + e);
            d = fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, fmaf(a.w, b.w, d))));
        }
    }
#pragma unroll
    for (int x = kLanes / 2; x > 0; x >>= 1) d += __shfl_xor_sync(0xffffffffu, d, x);
    if (in && i % kLanes == 0) {
        rz[row] = 1.0f / (den[row] + eps);
        r[row] = d;
    }
}

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

constexpr size_t kSmemF = 3 * 64 * kPitch * sizeof(float), kSmemE = 4 * 64 * kPitch * sizeof(float),
                 kSmemS = 2 * 64 * kPitch * sizeof(float);

// The states of a sweep, or of two at once.
template <typename T>
cudaError_t states(const Sweep& s, const Sweep* g, int BH, bool chained, cudaStream_t st)
{
    const unsigned n = g ? 2 * BH : BH;
    if (s.nc > 0) {   // L == 0: the walk has no chunk and hands its state on
        TraceScope trace_("simt_decay_state", st);
        const cudaError_t e = launch_in_chain(!chained, k_dec_state<T>, dim3(s.nc, (s.F + 63) / 64, n), kNT, kSmemS, st, s,
                                              g ? *g : s, BH);
        if (e != cudaSuccess) return e;
        chained = true;
    }
    const int sb = (s.F * 16 + kNT - 1) / kNT, zb = s.sz ? (s.F + kNT - 1) / kNT : 0;
    TraceScope trace_("simt_decay_scan", st);
    return launch_in_chain(!chained, k_dec_scan, dim3(sb + zb, n), kNT, 0, st, s, g ? *g : s, BH, sb);
}

template <typename T>
cudaError_t prepare_smem()
{
    cudaError_t e = cudaFuncSetAttribute(k_dec_fwd<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemF);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(k_dec_grads<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemE);
    return e;
}

struct Carve {
    float *st, *sz, *gt, *gz, *rz, *r;
    size_t bytes;
};

Carve carve(const DecayArgs& a, bool bwd, void* ws)
{
    const int64_t BH = static_cast<int64_t>(a.B) * a.H, nc = (a.L + kC - 1) / kC;
    char* p = static_cast<char*>(ws);
    size_t o = 0;
    auto take = [&](size_t floats) {
        float* q = reinterpret_cast<float*>(p + o);
        o += align256(floats * 4);
        return q;
    };
    Carve c{};
    c.st = take(static_cast<size_t>(BH) * nc * a.F * 64);
    c.sz = take(static_cast<size_t>(BH) * nc * a.F);
    if (bwd) {
        c.gt = take(static_cast<size_t>(BH) * nc * a.F * 64);
        c.gz = take(static_cast<size_t>(BH) * nc * a.F);
        c.rz = take(static_cast<size_t>(BH) * a.L);
        c.r = take(static_cast<size_t>(BH) * a.L);
    }
    c.bytes = o;
    return c;
}

Sweep base(const DecayArgs& a, const Carve& c)
{
    Sweep s{};
    s.log_decay = a.log_decay;
    s.lengths = a.lengths;
    s.H = a.H;
    s.L = a.L;
    s.F = a.F;
    s.nc = (a.L + kC - 1) / kC;
    s.st = c.st;
    s.sz = a.norm ? c.sz : nullptr;
    return s;
}

template <typename T>
cudaError_t fwd_t(const DecayArgs& a, void* ws, cudaStream_t st)
{
    const Carve c = carve(a, false, ws);
    const int BH = a.B * a.H;
    cudaError_t e = prepare_smem<T>();
    if (e != cudaSuccess) return e;
    Sweep s = base(a, c);
    s.fq = a.phq;
    s.fs = a.phk;
    s.es = a.v;
    s.first = a.S_in;
    s.first_z = a.z_in;
    s.last = a.S_out;
    s.last_z = a.z_out;
    if ((e = states<T>(s, nullptr, BH, false, st)) != cudaSuccess || s.nc == 0) return e;
    TraceScope trace_("simt_decay_out", st);
    return launch_in_chain(false, k_dec_fwd<T>, dim3(s.nc, BH), kNT, kSmemF, st, s, static_cast<T*>(a.out_w), a.den_w, a.norm,
                           a.eps);
}

template <typename T>
cudaError_t bwd_t(const DecayArgs& a, void* ws, cudaStream_t st)
{
    const Carve c = carve(a, true, ws);
    const int BH = a.B * a.H;
    cudaError_t e = prepare_smem<T>();
    if (e != cudaSuccess) return e;
    const bool stats = a.norm && a.L > 0;
    if (stats && (e = decay_row_stats(a, c.rz, c.r, st)) != cudaSuccess) return e;
    const float *rz = a.norm ? c.rz : nullptr, *r = a.norm ? c.r : nullptr;
    Sweep s = base(a, c);   // dphq from the states before each token
    s.fs = a.phk;
    s.es = a.v;
    s.eq = a.dout;
    s.q_mul = rz;
    s.q_off = r;
    s.first = a.S_in;
    s.first_z = a.z_in;
    Sweep g = base(a, c);   // dphk and dv from the states after each token
    g.st = c.gt;
    g.sz = a.norm ? c.gz : nullptr;
    g.rev = true;
    g.fs = a.phq;
    g.es = a.dout;
    g.s_mul = rz;
    g.s_off = r;
    g.z_delta = a.norm;
    g.eq = a.v;
    g.fq = a.phk;
    g.first = a.dS_out;
    g.first_z = a.dz_out;
    g.last = a.dS_in;
    g.last_z = a.dz_in;
    if (s.nc == 0) return states<T>(g, nullptr, BH, false, st);
    if ((e = states<T>(s, &g, BH, stats, st)) != cudaSuccess) return e;
    // few CTAs: the column blocks of the F-wide outputs go to CTAs of their own
    const int nfb = (a.F + 63) / 64;
    const int64_t ctas = 3 * static_cast<int64_t>(BH) * s.nc;
    const int zsplit = static_cast<int>(ctas >= 296 ? 1 : std::min<int64_t>(nfb, (296 + ctas - 1) / ctas));
    TraceScope trace_("simt_decay_out", st);
    return launch_in_chain(false, k_dec_grads<T>, dim3(s.nc, 3 * BH, zsplit), kNT, kSmemE, st, s, g, static_cast<T*>(a.dphq),
                           static_cast<T*>(a.dphk), static_cast<T*>(a.dv), BH, a.norm);
}

}  // namespace

cudaError_t decay_row_stats(const DecayArgs& a, float* rz, float* r, cudaStream_t st)
{
    const int64_t rows = static_cast<int64_t>(a.B) * a.H * a.L, HL = static_cast<int64_t>(a.H) * a.L;
    const int lanes = a.dt == SLAY_F32 ? 16 : 8;
    const unsigned grid = static_cast<unsigned>((rows * lanes + 255) / 256);
    TraceScope trace_("simt_decay_row_stats", st);
    if (a.dt == SLAY_F32)
        k_dec_row_stats<float><<<grid, 256, 0, st>>>(static_cast<const float*>(a.out), static_cast<const float*>(a.dout), a.den,
                                                     rz, r, rows, a.eps, a.lengths, HL, a.L);
    else
        k_dec_row_stats<__nv_bfloat16><<<grid, 256, 0, st>>>(static_cast<const __nv_bfloat16*>(a.out),
                                                             static_cast<const __nv_bfloat16*>(a.dout), a.den, rz, r, rows,
                                                             a.eps, a.lengths, HL, a.L);
    return cudaGetLastError();
}

size_t decay_simt_ws(const DecayArgs& a, bool bwd) { return carve(a, bwd, nullptr).bytes; }

cudaError_t decay_simt_fwd(const DecayArgs& a, void* ws, cudaStream_t st)
{
    return a.dt == SLAY_F32 ? fwd_t<float>(a, ws, st) : fwd_t<__nv_bfloat16>(a, ws, st);
}

cudaError_t decay_simt_bwd(const DecayArgs& a, void* ws, cudaStream_t st)
{
    return a.dt == SLAY_F32 ? bwd_t<float>(a, ws, st) : bwd_t<__nv_bfloat16>(a, ws, st);
}

}  // namespace slay
