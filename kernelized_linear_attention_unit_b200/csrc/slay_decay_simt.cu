// slay_decay_simt.cu -- CUDA-core sweeps of linear attention with a decay for each head (fp32
// mode, and the bf16 sizes the tensor-core sweeps do not take).  The recurrence and its roles
// are described in slay_decay.h.
//
// Three kernels over 64-token chunks, every product a 64 x 64 block of a 256-thread CTA held
// as 4 x 4 fp32 accumulators per thread, operands in shared memory as fp32, two products an
// instruction (B4 H16 L1024 F64 forward 106 us one by one, 100 in pairs; 81 with the loads
// asynchronous and the first of them ahead of the wait for the kernel in front):
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

// `rows` rows of x [.., W], columns [c0, c0 + 64) -> dst [rows][kPitch] fp32, times mul[row]
// when given; rows past n and columns past W are zero.  fp32 without mul arrives asynchronously:
// loads_done() before it is read.
template <typename T>
__device__ __forceinline__ void load_block(float* dst, const T* x, int rows, int n, int W, int c0,
                                           const float* mul = nullptr)
{
    constexpr bool kAsync = sizeof(T) == 4;
    const int wc = min(64, W - c0);
    if ((W & 3) == 0) {
        for (int i = threadIdx.x; i < rows * 16; i += kNT) {
            const int r = i >> 4, c = (i & 15) * 4;
            const bool in = r < n && c < wc;
            const T* from = in ? x + static_cast<int64_t>(r) * W + c0 + c : x;
            if (kAsync && !mul) {
                const uint32_t to = static_cast<uint32_t>(__cvta_generic_to_shared(dst + r * kPitch + c));
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(in ? 16 : 0) : "memory");
                continue;
            }
            float4 w = make_float4(0.f, 0.f, 0.f, 0.f);
            if (in) {
                w = ld4(from);
                if (mul) { const float m = mul[r]; w.x *= m; w.y *= m; w.z *= m; w.w *= m; }
            }
            *reinterpret_cast<float4*>(dst + r * kPitch + c) = w;
        }
    } else {
        for (int i = threadIdx.x; i < rows * 64; i += kNT) {
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
__device__ __forceinline__ void loads_sent() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kOpen>   // but the last kOpen groups sent
__device__ __forceinline__ void loads_done() { asm volatile("cp.async.wait_group %0;" ::"n"(kOpen) : "memory"); }

// d += a b on two floats at once
__device__ __forceinline__ void fma2(float2& d, float2 a, float2 b)
{
    asm("fma.rn.f32x2 %0, %1, %2, %0;"
        : "+l"(reinterpret_cast<uint64_t&>(d))
        : "l"(reinterpret_cast<const uint64_t&>(a)), "l"(reinterpret_cast<const uint64_t&>(b)));
}

// acc[i][..] += a[i] b[..] for a thread's R x 4 block
template <int R>
__device__ __forceinline__ void outer(float2 (&acc)[R][2], const float (&a)[R], float4 b)
{
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const float2 w = make_float2(a[i], a[i]);
        fma2(acc[i][0], w, make_float2(b.x, b.y));
        fma2(acc[i][1], w, make_float2(b.z, b.w));
    }
}

// acc[a][b] += sum_k A[ty + 16 a][k] B[tx + 16 b][k], k < 64
template <int R>
__device__ __forceinline__ void mma_nt(float (&acc)[R][4], const float* A, const float* B, int ty, int tx)
{
    float2 even_odd[R][4] = {};   // sums over even and over odd k
#pragma unroll 4
    for (int k = 0; k < 64; k += 4) {
        float4 a[R], b[4];
#pragma unroll
        for (int i = 0; i < R; ++i) a[i] = *reinterpret_cast<const float4*>(A + (ty + 16 * i) * kPitch + k);
#pragma unroll
        for (int j = 0; j < 4; ++j) b[j] = *reinterpret_cast<const float4*>(B + (tx + 16 * j) * kPitch + k);
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                fma2(even_odd[i][j], make_float2(a[i].x, a[i].y), make_float2(b[j].x, b[j].y));
                fma2(even_odd[i][j], make_float2(a[i].z, a[i].w), make_float2(b[j].z, b[j].w));
            }
    }
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] += even_odd[i][j].x + even_odd[i][j].y;
}

// acc[a] (columns 4 tx to 4 tx + 3) += sum_k A[ty + 16 a][k] B[k][..], k < 64
template <int R>
__device__ __forceinline__ void mma_nn(float2 (&acc)[R][2], const float* A, const float* B, int ty, int tx)
{
#pragma unroll 4
    for (int k = 0; k < 64; k += 4) {
        float a[4][R];
        float4 b[4];
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const float4 w = *reinterpret_cast<const float4*>(A + (ty + 16 * i) * kPitch + k);
            a[0][i] = w.x;
            a[1][i] = w.y;
            a[2][i] = w.z;
            a[3][i] = w.w;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) b[i] = *reinterpret_cast<const float4*>(B + (k + i) * kPitch + 4 * tx);
#pragma unroll
        for (int i = 0; i < 4; ++i) outer<R>(acc, a[i], b[i]);
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
    load_block(fsm, static_cast<const T*>(s.fs) + row0 * s.F, kC, n, s.F, f0);
    loads_sent();
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
    load_block(esm, static_cast<const T*>(s.es) + row0 * 64, kC, n, 64, 0, w);
    loads_done<0>();
    __syncthreads();
    float2 acc[4][2] = {};
#pragma unroll 8
    for (int j = 0; j < kC; ++j) {
        const float4 a = *reinterpret_cast<const float4*>(fsm + j * kPitch + 4 * ty);
        outer<4>(acc, {a.x, a.y, a.z, a.w}, *reinterpret_cast<const float4*>(esm + j * kPitch + 4 * tx));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (f0 + 4 * ty + i < s.F)
            *reinterpret_cast<float4*>(st + (4 * ty + i) * 64 + 4 * tx) =
                make_float4(acc[i][0].x, acc[i][0].y, acc[i][1].x, acc[i][1].y);
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
    const float g = s.log_decay[bh % s.H], g2 = g * kLog2e;
    ChunkDecay lam_c(g, g2, kC);
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
                run = step(nn == kC ? lam_c.next() : decay_pow(g2, nn), run, t[i]);
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

// The outputs' kernels take R x 16 of the chunk's queries a CTA, R rows a thread; what they
// read of the call's own inputs (nothing in the chain writes those) is on its way before the
// kernels in front of them have ended.

// ----------------------------------------------------- outputs 64 wide (out, dv)
template <typename T, int R>
__device__ __forceinline__ void out_f(const Sweep& s, float* sm, int64_t bh, int part, T* o, float* den, bool norm, float eps)
{
    constexpr int kRows = 16 * R;
    float* fqs = sm;                        // [kRows i][64 f]
    float* fss = fqs + 64 * kPitch;         // [64 j][64 f]; then the scores [kRows i][64 j]
    float* ms = fss + 64 * kPitch;          // [64 f][64 e]
    float* ess = ms + 64 * kPitch;          // [64 j][64 e]
    __shared__ float pw[kC], smul[kC], zs[64], dsum[kRows];
    const int c = blockIdx.x, i0 = part * kRows;
    const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
    const int t0 = c * kC, n = min(kC, seq_len(s.lengths, static_cast<int>(bh / s.H), s.L) - t0);
    const float g2 = s.log_decay[bh % s.H] * kLog2e;
    const int64_t row0 = bh * s.L + t0;
    auto load_rows = [&](int f0) {
        load_block(fqs, static_cast<const T*>(s.fq) + (row0 + i0) * s.F, kRows, n - i0, s.F, f0);
        load_block(fss, static_cast<const T*>(s.fs) + row0 * s.F, kC, n, s.F, f0);
    };
    auto load_state = [&](int f0) {
        load_block(ms, s.st + ((bh * s.nc + c) * s.F + f0) * 64, 64, min(64, s.F - f0), 64, 0);
        if (norm && tid < 64) zs[tid] = f0 + tid < s.F ? s.sz[(bh * s.nc + c) * s.F + f0 + tid] : 0.0f;
    };
    if (n > i0) load_rows(0);
    if (tid < kC) pw[tid] = decay_pow(g2, tid);
    if (tid < kRows) dsum[tid] = 0.0f;
    after_previous_kernel();
    if (n <= i0) return;
    load_state(0);
    loads_sent();
    load_block(ess, static_cast<const T*>(s.es) + row0 * 64, kC, n, 64, 0);
    loads_sent();
    if (tid < kC) smul[tid] = tid < n && s.s_mul ? s.s_mul[row0 + tid] : 1.0f;
    float p[R][4] = {}, dz = 0.0f;
    float2 acc[R][2] = {};
    constexpr int kLanes = kNT / kRows, kEach = 64 / kLanes;   // threads of a row and their features of z
    loads_done<1>();
    for (int f0 = 0;;) {
        __syncthreads();
        mma_nt<R>(p, fqs, fss, ty, tx);
        mma_nn<R>(acc, fqs, ms, ty, tx);
        if (norm) {
            const int i = tid / kLanes, k0 = (tid % kLanes) * kEach;
#pragma unroll
            for (int k = 0; k < kEach; ++k) dz = fmaf(fqs[i * kPitch + k0 + k], zs[k0 + k], dz);
        }
        __syncthreads();
        f0 += 64;
        if (f0 >= s.F) break;
        load_rows(f0);
        load_state(f0);
        loads_sent();
        loads_done<0>();
    }
    float rs[R] = {};
#pragma unroll
    for (int a = 0; a < R; ++a)
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const int i = ty + 16 * a, j = tx + 16 * b;
            const float w = score(p[a][b], i0 + i, j, n, s.rev, 0.0f, 0.0f, 1.0f, smul, pw);
            fss[i * kPitch + j] = w;
            rs[a] += w;
        }
    if (norm) {
#pragma unroll
        for (int a = 0; a < R; ++a) {
            for (int x = 8; x > 0; x >>= 1) rs[a] += __shfl_xor_sync(0xffffffffu, rs[a], x);
            if (tx == 0) dsum[ty + 16 * a] = rs[a];
        }
#pragma unroll
        for (int x = 1; x < kLanes; x *= 2) dz += __shfl_xor_sync(0xffffffffu, dz, x);
    }
    loads_done<0>();
    __syncthreads();
    if (norm && tid % kLanes == 0) {
        const int i = tid / kLanes;
        const float d = fmaf(decay_pow(g2, s.rev ? max(n - 1 - i0 - i, 0) : i0 + i + 1), dz, dsum[i]);
        dsum[i] = d;
        if (den && i0 + i < n) den[row0 + i0 + i] = d;
    }
#pragma unroll
    for (int a = 0; a < R; ++a) {
        const int i = i0 + ty + 16 * a;
        const float fac = decay_pow(g2, s.rev ? max(n - 1 - i, 0) : i + 1);
#pragma unroll
        for (int b = 0; b < 2; ++b) acc[a][b] = make_float2(acc[a][b].x * fac, acc[a][b].y * fac);
    }
    mma_nn<R>(acc, fss, ess, ty, tx);
    if (norm) __syncthreads();
#pragma unroll
    for (int a = 0; a < R; ++a) {
        const int i = ty + 16 * a;
        if (i0 + i >= n) continue;
        const float rden = norm ? dsum[i] + eps : 1.0f;
        float4 w = make_float4(acc[a][0].x, acc[a][0].y, acc[a][1].x, acc[a][1].y);
        if (norm) { w.x /= rden; w.y /= rden; w.z /= rden; w.w /= rden; }
        st4(o + (row0 + i0 + i) * 64 + 4 * tx, w);
    }
}

// ----------------------------------------------------- outputs F wide (dphq, dphk)
template <typename T, int R>
__device__ __forceinline__ void out_e(const Sweep& s, float* sm, int64_t bh, int part, int group, int groups, T* o, bool norm)
{
    constexpr int kRows = 16 * R;
    float* eqs = sm;                        // [kRows i][64 e]
    float* ps = eqs + 64 * kPitch;          // E side of the state, then the scores [kRows i][64 j]
    float* fss = ps + 64 * kPitch;          // [64 j][64 f]
    float* ms = fss + 64 * kPitch;          // [64 f][64 e]
    __shared__ float pw[kC], smul[kC], soff[kC], zs[64];
    const int c = blockIdx.x, i0 = part * kRows;
    const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
    const int t0 = c * kC, n = min(kC, seq_len(s.lengths, static_cast<int>(bh / s.H), s.L) - t0);
    const float g2 = s.log_decay[bh % s.H] * kLog2e;
    const int64_t row0 = bh * s.L + t0;
    auto load_rows = [&](int f0) { load_block(fss, static_cast<const T*>(s.fs) + row0 * s.F, kC, n, s.F, f0); };
    auto load_state = [&](int f0) {
        load_block(ms, s.st + ((bh * s.nc + c) * s.F + f0) * 64, 64, min(64, s.F - f0), 64, 0);
        if (tid < 64) zs[tid] = norm && f0 + tid < s.F ? s.sz[(bh * s.nc + c) * s.F + f0 + tid] : 0.0f;
    };
    int f0 = group * 64;
    if (n > i0) {
        load_block(eqs, static_cast<const T*>(s.eq) + (row0 + i0) * 64, kRows, n - i0, 64, 0);
        load_block(ps, static_cast<const T*>(s.es) + row0 * 64, kC, n, 64, 0);
        loads_sent();
        load_rows(f0);
    }
    after_previous_kernel();
    if (n <= i0) return;
    load_state(f0);
    loads_sent();
    if (tid < kC) {
        const bool in = tid < n;
        pw[tid] = decay_pow(g2, tid);
        smul[tid] = in && s.s_mul ? s.s_mul[row0 + tid] : 1.0f;
        soff[tid] = in && s.s_off ? s.s_off[row0 + tid] : 0.0f;
    }
    loads_done<1>();
    __syncthreads();
    float p[R][4] = {};
    mma_nt<R>(p, eqs, ps, ty, tx);
    __syncthreads();
    // per query row: the score's scalars, the state's factor and the weight of its z column
    float fac[R], zc[R];
#pragma unroll
    for (int a = 0; a < R; ++a) {
        const int i = i0 + ty + 16 * a;
        const bool in = i < n;
        const float qm = in && s.q_mul ? s.q_mul[row0 + i] : 1.0f;
        const float qo = in && s.q_off ? s.q_off[row0 + i] : 0.0f;
        fac[a] = qm * decay_pow(g2, s.rev ? max(n - 1 - i, 0) : i + 1);
        zc[a] = s.q_off ? -qo : 1.0f;
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const int j = tx + 16 * b;
            ps[(ty + 16 * a) * kPitch + j] = score(p[a][b], i, j, n, s.rev, qo, soff[j], qm, smul, pw);
        }
    }
    const bool vec = (s.F & 3) == 0;
    for (;;) {
        loads_done<0>();
        __syncthreads();
        // inter-chunk part with columns tx + 16 b; through shared memory to columns 4 tx + b
        float t[R][4] = {};
        float2 acc[R][2] = {};
        mma_nt<R>(t, eqs, ms, ty, tx);
        __syncthreads();
#pragma unroll
        for (int a = 0; a < R; ++a)
#pragma unroll
            for (int b = 0; b < 4; ++b)
                ms[(ty + 16 * a) * kPitch + tx + 16 * b] = fac[a] * fmaf(zc[a], zs[tx + 16 * b], t[a][b]);
        __syncthreads();
        mma_nn<R>(acc, ps, fss, ty, tx);
#pragma unroll
        for (int a = 0; a < R; ++a) {
            const int i = ty + 16 * a, f = f0 + 4 * tx;
            if (i0 + i >= n) continue;
            const float4 m = *reinterpret_cast<const float4*>(ms + i * kPitch + 4 * tx);
            const float4 w = make_float4(acc[a][0].x + m.x, acc[a][0].y + m.y, acc[a][1].x + m.z, acc[a][1].y + m.w);
            T* dst = o + (row0 + i0 + i) * s.F + f;
            if (vec) {
                if (f < s.F) st4(dst, w);
            } else {
                if (f < s.F) stf(dst, w.x);
                if (f + 1 < s.F) stf(dst + 1, w.y);
                if (f + 2 < s.F) stf(dst + 2, w.z);
                if (f + 3 < s.F) stf(dst + 3, w.w);
            }
        }
        f0 += groups * 64;
        if (f0 >= s.F) break;
        __syncthreads();
        load_rows(f0);
        load_state(f0);
        loads_sent();
    }
}

// grid (nc, BH, 4 / R)
template <typename T, int R>
__global__ void __launch_bounds__(kNT) k_dec_fwd(Sweep s, T* o, float* den, bool norm, float eps)
{
    extern __shared__ __align__(16) float sm[];
    out_f<T, R>(s, sm, blockIdx.y, blockIdx.z, o, den, norm, eps);
}

// The three gradients side by side: grid (nc, 3 BH, 4 / R x column groups of the F-wide ones)
template <typename T, int R>
__global__ void __launch_bounds__(kNT) k_dec_grads(Sweep s, Sweep g, T* dphq, T* dphk, T* dv, int BH, bool norm)
{
    extern __shared__ __align__(16) float sm[];
    constexpr int kParts = 4 / R;
    const int role = blockIdx.y / BH, bh = blockIdx.y % BH, part = blockIdx.z % kParts, group = blockIdx.z / kParts;
    if (role < 2) out_e<T, R>(role ? g : s, sm, bh, part, group, gridDim.z / kParts, role ? dphk : dphq, norm);
    else if (group == 0) out_f<T, R>(g, sm, bh, part, dv, nullptr, false, 0.0f);
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

constexpr size_t kSmemS = 2 * 64 * kPitch * sizeof(float), kSmemO = 4 * 64 * kPitch * sizeof(float);
// Up to this many CTAs, the outputs' kernels take half a chunk's queries each (R = 2): the
// halves still find an SM each.  B1 H3 L512 F128 forward (24 CTAs) 20.5 us with halves against 22.8
// with whole chunks, backward B1 H2 F64 (48) 17.5 / 19.5; beyond, the features decide and the rule
// takes the safer side: 120 CTAs forward F128 30.8 / 34.9, F64 22.6 / 20.5, backward F64 (72)
// 25.0 / 19.6.
constexpr int64_t kFew = 64;

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

template <typename K, typename... A>
cudaError_t outputs(K* kernel, dim3 grid, cudaStream_t st, A... args)
{
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemO);
    if (e != cudaSuccess) return e;
    TraceScope trace_("simt_decay_out", st);
    return launch_in_chain(false, kernel, grid, kNT, kSmemO, st, args...);
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
    cudaError_t e;
    Sweep s = base(a, c);
    s.fq = a.phq;
    s.fs = a.phk;
    s.es = a.v;
    s.first = a.S_in;
    s.first_z = a.z_in;
    s.last = a.S_out;
    s.last_z = a.z_out;
    if ((e = states<T>(s, nullptr, BH, false, st)) != cudaSuccess || s.nc == 0) return e;
    const bool few = static_cast<int64_t>(s.nc) * BH <= kFew;
    return outputs(few ? k_dec_fwd<T, 2> : k_dec_fwd<T, 4>, dim3(s.nc, BH, few ? 2 : 1), st, s, static_cast<T*>(a.out_w),
                   a.den_w, a.norm, a.eps);
}

template <typename T>
cudaError_t bwd_t(const DecayArgs& a, void* ws, cudaStream_t st)
{
    const Carve c = carve(a, true, ws);
    const int BH = a.B * a.H;
    cudaError_t e;
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
    const int groups = static_cast<int>(ctas >= 296 ? 1 : std::min<int64_t>(nfb, (296 + ctas - 1) / ctas));
    const bool few = ctas * groups <= kFew;
    return outputs(few ? k_dec_grads<T, 2> : k_dec_grads<T, 4>, dim3(s.nc, 3 * BH, few ? 2 * groups : groups), st, s, g,
                   static_cast<T*>(a.dphq), static_cast<T*>(a.dphk), static_cast<T*>(a.dv), BH, a.norm);
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
