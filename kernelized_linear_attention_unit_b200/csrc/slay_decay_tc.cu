// slay_decay_tc.cu -- tensor-core sweeps of linear attention with a decay for each head (bf16
// operands).  The recurrence and the roles its operands take are described in slay_decay.h.
//
// One CTA walks the 128-token chunks of one segment of one (b, h) with the running state M
// [F][64] in the fp32 registers of its epilogue warps.  Per chunk, over 64-feature slices of
// the F-side rows and with every accumulator in tensor memory:
//   scores  P  = x y^T                      (M = N = 128)
//   state   T  = sum_j y_j (w_j u_j)^T      (M = 128 features, N = 64, K = 128 tokens)
//   outputs Oi = P~ u,  Oe = x M            (P~: P masked, decayed, rounded to bf16)
//   o_i = Oi + lambda^(i+1) Oe,  M <- lambda^n M + T.
// Oi and Oe stay apart so that the row factor lambda^(i+1) is applied in fp32.
//
// Roundings to bf16 (all else is fp32): P~ and the copy of M that the tensor core reads, one
// each, so an output sees two besides its own; the decay weight of a token's state term is
// folded into the 64-wide side as w_j u_j = hi + mid + lo, three bf16 limbs accumulated in the
// same accumulator, so the fp32 states that leave the call are as exact as fp32 sums (one limb
// alone would be off by 2^-9, two by 2^-17).  The z column (the ones column of u) takes its
// weights as three bf16 columns of a 16-wide operand, exactly as well, and so does the
// denominator's state part; the denominator's other part is summed in fp32 from the scores.
//
// Bound: HBM.  A 128-token chunk at F = 256 moves 164 KB (7000 clocks at an SM's share of the
// bandwidth) and needs about 1800 clocks of tensor-core time, three state limbs included.  When
// there are fewer (b, h) than SMs the sequence is cut into segments: k_tc_dec<kState> sums each
// segment's own state (reading the F side and the 64-wide side once more), k_dec_seg_scan
// turns those into the states entering each segment, and the output sweeps start from them.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "slay_decay.h"
#include "slay_tc_common.cuh"
#include "slay_tc_ptx.cuh"

namespace slay {

using namespace tc;

namespace {

constexpr int kT = 128;               // tokens per chunk
constexpr int kTile = kT * 128;       // [128][64] bf16, 128-byte swizzle = 16 KiB
constexpr int kSlab = 64 * 128;       // [64 f][64 e] bf16 = 8 KiB
constexpr int kExt = 16 * 128;        // [16][64] bf16 = 2 KiB
constexpr int kThreads = 32 * 10;     // MMA warp, TMA warp, 8 epilogue warps
constexpr int kNumSMs = 148;
constexpr int kMaxFw = 256;           // features of one sweep

enum Mode { kState = 0, kOutF = 1, kOutE = 2 };

// tensor memory columns
constexpr uint32_t kColP = 0, kColPt = 128, kColT = 192, kColO = 352;
constexpr uint32_t kTStride = 80;     // T of 128 features: 64 columns and 16 for z

enum {
    B_FSF = 0, B_FSE = 4, B_FQF = 8, B_FQE = 10, B_ESF = 12, B_ESE = 14, B_YF = 16, B_MF, B_PF, B_PT, B_TF,
    B_OF = 21, B_OE = 23, B_NUM = 25
};

struct Layout {
    uint32_t fs, fq, es, eq, y, m, zext, wext, pw, smul, soff, dsum, zf, bar, tmem, total;
};

__host__ __device__ constexpr Layout layout(int mode)
{
    Layout l{};
    uint32_t o = 0;
    l.fs = o; o += 4 * kTile;                           // ring of four F-side slices
    l.fq = o; o += mode == kOutF ? 2 * kTile : 0;       // ring of two query slices
    l.es = o; o += 2 * kTile;                           // 64-wide side, two chunks
    l.eq = o; o += mode == kOutE ? 2 * kTile : 0;       // 64-wide queries, two chunks
    l.y = o; o += 3 * kTile;                            // weighted rows, three limbs
    l.m = o; o += mode == kState ? 0 : 4 * kSlab;       // the state as an operand
    l.zext = o; o += mode == kOutF ? 4 * kExt : 0;      // its z column, three limbs of 16 columns
    l.wext = o; o += 2 * kExt;                          // z weights of the chunk's tokens, likewise
    l.pw = o; o += 128 * 4;                             // lambda^d
    l.smul = o; o += 2 * 128 * 4;                       // score scalars of the state tokens
    l.soff = o; o += 2 * 128 * 4;
    l.dsum = o; o += mode == kOutF ? 2 * 2 * 128 * 4 : 0;                   // row sums of the scores, by column half
    l.zf = o; o += mode == kOutE ? 2 * kMaxFw * 4 : 0;                      // z in fp32
    l.bar = o; o += B_NUM * 8;
    l.tmem = o; o += 16;
    l.total = o;
    return l;
}

struct P {
    const float* log_decay;
    const int32_t* lengths;
    const float *s_mul, *s_off, *q_mul, *q_off;   // row scalars, null: 1 / 0
    const float *first, *first_z;                 // states entering: [BH][nseg] (or [BH]), null: zero
    float *last, *last_z;                         // states leaving, likewise, null: not wanted
    __nv_bfloat16* o;
    float* den;
    float *part, *part_den;                       // numerators and denominators over features [BH][L][64], [BH][L]
    int part_mode;                                // 0: none, 1: store them, 2: add them to this block's
    float eps;
    int H, L, F, nseg, nfb, fw, fb0;
    int rev, has_z, z_delta, has_den;
    int* err;
};

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// x = l0 + l1 + l2 to 2^-24, each a bf16 (bit patterns)
__device__ __forceinline__ void limbs3(float x, uint16_t (&l)[3])
{
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        const __nv_bfloat16 b = __float2bfloat16_rn(x);
        l[i] = __bfloat16_as_ushort(b);
        x -= __bfloat162float(b);
    }
}

__device__ __forceinline__ void st_shared_u16(uint32_t addr, uint16_t x)
{
    asm volatile("st.shared.u16 [%0], %1;" ::"r"(addr), "h"(x) : "memory");
}

template <int kMode>
__global__ void __launch_bounds__(kThreads, 1)
k_tc_dec(const __grid_constant__ CUtensorMap tfs, const __grid_constant__ CUtensorMap tfq,
         const __grid_constant__ CUtensorMap tes, const __grid_constant__ CUtensorMap teq, const P p)
{
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char* sm = aligned_smem(smem_raw);
    constexpr Layout Lo = layout(kMode);
    uint64_t* bar = reinterpret_cast<uint64_t*>(sm + Lo.bar);
    uint32_t* tslot = reinterpret_cast<uint32_t*>(sm + Lo.tmem);
    const uint32_t sbase = smem_u32(sm);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    // this CTA's feature block, segment and sequence
    int x = blockIdx.x;
    const int fb = kMode == kOutF ? p.fb0 : x % p.nfb;
    if (kMode != kOutF) x /= p.nfb;
    const int seg = x % p.nseg, bh = x / p.nseg;
    const int f0 = fb * p.fw, fv = min(p.fw, p.F - f0);
    const int ns = (fv + 63) >> 6, nsE = (ns + 1) & ~1;   // 64-feature slices; as whole pairs
    const int len = p.lengths ? min(max(p.lengths[bh / p.H], 0), p.L) : p.L;
    const int nch = (len + kT - 1) / kT;
    const int c_lo = static_cast<int>(static_cast<int64_t>(seg) * nch / p.nseg);
    const int count = static_cast<int>(static_cast<int64_t>(seg + 1) * nch / p.nseg) - c_lo;
    auto chunk_of = [&](int i) { return p.rev ? c_lo + count - 1 - i : c_lo + i; };
    const float g2 = p.log_decay[bh % p.H] * kLog2e;
    // without decay and row scalars the weights are 1 and one limb is exact
    const int nl = g2 == 0.0f && !p.s_mul ? 1 : 3;

    if (warp == 0) {
        tmem_alloc(tslot, 512);
        tmem_relinquish();
    }
    for (uint32_t i = Lo.zext / 4 + tid; i < Lo.pw / 4; i += kThreads) reinterpret_cast<uint32_t*>(sm)[i] = 0u;
    if (tid < kT) reinterpret_cast<float*>(sm + Lo.pw)[tid] = decay_pow(g2, tid);
    if (tid == 0) {
        for (int i = 0; i < B_NUM; ++i)
            mbar_init(&bar[i], i == B_YF || i == B_MF || i == B_PT || i == B_OE || i == B_OE + 1 ? 8 : 1);
        mbar_fence_init();
        tma_prefetch_desc(&tfs);
        tma_prefetch_desc(&tes);
        if (kMode == kOutF) tma_prefetch_desc(&tfq);
        if (kMode == kOutE) tma_prefetch_desc(&teq);
    }
    fence_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tslot;
    Waiter wt;
    // waits on the k-th completion (k >= 0) of a barrier
    auto wait_k = [&](int b, int k) {
        uint32_t ph = static_cast<uint32_t>(k & 1);
        wt.wait(&bar[b], ph);
    };

    if (warp == 1) {
        // ------------------------------------------------------------------ TMA loads
        if (lane == 0) {
            for (int i = 0; i < count && wt.ok; ++i) {
                const int t0 = chunk_of(i) * kT, b = i & 1;
                if (i >= 2) wait_k(B_ESE + b, (i >> 1) - 1);
                mbar_arrive_expect_tx(&bar[B_ESF + b], kMode == kOutE ? 2 * kTile : kTile);
                tma_load_3d(sm + Lo.es + b * kTile, &tes, &bar[B_ESF + b], 0, t0, bh);
                if (kMode == kOutE) tma_load_3d(sm + Lo.eq + b * kTile, &teq, &bar[B_ESF + b], 0, t0, bh);
                for (int s = 0; s < nsE; ++s) {
                    const int u = i * nsE + s, sl = u & 3;
                    if (u >= 4) wait_k(B_FSE + sl, (u >> 2) - 1);
                    if (s < ns) {
                        mbar_arrive_expect_tx(&bar[B_FSF + sl], kTile);
                        tma_load_3d(sm + Lo.fs + sl * kTile, &tfs, &bar[B_FSF + sl], f0 + 64 * s, t0, bh);
                    } else {
                        mbar_arrive(&bar[B_FSF + sl]);   // the second half of the last pair: not read
                    }
                    if (kMode == kOutF && s < ns) {
                        const int u2 = i * ns + s, q = u2 & 1;
                        if (u2 >= 2) wait_k(B_FQE + q, (u2 >> 1) - 1);
                        mbar_arrive_expect_tx(&bar[B_FQF + q], kTile);
                        tma_load_3d(sm + Lo.fq + q * kTile, &tfq, &bar[B_FQF + q], f0 + 64 * s, t0, bh);
                    }
                }
            }
        }
        __syncwarp();
    } else if (warp == 0) {
        // ------------------------------------------------------------------ MMA issue
        constexpr uint32_t idP = idesc_bf16(128, 128, 0, 0);
        constexpr uint32_t idKM = idesc_bf16(128, 64, 0, 1);    // A K-major (or tensor memory), B MN-major
        constexpr uint32_t idKK = idesc_bf16(128, 64, 0, 0);
        constexpr uint32_t idMM = idesc_bf16(128, 64, 1, 1);
        constexpr uint32_t idMz = idesc_bf16(128, 16, 1, 0);
        constexpr uint32_t idKz = idesc_bf16(128, 16, 0, 0);
        const uint64_t dfs = sdesc(sbase + Lo.fs, 16, 1024, kLayoutSW128);
        const uint64_t dfsT = sdesc(sbase + Lo.fs, kTile, 1024, kLayoutSW128);   // M = 128 over two slices
        const uint64_t dfq = sdesc(sbase + Lo.fq, 16, 1024, kLayoutSW128);
        const uint64_t des = sdesc(sbase + Lo.es, 16, 1024, kLayoutSW128);
        const uint64_t deq = sdesc(sbase + Lo.eq, 16, 1024, kLayoutSW128);
        const uint64_t dy = sdesc(sbase + Lo.y, 16, 1024, kLayoutSW128);
        const uint64_t dm = sdesc(sbase + Lo.m, 16, 1024, kLayoutSW128);
        const uint64_t dze = sdesc(sbase + Lo.zext, 16, 1024, kLayoutSW128);
        const uint64_t dwe = sdesc(sbase + Lo.wext, 16, 1024, kLayoutSW128);
        constexpr uint32_t kTd = kTile >> 4, kSd = kSlab >> 4, kEd = kExt >> 4;
        const bool lead = lane == 0;
        auto wait_m = [&](int b, int k) {
            wait_k(b, k);
            tc_fence_after();
        };
        for (int i = 0; i < count && wt.ok; ++i) {
            const int t0 = chunk_of(i) * kT, n = min(kT, len - t0), eb = i & 1;
            const uint64_t desi = des + eb * kTd;
            // rows of the tensor behind this sequence may hold anything: cleared in the slice,
            // since they enter sums over tokens (rows past L arrive as zero)
            const bool clear = n < kT && t0 + n < p.L;
            auto slice = [&](int s) {   // F-side slice s of the chunk, complete and clean
                const int u = i * nsE + s, sl = u & 3;
                wait_m(B_FSF + sl, u >> 2);
                if (clear) {
                    for (int a = n * 8 + lane; a < kT * 8; a += 32)
                        st_shared_v4(sbase + Lo.fs + sl * kTile + a * 16, 0u, 0u, 0u, 0u);
                    fence_async_smem();
                    __syncwarp();
                }
                return sl;
            };
            auto state_pair = [&](int s) {   // T of the pair whose last slice is s
                const uint64_t da = dfsT + ((i * nsE + (s & ~1)) & 3) * kTd;
                const uint32_t t = tmem + kColT + kTStride * (s >> 1);
                for (int l = 0; l < nl; ++l)
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk)
                        umma_bf16(t, da + 128 * kk, dy + l * kTd + 128 * kk, idMM, (l > 0 || kk > 0) ? 1u : 0u);
                if (p.has_z)
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk)
                        umma_bf16(t + 64, da + 128 * kk, dwe + (kk >> 2) * kEd + 2 * (kk & 3), idMz, kk > 0 ? 1u : 0u);
            };
            auto free_pair = [&](int s) {
                const int sl = (i * nsE + (s & ~1)) & 3;
                umma_commit(&bar[B_FSE + sl]);
                umma_commit(&bar[B_FSE + sl + 1]);
            };
            if (kMode == kOutE) {
                wait_m(B_ESF + eb, i >> 1);
                const int v = i * ns - 1, vo = (v & 1) ? v : v - 1;   // last use of the buffer over P
                if (vo >= 1) wait_m(B_OE + 1, vo >> 1);
                if (lead) {
                    const uint64_t deqi = deq + eb * kTd;
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        umma_bf16(tmem + kColP, deqi + 2 * kk, desi + 2 * kk, idP, kk > 0 ? 1u : 0u);
                    umma_commit(&bar[B_PF]);
                }
            }
            for (int s = 0; s < ns; ++s) {
                const int sl = slice(s);
                const bool pair_done = (s & 1) || s == ns - 1;
                if (kMode == kOutF) {
                    const int u2 = i * ns + s, q = u2 & 1;
                    wait_m(B_FQF + q, u2 >> 1);
                    const uint64_t dx = dfq + q * kTd, dyy = dfs + sl * kTd;
                    if (lead) {
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            umma_bf16(tmem + kColP, dx + 2 * kk, dyy + 2 * kk, idP, (s > 0 || kk > 0) ? 1u : 0u);
                        if (s == ns - 1) umma_commit(&bar[B_PF]);
                    }
                    if (s == 0) {
                        wait_m(B_MF, i);
                        if (i >= 1) wait_m(B_OE, i - 1);
                    }
                    if (lead) {
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            umma_bf16(tmem + kColO + 64, dx + 2 * kk, dm + s * kSd + 128 * kk, idKM,
                                      (s > 0 || kk > 0) ? 1u : 0u);
                        if (p.has_den)
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk)
                                umma_bf16(tmem + kColO + 128, dx + 2 * kk, dze + s * kEd + 2 * kk, idKz,
                                          (s > 0 || kk > 0) ? 1u : 0u);
                        umma_commit(&bar[B_FQE + q]);
                    }
                }
                if (!pair_done) continue;
                if (s <= 1) {
                    wait_m(B_YF, i);
                    if (kMode != kOutF) wait_m(B_MF, i);
                }
                if (lead) state_pair(s);
                if (kMode == kOutE) {
                    if (s <= 1) wait_m(B_PT, i);
                    for (int r = s & ~1; r <= s; ++r) {
                        const int v = i * ns + r, ob = v & 1;
                        if (v >= 2) wait_m(B_OE + ob, (v >> 1) - 1);
                        const uint32_t oi = tmem + (ob ? kColP : kColO);
                        const uint64_t du = dfs + ((i * nsE + r) & 3) * kTd, deqi = deq + eb * kTd;
                        if (lead) {
#pragma unroll
                            for (int kk = 0; kk < 8; ++kk)
                                umma_bf16_ts(oi, tmem + kColPt + 8 * kk, du + 128 * kk, idKM, kk > 0 ? 1u : 0u);
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk)
                                umma_bf16(oi + 64, deqi + 2 * kk, dm + r * kSd + 2 * kk, idKK, kk > 0 ? 1u : 0u);
                            umma_commit(&bar[B_OF + ob]);
                        }
                    }
                }
                if (lead) free_pair(s);
            }
            if (lead) umma_commit(&bar[B_TF]);
            if (kMode == kOutF) {
                wait_m(B_PT, i);
                if (lead) {
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk)
                        umma_bf16_ts(tmem + kColO, tmem + kColPt + 8 * kk, desi + 128 * kk, idKM, kk > 0 ? 1u : 0u);
                    umma_commit(&bar[B_OF]);
                }
            }
            if (lead) umma_commit(&bar[B_ESE + eb]);
            __syncwarp();
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------------ epilogue
        // (no early exit on a wait that ran out: the named barriers want every warp)
        const int q = warp & 3, half = (warp - 2) >> 2;
        const int row = 32 * q + lane;           // token of scores and outputs; feature of T
        const uint32_t trow = tmem + ((32u * q) << 16);
        const float* pw = reinterpret_cast<const float*>(sm + Lo.pw);
        float* smul = reinterpret_cast<float*>(sm + Lo.smul);
        float* soff = reinterpret_cast<float*>(sm + Lo.soff);
        float* dsum = reinterpret_cast<float*>(sm + Lo.dsum);
        float* zf = reinterpret_cast<float*>(sm + Lo.zf);
        const int64_t sidx = static_cast<int64_t>(bh) * p.nseg + seg;
        float run[2][32], zrun = 0.0f;           // M at (f = 128 b + row, e = 32 half + c); z at b = half
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const int f = 128 * b + row;
            const bool in = p.first && f < fv;
            const float4* src = reinterpret_cast<const float4*>(p.first + ((sidx * p.F) + f0 + f) * 64 + 32 * half);
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                const float4 w = in ? src[c] : make_float4(0.f, 0.f, 0.f, 0.f);
                run[b][4 * c] = w.x;
                run[b][4 * c + 1] = w.y;
                run[b][4 * c + 2] = w.z;
                run[b][4 * c + 3] = w.w;
            }
            if (b == half && in && p.has_z) zrun = p.first_z[sidx * p.F + f0 + f];
        }
        // the operand copy of M, and its z column, for chunk i
        auto write_m = [&](int i) {
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const int f = 128 * b + row;
                if (f < 64 * ns) {
                    const uint32_t slab = sbase + Lo.m + (f >> 6) * kSlab;
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        st_shared_v4(slab + sw128_off(f & 63, 4 * half + c),
                                     pack_bf16(run[b][8 * c], run[b][8 * c + 1]), pack_bf16(run[b][8 * c + 2], run[b][8 * c + 3]),
                                     pack_bf16(run[b][8 * c + 4], run[b][8 * c + 5]), pack_bf16(run[b][8 * c + 6], run[b][8 * c + 7]));
                    if (b == half && p.has_z) {
                        if (kMode == kOutF) {
                            uint16_t l[3];
                            limbs3(zrun, l);
                            const uint32_t t = sbase + Lo.zext + (f >> 6) * kExt;
#pragma unroll
                            for (int k = 0; k < 3; ++k) st_shared_u16(t + sw128_off(k, (f & 63) >> 3) + (f & 7) * 2, l[k]);
                        } else {
                            zf[(i & 1) * kMaxFw + f] = zrun;
                        }
                    }
                }
            }
            fence_async_smem();
        };
        // the weighted rows of chunk i (this thread: token `row`, 32 of its columns) in limbs,
        // the z weights and the score scalars of its tokens
        auto write_y = [&](int i) {
            const int t0 = chunk_of(i) * kT, n = min(kT, len - t0), eb = i & 1;
            const bool in = row < n;
            const int64_t grow = static_cast<int64_t>(bh) * p.L + t0 + row;
            const float mul = in && p.s_mul ? p.s_mul[grow] : 1.0f;
            const float off = in && p.s_off ? p.s_off[grow] : 0.0f;
            const float w = in ? decay_pow(g2, p.rev ? row + 1 : n - 1 - row) : 0.0f;
            const float a = w * mul;
            wait_k(B_ESF + eb, i >> 1);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const uint32_t o = sw128_off(row, 4 * half + c);
                uint4* src = reinterpret_cast<uint4*>(sm + Lo.es + eb * kTile + o);
                const uint4 r = *src;
                uint32_t v[4] = {r.x, r.y, r.z, r.w};
                if (!in) {
                    v[0] = v[1] = v[2] = v[3] = 0u;
                    if (kMode == kOutF) *src = make_uint4(0u, 0u, 0u, 0u);   // they are an operand as they are, too
                }
                if (nl == 1) {
                    st_shared_v4(sbase + Lo.y + o, v[0], v[1], v[2], v[3]);
                    continue;
                }
                uint32_t l[3][4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float y0 = a * bf_lo(v[e]), y1 = a * bf_hi(v[e]);
#pragma unroll
                    for (int k = 0; k < 3; ++k) {
                        l[k][e] = pack_bf16(y0, y1);
                        y0 -= bf_lo(l[k][e]);
                        y1 -= bf_hi(l[k][e]);
                    }
                }
#pragma unroll
                for (int k = 0; k < 3; ++k)
                    st_shared_v4(sbase + Lo.y + k * kTile + o, l[k][0], l[k][1], l[k][2], l[k][3]);
            }
            if (half == 0) {
                if (p.has_z) {
                    uint16_t l[3];
                    limbs3(p.z_delta ? -a * off : w, l);
                    const uint32_t t = sbase + Lo.wext + (row >> 6) * kExt;
#pragma unroll
                    for (int k = 0; k < 3; ++k) st_shared_u16(t + sw128_off(k, (row & 63) >> 3) + (row & 7) * 2, l[k]);
                }
                smul[(i & 1) * kT + row] = mul;
                soff[(i & 1) * kT + row] = off;
            }
            fence_async_smem();
            warp_arrive(&bar[B_YF]);
        };
        if (count > 0) {
            if (kMode != kState) write_m(0);
            warp_arrive(&bar[B_MF]);
            write_y(0);
            named_bar_sync(1, 256);
        }
        for (int i = 0; i < count; ++i) {
            const int t0 = chunk_of(i) * kT, n = min(kT, len - t0), par = i & 1;
            const int64_t grow = static_cast<int64_t>(bh) * p.L + t0 + row;
            const bool valid = row < n;
            float fac = decay_pow(g2, p.rev ? max(n - 1 - row, 0) : row + 1), qo = 0.0f, qm = 1.0f;
            if (kMode == kOutE && valid) {
                if (p.q_mul) qm = p.q_mul[grow];
                if (p.q_off) qo = p.q_off[grow];
            }
            if (kMode != kState) {
                // masked, decayed scores -> P~ (this warp's half of the columns)
                wait_k(B_PF, i);
                tc_fence_after();
                float rs = 0.0f;
                const bool cols = p.s_mul != nullptr;
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) {
                    uint32_t r[32], pk[16];
                    tmem_ld32(trow + kColP + 64 * half + 32 * hh, r);
                    tmem_wait_ld();
                    reg_fence(r);
                    const int j0 = 64 * half + 32 * hh;
                    float w[32];
#pragma unroll
                    for (int c = 0; c < 32; ++c) {
                        const int j = j0 + c, d = p.rev ? j - row : row - j;
                        float sc = __uint_as_float(r[c]);
                        if (kMode == kOutE) sc -= qo;
                        if (cols) sc = (kMode == kOutE ? sc - soff[par * kT + j] : sc) * smul[par * kT + j];
                        w[c] = d >= 0 && j < n ? sc * pw[max(d, 0)] : 0.0f;
                    }
#pragma unroll
                    for (int c = 0; c < 16; ++c) {
                        if (kMode == kOutE) { w[2 * c] *= qm; w[2 * c + 1] *= qm; }
                        if (kMode == kOutF) rs += w[2 * c] + w[2 * c + 1];
                        pk[c] = pack_bf16(w[2 * c], w[2 * c + 1]);
                    }
                    tmem_st16(trow + kColPt + 32 * half + 16 * hh, pk);
                }
                tmem_wait_st();
                if (kMode == kOutF && p.has_den) dsum[(par * 2 + half) * kT + row] = rs;
                tc_fence_before();
                warp_arrive(&bar[B_PT]);
            }
            if (kMode == kOutE) {
                // outputs, 64 features at a time
                const float fq = fac * qm, zc = p.q_off ? -qo : 1.0f;
                for (int s = 0; s < ns; ++s) {
                    const int v = i * ns + s, ob = v & 1;
                    wait_k(B_OF + ob, v >> 1);
                    tc_fence_after();
                    uint32_t a[32], e[32];
                    const uint32_t oc = trow + (ob ? kColP : kColO) + 32 * half;
                    tmem_ld32(oc, a);
                    tmem_ld32(oc + 64, e);
                    tmem_wait_ld();
                    reg_fence(a);
                    reg_fence(e);
                    tc_fence_before();
                    warp_arrive(&bar[B_OE + ob]);
                    const int fl = 64 * s + 32 * half;
                    __nv_bfloat16* dst = p.o + grow * p.F + f0 + fl;
                    const float4* z4 = reinterpret_cast<const float4*>(zf + par * kMaxFw + fl);
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        float t[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k) t[k] = __uint_as_float(e[8 * c + k]);
                        if (p.has_z) {
                            const float4 z0 = z4[2 * c], z1 = z4[2 * c + 1];
                            t[0] = fmaf(zc, z0.x, t[0]); t[1] = fmaf(zc, z0.y, t[1]);
                            t[2] = fmaf(zc, z0.z, t[2]); t[3] = fmaf(zc, z0.w, t[3]);
                            t[4] = fmaf(zc, z1.x, t[4]); t[5] = fmaf(zc, z1.y, t[5]);
                            t[6] = fmaf(zc, z1.z, t[6]); t[7] = fmaf(zc, z1.w, t[7]);
                        }
#pragma unroll
                        for (int k = 0; k < 8; ++k) t[k] = fmaf(fq, t[k], __uint_as_float(a[8 * c + k]));
                        if (valid && fl + 8 * c < fv)
                            *reinterpret_cast<uint4*>(dst + 8 * c) = make_uint4(pack_bf16(t[0], t[1]), pack_bf16(t[2], t[3]),
                                                                                pack_bf16(t[4], t[5]), pack_bf16(t[6], t[7]));
                    }
                }
            }
            // the state that leaves the chunk
            wait_k(B_TF, i);
            tc_fence_after();
            const float lam = decay_pow(g2, n);
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                if (2 * b >= ns) break;
                uint32_t t[32], z0 = 0, z1 = 0, z2 = 0;
                tmem_ld32(trow + kColT + kTStride * b + 32 * half, t);
                if (p.has_z && b == half) {
                    tmem_ld1(trow + kColT + kTStride * b + 64, z0);
                    tmem_ld1(trow + kColT + kTStride * b + 65, z1);
                    tmem_ld1(trow + kColT + kTStride * b + 66, z2);
                }
                tmem_wait_ld();
                reg_fence(t);
                reg_fence1(z0);
                reg_fence1(z1);
                reg_fence1(z2);
#pragma unroll
                for (int c = 0; c < 32; ++c) run[b][c] = fmaf(lam, run[b][c], __uint_as_float(t[c]));
                if (p.has_z && b == half)
                    zrun = fmaf(lam, zrun, __uint_as_float(z0) + (__uint_as_float(z1) + __uint_as_float(z2)));
            }
            tc_fence_before();
            if (i + 1 < count) {
                if (kMode != kState) write_m(i + 1);
                warp_arrive(&bar[B_MF]);
                write_y(i + 1);
            }
            if (kMode != kState) named_bar_sync(1, 256);
            if (kMode == kOutF) {
                wait_k(B_OF, i);
                tc_fence_after();
                uint32_t a[32], e[32], d0 = 0, d1 = 0, d2 = 0;
                tmem_ld32(trow + kColO + 32 * half, a);
                tmem_ld32(trow + kColO + 64 + 32 * half, e);
                if (p.has_den) {
                    tmem_ld1(trow + kColO + 128, d0);
                    tmem_ld1(trow + kColO + 129, d1);
                    tmem_ld1(trow + kColO + 130, d2);
                }
                tmem_wait_ld();
                reg_fence(a);
                reg_fence(e);
                reg_fence1(d0);
                reg_fence1(d1);
                reg_fence1(d2);
                tc_fence_before();
                warp_arrive(&bar[B_OE]);
                if (valid) {
                    float t[32], dn = 0.0f;
#pragma unroll
                    for (int c = 0; c < 32; ++c) t[c] = fmaf(fac, __uint_as_float(e[c]), __uint_as_float(a[c]));
                    if (p.has_den)
                        dn = fmaf(fac, __uint_as_float(d0) + (__uint_as_float(d1) + __uint_as_float(d2)),
                                  dsum[par * 2 * kT + row] + dsum[(par * 2 + 1) * kT + row]);
                    if (p.part_mode) {
                        float4* pp = reinterpret_cast<float4*>(p.part + grow * 64 + 32 * half);
                        if (p.part_mode == 1) {
#pragma unroll
                            for (int c = 0; c < 8; ++c) pp[c] = make_float4(t[4 * c], t[4 * c + 1], t[4 * c + 2], t[4 * c + 3]);
                            if (half == 0) p.part_den[grow] = dn;
                        } else {
#pragma unroll
                            for (int c = 0; c < 8; ++c) {
                                const float4 w = pp[c];
                                t[4 * c] += w.x;
                                t[4 * c + 1] += w.y;
                                t[4 * c + 2] += w.z;
                                t[4 * c + 3] += w.w;
                            }
                            dn += p.part_den[grow];
                        }
                    }
                    if (p.part_mode != 1) {
                        if (p.has_den) {
                            if (p.den && half == 0) p.den[grow] = dn;
                            const float rd = 1.0f / (dn + p.eps);
#pragma unroll
                            for (int c = 0; c < 32; ++c) t[c] *= rd;
                        }
                        uint4* dst = reinterpret_cast<uint4*>(p.o + grow * 64 + 32 * half);
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            dst[c] = make_uint4(pack_bf16(t[8 * c], t[8 * c + 1]), pack_bf16(t[8 * c + 2], t[8 * c + 3]),
                                                pack_bf16(t[8 * c + 4], t[8 * c + 5]), pack_bf16(t[8 * c + 6], t[8 * c + 7]));
                    }
                }
            }
        }
        if (p.last) {
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const int f = 128 * b + row;
                if (f >= fv) continue;
                float4* dst = reinterpret_cast<float4*>(p.last + ((sidx * p.F) + f0 + f) * 64 + 32 * half);
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    dst[c] = make_float4(run[b][4 * c], run[b][4 * c + 1], run[b][4 * c + 2], run[b][4 * c + 3]);
                if (b == half && p.has_z && p.last_z) p.last_z[sidx * p.F + f0 + f] = zrun;
            }
        }
    }
    wt.report(p.err);
    drain_after_failure(wt.ok);
    tc_fence_before();
    __syncthreads();
    if (warp == 0) tmem_dealloc(tmem, 512);
}

// Segment sums -> the states entering the segments, in place, S and z in one launch; first
// and last as in k_dec_scan.  grid (ceil(F * 65 / 256), BH)
__global__ void __launch_bounds__(256) k_dec_seg_scan(float* st, float* sz, const float* first, const float* first_z,
                                                      float* last, float* last_z, int F, int nseg, int rev,
                                                      const float* log_decay, const int32_t* lengths, int H, int L)
{
    const int64_t bh = blockIdx.y;
    int x = blockIdx.x * 256 + threadIdx.x;
    int64_t w = static_cast<int64_t>(F) * 64;
    if (x >= w) {
        if (!sz || x >= w + F) return;
        x -= static_cast<int>(w);
        w = F;
        st = sz;
        first = first_z;
        last = last_z;
    }
    const int len = lengths ? min(max(lengths[bh / H], 0), L) : L;
    const int nch = (len + kT - 1) / kT;
    const float g2 = log_decay[bh % H] * kLog2e;
    float run = first ? first[bh * w + x] : 0.0f;
    float* q = st + bh * nseg * w + x;
#pragma unroll 4
    for (int i = 0; i < nseg; ++i) {
        const int s = rev ? nseg - 1 - i : i;
        const int lo = static_cast<int>(static_cast<int64_t>(s) * nch / nseg) * kT;
        const int hi = min(static_cast<int>(static_cast<int64_t>(s + 1) * nch / nseg) * kT, len);
        const float t = q[s * w];
        q[s * w] = run;
        run = fmaf(decay_pow(g2, max(hi - lo, 0)), run, t);
    }
    if (last) last[bh * w + x] = run;
}

// [BH][L][cols] bf16 as a 3-D tensor, boxes of 64 columns x 128 tokens, 128-byte swizzle;
// columns past `cols` and rows past L read as zero.
bool map_rows(CUtensorMap* m, const void* base, int cols, int L, int64_t BH)
{
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(L), static_cast<cuuint64_t>(BH)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(cols) * 2, static_cast<cuuint64_t>(L) * cols * 2};
    const cuuint32_t box[3] = {64, kT, 1};
    const cuuint32_t es[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// How a call is cut: feature blocks of at most 256, and segments of the sequence.
struct Plan {
    int nfb, fw, nseg;
    int64_t BH;
};

Plan plan(const DecayArgs& a)
{
    Plan c{};
    c.BH = static_cast<int64_t>(a.B) * a.H;
    c.nfb = (a.F + kMaxFw - 1) / kMaxFw;
    c.fw = ((a.F + c.nfb - 1) / c.nfb + 63) & ~63;
    const int nch = (a.L + kT - 1) / kT;
    c.nseg = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(kNumSMs / c.BH, nch)));
    return c;
}

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

struct Carve {
    float *st, *sz, *part, *part_den, *rz, *r;
    size_t bytes;
};

Carve carve(const DecayArgs& a, const Plan& c, bool bwd, void* ws)
{
    char* base = static_cast<char*>(ws);
    size_t o = 0;
    auto take = [&](size_t floats) {
        float* q = reinterpret_cast<float*>(base + o);
        o += align256(floats * 4);
        return q;
    };
    Carve k{};
    const size_t rows = static_cast<size_t>(c.BH) * a.L;
    if (c.nseg > 1) {
        k.st = take(static_cast<size_t>(c.BH) * c.nseg * a.F * 64);
        k.sz = take(static_cast<size_t>(c.BH) * c.nseg * a.F);
    }
    if (c.nfb > 1) {
        k.part = take(rows * 64);
        k.part_den = take(rows);
    }
    if (bwd) {
        k.rz = take(rows);
        k.r = take(rows);
    }
    k.bytes = o;
    return k;
}

template <int kMode>
cudaError_t launch(const char* name, const CUtensorMap& fs, const CUtensorMap& fq, const CUtensorMap& es,
                   const CUtensorMap& eq, const P& p, const Plan& c, cudaStream_t st)
{
    constexpr size_t smem = layout(kMode).total + 1024;
    static_assert(smem <= 232448, "shared memory of one CTA");
    const cudaError_t e = cudaFuncSetAttribute(k_tc_dec<kMode>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    const int64_t grid = c.BH * p.nseg * (kMode == kOutF ? 1 : p.nfb);
    TraceScope trace_(name, st);
    k_tc_dec<kMode><<<static_cast<unsigned>(grid), kThreads, smem, st>>>(fs, fq, es, eq, p);
    return cudaGetLastError();
}

P base(const DecayArgs& a, const Plan& c, int* err)
{
    P p{};
    p.log_decay = a.log_decay;
    p.lengths = a.lengths;
    p.H = a.H;
    p.L = a.L;
    p.F = a.F;
    p.nseg = c.nseg;
    p.nfb = c.nfb;
    p.fw = c.fw;
    p.has_z = a.norm;
    p.eps = a.eps;
    p.err = err;
    return p;
}

// The states entering each segment: from `first` through the segments' own sums; leaves p
// ready for the output sweeps (the last state written here, or by the sweep that `p.last`
// is left for when there is one segment).
cudaError_t segment_states(const DecayArgs& a, const Plan& c, const Carve& k, P& p, const CUtensorMap& fs,
                           const CUtensorMap& es, const float* first, const float* first_z, float* last,
                           float* last_z, cudaStream_t st)
{
    p.first = first;
    p.first_z = first_z;
    if (c.nseg == 1) return cudaSuccess;
    P q = p;
    q.first = q.first_z = nullptr;
    q.last = k.st;
    q.last_z = k.sz;
    cudaError_t e = launch<kState>("tc_decay_state", fs, fs, es, es, q, c, st);
    if (e != cudaSuccess) return e;
    TraceScope trace_("decay_seg_scan", st);
    k_dec_seg_scan<<<dim3((a.F * 65 + 255) / 256, static_cast<unsigned>(c.BH)), 256, 0, st>>>(
        k.st, a.norm ? k.sz : nullptr, first, first_z, last, last_z, a.F, c.nseg, p.rev, a.log_decay, a.lengths, a.H, a.L);
    p.first = k.st;
    p.first_z = k.sz;
    return cudaGetLastError();
}

// A sweep whose queries are on the F side: one launch per feature block, the blocks'
// numerators and denominators added in fp32.
cudaError_t out_f(const CUtensorMap& fs, const CUtensorMap& fq, const CUtensorMap& es, P p, const Plan& c,
                  const Carve& k, cudaStream_t st)
{
    p.part = k.part;
    p.part_den = k.part_den;
    for (int fb = 0; fb < c.nfb; ++fb) {
        p.fb0 = fb;
        p.part_mode = c.nfb == 1 ? 0 : fb == 0 ? 1 : 2;
        const cudaError_t e = launch<kOutF>("tc_decay_out_f", fs, fq, es, es, p, c, st);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace

bool decay_tc_supported(const DecayArgs& a)
{
    return a.dt == SLAY_BF16 && a.L > 0 && a.F % 8 == 0 && a.F <= 2 * kMaxFw;
}

size_t decay_tc_ws(const DecayArgs& a, bool bwd) { return carve(a, plan(a), bwd, nullptr).bytes; }

cudaError_t decay_tc_fwd(const DecayArgs& a, void* ws, int* err, cudaStream_t st)
{
    const Plan c = plan(a);
    const Carve k = carve(a, c, false, ws);
    CUtensorMap mq, mk, mv;
    if (!map_rows(&mq, a.phq, a.F, a.L, c.BH) || !map_rows(&mk, a.phk, a.F, a.L, c.BH) || !map_rows(&mv, a.v, 64, a.L, c.BH))
        return cudaErrorInvalidValue;
    P p = base(a, c, err);
    cudaError_t e = segment_states(a, c, k, p, mk, mv, a.S_in, a.z_in, a.S_out, a.z_out, st);
    if (e != cudaSuccess) return e;
    if (c.nseg == 1) {
        p.last = a.S_out;
        p.last_z = a.z_out;
    }
    p.has_den = a.norm;
    p.o = static_cast<__nv_bfloat16*>(a.out_w);
    p.den = a.den_w;
    return out_f(mk, mq, mv, p, c, k, st);
}

cudaError_t decay_tc_bwd(const DecayArgs& a, void* ws, int* err, cudaStream_t st)
{
    const Plan c = plan(a);
    const Carve k = carve(a, c, true, ws);
    CUtensorMap mq, mk, mv, mo;
    if (!map_rows(&mq, a.phq, a.F, a.L, c.BH) || !map_rows(&mk, a.phk, a.F, a.L, c.BH) ||
        !map_rows(&mv, a.v, 64, a.L, c.BH) || !map_rows(&mo, a.dout, 64, a.L, c.BH))
        return cudaErrorInvalidValue;
    cudaError_t e = a.norm ? decay_row_stats(a, k.rz, k.r, st) : cudaSuccess;
    if (e != cudaSuccess) return e;
    const float *rz = a.norm ? k.rz : nullptr, *r = a.norm ? k.r : nullptr;
    P s = base(a, c, err);   // dphq from the states before each token
    if ((e = segment_states(a, c, k, s, mk, mv, a.S_in, a.z_in, nullptr, nullptr, st)) != cudaSuccess) return e;
    s.q_mul = rz;
    s.q_off = r;
    s.o = static_cast<__nv_bfloat16*>(a.dphq);
    if ((e = launch<kOutE>("tc_decay_out_e", mk, mk, mv, mo, s, c, st)) != cudaSuccess) return e;
    P g = base(a, c, err);   // dphk and dv from the states after each token
    g.rev = 1;
    g.s_mul = rz;
    g.s_off = r;
    g.z_delta = a.norm;
    if ((e = segment_states(a, c, k, g, mq, mo, a.dS_out, a.dz_out, a.dS_in, a.dz_in, st)) != cudaSuccess) return e;
    g.o = static_cast<__nv_bfloat16*>(a.dphk);
    if ((e = launch<kOutE>("tc_decay_out_e", mq, mq, mo, mv, g, c, st)) != cudaSuccess) return e;
    if (c.nseg == 1) {       // (the sweep that writes over dS_out when dS_in is dS_out: the last one)
        g.last = a.dS_in;
        g.last_z = a.dz_in;
    }
    g.o = static_cast<__nv_bfloat16*>(a.dv);
    return out_f(mq, mk, mo, g, c, k, st);
}

}  // namespace slay
