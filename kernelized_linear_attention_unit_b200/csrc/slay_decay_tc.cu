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
// each, so an output sees two besides its own (the normalized dphq takes both in two limbs);
// the decay weight of a token's state term is folded into the 64-wide side as w_j u_j = hi +
// mid + lo, three bf16 limbs, where the fp32 state leaves the call, so that it is as exact as an
// fp32 sum (one limb alone would be off by up to 2^-8), and two (2^-16) where only its bf16 copy is
// read.  The z column (the ones column of u) takes its weights as three bf16 columns of a
// 16-wide operand, and so does the denominator's state part; the denominator's other part is
// summed in fp32 from the scores.
//
// Bounds.  HBM's floor is 2 (2 F + 128) bytes per token and head forward, 2 (4 F + 256)
// backward; a 128-token chunk at F = 256 is 164 KB, 7000 clocks at an SM's share of the
// bandwidth.  The MMAs read their operands from shared memory (M = 128, K = 16: 4 KB of A and
// 2 KB of B per 64 columns, 128 bytes a clock), 4000 of them for the 88 MMAs of a forward
// chunk, which is why accumulators are as wide as tensor memory allows; P~ is read from tensor
// memory.  The chain of a chunk (scores, masking, state sum, its bf16 copy, the next scores)
// takes 8000 to 9000 clocks: forward B32 H12 L1024 F256 in 106 us, 4.8 TB/s, 73% of the copy
// bandwidth (tensor pipe 32% active); with fewer (b, h) than SMs the sequence is cut into segments, whose sums
// (k_tc_dec<kState>) read the F side once more, at 54% of the DRAM peak (B1 H16 L16384 F256).  Measured alternatives: 512 threads with four
// state warps in kOutF, too, 121 against 104 us; MMA loops not unrolled 126 us; roles chosen at
// run time 162 us (the code outgrew the instruction cache).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
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
constexpr int kNumSMs = 148;
constexpr int kMaxFw = 256;           // features of one sweep

enum Mode { kState = 0, kOutF = 1, kOutE = 2 };

// Warps: 0 issues the MMAs, 1 the TMA loads (2 the query slices'); 4 on are the epilogue.  kOutE, whose
// outputs are F wide, gives the state four warps of its own beside eight for scores and
// outputs; elsewhere eight do both (and hold half as much of the state each).
__host__ __device__ constexpr bool split(int mode) { return mode == kOutE; }
__host__ __device__ constexpr int threads(int mode) { return 32 * (split(mode) ? 16 : 12); }

// tensor memory columns.  P~ replaces the scores' first 64 columns; an output accumulator
// takes the other 64.  T of 128 features: the first limb's 64 columns, in the modes with
// room a second limb's (kState: a third's), and 16 for z.
constexpr uint32_t kColP = 0, kColOi = 64, kColDen = 128, kColOe = 144;   // (the scores' product is 144 wide with kColDen)
// kOutE: two output buffers; the one-limb form puts the second one's Oi over the scores, the
// two-limb form (128 features) has room beside them
__host__ __device__ constexpr uint32_t col_oi(bool limbs, int b) { return limbs ? 128 + 128 * b : b ? 64 : 128; }
__host__ __device__ constexpr uint32_t col_oe(bool limbs, int b) { return limbs ? 192 + 128 * b : b ? 256 : 192; }
__host__ __device__ constexpr uint32_t col_t(int mode, bool limbs) { return limbs ? 384 : mode == kOutE ? 352 : mode == kOutF ? 208 : 0; }
__host__ __device__ constexpr uint32_t col_z(int mode) { return mode == kOutE ? 64 : mode == kOutF ? 128 : 192; }
__host__ __device__ constexpr uint32_t t_stride(int mode) { return mode == kOutE ? 80 : mode == kOutF ? 144 : 208; }
__host__ __device__ constexpr int limb_tiles(int mode) { return mode == kState ? 8 : mode == kOutE ? 2 : 3; }

enum {
    B_FSF = 0, B_FSE = 4, B_FQF = 8, B_ESF = 12, B_ESE = 14, B_YF = 16, B_MF = 18, B_PF = 20, B_PT, B_OD,
    B_TF = 23, B_OF = 25, B_OE = 27, B_FQE = 29, B_NUM = 33
};

// An F-side slice in the ring; in kOutF, behind its 128 rows, 16 of the z column's limbs (three
// used): the scores' product carries the denominator's state part along.
__host__ __device__ constexpr uint32_t slot(int mode) { return kTile + (mode == kOutF ? kExt : 0); }

struct Layout {
    uint32_t fs, fq, es, eq, y, m, wext, stg, pw, smul, soff, dsum, zf, bar, tmem, total;
};

__host__ __device__ constexpr Layout layout(int mode)
{
    Layout l{};
    uint32_t o = 0;
    l.fs = o; o += 4 * slot(mode);                      // ring of four F-side slices
    l.fq = o; o += mode == kOutF ? 3 * kTile : 0;       // ring of query slices: four, or three and
    l.y = o; o += limb_tiles(mode) * kTile;             // the third of the weighted rows' limbs in that tile
    l.es = o; o += (mode == kOutF ? 1 : 2) * kTile;     // 64-wide side, two chunks (kOutF: one)
    l.eq = o; o += mode == kOutE ? 2 * kTile : 0;       // 64-wide queries, two chunks
    l.m = o; o += mode == kState ? 0 : 4 * kSlab;       // the state as an operand
    l.wext = o; o += mode == kState ? 0 : 2 * kExt;     // z weights of the chunk's tokens (kState: a fourth tile)
    l.stg = o; o += mode == kOutE ? 8 * 32 * 64 : 0;    // outputs on their way to the TMA store, 2 KiB a warp
    l.pw = o; o += 128 * 4;                             // lambda^d
    l.smul = o; o += mode == kState ? 0 : 2 * 128 * 4;  // score scalars of the state tokens
    l.soff = o; o += mode == kState ? 0 : 2 * 128 * 4;
    l.dsum = o; o += mode == kOutF ? 2 * 2 * 128 * 4 : 0;   // row sums of the scores, by column half
    l.zf = o; o += mode == kOutE ? 2 * kMaxFw * 4 : 0;  // z in fp32, two chunks
    l.bar = o; o += B_NUM * 8;
    l.tmem = o; o += 16;
    l.total = o;
    return l;
}

// The segments' sums and starting states, private to a call: per (b, h, segment) the float4s
// [128 features][16 of a row][128 rows], in the order in which a warp reads and writes them.
__host__ __device__ __forceinline__ int64_t sums_floats(int F) { return static_cast<int64_t>((F + 127) / 128) * 128 * 64; }
__device__ __forceinline__ int64_t sums_at(int f, int e4)   // in float4s
{
    return (static_cast<int64_t>(f >> 7) * 16 + e4) * 128 + (f & 127);
}

struct P {
    const float* log_decay;
    const int32_t* lengths;
    const float *s_mul, *s_off, *q_mul, *q_off;   // row scalars, null: 1 / 0
    const float *first, *first_z;                 // states entering the walk [BH], null: zero
    const float *sums, *sums_z;                   // the segments' own sums [BH][nseg]: a sweep adds up those
                                                  // before its segment; null: one segment, or
    const float *starts, *starts_z;               // the states entering the segments [BH][nseg]
    float *last, *last_z;                         // states leaving: the walk [BH]; kState: the sums [BH][nseg]
    __nv_bfloat16* o;
    float* den;
    float *part, *part_den;                       // numerators and denominators over features, by chunk
    int part_mode;                                // 0: none, 1: store them, 2: add them to this block's
    float eps;
    int H, L, F, nseg, nfb, fw, fb0;
    int seg0, nsl;                                // segments of this launch: seg0 .. seg0 + nsl - 1
    int z_state;                                  // keep z (kOutF backward: only where it is wanted)
    // kState in pairs: the direction, and a second walk of the same launch, from CTA n0 on (its
    // operands are the maps tfq and teq)
    int rev, n0;
    struct Walk {
        const float *s_mul, *s_off;
        float *last, *last_z;
        int rev, nseg, seg0, nsl;
    } second;
    int* err;
    int withhold;                                 // test hook, 0 in every normal call: see slay_debug_expire_wait
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

__device__ __forceinline__ float2 fadd2(float2 a, float2 b) { return ffma2(a, make_float2(1.0f, 1.0f), b); }

__device__ __forceinline__ void st_shared_u16(uint32_t addr, uint16_t x)
{
    asm volatile("st.shared.u16 [%0], %1;" ::"r"(addr), "h"(x) : "memory");
}

// A wait on the completion of `phase`, bounded in time (kWaitNs; the low word of the clock turns
// over after 4.3 s).  The clock is read only once a first try, which suspends the thread for a
// while, has come back empty; after a wait that ran out, each further one is a single try.
struct Bounded {
    bool ok = true;
    uint32_t where = 0;
    __device__ __forceinline__ void wait(uint64_t* bar, uint32_t phase)
    {
        const uint32_t addr = smem_u32(bar);
        if (mbar_try_wait(addr, phase)) return;
        if (ok) {
            const uint32_t t0 = clock_ns();
            do {
                if (mbar_try_wait(addr, phase)) return;
            } while (clock_ns() - t0 <= static_cast<uint32_t>(kWaitNs));
            where = 0x10000u | (addr & 0xFFFFu);
        }
        ok = false;
    }
    static __device__ __forceinline__ uint32_t clock_ns()
    {
        uint32_t t;
        asm volatile("mov.u32 %0, %%globaltimer_lo;" : "=r"(t));
        return t;
    }
    __device__ __forceinline__ void report(int* status) const
    {
        if (!ok) atomicCAS(status, 0, static_cast<int>(where));
    }
};

// One lane of a converged warp; the compiler knows that a single thread runs what it guards.
__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

// kRev: the sweep walks the chunks backward (kPair: as each of the two walks says).  kNorm: the normalized form, whose backward puts
// its row scalars on the state tokens (kRev) or on the query tokens (kOutE forward).
template <int kMode, bool kRev, bool kNorm, bool kPair = false, bool kIdle = false>
__device__ __forceinline__ void sweep(const CUtensorMap& tfs, const CUtensorMap& tfq, const CUtensorMap& tes,
                                      const CUtensorMap& teq, const CUtensorMap& tout, const P& p, int block)
{
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);   // (stays a shared address)
    constexpr bool kSplit = split(kMode);
    constexpr int kThreads = threads(kMode), kEs = kMode == kOutF ? 1 : 2;
    constexpr bool kCols = kRev && kNorm, kRows = kMode == kOutE && !kRev && kNorm, kDen = kMode == kOutF && !kRev && kNorm;
    // The normalized dphq is a difference (c_ij has no weighted mean over j) that loses a bit or
    // two: its scores and its copy of the state go in as two bf16 limbs, over half as many
    // features a CTA (one limb: 3.1e-3 off in relative L2, two: 1.7e-3, bf16's own rounding).
    constexpr bool kLimb = kRows;
    constexpr Layout Lo = layout(kMode);
    constexpr uint32_t kSlot = slot(kMode);
    uint64_t* bar = reinterpret_cast<uint64_t*>(sm + Lo.bar);
    uint32_t* tslot = reinterpret_cast<uint32_t*>(sm + Lo.tmem);
    const uint32_t sbase = smem_u32(sm);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    // this CTA's feature block, segment and sequence
    int x = block;
    const bool second = kPair && x >= p.n0;
    if (second) x -= p.n0;
    const bool rev = kPair ? (second ? p.second.rev : p.rev) != 0 : kRev;
    const int nseg = second ? p.second.nseg : p.nseg, nsl = second ? p.second.nsl : p.nsl;
    const int fb = kMode == kOutF ? p.fb0 : x % p.nfb;
    if (kMode != kOutF) x /= p.nfb;
    const int seg = (second ? p.second.seg0 : p.seg0) + x % nsl, bh = x / nsl;
    const int f0 = fb * p.fw, fv = min(p.fw, p.F - f0);
    const int ns = (fv + 63) >> 6, nsE = (ns + 1) & ~1;   // 64-feature slices; as whole pairs
    const int len = p.lengths ? min(max(p.lengths[bh / p.H], 0), p.L) : p.L;
    const int nch = (len + kT - 1) / kT;
    auto seg_lo = [&](int s) { return s * nch / nseg; };   // (at most 32768 chunks, 148 segments)
    const int c_lo = seg_lo(seg), count = seg_lo(seg + 1) - c_lo;
    // whether the state that leaves this CTA's walk is an output
    const bool leaves = p.last && (kMode == kState || seg == (kRev ? 0 : nseg - 1));
    auto chunk_of = [&](int i) { return rev ? c_lo + count - 1 - i : c_lo + i; };
    const float g2 = p.log_decay[bh % p.H] * kLog2e;
    // limbs of the weighted rows: three where the fp32 state leaves the call, two (2^-16) where
    // only its bf16 copy is read; without decay and row scalars the weights are 1, one is exact
    const bool has_z = kNorm && (kMode != kOutF || !kRev || p.z_state);
    const int nl = kMode == kState ? 3 : g2 == 0.0f && !kCols ? 1 : kMode == kOutF && leaves ? 3 : 2;

    // kOutF: limb tiles 0, 1 at y + 16 KiB, 2 at y, which is the query ring's fourth slot otherwise
    const int nfq = nl == 3 ? 3 : 4;
    constexpr uint32_t kY = kMode == kOutF ? Lo.y + kTile : Lo.y;
    if (warp == 0) {
        tmem_alloc(tslot, 512);
        tmem_relinquish();
    }
    for (uint32_t i = Lo.wext / 4 + tid; i < Lo.stg / 4; i += kThreads) reinterpret_cast<uint32_t*>(sm)[i] = 0u;
    if (kMode == kState)   // the z weights' 16 columns, of which three are used
        for (int i = tid; i < 2 * kT; i += kThreads) {
            const uint32_t t = sbase + Lo.y + ((i >> 7) * 4 + 3) * kTile;
            st_shared_v4(t + sw128_off(i & 127, 0), 0u, 0u, 0u, 0u);
            st_shared_v4(t + sw128_off(i & 127, 1), 0u, 0u, 0u, 0u);
        }
    if (kDen)
        for (int i = tid; i < kExt; i += kThreads)
            reinterpret_cast<uint32_t*>(sm + Lo.fs + (i >> 9) * kSlot + kTile)[i & 511] = 0u;
    // lambda powers: within a diagonal block of scores, at 31 + distance (zero where it is masked),
    // then the column factors of a block inside the mask
    if (tid < 64) reinterpret_cast<float*>(sm + Lo.pw)[tid] = tid >= 31 && tid < 63 ? decay_pow(g2, tid - 31) : 0.0f;
    if (tid < 32) reinterpret_cast<float*>(sm + Lo.pw)[64 + tid] = decay_pow(g2, kRev ? tid : 31 - tid);
    if (tid == 0) {
        for (int i = 0; i < B_NUM; ++i)
            mbar_init(&bar[i], i >= B_YF && i < B_YF + 4 ? (kSplit ? 4 : 8) : i == B_PT || i == B_OE || i == B_OE + 1 ? 8 : 1);
        mbar_fence_init();
        tma_prefetch_desc(second ? &tfq : &tfs);
        tma_prefetch_desc(second ? &teq : &tes);
        if (kMode == kOutF) tma_prefetch_desc(&tfq);
        if (kMode == kOutE) tma_prefetch_desc(&teq);
    }
    fence_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    after_previous_kernel();
    constexpr uint32_t tmem = 0;   // all 512 columns are this CTA's
    Bounded wt;
    if (*tslot != tmem) {
        wt.ok = false;
        wt.where = 0x20000u;
    }
    // waits on the k-th completion (k >= 0) of a barrier
    auto wait_k = [&](int b, int k) { wt.wait(&bar[b], static_cast<uint32_t>(k & 1)); };

    // Registers: the loading warpgroup gives some of its share to the warps that hold the
    // state.  384 threads launch with 168 each: 88 + 2 x 208 = 3 x 168; 512 with 128:
    // 96 + 192 + 2 x 112 = 4 x 128 (64 + 192 + 2 x 128 spilled in the loading warps: dphk of
    // B2 H16 L8192 F512 174 against 162 us), or, with half the state and two limbs of scores,
    // 64 + 128 + 2 x 160.  A fourth warpgroup that does nothing (kIdle): 24 + 88 + 2 x 200.
    if (warp < 4) {
        regs_dec<kLimb ? 64 : kSplit ? 96 : 88>();
        if (warp == 1 && lane == 0) {
            // -------------------------------------------------------------- TMA loads
            // (under the test hook the first CTA loads nothing)
            for (int i = p.withhold && block == 0 ? count : 0; i < count && wt.ok; ++i) {
                const int t0 = chunk_of(i) * kT, b = i % kEs;
                auto load_e = [&] {   // the 64-wide rows
                    if (i >= kEs) wait_k(B_ESE + b, i / kEs - 1);
                    mbar_arrive_expect_tx(&bar[B_ESF + b], kMode == kOutE ? 2 * kTile : kTile);
                    tma_load_3d(sm + Lo.es + b * kTile, second ? &teq : &tes, &bar[B_ESF + b], 0, t0, bh);
                    if (kMode == kOutE) tma_load_3d(sm + Lo.eq + b * kTile, &teq, &bar[B_ESF + b], 0, t0, bh);
                };
                if (kMode != kOutF || i == 0) load_e();
                for (int s = 0; s < nsE; ++s) {
                    const int u = i * nsE + s, sl = u & 3;
                    if (u >= 4) wait_k(B_FSE + sl, (u >> 2) - 1);
                    if (s < ns) {
                        mbar_arrive_expect_tx(&bar[B_FSF + sl], kTile);
                        tma_load_3d(sm + Lo.fs + sl * kSlot, second ? &tfq : &tfs, &bar[B_FSF + sl], f0 + 64 * s, t0, bh);
                    } else {
                        mbar_arrive(&bar[B_FSF + sl]);   // the second half of the last pair: not read
                    }
                }
                if (kMode == kOutF && i > 0) load_e();   // its one buffer is freed after the slices'
            }
        } else if (kMode == kOutF && warp == 2 && lane == 0) {
            int fq = 0, fqr = 0;   // query slot, its use
            for (int i = 0; i < count && wt.ok; ++i) {
                for (int s = 0; s < ns; ++s) {
                    if (fqr >= 1) wait_k(B_FQE + fq, fqr - 1);
                    mbar_arrive_expect_tx(&bar[B_FQF + fq], kTile);
                    tma_load_3d(sm + Lo.fq + fq * kTile, &tfq, &bar[B_FQF + fq], f0 + 64 * s, chunk_of(i) * kT, bh);
                    if (++fq == nfq) {
                        fq = 0;
                        ++fqr;
                    }
                }
            }
        } else if (warp == 0) {
            // -------------------------------------------------------------- MMA issue
            constexpr uint32_t idP = idesc_bf16(128, 128, 0, 0);
            constexpr uint32_t idKM = idesc_bf16(128, 64, 0, 1);    // A K-major (or tensor memory), B MN-major
            constexpr uint32_t idKK = idesc_bf16(128, 64, 0, 0);
            constexpr uint32_t idMM = idesc_bf16(128, 64, 1, 1);
            constexpr uint32_t idMM2 = idesc_bf16(128, 128, 1, 1);
            constexpr uint32_t idMz = idesc_bf16(128, 16, 1, 0);
            constexpr uint32_t idPz = idesc_bf16(128, 144, 0, 0);
            constexpr uint32_t kLd = kSlot >> 4, kTd = kTile >> 4, kSd = kSlab >> 4, kEd = kExt >> 4;
            const uint64_t d0 = sdesc(sbase, 16, 1024, kLayoutSW128);
            const uint64_t dT = sdesc(sbase, kTile, 1024, kLayoutSW128);   // the next 64 rows or columns one tile on,
            const uint64_t dF = sdesc(sbase, kSlot, 1024, kLayoutSW128);   // or one ring slot on
            constexpr uint32_t oFs = Lo.fs >> 4, oFq = Lo.fq >> 4, oEs = Lo.es >> 4, oEq = Lo.eq >> 4, oY = kY >> 4,
                               oM = Lo.m >> 4, oWe = Lo.wext >> 4;
            auto wait_m = [&](int b, int k) {
                wait_k(b, k);
                tc_fence_after();
            };
            int fq = 0, fqr = 0;   // query slot, its use
            for (int i = 0; i < count; ++i) {
                if (!__all_sync(0xffffffffu, wt.ok)) break;   // the warp leaves as one: elect_one needs all of it
                const int t0 = chunk_of(i) * kT, n = min(kT, len - t0), eb = i % kEs;
                // rows of the tensor behind this sequence may hold anything: cleared in the
                // tiles, since they enter sums over tokens (rows past L arrive as zero)
                const bool clear = n < kT && t0 + n < p.L;
                auto clear_rows = [&](uint32_t tile) {
                    for (int a = n * 8 + lane; a < kT * 8; a += 32) st_shared_v4(sbase + tile + a * 16, 0u, 0u, 0u, 0u);
                    fence_async_smem();
                    __syncwarp();
                };
                auto slice = [&](int s) {   // F-side slice s of the chunk, complete and clean
                    const int u = i * nsE + s, sl = u & 3;
                    wait_m(B_FSF + sl, u >> 2);
                    if (clear) clear_rows(Lo.fs + sl * kSlot);
                    return sl;
                };
                auto state_pair = [&](int s) {   // T of the pair of slices s, s + 1
                    const uint64_t da = dF + oFs + ((i * nsE + s) & 3) * kLd;
                    const uint32_t t = tmem + col_t(kMode, kLimb) + t_stride(kMode) * (s >> 1);
                    const uint32_t oy = oY + (kMode == kState ? eb * 4 * kTd : 0);
                    if (kMode == kState) {   // three limbs and the z weights side by side
                        constexpr uint32_t id = idesc_bf16(128, kNorm ? 208 : 192, 1, 1);
#pragma unroll
                        for (int kk = 0; kk < 8; ++kk) umma_bf16(t, da + 128 * kk, dT + oy + 128 * kk, id, kk > 0 ? 1u : 0u);
                        return;
                    }
                    int l = 0;
                    if (kMode != kOutE && nl > 1) {   // two limbs side by side: the F side is read once
#pragma unroll
                        for (int kk = 0; kk < 8; ++kk) umma_bf16(t, da + 128 * kk, dT + oy + 128 * kk, idMM2, kk > 0 ? 1u : 0u);
                        l = 2;
                    }
                    for (; l < nl; ++l)
#pragma unroll
                        for (int kk = 0; kk < 8; ++kk)
                            umma_bf16(t, da + 128 * kk, d0 + (kMode == kOutF && l == 2 ? Lo.y >> 4 : oy + l * kTd) + 128 * kk, idMM, (l > 0 || kk > 0) ? 1u : 0u);
                    if (has_z) {
                        const uint64_t dw = d0 + oWe;
#pragma unroll
                        for (int kk = 0; kk < 8; ++kk)
                            umma_bf16(t + col_z(kMode), da + 128 * kk, dw + (kk >> 2) * kEd + 2 * (kk & 3), idMz, kk > 0 ? 1u : 0u);
                    }
                };
                auto free_pair = [&](int s) {
                    const int sl = (i * nsE + s) & 3;
                    umma_commit(&bar[B_FSE + sl]);
                    umma_commit(&bar[B_FSE + sl + 1]);
                };
                const uint64_t des = d0 + oEs + eb * kTd, deq = d0 + oEq + eb * kTd;
                if (kMode == kOutF) {
                    // the scores and the state's part take the place of the last chunk's outputs
                    if (i >= 1) wait_m(B_OE, i - 1);
                    if (kDen) wait_m(B_MF, i);   // z is behind the slices
                    for (int s = 0; s < ns; ++s) {
                        const int sl = slice(s);
                        wait_m(B_FQF + fq, fqr);
                        const uint64_t dx = d0 + oFq + fq * kTd, dyy = d0 + oFs + sl * kLd;
                        if (elect_one()) {
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk)
                                umma_bf16(tmem + kColP, dx + 2 * kk, dyy + 2 * kk, kDen ? idPz : idP, (s > 0 || kk > 0) ? 1u : 0u);
                            if (s == ns - 1) umma_commit(&bar[B_PF]);
                        }
                        if (!kDen && s == 0) wait_m(B_MF, i);
                        if (elect_one()) {
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk)
                                umma_bf16(tmem + kColOe, dx + 2 * kk, d0 + oM + s * kSd + 128 * kk, idKM,
                                          (s > 0 || kk > 0) ? 1u : 0u);
                            umma_commit(&bar[B_FQE + fq]);
                        }
                        if (++fq == nfq) {
                            fq = 0;
                            ++fqr;
                        }
                    }
                    wait_m(B_YF, i);
                    if (elect_one()) {
                        for (int s = 0; s < ns; s += 2) {
                            state_pair(s);
                            free_pair(s);
                        }
                        umma_commit(&bar[B_TF]);
                    }
                    wait_m(B_PT, i);
                    if (elect_one()) {
#pragma unroll
                        for (int kk = 0; kk < 8; ++kk)
                            umma_bf16_ts(tmem + kColOi, tmem + kColP + 8 * kk, des + 128 * kk, idKM, kk > 0 ? 1u : 0u);
                        umma_commit(&bar[B_OF]);
                        umma_commit(&bar[B_ESE + eb]);
                    }
                } else if (kMode == kOutE) {
                    wait_m(B_ESF + eb, i / kEs);
                    if (clear) clear_rows(Lo.es + eb * kTile);
                    const int v1 = i * ns - 1, vo = (v1 & 1) ? v1 : v1 - 1;   // last use of the buffer over P
                    if (!kLimb && vo >= 1) wait_m(B_OE + 1, vo >> 1);
                    if (elect_one()) {
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            umma_bf16(tmem + kColP, deq + 2 * kk, des + 2 * kk, idP, kk > 0 ? 1u : 0u);
                        umma_commit(&bar[B_PF]);
                    }
                    wait_m(B_YF, i);
                    for (int s = 0; s < ns; s += 2) {   // while the scores are masked
                        slice(s);
                        if (s + 1 < ns) slice(s + 1);
                        if (elect_one()) state_pair(s);
                    }
                    if (elect_one()) umma_commit(&bar[B_TF]);
                    wait_m(B_PT, i);
                    wait_m(B_MF, i);
                    for (int r = 0; r < ns; ++r) {
                        const int v = i * ns + r, ob = v & 1;
                        if (v >= 2) wait_m(B_OE + ob, (v >> 1) - 1);
                        const uint32_t oi = tmem + col_oi(kLimb, ob), oe = tmem + col_oe(kLimb, ob);
                        const uint64_t du = d0 + oFs + ((i * nsE + r) & 3) * kLd;
                        if (elect_one()) {
#pragma unroll
                            for (int kk = 0; kk < 8; ++kk)
                                umma_bf16_ts(oi, tmem + kColP + 8 * kk, du + 128 * kk, idKM, kk > 0 ? 1u : 0u);
                            if (kLimb)
#pragma unroll
                                for (int kk = 0; kk < 8; ++kk)
                                    umma_bf16_ts(oi, tmem + kColP + 64 + 8 * kk, du + 128 * kk, idKM, 1u);
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk)
                                umma_bf16(oe, deq + 2 * kk, d0 + oM + r * kSd + 2 * kk, idKK, kk > 0 ? 1u : 0u);
                            if (kLimb)
#pragma unroll
                                for (int kk = 0; kk < 4; ++kk)
                                    umma_bf16(oe, deq + 2 * kk, d0 + oM + (r + 2) * kSd + 2 * kk, idKK, 1u);
                            umma_commit(&bar[B_OF + ob]);
                            if ((r & 1) || r == ns - 1) free_pair(r & ~1);
                        }
                    }
                    if (elect_one()) {
                        umma_commit(&bar[B_OD]);
                        umma_commit(&bar[B_ESE + eb]);
                    }
                } else {
                    wait_m(B_YF + eb, i >> 1);
                    for (int s = 0; s < ns; s += 2) {   // a pair's T is read while the other's is summed
                        slice(s);
                        if (s + 1 < ns) slice(s + 1);
                        wait_m(B_MF + (s >> 1), i);
                        if (elect_one()) {
                            state_pair(s);
                            free_pair(s);
                            umma_commit(&bar[B_TF + (s >> 1)]);
                        }
                    }
                    if (elect_one()) umma_commit(&bar[B_ESE + eb]);
                }
                __syncwarp();
            }
        }
        __syncwarp();
    } else if (kIdle && warp >= threads(kMode) / 32) {
        regs_dec<24>();
    } else {
        // ------------------------------------------------------------------ epilogue
        // (no early exit on a wait that ran out: the pairs of warps share named barriers)
        const int q = warp & 3, ew = warp - (kSplit ? 8 : 4), half = kSplit && warp < 8 ? 0 : ew >> 2;
        constexpr int kW = kSplit ? 64 : 32;   // columns of M a state thread holds
        const int row = 32 * q + lane;   // token of scores, outputs and weighted rows; feature of T
        const uint32_t trow = tmem + ((32u * q) << 16);
        const float* pw = reinterpret_cast<const float*>(sm + Lo.pw);
        float* smul = reinterpret_cast<float*>(sm + Lo.smul);
        float* soff = reinterpret_cast<float*>(sm + Lo.soff);
        float* dsum = reinterpret_cast<float*>(sm + Lo.dsum);
        float* zf = reinterpret_cast<float*>(sm + Lo.zf);
        const int64_t sidx = static_cast<int64_t>(bh) * nseg + seg;
        // the scalars of four query / state tokens: off the raw scores, onto the weights
        auto scale = [&](int par, int j, float2 off, float2& s0, float2& s1, float2& w0, float2& w1) {
            if (kRows) {
                s0 = fadd2(s0, off);
                s1 = fadd2(s1, off);
            }
            if (kCols) {
                const float4 m = *reinterpret_cast<const float4*>(smul + par * kT + j);
                w0 = fmul2(w0, make_float2(m.x, m.y));
                w1 = fmul2(w1, make_float2(m.z, m.w));
                if (kMode == kOutE) {
                    const float4 o = *reinterpret_cast<const float4*>(soff + par * kT + j);
                    s0 = fadd2(s0, make_float2(-o.x, -o.y));
                    s1 = fadd2(s1, make_float2(-o.z, -o.w));
                }
            }
        };
        // Masked, decayed scores -> P~.  A warp has two 32-column blocks of its 32 rows; a block
        // is wholly inside the mask (lambda^(i-j) as a row times a column factor, both <= 1), on
        // the diagonal, or wholly outside.  Returns the sum over this thread's columns.
        auto scores = [&](int i, float qo, float qm) {
            const int par = i & 1;
            if (kCols) wait_k(B_YF, i);   // smul, soff of this chunk
            wait_k(B_PF, i);
            tc_fence_after();
            float2 rs = make_float2(0.0f, 0.0f);
            uint32_t pk[2][16], pl[2][16];   // P~ in one limb or two
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
                const int cb = half + 2 * hh, j0 = 32 * cb;
                const int side = kRev ? cb - q : q - cb;   // > 0: inside, 0: diagonal
                auto put = [&](int c, float2 x) {
                    const uint32_t l = pack_bf16(x.x, x.y);
                    pk[hh][c / 2] = l;
                    if (kLimb) pl[hh][c / 2] = pack_bf16(x.x - bf_lo(l), x.y - bf_hi(l));
                };
                if (side < 0) {
#pragma unroll
                    for (int c = 0; c < 16; ++c) pk[hh][c] = pl[hh][c] = 0u;
                    continue;
                }
                uint32_t r[32];
                tmem_ld32(trow + kColP + j0, r);
                tmem_wait_ld();
                reg_fence(r);
                // (query rows behind the sequence keep whatever comes out: it reaches their own
                // output rows only, which are not stored)
                const float2 off = make_float2(-qo, -qo);
                if (side > 0) {
                    const float f = qm * decay_pow(g2, kRev ? j0 - row : row - j0 - 31);
                    const float2 rf = make_float2(f, f);
#pragma unroll
                    for (int c = 0; c < 32; c += 4) {
                        const float4 t = *reinterpret_cast<const float4*>(pw + 64 + c);
                        float2 w0 = fmul2(rf, make_float2(t.x, t.y)), w1 = fmul2(rf, make_float2(t.z, t.w));
                        float2 s0 = make_float2(__uint_as_float(r[c]), __uint_as_float(r[c + 1]));
                        float2 s1 = make_float2(__uint_as_float(r[c + 2]), __uint_as_float(r[c + 3]));
                        scale(par, j0 + c, off, s0, s1, w0, w1);
                        if (kDen) {
                            rs = ffma2(s0, w0, rs);
                            rs = ffma2(s1, w1, rs);
                        }
                        put(c, fmul2(s0, w0));
                        put(c + 2, fmul2(s1, w1));
                    }
                } else {
                    const float* pd = pw + 31 + (kRev ? -lane : lane);
                    const float2 rf = make_float2(qm, qm);
#pragma unroll
                    for (int c = 0; c < 32; c += 4) {
                        float2 w0 = make_float2(pd[kRev ? c : -c], pd[kRev ? c + 1 : -c - 1]);
                        float2 w1 = make_float2(pd[kRev ? c + 2 : -c - 2], pd[kRev ? c + 3 : -c - 3]);
                        if (kRows) {
                            w0 = fmul2(rf, w0);
                            w1 = fmul2(rf, w1);
                        }
                        float2 s0 = make_float2(__uint_as_float(r[c]), __uint_as_float(r[c + 1]));
                        float2 s1 = make_float2(__uint_as_float(r[c + 2]), __uint_as_float(r[c + 3]));
                        scale(par, j0 + c, off, s0, s1, w0, w1);
                        s0 = fmul2(s0, w0);
                        s1 = fmul2(s1, w1);
                        // (what is masked may be infinite: selected, not multiplied away)
                        if (kRev ? c < lane : c > lane) s0.x = 0.0f;
                        if (kRev ? c + 1 < lane : c + 1 > lane) s0.y = 0.0f;
                        if (kRev ? c + 2 < lane : c + 2 > lane) s1.x = 0.0f;
                        if (kRev ? c + 3 < lane : c + 3 > lane) s1.y = 0.0f;
                        if (kDen) {
                            rs.x += s0.x + s1.x;
                            rs.y += s0.y + s1.y;
                        }
                        put(c, s0);
                        put(c + 2, s1);
                    }
                }
            }
            if (kDen) dsum[(par * 2 + half) * kT + row] = rs.x + rs.y;
            // P~ goes over the scores once both warps of these rows have read theirs
            tc_fence_before();
            named_bar_sync(1 + q, 64);
            tc_fence_after();
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
                tmem_st16(trow + kColP + 16 * (half + 2 * hh), pk[hh]);
                if (kLimb) tmem_st16(trow + kColP + 64 + 16 * (half + 2 * hh), pl[hh]);
            }
            tmem_wait_st();
            // (before PT: no barrier may run two phases ahead of a thread that waits on it)
            if (kMode == kOutE && has_z) wait_k(B_MF, i);   // zf of this chunk
            tc_fence_before();
            warp_arrive(&bar[B_PT]);
        };
        // a chunk's F-wide outputs
        auto out_e = [&](int i) {
            const int t0 = chunk_of(i) * kT, n = min(kT, len - t0), par = i & 1;
            const int64_t grow = static_cast<int64_t>(bh) * p.L + t0 + row;
            const bool valid = row < n;
            const float fac = decay_pow(g2, kRev ? max(n - 1 - row, 0) : row + 1);
            float qo = 0.0f, qm = 1.0f;
            if (kRows && valid) {
                qm = p.q_mul[grow];
                qo = p.q_off[grow];
            }
            scores(i, qo, qm);
            // outputs, 64 features at a time; through the warp's staging box and a TMA store
            // unless rows of the tensor behind the sequence have to stay
            const float fq = fac * qm, zc = kRows ? -qo : 1.0f;
            const bool whole = n == kT || t0 + n == p.L;
            const uint32_t box = sbase + Lo.stg + ew * 2048;
            for (int s = 0; s < ns; ++s) {
                const int v = i * ns + s, ob = v & 1;
                wait_k(B_OF + ob, v >> 1);
                tc_fence_after();
                uint32_t a[32], e[32];
                tmem_ld32(trow + col_oi(kLimb, ob) + 32 * half, a);
                tmem_ld32(trow + col_oe(kLimb, ob) + 32 * half, e);
                tmem_wait_ld();
                reg_fence(a);
                reg_fence(e);
                tc_fence_before();
                warp_arrive(&bar[B_OE + ob]);
                const int fl = 64 * s + 32 * half;
                uint32_t o[16];
                const float2 fq2 = make_float2(fq, fq), zc2 = make_float2(zc, zc);
                const float4* z4 = reinterpret_cast<const float4*>(zf + par * kMaxFw + fl);
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    float2 e0 = make_float2(__uint_as_float(e[4 * c]), __uint_as_float(e[4 * c + 1]));
                    float2 e1 = make_float2(__uint_as_float(e[4 * c + 2]), __uint_as_float(e[4 * c + 3]));
                    if (has_z) {
                        const float4 z = z4[c];
                        e0 = ffma2(zc2, make_float2(z.x, z.y), e0);
                        e1 = ffma2(zc2, make_float2(z.z, z.w), e1);
                    }
                    e0 = ffma2(fq2, e0, make_float2(__uint_as_float(a[4 * c]), __uint_as_float(a[4 * c + 1])));
                    e1 = ffma2(fq2, e1, make_float2(__uint_as_float(a[4 * c + 2]), __uint_as_float(a[4 * c + 3])));
                    o[2 * c] = pack_bf16(e0.x, e0.y);
                    o[2 * c + 1] = pack_bf16(e1.x, e1.y);
                }
                if (whole) {
                    if (lane == 0) bulk_wait_read<0>();   // the box's last store has read it
                    __syncwarp();
                    const uint32_t rsw = (static_cast<uint32_t>(lane) >> 1) & 3u;   // 64-byte swizzle
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        st_shared_v4(box + lane * 64u + ((static_cast<uint32_t>(c) ^ rsw) << 4), o[4 * c], o[4 * c + 1],
                                     o[4 * c + 2], o[4 * c + 3]);
                    fence_async_smem();
                    __syncwarp();
                    if (lane == 0 && fl < fv) {
                        tma_store_3d(&tout, sm + Lo.stg + ew * 2048, f0 + fl, t0 + 32 * q, bh);
                        bulk_commit_group();
                    }
                } else if (valid) {
                    __nv_bfloat16* dst = p.o + grow * p.F + f0 + fl;
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        if (fl + 8 * c < fv)
                            *reinterpret_cast<uint4*>(dst + 8 * c) = make_uint4(o[4 * c], o[4 * c + 1], o[4 * c + 2], o[4 * c + 3]);
                }
            }
        };
        if (kSplit && warp >= 8) {
            if (kLimb) regs_inc<160>();
            else regs_dec<112>();
            for (int i = 0; i < count; ++i) out_e(i);
            if (lane == 0) bulk_wait<0>();   // this warp's stores have landed
        } else {
        if (!kLimb) regs_inc<kSplit ? 192 : kIdle ? 200 : 208>();
        constexpr int kNb = kLimb ? 1 : 2;      // 128-feature blocks
        float run[kNb][kW], zrun[kNb] = {};   // M at (f = 128 b + row, e = 32 half + c); z at b
        auto has_zrow = [&](int b) { return has_z && (kSplit || b == half); };
        // the state entering the segment: M <- lambda^n M + (its sums) over the segments before it
        auto add_state = [&](const float* S, const float* z, int64_t at, float lam, bool own) {
#pragma unroll
            for (int b = 0; b < kNb; ++b) {
                const int f = 128 * b + row;
                if (f >= fv) continue;
                const float4* src = own ? reinterpret_cast<const float4*>(S + at * sums_floats(p.F)) + sums_at(f0 + f, 8 * half)
                                        : reinterpret_cast<const float4*>(S + (at * p.F + f0 + f) * 64 + 32 * half);
                const int step = own ? 128 : 1;
#pragma unroll
                for (int c = 0; c < kW / 4; ++c) {
                    const float4 w = src[c * step];
                    run[b][4 * c] = fmaf(lam, run[b][4 * c], w.x);
                    run[b][4 * c + 1] = fmaf(lam, run[b][4 * c + 1], w.y);
                    run[b][4 * c + 2] = fmaf(lam, run[b][4 * c + 2], w.z);
                    run[b][4 * c + 3] = fmaf(lam, run[b][4 * c + 3], w.w);
                }
                if (has_zrow(b)) zrun[b] = fmaf(lam, zrun[b], z[at * p.F + f0 + f]);
            }
        };
#pragma unroll
        for (int b = 0; b < kNb; ++b)
#pragma unroll
            for (int c = 0; c < kW; ++c) run[b][c] = 0.0f;
        if (p.starts) {
            add_state(p.starts, p.starts_z, sidx, 1.0f, true);
        } else {
            if (p.first) add_state(p.first, p.first_z, bh, 1.0f, false);
            if (p.sums)
                for (int i = 0; i < (kRev ? nseg - 1 - seg : seg); ++i) {
                    const int s = kRev ? nseg - 1 - i : i;
                    add_state(p.sums, p.sums_z, static_cast<int64_t>(bh) * nseg + s,
                              decay_pow(g2, max(min(seg_lo(s + 1) * kT, len) - seg_lo(s) * kT, 0)), true);
                }
        }
        // the operand copy of M, and its z column, for chunk i
        auto write_m = [&](int i) {
#pragma unroll
            for (int b = 0; b < kNb; ++b) {
                const int f = 128 * b + row;
                if (f < 64 * ns) {
                    const uint32_t slab = sbase + Lo.m + (f >> 6) * kSlab;
#pragma unroll
                    for (int c = 0; c < kW / 8; ++c)
                        st_shared_v4(slab + sw128_off(f & 63, 4 * half + c),
                                     pack_bf16(run[b][8 * c], run[b][8 * c + 1]), pack_bf16(run[b][8 * c + 2], run[b][8 * c + 3]),
                                     pack_bf16(run[b][8 * c + 4], run[b][8 * c + 5]), pack_bf16(run[b][8 * c + 6], run[b][8 * c + 7]));
                    if (kLimb && b == 0)   // the second limb, two slabs on
#pragma unroll
                        for (int c = 0; c < kW / 8; ++c) {
                            uint32_t l[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const float x = run[b][8 * c + 2 * k], y = run[b][8 * c + 2 * k + 1];
                                const uint32_t hi = pack_bf16(x, y);
                                l[k] = pack_bf16(x - bf_lo(hi), y - bf_hi(hi));
                            }
                            st_shared_v4(slab + 2 * kSlab + sw128_off(f & 63, 4 * half + c), l[0], l[1], l[2], l[3]);
                        }
                    if (has_zrow(b)) {
                        if (kDen) {
                            uint16_t l[3];
                            limbs3(zrun[b], l);
                            const uint32_t t = sbase + Lo.fs + ((i * nsE + (f >> 6)) & 3) * kSlot + kTile;
#pragma unroll
                            for (int k = 0; k < 3; ++k) st_shared_u16(t + sw128_off(k, (f & 63) >> 3) + (f & 7) * 2, l[k]);
                        } else if (kMode == kOutE) {
                            zf[(i & 1) * kMaxFw + f] = zrun[b];
                        }
                    }
                }
            }
            fence_async_smem();
            warp_arrive(&bar[B_MF]);
        };
        // the weighted rows of chunk i (this thread: token `row`, 32 of its columns) in limbs,
        // the z weights and the score scalars of its tokens
        auto write_y = [&](int i) {
            const int t0 = chunk_of(i) * kT, n = min(kT, len - t0), eb = i % kEs;
            const bool in = row < n;
            const int64_t grow = static_cast<int64_t>(bh) * p.L + t0 + row;
            const bool cols = kPair ? kNorm && rev : kCols;   // row scalars on the state tokens
            const float mul = cols && in ? (second ? p.second.s_mul : p.s_mul)[grow] : 1.0f;
            const float off = cols && in ? (second ? p.second.s_off : p.s_off)[grow] : 0.0f;
            const float w = in ? decay_pow(g2, rev ? row + 1 : n - 1 - row) : 0.0f;
            const float a = w * mul;
            const uint32_t ybase = sbase + kY + (kMode == kState ? eb * 4 * kTile : 0);
            wait_k(B_ESF + eb, i / kEs);
            uint4 r[kW / 8];
#pragma unroll
            for (int c = 0; c < kW / 8; ++c)
                r[c] = *reinterpret_cast<const uint4*>(sm + Lo.es + eb * kTile + sw128_off(row, 4 * half + c));
#pragma unroll
            for (int c = 0; c < kW / 8; ++c) {
                const uint32_t o = sw128_off(row, 4 * half + c);
                uint32_t v[4] = {r[c].x, r[c].y, r[c].z, r[c].w};
                if (!in) {
                    v[0] = v[1] = v[2] = v[3] = 0u;
                    if (kMode == kOutF) st_shared_v4(sbase + Lo.es + eb * kTile + o, 0u, 0u, 0u, 0u);   // an operand itself
                }
                if (nl == 1) {
                    st_shared_v4(ybase + o, v[0], v[1], v[2], v[3]);
                    continue;
                }
                float2 y[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) y[e] = fmul2(make_float2(a, a), make_float2(bf_lo(v[e]), bf_hi(v[e])));
#pragma unroll
                for (int k = 0; k < 3; ++k) {
                    if (k >= (kMode == kOutE ? 2 : nl)) break;
                    uint32_t l[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        l[e] = pack_bf16(y[e].x, y[e].y);
                        y[e] = ffma2(make_float2(-1.0f, -1.0f), make_float2(bf_lo(l[e]), bf_hi(l[e])), y[e]);
                    }
                    st_shared_v4((kMode == kOutF && k == 2 ? sbase + Lo.y : ybase + k * kTile) + o, l[0], l[1], l[2], l[3]);
                }
            }
            if (half == 0) {
                if (has_z) {
                    uint16_t l[3];
                    limbs3(cols ? -a * off : w, l);
                    if (kMode == kState) {
                        const uint32_t lo = l[0] | (static_cast<uint32_t>(l[1]) << 16);
                        st_shared_v4(ybase + 3 * kTile + sw128_off(row, 0), lo, l[2], 0u, 0u);
                    } else {
                        const uint32_t t = sbase + Lo.wext + (row >> 6) * kExt;
#pragma unroll
                        for (int k = 0; k < 3; ++k) st_shared_u16(t + sw128_off(k, (row & 63) >> 3) + (row & 7) * 2, l[k]);
                    }
                }
                if (kCols && kMode != kState) {   // (kState masks no scores and has no room for them)
                    smul[(i & 1) * kT + row] = mul;
                    soff[(i & 1) * kT + row] = off;
                }
            }
            fence_async_smem();
            warp_arrive(&bar[kMode == kState ? B_YF + eb : B_YF]);
        };
        // M <- lambda^n M + T
        ChunkDecay lam_c(p.log_decay[bh % p.H], g2, kT);
        auto update_m = [&](int i) {
            const int n = min(kT, len - chunk_of(i) * kT);
            const float lam = n == kT ? lam_c.next() : decay_pow(g2, n);
            const bool two = kMode != kOutE && nl > 1;
            if (kMode != kState) {
                wait_k(B_TF, i);
                tc_fence_after();
            }
#pragma unroll
            for (int b = 0; b < kNb; ++b) {
                if (2 * b >= ns) break;
                if (kMode == kState) {
                    wait_k(B_TF + b, i);
                    tc_fence_after();
                }
                const uint32_t tc = trow + col_t(kMode, kLimb) + t_stride(kMode) * b;
#pragma unroll
                for (int hh = 0; hh < kW / 32; ++hh) {
                uint32_t t[32], t2[32], t3[32], z0 = 0, z1 = 0, z2 = 0;
                tmem_ld32(tc + 32 * (half + hh), t);
                if (two) tmem_ld32(tc + 64 + 32 * half, t2);
                if (kMode == kState) tmem_ld32(tc + 128 + 32 * half, t3);
                if (hh == 0 && has_zrow(b)) {
                    tmem_ld1(tc + col_z(kMode), z0);
                    tmem_ld1(tc + col_z(kMode) + 1, z1);
                    tmem_ld1(tc + col_z(kMode) + 2, z2);
                }
                tmem_wait_ld();
                reg_fence(t);
                reg_fence(t2);
                reg_fence(t3);
                reg_fence1(z0);
                reg_fence1(z1);
                reg_fence1(z2);
#pragma unroll
                for (int c = 0; c < 32; c += 2) {
                    float2 w = make_float2(__uint_as_float(t[c]), __uint_as_float(t[c + 1]));
                    if (kMode == kState) {   // the small limbs first
                        const float2 w3 = make_float2(__uint_as_float(t3[c]), __uint_as_float(t3[c + 1]));
                        w = fadd2(w, fadd2(w3, make_float2(__uint_as_float(t2[c]), __uint_as_float(t2[c + 1]))));
                    } else if (two) {
                        w = fadd2(w, make_float2(__uint_as_float(t2[c]), __uint_as_float(t2[c + 1])));
                    }
                    const float2 r = ffma2(make_float2(lam, lam), make_float2(run[b][32 * hh + c], run[b][32 * hh + c + 1]), w);
                    run[b][32 * hh + c] = r.x;
                    run[b][32 * hh + c + 1] = r.y;
                }
                if (hh == 0 && has_zrow(b))
                    zrun[b] = fmaf(lam, zrun[b], __uint_as_float(z0) + (__uint_as_float(z1) + __uint_as_float(z2)));
                }
                if (kMode == kState) {
                    tc_fence_before();
                    warp_arrive(&bar[B_MF + b]);   // T has been read
                }
            }
            tc_fence_before();
        };
        if (count > 0) {
            if (kMode != kState) {
                write_m(0);
            } else {
                warp_arrive(&bar[B_MF]);
                warp_arrive(&bar[B_MF + 1]);
            }
            write_y(0);
        }
        for (int i = 0; i < count; ++i) {
            const bool more = i + 1 < count;
            if (kMode == kState) {
                if (more) write_y(i + 1);   // the other limb buffer: off the state's chain
                update_m(i);
            } else if (kSplit) {
                update_m(i);
                if (more) {
                    // the output warps have passed their wait for this chunk's scalars
                    if (kCols) wait_k(B_PT, i);
                    write_y(i + 1);
                    wait_k(B_OD, i);   // the state's operand is read until the chunk's last output
                    write_m(i + 1);
                }
            } else {
                const int t0 = chunk_of(i) * kT, n = min(kT, len - t0), par = i & 1;
                const int64_t grow = static_cast<int64_t>(bh) * p.L + t0 + row;
                const bool valid = row < n;
                const float fac = decay_pow(g2, kRev ? max(n - 1 - row, 0) : row + 1);
                scores(i, 0.0f, 1.0f);
                // the earlier feature blocks' sums: [chunk][16 float4 of a row][128 rows], so that a
                // warp's accesses are whole lines; on their way while the state is summed
                const int64_t pc = static_cast<int64_t>(bh) * ((p.L + kT - 1) / kT) + chunk_of(i);
                float4* pp = reinterpret_cast<float4*>(p.part) + (pc * 16 + 8 * half) * kT + row;
                float* pd = p.part_den + pc * kT + row;
                float4 part[8];
                float part_dn = 0.0f;
                if (p.part_mode == 2) {
#pragma unroll
                    for (int c = 0; c < 8; ++c) part[c] = pp[c * kT];
                    if (kDen) part_dn = *pd;
                }
                update_m(i);
                if (more) write_m(i + 1);   // the next chunk's products want the state first
                wait_k(B_OF, i);
                tc_fence_after();
                uint32_t a[32], e[32], d0 = 0, d1 = 0, d2 = 0;
                tmem_ld32(trow + kColOi + 32 * half, a);
                tmem_ld32(trow + kColOe + 32 * half, e);
                if (kDen) {
                    tmem_ld1(trow + kColDen, d0);
                    tmem_ld1(trow + kColDen + 1, d1);
                    tmem_ld1(trow + kColDen + 2, d2);
                }
                tmem_wait_ld();
                reg_fence(a);
                reg_fence(e);
                reg_fence1(d0);
                reg_fence1(d1);
                reg_fence1(d2);
                tc_fence_before();
                warp_arrive(&bar[B_OE]);
                float t[32], dn = 0.0f;
#pragma unroll
                for (int c = 0; c < 32; ++c) t[c] = fmaf(fac, __uint_as_float(e[c]), __uint_as_float(a[c]));
                if (kDen)
                    dn = fmaf(fac, __uint_as_float(d0) + (__uint_as_float(d1) + __uint_as_float(d2)),
                              dsum[par * 2 * kT + row] + dsum[(par * 2 + 1) * kT + row]);
                if (p.part_mode == 1) {
#pragma unroll
                    for (int c = 0; c < 8; ++c) pp[c * kT] = make_float4(t[4 * c], t[4 * c + 1], t[4 * c + 2], t[4 * c + 3]);
                    if (half == 0) *pd = dn;
                } else if (p.part_mode == 2) {
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        t[4 * c] += part[c].x;
                        t[4 * c + 1] += part[c].y;
                        t[4 * c + 2] += part[c].z;
                        t[4 * c + 3] += part[c].w;
                    }
                    dn += part_dn;
                }
                if (p.part_mode != 1) {
                    if (kDen) {
                        if (p.den && half == 0 && valid) p.den[grow] = dn;
                        const float rd = 1.0f / (dn + p.eps);
#pragma unroll
                        for (int c = 0; c < 32; ++c) t[c] *= rd;
                    }
                    uint32_t o[4][4];   // 16-byte chunks of this row's 64 bytes
#pragma unroll
                    for (int c = 0; c < 16; ++c) o[c >> 2][c & 3] = pack_bf16(t[2 * c], t[2 * c + 1]);
                    // four lanes trade chunks, so that one store writes 64 bytes of 8 rows and not
                    // 16 bytes of 32: o[r] becomes chunk (lane & 3) of row (lane & ~3) + r
#pragma unroll
                    for (int m = 1; m <= 2; m *= 2)
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            if (c & m) continue;
#pragma unroll
                            for (int w = 0; w < 4; ++w) {
                                const bool up = (lane & m) != 0;
                                const uint32_t give = up ? o[c][w] : o[c + m][w];
                                const uint32_t got = __shfl_xor_sync(0xffffffffu, give, m);
                                if (up) o[c][w] = got; else o[c + m][w] = got;
                            }
                        }
                    const int r0 = 32 * q + (lane & ~3);
                    __nv_bfloat16* dst = p.o + (grow - row + r0) * 64 + 32 * half + 8 * (lane & 3);
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        if (r0 + r < n) *reinterpret_cast<uint4*>(dst + r * 64) = make_uint4(o[r][0], o[r][1], o[r][2], o[r][3]);
                }
                if (more) write_y(i + 1);
            }
        }
        if (leaves) {
            const int64_t at = kMode == kState ? sidx : bh;
            float *const last = second ? p.second.last : p.last, *const last_z = second ? p.second.last_z : p.last_z;
#pragma unroll
            for (int b = 0; b < kNb; ++b) {
                const int f = 128 * b + row;
                if (f >= fv) continue;
                float4* dst = kMode == kState ? reinterpret_cast<float4*>(last + at * sums_floats(p.F)) + sums_at(f0 + f, 8 * half)
                                              : reinterpret_cast<float4*>(last + (at * p.F + f0 + f) * 64 + 32 * half);
#pragma unroll
                for (int c = 0; c < kW / 4; ++c)
                    dst[c * (kMode == kState ? 128 : 1)] = make_float4(run[b][4 * c], run[b][4 * c + 1], run[b][4 * c + 2], run[b][4 * c + 3]);
                if (has_zrow(b) && last_z) last_z[at * p.F + f0 + f] = zrun[b];
            }
        }
        }
    }
    wt.report(p.err);
    drain_after_failure(wt.ok);
    tc_fence_before();
    __syncthreads();
    if (warp == 0) tmem_dealloc(tmem, 512);
}

template <int kMode, bool kRev, bool kNorm, bool kPair>
__global__ void __launch_bounds__(threads(kMode), 1)
k_tc_dec(const __grid_constant__ CUtensorMap tfs, const __grid_constant__ CUtensorMap tfq,
         const __grid_constant__ CUtensorMap tes, const __grid_constant__ CUtensorMap teq,
         const __grid_constant__ CUtensorMap tout, const __grid_constant__ P p)
{
    sweep<kMode, kRev, kNorm, kPair>(tfs, tfq, tes, teq, tout, p, blockIdx.x);
}

// The gradients' sweeps in one launch: dphq (the first n0 CTAs), dphk (the next n1) and, where
// it has one block of features, dv, whose CTAs leave four warps idle.
template <bool kNorm>
__global__ void __launch_bounds__(threads(kOutE), 1)
k_tc_dec_grads(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
               const __grid_constant__ CUtensorMap tdo, const __grid_constant__ CUtensorMap tq,
               const __grid_constant__ CUtensorMap tdq, const __grid_constant__ CUtensorMap tdk,
               const __grid_constant__ P pq, const __grid_constant__ P pk, const __grid_constant__ P pv, int n0, int n1)
{
    const int x = blockIdx.x;
    if (x < n0)
        sweep<kOutE, false, kNorm>(tk, tk, tv, tdo, tdq, pq, x);
    else if (x < n0 + n1)
        sweep<kOutE, true, kNorm>(tq, tq, tdo, tv, tdk, pk, x - n0);
    else
        sweep<kOutF, true, kNorm, false, true>(tq, tk, tdo, tdo, tq, pv, x - n0 - n1);
}

// Segment sums -> the states entering the segments, in place, S (four elements a thread) and z
// in one launch; first: the state entering the walk (null: zero), last: the one leaving it
// (null: not wanted; may be first).  Loads run eight segments ahead of the stores (L2 latency
// would be paid per segment otherwise).  grid (ceil((sums_floats(F) / 4 + F) / 256), BH)
__global__ void __launch_bounds__(256) k_dec_seg_scan(float* st, float* sz, const float* first, const float* first_z,
                                                      float* last, float* last_z, int F, int nseg, bool rev,
                                                      const float* log_decay, const int32_t* lengths, int H, int L)
{
    __shared__ float lam[kNumSMs];
    const int bh = blockIdx.y;
    {
        const int len = lengths ? min(max(lengths[bh / H], 0), L) : L;
        const int nch = (len + kT - 1) / kT;
        const float g2 = log_decay[bh % H] * kLog2e;
        for (int s = threadIdx.x; s < nseg; s += 256)
            lam[s] = decay_pow(g2, max(min((s + 1) * nch / nseg * kT, len) - s * nch / nseg * kT, 0));
    }
    after_previous_kernel();
    __syncthreads();
    constexpr int kAhead = 8;
    auto walk = [&](auto* q, int64_t w, auto run, auto* to, auto step) {
        for (int i0 = 0; i0 < nseg; i0 += kAhead) {
            decltype(run) t[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; ++i)
                if (i0 + i < nseg) t[i] = q[(rev ? nseg - 1 - i0 - i : i0 + i) * w];
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                if (i0 + i >= nseg) break;
                const int s = rev ? nseg - 1 - i0 - i : i0 + i;
                q[s * w] = run;
                run = step(lam[s], run, t[i]);
            }
        }
        if (to) *to = run;
    };
    const int x = blockIdx.x * 256 + threadIdx.x;
    const int64_t w = sums_floats(F) / 4;
    if (x < w) {
        const int f = ((x >> 7) >> 4) * 128 + (x & 127);
        if (f >= F) return;
        const int64_t at = (static_cast<int64_t>(bh) * F + f) * 16 + ((x >> 7) & 15);
        walk(reinterpret_cast<float4*>(st) + bh * nseg * w + x, w,
             first ? reinterpret_cast<const float4*>(first)[at] : make_float4(0.f, 0.f, 0.f, 0.f),
             last ? reinterpret_cast<float4*>(last) + at : nullptr, [](float l, float4 a, float4 b) {
                 return make_float4(fmaf(l, a.x, b.x), fmaf(l, a.y, b.y), fmaf(l, a.z, b.z), fmaf(l, a.w, b.w));
             });
    } else if (sz && x < w + F) {
        const int f = x - static_cast<int>(w);
        const int64_t at = static_cast<int64_t>(bh) * F + f;
        walk(sz + static_cast<int64_t>(bh) * nseg * F + f, F, first_z ? first_z[at] : 0.0f, last_z ? last_z + at : nullptr,
             [](float l, float a, float b) { return fmaf(l, a, b); });
    }
}

// [BH][L][cols] bf16 as a 3-D tensor, boxes of 64 columns x 128 tokens, 128-byte swizzle;
// columns past `cols` and rows past L read as zero.  out: boxes of 32 columns x 32 tokens,
// 64-byte swizzle, for stores; what lies past the edges is not written.
bool map_rows(CUtensorMap* m, const void* base, int cols, int L, int64_t BH, bool out = false)
{
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(L), static_cast<cuuint64_t>(BH)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(cols) * 2, static_cast<cuuint64_t>(L) * cols * 2};
    const cuuint32_t box[3] = {out ? 32u : 64u, out ? 32u : static_cast<cuuint32_t>(kT), 1};
    const cuuint32_t es[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, out ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
              out ? CU_TENSOR_MAP_L2_PROMOTION_NONE : CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// How a sweep is cut: blocks of at most `block` features, and segments of the sequence, as many
// as shorten it while each CTA finds an SM.  More of them cost more than they balance: forward
// B4 H8 L2048 F256 40 us with four, 54 with eight; backward B2 H16 L8192 F512 657 with four, 694
// with nine (1.95 waves instead of 0.86); ragged batches too, forward B8 H16 L1500 F128 43 with
// one, 56 with two.  Short sequences stay whole: forward B3 H24 L384 F128 16 us with one, 18.6
// with two; B3 H24 L640 F256 (two) 34, with one 35.
struct Plan {
    int nfb, fw, nseg;
    int64_t BH;
};

int chunks(const DecayArgs& a) { return (a.L + kT - 1) / kT; }
int64_t waves(int64_t ctas) { return (ctas + kNumSMs - 1) / kNumSMs; }

Plan plan(const DecayArgs& a, int block, bool blocks_in_grid)
{
    Plan c{};
    c.BH = static_cast<int64_t>(a.B) * a.H;
    c.nfb = (a.F + block - 1) / block;
    c.fw = ((a.F + c.nfb - 1) / c.nfb + 63) & ~63;
    const int64_t units = c.BH * (blocks_in_grid ? c.nfb : 1);
    const int nch = chunks(a);
    const int most = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(kNumSMs / units, nch)));
    // the fewest segments of the shortest time: a walk's chunks, and one and a half more for the
    // states that segments need first
    const int len = (nch + most - 1) / most;
    c.nseg = 2 * len + 3 < 2 * nch ? (nch + len - 1) / len : 1;
    return c;
}

// out, dv, dphk: the feature blocks of a 64-wide output follow one another, so (b, h) and
// segments fill the GPU; dphk shares dv's segments and their states.
Plan plan_f(const DecayArgs& a) { return plan(a, kMaxFw, false); }
// dphq: the normalized form's two limbs leave room for 128 features; otherwise 256, unless
// blocks of 128 fill the GPU without segments, whose states are a pass of their own.
Plan plan_q(const DecayArgs& a)
{
    const Plan h = plan(a, kMaxFw / 2, true);
    if (a.norm || (h.nseg == 1 && h.BH * h.nfb <= kNumSMs)) return h;
    return plan(a, kMaxFw, true);
}

// The backward's: its three sweeps side by side fill the GPU with a third of the segments, often
// without any.  Compared in half chunks of a CTA (launches and states included): that, with the
// same segments for both walks, whose sums share a launch, and one sweep after the other, each
// cut for itself.  The latter and the former, measured: B2 H16 L2048 F256 115 and 80 us, B4 H12
// L1024 F64 normalized 63 and 39, B8 H8 L1111 F128 ragged 59 and 49; but B1 H16 L4096 F128 76
// and 85.
struct BwdPlan {
    Plan k, q;   // dphk and dv, dphq
};

BwdPlan plan_bwd(const DecayArgs& a)
{
    BwdPlan b{plan_f(a), plan_q(a)};
    const int64_t BH = b.k.BH, cs = plan(a, kMaxFw, true).nfb;
    const int nch = chunks(a);
    auto len = [&](int n) { return static_cast<int64_t>((nch + n - 1) / n); };
    auto sums = [&](int n) { return n > 1 ? 3 + waves(BH * cs * n) * len(n) : 0; };
    int64_t best = 4 * (2 * (waves(BH * b.q.nfb * b.q.nseg) * len(b.q.nseg) +
                             (waves(BH * b.k.nfb * b.k.nseg) + b.k.nfb * waves(BH * b.k.nseg)) * len(b.k.nseg)) +
                        4 + sums(b.q.nseg) + sums(b.k.nseg));
    const int most = static_cast<int>(std::min<int64_t>(std::max<int64_t>(1, kNumSMs / (2 * BH * cs)), nch));
    int joined = 0;
    // (of the numbers of segments that give the same length, the least)
    for (int n = 1; n <= most; n = len(n) > 1 ? (nch + static_cast<int>(len(n)) - 2) / (static_cast<int>(len(n)) - 1) : most + 1) {
        // (with a second block of dv's features it has to be clearly shorter)
        const int64_t t = (b.k.nfb > 1 ? 5 : 4) *
                          (2 * (waves(BH * (b.q.nfb + b.k.nfb + 1) * n) + (b.k.nfb - 1) * waves(BH * n)) * len(n) +
                           (n > 1 ? 3 + 2 * len(n) : 0));
        if (joined ? t < best : t <= best) {
            best = t;
            joined = n;
        }
    }
    if (joined) b.k.nseg = b.q.nseg = joined;
    return b;
}

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

// Sums (or starting states) of a walk's segments.
struct Segs {
    float *st, *sz;
};

struct Carve {
    Segs walk, walk_q;   // of the walk that the 64-wide output shares, and of dphq's
    float *in, *in_z, *part, *part_den, *rz, *r;
    size_t bytes;
};

Carve carve(const DecayArgs& a, bool bwd, void* ws)
{
    char* base = static_cast<char*>(ws);
    size_t o = 0;
    auto take = [&](size_t floats) {
        float* q = reinterpret_cast<float*>(base + o);
        o += align256(floats * 4);
        return q;
    };
    Carve k{};
    const Plan c = plan_f(a);
    const size_t rows = static_cast<size_t>(c.BH) * a.L;
    auto segs = [&](int nseg) {
        Segs s{};
        if (nseg > 1) {
            s.st = take(static_cast<size_t>(c.BH) * nseg * sums_floats(a.F));
            s.sz = take(static_cast<size_t>(c.BH) * nseg * a.F);
        }
        return s;
    };
    int nseg = c.nseg, nseg_q = 1;
    if (bwd) {                  // (the size of a workspace serves either form)
        DecayArgs other = a;
        other.norm = !a.norm;
        const BwdPlan x = plan_bwd(a), y = plan_bwd(other);
        nseg = std::max(x.k.nseg, y.k.nseg);
        nseg_q = std::max(x.q.nseg, y.q.nseg);
    }
    k.walk = segs(nseg);
    if (nseg > 1) {
        k.in = take(static_cast<size_t>(c.BH) * a.F * 64);
        k.in_z = take(static_cast<size_t>(c.BH) * a.F);
    }
    if (c.nfb > 1) {
        const size_t padded = static_cast<size_t>(c.BH) * ((a.L + kT - 1) / kT) * kT;
        k.part = take(padded * 64);
        k.part_den = take(padded);
    }
    if (bwd) {
        k.rz = take(rows);
        k.r = take(rows);
        k.walk_q = segs(nseg_q);
    }
    k.bytes = o;
    return k;
}

template <int kMode, bool kRev, bool kNorm, bool kPair = false>
cudaError_t launch1(const CUtensorMap& fs, const CUtensorMap& fq, const CUtensorMap& es, const CUtensorMap& eq,
                    const CUtensorMap& out, const P& p, const Plan& c, bool& chained, cudaStream_t st)
{
    constexpr size_t smem = layout(kMode).total + 1024;
    static_assert(smem <= 232448, "shared memory of one CTA");
    const auto kernel = k_tc_dec<kMode, kRev, kNorm, kPair>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    const int64_t grid = c.BH * (p.nsl + (kPair ? p.second.nsl : 0)) * (kMode == kOutF ? 1 : p.nfb);
    const bool first = !chained;
    chained = true;
    return launch_in_chain(first, +kernel, dim3(static_cast<unsigned>(grid)), threads(kMode), smem, st, fs, fq, es, eq, out, p);
}

template <int kMode>
cudaError_t launch(const char* name, const CUtensorMap& fs, const CUtensorMap& fq, const CUtensorMap& es,
                   const CUtensorMap& eq, const CUtensorMap& out, const P& p, const Plan& c, bool rev, bool norm,
                   bool& chained, cudaStream_t st)
{
    TraceScope trace_(name, st);
    if constexpr (kMode == kState)
        if (p.second.nsl > 0)
            return norm ? launch1<kMode, false, true, true>(fs, fq, es, eq, out, p, c, chained, st) : launch1<kMode, false, false, true>(fs, fq, es, eq, out, p, c, chained, st);
    if (rev) return norm ? launch1<kMode, true, true>(fs, fq, es, eq, out, p, c, chained, st) : launch1<kMode, true, false>(fs, fq, es, eq, out, p, c, chained, st);
    return norm ? launch1<kMode, false, true>(fs, fq, es, eq, out, p, c, chained, st) : launch1<kMode, false, false>(fs, fq, es, eq, out, p, c, chained, st);
}

// Armed by slay_debug_expire_wait(2), consumed by the next call that runs these sweeps.
std::atomic<int> g_wait_fault{0};

P base(const DecayArgs& a, const Plan& c, int* err, bool withhold)
{
    P p{};
    p.withhold = withhold;
    p.log_decay = a.log_decay;
    p.lengths = a.lengths;
    p.H = a.H;
    p.L = a.L;
    p.F = a.F;
    p.nseg = p.nsl = c.nseg;
    p.nfb = c.nfb;
    p.fw = c.fw;
    p.eps = a.eps;
    p.err = err;
    return p;
}

// What the output sweeps start from, and the state that the walk leaves.  Up to kMaxSums
// segments, each sweep adds up the sums of the segments before its own (66 KB each from L2, at
// F = 256) and the one that walks last writes the state; beyond, a scan kernel does both.  A
// state that enters the walk counts as two more.  Forward at F = 256: four segments (B4 H8 L2048)
// 40 us against 44 with the scan, nine (B1 H16 L16384) 128 against 118, three and a carried
// state (B1 H4 L384) 22.6 against 18.5.
constexpr int kMaxSums = 4;

// A walk whose segments' states are wanted.
struct Start {
    const Plan* c;
    Segs segs;
    P* p;                          // its sweeps' parameters
    const CUtensorMap *fs, *es;
    bool rev;
    const float *first, *first_z;
    float *last, *last_z;
    bool scan() const { return c->nseg - 1 + (first ? 2 : 0) > kMaxSums - 1; }
    int summed() const { return scan() ? c->nseg : c->nseg - 1; }   // (without a scan nobody adds the last segment's)
};

// Two walks' sums come from one launch where its CTAs still find an SM each: backward B1 H4
// L1000 F256 41 us, 47 one after the other; beyond, the sweep that follows a walk's own launch
// finds its rows in L2, B1 H8 L16000 F256 170 us against 181.
bool together(const DecayArgs& a, const Start& x, const Start& y)
{
    const Plan cs = plan(a, kMaxFw, true);
    return x.c->nseg > 1 && y.c->nseg > 1 && cs.BH * cs.nfb * (x.summed() + y.summed()) <= kNumSMs;
}

// For one walk or two.
cudaError_t segment_states(const DecayArgs& a, const Carve& k, Start* const* walks, int n, bool& chained, cudaStream_t st)
{
    Start* cut[2];
    int m = 0;
    for (int i = 0; i < n; ++i) {
        Start& w = *walks[i];
        P& p = *w.p;
        p.first = w.first;
        p.first_z = w.first_z;
        p.last = w.last;
        p.last_z = w.last_z;
        if (w.c->nseg == 1) continue;
        if (!w.scan() && w.first && (w.last == w.first || (w.last_z && w.last_z == w.first_z))) {
            // in place: the CTAs read a copy, one of them writes the state while others start
            const size_t floats = static_cast<size_t>(w.c->BH) * a.F * sizeof(float);
            cudaError_t e = cudaMemcpyAsync(k.in, w.first, floats * 64, cudaMemcpyDeviceToDevice, st);
            if (e == cudaSuccess && w.first_z) e = cudaMemcpyAsync(k.in_z, w.first_z, floats, cudaMemcpyDeviceToDevice, st);
            if (e != cudaSuccess) return e;
            p.first = k.in;
            p.first_z = w.first_z ? k.in_z : nullptr;
            chained = false;             // the next kernel follows a copy
        }
        cut[m++] = &w;
    }
    if (m == 0) return cudaSuccess;
    auto walk = [&](const Start& w) {
        return P::Walk{w.p->s_mul, w.p->s_off, w.segs.st, w.segs.sz, w.rev ? 1 : 0, w.c->nseg,
                       w.rev ? w.c->nseg - w.summed() : 0, w.summed()};
    };
    const Plan cs = plan(a, kMaxFw, true);   // (the sums go by blocks of 256 whatever the sweep's)
    P q = *cut[0]->p;
    q.nfb = cs.nfb;
    q.fw = cs.fw;
    q.first = q.first_z = nullptr;
    const P::Walk w0 = walk(*cut[0]);
    q.last = w0.last;
    q.last_z = w0.last_z;
    q.rev = w0.rev;
    q.nsl = w0.nsl;
    q.seg0 = w0.seg0;
    q.n0 = static_cast<int>(cs.BH * w0.nsl * cs.nfb);
    if (m == 2) q.second = walk(*cut[1]);
    const Start& o = *cut[m - 1];
    cudaError_t e = launch<kState>("tc_decay_state", *cut[0]->fs, *o.fs, *cut[0]->es, *o.es, *cut[0]->fs, q, cs, cut[0]->rev, a.norm, chained, st);
    for (int i = 0; i < m && e == cudaSuccess; ++i) {
        const Start& w = *cut[i];
        P& p = *w.p;
        if (!w.scan()) {
            p.sums = w.segs.st;
            p.sums_z = w.segs.sz;
            continue;
        }
        TraceScope trace_("decay_seg_scan", st);
        e = launch_in_chain(false, k_dec_seg_scan, dim3(static_cast<unsigned>((sums_floats(a.F) / 4 + a.F + 255) / 256), static_cast<unsigned>(w.c->BH)),
                            256, 0, st, w.segs.st, a.norm ? w.segs.sz : nullptr, w.first, w.first_z, w.last, w.last_z, a.F,
                            w.c->nseg, w.rev, a.log_decay, a.lengths, a.H, a.L);
        p.starts = w.segs.st;
        p.starts_z = w.segs.sz;
        p.last = p.last_z = nullptr;
    }
    return e;
}

template <bool kNorm>
cudaError_t launch_grads(const CUtensorMap& k, const CUtensorMap& v, const CUtensorMap& dout, const CUtensorMap& q,
                         const CUtensorMap& dq, const CUtensorMap& dk, const P& pq, const P& pk, const P* pv, int64_t BH,
                         bool& chained, cudaStream_t st)
{
    constexpr size_t smem = std::max(layout(kOutE).total, layout(kOutF).total) + 1024;
    const auto kernel = k_tc_dec_grads<kNorm>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    const int n0 = static_cast<int>(BH * pq.nsl * pq.nfb), n1 = static_cast<int>(BH * pk.nsl * pk.nfb);
    const int n2 = pv ? static_cast<int>(BH * pv->nsl) : 0;
    const bool first = !chained;
    chained = true;
    TraceScope trace_("tc_decay_grads", st);
    return launch_in_chain(first, +kernel, dim3(static_cast<unsigned>(n0 + n1 + n2)), threads(kOutE), smem, st, k, v, dout, q, dq, dk,
                           pq, pk, pv ? *pv : pk, n0, n1);
}

// Whether the gradients' sweeps, of n0, n1 and n2 CTAs, share a launch: sequences of their own
// lengths even out, so do several waves of CTAs, and few CTAs fill each other's idle SMs.
// Backward, apart and together: B8 H8 L1111 F128 ragged (in two segments) 69 and 59 us; B32 H12
// L1024 F256 383 and 351; B1 H4 L1000 F256 41 and 27.  Where each fills most of the GPU once, they had better
// follow one another: B8 H16 L1000 F128 122 apart, 127 together.  (The host does not see the lengths: a
// ragged batch whose sequences are all long takes the latter.)
bool one_launch(const DecayArgs& a, int64_t n0, int64_t n1, int64_t n2)
{
    return a.lengths || std::max(n0, n1) > kNumSMs || waves(n0 + n1 + n2) < waves(n0) + waves(n1) + waves(n2);
}

// A sweep whose queries are on the F side: one launch per feature block, the blocks'
// numerators and denominators added in fp32.
cudaError_t out_f(const CUtensorMap& fs, const CUtensorMap& fq, const CUtensorMap& es, P p, const Plan& c,
                  const Carve& k, bool rev, bool norm, bool& chained, cudaStream_t st)
{
    p.part = k.part;
    p.part_den = k.part_den;
    for (int fb = 0; fb < c.nfb; ++fb) {
        p.fb0 = fb;
        p.part_mode = c.nfb == 1 ? 0 : fb == 0 ? 1 : 2;
        const cudaError_t e = launch<kOutF>("tc_decay_out_f", fs, fq, es, es, fs, p, c, rev, norm, chained, st);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace

void decay_arm_wait_fault(bool on) { g_wait_fault.store(on ? 1 : 0); }

bool decay_tc_supported(const DecayArgs& a)
{
    return a.dt == SLAY_BF16 && a.L > 0 && a.F % 8 == 0 && a.F <= 2 * kMaxFw;
}

size_t decay_tc_ws(const DecayArgs& a, bool bwd) { return carve(a, bwd, nullptr).bytes; }

cudaError_t decay_tc_fwd(const DecayArgs& a, void* ws, int* err, cudaStream_t st)
{
    const Plan c = plan_f(a);
    const Carve k = carve(a, false, ws);
    CUtensorMap mq, mk, mv;
    if (!map_rows(&mq, a.phq, a.F, a.L, c.BH) || !map_rows(&mk, a.phk, a.F, a.L, c.BH) || !map_rows(&mv, a.v, 64, a.L, c.BH))
        return cudaErrorInvalidValue;
    P p = base(a, c, err, g_wait_fault.exchange(0) != 0);
    bool chained = false;   // whether a kernel of this call runs before
    Start w{&c, k.walk, &p, &mk, &mv, false, a.S_in, a.z_in, a.S_out, a.z_out}, *walks[] = {&w};
    cudaError_t e = segment_states(a, k, walks, 1, chained, st);
    if (e != cudaSuccess) return e;
    p.o = static_cast<__nv_bfloat16*>(a.out_w);
    p.den = a.den_w;
    return out_f(mk, mq, mv, p, c, k, false, a.norm, chained, st);
}

cudaError_t decay_tc_bwd(const DecayArgs& a, void* ws, int* err, cudaStream_t st)
{
    const BwdPlan b = plan_bwd(a);
    const Plan &c = b.k, &cq = b.q;
    const Carve k = carve(a, true, ws);
    CUtensorMap mq, mk, mv, mo, mdq, mdk;
    if (!map_rows(&mq, a.phq, a.F, a.L, c.BH) || !map_rows(&mk, a.phk, a.F, a.L, c.BH) ||
        !map_rows(&mv, a.v, 64, a.L, c.BH) || !map_rows(&mo, a.dout, 64, a.L, c.BH) ||
        !map_rows(&mdq, a.dphq, a.F, a.L, c.BH, true) || !map_rows(&mdk, a.dphk, a.F, a.L, c.BH, true))
        return cudaErrorInvalidValue;
    bool chained = a.norm;   // whether a kernel of this call runs before
    cudaError_t e = a.norm ? decay_row_stats(a, k.rz, k.r, st) : cudaSuccess;
    if (e != cudaSuccess) return e;
    const float *rz = a.norm ? k.rz : nullptr, *r = a.norm ? k.r : nullptr;
    const bool withhold = g_wait_fault.exchange(0) != 0;
    P s = base(a, cq, err, withhold);   // dphq from the states before each token
    P g = base(a, c, err, withhold);    // dphk and dv from the states after each token
    g.s_mul = rz;
    g.s_off = r;
    Start before{&cq, k.walk_q, &s, &mk, &mv, false, a.S_in, a.z_in, nullptr, nullptr};
    Start after{&c, k.walk, &g, &mq, &mo, true, a.dS_out, a.dz_out, a.dS_in, a.dz_in}, *walks[] = {&after, &before};
    const bool both = together(a, after, before);
    if ((e = segment_states(a, k, both ? walks : walks + 1, both ? 2 : 1, chained, st)) != cudaSuccess) return e;
    s.q_mul = rz;
    s.q_off = r;
    s.o = static_cast<__nv_bfloat16*>(a.dphq);
    auto params_k = [&] {
        P w = g;              // (the state that the walk leaves is dv's sweep to write)
        w.last = w.last_z = nullptr;
        w.o = static_cast<__nv_bfloat16*>(a.dphk);
        return w;
    };
    // The three sweeps in one launch, once the states are there.  (A state that dv's updates in
    // place is dphk's to read first.)
    const bool in_place = c.nseg == 1 && ((a.dS_in && a.dS_in == a.dS_out) || (a.dz_in && a.dz_in == a.dz_out));
    const bool three = c.nfb == 1 && !in_place;
    if ((both || c.nseg == 1) && one_launch(a, c.BH * cq.nseg * cq.nfb, c.BH * c.nseg * c.nfb, three ? c.BH * c.nseg : 0)) {
        if (!both && (e = segment_states(a, k, walks, 1, chained, st)) != cudaSuccess) return e;
        g.z_state = g.last_z != nullptr;
        g.o = static_cast<__nv_bfloat16*>(a.dv);
        e = a.norm ? launch_grads<true>(mk, mv, mo, mq, mdq, mdk, s, params_k(), three ? &g : nullptr, c.BH, chained, st)
                   : launch_grads<false>(mk, mv, mo, mq, mdq, mdk, s, params_k(), three ? &g : nullptr, c.BH, chained, st);
        if (e != cudaSuccess || three) return e;
    } else {
        if ((e = launch<kOutE>("tc_decay_out_e", mk, mk, mv, mo, mdq, s, cq, false, a.norm, chained, st)) != cudaSuccess) return e;
        if (!both && (e = segment_states(a, k, walks, 1, chained, st)) != cudaSuccess) return e;
        if ((e = launch<kOutE>("tc_decay_out_e", mq, mq, mo, mv, mdk, params_k(), c, true, a.norm, chained, st)) != cudaSuccess) return e;
    }
    g.z_state = g.last_z != nullptr;
    g.o = static_cast<__nv_bfloat16*>(a.dv);
    return out_f(mq, mk, mo, g, c, k, true, a.norm, chained, st);
}

}  // namespace slay
