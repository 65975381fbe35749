// slay_pool.cu -- states of running sequences in the slots of a pool: one decayed decode step
// on the slots a batch names, and copies between slots (fork, move, clear).
//
// Both move each state once each way and compute next to nothing, so HBM bounds them:
// 8 F 65 bytes per head and step, 4 F 65 bytes read and written per head and copied slot.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "slay_decay.h"

namespace slay {
namespace {

namespace cg = cooperative_groups;

constexpr int kNT = 256;
constexpr int kNumSMs = 148;
constexpr int kRows = 4;        // rows of S a decode thread loads ahead
constexpr int kCopySmem = 128 * 1024;   // of a copying CTA at most: 32 KiB of lists, then 64 KiB of table or stage for 4096 pairs

__device__ __forceinline__ float ldf(const float* p) { return *p; }
__device__ __forceinline__ float ldf(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void stf(float* p, float x) { *p = x; }
__device__ __forceinline__ void stf(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

// ------------------------------------------------------------------------ decode
// S <- lambda S + k v^T, z <- lambda z + k, out = q^T S (/ (q . z + eps)) for batch row b and
// head h on slot slots[b].  A cluster of CTAs shares one (b, h), each a contiguous share of
// the F rows of S; 16 threads cover a row's 64 columns, and the partial numerators and
// denominators join in the first CTA through distributed shared memory.
// Bt 256, H 16, F 512 (1.07 GB): 175 us, 6.1 TB/s, 93% of the copy bandwidth; Bt 1, H 16,
// F 256: 6 us on the GPU, launch and latency.
// A row whose slot is outside the pool, or was already named by an earlier row, is left out:
// its out row and the slot stay as they were (two rows must not step one state at once).
template <typename T>
__global__ void __launch_bounds__(kNT) k_decay_decode(const T* __restrict__ phq, const T* __restrict__ phk,
                                                      const T* __restrict__ v, const float* __restrict__ log_decay,
                                                      float* __restrict__ S, float* __restrict__ z,
                                                      const int32_t* __restrict__ slots, T* __restrict__ out, int H,
                                                      int F, int n_slots, int norm, float eps)
{
    extern __shared__ __align__(16) float sm[];   // q and k of this CTA's features
    __shared__ float red[16][64];
    __shared__ float part[65];
    __shared__ float dred[kNT / 32];
    cg::cluster_group cl = cg::this_cluster();
    const int cs = cl.num_blocks(), rank = cl.block_rank();
    const int64_t bh = blockIdx.x / cs;
    const int b = static_cast<int>(bh / H), h = static_cast<int>(bh % H), tid = threadIdx.x;
    const int slot = slots ? slots[b] : b;
    if (slot < 0 || slot >= n_slots) return;      // the whole cluster sees the same slot
    const int share = (F + cs - 1) / cs, f0 = min(rank * share, F), n = min(share, F - f0);
    const int e4 = (tid & 15) * 4, fr = tid >> 4;
    const int64_t sh = static_cast<int64_t>(slot) * H + h;
    // the state streams through registers, kRows rows of F a thread ahead; the first of them
    // are on their way while the row's place in the batch is checked and q, k arrive
    float4* Sp = reinterpret_cast<float4*>(S + (sh * F + f0) * 64 + e4);
    float4 s[kRows];
    auto load = [&](int f) {
#pragma unroll
        for (int i = 0; i < kRows; ++i)
            if (f + 16 * i < n) s[i] = __ldcs(Sp + (f + 16 * i) * 16);
    };
    load(fr);
    int named = 0;
    if (slots)
        for (int i = tid; i < b; i += kNT) named |= slots[i] == slot;
    float* qs = sm;
    float* ks = sm + share;
    for (int f = tid; f < n; f += kNT) {
        qs[f] = ldf(phq + bh * F + f0 + f);
        ks[f] = ldf(phk + bh * F + f0 + f);
    }
    // a state lives through thousands of steps: near 1, lambda S is S + (lambda - 1) S, whose factor
    // is not off by lambda's own rounding (4096 steps of log_decay -9.78e-4: S would be 2.8e-5 off)
    const float lam = expf(log_decay[h]), drop = expm1f(log_decay[h]);
    const bool near = drop < 0.0f && drop > -0.5f;
    const float fac = near ? drop : lam;
    auto step = [&](float s, float a, float x) { return fmaf(fac, s, near ? fmaf(a, x, s) : a * x); };
    const T* vp = v + bh * 64 + e4;
    const float4 vv = make_float4(ldf(vp), ldf(vp + 1), ldf(vp + 2), ldf(vp + 3));
    if (__syncthreads_or(named)) return;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int f = fr; f < n; f += 16 * kRows) {
        float4 t[kRows];
#pragma unroll
        for (int i = 0; i < kRows; ++i) t[i] = s[i];
        if (f + 16 * kRows < n) load(f + 16 * kRows);
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const int g = f + 16 * i;
            if (g >= n) break;
            const float a = ks[g], c = qs[g];
            t[i].x = step(t[i].x, a, vv.x);
            t[i].y = step(t[i].y, a, vv.y);
            t[i].z = step(t[i].z, a, vv.z);
            t[i].w = step(t[i].w, a, vv.w);
            __stcs(Sp + g * 16, t[i]);
            acc.x = fmaf(c, t[i].x, acc.x);
            acc.y = fmaf(c, t[i].y, acc.y);
            acc.z = fmaf(c, t[i].z, acc.z);
            acc.w = fmaf(c, t[i].w, acc.w);
        }
    }
    *reinterpret_cast<float4*>(&red[fr][e4]) = acc;
    if (norm) {
        float d = 0.0f;
        float* zp = z + sh * F + f0;
        for (int f = tid; f < n; f += kNT) {
            const float w = step(zp[f], ks[f], 1.0f);
            zp[f] = w;
            d = fmaf(qs[f], w, d);
        }
        for (int x = 16; x > 0; x >>= 1) d += __shfl_xor_sync(0xffffffffu, d, x);
        if ((tid & 31) == 0) dred[tid >> 5] = d;
    }
    __syncthreads();
    if (tid < 64) {
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) s += red[i][tid];
        part[tid] = s;
    } else if (tid == 64) {
        float d = 0.0f;
        for (int i = 0; i < kNT / 32; ++i) d += norm ? dred[i] : 0.0f;
        part[64] = d;
    }
    cl.sync();
    if (rank == 0 && tid < 64) {
        float s = 0.0f, d = 0.0f;
        for (int i = 0; i < cs; ++i) {
            const float* p = cl.map_shared_rank(part, i);
            s += p[tid];
            d += p[64];
        }
        stf(out + bh * 64 + tid, norm ? s / (d + eps) : s);
    }
    cl.sync();   // the peers' shared memory stays until it has been read
}

template <typename T>
cudaError_t decode_t(const DecodeArgs& a, cudaStream_t st)
{
    // one CTA per (row, head) when those fill the GPU, else up to 8 that share it (at least 16
    // features each: one pass of the CTA).  H 16, F 512, one row: 3.8 us with 8, 6.4 with one;
    // 8 rows 6.7 with 2, 7.0 with one or 4, 9.8 with 8; 18 rows, F 256: 6.6 with one, 6.9 with 2
    const int64_t bh = static_cast<int64_t>(a.B) * a.H;
    int cs = 1;
    while (cs < 8 && bh * cs < kNumSMs && a.F >= 32 * cs) cs *= 2;
    const size_t smem = 2 * static_cast<size_t>((a.F + cs - 1) / cs) * sizeof(float);
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(bh * cs));
    cfg.blockDim = dim3(kNT);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = cs;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    TraceScope trace_("decay_decode", st);
    return cudaLaunchKernelEx(&cfg, k_decay_decode<T>, static_cast<const T*>(a.phq), static_cast<const T*>(a.phk),
                              static_cast<const T*>(a.v), a.log_decay, a.S, a.z, a.slots, static_cast<T*>(a.out), a.H,
                              a.F, a.n_slots, a.norm ? 1 : 0, a.eps);
}

// ------------------------------------------------------------------------- copies
// dst[i] <- src[i] for n pairs of slots, every source read as it was before the call.  A CTA
// owns a range of columns (`width` bytes of every slot): it reads its columns of all sources
// into shared memory, then writes them to the destinations, so a slot may be both a source
// and a destination, in any cycle, with no order between CTAs.  Where a destination is named
// more than once the last pair wins: a hash table in shared memory keeps, per destination,
// the highest pair index.
// B200: 128 slots of 2.1 MB (477 MB moved) in 90 us, 5.3 TB/s, 81% of the copy bandwidth.
// Ranges of 512 bytes (64 KiB a CTA, three to an SM) measured best: 256 bytes 97 us, 1 KiB with
// one CTA 94 us; bulk asynchronous copies of the same ranges 93 us in one stage or two.  The range
// shrinks as the pairs share a CTA's memory: 512 slots of 266 KB 63 us (4.3 TB/s), 2000 (32 bytes)
// 766 us (1.4), 4096 (16 bytes) 3.4 ms (0.6); of 16.6 KB, 4096 slots 62 us (2.2).
template <typename U>
__device__ __forceinline__ void copy_columns(const U* src_base, U* dst_base, int64_t slot_units, int64_t c0, int wu,
                                             int n, const int* src, const int* dst, U* stage)
{
    // wu units (a power of two) of each of n slots, columns [c0, c0 + wu) cut at slot_units
    for (int i = threadIdx.x; i < n * wu; i += kNT) {
        const int p = i / wu, c = i & (wu - 1);
        if (dst[p] < 0 || c0 + c >= slot_units) continue;
        if (src[p] >= 0) {
            const uint32_t s = static_cast<uint32_t>(__cvta_generic_to_shared(stage + i));
            const U* g = src_base + src[p] * slot_units + c0 + c;
            if (sizeof(U) == 16)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(s), "l"(g) : "memory");
            else
                asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(s), "l"(g) : "memory");
        } else {
            stage[i] = U{};
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
    for (int i = threadIdx.x; i < n * wu; i += kNT) {
        const int p = i / wu, c = i & (wu - 1);
        if (dst[p] < 0 || c0 + c >= slot_units) continue;
        dst_base[dst[p] * slot_units + c0 + c] = stage[i];
    }
    __syncthreads();   // the stage is free again
}

__global__ void __launch_bounds__(kNT) k_state_copy(CopyArgs a, int wS, int nS, int wZ, int nZ, int z16, int table)
{
    extern __shared__ __align__(16) unsigned char raw[];
    int* src = reinterpret_cast<int*>(raw);
    int* dst = src + ((a.n + 3) & ~3);
    int* key = dst + ((a.n + 3) & ~3);   // [table], then the highest pair index [table]
    int* top = key + table;
    unsigned char* stage = reinterpret_cast<unsigned char*>(dst + ((a.n + 3) & ~3));   // after the table's use
    const int tid = threadIdx.x;
    for (int i = tid; i < table; i += kNT) { key[i] = -1; top[i] = -1; }
    __syncthreads();
    for (int i = tid; i < a.n; i += kNT) {
        const int s = a.src[i], d = a.dst[i];
        const bool ok = d >= 0 && d < a.n_dst && s >= -1 && s < a.n_src;
        src[i] = s;
        dst[i] = ok ? d : -1;
        if (!ok) continue;
        uint32_t at = (static_cast<uint32_t>(d) * 2654435761u) & (table - 1);
        for (int probe = 0; probe < table; ++probe) {
            const int was = atomicCAS(&key[at], -1, d);
            if (was == -1 || was == d) { atomicMax(&top[at], i); break; }
            at = (at + 1) & (table - 1);
        }
    }
    __syncthreads();
    for (int i = tid; i < a.n; i += kNT) {
        const int d = dst[i];
        if (d < 0) continue;
        uint32_t at = (static_cast<uint32_t>(d) * 2654435761u) & (table - 1);
        for (int probe = 0; probe < table && key[at] != d; ++probe) at = (at + 1) & (table - 1);
        if (top[at] != i) dst[i] = -1;   // a later pair writes this destination
    }
    __syncthreads();
    for (int w = blockIdx.x; w < nS + nZ; w += gridDim.x) {
        if (w < nS)
            copy_columns(reinterpret_cast<const float4*>(a.S_src), reinterpret_cast<float4*>(a.S_dst), a.hf * 16,
                         static_cast<int64_t>(w) * wS, wS, a.n, src, dst, reinterpret_cast<float4*>(stage));
        else if (z16)
            copy_columns(reinterpret_cast<const float4*>(a.z_src), reinterpret_cast<float4*>(a.z_dst), a.hf / 4,
                         static_cast<int64_t>(w - nS) * wZ, wZ, a.n, src, dst, reinterpret_cast<float4*>(stage));
        else
            copy_columns(a.z_src, a.z_dst, a.hf, static_cast<int64_t>(w - nS) * wZ, wZ, a.n, src, dst,
                         reinterpret_cast<float*>(stage));
    }
}

}  // namespace

cudaError_t decay_decode(const DecodeArgs& a, cudaStream_t st)
{
    return a.dt == SLAY_F32 ? decode_t<float>(a, st) : decode_t<__nv_bfloat16>(a, st);
}

cudaError_t state_copy(const CopyArgs& a, cudaStream_t st)
{
    int table = 32;
    while (table < 2 * a.n) table *= 2;
    const size_t lists = 2 * static_cast<size_t>((a.n + 3) & ~3) * sizeof(int);
    // column width in 16-byte units: the widest power of two, at most 64 (1 KiB), whose
    // stage leaves room for two CTAs on an SM and that gives every SM two ranges of columns
    const size_t budget = 100 * 1024 - lists;
    auto width = [&](int64_t units, size_t unit) {
        int w = 64;
        while (w > 1 && (static_cast<size_t>(a.n) * w * unit > budget || (units + w - 1) / w < 2 * kNumSMs)) w /= 2;
        return w;
    };
    const int64_t uS = a.hf * 16;
    const int wS = width(uS, 16);
    const int nS = static_cast<int>((uS + wS - 1) / wS);
    const int z16 = a.z_dst && a.hf % 4 == 0;
    const int64_t uZ = a.z_dst ? (z16 ? a.hf / 4 : a.hf) : 0;
    const int wZ = width(uZ, 16);
    const int nZ = static_cast<int>((uZ + wZ - 1) / wZ);
    const size_t stage = static_cast<size_t>(a.n) * std::max(wS, wZ) * 16;
    const size_t smem = lists + std::max(stage, 2 * static_cast<size_t>(table) * sizeof(int));
    // (the same limit whatever the call needs: another host thread may set it in between)
    if (smem > kCopySmem) return cudaErrorInvalidValue;
    cudaError_t e = cudaFuncSetAttribute(k_state_copy, cudaFuncAttributeMaxDynamicSharedMemorySize, kCopySmem);
    if (e != cudaSuccess) return e;
    int per_sm = 1;
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, k_state_copy, kNT, smem);
    if (e != cudaSuccess) return e;
    const int grid = std::min(nS + nZ, std::max(1, per_sm) * kNumSMs);
    TraceScope trace_("state_copy", st);
    k_state_copy<<<grid, kNT, smem, st>>>(a, wS, nS, wZ, nZ, z16, table);
    return cudaGetLastError();
}

}  // namespace slay
