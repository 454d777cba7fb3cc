// Device helpers of the 8-bit block cache (block8_*): the quantiser, the
// queries' limits, exact conversions of 8-bit codes to fp16 pairs.
#pragma once

#include <atomic>

#include "kvq_common.cuh"

namespace kvq {
namespace b8 {

constexpr float kSmallestScale = 5.421010862427522e-20f;    // 2^-64

// Largest code magnitude and its rounded reciprocal (the quantiser multiplies by it).
template <int CODE> struct Code;
template <> struct Code<KVQ_CODE_E4M3> {
    static constexpr float kInvMax = 1.0f / 448.0f;
};
template <> struct Code<KVQ_CODE_INT8> {
    static constexpr float kInvMax = 1.0f / 127.0f;
};
constexpr float kInv127 = 1.0f / 127.0f;

__device__ __forceinline__ float scale_of(float amax, float inv_max) {
    return fmaxf(__fmul_rn(amax, inv_max), kSmallestScale);
}

__device__ __forceinline__ unsigned long long f2_mul(unsigned long long a, unsigned long long b) {
    unsigned long long d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// Four codes RN(x * inv), x0's in the low byte.  No clamp is needed: |x| <= amax and inv is at most
// 1 / fp32(amax / Q), so the product stays below Q (1 + 2^-22), which rounds to Q.  int8: adding
// 1.5 2^23 rounds to a whole number (ties to even) that the low byte holds in two's complement.
// (The product and the addition are scalar: the assembler joins packed ones into one fused operation,
// which rounds otherwise.)
template <int CODE>
__device__ __forceinline__ uint32_t code_four(float x0, float x1, float x2, float x3, float inv) {
    if constexpr (CODE == KVQ_CODE_E4M3) {
        const unsigned long long inv2 = f2_pack(inv, inv);
        float y0, y1, y2, y3;
        f2_unpack(f2_mul(f2_pack(x0, x1), inv2), y0, y1);
        f2_unpack(f2_mul(f2_pack(x2, x3), inv2), y2, y3);
        uint16_t lo, hi;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(y1), "f"(y0));
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(y3), "f"(y2));
        return (uint32_t)lo | ((uint32_t)hi << 16);
    } else {
        const float magic = 12582912.0f;
        const uint32_t y0 = __float_as_uint(__fadd_rn(__fmul_rn(x0, inv), magic)),
                       y1 = __float_as_uint(__fadd_rn(__fmul_rn(x1, inv), magic)),
                       y2 = __float_as_uint(__fadd_rn(__fmul_rn(x2, inv), magic)),
                       y3 = __float_as_uint(__fadd_rn(__fmul_rn(x3, inv), magic));
        return __byte_perm(__byte_perm(y0, y1, 0x0040), __byte_perm(y2, y3, 0x0040), 0x5410);
    }
}

// Rows of the call that sequence b has; a bad entry is clamped and reported.
__device__ __forceinline__ int new_rows(const int32_t* n_new, int b, int n, uint32_t* status) {
    if (n_new == nullptr) return n;
    const int m = n_new[b];
    if (m >= 0 && m <= n) return m;
    atomicOr(status, kDevCheck);
    return m < 0 ? 0 : n;
}

// Tokens of a unit with count tokens that query t of m sees.
__device__ __forceinline__ int query_limit(int count, int m, int t) { return t < m ? max(0, count - m + t + 1) : 0; }

// Key of a score for top-k: NaN above everything, -0 equal to +0.
__device__ __forceinline__ uint32_t rank_key(float f) {
    if (isnan(f)) return 0xffffffffu;
    const uint32_t u = __float_as_uint(f + 0.0f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Work units 0 .. works - 1 of tiles(i) tiles each, as one list of places that is cut into equal runs
// for the grid's CTAs, whatever the units' sizes (known on the device only): every CTA adds all of them
// up.  Starting on a unit costs a CTA the time of about eight tiles (counters, table, first tile).  So
//  - where the grid has a CTA for every `least` tiles of every unit, a unit's tiles are filled up to a
//    multiple of `least` places and a run is `least` places: no CTA comes to a second unit (32 ragged
//    units of up to 64 tokens 14.6 -> 7.1 us);
//  - else a unit's first tile stands behind `start` places without work, at most a quarter of a CTA's
//    tiles (attn of 32 units of 4096 tokens 15.2 -> 13.4 us, ragged 256 units 58 -> 56).
template <int LEAST>
struct Run {
    int from, to;               // the CTA's places in the list
    int work, before;           // unit of the first place, and the places ahead of that unit
    bool whole;                 // the first of the two ways
    int start;                  // places ahead of a unit's tiles
    int per;                    // places per CTA (CTA c: [c per, c per + per))

    __device__ __forceinline__ int places(int tiles) const {
        return whole ? (tiles + LEAST - 1) / LEAST * LEAST : tiles > 0 ? start + tiles : 0;
    }
};
template <int THREADS>
struct RunShared {
    int scan[THREADS / 32][3];
    int at[2];
};

// The whole CTA calls this.
template <int THREADS, int LEAST, typename TilesFn>
__device__ __forceinline__ Run<LEAST> find_run(int works, TilesFn tiles, RunShared<THREADS>& sh) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int each = (works + THREADS - 1) / THREADS, w0 = min((int)threadIdx.x * each, works), w1 = min(w0 + each, works);
    int sum[3] = {0, 0, 0};                     // tiles, units that have any, runs of LEAST tiles
    for (int i = w0; i < w1; ++i) {
        const int n = tiles(i);
        sum[0] += n;
        sum[1] += n > 0 ? 1 : 0;
        sum[2] += (n + LEAST - 1) / LEAST;
    }
    int incl[3] = {sum[0], sum[1], sum[2]};
#pragma unroll
    for (int o = 1; o < 32; o <<= 1)
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            const int x = __shfl_up_sync(0xffffffffu, incl[k], o);
            if (lane >= o) incl[k] += x;
        }
    if (lane == 31)
#pragma unroll
        for (int k = 0; k < 3; ++k) sh.scan[warp][k] = incl[k];
    __syncthreads();
    int all[3] = {0, 0, 0};
#pragma unroll
    for (int i = 0; i < THREADS / 32; ++i)
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            const int x = sh.scan[i][k];
            if (i < warp) incl[k] += x;
            all[k] += x;
        }
    const int grid = (int)gridDim.x;
    const bool whole = all[2] <= grid;
    Run<LEAST> r;
    r.whole = whole;
    r.start = whole ? 0 : min(8, all[0] / grid / 4);
    const int list = whole ? all[2] * LEAST : all[0] + r.start * all[1];
    r.per = max((list + grid - 1) / grid, LEAST);
    r.from = (int)min((long long)blockIdx.x * r.per, (long long)list);
    r.to = min(r.from + r.per, list);
    int at = whole ? (incl[2] - sum[2]) * LEAST : incl[0] - sum[0] + r.start * (incl[1] - sum[1]);
    const int own = whole ? sum[2] * LEAST : sum[0] + r.start * sum[1];
    if (r.from < list && r.from >= at && r.from < at + own) {
        int i = w0;
        for (;; ++i) {
            const int p = r.places(tiles(i));
            if (r.from < at + p) break;
            at += p;
        }
        sh.at[0] = i;
        sh.at[1] = at;
    }
    __syncthreads();
    r.work = sh.at[0];
    r.before = sh.at[1];
    return r;
}

// CTAs of the kernel that the current device holds at once.
template <typename K>
inline cudaError_t resident_ctas(K kernel, int threads, size_t smem, std::atomic<int>* known, int* out) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 64 && (*out = known[dev].load(std::memory_order_relaxed)) > 0) return cudaSuccess;
    int sms = 0, per = 0;
    e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kernel, threads, smem);
    if (e != cudaSuccess) return e;
    *out = sms * per > 0 ? sms * per : 1;
    if (dev < 64) known[dev].store(*out, std::memory_order_relaxed);
    return cudaSuccess;
}

// 16 bytes that are read once.
__device__ __forceinline__ uint4 load16(const uint8_t* p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}
// Four codes as two fp16 pairs, exactly.  int8: the byte with its sign bit flipped, under the
// exponent of 1024, is 1152 + code.
template <int CODE>
__device__ __forceinline__ void to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
    if constexpr (CODE == KVQ_CODE_E4M3) {
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(lo) : "h"((uint16_t)w));
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(hi) : "h"((uint16_t)(w >> 16)));
    } else {
        const uint32_t x = w ^ 0x80808080u;
        const __half2 bias = __half2half2(__ushort_as_half(0x6480));
        uint32_t l = __byte_perm(x, 0x64646464u, 0x4140), h = __byte_perm(x, 0x64646464u, 0x4342);
        __half2 a = __hsub2(*reinterpret_cast<__half2*>(&l), bias), b = __hsub2(*reinterpret_cast<__half2*>(&h), bias);
        lo = *reinterpret_cast<uint32_t*>(&a);
        hi = *reinterpret_cast<uint32_t*>(&b);
    }
}

__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

}  // namespace b8
}  // namespace kvq
