// prefill_attn_bwd: gradients of q, k and v through prefill_attn_scores' o and lse, the probabilities recomputed.
//
//   P_ij = exp(sigma q_i.k_j - lse_i) for j <= i, 0 above;   delta_i = do_i.o_i - dlse_i
//   dS_ij = P_ij (do_i.v_j - delta_i)
//   dV_j = sum_i P_ij do_i;   dK_j = sigma sum_i dS_ij q_i;   dQ_i = sigma sum_j dS_ij k_j
//
// Two kernels over 128 x 128 tiles, so that every sum stays in one CTA's tensor memory (where key tiles are few, a
// cluster's, added up in the order of its CTAs) in a fixed order: no atomics, no float32 buffer, and a call repeats itself
// bit for bit.  The price is that S and dO V^T are computed in both (seven products for the five of the formulas).
//   dkv: CTA = (KV head, key tile), over the query heads of its group and their query tiles at and below the diagonal,
//        S^T = K Q^T, dP^T = V dO^T, then dV += P^T dO and dK += dS^T Q with P^T and dS^T read from tensor memory.
//   dq:  CTA = (query head, query tile), over the key tiles up to the diagonal: S = Q K^T, dP = dO V^T, dQ += dS K.
// Sixteen warps do the exponentials and dS (four warpgroups, each a quarter of a tile's columns), one warp issues the
// copies, one the products, in dkv one brings the rows' lse and delta.
// A first kernel computes delta and brings lse to base 2.
//
// Rounding: P and dS enter their products in the inputs' type, which the products take: up to half a step of each term
// (2^-8 in bf16), as much as the output's own rounding; against float64 a gradient is off by 2.4e-3 in bf16 and 2.9e-4 in
// fp16, where one computed in float32 and rounded at the end is off by 1.7e-3 and 2.1e-4.  fp16 has a problem of range
// besides: P of long rows and dS of small gradients fall below its normal numbers.  So P is kept times 2^15 (P <= 1) and
// dS times a power of two c as well, so that |do_i.v_j - delta_i| c <= 1 by |do_i|, |v_j| (2-norms) and |delta_i|: for dK,
// whose sums run over rows, one c for a key tile, from the rows of its query tiles; for dQ one for each row, from
// |delta_i| and its |do_i|, which the first kernel leaves as four bits below its tile's largest.  The sums' factors are
// undone in the epilogue.  (With one c for a head, dq of rows whose do is 2^16 below the largest was off by 6e-4 at 4096
// tokens and 2e-3 at 16384; 3e-4 now, as for all rows.)
//
// Bound: the tensor pipe and in dkv at D = 128 the waits between its products, and for large calls the card's power.  A tile
// of 128 x 128 pairs at D = 128 takes about 2600 clocks in dkv (products 2048) and 1800 in dq (1536).  4 x 32/8 heads x
// 4096 tokens: 1320 us, 1.04 PFLOP/s of the five products, 1.46 of the seven; 8/2 x 16384: 1235 us, 1.11 and 1.56.  At
// D = 64 the softmax warps are the longer side: 8 x 16 heads x 2048 tokens 322 us.
//
// Every mbarrier wait is bounded; a CTA that gives up drains its copies and products, frees TMEM, stores nothing and
// records KVQ_ETIMEOUT in the device status word.
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "grad_device.cuh"
#include "kvq_common.cuh"
#include "kvq_internal.h"
#include "prefill_tiles.cuh"

namespace kvq {

KVQ_DEFINE_STATUS(prefill_bwd)

namespace {

constexpr int kSoftWarps = 16;                        // four warpgroups, each a quarter of a tile's columns
constexpr int kDkvThreads = 32 * (kSoftWarps + 3);   // + copies, products, row statistics
constexpr int kDqThreads = 32 * (kSoftWarps + 2);
constexpr int kPrepThreads = 256;
constexpr uint32_t kTmemCols = 512;

// What the first kernel leaves in the workspace (n_t tiles, Tp = 128 n_t rows a head).
struct BwdWs {
    float* nlse;        // [B*Hq][Tp] minus lse in base 2, plus the probabilities' shift; -inf behind the last row
    float* delta;       // [B*Hq][Tp]
    float* do_max;      // [B*Hq][n_t] largest 2-norm of a row of do        (fp16 only, also the next three)
    float* dl_max;      // [B*Hq][n_t] largest |delta|
    float* v_max;       // [B*Hkv][n_t] largest 2-norm of a row of v
    uint32_t* below;    // [B*Hq][n_t][16] four bits a row, row 0 the lowest: its do's 2-norm is at most do_max 2^-bits
};

struct BwdArgs {
    BwdWs ws;
    int B, Hq, Hkv, T_len, n_t;
    float sm_scale, scale_log2;
    int group;          // heads (dkv: KV heads) whose tiles are launched side by side
    int split;          // dkv: CTAs of a cluster that share a tile's query tiles
};

// Bounded wait of a whole warp, the same outcome in every lane; the loop is kept out of the callers' code.
__device__ __noinline__ bool bwd_wait_on(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag)) != 0;
}
__device__ __forceinline__ bool bwd_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    return bwd_wait_on(bar, parity, abort_flag);
}

__device__ __forceinline__ void bwd_give_up(volatile int* abort_flag) {
    *abort_flag = 1;
    atomicOr(&g_status_prefill_bwd, kDevTimeout);
}

template <int N> using Int = std::integral_constant<int, N>;

// Probabilities are kept times 2^kShift.
template <int AB> struct Shift { static constexpr float value = AB == 0 ? 15.0f : 0.0f; };

// ------------------------------------------------------------------ row statistics

// CTA = (tile of 128 rows, query head); D / 8 lanes of 16 bytes per row.
template <typename T, int AB, int D>
__global__ void __launch_bounds__(kPrepThreads)
    bwd_prep_kernel(const T* __restrict__ o, const T* __restrict__ go, const T* __restrict__ v,
                    const float* __restrict__ lse, const float* __restrict__ glse, const BwdArgs a) {
    constexpr int kLanes = D / 8, kRows = kPrepThreads / kLanes;
    grid_launch_dependents();
    const int tile = (int)blockIdx.x % a.n_t, bh = (int)blockIdx.x / a.n_t;
    const int b = bh / a.Hq, hq = bh % a.Hq, g = a.Hq / a.Hkv;
    const int l = threadIdx.x % kLanes, sub = threadIdx.x / kLanes;
    const int64_t Tp = (int64_t)a.n_t * kTile;
    const bool with_v = AB == 0 && hq % g == 0;
    const int u = b * a.Hkv + hq / g;
    float most_do = 0.0f, most_dl = 0.0f, most_v = 0.0f;
    __shared__ float row_sq[AB == 0 ? kTile : 1];       // the rows' |do|^2
#pragma unroll 4
    for (int r0 = 0; r0 < kTile; r0 += kRows) {
        const int i = tile * kTile + r0 + sub;
        const bool there = i < a.T_len;
        float dot = 0.0f, sq = 0.0f, vv = 0.0f;
        if (there) {
            const int64_t at = ((int64_t)bh * a.T_len + i) * kLanes + l;
            const uint4 x = reinterpret_cast<const uint4*>(o)[at], y = reinterpret_cast<const uint4*>(go)[at];
            const T *xe = reinterpret_cast<const T*>(&x), *ye = reinterpret_cast<const T*>(&y);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float d = Elem<T>::to_f(ye[e]);
                dot = fmaf(Elem<T>::to_f(xe[e]), d, dot);
                sq = fmaf(d, d, sq);
            }
            if (with_v) {
                const uint4 z = reinterpret_cast<const uint4*>(v)[((int64_t)u * a.T_len + i) * kLanes + l];
                const T* ze = reinterpret_cast<const T*>(&z);
#pragma unroll
                for (int e = 0; e < 8; ++e) vv = fmaf(Elem<T>::to_f(ze[e]), Elem<T>::to_f(ze[e]), vv);
            }
        }
#pragma unroll
        for (int m = kLanes / 2; m > 0; m >>= 1) {
            dot += __shfl_xor_sync(0xffffffffu, dot, m);
            if (AB == 0) sq += __shfl_xor_sync(0xffffffffu, sq, m);
            if (AB == 0) vv += __shfl_xor_sync(0xffffffffu, vv, m);
        }
        float nl = -__int_as_float(0x7f800000), dl = 0.0f;
        if (there) {
            const int64_t row = (int64_t)bh * a.T_len + i;
            dl = dot - (glse ? glse[row] : 0.0f);
            const float x = lse[row];
            if (!isinf(x)) nl = Shift<AB>::value - x * kLog2e;
            else dl = sq = 0.0f;                                    // a row that saw nothing has no gradient
        }
        if (l == 0) {
            a.ws.nlse[bh * Tp + i] = nl;
            a.ws.delta[bh * Tp + i] = dl;
            if (AB == 0) row_sq[r0 + sub] = sq;
        }
        if (AB == 0) {
            most_do = fmaxf(most_do, sq), most_dl = fmaxf(most_dl, fabsf(dl)), most_v = fmaxf(most_v, vv);
        }
    }
    if (AB == 0) {
        __shared__ float red[kPrepThreads / 32][3];
        __shared__ uint32_t bits[kTile / 8];
        if (threadIdx.x < kTile / 8) bits[threadIdx.x] = 0;
#pragma unroll
        for (int m = 16; m > 0; m >>= 1) {
            most_do = fmaxf(most_do, __shfl_xor_sync(0xffffffffu, most_do, m));
            most_dl = fmaxf(most_dl, __shfl_xor_sync(0xffffffffu, most_dl, m));
            most_v = fmaxf(most_v, __shfl_xor_sync(0xffffffffu, most_v, m));
        }
        if ((threadIdx.x & 31) == 0) {
            float* x = red[threadIdx.x >> 5];
            x[0] = most_do, x[1] = most_dl, x[2] = most_v;
        }
        __syncthreads();
        for (int w = 0; w < kPrepThreads / 32; ++w) {
            most_do = fmaxf(most_do, red[w][0]), most_dl = fmaxf(most_dl, red[w][1]), most_v = fmaxf(most_v, red[w][2]);
        }
        if (threadIdx.x < kTile) {
            const float ratio = most_do / row_sq[threadIdx.x];      // of squares; infinite or NaN for a row of zeros
            const uint32_t b = ratio < 0x1p30f ? (uint32_t)ilogbf(fmaxf(ratio, 1.0f)) / 2 : 15;
            atomicOr(&bits[threadIdx.x / 8], b << (4 * (threadIdx.x & 7)));
        }
        __syncthreads();
        if (threadIdx.x < kTile / 8)
            a.ws.below[((int64_t)bh * a.n_t + tile) * (kTile / 8) + threadIdx.x] = bits[threadIdx.x];
        if (threadIdx.x == 0) {
            a.ws.do_max[(int64_t)bh * a.n_t + tile] = sqrtf(most_do);
            a.ws.dl_max[(int64_t)bh * a.n_t + tile] = most_dl;
            if (with_v) a.ws.v_max[(int64_t)u * a.n_t + tile] = sqrtf(most_v);
        }
    }
}

// The power of two c with `most` c <= 1, most >= |do_i.v_j - delta_i| (fp16; else 1).
template <int AB> __device__ __forceinline__ float ds_scale(float most) {
    if (AB != 0 || !(most > 0.0f)) return 1.0f;
    const int e = most < 1e30f ? min(max(ilogbf(most) + 1, -60), 60) : 60;
    return __int_as_float((127 - e) << 23);
}

__device__ __forceinline__ float warp_most(float x) {
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, m));
    return x;
}

// That of key tile kt of unit u and the query tiles at and below it of the nh query heads from h0 on, by a warp.
template <int AB> __device__ __forceinline__ float key_tile_scale(const BwdArgs& a, int h0, int nh, int u, int kt, int lane) {
    if (AB != 0) return 1.0f;
    float x = 0.0f, d = 0.0f;
    for (int h = 0; h < nh; ++h) {
#pragma unroll 4
        for (int i = kt + lane; i < a.n_t; i += 32) {
            x = fmaxf(x, __ldcg(a.ws.do_max + (int64_t)(h0 + h) * a.n_t + i));
            d = fmaxf(d, __ldcg(a.ws.dl_max + (int64_t)(h0 + h) * a.n_t + i));
        }
    }
    return ds_scale<AB>(fmaf(warp_most(x), __ldcg(a.ws.v_max + (int64_t)u * a.n_t + kt), warp_most(d)));
}

// The largest |do_i| |v_j| of query tile qt of head bh with its keys, by a warp.
__device__ __forceinline__ float query_tile_most(const BwdArgs& a, int bh, int u, int qt, int lane) {
    float v = 0.0f;
#pragma unroll 4
    for (int i = lane; i <= qt; i += 32) v = fmaxf(v, __ldcg(a.ws.v_max + (int64_t)u * a.n_t + i));
    return __ldcg(a.ws.do_max + (int64_t)bh * a.n_t + qt) * warp_most(v);
}

// block -> (tile rank, head): heads in groups, all tiles of a group before the next group, the longest tiles of
// every head first.  A group's streamed operands stay in L2 while its CTAs run.
__device__ __forceinline__ void place(const BwdArgs& a, int block, int heads, int& rank, int& head) {
    const int per = a.group * a.n_t, g = block / per, in = block % per;
    const int size = min(a.group, heads - g * a.group);
    rank = in / size;
    head = g * a.group + in % size;
}

// Shared memory of both kernels: dkv has K, V, three stages of Q and two of dO; dq has dO, four stages of K (from A1 on)
// and two of V.
template <int D> struct BwdLayout {
    static constexpr uint32_t kTileBytes = kTile * D * 2;
    static constexpr uint32_t A0 = 0, A1 = kTileBytes;
    static constexpr uint32_t S0 = 2 * kTileBytes;
    static constexpr uint32_t S1 = S0 + 3 * kTileBytes;
    static constexpr uint32_t STAT = S1 + 2 * kTileBytes;       // dkv: 2 stages of 128 (nlse) and 128 (delta) floats
    static constexpr uint32_t SCALE = STAT + 2048;              // dkv: key_tile_scale(); dq: query_tile_most()
    static constexpr uint32_t BAR = SCALE + 16;
    // no alignment slack at D = 128: the kernels require (and check) a 1024-aligned base
    static constexpr uint32_t BYTES = BAR + 256;
};
static_assert(BwdLayout<128>::BYTES <= 232448, "shared memory");

// C = A B^T of two K-major tiles of 128 rows (one thread).
template <int D> __device__ __forceinline__ void products_k(uint32_t c, uint32_t ta, uint32_t tb, uint32_t idesc) {
    const uint64_t da = kmajor_desc(ta, 0), db = kmajor_desc(tb, 0);
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
        const uint64_t off = ((uint32_t)(kk >> 2) * kHalfBytes + (uint32_t)(kk & 3) * 32u) >> 4;
        tc_mma_f16(c, da + off, db + off, idesc, kk > 0);
    }
}

// The same with A packed in tensor memory.
template <int D> __device__ __forceinline__ void products_k_ta(uint32_t c, uint32_t ta, uint32_t tb, uint32_t idesc) {
    const uint64_t db = kmajor_desc(tb, 0);
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
        const uint64_t off = ((uint32_t)(kk >> 2) * kHalfBytes + (uint32_t)(kk & 3) * 32u) >> 4;
        tc_mma_f16_ta(c, ta + (uint32_t)kk * 8u, db + off, idesc, kk > 0);
    }
}

// C (+)= A B, A [128, 128] packed pairs in tensor memory (every 32 values in 16 columns, STEP columns apart), B a tile of
// 128 rows (one thread).
template <int STEP>
__device__ __forceinline__ void products_mn(uint32_t c, uint32_t ta, uint32_t tb, uint32_t idesc, bool accumulate) {
    const uint64_t db = mnmajor_desc(tb, 0);
#pragma unroll
    for (int kk = 0; kk < 8; ++kk)
        tc_mma_f16_ta(c, ta + (uint32_t)(kk >> 1) * STEP + (uint32_t)(kk & 1) * 8u, db + (uint64_t)(kk * 16 * 128 >> 4), idesc,
                      kk > 0 || accumulate);
}

// 32 values of a thread's row as 16 columns of packed pairs.
template <typename T> __device__ __forceinline__ void store_pairs(uint32_t taddr, const float* x) {
    uint32_t w[16];
#pragma unroll
    for (int c = 0; c < 16; ++c) w[c] = Pack2<T>::pack(x[2 * c], x[2 * c + 1]);
    tmem_st16(taddr, w);
}

// A warp's 32 keys by 32 queries, as [16 queries][16 keys][tile of 8 queries][8 keys][2 queries] a thread, and their pairs
// in the first 16 of the 32 columns.
__device__ __forceinline__ void load_frags(uint32_t taddr, float* x) {
    tmem_ld_frag16(taddr, x);
    tmem_ld_frag16(taddr + (16u << 16), x + 8);
    tmem_ld_frag16(taddr + 16u, x + 16);
    tmem_ld_frag16(taddr + 16u + (16u << 16), x + 24);
    tmem_wait_ld();
}
__device__ __forceinline__ void store_frags(uint32_t taddr, const uint32_t* w) {
    tmem_st_frag8(taddr, w);
    tmem_st_frag8(taddr + (16u << 16), w + 4);
    tmem_st_frag8(taddr + 8u, w + 8);
    tmem_st_frag8(taddr + 8u + (16u << 16), w + 12);
    tmem_wait_st();
}

// Zeros where the query comes before the key, in a thread's 16 keys by 16 queries; d: query - key of element 0.
__device__ __forceinline__ void mask16(float* x, int d) {
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = d + 8 * ((i >> 2) & 1) + (i & 1) - 16 * (i >> 3) - 8 * ((i >> 1) & 1) >= 0 ? x[i] : 0.0f;
}

// N float32 TMEM columns of a thread's row (lane r), times f, in T to a 64-column half of a swizzled tile in shared memory,
// from its column c0 on.
template <typename T, int N>
__device__ __forceinline__ void stage_row(uint32_t taddr, float f, uint8_t* half, int r, int c0) {
    uint8_t* row = half + r * 128;
#pragma unroll
    for (int c4 = 0; c4 < N / 32; ++c4) {
        float x[32];
        tmem_ld32(taddr + (uint32_t)c4 * 32u, x);
        tmem_wait_ld();
#pragma unroll
        for (int c8 = 0; c8 < 4; ++c8) {
            uint4 w;
            w.x = Pack2<T>::pack(x[c8 * 8 + 0] * f, x[c8 * 8 + 1] * f);
            w.y = Pack2<T>::pack(x[c8 * 8 + 2] * f, x[c8 * 8 + 3] * f);
            w.z = Pack2<T>::pack(x[c8 * 8 + 4] * f, x[c8 * 8 + 5] * f);
            w.w = Pack2<T>::pack(x[c8 * 8 + 6] * f, x[c8 * 8 + 7] * f);
            *reinterpret_cast<uint4*>(row + ((c0 / 8 + c4 * 4 + c8) ^ (r & 7)) * 16) = w;
        }
    }
}

// ------------------------------------------------------------------ dK and dV

enum DkvBar { V_KV = 0, V_QF = 1, V_QE = 4, V_GF = 7, V_GE = 9, V_TF = 11, V_TE = 13, V_SF = 15, V_PR = 16, V_DF = 17,
              V_DR = 18, V_END = 19, DKV_NBAR = 20 };

template <typename T, int AB, int D>
__global__ void __launch_bounds__(kDkvThreads, 1)
    bwd_dkv_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                   const __grid_constant__ CUtensorMap tv, const __grid_constant__ CUtensorMap tg,
                   const __grid_constant__ CUtensorMap tdk, const __grid_constant__ CUtensorMap tdv, T* __restrict__ dk,
                   T* __restrict__ dv, const BwdArgs a) {
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t base = smem_u32(smem);
    if (base & 1023u) {                                 // layout assumption broken: do nothing
        if (threadIdx.x == 0) atomicOr(&g_status_prefill_bwd, kDevCheck);
        return;
    }
    using Lay = BwdLayout<D>;
    constexpr uint32_t kTileBytes = Lay::kTileBytes;
    constexpr int kHalves = D / 64;
    const uint32_t sK = base + Lay::A0, sV = base + Lay::A1, sQ = base + Lay::S0, sG = base + Lay::S1;
    auto BAR = [&](int i) -> uint32_t { return base + Lay::BAR + 8u * (uint32_t)i; };
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Lay::BAR + 8 * DKV_NBAR);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Lay::BAR + 8 * DKV_NBAR + 4);
    float* scale = reinterpret_cast<float*>(smem + Lay::SCALE);

    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    int kt, u;
    place(a, (int)blockIdx.x / a.split, a.B * a.Hkv, kt, u);
    const int g = a.Hq / a.Hkv, h0 = u * g;             // head u * g + h of all B * Hq is the unit's h-th
    if (threadIdx.x == 0) prefetch_tmap(&tk), prefetch_tmap(&tq), prefetch_tmap(&tv), prefetch_tmap(&tg);
    // query tiles of a head; tiles of all heads, of which this CTA of the cluster has n from `from` on
    const int m = a.n_t - kt, mine_of = (int)blockIdx.x % a.split, from = g * m * mine_of / a.split;
    const int n = g * m * (mine_of + 1) / a.split - from;

    // (one lane) tile it of Q or dO into its stage
    auto load_q = [&](int it) {
        const int s = it % 3;
        mbar_expect_tx(BAR(V_QF + s), kTileBytes);
        for (int hf = 0; hf < kHalves; ++hf)
            tma_load_3d(sQ + s * kTileBytes + hf * kHalfBytes, &tq, 64 * hf, (kt + (from + it) % m) * kTile, h0 + (from + it) / m,
                        BAR(V_QF + s));
    };
    auto load_g = [&](int it) {
        const int s = it & 1;
        mbar_expect_tx(BAR(V_GF + s), kTileBytes);
        for (int hf = 0; hf < kHalves; ++hf)
            tma_load_3d(sG + s * kTileBytes + hf * kHalfBytes, &tg, 64 * hf, (kt + (from + it) % m) * kTile, h0 + (from + it) / m,
                        BAR(V_GF + s));
    };
    if (warp == kSoftWarps) {
        // a lane per barrier; the softmax warps all arrive at some
        constexpr uint32_t kMany = 1u << V_TE | 1u << (V_TE + 1) | 1u << V_PR | 1u << V_DR;
        if (lane < DKV_NBAR) mbar_init(BAR(lane), kMany >> lane & 1 ? kSoftWarps : 1);
        if (lane == 0) *abort_flag = 0;
        fence_mbar_init();
    }
    __syncwarp();
    if (warp == kSoftWarps && lane == 0) {
        // the first copies do not wait for the rest of the CTA, nor for the grid before this one
        if (n > 0) {
            mbar_expect_tx(BAR(V_KV), 2 * kTileBytes);
            for (int hf = 0; hf < kHalves; ++hf) tma_load_3d(sK + hf * kHalfBytes, &tk, 64 * hf, kt * kTile, u, BAR(V_KV));
            load_q(0);
            for (int hf = 0; hf < kHalves; ++hf) tma_load_3d(sV + hf * kHalfBytes, &tv, 64 * hf, kt * kTile, u, BAR(V_KV));
            load_g(0);
        }
    }
    if (warp == kSoftWarps + 1) tmem_alloc(smem_u32(tmem_slot), kTmemCols);
    grid_dependency_wait();                             // the rows' statistics
    grid_launch_dependents();                           // dQ's CTAs take the SMs that this grid leaves free
    float4 stat_l = make_float4(0.0f, 0.0f, 0.0f, 0.0f), stat_d = stat_l;   // of the lane's four rows, a tile ahead
    auto load_stat = [&](int it) {
        const int64_t row = (int64_t)(h0 + (from + it) / m) * a.n_t * kTile + (kt + (from + it) % m) * kTile + 4 * lane;
        stat_l = *reinterpret_cast<const float4*>(a.ws.nlse + row);
        stat_d = *reinterpret_cast<const float4*>(a.ws.delta + row);
    };
    if (warp == kSoftWarps + 2 && n > 0) load_stat(0);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
    // S^T, dP^T, dV, dK; packed P^T and dS^T beside them at D = 64 (32 queries in 16 columns), at D = 128, where tensor
    // memory has no more room, in their place (32 queries in the first 16 of their 32 columns)
    constexpr bool kBeside = D == 64;
    constexpr uint32_t kStep = kBeside ? 16 : 32;
    const uint32_t tS = tmem, tP = tmem + 128, tDV = tmem + 256, tDK = tmem + 256 + D;
    const uint32_t tPw = kBeside ? tmem + 384 : tS, tDw = kBeside ? tmem + 448 : tP;

    if (warp == kSoftWarps) {
        if (lane == 0 && n > 0) {
            int it = 1, lastq[3] = {0, -1, -1}, lastg[2] = {0, -1};
            for (; it < n; ++it) {
                if (it >= 3 && !mbar_wait(BAR(V_QE + it % 3), (it / 3 - 1) & 1, abort_flag)) break;
                load_q(it);
                lastq[it % 3] = it / 3;
                if (it >= 2 && !mbar_wait(BAR(V_GE + (it & 1)), (it / 2 - 1) & 1, abort_flag)) break;
                load_g(it);
                lastg[it & 1] = it / 2;
            }
            if (it < n) bwd_give_up(abort_flag);
            // every issued copy has landed before the CTA may exit
            mbar_wait(BAR(V_KV), 0, nullptr);
            for (int s = 0; s < 3; ++s)
                if (lastq[s] >= 0) mbar_wait(BAR(V_QF + s), lastq[s] & 1, nullptr);
            for (int s = 0; s < 2; ++s)
                if (lastg[s] >= 0) mbar_wait(BAR(V_GF + s), lastg[s] & 1, nullptr);
        }
    } else if (warp == kSoftWarps + 1) {
        constexpr uint32_t idS = idesc_f16(AB, 128, 128, 0), idD = idesc_f16(AB, 128, D, 1);
        // (one lane) S^T = K Q^T, dP^T = V dO^T with the streamed tile in stage s
        auto scores = [&](int s) {
            products_k<D>(tS, sK, sQ + (uint32_t)s * kTileBytes, idS);
            tc_commit(BAR(V_SF));
        };
        auto grads = [&](int s) {
            products_k<D>(tP, sV, sG + (uint32_t)s * kTileBytes, idS);
            tc_commit(BAR(V_DF));
        };
        auto wait = [&](int bar, int parity) { return mbar_wait(BAR(bar), (uint32_t)(parity & 1), abort_flag); };
        auto q_there = [&](int it, int s) { return wait(V_QF + s, it / 3); };
        auto g_there = [&](int it, int s) { return wait(V_GF + s, it / 2); };
        // One tile, PH = it mod 6: the stages are constants, so that descriptors stay in uniform registers (computed from
        // the tile's number they made a product's issue three times as long).
        // The next S^T and dP^T are issued behind dV and dK.  Only products of one sum are sure to run in the order of their
        // issue, so what replaces an operand in tensor memory waits until the product that reads it is done.  At D = 64 that
        // costs nothing: P^T and dS^T lie beside S^T and dP^T, and the softmax warps write the next ones after V_SF and V_DF,
        // whose commits cover the dV and dK before them.  At D = 128 they lie in the place of S^T and dP^T, and the issuing
        // lane waits (4 x 32/8 x 4096: 5 % of the call; dK before the next S^T, so that the pipe has work during the waits:
        // 8 %, the softmax warps then have too little time).
        // A wait costs one to three products' time even where there is nothing to wait for, and the tensor pipe has about
        // four products ahead of it: else no two waits follow one another without products between.
        auto step = [&](auto phase, int it) -> bool {
            constexpr int PH = decltype(phase)::value, q0 = PH % 3, q1 = (PH + 1) % 3, q2 = (PH + 2) % 3, g0 = PH & 1, g1 = g0 ^ 1;
            const bool more = it + 1 < n;
            if (!wait(V_PR, PH)) return false;
            tc_fence_after();
            products_mn<kStep>(tDV, tPw, sG + (uint32_t)g0 * kTileBytes, idD, it > 0);      // dV += P^T dO
            tc_commit(BAR(V_GE + g0));
            if (more) {
                if (!g_there(it + 1, g1) || (!kBeside && !wait(V_GE + g0, it / 2))) return false;
                scores(q1);
            }
            if (!wait(V_DR, PH)) return false;
            tc_fence_after();
            products_mn<kStep>(tDK, tDw, sQ + (uint32_t)q0 * kTileBytes, idD, it > 0);      // dK += dS^T Q
            tc_commit(BAR(V_QE + q0));
            if (it + 2 < n && !q_there(it + 2, q2)) return false;
            if (more) {
                if (!kBeside && !wait(V_QE + q0, it / 3)) return false;
                grads(g1);
            }
            return true;
        };
        if (elect_one()) {
            bool ok = n == 0 || (wait(V_KV, 0) && q_there(0, 0) && g_there(0, 0) && (n == 1 || q_there(1, 1)));
            if (ok && n > 0) scores(0), grads(0);
            for (int it = 0; ok && it < n; it += 6) {
                ok = step(Int<0>{}, it) && (it + 1 >= n || step(Int<1>{}, it + 1)) && (it + 2 >= n || step(Int<2>{}, it + 2)) &&
                     (it + 3 >= n || step(Int<3>{}, it + 3)) && (it + 4 >= n || step(Int<4>{}, it + 4)) &&
                     (it + 5 >= n || step(Int<5>{}, it + 5));
            }
            if (!ok) bwd_give_up(abort_flag);
            // all products complete before the sums are read and TMEM is released
            tc_commit(BAR(V_END));
            mbar_wait(BAR(V_END), 0, nullptr);
        }
        __syncwarp();
    } else if (warp == kSoftWarps + 2) {
        // the scale, and the query rows' statistics, delta times it
        const float c = key_tile_scale<AB>(a, h0, g, u, kt, lane);
        if (lane == 0) *scale = c;
        bool ok = true;
        for (int it = 0; it < n; ++it) {
            const int s = it & 1;
            const float4 x = stat_l;
            const float4 y = make_float4(-c * stat_d.x, -c * stat_d.y, -c * stat_d.z, -c * stat_d.w);
            if (it + 1 < n) load_stat(it + 1);
            if (it >= 2 && !(ok = bwd_wait(BAR(V_TE + s), (it / 2 - 1) & 1, abort_flag))) break;
            float4* to = reinterpret_cast<float4*>(smem + Lay::STAT + s * 1024);
            to[lane] = x;
            to[32 + lane] = y;
            __syncwarp();
            if (lane == 0) mbar_arrive(BAR(V_TF + s));
        }
        if (!ok) bwd_give_up(abort_flag);
    } else {
        // Warpgroup wg has queries 32 wg .. 32 wg + 31 of each tile, warp w of it keys 32 w .. 32 w + 31, in fragments: a
        // thread has 4 keys and 8 queries, so that it needs the statistics of 8 queries only (with a thread per key the
        // broadcasts of 32 took as many cycles of shared memory as the tensor pipe's operands left).
        const int wg = warp >> 2, r = threadIdx.x & 127;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t mine = lanes + 32u * (uint32_t)wg, packed = lanes + kStep * (uint32_t)wg;
        const int first = 32 * wg + 2 * (lane & 3) - (32 * (warp & 3) + (lane >> 2));    // query - key of element 0
        const unsigned long long sc2 = f2_pack(a.scale_log2, a.scale_log2);
        float c = 1.0f;
        bool ok = true;
        for (int it = 0; it < n; ++it) {
            const int s = it & 1;
            const bool diag = (from + it) % m == 0;
            if (!bwd_wait(BAR(V_TF + s), (it / 2) & 1, abort_flag)) { ok = false; break; }
            if (AB == 0 && it == 0) c = *scale;         // written before the first statistics
            const unsigned long long c2 = f2_pack(c, c);
            const unsigned long long* stat =
                reinterpret_cast<const unsigned long long*>(smem + Lay::STAT + s * 1024 + 128 * wg) + (lane & 3);
            unsigned long long nl[4], nd[4];
#pragma unroll
            for (int t = 0; t < 4; ++t) nl[t] = stat[4 * t], nd[t] = stat[64 + 4 * t];
            if (!bwd_wait(BAR(V_SF), it & 1, abort_flag)) { ok = false; break; }
            tc_fence_after();
            float p[32];                                // [16 queries][16 keys][tile of 8 queries][8 keys][2 queries]
            uint32_t w[16];
            load_frags(tS + mine, p);
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
                float e0, e1;
                f2_unpack(f2_fma(f2_pack(p[i], p[i + 1]), sc2, nl[2 * (i >> 4) + ((i >> 2) & 1)]), e0, e1);
                p[i] = ex2_approx(e0), p[i + 1] = ex2_approx(e1);
            }
            if (diag) mask16(p, first), mask16(p + 16, first + 16);
#pragma unroll
            for (int i = 0; i < 16; ++i) w[i] = Pack2<T>::pack(p[2 * i], p[2 * i + 1]);
            store_frags(tPw + packed, w);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(BAR(V_PR));
            if (!bwd_wait(BAR(V_DF), it & 1, abort_flag)) { ok = false; break; }
            tc_fence_after();
            float d[32];
            load_frags(tP + mine, d);
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
                f2_unpack(f2_mul(f2_pack(p[i], p[i + 1]),
                                 f2_fma(f2_pack(d[i], d[i + 1]), c2, nd[2 * (i >> 4) + ((i >> 2) & 1)])),
                          d[i], d[i + 1]);
            }
            if (diag) mask16(d, first), mask16(d + 16, first + 16);
#pragma unroll
            for (int i = 0; i < 16; ++i) w[i] = Pack2<T>::pack(d[2 * i], d[2 * i + 1]);
            store_frags(tDw + packed, w);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(BAR(V_DR));
                mbar_arrive(BAR(V_TE + s));
            }
        }
        if (!ok) bwd_give_up(abort_flag);
        if (!bwd_wait(BAR(V_END), 0, nullptr)) bwd_give_up(abort_flag);
        tc_fence_after();
        // dV (warpgroups 0 and 1, half of the columns each) and dK (2 and 3) through the stages that held Q
        const float unshift = AB == 0 ? 0x1p-15f : 1.0f;
        const int part = wg & 1, to_dk = wg >> 1;
        const uint32_t sums = (to_dk ? tDK : tDV) + lanes + (uint32_t)(part * (D / 2));
        if (a.split == 1) {
            uint8_t* half = smem + Lay::S0 + (uint32_t)(to_dk * kHalves + (D == 128 ? part : 0)) * kHalfBytes;
            stage_row<T, D / 2>(sums, to_dk ? a.sm_scale * unshift / c : unshift, half, r, D == 128 ? 0 : 32 * part);
            fence_proxy_async_smem();
            named_barrier_sync(1, 32 * kSoftWarps);
            if (threadIdx.x == 0 && !*abort_flag) {
                for (int hf = 0; hf < kHalves; ++hf) {
                    tma_store_3d(&tdv, sQ + (uint32_t)hf * kHalfBytes, 64 * hf, kt * kTile, u);
                    tma_store_3d(&tdk, sQ + (uint32_t)(kHalves + hf) * kHalfBytes, 64 * hf, kt * kTile, u);
                }
                bulk_store_done();
            }
        } else {
            // the cluster's sums meet in shared memory: row r has 2 D floats, dV then dK, 16-byte pieces swizzled
            float4* row = reinterpret_cast<float4*>(smem + Lay::S0) + r * (D / 2);
#pragma unroll
            for (int c4 = 0; c4 < D / 64; ++c4) {
                float x[32];
                if (n > 0) {
                    tmem_ld32(sums + (uint32_t)c4 * 32u, x);
                    tmem_wait_ld();
                } else {
#pragma unroll
                    for (int e = 0; e < 32; ++e) x[e] = 0.0f;
                }
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    row[((to_dk * D + part * (D / 2)) / 4 + c4 * 8 + e) ^ (r & 7)] =
                        make_float4(x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]);
            }
        }
    }
    if (a.split > 1) {
        __syncwarp();
        cluster_arrive_release();
        cluster_wait_acquire();
        if (warp < kSoftWarps) {
            // every CTA adds up its share of the rows, always in the order of the CTAs
            bool fine = true;
            const uint32_t flag = smem_u32(const_cast<int*>(abort_flag)), at = base + Lay::S0;
            for (int p = 0; p < a.split; ++p) fine = fine && cluster_ld_u32(cluster_map(flag, (uint32_t)p)) == 0;
            const float unshift = AB == 0 ? 0x1p-15f : 1.0f, fk = a.sm_scale * unshift / *scale;
            const int rows = kTile / a.split;
            for (int e = threadIdx.x; e < rows * (D / 2); e += 32 * kSoftWarps) {
                const int r = mine_of * rows + e / (D / 2), piece = e % (D / 2);
                const uint32_t off = at + (uint32_t)(r * (D / 2) + (piece ^ (r & 7))) * 16u;
                float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                for (int p = 0; p < a.split; ++p) {
                    const float4 y = cluster_ld_f4(cluster_map(off, (uint32_t)p));
                    x.x += y.x, x.y += y.y, x.z += y.z, x.w += y.w;
                }
                const bool to_dk = piece >= D / 4;
                const float f = to_dk ? fk : unshift;
                const int j = kt * kTile + r;
                if (fine && j < a.T_len) {
                    uint2 w;
                    w.x = Pack2<T>::pack(x.x * f, x.y * f);
                    w.y = Pack2<T>::pack(x.z * f, x.w * f);
                    *reinterpret_cast<uint2*>((to_dk ? dk : dv) + ((int64_t)u * a.T_len + j) * D + 4 * (piece % (D / 4))) = w;
                }
            }
        }
        __syncwarp();
        cluster_arrive_release();                       // nobody reads this CTA's memory any more
        cluster_wait_acquire();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kSoftWarps + 1) tmem_dealloc(tmem, kTmemCols);
}

// ------------------------------------------------------------------ dQ

enum DqBar { W_QG = 0, W_KF = 1, W_KE = 5, W_VF = 9, W_VE = 11, W_SF = 13, W_SC = 14, W_DF = 15, W_DC = 16, W_DR = 17,
             W_DE = 18, W_END = 19, W_AT = 20, W_CS = 21, DQ_NBAR = 22 };

template <typename T, int AB, int D>
__global__ void __launch_bounds__(kDqThreads, 1)
    bwd_dq_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                  const __grid_constant__ CUtensorMap tg,
                  const __grid_constant__ CUtensorMap tdq, const T* __restrict__ q, const T* __restrict__ go,
                  const BwdArgs a) {
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t base = smem_u32(smem);
    if (base & 1023u) {                                 // layout assumption broken: do nothing
        if (threadIdx.x == 0) atomicOr(&g_status_prefill_bwd, kDevCheck);
        return;
    }
    using Lay = BwdLayout<D>;
    constexpr uint32_t kTileBytes = Lay::kTileBytes;
    constexpr int kHalves = D / 64;
    const uint32_t sG = base + Lay::A0, sK = base + Lay::A1, sV = base + Lay::S1;   // four stages of K, two of V
    auto BAR = [&](int i) -> uint32_t { return base + Lay::BAR + 8u * (uint32_t)i; };
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Lay::BAR + 8 * DQ_NBAR);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Lay::BAR + 8 * DQ_NBAR + 4);
    float* scale = reinterpret_cast<float*>(smem + Lay::SCALE);

    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    int rank, bh;
    place(a, (int)blockIdx.x, a.B * a.Hq, rank, bh);
    const int qt = a.n_t - 1 - rank, n = qt + 1;
    const int u = bh / a.Hq * a.Hkv + bh % a.Hq / (a.Hq / a.Hkv);
    const int wg = warp >> 2, r = threadIdx.x & 127, i = qt * kTile + r;
    if (threadIdx.x == 0) prefetch_tmap(&tk), prefetch_tmap(&tg), prefetch_tmap(&tv);

    // (one lane) tile it of K or V into its stage
    auto load_k = [&](int it) {
        const int s = it & 3;
        mbar_expect_tx(BAR(W_KF + s), kTileBytes);
        for (int hf = 0; hf < kHalves; ++hf)
            tma_load_3d(sK + s * kTileBytes + hf * kHalfBytes, &tk, 64 * hf, it * kTile, u, BAR(W_KF + s));
    };
    auto load_v = [&](int it) {
        const int s = it & 1;
        mbar_expect_tx(BAR(W_VF + s), kTileBytes);
        for (int hf = 0; hf < kHalves; ++hf)
            tma_load_3d(sV + s * kTileBytes + hf * kHalfBytes, &tv, 64 * hf, it * kTile, u, BAR(W_VF + s));
    };
    // The thread's share of Q (at D = 64 and dO), for tensor memory: as the products' first operands they would take as
    // much of shared memory's bandwidth as the second ones.
    constexpr bool kBoth = D == 64;
    uint32_t mine_q[16];
    if (warp < kSoftWarps) {
        constexpr int kChunks = D / 32;                 // 16-byte pieces of a warpgroup's columns
        const int64_t row = ((int64_t)bh * a.T_len + (i < a.T_len ? i : 0)) * D + 8 * kChunks * wg;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const T* from = (kBoth && e >= 2 ? go : q) + row;
            const uint4 y = i < a.T_len ? reinterpret_cast<const uint4*>(from)[e % kChunks] : make_uint4(0, 0, 0, 0);
            mine_q[4 * e] = y.x, mine_q[4 * e + 1] = y.y, mine_q[4 * e + 2] = y.z, mine_q[4 * e + 3] = y.w;
        }
    }
    if (warp == kSoftWarps) {
        constexpr uint32_t kMany = 1u << W_SC | 1u << W_DC | 1u << W_DR | 1u << W_AT;
        if (lane < DQ_NBAR) mbar_init(BAR(lane), kMany >> lane & 1 ? kSoftWarps : 1);
        if (lane == 0) *abort_flag = 0;
        fence_mbar_init();
    }
    __syncwarp();
    if (warp == kSoftWarps && lane == 0) {
        load_k(0);                                      // the first copies, see dkv
        if (!kBoth) {
            mbar_expect_tx(BAR(W_QG), kTileBytes);
            for (int hf = 0; hf < kHalves; ++hf) tma_load_3d(sG + hf * kHalfBytes, &tg, 64 * hf, qt * kTile, bh, BAR(W_QG));
        }
        load_v(0);
    }
    if (warp == kSoftWarps + 1) tmem_alloc(smem_u32(tmem_slot), kTmemCols);
    // No wait for the grid before this one: it waited for the statistics' grid before it let this one start (the
    // statistics are read from L2).
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
    // S, dP, packed dS, packed Q (at D = 64 and packed dO), dQ
    const uint32_t tS = tmem, tP = tmem + 128, tDS = tmem + 256, tQ = tmem + 320, tG = tmem + 352, tDQ = tmem + 384;

    if (warp == kSoftWarps) {
        if (lane == 0) {
            int it = 1, lastk[4] = {0, -1, -1, -1}, lastv[2] = {0, -1};
            for (; it < n; ++it) {
                if (it >= 4 && !mbar_wait(BAR(W_KE + (it & 3)), (it / 4 - 1) & 1, abort_flag)) break;
                load_k(it);
                lastk[it & 3] = it / 4;
                if (it >= 2 && !mbar_wait(BAR(W_VE + (it & 1)), (it / 2 - 1) & 1, abort_flag)) break;
                load_v(it);
                lastv[it & 1] = it / 2;
            }
            if (it < n) bwd_give_up(abort_flag);
            if (!kBoth) mbar_wait(BAR(W_QG), 0, nullptr);
            for (int s = 0; s < 4; ++s)
                if (lastk[s] >= 0) mbar_wait(BAR(W_KF + s), lastk[s] & 1, nullptr);
            for (int s = 0; s < 2; ++s)
                if (lastv[s] >= 0) mbar_wait(BAR(W_VF + s), lastv[s] & 1, nullptr);
        }
    } else if (warp == kSoftWarps + 1) {
        constexpr uint32_t idS = idesc_f16(AB, 128, 128, 0), idD = idesc_f16(AB, 128, D, 1);
        if (AB == 0) {                                  // for the scales, while the first tiles are on their way
            const float most = query_tile_most(a, bh, u, qt, lane);
            if (lane == 0) {
                *scale = most;
                mbar_arrive(BAR(W_CS));
            }
            __syncwarp();
        }
        // (one lane) S = Q K^T, dP = dO V^T with the streamed tile in stage s
        auto scores = [&](int s) {
            products_k_ta<D>(tS, tQ, sK + (uint32_t)s * kTileBytes, idS);
            tc_commit(BAR(W_SF));
        };
        auto grads = [&](int s) {
            if (kBoth) products_k_ta<D>(tP, tG, sV + (uint32_t)s * kTileBytes, idS);
            else products_k<D>(tP, sG, sV + (uint32_t)s * kTileBytes, idS);
            tc_commit(BAR(W_DF));
            tc_commit(BAR(W_VE + s));
        };
        auto wait = [&](int bar, int parity) { return mbar_wait(BAR(bar), (uint32_t)(parity & 1), abort_flag); };
        auto k_there = [&](int it, int s) { return wait(W_KF + s, it / 4); };
        auto v_there = [&](int it, int s) { return wait(W_VF + s, it / 2); };
        auto step = [&](auto phase, int it) -> bool {   // PH = it mod 4, see dkv
            constexpr int PH = decltype(phase)::value, k0 = PH, k1 = (PH + 1) % 4, k2 = (PH + 2) % 4, v1 = (PH & 1) ^ 1;
            if (it + 1 < n) {
                if (!wait(W_SC, PH)) return false;
                tc_fence_after();
                scores(k1);
                if (!v_there(it + 1, v1) || (it + 2 < n && !k_there(it + 2, k2)) || !wait(W_DC, PH)) return false;
                tc_fence_after();
                grads(v1);
            }
            if (!wait(W_DR, PH)) return false;
            tc_fence_after();
            products_mn<16>(tDQ, tDS, sK + (uint32_t)k0 * kTileBytes, idD, it > 0);         // dQ += dS K
            tc_commit(BAR(W_KE + k0));
            tc_commit(BAR(W_DE));
            return true;
        };
        if (elect_one()) {
            bool ok = wait(W_AT, 0) && (kBoth || wait(W_QG, 0)) && k_there(0, 0) && v_there(0, 0) && (n == 1 || k_there(1, 1));
            if (ok) {
                tc_fence_after();
                scores(0), grads(0);
            }
            for (int it = 0; ok && it < n; it += 4) {
                ok = step(Int<0>{}, it) && (it + 1 >= n || step(Int<1>{}, it + 1)) && (it + 2 >= n || step(Int<2>{}, it + 2)) &&
                     (it + 3 >= n || step(Int<3>{}, it + 3));
            }
            if (!ok) bwd_give_up(abort_flag);
            tc_commit(BAR(W_END));
            mbar_wait(BAR(W_END), 0, nullptr);
        }
        __syncwarp();
    } else {
        // thread r of warpgroup wg owns query r and keys 32 wg .. 32 wg + 31 of each tile
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t mine = lanes + 32u * (uint32_t)wg;
        const int64_t stat = (int64_t)bh * a.n_t * kTile + i;
        const float nl = __ldcg(a.ws.nlse + stat), delta = __ldcg(a.ws.delta + stat);
        const int below = AB == 0 ? __ldcg(a.ws.below + stat / 8) >> (4 * (r & 7)) & 15 : 0;
        const unsigned long long sc2 = f2_pack(a.scale_log2, a.scale_log2), nl2 = f2_pack(nl, nl);
        bool ok = true;
        if (kBoth) {
            tmem_st8(tQ + lanes + 8u * (uint32_t)wg, mine_q);
            tmem_st8(tG + lanes + 8u * (uint32_t)wg, mine_q + 8);
        } else {
            tmem_st16(tQ + lanes + 16u * (uint32_t)wg, mine_q);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(BAR(W_AT));
        if (AB == 0 && !bwd_wait(BAR(W_CS), 0, abort_flag)) ok = false;
        const float c = AB == 0 && ok ? ds_scale<AB>(fmaf(*scale, __int_as_float((127 - below) << 23), fabsf(delta))) : 1.0f;
        const float nd = -c * delta;
        const unsigned long long c2 = f2_pack(c, c), nd2 = f2_pack(nd, nd);
        for (int it = 0; ok && it < n; ++it) {
            const bool diag = it == qt;
            if (!bwd_wait(BAR(W_SF), it & 1, abort_flag)) { ok = false; break; }
            tc_fence_after();
            float p[32];
            tmem_ld32(tS + mine, p);
            tmem_wait_ld();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(BAR(W_SC));
#pragma unroll
            for (int q = 0; q < 32; q += 2) {
                float e0, e1;
                f2_unpack(f2_fma(f2_pack(p[q], p[q + 1]), sc2, nl2), e0, e1);
                p[q] = ex2_approx(e0), p[q + 1] = ex2_approx(e1);
            }
            if (!bwd_wait(BAR(W_DF), it & 1, abort_flag)) { ok = false; break; }
            tc_fence_after();
            float d[32];
            tmem_ld32(tP + mine, d);
            tmem_wait_ld();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(BAR(W_DC));
#pragma unroll
            for (int q = 0; q < 32; q += 2) {
                f2_unpack(f2_mul(f2_pack(p[q], p[q + 1]), f2_fma(f2_pack(d[q], d[q + 1]), c2, nd2)), d[q], d[q + 1]);
            }
            if (diag) {
#pragma unroll
                for (int q = 0; q < 32; ++q) d[q] = 32 * wg + q <= r ? d[q] : 0.0f;
            }
            if (it >= 1 && !bwd_wait(BAR(W_DE), (it - 1) & 1, abort_flag)) { ok = false; break; }
            tc_fence_after();
            store_pairs<T>(tDS + lanes + 16u * (uint32_t)wg, d);
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(BAR(W_DR));
        }
        if (!ok) bwd_give_up(abort_flag);
        if (!bwd_wait(BAR(W_END), 0, nullptr)) bwd_give_up(abort_flag);
        tc_fence_after();
        // 32 columns a warpgroup, through the stages that held K
        const float f = a.sm_scale * (AB == 0 ? 0x1p-15f : 1.0f) / c;
        if (32 * wg < D) stage_row<T, 32>(tDQ + mine, f, smem + Lay::A1 + (uint32_t)(wg >> 1) * kHalfBytes, r, 32 * (wg & 1));
        fence_proxy_async_smem();
        named_barrier_sync(1, 32 * kSoftWarps);
        if (threadIdx.x == 0 && !*abort_flag) {
            for (int hf = 0; hf < kHalves; ++hf) tma_store_3d(&tdq, sK + (uint32_t)hf * kHalfBytes, 64 * hf, qt * kTile, bh);
            bulk_store_done();
        }
    }
    // What follows this grid on the stream may start when it is done: the last CTA stays until the grid before it is too.
    if (blockIdx.x == gridDim.x - 1) grid_dependency_wait();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kSoftWarps + 1) tmem_dealloc(tmem, kTmemCols);
}

// ------------------------------------------------------------------ host

size_t ws_layout(int B, int Hq, int Hkv, int T, char* base, BwdWs* w) {
    const size_t n_t = (size_t)(T + kTile - 1) / kTile, rows = (size_t)B * Hq * n_t * kTile, tiles = (size_t)B * Hq * n_t;
    size_t at = 0;
    auto take = [&](size_t floats) {
        float* p = reinterpret_cast<float*>(base + at);
        at += (floats * sizeof(float) + 255) / 256 * 256;
        return p;
    };
    BwdWs x;
    x.nlse = take(rows), x.delta = take(rows), x.do_max = take(tiles), x.dl_max = take(tiles);
    x.v_max = take((size_t)B * Hkv * n_t);
    x.below = reinterpret_cast<uint32_t*>(take(tiles * (kTile / 8)));
    if (w) *w = x;
    return at;
}

// Heads launched side by side: groups of one size, the largest that keeps `bytes` a head within a third of L2.
int head_group(int heads, long long bytes) {
    const long long most = std::max<long long>(1, (40ll << 20) / std::max<long long>(bytes, 1));
    const int groups = (int)((heads + most - 1) / most);
    return (heads + groups - 1) / groups;
}

// CTAs that share a key tile in dkv (a cluster that adds up its sums through shared memory).  In thousands of clocks, a
// tile takes about 2.3 (D = 128: 2.6) in dkv and 1.9 in dq, a CTA's start and end 6 and with a cluster's sum 16; the call
// takes at least its longest CTA and, as dq fills the SMs that dkv leaves, all work over the SMs.  The size with the least
// such bound.
// (32/4 heads x 1024 tokens: 4 CTAs 48 us, one 92; 2 heads x 256: dkv alone 10 us with one, 14 with 8.)
int cluster_size(int units, int g, int n_t) {
    const int sms = device_sms(nullptr);
    const double tiles = 0.5 * units * g * n_t * (n_t + 1.0), ctas = (double)units * n_t;
    int best = 1;
    double least = 0.0;
    for (int c = 1; c <= 8; c *= 2) {
        const double longest = 2.3 * g * n_t / c + (c > 1 ? 16.0 : 6.0);
        const double all = (4.2 * tiles + ctas * (c * (c > 1 ? 16.0 : 6.0) + 6.0 * g)) / sms;
        const double bound = std::max(longest, all);
        if (c == 1 || bound < 0.95 * least) best = c, least = bound;
    }
    return best;
}

// A launch whose CTAs may start while the grid before it still runs (they wait for it where they need it).
template <typename... Params, typename... Args>
cudaError_t launch_early(void (*kernel)(Params...), int ctas, int cluster, int threads, size_t smem, cudaStream_t s,
                         Args... args) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = (unsigned)cluster;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = at;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <typename T, int AB, int D>
kvq_status run_typed(const PrefillBwdCall& c, cudaStream_t s) {
    using Lay = BwdLayout<D>;
    CUtensorMap mq, mk, mv, mg, mdq, mdk, mdv;
    const int dt = AB == 0 ? KVQ_F16 : KVQ_BF16;
    if (!make_map(&mq, c.q, dt, c.B * c.Hq, c.T, D) || !make_map(&mk, c.k, dt, c.B * c.Hkv, c.T, D) ||
        !make_map(&mv, c.v, dt, c.B * c.Hkv, c.T, D) || !make_map(&mg, c.go, dt, c.B * c.Hq, c.T, D) ||
        !make_map(&mdq, c.dq, dt, c.B * c.Hq, c.T, D) || !make_map(&mdk, c.dk, dt, c.B * c.Hkv, c.T, D) ||
        !make_map(&mdv, c.dv, dt, c.B * c.Hkv, c.T, D)) {
        set_error("prefill_attn_bwd: tensor map encoding failed");
        return KVQ_ECUDA;
    }
    static std::atomic<uint64_t> ready{0};              // devices whose attributes are set
    int dev = -1;
    device_sms(&dev);
    cudaError_t e = cudaSuccess;
    if (dev < 0 || dev > 63 || !(ready.load(std::memory_order_acquire) >> dev & 1)) {
        e = cudaFuncSetAttribute(bwd_dkv_kernel<T, AB, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Lay::BYTES);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(bwd_dq_kernel<T, AB, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Lay::BYTES);
        if (e == cudaSuccess && dev >= 0 && dev < 64) ready.fetch_or(1ull << dev, std::memory_order_release);
    }
    if (e == cudaSuccess) {
        BwdArgs a;
        ws_layout(c.B, c.Hq, c.Hkv, c.T, (char*)c.ws, &a.ws);
        a.B = c.B, a.Hq = c.Hq, a.Hkv = c.Hkv, a.T_len = c.T, a.n_t = (c.T + kTile - 1) / kTile;
        a.sm_scale = c.sm_scale, a.scale_log2 = c.sm_scale * kLog2e;
        a.group = a.split = 1;
        const int g = c.Hq / c.Hkv;
        bwd_prep_kernel<T, AB, D><<<a.n_t * c.B * c.Hq, kPrepThreads, 0, s>>>(
            (const T*)c.o, (const T*)c.go, (const T*)c.v, c.lse, c.glse, a);
        e = cudaGetLastError();
        if (e == cudaSuccess) {
            a.group = head_group(c.B * c.Hkv, (long long)c.T * D * 4 * g);
            a.split = cluster_size(c.B * c.Hkv, g, a.n_t);
            e = launch_early(bwd_dkv_kernel<T, AB, D>, a.n_t * c.B * c.Hkv * a.split, a.split, kDkvThreads, Lay::BYTES, s, mq,
                             mk, mv, mg, mdk, mdv, (T*)c.dk, (T*)c.dv, a);
        }
        if (e == cudaSuccess) {
            a.group = head_group(c.B * c.Hq, (long long)c.T * D * 4 / g);
            e = launch_early(bwd_dq_kernel<T, AB, D>, a.n_t * c.B * c.Hq, 1, kDqThreads, Lay::BYTES, s, mk, mv, mg, mdq,
                             (const T*)c.q, (const T*)c.go, a);
        }
    }
    if (e != cudaSuccess) {
        set_error("prefill_attn_bwd launch: %s", cudaGetErrorString(e));
        return KVQ_ECUDA;
    }
    return KVQ_OK;
}

}  // namespace

size_t prefill_bwd_bytes(int B, int Hq, int Hkv, int T) { return ws_layout(B, Hq, Hkv, T, nullptr, nullptr); }

kvq_status run_prefill_bwd(const PrefillBwdCall& c, cudaStream_t s) {
    if (c.dt == KVQ_F16) return c.D == 64 ? run_typed<__half, 0, 64>(c, s) : run_typed<__half, 0, 128>(c, s);
    return c.D == 64 ? run_typed<__nv_bfloat16, 1, 64>(c, s) : run_typed<__nv_bfloat16, 1, 128>(c, s);
}

}  // namespace kvq
