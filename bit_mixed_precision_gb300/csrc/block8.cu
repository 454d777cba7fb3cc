// The 8-bit block cache: reset, append, block selection and eviction (the
// attention over it is in block8_attn.cu; include/kvq.h has the format).
//
// append   one CTA per (unit, touched block): the rows of the block are held
//          in registers, one pass finds the largest magnitude and the keys'
//          minimum and maximum per channel, a second one (from registers)
//          writes the codes.  Bound by HBM: 16-bit rows in, 8-bit codes out.
// select   a score kernel (exact products of the 8-bit queries with the 8-bit
//          key bounds on the tensor cores) and, as its programmatic dependent, a
//          top-k kernel (one CTA per query and unit).
// evict    one CTA per unit: top-k over the blocks' accumulated weights and a
//          stable partition of the table row; no codes move.
#include <algorithm>
#include <type_traits>

#include "block8_device.cuh"
#include "kvq_internal.h"
#include "topk_device.cuh"

namespace kvq {

KVQ_DEFINE_STATUS(block8)

namespace {

using namespace b8;

// ------------------------------------------------------------------ reset

__global__ void reset_kernel(kvq_block8 c, const int32_t* __restrict__ mask) {
    const int u = blockIdx.x * blockDim.x + threadIdx.x;
    if (u >= c.B * c.Hkv || (mask && mask[u] == 0)) return;
    c.count[u] = 0;
    c.seq_len[u] = 0;
}

// ------------------------------------------------------------------ append

struct AppendArgs {
    kvq_block8 c;
    const void *k, *v;
    int64_t ks[3], vs[3];           // element strides b, h, t
    int n;
    const int32_t* n_new;
    const float* colscore;
};

// What a call does to unit u: its tokens before, the new ones (0: nothing), the touched blocks.
struct Plan {
    int count, n, first, last;      // blocks [first, last]
};

// The whole CTA calls this; all threads get the same answer.  `all`: checks every table entry that
// the call needs, so that a unit is appended to as a whole or left alone.  Only the CTA that may
// write the unit's open block and tail and the one that sets its counters need that: what the others
// write lies in the unit's free blocks.
template <int P>
__device__ Plan append_plan(const AppendArgs& a, int u, bool all, bool report) {
    static_assert((P & (P - 1)) == 0, "a power of two");
    Plan p;
    p.count = a.c.count[u];
    p.n = a.n_new ? a.n_new[u / a.c.Hkv] : a.n;
    bool bad = p.n < 0 || p.n > a.n;
    p.n = min(max(p.n, 0), a.n);
    bool fits = p.count >= 0 && (unsigned)p.count + (unsigned)p.n <= (unsigned)(a.c.max_blocks * P);
    p.first = p.count / P;
    p.last = p.n > 0 ? (p.count + p.n - 1) / P : p.first - 1;
    if (all && fits && p.n > 0) {
        const int32_t* row = a.c.table + (size_t)u * a.c.max_blocks;
        bool ok = true;
        for (int i = p.first + (int)threadIdx.x; i <= p.last; i += blockDim.x)
            ok = ok && (unsigned)row[i] < (unsigned)a.c.n_blocks;
        fits = __syncthreads_and(ok);
    }
    if (!fits) {
        bad = true;
        p.n = 0;
        p.last = p.first - 1;
    }
    if (bad && report && threadIdx.x == 0) atomicOr(&g_status_block8, kDevCheck);
    return p;
}

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.u16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

template <typename T> struct Packed2;
template <> struct Packed2<__half> {
    using type = __half2;
    static constexpr uint32_t kInf = 0x7c00u;
};
template <> struct Packed2<__nv_bfloat16> {
    using type = __nv_bfloat162;
    static constexpr uint32_t kInf = 0x7f80u;
};

// Minimum and maximum of pairs; a NaN wins both.
template <typename T>
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
    using P = typename Packed2<T>::type;
    P r = __hmin2_nan(*reinterpret_cast<P*>(&a), *reinterpret_cast<P*>(&b));
    return *reinterpret_cast<uint32_t*>(&r);
}
template <typename T>
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    using P = typename Packed2<T>::type;
    P r = __hmax2_nan(*reinterpret_cast<P*>(&a), *reinterpret_cast<P*>(&b));
    return *reinterpret_cast<uint32_t*>(&r);
}
template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t a) {
    T* h = reinterpret_cast<T*>(&a);
    return make_float2(Elem<T>::to_f(h[0]), Elem<T>::to_f(h[1]));
}

template <int THREADS>
struct AppendShared {
    uint32_t amax[THREADS / 32][2];     // keys, values
    float sum[THREADS / 32];
    uint32_t lo[THREADS / 32][64], hi[THREADS / 32][64];        // packed channel pairs per warp
};

// Codes of the thread's rows of one tensor (keys or values) of a block, and its new rows into the
// tail while the block stays open.
template <typename T, int D, int CODE, int THREADS, int PASSES, bool FULL>
__device__ __forceinline__ void write_codes(const uint4 (&r)[PASSES], uint8_t* codes, T* tail, int from, int fill, int end,
                                            bool open, bool finite, float s) {
    constexpr int TPR = D / 8, RPP = THREADS / TPR;
    const int col = threadIdx.x % TPR, row0 = threadIdx.x / TPR;
    const float inv = __frcp_rn(s);
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
        const int row = p * RPP + row0;
        if (!FULL && (row < from || row >= end)) continue;
        uint2 q = make_uint2(0, 0);
        if (finite) {
            const float2 f0 = unpack2<T>(r[p].x), f1 = unpack2<T>(r[p].y), f2 = unpack2<T>(r[p].z), f3 = unpack2<T>(r[p].w);
            q.x = code_four<CODE>(f0.x, f0.y, f1.x, f1.y, inv);
            q.y = code_four<CODE>(f2.x, f2.y, f3.x, f3.y, inv);
        }
        *reinterpret_cast<uint2*>(codes + row * D + col * 8) = q;
        if (!FULL && open && row >= fill) *reinterpret_cast<uint4*>(tail + row * D + col * 8) = r[p];
    }
}

// Packed channel minima and maxima of the thread's rows [from, end).
template <typename T, int RPP, int PASSES, bool FULL>
__device__ __forceinline__ void channel_range(const uint4 (&r)[PASSES], int row0, int from, int end, uint32_t (&lo)[4],
                                              uint32_t (&hi)[4]) {
    constexpr uint32_t kInf2 = Packed2<T>::kInf * 0x10001u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        lo[i] = kInf2;
        hi[i] = kInf2 | 0x80008000u;
    }
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
        const int row = p * RPP + row0;
        if (FULL || (row >= from && row < end)) {
            const uint32_t w[4] = {r[p].x, r[p].y, r[p].z, r[p].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                lo[i] = min2<T>(lo[i], w[i]);
                hi[i] = max2<T>(hi[i], w[i]);
            }
        }
    }
}

// Largest magnitude as 16-bit pairs, NaN and infinity above all numbers.
template <int PASSES>
__device__ __forceinline__ uint32_t largest(const uint4 (&r)[PASSES]) {
    uint32_t m = 0;
#pragma unroll
    for (int p = 0; p < PASSES; ++p)
        m = max_u16x2(m, max_u16x2(max_u16x2(r[p].x & 0x7fff7fffu, r[p].y & 0x7fff7fffu),
                                 max_u16x2(r[p].z & 0x7fff7fffu, r[p].w & 0x7fff7fffu)));
    return m;
}

// One block of one unit.  Rows [0, fill) are the open block's 16-bit rows in the tail, rows
// [fill, end) new ones; the block stays open if end < block.  Thread i holds 8 channels of row
// i / (D/8), + RPP, + 2 RPP ..., of keys and values at once: at most four pieces each, all
// requested before the first is used (THREADS grows with the block), and two barriers a block.
//
// 16 x 32 prompts of 16384 tokens of 128 channels, blocks of 32, int8, with column scores: 1077 us,
// 0.90 of the measured HBM rate (2910 us with 256 threads a block and the tensors one after the other;
// blocks that are not FULL on the same path as the others, and divisions by a block size that the compiler
// does not know, 1285).  A step's row of 512 units: four dependent loads and the launch, 6.1 to 6.7 us where
// no scale grows, 8.2 where all do; 8.5 with the copy that sets counters and scales back between calls.
// All variants use 64 registers; they spill 8 to 80 bytes.
//
// A block whose scales do not grow needs only its new rows: the codes of the others stand, and
// the bounds are the old ones widened by the new rows' (floor and ceil are monotone), exactly
// what a quantisation of all rows gives.  A scale grows 1/fill of the time, so a decode step
// reads one row instead of the whole open block.
//
// FULL: a block that this call fills from its first row to its last (most of a prompt's).
template <typename T, int D, int CODE, int THREADS, int PASSES, bool FULL>
__device__ void append_one(const AppendArgs& a, const Plan& pl, int u, int block, AppendShared<THREADS>& sh) {
    constexpr int TPR = D / 8, RPP = THREADS / TPR, W = THREADS / 32, P = RPP * PASSES;
    constexpr uint32_t kInf = Packed2<T>::kInf;
    const kvq_block8& c = a.c;
    const int col = threadIdx.x % TPR, row0 = threadIdx.x / TPR, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int b = u / c.Hkv, h = u % c.Hkv;
    const int fill = FULL ? 0 : max(0, pl.count - block * P), end = FULL ? P : min(P, pl.count + pl.n - block * P);
    const int t0 = block * P + fill - pl.count;                 // the block's first new token
    const int phys = c.table[(size_t)u * c.max_blocks + block];
    if ((unsigned)phys >= (unsigned)c.n_blocks) return;         // reported with the unit's whole range
    T* tk = (T*)c.tail_k + (size_t)u * P * D + col * 8;
    T* tv = (T*)c.tail_v + (size_t)u * P * D + col * 8;
    uint4 rk[PASSES], rv[PASSES];
    {
        const int64_t t = t0 + row0 - fill;                     // below 0 for rows that are not loaded
        const T* k = (const T*)a.k + b * a.ks[0] + h * a.ks[1] + t * a.ks[2] + col * 8;
        const T* v = (const T*)a.v + b * a.vs[0] + h * a.vs[1] + t * a.vs[2] + col * 8;
#pragma unroll
        for (int p = 0; p < PASSES; ++p, k += RPP * a.ks[2], v += RPP * a.vs[2]) {
            const int row = p * RPP + row0;
            rk[p] = rv[p] = make_uint4(0, 0, 0, 0);
            if (FULL || (row >= fill && row < end)) {
                rk[p] = __ldcs(reinterpret_cast<const uint4*>(k));
                rv[p] = __ldcs(reinterpret_cast<const uint4*>(v));
            }
        }
    }
    float sum = 0.0f;
    if (a.colscore) {
        const int g = c.Hq / c.Hkv, m = end - fill;
        const float* cs = a.colscore + ((size_t)b * c.Hq + (size_t)h * g) * a.n + t0;
        for (int x = 0; x < g; ++x, cs += a.n)
            for (int i = threadIdx.x; i < m; i += THREADS) sum += cs[i];
#pragma unroll
        for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (lane == 0) sh.sum[warp] = sum;
    }
    const float old_k = fill ? c.k_scale[phys] : 0.0f, old_v = fill ? c.v_scale[phys] : 0.0f,
                old_b = fill ? c.bound_scale[phys] : 0.0f;
    int from_k = fill, from_v = fill;   // the rows that count from here on
    float sk, sv, sb;
    bool fin_k, fin_v;
    uint32_t lo[4], hi[4];              // the keys' range per channel, over the thread's rows
    for (;;) {
        uint32_t mk = 0, mv = largest(rv);
        channel_range<T, RPP, PASSES, FULL>(rk, row0, from_k, end, lo, hi);
        constexpr uint32_t kInf2 = kInf * 0x10001u;
        if (FULL || lo[0] != kInf2 || hi[0] != (kInf2 | 0x80008000u))   // as they start: the thread has no rows
#pragma unroll
            for (int i = 0; i < 4; ++i) mk = max_u16x2(mk, max_u16x2(lo[i] & 0x7fff7fffu, hi[i] & 0x7fff7fffu));
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            mk = max_u16x2(mk, __shfl_xor_sync(0xffffffffu, mk, o));
            mv = max_u16x2(mv, __shfl_xor_sync(0xffffffffu, mv, o));
        }
        if (lane == 0) {
            sh.amax[warp][0] = mk;
            sh.amax[warp][1] = mv;
        }
        __syncthreads();
        mk = mv = 0;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            mk = max_u16x2(mk, sh.amax[w][0]);
            mv = max_u16x2(mv, sh.amax[w][1]);
        }
        mk = max(mk & 0xffffu, mk >> 16);
        mv = max(mv & 0xffffu, mv >> 16);
        const float nan = __int_as_float(0x7fc00000);
        fin_k = mk < kInf;
        fin_v = mv < kInf;
        sk = fin_k ? scale_of(unpack2<T>(mk).x, Code<CODE>::kInvMax) : nan;
        sb = fin_k ? scale_of(unpack2<T>(mk).x, kInv127) : nan;
        sv = fin_v ? scale_of(unpack2<T>(mv).x, Code<CODE>::kInvMax) : nan;
        const bool grow_k = from_k > 0 && !(sk <= old_k && sb <= old_b), grow_v = from_v > 0 && !(sv <= old_v);
        if (FULL || (!grow_k && !grow_v)) break;
        // a scale grows: every row of that tensor counts
        __syncthreads();
#pragma unroll
        for (int p = 0; p < PASSES; ++p) {
            const int row = p * RPP + row0;
            if (row < fill) {
                if (grow_k) rk[p] = *reinterpret_cast<const uint4*>(tk + (size_t)row * D);
                if (grow_v) rv[p] = *reinterpret_cast<const uint4*>(tv + (size_t)row * D);
            }
        }
        if (grow_k) from_k = 0;
        if (grow_v) from_v = 0;
    }
    const bool widen = from_k > 0;      // the old scales stand
    if (widen) {
        sk = old_k;
        sb = old_b;
    }
    if (from_v > 0) sv = old_v;
    // bounds: minimum and maximum per channel, over the warp's rows and then the CTA's
#pragma unroll
    for (int o = TPR; o < 32; o <<= 1)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            lo[i] = min2<T>(lo[i], __shfl_xor_sync(0xffffffffu, lo[i], o));
            hi[i] = max2<T>(hi[i], __shfl_xor_sync(0xffffffffu, hi[i], o));
        }
    if (lane < TPR)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            sh.lo[warp][lane * 4 + i] = lo[i];
            sh.hi[warp][lane * 4 + i] = hi[i];
        }
    write_codes<T, D, CODE, THREADS, PASSES, FULL>(rk, c.k_codes + (size_t)phys * P * D, tk - col * 8, from_k, fill, end, end < P,
                                             fin_k, sk);
    write_codes<T, D, CODE, THREADS, PASSES, FULL>(rv, c.v_codes + (size_t)phys * P * D, tv - col * 8, from_v, fill, end, end < P,
                                             fin_v, sv);
    __syncthreads();
    for (int x = threadIdx.x; x < D / 2; x += THREADS) {
        uint32_t l = sh.lo[0][x], hh = sh.hi[0][x];
#pragma unroll
        for (int w = 1; w < W; ++w) {
            l = min2<T>(l, sh.lo[w][x]);
            hh = max2<T>(hh, sh.hi[w][x]);
        }
        const float ib = __frcp_rn(sb);
        const float2 fl = unpack2<T>(l), fh = unpack2<T>(hh);
        int l0 = 0, l1 = 0, h0 = 0, h1 = 0;
        if (fin_k) {
            l0 = (int)fmaxf(-127.0f, fminf(127.0f, floorf(__fmul_rn(fl.x, ib))));
            l1 = (int)fmaxf(-127.0f, fminf(127.0f, floorf(__fmul_rn(fl.y, ib))));
            h0 = (int)fmaxf(-127.0f, fminf(127.0f, ceilf(__fmul_rn(fh.x, ib))));
            h1 = (int)fmaxf(-127.0f, fminf(127.0f, ceilf(__fmul_rn(fh.y, ib))));
        }
        char2* lp = reinterpret_cast<char2*>(c.k_bound + (size_t)phys * 2 * D) + x;
        char2* hp = lp + D / 2;
        if (widen) {
            const char2 ol = *lp, oh = *hp;
            l0 = min(l0, (int)ol.x);
            l1 = min(l1, (int)ol.y);
            h0 = max(h0, (int)oh.x);
            h1 = max(h1, (int)oh.y);
        }
        *lp = make_char2((signed char)l0, (signed char)l1);
        *hp = make_char2((signed char)h0, (signed char)h1);
    }
    if (threadIdx.x == 0) {
        c.k_scale[phys] = sk;
        c.bound_scale[phys] = sb;
        c.v_scale[phys] = sv;
        if (fill == 0) c.block_pos[phys] = c.seq_len[u] + block * P - pl.count;
        sum = 0.0f;
        if (a.colscore)
            for (int w = 0; w < W; ++w) sum += sh.sum[w];
        if (fill == 0 || a.colscore) c.acc[phys] = (fill == 0 ? 0.0f : c.acc[phys]) + sum;
    }
}

// Grid: x = j + per * unit.  CTA j takes block first + j; CTA 0 takes, where the first touched
// block was open, the last one too if that stays open: both use the unit's tail rows, and the
// first reads them before the last writes them.  commit: the CTA is alone (n <= block touches at
// most those two blocks) and sets the counters itself.
template <typename T, int D, int CODE, int THREADS, int PASSES>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) append_kernel(AppendArgs a, unsigned per, int commit) {
    constexpr int P = THREADS * PASSES * 8 / D;
    __shared__ AppendShared<THREADS> sh;
    const int u = blockIdx.x / per, j = blockIdx.x % per;
    const Plan p = append_plan<P>(a, u, j == 0, j == 0);
    if (p.n == 0) return;
    const bool open_first = p.count % P != 0, open_last = (p.count + p.n) % P != 0;
    const bool pair = open_first && open_last && p.last > p.first;
    int block = p.first + j;
    if (block > p.last) return;
    const bool full = block * P >= p.count && (block + 1) * P <= p.count + p.n;
    if (full) {
        append_one<T, D, CODE, THREADS, PASSES, true>(a, p, u, block, sh);
    } else if (!(pair && j > 0)) {
        for (;; block = p.last) {
            append_one<T, D, CODE, THREADS, PASSES, false>(a, p, u, block, sh);
            if (!pair || block == p.last) break;
            __syncthreads();
        }
    }
    if (commit && threadIdx.x == 0) {
        a.c.count[u] = p.count + p.n;
        a.c.seq_len[u] += p.n;
    }
}

template <int P>
__global__ void __launch_bounds__(256) append_commit_kernel(AppendArgs a) {
    const int u = blockIdx.x;
    const Plan p = append_plan<P>(a, u, true, false);
    if (threadIdx.x == 0 && p.n > 0) {
        a.c.count[u] = p.count + p.n;
        a.c.seq_len[u] += p.n;
    }
}

template <typename T, int D, int CODE, int THREADS, int PASSES>
cudaError_t launch_append_threads(const AppendArgs& a, cudaStream_t s) {
    constexpr int P = THREADS * PASSES * 8 / D;
    const unsigned units = (unsigned)(a.c.B * a.c.Hkv);
    if (a.n <= P) {
        append_kernel<T, D, CODE, THREADS, PASSES><<<units, THREADS, 0, s>>>(a, 1, 1);
        return cudaGetLastError();
    }
    const unsigned per = (unsigned)((a.n + P - 2) / P + 1);
    append_kernel<T, D, CODE, THREADS, PASSES><<<units * per, THREADS, 0, s>>>(a, per, 0);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    append_commit_kernel<P><<<units, 256, 0, s>>>(a);
    return cudaGetLastError();
}

// Threads so that each holds at most four 16-byte pieces of the block's keys (and of its values), 64
// at least; threads, passes and D give the block's size.
template <typename T, int D, int CODE, int P>
cudaError_t launch_append_block(const AppendArgs& a, cudaStream_t s) {
    constexpr int kPieces = P * D / 8, kThreads = kPieces / 4 < 64 ? 64 : kPieces / 4;
    return launch_append_threads<T, D, CODE, kThreads, kPieces / kThreads>(a, s);
}

template <typename T, int D, int CODE>
cudaError_t launch_append_typed(const AppendArgs& a, cudaStream_t s) {
    switch (a.c.block) {
        case 16: return launch_append_block<T, D, CODE, 16>(a, s);
        case 32: return launch_append_block<T, D, CODE, 32>(a, s);
        case 64: return launch_append_block<T, D, CODE, 64>(a, s);
        default: return launch_append_block<T, D, CODE, 128>(a, s);
    }
}

// ------------------------------------------------------------------ select

struct SelectArgs {
    kvq_block8 c;
    const void* q;
    int64_t qs[3];
    int n_q;
    const int32_t* n_new;
    int n_sel, n_first, n_last;
    int32_t *idx_out, *n_out;
    float* score;                   // workspace [u][n_q][max_blocks]
};

constexpr int kScoreThreads = 128, kScoreWarps = kScoreThreads / 32;

__device__ __forceinline__ float max_or_nan(float a, float b) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}

// Blocks that query t of the unit of row (unit, t) sees, or 0 where all of them are chosen anyway.
__device__ __forceinline__ int blocks_to_score(const SelectArgs& a, int row) {
    const kvq_block8& c = a.c;
    const int u = row / a.n_q, t = row % a.n_q;
    const int m = new_rows(a.n_new, u / c.Hkv, a.n_q, &g_status_block8);
    const int limit = min(query_limit(c.count[u], m, t), c.max_blocks * c.block);
    const int nb = (limit + c.block - 1) / c.block;
    return nb > a.n_sel ? nb : 0;
}

// Scores of blocks for the queries of their unit: sum_c max(q8 low, q8 high) = q8- . low + q8+ . high
// is one product of the bounds (16 blocks are the rows of an MMA, their 2 D bounds its k axis) with
// the group's queries, eight heads to a column block.  Whole numbers below 2^21 in fp16 operands and
// float32 sums: exact.  Bound rows go from global memory into the fragments, a lane's 16-byte pieces
// being the k elements of four MMAs.  All queries' groups of 16 blocks form one list that is split over
// the resident CTAs; a CTA quantises a query once per run of groups, its warps take the groups in turn,
// each with the next group's bounds requested before the current ones are used.
// 128 units of up to 2048 blocks: the call 22 us against 7.5 of HBM time; the groups stream at 7.6 TB/s,
// but the first ones arrive 4 us after the start (counters, table, bounds) and a second unit in a run
// costs 3 us.  One thread per block with four-byte dot products: 31 us; grids of 64 to 512 blocks per
// CTA: 20 (for these units, 15 for eight) to 33.
template <typename T, int D>
__global__ void __launch_bounds__(kScoreThreads, 5) score_kernel(SelectArgs a) {
    constexpr int S = 2 * D / 16, PAD = 2 * D + 4;      // MMA steps; halves per head in shared memory
    extern __shared__ __align__(16) __half q8[];        // [heads, a multiple of 8][2][D], rows padded
    __shared__ float sq[KVQ_BLOCK8_MAX_GROUP];
    __shared__ RunShared<kScoreThreads> run_sh;
    const kvq_block8& c = a.c;
    const int g = c.Hq / c.Hkv, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, lg = lane >> 2, lt = lane & 3;
    const auto run = find_run<kScoreThreads, kScoreWarps>(
        c.B * c.Hkv * a.n_q, [&](int i) { return (blocks_to_score(a, i) + 15) / 16; }, run_sh);
    grid_launch_dependents();
    for (int row = run.work, from = run.from, before = run.before; from < run.to; ++row) {
        const int nb = blocks_to_score(a, row), groups = (nb + 15) / 16;
        if (groups == 0) continue;
        const int u = row / a.n_q, t = row % a.n_q, b = u / c.Hkv, h = u % c.Hkv;
        // groups of this query: [first, last)
        const int first = max(from - before - run.start, 0), last = min(groups, run.to - before - run.start);
        if (last <= 0) break;                           // the run ends ahead of the query's groups
        const int32_t* table = a.c.table + (size_t)u * c.max_blocks;
        uint4 r[2][S / 4];                              // rows lg, lg + 8: low, then high bounds
        float scale[2];
        bool there[2];
        // pool blocks of two of the warp's groups, i and i + kScoreWarps, one a lane; asked for two
        // groups before they are used
        auto find = [&](int i) {
            const int at = 16 * (i + (lane >> 4) * kScoreWarps) + (lane & 15);
            return at < nb && i < last ? table[at] : 0;
        };
        int i = first + warp, ids = find(i), ids2 = find(i + 2 * kScoreWarps);
        auto request = [&](int half) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int phys = __shfl_sync(0xffffffffu, ids, half * 16 + lg + 8 * x);
                there[x] = (unsigned)phys < (unsigned)c.n_blocks;
                const int at = there[x] ? phys : 0;
                const uint8_t* p = (const uint8_t*)c.k_bound + (size_t)at * 2 * D + lt * 16;
#pragma unroll
                for (int y = 0; y < S / 4; ++y) r[x][y] = load16(p + y * 64);
                scale[x] = c.bound_scale[at];
            }
        };
        // the first query row's load and the table's are on their way together
        const T* q = (const T*)a.q + b * a.qs[0] + (int64_t)(h * g) * a.qs[1] + t * a.qs[2] + lane * 4;
        uint2 w = make_uint2(0, 0);
        if (warp < g && lane < D / 4) w = *reinterpret_cast<const uint2*>(q + warp * a.qs[1]);
        if (i < last) request(0);
        for (int hh = warp; hh < ((g + 7) & ~7); hh += kScoreWarps) {
            float x[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            if (hh >= kScoreWarps && hh < g && lane < D / 4) w = *reinterpret_cast<const uint2*>(q + hh * a.qs[1]);
            if (hh < g && lane < D / 4) {
                const T* e = reinterpret_cast<const T*>(&w);
#pragma unroll
                for (int j = 0; j < 4; ++j) x[j] = Elem<T>::to_f(e[j]);
            }
            uint32_t mx = 0;                            // magnitudes as bits: NaN and infinity rank above all
#pragma unroll
            for (int j = 0; j < 4; ++j) mx = max(mx, __float_as_uint(x[j]) & 0x7fffffffu);
            mx = __reduce_max_sync(0xffffffffu, mx);
            const bool finite = mx < 0x7f800000u;
            const float s = finite ? scale_of(__uint_as_float(mx), kInv127) : __int_as_float(0x7fc00000);
            const float inv = __frcp_rn(s);
            if (lane < D / 4)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float v = finite ? fminf(127.0f, fmaxf(-127.0f, rintf(__fmul_rn(x[j], inv)))) : 0.0f;
                    q8[hh * PAD + lane * 4 + j] = __float2half_rn(fminf(v, 0.0f));
                    q8[hh * PAD + D + lane * 4 + j] = __float2half_rn(fmaxf(v, 0.0f));
                }
            if (lane == 0 && hh < g) sq[hh] = s;
        }
        __syncthreads();
        const __half* mine = q8 + lg * PAD + lt * 16;   // fragments: channels in the order of the lane's pieces
        for (int half = 1; i < last; i += kScoreWarps, half ^= 1) {
            const float bs[2] = {scale[0], scale[1]};
            const bool ok[2] = {there[0], there[1]};
            float best[2] = {-INFINITY, -INFINITY};
            for (int h0 = 0; h0 < g; h0 += 8) {
                float d[4] = {0.0f, 0.0f, 0.0f, 0.0f}, d2[4] = {0.0f, 0.0f, 0.0f, 0.0f};     // two chains of products
#pragma unroll
                for (int s = 0; s < S; ++s) {
                    const uint4 x = r[0][s / 4], y = r[1][s / 4];
                    const uint2 q = *reinterpret_cast<const uint2*>(mine + h0 * PAD + (s / 4) * 64 + (s % 4) * 4);
                    uint32_t a0, a1, a2, a3;
                    to_f16<KVQ_CODE_INT8>(s % 4 == 0 ? x.x : s % 4 == 1 ? x.y : s % 4 == 2 ? x.z : x.w, a0, a2);
                    to_f16<KVQ_CODE_INT8>(s % 4 == 0 ? y.x : s % 4 == 1 ? y.y : s % 4 == 2 ? y.z : y.w, a1, a3);
                    mma(s & 1 ? d2 : d, a0, a1, a2, a3, q.x, q.y);
                }
                if (h0 + 8 >= g) {                      // the bounds are read: ask for the next ones
                    if (half == 0) {
                        ids = ids2;
                        ids2 = find(i + 3 * kScoreWarps);
                    }
                    if (i + kScoreWarps < last) request(half);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) d[e] += d2[e];
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    if (h0 + 2 * lt + e < g) {
                        best[0] = max_or_nan(best[0], __fmul_rn(d[e], sq[h0 + 2 * lt + e]));
                        best[1] = max_or_nan(best[1], __fmul_rn(d[2 + e], sq[h0 + 2 * lt + e]));
                    }
            }
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                best[x] = max_or_nan(best[x], __shfl_xor_sync(0xffffffffu, best[x], 1));
                best[x] = max_or_nan(best[x], __shfl_xor_sync(0xffffffffu, best[x], 2));
                const int at = 16 * i + lg + 8 * x;
                if (lt == 0 && at < nb) {
                    if (!ok[x]) atomicOr(&g_status_block8, kDevCheck);
                    a.score[(size_t)row * c.max_blocks + at] = ok[x] ? __fmul_rn(best[x], bs[x]) : -INFINITY;
                }
            }
        }
        __syncthreads();                                // q8 and sq are written again
        before += run.places(groups);
        from = before;
    }
}

// ------------------------------------------------------------------ top-k in order

// Which of the keys key(0) .. key(n - 1) are the k largest, ties to the lower index: put(i, chosen,
// before) for each i, before = how many of lower index are chosen.  k < n.
//
// The keys stay in registers, KPT a thread, in index order.  The k-th largest is found two bits a
// round from the highest bit in which the keys differ: one count of the CTA against three candidates,
// one barrier.  As soon as a count is k exactly there is nothing more to find (for keys without ties
// after about log2 n bits).  One scan gives every key its place.  At 2048 keys about 6 us with the launch,
// against 9 of the radix select's four passes over memory and one bit a round in 512 threads.
template <int KPT, typename KeyFn, typename PutFn>
__device__ void choose_regs(KeyFn key, int n, int k, TopkShared& sh, PutFn put) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5, i0 = threadIdx.x * KPT;
    uint32_t x[KPT], lo = 0xffffffffu, hi = 0u;
#pragma unroll
    for (int j = 0; j < KPT; ++j) {
        x[j] = i0 + j < n ? key(i0 + j) : 0u;           // 0 is no key (rank_key > 0) and never counted
        hi = max(hi, x[j]);
        if (i0 + j < n) lo = min(lo, x[j]);
    }
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    uint2* buf = reinterpret_cast<uint2*>(sh.hist);     // two halves of 32, used in turn
    if (lane == 0) buf[warp] = make_uint2(lo, hi);
    __syncthreads();
    const uint2 ends = lane < nw ? buf[lane] : make_uint2(0xffffffffu, 0u);
    lo = __reduce_min_sync(0xffffffffu, ends.x);
    hi = __reduce_max_sync(0xffffffffu, ends.y);
    uint32_t at = hi;                                   // all keys equal: the k-th largest
    bool exact = false;
    if (lo != hi) {
        int bit = (31 - __clz(lo ^ hi)) & ~1;           // rounds of bits (bit + 1, bit)
        at = hi >> bit >> 1 >> 1 << bit << 1 << 1;      // what all keys share
        for (int half = 32; bit >= 0 && !exact; bit -= 2, half ^= 32) {
            const uint32_t c1 = at | (1u << bit), c2 = at | (2u << bit), c3 = at | (3u << bit);
            uint32_t n1 = 0, n23 = 0;
#pragma unroll
            for (int j = 0; j < KPT; ++j) {
                n1 += x[j] >= c1 ? 1u : 0u;
                n23 += (x[j] >= c2 ? 1u : 0u) + (x[j] >= c3 ? 0x10000u : 0u);
            }
            n1 = __reduce_add_sync(0xffffffffu, n1);
            n23 = __reduce_add_sync(0xffffffffu, n23);
            if (lane == 0) buf[half + warp] = make_uint2(n1, n23);
            __syncthreads();
            const uint2 y = lane < nw ? buf[half + lane] : make_uint2(0u, 0u);
            n1 = __reduce_add_sync(0xffffffffu, y.x);
            n23 = __reduce_add_sync(0xffffffffu, y.y);
            const uint32_t kk = (uint32_t)k, n2 = n23 & 0xffffu, n3 = n23 >> 16;
            exact = n1 == kk || n2 == kk || n3 == kk;
            if (n3 >= kk) at = c3;
            else if (n2 >= kk) at = c2;
            else if (n1 >= kk) at = c1;
        }
    }
    uint32_t gt = 0, eq = 0;
#pragma unroll
    for (int j = 0; j < KPT; ++j) {
        gt += (exact ? x[j] >= at : x[j] > at) ? 1u : 0u;
        eq += !exact && x[j] == at ? 1u : 0u;
    }
    uint32_t total;
    const uint32_t before = block_excl_scan(gt << 16 | eq, sh, &total);
    const uint32_t take = (uint32_t)k - (total >> 16);  // equal keys that are chosen
    uint32_t g = before >> 16, e = before & 0xffffu;
#pragma unroll
    for (int j = 0; j < KPT; ++j) {
        const bool more = exact ? x[j] >= at : x[j] > at, same = !exact && x[j] == at;
        if (i0 + j < n) put(i0 + j, more || (same && e < take), g + min(e, take));
        g += more ? 1u : 0u;
        e += same ? 1u : 0u;
    }
}

// The same for any n: radix select with the keys read again in every pass.
template <typename KeyFn, typename PutFn>
__device__ void choose_many(KeyFn key, int n, int k, TopkShared& sh, PutFn put) {
    uint32_t kstar = 0xffffffffu, take_eq = 0;
    if (k > 0) block_radix_select(key, n, k, sh, &kstar, &take_eq);
    uint32_t eq_base = 0, sel_base = 0;
    for (int c0 = 0; c0 < n; c0 += blockDim.x) {
        const int i = c0 + threadIdx.x;
        const uint32_t kv = i < n ? key(i) : 0u;
        const uint32_t eq = k > 0 && i < n && kv == kstar ? 1u : 0u;
        uint32_t tot;
        const uint32_t eq_rank = block_excl_scan(eq, sh, &tot);
        const uint32_t sel = k > 0 && i < n && (kv > kstar || (eq && eq_base + eq_rank < take_eq)) ? 1u : 0u;
        eq_base += tot;
        const uint32_t before = block_excl_scan(sel, sh, &tot);
        if (i < n) put(i, sel != 0, sel_base + before);
        sel_base += tot;
    }
}

constexpr int kChooseThreads = 256;

// KPT keys a thread in registers, or 0: any number of keys.  The launch takes the smallest that holds
// max_blocks keys (8 a thread leave six CTAs per SM, 32 two; evict of 512 units of 2000 blocks with all
// three in one kernel ran in two waves).
template <int KPT, typename KeyFn, typename PutFn>
__device__ __forceinline__ void choose(KeyFn key, int n, int k, TopkShared& sh, PutFn put) {
    if (k == 0) {
        for (int i = threadIdx.x; i < n; i += blockDim.x) put(i, false, 0u);
    } else {
        if constexpr (KPT > 0) choose_regs<KPT>(key, n, k, sh, put);
        else choose_many(key, n, k, sh, put);
    }
}

template <typename F>
cudaError_t by_keys(int most, F f) {
    if (most <= 8 * kChooseThreads) return f(std::integral_constant<int, 8>{});
    if (most <= 32 * kChooseThreads) return f(std::integral_constant<int, 32>{});
    return f(std::integral_constant<int, 0>{});
}

template <int KPT>
__global__ void __launch_bounds__(kChooseThreads) choose_kernel(SelectArgs a) {
    __shared__ __align__(16) TopkShared sh;
    const kvq_block8& c = a.c;
    const int row = blockIdx.x, u = row / a.n_q, t = row % a.n_q;
    const int m = new_rows(a.n_new, u / c.Hkv, a.n_q, &g_status_block8);
    const int limit = min(query_limit(c.count[u], m, t), c.max_blocks * c.block);
    const int nb = (limit + c.block - 1) / c.block;
    int32_t* out = a.idx_out + (size_t)row * a.n_sel;
    if (threadIdx.x == 0) a.n_out[row] = min(nb, a.n_sel);
    if (nb <= a.n_sel) {
        for (int i = threadIdx.x; i < a.n_sel; i += blockDim.x) out[i] = i < nb ? i : -1;
        grid_dependency_wait();         // what follows in the stream follows both kernels
        return;
    }
    grid_dependency_wait();
    const float* score = a.score + (size_t)row * c.max_blocks + a.n_first;
    for (int i = threadIdx.x; i < a.n_first; i += blockDim.x) out[i] = i;
    for (int i = threadIdx.x; i < a.n_last; i += blockDim.x) out[a.n_sel - a.n_last + i] = nb - a.n_last + i;
    choose<KPT>([&](int i) { return rank_key(score[i]); }, nb - a.n_first - a.n_last, a.n_sel - a.n_first - a.n_last, sh,
           [&](int i, bool chosen, uint32_t before) {
               if (chosen) out[a.n_first + before] = a.n_first + i;
           });
}

// ------------------------------------------------------------------ evict

// ids: the unit's table row, read once; the new row is written from it.  Where the keys do not fit
// the registers they are gathered again from acc in every pass.  Bound by latency (counter, row, weights
// at random places of acc, about ten rounds of counting): 512 units of up to 2048 blocks 16 us with a
// copy of the table.
template <int KPT>
__global__ void __launch_bounds__(kChooseThreads) evict_kernel(kvq_block8 c, const int32_t* __restrict__ keep, int n_first,
                                                              int n_last, int32_t* __restrict__ n_evicted) {
    extern __shared__ int32_t ids[];
    __shared__ __align__(16) TopkShared sh;
    const int u = blockIdx.x, count = min(max(c.count[u], 0), c.max_blocks * c.block);
    const int nb = (count + c.block - 1) / c.block;
    const int want = max(keep[u], n_first + n_last);
    if (nb <= want) {
        if (threadIdx.x == 0 && n_evicted) n_evicted[u] = 0;
        return;
    }
    int32_t* row = c.table + (size_t)u * c.max_blocks;
    for (int i = threadIdx.x; i < nb; i += blockDim.x) ids[i] = row[i];
    __syncthreads();
    const int mid = want - n_first - n_last;
    choose<KPT>(
        [&](int i) {
            const int phys = ids[n_first + i];
            if ((unsigned)phys < (unsigned)c.n_blocks) return rank_key(c.acc[phys]);
            atomicOr(&g_status_block8, kDevCheck);
            return 1u;                                  // a lost block goes first
        },
        nb - n_first - n_last, mid, sh,
        [&](int i, bool chosen, uint32_t before) {
            row[chosen ? n_first + (int)before : want + i - (int)before] = ids[n_first + i];
        });
    for (int i = threadIdx.x; i < n_last; i += blockDim.x) row[want - n_last + i] = ids[nb - n_last + i];
    if (threadIdx.x == 0) {
        c.count[u] = count - (nb - want) * c.block;
        if (n_evicted) n_evicted[u] = nb - want;
    }
}

template <typename F>
cudaError_t by_type(const kvq_block8& c, F f) {
    if (c.dtype == KVQ_F16) return c.D == 64 ? f(__half{}, std::integral_constant<int, 64>{})
                                             : f(__half{}, std::integral_constant<int, 128>{});
    return c.D == 64 ? f(__nv_bfloat16{}, std::integral_constant<int, 64>{})
                     : f(__nv_bfloat16{}, std::integral_constant<int, 128>{});
}

}  // namespace

cudaError_t launch_block8_reset(const kvq_block8& c, const int32_t* mask, cudaStream_t s) {
    const unsigned units = (unsigned)(c.B * c.Hkv);
    reset_kernel<<<(units + 127) / 128, 128, 0, s>>>(c, mask);
    return cudaGetLastError();
}

cudaError_t launch_block8_append(const kvq_block8& c, const void* k, const int64_t* ks, const void* v,
                                 const int64_t* vs, int n, const int32_t* n_new, const float* colscore,
                                 cudaStream_t s) {
    AppendArgs a;
    a.c = c;
    a.k = k;
    a.v = v;
    for (int i = 0; i < 3; ++i) {
        a.ks[i] = ks[i];
        a.vs[i] = vs[i];
    }
    a.n = n;
    a.n_new = n_new;
    a.colscore = colscore;
    return by_type(c, [&](auto t, auto d) {
        using T = decltype(t);
        constexpr int D = decltype(d)::value;
        return c.code == KVQ_CODE_E4M3 ? launch_append_typed<T, D, KVQ_CODE_E4M3>(a, s)
                                       : launch_append_typed<T, D, KVQ_CODE_INT8>(a, s);
    });
}

size_t block8_select_bytes(const kvq_block8& c, int n_q) {
    return (size_t)c.B * c.Hkv * n_q * c.max_blocks * sizeof(float);
}

cudaError_t launch_block8_select(const void* q, const int64_t* qs, int n_q, const int32_t* n_new, const kvq_block8& c,
                                 int n_sel, int n_first, int n_last, int32_t* idx_out, int32_t* n_out, void* ws,
                                 cudaStream_t s) {
    SelectArgs a;
    a.c = c;
    a.q = q;
    for (int i = 0; i < 3; ++i) a.qs[i] = qs[i];
    a.n_q = n_q;
    a.n_new = n_new;
    a.n_sel = n_sel;
    a.n_first = n_first;
    a.n_last = n_last;
    a.idx_out = idx_out;
    a.n_out = n_out;
    a.score = (float*)ws;
    const unsigned rows = (unsigned)(c.B * c.Hkv * n_q);
    if (c.max_blocks > n_sel) {
        cudaError_t e = by_type(c, [&](auto t, auto d) {
            using T = decltype(t);
            constexpr int D = decltype(d)::value;
            static std::atomic<int> known[64];
            const size_t smem = (size_t)((c.Hq / c.Hkv + 7) & ~7) * (2 * D + 4) * sizeof(__half);
            int ctas = 0;
            cudaError_t r = resident_ctas(score_kernel<T, D>, kScoreThreads, 0, known, &ctas);
            if (r != cudaSuccess) return r;
            const int run = kScoreWarps * 16;           // blocks of a round
            const unsigned grid = (unsigned)std::min<long long>(ctas, (long long)rows * ((c.max_blocks + run - 1) / run));
            score_kernel<T, D><<<grid, kScoreThreads, smem, s>>>(a);
            return cudaGetLastError();
        });
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(rows);
    cfg.blockDim = dim3(kChooseThreads);
    cfg.stream = s;
    cfg.attrs = at;
    cfg.numAttrs = c.max_blocks > n_sel ? 1 : 0;
    return by_keys(c.max_blocks, [&](auto k) { return cudaLaunchKernelEx(&cfg, choose_kernel<decltype(k)::value>, a); });
}

cudaError_t launch_block8_evict(const kvq_block8& c, const int32_t* keep, int n_first, int n_last, int32_t* n_evicted,
                                cudaStream_t s) {
    const size_t smem = (size_t)c.max_blocks * sizeof(int32_t);
    return by_keys(c.max_blocks, [&](auto k) {
        auto kernel = evict_kernel<decltype(k)::value>;
        if (smem > 40 * 1024) {
            cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 51200 * 4);
            if (e != cudaSuccess) return e;
        }
        kernel<<<(unsigned)(c.B * c.Hkv), kChooseThreads, smem, s>>>(c, keep, n_first, n_last, n_evicted);
        return cudaGetLastError();
    });
}

}  // namespace kvq
