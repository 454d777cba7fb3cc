// The 8-bit block cache: reset, append, block selection and eviction (the
// attention over it is in block8_attn.cu; include/kvq.h has the format).
//
// append   one CTA per (unit, touched block): the rows of the block are held
//          in registers, one pass finds the largest magnitude and the keys'
//          minimum and maximum per channel, a second one (from registers)
//          writes the codes.  Bound by HBM: 16-bit rows in, 8-bit codes out.
// select   a score kernel (one thread per block and query: exact integer dot
//          products of the 8-bit query with the 8-bit key bounds) and a top-k
//          kernel (one CTA per query and unit).
// evict    one CTA per unit: top-k over the blocks' accumulated weights and a
//          stable partition of the table row; no codes move.
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

constexpr int kAppendThreads = 256;

// What a call does to unit u: its tokens before, the new ones (0: nothing), the touched blocks.
struct Plan {
    int count, n, first, last;      // blocks [first, last]
};

// The whole CTA calls this.  Checks the unit's room and every table entry the call needs; all
// threads get the same answer, so that a unit is either appended to as a whole or left alone.
__device__ Plan append_plan(const AppendArgs& a, int u, bool report) {
    Plan p;
    p.count = a.c.count[u];
    p.n = a.n_new ? a.n_new[u / a.c.Hkv] : a.n;
    bool bad = p.n < 0 || p.n > a.n;
    p.n = min(max(p.n, 0), a.n);
    const long long end = (long long)p.count + p.n;
    p.first = p.count / a.c.block;
    p.last = p.n > 0 ? (int)((end - 1) / a.c.block) : p.first - 1;
    bool fits = p.count >= 0 && end <= (long long)a.c.max_blocks * a.c.block;
    if (fits && p.n > 0) {
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

template <typename T> struct Packed2;
template <> struct Packed2<__half> {
    using type = __half2;
    static constexpr uint32_t kInf = 0x7c00u;
};
template <> struct Packed2<__nv_bfloat16> {
    using type = __nv_bfloat162;
    static constexpr uint32_t kInf = 0x7f80u;
};

template <typename T>
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
    using P = typename Packed2<T>::type;
    P r = __hmin2(*reinterpret_cast<P*>(&a), *reinterpret_cast<P*>(&b));
    return *reinterpret_cast<uint32_t*>(&r);
}
template <typename T>
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    using P = typename Packed2<T>::type;
    P r = __hmax2(*reinterpret_cast<P*>(&a), *reinterpret_cast<P*>(&b));
    return *reinterpret_cast<uint32_t*>(&r);
}
template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t a) {
    T* h = reinterpret_cast<T*>(&a);
    return make_float2(Elem<T>::to_f(h[0]), Elem<T>::to_f(h[1]));
}

struct AppendShared {
    uint32_t amax[kAppendThreads / 32];
    uint32_t lo[kAppendThreads / 32][64], hi[kAppendThreads / 32][64];  // packed channel pairs per warp
    float sum[kAppendThreads / 32];
};

// Keys or values of one block.  Rows [0, fill) are the open block's 16-bit rows, rows
// [fill, end) new ones (row r is x + (r - fill) * stride); the block stays open if end < P.
// PASSES rows per thread: thread i holds 8 channels of row i / (D/8), + RPP, + 2 RPP ...
//
// A block whose scale does not grow needs only its new rows: the codes of the others stand, and
// the bounds are the old ones widened by the new rows' (floor and ceil are monotone), exactly
// what a quantisation of all rows gives.  A scale grows 1/fill of the time, so a decode step
// reads one row instead of the whole open block.
template <typename T, int D, int CODE, int PASSES, bool IS_K>
__device__ void append_block(const kvq_block8& c, int phys, int fill, int end, const T* x, int64_t stride, T* tail,
                             AppendShared& sh) {
    constexpr int TPR = D / 8, RPP = kAppendThreads / TPR;
    const int col = threadIdx.x % TPR, row0 = threadIdx.x / TPR, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    constexpr uint32_t kInf2 = Packed2<T>::kInf * 0x10001u;
    float* scale = IS_K ? c.k_scale : c.v_scale;
    uint8_t* codes = (IS_K ? c.k_codes : c.v_codes) + (size_t)phys * c.block * D;
    const float old_s = scale[phys], old_b = IS_K ? c.bound_scale[phys] : 0.0f;
    uint4 r[PASSES];
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
        const int row = p * RPP + row0;
        r[p] = make_uint4(0, 0, 0, 0);
        if (row >= fill && row < end)
            r[p] = *reinterpret_cast<const uint4*>(x + (int64_t)(row - fill) * stride + col * 8);
    }
    int from = fill;                    // first row that counts below
    bool grow, finite;
    float s, sb;
    for (;;) {
        uint32_t m = 0;
#pragma unroll
        for (int p = 0; p < PASSES; ++p) {
            m = __vmaxu2(m, __vmaxu2(__vmaxu2(r[p].x & 0x7fff7fffu, r[p].y & 0x7fff7fffu),
                                     __vmaxu2(r[p].z & 0x7fff7fffu, r[p].w & 0x7fff7fffu)));
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, o));
        if (lane == 0) sh.amax[warp] = m;
        __syncthreads();
        m = 0;
#pragma unroll
        for (int w = 0; w < kAppendThreads / 32; ++w) m = __vmaxu2(m, sh.amax[w]);
        __syncthreads();
        m = max(m & 0xffffu, m >> 16);
        finite = m < Packed2<T>::kInf;
        const float amax = unpack2<T>(m).x;
        s = finite ? scale_of(amax, Code<CODE>::kInvMax) : __int_as_float(0x7fc00000);
        sb = finite ? scale_of(amax, kInv127) : __int_as_float(0x7fc00000);
        grow = from > 0 && !(s <= old_s && (!IS_K || sb <= old_b));
        if (!grow) break;
        // the scale grows: every row of the block counts
#pragma unroll
        for (int p = 0; p < PASSES; ++p) {
            const int row = p * RPP + row0;
            if (row < fill) r[p] = *reinterpret_cast<const uint4*>(tail + (size_t)row * D + col * 8);
        }
        from = 0;
    }
    const bool widen = from > 0;        // the old scale stands
    if (widen) {
        s = old_s;
        sb = old_b;
    }
    const float inv = __frcp_rn(s);
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
        const int row = p * RPP + row0;
        if (row >= from && row < end) {
            uint2 q = make_uint2(0, 0);
            if (finite) {
                const float2 f0 = unpack2<T>(r[p].x), f1 = unpack2<T>(r[p].y), f2 = unpack2<T>(r[p].z),
                             f3 = unpack2<T>(r[p].w);
                q.x = code_pair<CODE>(f0.x, f0.y, inv) | (code_pair<CODE>(f1.x, f1.y, inv) << 16);
                q.y = code_pair<CODE>(f2.x, f2.y, inv) | (code_pair<CODE>(f3.x, f3.y, inv) << 16);
            }
            *reinterpret_cast<uint2*>(codes + (size_t)row * D + col * 8) = q;
            if (end < c.block && row >= fill) *reinterpret_cast<uint4*>(tail + (size_t)row * D + col * 8) = r[p];
        }
    }
    if constexpr (IS_K) {
        uint32_t lo[4], hi[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            lo[i] = kInf2;
            hi[i] = kInf2 | 0x80008000u;
        }
#pragma unroll
        for (int p = 0; p < PASSES; ++p) {
            const int row = p * RPP + row0;
            if (row >= from && row < end) {
                const uint32_t w[4] = {r[p].x, r[p].y, r[p].z, r[p].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    lo[i] = min2<T>(lo[i], w[i]);
                    hi[i] = max2<T>(hi[i], w[i]);
                }
            }
        }
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
        __syncthreads();
        if (threadIdx.x < D / 2) {
            uint32_t l = sh.lo[0][threadIdx.x], h = sh.hi[0][threadIdx.x];
#pragma unroll
            for (int w = 1; w < kAppendThreads / 32; ++w) {
                l = min2<T>(l, sh.lo[w][threadIdx.x]);
                h = max2<T>(h, sh.hi[w][threadIdx.x]);
            }
            const float ib = __frcp_rn(sb);
            const float2 fl = unpack2<T>(l), fh = unpack2<T>(h);
            int l0 = 0, l1 = 0, h0 = 0, h1 = 0;
            if (finite) {
                l0 = (int)fmaxf(-127.0f, fminf(127.0f, floorf(__fmul_rn(fl.x, ib))));
                l1 = (int)fmaxf(-127.0f, fminf(127.0f, floorf(__fmul_rn(fl.y, ib))));
                h0 = (int)fmaxf(-127.0f, fminf(127.0f, ceilf(__fmul_rn(fh.x, ib))));
                h1 = (int)fmaxf(-127.0f, fminf(127.0f, ceilf(__fmul_rn(fh.y, ib))));
            }
            char2* lp = reinterpret_cast<char2*>(c.k_bound + (size_t)phys * 2 * D) + threadIdx.x;
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
        __syncthreads();                // sh is used again
    }
    if (threadIdx.x == 0) {
        scale[phys] = s;
        if (IS_K) c.bound_scale[phys] = sb;
    }
}

template <typename T, int D, int CODE, int PASSES>
__device__ void append_one(const AppendArgs& a, const Plan& p, int u, int block, AppendShared& sh) {
    const kvq_block8& c = a.c;
    const int P = c.block, b = u / c.Hkv, h = u % c.Hkv;
    const int fill = max(0, p.count - block * P), end = min(P, p.count + p.n - block * P);
    const int t0 = block * P + fill - p.count;                  // the block's first new token
    const int phys = c.table[(size_t)u * c.max_blocks + block];
    const T* k = (const T*)a.k + b * a.ks[0] + h * a.ks[1] + t0 * a.ks[2];
    const T* v = (const T*)a.v + b * a.vs[0] + h * a.vs[1] + t0 * a.vs[2];
    T* tk = (T*)c.tail_k + (size_t)u * P * D;
    T* tv = (T*)c.tail_v + (size_t)u * P * D;
    append_block<T, D, CODE, PASSES, true>(c, phys, fill, end, k, a.ks[2], tk, sh);
    append_block<T, D, CODE, PASSES, false>(c, phys, fill, end, v, a.vs[2], tv, sh);
    float sum = 0.0f;
    if (a.colscore) {
        const int g = c.Hq / c.Hkv, m = end - fill;
        const float* cs = a.colscore + ((size_t)b * c.Hq + (size_t)h * g) * a.n + t0;
        for (int i = threadIdx.x; i < g * m; i += kAppendThreads) sum += cs[(size_t)(i / m) * a.n + i % m];
#pragma unroll
        for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if ((threadIdx.x & 31) == 0) sh.sum[threadIdx.x >> 5] = sum;
        __syncthreads();
        sum = 0.0f;
        for (int w = 0; w < kAppendThreads / 32; ++w) sum += sh.sum[w];
    }
    if (threadIdx.x == 0) {
        if (fill == 0) c.block_pos[phys] = c.seq_len[u] + block * P - p.count;
        if (fill == 0 || a.colscore) c.acc[phys] = (fill == 0 ? 0.0f : c.acc[phys]) + sum;
    }
    __syncthreads();
}

// Grid: x = unit + units * j.  CTA j = 0 of a unit takes the first touched block and, where that
// one was open, the last one too if it stays open: both use the unit's tail rows, the first reads
// them before the last one writes them.  CTA j takes block first + j.  commit: the CTA is alone
// (n <= block touches at most those two blocks) and sets the counters itself.
template <typename T, int D, int CODE, int PASSES>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(AppendArgs a, int commit) {
    __shared__ AppendShared sh;
    const int units = a.c.B * a.c.Hkv, u = blockIdx.x % units, j = blockIdx.x / units;
    const Plan p = append_plan(a, u, j == 0);
    if (p.n == 0) return;
    const bool open_first = p.count % a.c.block != 0, open_last = (p.count + p.n) % a.c.block != 0;
    const bool pair = open_first && open_last && p.last > p.first;
    if (p.first + j < p.last || (p.first + j == p.last && !(pair && j > 0)))
        append_one<T, D, CODE, PASSES>(a, p, u, p.first + j, sh);
    if (j == 0 && pair) append_one<T, D, CODE, PASSES>(a, p, u, p.last, sh);
    if (commit && threadIdx.x == 0) {
        a.c.count[u] = p.count + p.n;
        a.c.seq_len[u] += p.n;
    }
}

__global__ void __launch_bounds__(kAppendThreads) append_commit_kernel(AppendArgs a) {
    const int u = blockIdx.x;
    const Plan p = append_plan(a, u, false);
    if (threadIdx.x == 0 && p.n > 0) {
        a.c.count[u] = p.count + p.n;
        a.c.seq_len[u] += p.n;
    }
}

template <typename T, int D, int CODE, int PASSES>
cudaError_t launch_append_passes(const AppendArgs& a, cudaStream_t s) {
    const unsigned units = (unsigned)(a.c.B * a.c.Hkv);
    if (a.n <= a.c.block) {
        append_kernel<T, D, CODE, PASSES><<<units, kAppendThreads, 0, s>>>(a, 1);
        return cudaGetLastError();
    }
    const unsigned per = (unsigned)((a.n + a.c.block - 2) / a.c.block + 1);
    append_kernel<T, D, CODE, PASSES><<<units * per, kAppendThreads, 0, s>>>(a, 0);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    append_commit_kernel<<<units, kAppendThreads, 0, s>>>(a);
    return cudaGetLastError();
}

template <typename T, int D, int CODE>
cudaError_t launch_append_typed(const AppendArgs& a, cudaStream_t s) {
    constexpr int RPP = kAppendThreads / (D / 8);
    const int passes = (a.c.block + RPP - 1) / RPP;
    if (passes <= 1) return launch_append_passes<T, D, CODE, 1>(a, s);
    if (passes <= 2) return launch_append_passes<T, D, CODE, 2>(a, s);
    if (passes <= 4) return launch_append_passes<T, D, CODE, 4>(a, s);
    return launch_append_passes<T, D, CODE, 8>(a, s);
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

constexpr int kScoreThreads = 128;
constexpr int kHeadTile = 8;        // heads whose sums a thread holds at once

// One thread per (block, query): sum_c max(q8 low, q8 high) = q8+ . high + q8- . low per head, exact
// in int32 (4-byte dot products), then the largest of the group's heads.  q8+ and q8- of the
// group sit in shared memory and are read by all lanes at once; a thread reads its own block's
// 2 D bytes of bounds in 16-byte pieces.
template <typename T, int D>
__global__ void __launch_bounds__(kScoreThreads) score_kernel(SelectArgs a) {
    extern __shared__ __align__(16) uint32_t q8[];      // [g][2][D/4]
    __shared__ float sq[KVQ_BLOCK8_MAX_GROUP];
    const kvq_block8& c = a.c;
    const int units = c.B * c.Hkv, rows = units * a.n_q;
    const int row = blockIdx.x % rows, chunk = blockIdx.x / rows;
    const int u = row / a.n_q, t = row % a.n_q, b = u / c.Hkv, h = u % c.Hkv, g = c.Hq / c.Hkv;
    const int m = new_rows(a.n_new, b, a.n_q, &g_status_block8);
    const int limit = min(query_limit(c.count[u], m, t), c.max_blocks * c.block);
    const int nb = (limit + c.block - 1) / c.block;
    if (chunk * kScoreThreads >= nb || nb <= a.n_sel) return;        // few blocks: all are chosen
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int hh = warp; hh < g; hh += kScoreThreads / 32) {
        const T* q = (const T*)a.q + b * a.qs[0] + (int64_t)(h * g + hh) * a.qs[1] + t * a.qs[2];
        float x[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        if (lane < D / 4) {
            const uint2 w = *reinterpret_cast<const uint2*>(q + lane * 4);
            const T* e = reinterpret_cast<const T*>(&w);
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = Elem<T>::to_f(e[i]);
        }
        uint32_t mx = 0;                                // magnitudes as bits: NaN and infinity rank above all
#pragma unroll
        for (int i = 0; i < 4; ++i) mx = max(mx, __float_as_uint(x[i]) & 0x7fffffffu);
        mx = __reduce_max_sync(0xffffffffu, mx);
        const bool finite = mx < 0x7f800000u;
        const float s = finite ? scale_of(__uint_as_float(mx), kInv127) : __int_as_float(0x7fc00000);
        const float inv = __frcp_rn(s);
        uint32_t pos = 0, neg = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int v = finite ? min(127, max(-127, __float2int_rn(__fmul_rn(x[i], inv)))) : 0;
            pos |= (uint32_t)(max(v, 0) & 255) << (8 * i);
            neg |= (uint32_t)(min(v, 0) & 255) << (8 * i);
        }
        if (lane < D / 4) {
            q8[(hh * 2 + 0) * (D / 4) + lane] = pos;
            q8[(hh * 2 + 1) * (D / 4) + lane] = neg;
        }
        if (lane == 0) sq[hh] = s;
    }
    __syncthreads();
    const int i = chunk * kScoreThreads + threadIdx.x;
    if (i >= nb) return;
    const int phys = c.table[(size_t)u * c.max_blocks + i];
    float best = -INFINITY;
    if ((unsigned)phys < (unsigned)c.n_blocks) {
        const uint4* bound = reinterpret_cast<const uint4*>(c.k_bound + (size_t)phys * 2 * D);
        bool nan = false;
        for (int h0 = 0; h0 < g; h0 += kHeadTile) {
            int acc[kHeadTile] = {};
            for (int ch = 0; ch < D / 16; ++ch) {
                const uint4 lo = bound[ch], hi = bound[D / 16 + ch];
#pragma unroll
                for (int k = 0; k < kHeadTile; ++k) {
                    if (h0 + k < g) {
                        const uint4 p = reinterpret_cast<const uint4*>(q8)[(h0 + k) * (2 * D / 16) + ch];
                        const uint4 n = reinterpret_cast<const uint4*>(q8)[(h0 + k) * (2 * D / 16) + D / 16 + ch];
                        int s = acc[k];
                        s = __dp4a((int)hi.x, (int)p.x, s);
                        s = __dp4a((int)hi.y, (int)p.y, s);
                        s = __dp4a((int)hi.z, (int)p.z, s);
                        s = __dp4a((int)hi.w, (int)p.w, s);
                        s = __dp4a((int)lo.x, (int)n.x, s);
                        s = __dp4a((int)lo.y, (int)n.y, s);
                        s = __dp4a((int)lo.z, (int)n.z, s);
                        s = __dp4a((int)lo.w, (int)n.w, s);
                        acc[k] = s;
                    }
                }
            }
#pragma unroll
            for (int k = 0; k < kHeadTile; ++k)
                if (h0 + k < g) {
                    const float f = __fmul_rn((float)acc[k], sq[h0 + k]);
                    nan = nan || isnan(f);
                    best = fmaxf(best, f);
                }
        }
        best = nan ? __int_as_float(0x7fc00000) : __fmul_rn(best, c.bound_scale[phys]);
    } else {
        atomicOr(&g_status_block8, kDevCheck);
    }
    a.score[(size_t)row * c.max_blocks + i] = best;
}

// Block [first, n - last) of n: writes the k of the largest key(i) in ascending order from out[at].
template <typename KeyFn, typename PutFn>
__device__ void choose(KeyFn key, int first, int n, int k, TopkShared& sh, PutFn put) {
    uint32_t kstar = 0, take_eq = 0;
    if (k > 0) block_radix_select([&](int i) { return key(first + i); }, n, k, sh, &kstar, &take_eq);
    uint32_t eq_base = 0;
    for (int c0 = 0; c0 < n; c0 += blockDim.x) {
        const int i = c0 + threadIdx.x;
        const uint32_t kv = i < n ? key(first + i) : 0u;
        const uint32_t gt = (k > 0 && i < n && kv > kstar) ? 1u : 0u;
        const uint32_t eq = (k > 0 && i < n && kv == kstar) ? 1u : 0u;
        uint32_t eq_tot;
        const uint32_t eq_rank = block_excl_scan(eq, sh, &eq_tot);
        put(first + i, i < n, gt | (eq & (eq_base + eq_rank < take_eq ? 1u : 0u)));
        eq_base += eq_tot;
    }
}

__global__ void __launch_bounds__(kTopkBlock) choose_kernel(SelectArgs a) {
    __shared__ TopkShared sh;
    const kvq_block8& c = a.c;
    const int row = blockIdx.x, u = row / a.n_q, t = row % a.n_q;
    const int m = new_rows(a.n_new, u / c.Hkv, a.n_q, &g_status_block8);
    const int limit = min(query_limit(c.count[u], m, t), c.max_blocks * c.block);
    const int nb = (limit + c.block - 1) / c.block;
    int32_t* out = a.idx_out + (size_t)row * a.n_sel;
    const int n = min(nb, a.n_sel);
    if (nb <= a.n_sel) {
        for (int i = threadIdx.x; i < a.n_sel; i += blockDim.x) out[i] = i < nb ? i : -1;
    } else {
        const float* score = a.score + (size_t)row * c.max_blocks;
        for (int i = threadIdx.x; i < a.n_first; i += blockDim.x) out[i] = i;
        for (int i = threadIdx.x; i < a.n_last; i += blockDim.x) out[a.n_sel - a.n_last + i] = nb - a.n_last + i;
        uint32_t base = (uint32_t)a.n_first;
        choose([&](int i) { return rank_key(score[i]); }, a.n_first, nb - a.n_first - a.n_last,
               a.n_sel - a.n_first - a.n_last, sh, [&](int i, bool, uint32_t sel) {
                   uint32_t tot;
                   const uint32_t pos = block_excl_scan(sel, sh, &tot);
                   if (sel) out[base + pos] = i;
                   base += tot;
               });
    }
    if (threadIdx.x == 0) a.n_out[row] = n;
}

// ------------------------------------------------------------------ evict

// keys[i]: the rank key of block i's weight; once block i has been placed, entry e <= i holds the
// e-th block that left (the table row is rewritten front to back, each entry after it was read).
__global__ void __launch_bounds__(kTopkBlock) evict_kernel(kvq_block8 c, const int32_t* __restrict__ keep, int n_first,
                                                          int n_last, int32_t* __restrict__ n_evicted) {
    extern __shared__ uint32_t keys[];
    __shared__ TopkShared sh;
    const int u = blockIdx.x, count = min(max(c.count[u], 0), c.max_blocks * c.block);
    const int nb = (count + c.block - 1) / c.block;
    const int want = max(keep[u], n_first + n_last);
    if (nb <= want) {
        if (threadIdx.x == 0 && n_evicted) n_evicted[u] = 0;
        return;
    }
    int32_t* row = c.table + (size_t)u * c.max_blocks;
    for (int i = threadIdx.x; i < nb; i += blockDim.x) {
        const int phys = row[i];
        const bool ok = (unsigned)phys < (unsigned)c.n_blocks;
        if (!ok) atomicOr(&g_status_block8, kDevCheck);
        keys[i] = ok ? rank_key(c.acc[phys]) : 0u;
    }
    __syncthreads();
    uint32_t kept = (uint32_t)n_first, gone = 0;
    choose([&](int i) { return keys[i]; }, n_first, nb - n_first - n_last, want - n_first - n_last, sh,
           [&](int i, bool in, uint32_t sel) {
               const int phys = in ? row[i] : 0;
               uint32_t tot, out_tot;
               const uint32_t pos = block_excl_scan(sel, sh, &tot);
               const uint32_t out = block_excl_scan(in && !sel ? 1u : 0u, sh, &out_tot);
               if (in && sel) row[kept + pos] = phys;
               if (in && !sel) keys[gone + out] = (uint32_t)phys;
               kept += tot;
               gone += out_tot;
               __syncthreads();
           });
    for (int i0 = 0; i0 < n_last; i0 += blockDim.x) {   // front to back: kept + i <= nb - n_last + i
        const int i = i0 + threadIdx.x;
        const int phys = i < n_last ? row[nb - n_last + i] : 0;
        __syncthreads();
        if (i < n_last) row[kept + i] = phys;
        __syncthreads();
    }
    for (uint32_t i = threadIdx.x; i < gone; i += blockDim.x) row[want + i] = (int32_t)keys[i];
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
        const unsigned chunks = (unsigned)((c.max_blocks + kScoreThreads - 1) / kScoreThreads);
        cudaError_t e = by_type(c, [&](auto t, auto d) {
            using T = decltype(t);
            constexpr int D = decltype(d)::value;
            score_kernel<T, D><<<rows * chunks, kScoreThreads, (size_t)(c.Hq / c.Hkv) * 2 * D, s>>>(a);
            return cudaGetLastError();
        });
        if (e != cudaSuccess) return e;
    }
    choose_kernel<<<rows, kTopkBlock, 0, s>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_block8_evict(const kvq_block8& c, const int32_t* keep, int n_first, int n_last, int32_t* n_evicted,
                                cudaStream_t s) {
    const size_t smem = (size_t)c.max_blocks * sizeof(uint32_t);
    if (smem > 40 * 1024) {
        cudaError_t e = cudaFuncSetAttribute(evict_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 51200 * 4);
        if (e != cudaSuccess) return e;
    }
    evict_kernel<<<(unsigned)(c.B * c.Hkv), kTopkBlock, smem, s>>>(c, keep, n_first, n_last, n_evicted);
    return cudaGetLastError();
}

}  // namespace kvq
