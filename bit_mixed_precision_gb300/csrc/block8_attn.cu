// block8_attn: attention of a few queries over the 8-bit block cache, over all
// tokens or over a list of blocks per query (include/kvq.h has the format).
//
// Mathematics.  A logit is s_j = (q . c_j) k_scale sigma log2(e): codes and
// 16-bit queries multiply exactly in fp16 MMAs with float32 sums.  With the
// value scale v as a power of two in the exponent, the second product is over the
// value codes with weights 2^(s_j + log2 v - M), M one running reference per query
// row, so blocks whose value scales lie many powers of two apart share one fp16
// range; a weight enters as a pair of fp16 numbers (22 bits).  The sum of the same
// weights times 1 / v beside it gives the softmax denominator, so that the
// rounding of log2 v (2^-22) only shifts a block's logits by as much.  bf16 value
// scales may be so far apart that float32 loses weights that count there: kFar below.
//
// Work.  The rows that read a unit together (queries x heads of the group, up to
// 8, 16 or 32 of them) and its tokens, or a query's listed blocks, form a work unit;
// its tokens are cut into tiles of 32 (16 for more than 8 rows).  All work units' tiles form one list, split
// evenly over the resident CTAs, whatever the lengths (each CTA adds up the
// units' tile counts itself).  In a CTA the four warps take the tiles of its run
// in turn, each with its own state: tokens are the M rows of the first MMA and
// channels those of the second, so that 8 rows cost one n = 8 column block.  The
// codes go from global memory straight to the registers where the fragments
// want them: a lane's 16-byte pieces of a key row are the k elements of four
// MMAs (the query fragments use the same channel order), and its 16-byte pieces
// of four value rows, transposed by byte permutes, are the fragments of eight.
// A tile's key registers are loaded again for the next tile as soon as the first
// product has read them, the value registers after the second.  At the end of
// a unit's run the warps meet in shared memory and the CTA writes one partial
// state; a second kernel, a programmatic dependent, joins the partials of a unit
// and, with accumulate, adds the blocks' shares of the weights, in a fixed order.
// Small caches (kDirectCells) take one CTA per work unit and no second kernel.
//
// Bound by HBM: 2 D bytes per token and KV head against 4 D g flop.  512 units of 32768 tokens, D 128,
// four heads, e4m3, weights accumulated: 678 us, 0.93 of the measured 6.79 TB/s; 256 ragged units of up
// to 8192, five heads, int8: 55 us, 0.78 (5 us go before the first tile, int8 codes take 380 warp
// instructions per 16 tokens).  With 32 rows the tensor cores' share is larger than HBM's: 64 units of up
// to 20011 tokens 88 us, 0.40, behind fixed-latency waits of two warps per scheduler.  With D 128 the
// variants of up to 16 rows use 168 registers, those of 32 rows 255, and spill up to 60 bytes.
#include <algorithm>
#include <type_traits>

#include "block8_device.cuh"
#include "kvq_internal.h"

namespace kvq {

KVQ_DEFINE_STATUS(block8_attn)

namespace {

using namespace b8;

constexpr int kWarps = 4, kThreads = kWarps * 32;
constexpr int kMaxCtas = 1024;          // CTAs of the first kernel at most (sizes the workspace)
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
// The reference starts 2^7 below a row's largest weight and moves only when one passes it by 2^15:
// weights fit fp16, and 2^-31 of the largest is still a weight.  kNone: no logit yet (finite, so that
// differences of references are numbers).
constexpr float kShift = 7.0f, kLift = 15.0f, kNone = -1.0e38f;

// The softmax denominator does not know the value scales, the exponents above do.  fp16 values keep
// log2 v within -64 .. 9.1, and what float32 flushes (2^-126) is then below 2^-53 of the denominator.
// bf16 values reach from -64 (a block of zeros) to 121.  So for bf16 a warp whose cells' log2 v span
// more than kFar takes the part of the lower ones in the denominator from a second exponential without
// log2 v (with kBias more: the largest value scale alone puts the denominator at 2^-114), beside the
// rare moves of the reference; and a reference that far below another lowers its denominator in two steps.
// It costs bf16 1 to 2 % (512 units of 32768 tokens 670 -> 678 us, 32 rows 86.1 -> 88.1, 32 units of up to
// 64 tokens 7.2 -> 7.6); tested in the loop for every tile, 32 rows took 90.5.
constexpr float kFar = 80.0f, kBias = 24.0f, kBiasInv = 1.0f / 16777216.0f;
template <typename T> constexpr bool kWide = std::is_same<T, __nv_bfloat16>::value;

// l 2^d, d <= 0: l may be as large as 2^(64 + kLift) a token while 2^d alone is flushed.
template <bool WIDE>
__device__ __forceinline__ float lowered(float l, float d) {
    if constexpr (!WIDE) return l * ex2_approx(d);
    const float f = ex2_approx(d < -64.0f ? 0.5f * d : d);
    return l * f * (d < -64.0f ? f : 1.0f);
}

// Work units of at most this many 16-token cells (twice as many where the units alone give every SM a
// CTA) are each taken by one CTA that writes o and lse itself, without the second kernel: 2 to 32 units
// of 64, 128 and 256 tokens 4.1 to 4.5, 4.3 to 4.7, 5.5 to 5.8 us against 6.3 to 7.7 the other way; of 512
// 7.5 to 7.9 against 7.2 to 7.9, of 1024 11.5 against 7.6.  512 units of 512 tokens 18.7 against 21.8, of
// 1024 35.6 against 31.8.  (By room, not by tokens held: the host does not know those.)
constexpr int kDirectCells = 16;

struct AttnArgs {
    kvq_block8 c;
    const void* q;
    int64_t qs[3];
    int n_q;
    const int32_t* n_new;
    float sm_scale;
    const int32_t *blocks, *list_len;
    int n_sel;
    void* o;
    float* lse;
    // derived
    int n_list;                         // entries of a list that can count
    int g, row_tiles, works;            // work units = units (x n_q with lists) x row_tiles
    int cells;                          // 16-token cells per work unit at most
    int direct;                         // one CTA per work unit that writes o and lse itself
    // workspace
    float *part, *ml, *mass;            // [slot][rows][D], [slot][rows][2], [work][cells][rows]
    int2* span;                         // [work] first and last CTA
};

// Shapes by the number of 8-row column blocks.  One (up to 8 rows): tiles of two cells, query fragments
// in registers, three CTAs per SM.  Two and four share a tile's converted codes among 16 or 32 rows;
// their accumulators leave room for one cell, and the fragments are read from shared memory.  32 rows in
// one pass of four column blocks took 86 us where two passes of two took 94 to 97.
template <int NT> struct Shape {
    static constexpr int C = NT == 1 ? 2 : 1;           // 16-token cells of a tile
    static constexpr int kCtas = NT == 4 ? 2 : 3;       // resident CTAs per SM
    static constexpr bool kSharedQ = NT > 1;
};

// What a work unit is and sees.
struct Work {
    int u, b, t0, rows;                 // unit, sequence, first query (the only one with lists), valid + padding rows
    int tiles, top;                     // tiles; tokens that its last query sees
    int list_n;                         // listed blocks
};

template <int NT, bool LIST>
__device__ __forceinline__ Work work_of(const AttnArgs& a, int w) {
    Work k;                             // one row tile, one query: the usual case, without the divisions
    const bool tiled = a.row_tiles > 1, one = a.n_q == 1;
    const int rt = tiled ? w % a.row_tiles : 0, x = tiled ? w / a.row_tiles : w;
    k.u = LIST && !one ? x / a.n_q : x;
    k.b = k.u / a.c.Hkv;
    const int m = a.n_new ? new_rows(a.n_new, k.b, a.n_q, &g_status_block8_attn) : a.n_q;
    const int count = min(a.c.count[k.u], a.c.max_blocks * a.c.block);
    const int r0 = rt * 8 * NT, all = LIST ? a.g : a.g * a.n_q;
    k.rows = min(8 * NT, all - r0);
    const int first = one ? 0 : LIST ? x % a.n_q : r0 / a.g, last = one ? 0 : LIST ? first : (r0 + k.rows - 1) / a.g;
    k.t0 = first;
    k.top = first < m ? query_limit(count, m, min(last, m - 1)) : 0;
    k.list_n = 0;
    if (LIST) {
        const int n = a.list_len[x];
        if (n < 0 || n > a.n_list) atomicOr(&g_status_block8_attn, kDevCheck);
        k.list_n = k.top > 0 ? min(max(n, 0), a.n_list) : 0;
        k.tiles = (k.list_n * (a.c.block / 16) + Shape<NT>::C - 1) / Shape<NT>::C;
    } else {
        k.tiles = (k.top + 16 * Shape<NT>::C - 1) / (16 * Shape<NT>::C);
    }
    return k;
}

// Query and head (within the group) of row i of a work unit.
template <int NT, bool LIST>
__device__ __forceinline__ int2 row_of(const AttnArgs& a, const Work& k, int w, int i) {
    const int r = a.row_tiles > 1 ? (w % a.row_tiles) * 8 * NT + i : i;
    return LIST || a.n_q == 1 ? make_int2(k.t0, r) : make_int2(r / a.g, r % a.g);
}

// ------------------------------------------------------------------ pieces of the inner loop

__device__ __forceinline__ uint2 load8(const uint8_t* p) {
    uint2 v;
    asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
    return v;
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// (a, b) rounded to an fp16 pair and the pair of the remainders.
__device__ __forceinline__ void split2(float a, float b, uint32_t& hi, uint32_t& lo) {
    __half2 h = __floats2half2_rn(a, b);
    const float2 f = __half22float2(h);
    __half2 r = __floats2half2_rn(a - f.x, b - f.y);
    hi = *reinterpret_cast<uint32_t*>(&h);
    lo = *reinterpret_cast<uint32_t*>(&r);
}

// One lane's registers of a 16-token cell.
template <int D> struct KeyRegs { uint4 r[2][D / 64]; };        // rows g, g + 8; pieces of 16 channels
template <int D> struct ValueRegs { uint32_t r[4][D / 32]; };   // rows 2t, 2t + 1, 2t + 8, 2t + 9; D/8 channels

template <int D>
__device__ __forceinline__ void load_keys(KeyRegs<D>& k, const uint8_t* codes, uint32_t cell, int g, int t) {
    if (cell == 0xffffffffu) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < D / 64; ++j) k.r[i][j] = make_uint4(0, 0, 0, 0);
        return;
    }
    const uint8_t* p = codes + (size_t)cell * (16 * D) + g * D + t * 16;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < D / 64; ++j) k.r[i][j] = load16(p + i * 8 * D + j * 64);
}

template <int D>
__device__ __forceinline__ void load_values(ValueRegs<D>& v, const uint8_t* codes, uint32_t cell, int g, int t) {
    if (cell == 0xffffffffu) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < D / 32; ++j) v.r[i][j] = 0;
        return;
    }
    const uint8_t* p = codes + (size_t)cell * (16 * D) + 2 * t * D + g * (D / 8);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint8_t* row = p + ((i & 1) + (i >> 1) * 8) * D;
        if constexpr (D == 128) {
            const uint4 x = load16(row);
            v.r[i][0] = x.x; v.r[i][1] = x.y; v.r[i][2] = x.z; v.r[i][3] = x.w;
        } else {
            const uint2 x = load8(row);
            v.r[i][0] = x.x; v.r[i][1] = x.y;
        }
    }
}

// Where a warp's next 32 / C tiles lie: lane C i + j holds cell j of its i-th tile.
struct Cells {
    uint32_t cell;                      // number of the 16-token cell in the pool, ~0 for none
    int slot;                           // its first token in the unit
    float ks, lv, rv;                   // k_scale sigma log2(e); log2 and reciprocal of v_scale (NaN: NaN and 0)
};

template <int C, bool LIST>
__device__ __forceinline__ Cells find_cells(const AttnArgs& a, const Work& k, int w, int tile, int end, int lane) {
    Cells x;
    x.cell = 0xffffffffu;
    x.slot = 0;
    x.ks = 0.0f;
    x.lv = 0.0f;
    x.rv = 1.0f;
    const int my = tile + (lane / C) * kWarps, cell = C * my + lane % C;
    if (my < end) {
        const int per = a.c.block / 16, j = cell / per, in = cell % per;
        int blk = j;
        bool there;
        if (LIST) {
            there = j < k.list_n;
            if (there) {
                blk = a.blocks[(size_t)(w / a.row_tiles) * a.n_sel + j];
                const int held = (min(a.c.count[k.u], a.c.max_blocks * a.c.block) + a.c.block - 1) / a.c.block;
                if ((unsigned)blk >= (unsigned)held) {
                    atomicOr(&g_status_block8_attn, kDevCheck);
                    there = false;
                }
            }
        } else {
            there = cell * 16 < k.top;
        }
        if (there) {
            x.slot = blk * a.c.block + in * 16;
            if (x.slot < k.top) {
                const int phys = a.c.table[(size_t)k.u * a.c.max_blocks + blk];
                if ((unsigned)phys < (unsigned)a.c.n_blocks) {
                    x.cell = (uint32_t)phys * per + in;
                    x.ks = a.c.k_scale[phys] * (a.sm_scale * kLog2e);
                    const float vs = a.c.v_scale[phys];
                    x.lv = log2f(vs);
                    x.rv = isnan(vs) ? 0.0f : __frcp_rn(vs);
                } else {
                    atomicOr(&g_status_block8_attn, kDevCheck);
                }
            }
        }
    }
    return x;
}

// Takes the lanes' log2 v into the warp's range: whether it is wider than kFar.
__device__ __forceinline__ bool scales_apart(float2& range, float lv, float2 before) {
    float hi = lv, lo = lv;
#pragma unroll
    for (int x = 1; x < 32; x <<= 1) {
        hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, x));
        lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, x));
    }
    hi = fmaxf(hi, before.x);
    lo = fminf(lo, before.y);
    __syncwarp();                       // `before` may be the range: every lane has read it
    if ((threadIdx.x & 31) == 0) range = make_float2(hi, lo);
    __syncwarp();
    return hi - lo > kFar;
}

// Asks L2 for the cells of tile i of those in `x`; nothing waits for them.  One tile ahead (the tile
// whose registers are loaded next): 712 -> 681 us on 512 units of 32768 tokens; two, three and five
// ahead 691, 695, 709.
template <int D, int C>
__device__ __forceinline__ void ask_l2(const kvq_block8& c, const Cells& x, int i, int lane) {
    if (lane / C == i && x.cell != 0xffffffffu) {
        bulk_prefetch_l2(c.k_codes + (size_t)x.cell * (16 * D), 16 * D);
        bulk_prefetch_l2(c.v_codes + (size_t)x.cell * (16 * D), 16 * D);
    }
}

// Channels d .. d + 3 of a row's output, and lse with the first ones.
template <typename T, int NT, bool LIST>
__device__ __forceinline__ void write_row(const AttnArgs& a, const Work& k, int w, int row, int d, float4 y, float ref,
                                          float sum) {
    const int2 th = row_of<NT, LIST>(a, k, w, row);
    const int m = a.n_new ? min(max(a.n_new[k.b], 0), a.n_q) : a.n_q;
    const bool sees = th.x < m && sum != 0.0f;
    const float inv = sees ? 1.0f / sum : 0.0f;
    const size_t orow = ((size_t)k.b * a.c.Hq + (size_t)(k.u % a.c.Hkv) * a.g + th.y) * a.n_q + th.x;
    T t[4] = {Elem<T>::from_f(sees ? y.x * inv : 0.0f), Elem<T>::from_f(sees ? y.y * inv : 0.0f),
              Elem<T>::from_f(sees ? y.z * inv : 0.0f), Elem<T>::from_f(sees ? y.w * inv : 0.0f)};
    *reinterpret_cast<uint2*>((T*)a.o + orow * a.c.D + d) = *reinterpret_cast<uint2*>(t);
    if (d == 0 && a.lse) a.lse[orow] = sees ? (ref + log2f(sum)) * kLn2 : -INFINITY;
}

template <int D, int NT>
struct alignas(16) Shared {
    float o[kWarps][8][D + 4];          // one column block at a time
    float ml[kWarps][8 * NT][2];
    __half q[Shape<NT>::kSharedQ ? 8 * NT : 1][D + 4];          // queries as fp16, rows padded
    float undo[8 * NT];
    float2 lv[kWarps];                  // largest and least log2 v of the cells that a warp has looked up
    RunShared<kThreads> run;
};

template <typename T, int D, int CODE, int NT, bool LIST, bool ACC>
__global__ void __launch_bounds__(kThreads, Shape<NT>::kCtas) attn_kernel(AttnArgs a) {
    constexpr int R = 8 * NT, C = Shape<NT>::C, LANES = 32 / C;
    constexpr bool SQ = Shape<NT>::kSharedQ;
    __shared__ Shared<D, NT> sh;
    const kvq_block8& c = a.c;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    Run<kWarps> run = {0, 1, (int)blockIdx.x, 0, true, 0, 1};   // direct: the CTA's own unit, whole
    if (!a.direct)
        run = find_run<kThreads, kWarps>(a.works, [&](int i) { return work_of<NT, LIST>(a, i).tiles; }, sh.run);
    grid_launch_dependents();
    for (int w = run.work, from = run.from, before = run.before; from < run.to; ++w) {
        const Work k = work_of<NT, LIST>(a, w);
        int s0 = 0, s1 = k.tiles;
        if (!a.direct) {
            if (k.tiles == 0) continue;
            s0 = max(from - before - run.start, 0);
            s1 = min(k.tiles, run.to - before - run.start);
            if (s1 <= 0) break;                 // the run ends ahead of the unit's tiles
            if (s0 == 0 && threadIdx.x == 0)
                a.span[w] = make_int2(blockIdx.x, (before + run.start + k.tiles - 1) / run.per);
        }
        // ---- requests, in the order of their latencies: the table, the queries, the first tile
        KeyRegs<D> kr[C];
        ValueRegs<D> vr[C];
        Cells cells = find_cells<C, LIST>(a, k, w, s0 + warp, s1, lane);
        // a column block's query row g: all column blocks where fragments stay in registers, else block
        // `warp` of this warp, for all warps
        constexpr int QN = SQ ? 1 : NT;
        uint4 raw[QN][D / 64][2];
#pragma unroll
        for (int n = 0; n < QN; ++n) {
            const int2 th = row_of<NT, LIST>(a, k, w, min(8 * (SQ ? warp : n) + g, k.rows - 1));
            const T* q = (const T*)a.q + k.b * a.qs[0] + (int64_t)((k.u % c.Hkv) * a.g + th.y) * a.qs[1] + th.x * a.qs[2] +
                         t * 16;
#pragma unroll
            for (int j = 0; j < D / 64; ++j)
#pragma unroll
                for (int e = 0; e < 2; ++e) raw[n][j][e] = *reinterpret_cast<const uint4*>(q + j * 64 + e * 8);
        }
        uint32_t cell[C];
#pragma unroll
        for (int j = 0; j < C; ++j) {
            cell[j] = __shfl_sync(0xffffffffu, cells.cell, j);
            load_keys<D>(kr[j], c.k_codes, cell[j], g, t);
        }
#pragma unroll
        for (int j = 0; j < C; ++j) load_values<D>(vr[j], c.v_codes, cell[j], g, t);
        // ---- the queries, channels in the keys' order, as fp16
        uint32_t qf[QN][D / 16][2];
        float undo[QN];                 // what undoes a row's factor
#pragma unroll
        for (int n = 0; n < QN; ++n) {
            float x[D / 4];
#pragma unroll
            for (int j = 0; j < D / 64; ++j)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const T* y = reinterpret_cast<const T*>(&raw[n][j][e]);
#pragma unroll
                    for (int z = 0; z < 8; ++z) x[j * 16 + e * 8 + z] = Elem<T>::to_f(y[z]);
                }
            undo[n] = 1.0f;
            if constexpr (std::is_same<T, __nv_bfloat16>::value) {
                // bf16 reaches further than fp16: a power of two brings the row's largest to 2^14 .. 2^15
                uint32_t mx = 0;
#pragma unroll
                for (int z = 0; z < D / 4; ++z) mx = max(mx, __float_as_uint(x[z]) & 0x7fffffffu);
                mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                const int e = min(max((int)(mx >> 23), 28), 254);
                const float f = mx < 0x7f800000u ? __uint_as_float((uint32_t)(127 + 14 + 127 - e) << 23) : 1.0f;
                undo[n] = mx < 0x7f800000u ? __uint_as_float((uint32_t)(e - 14) << 23) : 1.0f;
#pragma unroll
                for (int z = 0; z < D / 4; ++z) x[z] *= f;
            }
#pragma unroll
            for (int s = 0; s < D / 16; ++s) {
                __half2 h0 = __floats2half2_rn(x[4 * s], x[4 * s + 1]), h1 = __floats2half2_rn(x[4 * s + 2], x[4 * s + 3]);
                qf[n][s][0] = *reinterpret_cast<uint32_t*>(&h0);
                qf[n][s][1] = *reinterpret_cast<uint32_t*>(&h1);
            }
        }
        if constexpr (SQ) {             // (the CTA's last unit's queries were read before its merge's barrier)
            if (warp < NT) {
#pragma unroll
                for (int s = 0; s < D / 16; ++s)
                    *reinterpret_cast<uint2*>(&sh.q[8 * warp + g][(s / 4) * 64 + t * 16 + (s % 4) * 4]) =
                        make_uint2(qf[0][s][0], qf[0][s][1]);
                if (t == 0) sh.undo[8 * warp + g] = undo[0];
            }
            __syncthreads();
        }
        float qi[NT][2];                // undo for this lane's columns 2t, 2t + 1
        int lim[NT][2], least = k.top;  // tokens that the columns' queries see
        {
            const int m = a.n_new ? min(max(a.n_new[k.b], 0), a.n_q) : a.n_q;
            const int count = min(c.count[k.u], c.max_blocks * c.block);
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int col = 8 * n + 2 * t + e;
                    if constexpr (SQ) qi[n][e] = sh.undo[col];
                    else qi[n][e] = __shfl_sync(0xffffffffu, undo[n], (2 * t + e) * 4);
                    lim[n][e] = k.top;  // padding rows: as the last query; nobody reads them
                    const int tq = row_of<NT, LIST>(a, k, w, col).x;
                    if (col < k.rows && tq < m) lim[n][e] = query_limit(count, m, tq);
                    least = min(least, lim[n][e]);
                }
        }
        least = __reduce_min_sync(0xffffffffu, least);
        float o[NT][D / 16][4], M[NT][2], l[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int i = 0; i < D / 16; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[n][i][e] = 0.0f;
            M[n][0] = M[n][1] = kNone;
            l[n][0] = l[n][1] = 0.0f;
        }
        // ---- the warp's tiles
        int at = 0;                     // the tile's place among those of `cells`
        bool wide = false;              // value scales more than kFar apart so far (for the whole warp)
        if constexpr (kWide<T>) wide = scales_apart(sh.lv[warp], cells.lv, make_float2(-INFINITY, INFINITY));
        for (int tile = s0 + warp; tile < s1; tile += kWarps) {
            float ks[C], lv[C], rv[C];
            int slot[C];
#pragma unroll
            for (int j = 0; j < C; ++j) {
                ks[j] = __shfl_sync(0xffffffffu, cells.ks, C * at + j);
                lv[j] = __shfl_sync(0xffffffffu, cells.lv, C * at + j);
                rv[j] = __shfl_sync(0xffffffffu, cells.rv, C * at + j);
                slot[j] = __shfl_sync(0xffffffffu, cells.slot, C * at + j);
                if (cell[j] == 0xffffffffu) slot[j] = 0x40000000;       // nothing there: behind every limit
            }
            // where the next tile lies
            if (++at == LANES) {
                cells = find_cells<C, LIST>(a, k, w, tile + kWarps, s1, lane);
                at = 0;
                if constexpr (kWide<T>) wide = scales_apart(sh.lv[warp], cells.lv, sh.lv[warp]);
            }
            ask_l2<D, C>(c, cells, at, lane);
#pragma unroll
            for (int j = 0; j < C; ++j) cell[j] = __shfl_sync(0xffffffffu, cells.cell, C * at + j);
            if (tile + kWarps >= s1)
#pragma unroll
                for (int j = 0; j < C; ++j) cell[j] = 0xffffffffu;
            // ---- logits: tokens are rows, queries columns
            float s[C][NT][4];
#pragma unroll
            for (int j = 0; j < C; ++j) {
#pragma unroll
                for (int n = 0; n < NT; ++n) s[j][n][0] = s[j][n][1] = s[j][n][2] = s[j][n][3] = 0.0f;
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                    const uint4 lo = kr[j].r[0][i / 4], hi = kr[j].r[1][i / 4];
                    const uint32_t wl = i % 4 == 0 ? lo.x : i % 4 == 1 ? lo.y : i % 4 == 2 ? lo.z : lo.w;
                    const uint32_t wh = i % 4 == 0 ? hi.x : i % 4 == 1 ? hi.y : i % 4 == 2 ? hi.z : hi.w;
                    uint32_t a0, a1, a2, a3;
                    to_f16<CODE>(wl, a0, a2);
                    to_f16<CODE>(wh, a1, a3);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        uint2 q;
                        if constexpr (SQ)
                            q = *reinterpret_cast<const uint2*>(&sh.q[8 * n + g][(i / 4) * 64 + t * 16 + (i % 4) * 4]);
                        else
                            q = make_uint2(qf[n][i][0], qf[n][i][1]);
                        mma(s[j][n], a0, a1, a2, a3, q.x, q.y);
                    }
                }
                load_keys<D>(kr[j], c.k_codes, cell[j], g, t);
            }
            // ---- weights
#pragma unroll
            for (int j = 0; j < C; ++j) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int x = 0; x < 4; ++x) s[j][n][x] = fmaf(s[j][n][x], ks[j] * qi[n][x & 1], lv[j]);
                if (slot[j] + 16 > least) {
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int x = 0; x < 4; ++x)
                            if (slot[j] + g + (x >> 1) * 8 >= lim[n][x & 1]) s[j][n][x] = -INFINITY;
                }
            }
            // log2 of a cell's weights, whatever M is now or becomes; sum0 and sum1 count `unit` each
            [[maybe_unused]] auto put_mass = [&](int j, int n, float sum0, float sum1, float unit) {
#pragma unroll
                for (int x = 4; x < 32; x <<= 1) {
                    sum0 += __shfl_xor_sync(0xffffffffu, sum0, x);
                    sum1 += __shfl_xor_sync(0xffffffffu, sum1, x);
                }
                if (g == 0 && slot[j] < 0x40000000)
                    *reinterpret_cast<float2*>(a.mass + ((size_t)w * a.cells + C * tile + j) * R + 8 * n + 2 * t) =
                        make_float2(__log2f(sum0 * unit) + M[n][0], __log2f(sum1 * unit) + M[n][1]);
            };
            [[maybe_unused]] bool counted[C];
#pragma unroll
            for (int j = 0; j < C; ++j) counted[j] = false;
            float over = wide ? INFINITY : -INFINITY;
            auto column_max = [&](int n, int e) {
                float mx = fmaxf(s[0][n][e], s[0][n][2 + e]);
                if constexpr (C == 2) mx = fmaxf(mx, fmaxf(s[C - 1][n][e], s[C - 1][n][2 + e]));
                return mx;
            };
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) over = fmaxf(over, column_max(n, e) - M[n][e]);
            if (__any_sync(0xffffffffu, over > kLift)) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float mx = column_max(n, e);
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
                        const float now = fmaxf(M[n][e], mx - kShift), fac = ex2_approx(M[n][e] - now);
                        l[n][e] = lowered<kWide<T>>(l[n][e], M[n][e] - now);
                        M[n][e] = now;
#pragma unroll
                        for (int i = 0; i < D / 16; ++i) {
                            o[n][i][e] *= fac;
                            o[n][i][2 + e] *= fac;
                        }
                    }
                if constexpr (kWide<T>) {
#pragma unroll
                    for (int j = 0; j < C; ++j)
                        if (sh.lv[warp].x - lv[j] > kFar) {             // (the whole warp)
                            const float up = kBias - lv[j];
#pragma unroll
                            for (int n = 0; n < NT; ++n) {
                                float sum[2];
#pragma unroll
                                for (int e = 0; e < 2; ++e) {
                                    sum[e] = ex2_approx(s[j][n][e] - M[n][e] + up) + ex2_approx(s[j][n][2 + e] - M[n][e] + up);
                                    l[n][e] = fmaf(sum[e], kBiasInv, l[n][e]);
                                }
                                if constexpr (ACC) put_mass(j, n, sum[0], sum[1], kBiasInv);
                            }
                            rv[j] = 0.0f;
                            counted[j] = true;
                        }
                }
            }
            uint32_t bh[C][NT][2], bl[C][NT][2];
#pragma unroll
            for (int j = 0; j < C; ++j) {
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float p[4];
#pragma unroll
                    for (int x = 0; x < 4; ++x) p[x] = ex2_approx(s[j][n][x] - M[n][x & 1]);
                    const float sum0 = p[0] + p[2], sum1 = p[1] + p[3];
                    l[n][0] = fmaf(sum0, rv[j], l[n][0]);
                    l[n][1] = fmaf(sum1, rv[j], l[n][1]);
                    if constexpr (ACC)
                        if (!counted[j]) put_mass(j, n, sum0, sum1, rv[j]);
                    uint32_t h0, l0, h1, l1;
                    split2(p[0], p[1], h0, l0);
                    split2(p[2], p[3], h1, l1);
                    bh[j][n][0] = transpose8x8(h0);
                    bh[j][n][1] = transpose8x8(h1);
                    bl[j][n][0] = transpose8x8(l0);
                    bl[j][n][1] = transpose8x8(l1);
                }
                // ---- outputs: channels are rows, queries columns
                if (slot[j] + 16 > k.top) {             // rows behind the last token may hold anything: 0 x NaN
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (slot[j] + 2 * t + (i & 1) + (i >> 1) * 8 >= k.top)
#pragma unroll
                            for (int x = 0; x < D / 32; ++x) vr[j].r[i][x] = 0;
                }
#pragma unroll
                for (int i = 0; i < D / 32; ++i) {
                    const uint32_t p0 = __byte_perm(vr[j].r[0][i], vr[j].r[1][i], 0x5140);
                    const uint32_t p1 = __byte_perm(vr[j].r[0][i], vr[j].r[1][i], 0x7362);
                    const uint32_t p2 = __byte_perm(vr[j].r[2][i], vr[j].r[3][i], 0x5140);
                    const uint32_t p3 = __byte_perm(vr[j].r[2][i], vr[j].r[3][i], 0x7362);
                    uint32_t a0, a1, a2, a3;
                    to_f16<CODE>(p0, a0, a1);
                    to_f16<CODE>(p2, a2, a3);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        mma(o[n][2 * i], a0, a1, a2, a3, bh[j][n][0], bh[j][n][1]);
                        mma(o[n][2 * i], a0, a1, a2, a3, bl[j][n][0], bl[j][n][1]);
                    }
                    to_f16<CODE>(p1, a0, a1);
                    to_f16<CODE>(p3, a2, a3);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        mma(o[n][2 * i + 1], a0, a1, a2, a3, bh[j][n][0], bh[j][n][1]);
                        mma(o[n][2 * i + 1], a0, a1, a2, a3, bl[j][n][0], bl[j][n][1]);
                    }
                }
                load_values<D>(vr[j], c.v_codes, cell[j], g, t);
            }
        }
        // ---- the CTA's partial state of this work unit
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float x = l[n][e];
                x += __shfl_xor_sync(0xffffffffu, x, 4);
                x += __shfl_xor_sync(0xffffffffu, x, 8);
                x += __shfl_xor_sync(0xffffffffu, x, 16);
                if (g == 0) *reinterpret_cast<float2*>(sh.ml[warp][8 * n + 2 * t + e]) = make_float2(M[n][e], x);
            }
        const size_t slot = (size_t)blockIdx.x + w;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float* dst = &sh.o[warp][2 * t + e][g * (D / 8)];
#pragma unroll
                for (int i = 0; i < D / 16; ++i)
                    *reinterpret_cast<float2*>(dst + 2 * i) = make_float2(o[n][i][e], o[n][i][2 + e]);
            }
            __syncthreads();
            for (int x = threadIdx.x; x < 8 * (D / 4); x += kThreads) {
                const int col = x / (D / 4), row = 8 * n + col, d = x % (D / 4) * 4;
                float top = -INFINITY, sum = 0.0f;
#pragma unroll
                for (int i = 0; i < kWarps; ++i) top = fmaxf(top, sh.ml[i][row][0]);
                const float ref = top == -INFINITY ? 0.0f : top;
                float4 y = make_float4(0, 0, 0, 0);
#pragma unroll
                for (int i = 0; i < kWarps; ++i) {
                    const float fac = ex2_approx(sh.ml[i][row][0] - ref);
                    const float4 v = *reinterpret_cast<const float4*>(&sh.o[i][col][d]);
                    y.x = fmaf(v.x, fac, y.x);
                    y.y = fmaf(v.y, fac, y.y);
                    y.z = fmaf(v.z, fac, y.z);
                    y.w = fmaf(v.w, fac, y.w);
                    if constexpr (kWide<T>) sum += lowered<true>(sh.ml[i][row][1], sh.ml[i][row][0] - ref);
                    else sum = fmaf(sh.ml[i][row][1], fac, sum);
                }
                if (a.direct) {
                    if (row < k.rows) write_row<T, NT, LIST>(a, k, w, row, d, y, top, sum);
                } else {
                    *reinterpret_cast<float4*>(a.part + (slot * R + row) * D + d) = y;
                    if (d == 0) *reinterpret_cast<float2*>(a.ml + (slot * R + row) * 2) = make_float2(top, sum);
                }
            }
            __syncthreads();
        }
        if (a.direct) break;
        before += run.places(k.tiles);
        from = before;
    }
}

// ------------------------------------------------------------------ the second kernel

// A cell's weight (log2) as a part of its row's sum (log2; infinity for rows that count nothing, whose
// cells may hold anything).
__device__ __forceinline__ float part_of(float mass, float lse2) {
    return lse2 == INFINITY ? 0.0f : ex2_approx(mass - lse2);
}

constexpr int kJoinThreads = 256, kJoinWarps = kJoinThreads / 32;

// A row's partials j = first, first + step, ... <= last joined by one warp: the reference M and the
// sum l that belong to it, and D / 32 output channels a lane (o, if OUT).  Four partials are in flight
// at a time.
template <int D, int R, bool OUT, bool WIDE>
__device__ __forceinline__ float2 join_row(const AttnArgs& a, int w, int row, int first, int last, int step, int lane,
                                           float (&o)[D / 32]) {
    constexpr int V = D / 32;
    float M = -INFINITY, l = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) o[v] = 0.0f;
    for (int j = first; j <= last; j += 4 * step) {
        float2 ml[4];
        float x[4][V];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            ml[i] = make_float2(-INFINITY, 0.0f);
            const size_t at = ((size_t)(j + i * step) + w) * R + row;
            if (j + i * step <= last) {
                ml[i] = *reinterpret_cast<const float2*>(a.ml + at * 2);
                if (OUT) {
                    const float* p = a.part + at * D + lane * V;
                    if constexpr (V == 4) {
                        const float4 y = *reinterpret_cast<const float4*>(p);
                        x[i][0] = y.x; x[i][1] = y.y; x[i][2] = y.z; x[i][3] = y.w;
                    } else {
                        const float2 y = *reinterpret_cast<const float2*>(p);
                        x[i][0] = y.x; x[i][1] = y.y;
                    }
                }
            } else if (OUT) {
#pragma unroll
                for (int v = 0; v < V; ++v) x[i][v] = 0.0f;
            }
        }
        const float top = fmaxf(fmaxf(fmaxf(ml[0].x, ml[1].x), fmaxf(ml[2].x, ml[3].x)), M);
        const float ref = top == -INFINITY ? 0.0f : top, old = ex2_approx(M - ref);
        l = WIDE ? lowered<WIDE>(l, M - ref) : l * old;
        M = top;
#pragma unroll
        for (int v = 0; v < V; ++v) o[v] *= old;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float f = ex2_approx(ml[i].x - ref);
            l = WIDE ? l + lowered<WIDE>(ml[i].y, ml[i].x - ref) : fmaf(ml[i].y, f, l);
            if (OUT)
#pragma unroll
                for (int v = 0; v < V; ++v) o[v] = fmaf(x[i][v], f, o[v]);
        }
    }
    return make_float2(M, l);
}

// A few partials a row: bound by the latency of three dependent loads (span, partials, and the counters
// before them), so all of a row's are asked for at once, and what does not come from the first kernel is
// read before the wait (2 to 3 us less than one block per row that took the partials in turn).
// Blocks [0, works * R * SPLIT / kJoinWarps): SPLIT warps join one row of a work unit: o and lse.
// Blocks behind them (accumulate): the shares of kJoinThreads blocks of a unit, or of all listed blocks
// of a unit, one thread per block, summed over queries, heads and cells in a fixed order.
template <typename T, int D, int NT, bool LIST, bool ACC, int SPLIT>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(AttnArgs a, int row_blocks, int chunks) {
    constexpr int R = 8 * NT, V = D / 32;
    const kvq_block8& c = a.c;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if ((int)blockIdx.x < row_blocks) {
        __shared__ float2 sml[kJoinWarps];
        __shared__ float so[kJoinWarps][D];
        const int x = blockIdx.x * (kJoinWarps / SPLIT) + warp / SPLIT, w = x / R, i = x % R, part = warp % SPLIT;
        const Work k = work_of<NT, LIST>(a, w);
        const int m = new_rows(a.n_new, k.b, a.n_q, &g_status_block8_attn);
        const int2 th = row_of<NT, LIST>(a, k, w, min(i, k.rows - 1));
        const bool live = i < k.rows && k.tiles > 0 && th.x < m;
        grid_dependency_wait();
        float o[V], l = 0.0f, M = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) o[v] = 0.0f;
        if (live) {
            const int2 span = a.span[w];
            const float2 ml = join_row<D, R, true, kWide<T>>(a, w, i, span.x + part, span.y, SPLIT, lane, o);
            M = ml.x;
            l = ml.y;
        }
        if (SPLIT > 1) {
            if (lane == 0) sml[warp] = make_float2(M, l);
#pragma unroll
            for (int v = 0; v < V; ++v) so[warp][lane * V + v] = o[v];
            __syncthreads();
            if (part) return;
            float top = -INFINITY;
#pragma unroll
            for (int p = 0; p < SPLIT; ++p) top = fmaxf(top, sml[warp + p].x);
            const float ref = top == -INFINITY ? 0.0f : top;
            M = top;
            l = 0.0f;
#pragma unroll
            for (int v = 0; v < V; ++v) o[v] = 0.0f;
#pragma unroll
            for (int p = 0; p < SPLIT; ++p) {
                const float f = ex2_approx(sml[warp + p].x - ref);
                l = kWide<T> ? l + lowered<kWide<T>>(sml[warp + p].y, sml[warp + p].x - ref) : fmaf(sml[warp + p].y, f, l);
#pragma unroll
                for (int v = 0; v < V; ++v) o[v] = fmaf(so[warp + p][lane * V + v], f, o[v]);
            }
        }
        if (i >= k.rows) return;
        const bool sees = live && l != 0.0f;
        const float inv = sees ? 1.0f / l : 0.0f;
        const size_t orow = ((size_t)k.b * c.Hq + (size_t)(k.u % c.Hkv) * a.g + th.y) * a.n_q + th.x;
        T y[V];
#pragma unroll
        for (int v = 0; v < V; ++v) y[v] = Elem<T>::from_f(sees ? o[v] * inv : 0.0f);
        T* dst = (T*)a.o + orow * D + lane * V;
        if constexpr (V == 4) *reinterpret_cast<uint2*>(dst) = *reinterpret_cast<uint2*>(y);
        else *reinterpret_cast<uint32_t*>(dst) = *reinterpret_cast<uint32_t*>(y);
        if (lane == 0 && a.lse)
            a.lse[orow] = sees ? (M + log2f(l)) * kLn2 : -INFINITY;
        return;
    }
    if constexpr (ACC) {
        __shared__ float lse2[R];
        const int x = blockIdx.x - row_blocks, u = x / chunks, chunk = x % chunks;
        const int m = new_rows(a.n_new, u / c.Hkv, a.n_q, &g_status_block8_attn), per = c.block / 16;
        const int held = (min(c.count[u], c.max_blocks * c.block) + c.block - 1) / c.block;
        grid_dependency_wait();
        for (int t = 0; t < (LIST ? m : 1); ++t) {
            for (int rt = 0; rt < a.row_tiles; ++rt) {
                const int w = (LIST ? u * a.n_q + t : u) * a.row_tiles + rt;
                const Work k = work_of<NT, LIST>(a, w);
                const int n = LIST ? k.list_n : (k.top + c.block - 1) / c.block;
                if (n <= chunk * kJoinThreads) continue;
                const int2 span = a.span[w];
                __syncthreads();
                for (int i = warp; i < R; i += kJoinWarps) {
                    float none[V];
                    const float2 ml = join_row<D, R, false, kWide<T>>(a, w, i, span.x + lane, span.y, 32, lane, none);
                    float top = ml.x;
#pragma unroll
                    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                    const float ref = top == -INFINITY ? 0.0f : top;
                    float l = lowered<kWide<T>>(ml.y, ml.x - ref);
#pragma unroll
                    for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
                    const bool sees = i < k.rows && row_of<NT, LIST>(a, k, w, i).x < m && l != 0.0f;
                    if (lane == 0) lse2[i] = sees ? ref + log2f(l) : INFINITY;
                }
                __syncthreads();
                for (int j = chunk * kJoinThreads + threadIdx.x; j < (LIST ? n : min(n, (chunk + 1) * kJoinThreads));
                     j += kJoinThreads) {
                    const int blk = LIST ? a.blocks[(size_t)(u * a.n_q + t) * a.n_sel + j] : j;
                    if ((unsigned)blk >= (unsigned)held) continue;
                    const int phys = c.table[(size_t)u * c.max_blocks + blk];
                    if ((unsigned)phys >= (unsigned)c.n_blocks) continue;
                    const int cells = min(per, (k.top - blk * c.block + 15) / 16);
                    float share = 0.0f;
                    for (int y = 0; y < cells; ++y) {
                        const float* mass = a.mass + ((size_t)w * a.cells + (size_t)j * per + y) * R;
#pragma unroll
                        for (int i = 0; i < R; i += 4) {
                            const float4 z = *reinterpret_cast<const float4*>(mass + i);
                            share += part_of(z.x, lse2[i]) + part_of(z.y, lse2[i + 1]) +
                                     (part_of(z.z, lse2[i + 2]) + part_of(z.w, lse2[i + 3]));
                        }
                    }
                    if (LIST) atomicAdd(&c.acc[phys], share);       // a block listed twice adds twice
                    else c.acc[phys] += share;
                }
            }
        }
    }
}

// ------------------------------------------------------------------ host

struct Layout {
    int nt, row_tiles, works, cells;
    size_t part, ml, span, mass, total;
};

size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

Layout layout_of(const kvq_block8& c, int n_q, int n_sel, int accumulate) {
    Layout y;
    const int units = c.B * c.Hkv, g = c.Hq / c.Hkv, rows = n_sel ? g : g * n_q;
    y.nt = rows <= 8 ? 1 : rows <= 16 ? 2 : 4;
    y.row_tiles = (rows + 8 * y.nt - 1) / (8 * y.nt);
    y.works = units * (n_sel ? n_q : 1) * y.row_tiles;
    y.cells = (n_sel ? std::min(n_sel, c.max_blocks) : c.max_blocks) * (c.block / 16);
    const size_t slots = (size_t)kMaxCtas + y.works, r = 8 * y.nt;
    y.part = 0;
    y.ml = y.part + up256(slots * r * c.D * sizeof(float));
    y.span = y.ml + up256(slots * r * 2 * sizeof(float));
    y.mass = y.span + up256((size_t)y.works * sizeof(int2));
    y.total = y.mass + (accumulate ? up256((size_t)y.works * y.cells * r * sizeof(float)) : 0);
    return y;
}

template <typename T, int D, int NT, bool LIST, bool ACC, int SPLIT>
cudaError_t launch_join(const AttnArgs& a, cudaStream_t s) {
    const int units = a.c.B * a.c.Hkv, row_blocks = a.works * (NT * SPLIT);    // 8 rows each column block, 8 warps
    const int chunks = LIST ? 1 : (a.c.max_blocks + kJoinThreads - 1) / kJoinThreads;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3((unsigned)(row_blocks + (ACC ? units * chunks : 0)));
    cfg.blockDim = dim3(kJoinThreads);
    cfg.stream = s;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, join_kernel<T, D, NT, LIST, ACC, SPLIT>, a, row_blocks, chunks);
}

template <typename T, int D, int CODE, int NT, bool LIST, bool ACC>
cudaError_t launch(AttnArgs a, cudaStream_t s) {
    static std::atomic<int> known[64];
    auto kernel = attn_kernel<T, D, CODE, NT, LIST, ACC>;
    int ctas = 0;
    cudaError_t e = resident_ctas(kernel, kThreads, 0, known, &ctas);
    if (e != cudaSuccess) return e;
    if (!ACC && a.cells <= (a.works >= ctas / Shape<NT>::kCtas ? 2 : 1) * kDirectCells) {
        a.direct = 1;
        kernel<<<(unsigned)a.works, kThreads, 0, s>>>(a);
        return cudaGetLastError();
    }
    // no more CTAs than runs of kWarps tiles in full caches
    constexpr int kRun = kWarps * Shape<NT>::C;
    const int grid = (int)std::min<long long>(std::min(ctas, kMaxCtas), (long long)a.works * ((a.cells + kRun - 1) / kRun));
    kernel<<<grid, kThreads, 0, s>>>(a);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    // four warps a row where a unit has many partials, one where it has few
    return grid >= 4 * a.works ? launch_join<T, D, NT, LIST, ACC, 4>(a, s) : launch_join<T, D, NT, LIST, ACC, 1>(a, s);
}

}  // namespace

size_t block8_attn_bytes(const kvq_block8& c, int n_q, int n_sel, int accumulate) {
    return layout_of(c, n_q, n_sel, accumulate).total;
}

cudaError_t launch_block8_attn(const void* q, const int64_t* qs, int n_q, const int32_t* n_new, const kvq_block8& c,
                               float sm_scale, const int32_t* blocks, const int32_t* list_len, int n_sel,
                               int accumulate, void* o, float* lse, void* ws, cudaStream_t s) {
    const Layout y = layout_of(c, n_q, n_sel, accumulate);
    char* base = (char*)ws;
    AttnArgs a{c, q, {qs[0], qs[1], qs[2]}, n_q, n_new, sm_scale, blocks, list_len, n_sel, o, lse,
               std::min(n_sel, c.max_blocks), c.Hq / c.Hkv, y.row_tiles, y.works, y.cells, 0, (float*)(base + y.part),
               (float*)(base + y.ml), (float*)(base + y.mass), (int2*)(base + y.span)};
    // one switch after the other turns the runtime choices into template arguments
    auto on = [](bool x, auto f) { return x ? f(std::true_type{}) : f(std::false_type{}); };
    return on(c.dtype == KVQ_BF16, [&](auto bf) {
        using T = std::conditional_t<decltype(bf)::value, __nv_bfloat16, __half>;
        return on(c.D == 128, [&](auto wide) {
            constexpr int D = decltype(wide)::value ? 128 : 64;
            return on(c.code == KVQ_CODE_INT8, [&](auto i8) {
                constexpr int CODE = decltype(i8)::value ? KVQ_CODE_INT8 : KVQ_CODE_E4M3;
                return on(blocks != nullptr, [&](auto list) {
                    return on(accumulate != 0, [&](auto acc) {
                        constexpr bool LIST = decltype(list)::value, ACC = decltype(acc)::value;
                        return y.nt == 1   ? launch<T, D, CODE, 1, LIST, ACC>(a, s)
                               : y.nt == 2 ? launch<T, D, CODE, 2, LIST, ACC>(a, s)
                                           : launch<T, D, CODE, 4, LIST, ACC>(a, s);
                    });
                });
            });
        });
    });
}

}  // namespace kvq
