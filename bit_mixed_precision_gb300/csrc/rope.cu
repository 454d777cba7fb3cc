// qk_norm_rope and qk_norm_rope_bwd: a layer's projection [B, T, heads, D] to what attention and the caches take
// ([B, heads, T, D], queries and keys normed per head and rotated), and the gradient of that.
//
// Mathematics (x a head's row, w the norm's weight, f_i the frequency of pair i in radians per position):
//   r = 1 / sqrt(mean(x^2) + eps);  y = x r w;  pair (a, b) of y with phi = pos f: (a cos - b sin, b cos + a sin)
//   backward: dy = the pairs of d turned by -phi;  dw = sum over rows of dy x r;  g = dy w;
//             dx = r (g - (x r) mean(g (x r)))
// Angles: f is kept as a 64-bit fraction of a turn, so pos * f modulo a turn is one wrapping integer product, exact for
// every int32 position but for the fraction's own error times the position (2^-65 of a turn for a fraction rounded once;
// one formed in float64 has 2^-52 of f / 2 pi, so that f = 1 at position 2^20 loses at most 2^-34 of a turn); what is left,
// in [-1/2, 1/2) turns, becomes float32 and cosine and sine.
// Bound: HBM, each row is read and written once.  D / 16 lanes share a row, each with the two 16-byte pieces that hold
// the two sides of its eight pairs, so that the rotation needs no exchange and the norm's sum two or three shuffles; a
// warp holds 64 / (D / 8) rows of one token at a time, and the token's angles are computed once for all heads, a share
// by each lane.  The rows come through a ring in shared memory that every lane fills for itself with asynchronous
// copies: 5 KB a warp in flight (backward 8) without registers to hold it.
// All arithmetic is float32, two numbers to an instruction; an output is rounded once.
// Measured: 4 x 16384 tokens of 32/8 heads of 128 in bf16 236 us, 6.8 TB/s (loads to registers two groups ahead: 318);
// their gradient, 16 x 4096 tokens, 375 us, 6.1 TB/s (eight sines a lane and weights in registers: 523).  One token
// 2.8 us.
#include <algorithm>
#include <atomic>

#include "grad_device.cuh"
#include "kvq_common.cuh"
#include "kvq_internal.h"

namespace kvq {

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kStages = 5;          // forward: 1 KB each
constexpr int kBwdStages = 4;       // backward: 2 KB each
constexpr int kBwdCtas = 2;         // of an SM

template <typename T> struct RopeArgs {
    const T *q, *k, *v;             // raw rows [B, T, heads, D] (strides in elements, b, t, head)
    int64_t qs[3], ks[3], vs[3];
    T *qo, *ko, *vo;                // [B, heads, T, D]
    const int32_t* pos;             // [n_axes, B, T]
    const void *qw, *kw;            // [D] or NULL: no norm
    int w_f32;
    float eps;
    int B, T_len, Hq, Hkv;
    int rot, interleaved;
    unsigned long long axis[2];     // two bits per pair
    unsigned long long turn[64];
};

template <typename T> struct RopeBwdArgs {
    RopeArgs<T> f;                  // qo, ko, vo: the gradients that come in
    T *gq, *gk, *gv;                // [B, T, heads, D]
    int64_t gqs[3], gks[3], gvs[3];
    float* part;                    // [CTA][D] sums for the weights' gradients
};

// The 16 values of a lane: pieces c0 and c1 (eight channels each) of its row.
template <int D> struct Place {
    static constexpr int kLanes = D / 16;       // lanes of a row
    static constexpr int kRows = 32 / kLanes;   // rows of a warp
    int c0, c1, pair;                           // pieces; first pair (behind the last one where the lane has none)
    __device__ __forceinline__ Place(int lane, int rot, int interleaved) {
        const int l = lane % kLanes, n = rot / 16;
        pair = 8 * l;
        if (interleaved || l >= n) {
            c0 = 2 * l;
            c1 = c0 + 1;
        } else {
            c0 = l;
            c1 = l + n;
        }
    }
};

using F2 = unsigned long long;      // two float32, for packed arithmetic

// The lane's 16 channels as the sides a and b of its eight pairs, two pairs to an F2: from the 16-byte pieces c0 and c1,
// which are the sides themselves, or (IL, interleaved) hold pairs of neighbours.
struct Sides {
    F2 a[4], b[4];
};

template <typename T> __device__ __forceinline__ F2 widen(uint32_t w) {
    const T* e = reinterpret_cast<const T*>(&w);
    return f2_pack(Elem<T>::to_f(e[0]), Elem<T>::to_f(e[1]));
}

template <typename T> __device__ __forceinline__ uint32_t narrow(F2 x) {
    float lo, hi;
    f2_unpack(x, lo, hi);
    uint32_t w;
    T* e = reinterpret_cast<T*>(&w);
    e[0] = Elem<T>::from_f(lo), e[1] = Elem<T>::from_f(hi);
    return w;
}

// (x0, x1), (y0, y1) -> (x0, y0), (x1, y1)
__device__ __forceinline__ void unzip(F2& x, F2& y) {
    float x0, x1, y0, y1;
    f2_unpack(x, x0, x1);
    f2_unpack(y, y0, y1);
    x = f2_pack(x0, y0);
    y = f2_pack(x1, y1);
}

template <typename T, bool IL> __device__ __forceinline__ Sides sides(const uint4& c0, const uint4& c1) {
    Sides s = {{widen<T>(c0.x), widen<T>(c0.y), widen<T>(c0.z), widen<T>(c0.w)},
               {widen<T>(c1.x), widen<T>(c1.y), widen<T>(c1.z), widen<T>(c1.w)}};
    if (IL) {               // words in order hold pairs 0 .. 7
        Sides t;
        const F2 w[8] = {s.a[0], s.a[1], s.a[2], s.a[3], s.b[0], s.b[1], s.b[2], s.b[3]};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            t.a[i] = w[2 * i], t.b[i] = w[2 * i + 1];
            unzip(t.a[i], t.b[i]);
        }
        return t;
    }
    return s;
}

template <typename T, bool IL> __device__ __forceinline__ void pieces(Sides s, uint4& c0, uint4& c1) {
    if (IL) {
#pragma unroll
        for (int i = 0; i < 4; ++i) unzip(s.a[i], s.b[i]);
        c0 = make_uint4(narrow<T>(s.a[0]), narrow<T>(s.b[0]), narrow<T>(s.a[1]), narrow<T>(s.b[1]));
        c1 = make_uint4(narrow<T>(s.a[2]), narrow<T>(s.b[2]), narrow<T>(s.a[3]), narrow<T>(s.b[3]));
    } else {
        c0 = make_uint4(narrow<T>(s.a[0]), narrow<T>(s.a[1]), narrow<T>(s.a[2]), narrow<T>(s.a[3]));
        c1 = make_uint4(narrow<T>(s.b[0]), narrow<T>(s.b[1]), narrow<T>(s.b[2]), narrow<T>(s.b[3]));
    }
}

template <typename T, bool IL> __device__ __forceinline__ Sides load_weight(const void* w, int f32, int c0, int c1) {
    if (!f32) return sides<T, IL>(reinterpret_cast<const uint4*>(w)[c0], reinterpret_cast<const uint4*>(w)[c1]);
    Sides s;
    const F2* p = reinterpret_cast<const F2*>(w);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (IL) {
            s.a[i] = p[4 * (i < 2 ? c0 : c1) + 2 * (i & 1)], s.b[i] = p[4 * (i < 2 ? c0 : c1) + 2 * (i & 1) + 1];
            unzip(s.a[i], s.b[i]);
        } else {
            s.a[i] = p[4 * c0 + i], s.b[i] = p[4 * c1 + i];
        }
    }
    return s;
}

// Cosines and sines of a token: the warp's lanes take one pair each of 32 and hand them round through `table` (its own
// [2][64] floats), so that a lane computes two sines instead of the eight that it needs.
template <int D> struct Angles {
    static constexpr int kPer = D / 64;         // pairs that a lane computes
    unsigned long long turn[kPer];
    int64_t axis[kPer];                         // where the axis' positions start
    template <typename T> __device__ __forceinline__ Angles(const RopeArgs<T>& a, int lane, uint32_t n_tokens) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int p = lane + 32 * i;
            turn[i] = a.turn[p];                // 0 behind the last pair: cosine 1, sine 0
            axis[i] = ((a.axis[p >> 5] >> (2 * (p & 31))) & 3) * (int64_t)n_tokens;
        }
    }
    __device__ __forceinline__ void of(const int32_t* pos, bool any, uint32_t token, int lane, const int pair, float* table,
                                       F2* cs, F2* sn) const {
        __syncwarp();                           // the last token's have been read
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            float c = 1.0f, s = 0.0f;
            if (any) {
                const unsigned long long turns = (unsigned long long)(long long)pos[axis[i] + token] * turn[i];
                // the fraction of a turn in [-1/2, 1/2) as half turns in [-1, 1)
                sincospif((float)(int32_t)(turns >> 32) * 4.656612873077393e-10f, &s, &c);
            }
            table[lane + 32 * i] = c, table[64 + lane + 32 * i] = s;
        }
        __syncwarp();
        const ulonglong2* t = reinterpret_cast<const ulonglong2*>(table + pair);
        const ulonglong2 c0 = t[0], c1 = t[1], s0 = t[16], s1 = t[17];
        cs[0] = c0.x, cs[1] = c0.y, cs[2] = c1.x, cs[3] = c1.y;
        sn[0] = s0.x, sn[1] = s0.y, sn[2] = s1.x, sn[3] = s1.y;
    }
};

__device__ __forceinline__ F2 f2_neg(F2 x) { return x ^ 0x8000000080000000ull; }

// The pairs turned by phi, or with BACK by -phi.  A lane whose channels do not turn (all of its eight pairs or none do)
// leaves them alone: with cosine 1 and sine 0 an infinity would make its neighbour NaN.
template <bool BACK> __device__ __forceinline__ void turn_pairs(Sides& x, bool turns, const F2* cs, const F2* sn) {
    if (!turns) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const F2 a = x.a[i], b = x.b[i], s = BACK ? sn[i] : f2_neg(sn[i]), t = BACK ? f2_neg(sn[i]) : sn[i];
        x.a[i] = f2_fma(a, cs[i], f2_mul(b, s));
        x.b[i] = f2_fma(b, cs[i], f2_mul(a, t));
    }
}

__device__ __forceinline__ float f2_total(F2 x) {
    float lo, hi;
    f2_unpack(x, lo, hi);
    return lo + hi;
}

template <int LANES> __device__ __forceinline__ float row_sum(float x) {
#pragma unroll
    for (int m = LANES / 2; m > 0; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
    return x;
}

// The lane's part of a product of two rows.
__device__ __forceinline__ float dot(const Sides& x, const Sides& y) {
    F2 s = 0, t = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) s = f2_fma(x.a[i], y.a[i], s), t = f2_fma(x.b[i], y.b[i], t);
    return f2_total(f2_add(s, t));
}

template <int D> __device__ __forceinline__ float row_scale(const Sides& x, float eps) {
    return rsqrtf(row_sum<D / 16>(dot(x, x)) * (1.0f / D) + eps);
}

// A lane's own asynchronous copies: 16 bytes, zeros where there is nothing to read; each call of ring_commit() ends one
// stage's, ring_wait<N>() leaves the last N stages in flight.
__device__ __forceinline__ void ring_copy(uint4* to, const void* from, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(to)), "l"(from), "r"(there ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void ring_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void ring_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// ------------------------------------------------------------------ forward

// One warp per (token, share of its heads): the token's groups of kRows heads, first those of the queries, then the
// keys', then the values', are split into `parts` equal shares (one share for prompts; as many as there are groups for
// steps of few sequences, whose time is latency).
template <typename T, int D, bool IL>
__global__ void __launch_bounds__(kThreads, 3)
    rope_kernel(const __grid_constant__ RopeArgs<T> a, int parts, int per_part) {
    using P = Place<D>;
    __shared__ uint4 ring[kWarps][kStages][2][32];
    __shared__ __align__(16) float table[kWarps][128];
    const int lane = threadIdx.x & 31;
    uint4(*mine)[2][32] = ring[threadIdx.x >> 5];
    const uint32_t item = blockIdx.x * kWarps + (threadIdx.x >> 5), n_tokens = (uint32_t)a.B * (uint32_t)a.T_len;
    const uint32_t token = item / (uint32_t)parts;      // at most 2^30 tokens, in parts where they are few
    if (token >= n_tokens) return;
    const int b = (int)(token / (uint32_t)a.T_len), t = (int)(token % (uint32_t)a.T_len);
    const int gq = (a.Hq + P::kRows - 1) / P::kRows, gk = (a.Hkv + P::kRows - 1) / P::kRows;
    const int first = (int)(item % (uint32_t)parts) * per_part;
    const int last = min(first + per_part, gq + (a.v ? 2 : 1) * gk);
    const P at(lane, a.rot, IL);
    const int sub = lane / P::kLanes;
    const T* in_q = a.q + (int64_t)b * a.qs[0] + (int64_t)t * a.qs[1];
    const T* in_k = a.k + (int64_t)b * a.ks[0] + (int64_t)t * a.ks[1];
    const T* in_v = a.v + (int64_t)b * a.vs[0] + (int64_t)t * a.vs[1];
    auto request = [&](int p, int stage) {              // group p of the token into the ring
        if (p < last) {
            const bool q = p < gq, k = p < gq + gk;
            const int h = (p - (q ? 0 : k ? gq : gq + gk)) * P::kRows + sub;
            const bool there = h < (q ? a.Hq : a.Hkv);
            const T* row = (q ? in_q : k ? in_k : in_v) + (there ? h : 0) * (q ? a.qs[2] : k ? a.ks[2] : a.vs[2]);
            ring_copy(&mine[stage][0][lane], row + 8 * at.c0, there);
            ring_copy(&mine[stage][1][lane], row + 8 * at.c1, there);
        }
        ring_commit();
    };
#pragma unroll
    for (int i = 0; i < kStages; ++i) request(first + i, i);
    F2 cs[4], sn[4];
    Sides wt;
    if (first < gq + gk)
        Angles<D>(a, lane, n_tokens).of(a.pos, a.rot > 0, token, lane, at.pair, table[threadIdx.x >> 5], cs, sn);
    const void* w = nullptr;
    int stage = 0;
    for (int p = first; p < last; ++p) {
        const bool q = p < gq, k = p < gq + gk;
        if (p == first || p == gq) {                    // the weights of the queries, then of the keys
            w = q ? a.qw : k ? a.kw : nullptr;
            if (w) wt = load_weight<T, IL>(w, a.w_f32, at.c0, at.c1);
        }
        const int H = q ? a.Hq : a.Hkv, h = (p - (q ? 0 : k ? gq : gq + gk)) * P::kRows + sub;
        ring_wait<kStages - 1>();
        uint4 u0 = mine[stage][0][lane], u1 = mine[stage][1][lane];
        request(p + kStages, stage);
        stage = stage + 1 == kStages ? 0 : stage + 1;
        if (k) {
            Sides x = sides<T, IL>(u0, u1);
            if (w) {
                const float r = row_scale<D>(x, a.eps);
                const F2 r2 = f2_pack(r, r);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x.a[i] = f2_mul(f2_mul(x.a[i], r2), wt.a[i]);
                    x.b[i] = f2_mul(f2_mul(x.b[i], r2), wt.b[i]);
                }
            }
            turn_pairs<false>(x, at.pair < a.rot / 2, cs, sn);
            pieces<T, IL>(x, u0, u1);
        }
        if (h < H) {
            T* out = (q ? a.qo : k ? a.ko : a.vo) + (((int64_t)b * H + h) * a.T_len + t) * D;
            *reinterpret_cast<uint4*>(out + 8 * at.c0) = u0;
            *reinterpret_cast<uint4*>(out + 8 * at.c1) = u1;
        }
    }
}

// ------------------------------------------------------------------ backward

// CTAs below q_ctas have the queries, the others the keys and values, so that a lane keeps the weight and the weight's
// gradient of its 16 channels in registers; the warps of either stride over the tokens, their rings running on from one
// token to the next.  Sums go lane, warp, CTA, then over the CTAs in a second kernel, always in the same order.
template <typename T, int D, bool NORM, bool IL>
__global__ void __launch_bounds__(kThreads, kBwdCtas)
    rope_bwd_kernel(const __grid_constant__ RopeBwdArgs<T> p, int q_ctas) {
    using P = Place<D>;
    extern __shared__ uint4 ring_raw[];
    const RopeArgs<T>& a = p.f;
    grid_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint4* mine = ring_raw + warp * kBwdStages * 128 + lane;        // [stage][d, d, x, x][32]
    float* table = reinterpret_cast<float*>(ring_raw + kWarps * kBwdStages * 128) + warp * 128;
    const uint32_t T_len = (uint32_t)a.T_len, n_tokens = (uint32_t)a.B * T_len;     // at most 2^30
    const P at(lane, a.rot, IL);
    const int sub = lane / P::kLanes;
    const bool is_q = (int)blockIdx.x < q_ctas;
    const int H = is_q ? a.Hq : a.Hkv, groups = (H + P::kRows - 1) / P::kRows;
    const int all = groups * (is_q || !a.vo ? 1 : 2);               // groups of a token: keys, then values
    const void* w = is_q ? a.qw : a.kw;
    const bool norm = NORM && w;
    const T* raw = is_q ? a.q : a.k;
    const int64_t* st = is_q ? a.qs : a.ks;
    const uint32_t step = (is_q ? q_ctas : gridDim.x - q_ctas) * kWarps;
    const uint32_t start = (is_q ? blockIdx.x : blockIdx.x - q_ctas) * kWarps + warp;
    const Angles<D> angle(a, lane, n_tokens);
    // the weights of a lane's 16 channels, in shared memory to leave registers to the rest
    __shared__ __align__(16) F2 weight[4][D / 16][2];
    if (norm && warp == 0 && sub == 0) {
        const Sides x = load_weight<T, IL>(w, a.w_f32, at.c0, at.c1);
#pragma unroll
        for (int i = 0; i < 4; ++i) weight[i][lane][0] = x.a[i], weight[i][lane][1] = x.b[i];
    }
    if (NORM) __syncthreads();
    Sides dw = {{0, 0, 0, 0}, {0, 0, 0, 0}};
    // the next group to ask for: its number, its token, the lane's row in it (of d, of x)
    uint32_t ask = start;
    int ask_g = 0;
    const int64_t head = (int64_t)a.T_len * D, hop_d = P::kRows * head, hop_x = P::kRows * (norm ? st[2] : 0);
    const int c1 = 8 * (at.c1 - at.c0);                 // from a row's first piece to its second
    const T *ask_d = nullptr, *ask_x = nullptr;
    auto place = [&](const T* of) {                     // the first group of keys (queries) or of values
        const uint32_t b = ask / T_len, t = ask % T_len;
        ask_d = of + (int64_t)b * H * head + (int64_t)t * D + sub * head + 8 * at.c0;
        ask_x = norm ? raw + (int64_t)b * st[0] + (int64_t)t * st[1] + sub * st[2] + 8 * at.c0 : nullptr;
    };
    const T* first_of = is_q ? a.qo : a.ko;
    if (ask < n_tokens) place(first_of);
    auto request = [&](int stage) {
        if (ask < n_tokens) {
            const bool v = ask_g >= groups, there = (v ? ask_g - groups : ask_g) * P::kRows + sub < H;
            uint4* to = mine + stage * 128;
            const T* d = there ? ask_d : first_of;
            ring_copy(to, d, there);
            ring_copy(to + 32, d + (there ? c1 : 0), there);
            if (norm && !v) {
                const T* x = there ? ask_x : raw;
                ring_copy(to + 64, x, there);
                ring_copy(to + 96, x + (there ? c1 : 0), there);
            }
            ask_d += hop_d;
            ask_x += hop_x;
            if (++ask_g == all) {
                ask_g = 0, ask += step;
                if (ask < n_tokens) place(first_of);
            } else if (ask_g == groups) {
                place(a.vo);
            }
        }
        ring_commit();
    };
#pragma unroll
    for (int i = 0; i < kBwdStages; ++i) request(i);
    int stage = 0;
    for (uint32_t token = start; token < n_tokens; token += step) {
        const uint32_t b = token / T_len, t = token % T_len;
        const int64_t* gs = is_q ? p.gqs : p.gks;
        T* out = (is_q ? p.gq : p.gk) + (int64_t)b * gs[0] + (int64_t)t * gs[1] + sub * gs[2] + 8 * at.c0;
        int64_t hop = P::kRows * gs[2];
        F2 cs[4], sn[4];
        angle.of(a.pos, a.rot > 0, token, lane, at.pair, table, cs, sn);
#pragma unroll 1
        for (int g = 0; g < all; ++g) {
            const bool v = g >= groups;
            const int h = (v ? g - groups : g) * P::kRows + sub;
            if (g == groups) {                          // the values' turn
                out = p.gv + (int64_t)b * p.gvs[0] + (int64_t)t * p.gvs[1] + sub * p.gvs[2] + 8 * at.c0;
                hop = P::kRows * p.gvs[2];
            }
            ring_wait<kBwdStages - 1>();
            const uint4* from = mine + stage * 128;
            uint4 u0 = from[0], u1 = from[32];
            Sides d, x;
            if (!v) {
                d = sides<T, IL>(u0, u1);
                if (norm) x = sides<T, IL>(from[64], from[96]);
            }
            request(stage);
            stage = stage + 1 == kBwdStages ? 0 : stage + 1;
            if (!v) {
                turn_pairs<true>(d, at.pair < a.rot / 2, cs, sn);
                if (norm) {
                    // lanes without a head hold zeros, whose 1 / sqrt(0 + eps) may be infinite: 0 for them
                    const float s = row_scale<D>(x, a.eps), r = h < H ? s : 0.0f;
                    const F2 r2 = f2_pack(r, r);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        x.a[i] = f2_mul(x.a[i], r2), x.b[i] = f2_mul(x.b[i], r2);
                        dw.a[i] = f2_fma(d.a[i], x.a[i], dw.a[i]), dw.b[i] = f2_fma(d.b[i], x.b[i], dw.b[i]);
                        const ulonglong2 wt = *reinterpret_cast<const ulonglong2*>(weight[i][lane % P::kLanes]);
                        d.a[i] = f2_mul(d.a[i], wt.x), d.b[i] = f2_mul(d.b[i], wt.y);
                    }
                    const float m = row_sum<D / 16>(dot(d, x)) * (-1.0f / D);
                    const F2 m2 = f2_pack(m, m);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        d.a[i] = f2_mul(f2_fma(x.a[i], m2, d.a[i]), r2);
                        d.b[i] = f2_mul(f2_fma(x.b[i], m2, d.b[i]), r2);
                    }
                }
                pieces<T, IL>(d, u0, u1);
            }
            if (h < H) {
                *reinterpret_cast<uint4*>(out) = u0;
                *reinterpret_cast<uint4*>(out + c1) = u1;
            }
            out += hop;
        }
    }
    if (!NORM) return;
    // rows of the warp, then warps of the CTA
    __shared__ float sum[kWarps][D];
#pragma unroll
    for (int i = 0; i < 16; ++i) {                      // side b (i >= 8) or a of pair i mod 8
        float lo, hi;
        f2_unpack(i < 8 ? dw.a[i / 2] : dw.b[i / 2 - 4], lo, hi);
        float x = i & 1 ? hi : lo;
#pragma unroll
        for (int m = P::kLanes; m < 32; m <<= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
        const int j = i & 7;
        if (sub == 0) sum[warp][IL ? 8 * at.c0 + 2 * j + (i >> 3) : 8 * (i < 8 ? at.c0 : at.c1) + j] = x;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < D; i += kThreads) {
        float x = 0.0f;
#pragma unroll
        for (int k = 0; k < kWarps; ++k) x += sum[k][i];
        p.part[(int64_t)blockIdx.x * D + i] = x;
    }
}

// The CTAs' sums: one CTA per 32 of the 2 D channels (the queries' first), its warps striding over the parts.
__global__ void __launch_bounds__(1024)
    rope_weight_kernel(const float* __restrict__ part, int q_ctas, int ctas, int D, float* __restrict__ gqw,
                       float* __restrict__ gkw) {
    __shared__ float sum[32][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, i = blockIdx.x * 32 + lane;
    const bool k = i >= D;
    grid_dependency_wait();
    float x = 0.0f;
    for (int c = (k ? q_ctas : 0) + warp; c < (k ? ctas : q_ctas); c += 32) x += part[(int64_t)c * D + i % D];
    sum[warp][lane] = x;
    __syncthreads();
    if (warp == 0) {
        x = 0.0f;
#pragma unroll
        for (int w = 0; w < 32; ++w) x += sum[w][lane];
        float* out = k ? gkw : gqw;
        if (out) out[i % D] = x;
    }
}

template <typename T> RopeArgs<T> make_args(const RopeCall& c) {
    RopeArgs<T> a;
    a.q = (const T*)c.q, a.k = (const T*)c.k, a.v = (const T*)c.v;
    for (int i = 0; i < 3; ++i) a.qs[i] = c.strides[0][i], a.ks[i] = c.strides[1][i], a.vs[i] = c.strides[2][i];
    a.qo = (T*)c.qo, a.ko = (T*)c.ko, a.vo = (T*)c.vo;
    a.pos = c.pos, a.qw = c.qw, a.kw = c.kw, a.w_f32 = c.w_f32, a.eps = c.eps;
    a.B = c.B, a.T_len = c.T, a.Hq = c.Hq, a.Hkv = c.Hkv;
    a.rot = c.rope->rot, a.interleaved = c.rope->interleaved;
    a.axis[0] = a.axis[1] = 0;
    for (int i = 0; i < 64; ++i) {
        const bool there = i < c.rope->rot / 2;
        a.turn[i] = there ? c.rope->turn[i] : 0;
        if (there) a.axis[i >> 5] |= (unsigned long long)(c.rope->axis[i] & 3) << (2 * (i & 31));
    }
    return a;
}

template <typename T, int D> cudaError_t forward(const RopeCall& c, cudaStream_t s) {
    const RopeArgs<T> a = make_args<T>(c);
    constexpr int rows = Place<D>::kRows;
    const int groups = (c.Hq + rows - 1) / rows + (c.v ? 2 : 1) * ((c.Hkv + rows - 1) / rows);
    const int64_t tokens = (int64_t)c.B * c.T, want = (int64_t)device_sms(nullptr) * 16;
    const int split = (int)std::min<int64_t>(groups, (want + tokens - 1) / tokens);
    const int per_part = (groups + split - 1) / split, parts = (groups + per_part - 1) / per_part;
    const int64_t ctas = (tokens * parts + kWarps - 1) / kWarps;
    if (a.interleaved) rope_kernel<T, D, true><<<(unsigned)ctas, kThreads, 0, s>>>(a, parts, per_part);
    else rope_kernel<T, D, false><<<(unsigned)ctas, kThreads, 0, s>>>(a, parts, per_part);
    return cudaGetLastError();
}

template <typename T, int D> cudaError_t backward(const RopeCall& c, cudaStream_t s) {
    RopeBwdArgs<T> p;
    p.f = make_args<T>(c);
    p.gq = (T*)c.gq, p.gk = (T*)c.gk, p.gv = (T*)c.gv;
    for (int i = 0; i < 3; ++i) p.gqs[i] = c.gstrides[0][i], p.gks[i] = c.gstrides[1][i], p.gvs[i] = c.gstrides[2][i];
    p.part = (float*)c.ws;
    // CTAs by the bytes that queries, and keys with values, take
    const bool norm = c.qw || c.kw;
    const int ctas = rope_bwd_ctas(c.B, c.T);
    const double wq = c.Hq * (c.qw ? 3.0 : 2.0), wk = c.Hkv * ((c.kw ? 3.0 : 2.0) + (c.vo ? 2.0 : 0.0));
    const int q_ctas = std::min(ctas - 1, std::max(1, (int)(ctas * wq / (wq + wk) + 0.5)));
    constexpr size_t smem = kWarps * (kBwdStages * 128 * sizeof(uint4) + 128 * sizeof(float));
    auto kernel = p.f.interleaved ? (norm ? rope_bwd_kernel<T, D, true, true> : rope_bwd_kernel<T, D, false, true>)
                                  : (norm ? rope_bwd_kernel<T, D, true, false> : rope_bwd_kernel<T, D, false, false>);
    static std::atomic<uint64_t> ready[4];              // devices whose attribute is set, by kernel
    std::atomic<uint64_t>& done = ready[2 * p.f.interleaved + norm];
    int dev = -1;
    device_sms(&dev);
    cudaError_t e = cudaSuccess;
    if (dev < 0 || dev > 63 || !(done.load(std::memory_order_acquire) >> dev & 1)) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) done.fetch_or(1ull << dev, std::memory_order_release);
    }
    kernel<<<ctas, kThreads, smem, s>>>(p, q_ctas);
    e = cudaGetLastError();
    if (e != cudaSuccess || !norm) return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute early[1];
    early[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(2 * D / 32);
    cfg.blockDim = dim3(1024);
    cfg.stream = s;
    cfg.attrs = early;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, rope_weight_kernel, (const float*)p.part, q_ctas, ctas, D, c.qw ? c.gqw : (float*)nullptr,
                              c.kw ? c.gkw : (float*)nullptr);
}

}  // namespace

int rope_bwd_ctas(int B, int T) {
    const int64_t tokens = (int64_t)B * T;
    return (int)std::min<int64_t>(2 * ((tokens + kWarps - 1) / kWarps), (int64_t)device_sms(nullptr) * kBwdCtas);
}

cudaError_t launch_rope(const RopeCall& c, cudaStream_t s) {
    if (c.dt == KVQ_F16) return c.D == 64 ? forward<__half, 64>(c, s) : forward<__half, 128>(c, s);
    return c.D == 64 ? forward<__nv_bfloat16, 64>(c, s) : forward<__nv_bfloat16, 128>(c, s);
}

cudaError_t launch_rope_bwd(const RopeCall& c, cudaStream_t s) {
    if (c.dt == KVQ_F16) return c.D == 64 ? backward<__half, 64>(c, s) : backward<__half, 128>(c, s);
    return c.D == 64 ? backward<__nv_bfloat16, 64>(c, s) : backward<__nv_bfloat16, 128>(c, s);
}

}  // namespace kvq
