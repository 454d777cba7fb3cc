// qk_norm_rope and qk_norm_rope_bwd: a layer's projection [B, T, heads, D] to what attention and the caches take
// ([B, heads, T, D], queries and keys normed per head and rotated), and the gradient of that.
//
// Mathematics (x a head's row, w the norm's weight, f_i the frequency of pair i in radians per position):
//   r = 1 / sqrt(mean(x^2) + eps);  y = x r w;  pair (a, b) of y with phi = pos f: (a cos - b sin, b cos + a sin)
//   backward: dy = the pairs of d turned by -phi;  dw = sum over rows of dy x r;  g = dy w;
//             dx = r (g - (x r) mean(g (x r)))
// Angles: f is kept as a 64-bit fraction of a turn, so pos * f modulo a turn is one wrapping integer product, exact for
// every int32 position but for the fraction's own 2^-64 (positions of 2^20 lose 2^-44 of a turn); what is left, in
// [-1/2, 1/2) turns, becomes float32 and cosine and sine.
// Bound: HBM, each row is read and written once.  D / 16 lanes share a row, each with the two 16-byte pieces that hold
// the two sides of its eight pairs, so that the rotation needs no exchange and the norm's sum two or three shuffles; a
// warp holds 64 / (D / 8) rows of one token at a time and computes the token's eight angles a lane once for all heads.
// All arithmetic is float32; an output is rounded once.
#include <algorithm>

#include "kvq_common.cuh"
#include "kvq_internal.h"

namespace kvq {

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;

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
    float* part;                    // [CTA][2][D] sums for the weights' gradients
};

// The 16 values of a lane: pieces c0 and c1 (eight channels each) of its row.
template <int D> struct Place {
    static constexpr int kLanes = D / 16;       // lanes of a row
    static constexpr int kRows = 32 / kLanes;   // rows of a warp
    int c0, c1, pair;                           // pieces; first pair
    bool rotated;
    __device__ __forceinline__ Place(int lane, int rot, int interleaved) {
        const int l = lane % kLanes, n = rot / 16;
        pair = 8 * l;
        rotated = l < n;
        if (interleaved || l >= n) {
            c0 = 2 * l;
            c1 = c0 + 1;
        } else {
            c0 = l;
            c1 = l + n;
        }
    }
};

template <typename T> __device__ __forceinline__ void unpack8(const uint4& u, float* x) {
    const T* e = reinterpret_cast<const T*>(&u);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = Elem<T>::to_f(e[i]);
}

template <typename T> __device__ __forceinline__ uint4 pack8(const float* x) {
    uint4 u;
    T* e = reinterpret_cast<T*>(&u);
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = Elem<T>::from_f(x[i]);
    return u;
}

template <typename T> __device__ __forceinline__ void load_weight(const void* w, int f32, int c0, int c1, float* out) {
    if (f32) {
        const float4* p = reinterpret_cast<const float4*>(w);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float4 x = p[2 * (i < 2 ? c0 : c1) + (i & 1)];
            out[4 * i] = x.x, out[4 * i + 1] = x.y, out[4 * i + 2] = x.z, out[4 * i + 3] = x.w;
        }
    } else {
        const uint4* p = reinterpret_cast<const uint4*>(w);
        unpack8<T>(p[c0], out);
        unpack8<T>(p[c1], out + 8);
    }
}

// Cosine and sine of the lane's eight pairs at the token's positions.
template <typename T, int D>
__device__ __forceinline__ void angles(const RopeArgs<T>& a, const Place<D>& at, int64_t token, int64_t n_tokens,
                                       float* cs, float* sn) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        cs[j] = 1.0f, sn[j] = 0.0f;
        if (at.rotated) {
            const int p = at.pair + j;
            const int axis = (int)(a.axis[p >> 5] >> (2 * (p & 31))) & 3;
            const long long pos = a.pos[axis * n_tokens + token];
            const unsigned long long turns = (unsigned long long)pos * a.turn[p];
            // the fraction of a turn in [-1/2, 1/2) as half turns in [-1, 1)
            const float x = (float)(int32_t)(turns >> 32) * 4.656612873077393e-10f;
            sincospif(x, &sn[j], &cs[j]);
        }
    }
}

// The lane's pairs turned by phi (sign = 1) or back (-1): pair j is (x[j], x[8 + j]), interleaved (x[2 j], x[2 j + 1]).
template <int SIGN>
__device__ __forceinline__ void turn_pairs(float* x, const float* cs, const float* sn, int interleaved) {
    if (interleaved) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float a = x[2 * j], b = x[2 * j + 1], s = SIGN * sn[j];
            x[2 * j] = a * cs[j] - b * s;
            x[2 * j + 1] = b * cs[j] + a * s;
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float a = x[j], b = x[8 + j], s = SIGN * sn[j];
            x[j] = a * cs[j] - b * s;
            x[8 + j] = b * cs[j] + a * s;
        }
    }
}

template <int LANES> __device__ __forceinline__ float row_sum(float x) {
#pragma unroll
    for (int m = LANES / 2; m > 0; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
    return x;
}

template <int D> __device__ __forceinline__ float row_scale(const float* x, float eps) {
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) s = fmaf(x[i], x[i], s);
    return rsqrtf(row_sum<D / 16>(s) * (1.0f / D) + eps);
}

// ------------------------------------------------------------------ forward

// One warp per (token, share of its heads): the token's groups of kRows heads, first those of the queries, then the
// keys', then the values', are split into `parts` equal shares (one share for prompts; as many as there are groups for
// steps of few sequences, whose time is latency).
template <typename T, int D>
__global__ void __launch_bounds__(kThreads)
    rope_kernel(const __grid_constant__ RopeArgs<T> a, int parts, int per_part) {
    using P = Place<D>;
    const int lane = threadIdx.x & 31;
    const int64_t item = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    const int64_t n_tokens = (int64_t)a.B * a.T_len;
    const int64_t token = item / parts;
    if (token >= n_tokens) return;
    const int b = (int)(token / a.T_len), t = (int)(token % a.T_len);
    const int gq = (a.Hq + P::kRows - 1) / P::kRows, gk = (a.Hkv + P::kRows - 1) / P::kRows;
    const int first = (int)(item % parts) * per_part;
    const int last = min(first + per_part, gq + (a.v ? 2 : 1) * gk);
    const P at(lane, a.rot, a.interleaved);
    const int sub = lane / P::kLanes;
    float cs[8], sn[8];
    if (first < gq + gk) angles<T, D>(a, at, token, n_tokens, cs, sn);
#pragma unroll
    for (int kind = 0; kind < 3; ++kind) {
        const int from = kind == 0 ? 0 : kind == 1 ? gq : gq + gk;
        const int to = kind == 0 ? gq : kind == 1 ? gq + gk : gq + 2 * gk;
        const int H = kind == 0 ? a.Hq : a.Hkv;
        const T* in = kind == 0 ? a.q : kind == 1 ? a.k : a.v;
        const int64_t* st = kind == 0 ? a.qs : kind == 1 ? a.ks : a.vs;
        T* out = kind == 0 ? a.qo : kind == 1 ? a.ko : a.vo;
        const void* w = kind == 0 ? a.qw : kind == 1 ? a.kw : nullptr;
        const int g0 = max(first, from), g1 = min(last, to);
        if (g0 >= g1) continue;
        float wt[16];
        if (kind < 2 && w) load_weight<T>(w, a.w_f32, at.c0, at.c1, wt);
        in += (int64_t)b * st[0] + (int64_t)t * st[1];
        out += ((int64_t)b * H * a.T_len + t) * D;
#pragma unroll 2
        for (int g = g0; g < g1; ++g) {
            const int h = (g - from) * P::kRows + sub;
            uint4 u0 = make_uint4(0, 0, 0, 0), u1 = u0;
            if (h < H) {
                const uint4* p = reinterpret_cast<const uint4*>(in + h * st[2]);
                u0 = p[at.c0];
                u1 = p[at.c1];
            }
            if (kind < 2) {
                float x[16];
                unpack8<T>(u0, x);
                unpack8<T>(u1, x + 8);
                if (w) {
                    const float r = row_scale<D>(x, a.eps);
#pragma unroll
                    for (int i = 0; i < 16; ++i) x[i] = x[i] * r * wt[i];
                }
                turn_pairs<1>(x, cs, sn, a.interleaved);
                u0 = pack8<T>(x);
                u1 = pack8<T>(x + 8);
            }
            if (h < H) {
                uint4* p = reinterpret_cast<uint4*>(out + (int64_t)h * a.T_len * D);
                p[at.c0] = u0;
                p[at.c1] = u1;
            }
        }
    }
}

// ------------------------------------------------------------------ backward

// One warp per token at a time, the CTAs' warps striding over the tokens; each lane keeps the weights' gradients of its
// 16 channels in float32.  Sums go lane, warp, CTA, then over the CTAs in a second kernel, always in the same order.
template <typename T, int D, bool NORM>
__global__ void __launch_bounds__(kThreads)
    rope_bwd_kernel(const __grid_constant__ RopeBwdArgs<T> p) {
    using P = Place<D>;
    const RopeArgs<T>& a = p.f;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t n_tokens = (int64_t)a.B * a.T_len;
    const P at(lane, a.rot, a.interleaved);
    const int sub = lane / P::kLanes;
    float dw[2][16];
#pragma unroll
    for (int i = 0; i < 16; ++i) dw[0][i] = dw[1][i] = 0.0f;
    for (int64_t token = (int64_t)blockIdx.x * kWarps + warp; token < n_tokens; token += (int64_t)gridDim.x * kWarps) {
        const int b = (int)(token / a.T_len), t = (int)(token % a.T_len);
        float cs[8], sn[8];
        angles<T, D>(a, at, token, n_tokens, cs, sn);
#pragma unroll
        for (int kind = 0; kind < 3; ++kind) {
            const int H = kind == 0 ? a.Hq : a.Hkv;
            const T* raw = kind == 0 ? a.q : a.k;
            const int64_t* st = kind == 0 ? a.qs : a.ks;
            const T* in = kind == 0 ? a.qo : kind == 1 ? a.ko : a.vo;
            T* out = kind == 0 ? p.gq : kind == 1 ? p.gk : p.gv;
            const int64_t* gs = kind == 0 ? p.gqs : kind == 1 ? p.gks : p.gvs;
            const void* w = kind == 0 ? a.qw : kind == 1 ? a.kw : nullptr;
            if (kind == 2 && !in) continue;
            const bool norm = NORM && kind < 2 && w;
            float wt[16];
            if (norm) load_weight<T>(w, a.w_f32, at.c0, at.c1, wt);
            in += ((int64_t)b * H * a.T_len + t) * D;
            if (norm) raw += (int64_t)b * st[0] + (int64_t)t * st[1];
            out += (int64_t)b * gs[0] + (int64_t)t * gs[1];
#pragma unroll 1
            for (int h0 = 0; h0 < H; h0 += P::kRows) {
                const int h = h0 + sub;
                uint4 u0 = make_uint4(0, 0, 0, 0), u1 = u0, x0 = u0, x1 = u0;
                if (h < H) {
                    const uint4* q = reinterpret_cast<const uint4*>(in + (int64_t)h * a.T_len * D);
                    u0 = q[at.c0];
                    u1 = q[at.c1];
                    if (norm) {
                        const uint4* r = reinterpret_cast<const uint4*>(raw + h * st[2]);
                        x0 = r[at.c0];
                        x1 = r[at.c1];
                    }
                }
                if (kind < 2) {
                    float d[16];
                    unpack8<T>(u0, d);
                    unpack8<T>(u1, d + 8);
                    turn_pairs<-1>(d, cs, sn, a.interleaved);
                    if (norm) {
                        float x[16];
                        unpack8<T>(x0, x);
                        unpack8<T>(x1, x + 8);
                        const float r = row_scale<D>(x, a.eps);
                        float dot = 0.0f;
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            x[i] *= r;
                            dw[kind & 1][i] = fmaf(d[i], x[i], dw[kind & 1][i]);
                            d[i] *= wt[i];
                            dot = fmaf(d[i], x[i], dot);
                        }
                        dot = row_sum<D / 16>(dot) * (1.0f / D);
#pragma unroll
                        for (int i = 0; i < 16; ++i) d[i] = r * (d[i] - x[i] * dot);
                    }
                    u0 = pack8<T>(d);
                    u1 = pack8<T>(d + 8);
                }
                if (h < H) {
                    uint4* q = reinterpret_cast<uint4*>(out + h * gs[2]);
                    q[at.c0] = u0;
                    q[at.c1] = u1;
                }
            }
        }
    }
    if (!NORM) return;
    // rows of the warp, then warps of the CTA
    __shared__ float sum[kWarps][2][D];
#pragma unroll
    for (int kind = 0; kind < 2; ++kind)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float x = dw[kind][i];
#pragma unroll
            for (int m = P::kLanes; m < 32; m <<= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
            if (sub == 0) sum[warp][kind][8 * (i < 8 ? at.c0 : at.c1) + (i & 7)] = x;
        }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * D; i += kThreads) {
        float x = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) x += sum[w][i / D][i % D];
        p.part[(int64_t)blockIdx.x * 2 * D + i] = x;
    }
}

// The CTAs' sums: one CTA per 32 of the 2 D channels, its warps striding over the parts.
__global__ void __launch_bounds__(1024)
    rope_weight_kernel(const float* __restrict__ part, int n, int D, float* __restrict__ gqw, float* __restrict__ gkw) {
    __shared__ float sum[32][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, i = blockIdx.x * 32 + lane;
    grid_dependency_wait();
    float x = 0.0f;
    for (int c = warp; c < n; c += 32) x += part[(int64_t)c * 2 * D + i];
    sum[warp][lane] = x;
    __syncthreads();
    if (warp == 0) {
        x = 0.0f;
#pragma unroll
        for (int w = 0; w < 32; ++w) x += sum[w][lane];
        float* out = i < D ? gqw : gkw;
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
    rope_kernel<T, D><<<(unsigned)ctas, kThreads, 0, s>>>(a, parts, per_part);
    return cudaGetLastError();
}

template <typename T, int D> cudaError_t backward(const RopeCall& c, cudaStream_t s) {
    RopeBwdArgs<T> p;
    p.f = make_args<T>(c);
    p.gq = (T*)c.gq, p.gk = (T*)c.gk, p.gv = (T*)c.gv;
    for (int i = 0; i < 3; ++i) p.gqs[i] = c.gstrides[0][i], p.gks[i] = c.gstrides[1][i], p.gvs[i] = c.gstrides[2][i];
    p.part = (float*)c.ws;
    const int ctas = rope_bwd_ctas(c.B, c.T);
    if (!c.qw && !c.kw) {
        rope_bwd_kernel<T, D, false><<<ctas, kThreads, 0, s>>>(p);
        return cudaGetLastError();
    }
    rope_bwd_kernel<T, D, true><<<ctas, kThreads, 0, s>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    rope_weight_kernel<<<2 * D / 32, 1024, 0, s>>>(p.part, ctas, D, c.qw ? c.gqw : nullptr, c.kw ? c.gkw : nullptr);
    return cudaGetLastError();
}

}  // namespace

int rope_bwd_ctas(int B, int T) {
    const int64_t tokens = (int64_t)B * T;
    return (int)std::min<int64_t>((tokens + kWarps - 1) / kWarps, (int64_t)device_sms(nullptr) * 2);
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
