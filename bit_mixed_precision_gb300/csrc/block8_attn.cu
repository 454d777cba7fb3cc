// block8_attn: attention of a few queries over the 8-bit block cache, over all
// tokens or over a list of blocks per query (include/kvq.h has the format).
//
// One CTA per (unit, query, head).  Four warps take the blocks in turn, each
// with its own running maximum, sum and output; the CTA merges the four.  With
// accumulate a second kernel adds each block's softmax weight to its acc.
#include <type_traits>

#include "block8_device.cuh"
#include "kvq_internal.h"

namespace kvq {

KVQ_DEFINE_STATUS(block8_attn)

namespace {

using namespace b8;

struct AttnArgs {
    kvq_block8 c;
    const void* q;
    int64_t qs[3];
    int n_q;
    const int32_t* n_new;
    float sm_scale;
    const int32_t *blocks, *list_len;
    int n_sel, accumulate;
    void* o;
    float *lse, *lse2;              // lse2: workspace, per (unit, query, head)
};

constexpr int kWarps = 4;
constexpr float kLog2e = 1.4426950408889634f;

template <int CODE> __device__ __forceinline__ void four_codes(uint32_t w, float (&f)[4]) {
    if constexpr (CODE == KVQ_CODE_E4M3) {
        uint32_t a, b;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(a) : "h"((uint16_t)w));
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(b) : "h"((uint16_t)(w >> 16)));
        const float2 x = __half22float2(*reinterpret_cast<__half2*>(&a)), y = __half22float2(*reinterpret_cast<__half2*>(&b));
        f[0] = x.x; f[1] = x.y; f[2] = y.x; f[3] = y.y;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = (float)(int8_t)(w >> (8 * i));
    }
}

// The warp's dot product of its query with one token's codes.
template <int CODE>
__device__ __forceinline__ float logit(const float (&q)[4], const uint8_t* codes, bool mine) {
    float s = 0.0f;
    if (mine) {
        float f[4];
        four_codes<CODE>(*reinterpret_cast<const uint32_t*>(codes), f);
        s = q[0] * f[0] + q[1] * f[1] + q[2] * f[2] + q[3] * f[3];
    }
    for (int w = 16; w; w >>= 1) s += __shfl_xor_sync(0xffffffffu, s, w);
    return s;
}

template <typename T, int D, int CODE>
__global__ void __launch_bounds__(kWarps * 32) attn_kernel(AttnArgs a) {
    __shared__ float part[kWarps][D + 2];
    const kvq_block8& c = a.c;
    const int g = c.Hq / c.Hkv, hh = blockIdx.x % g, row = blockIdx.x / g, u = row / a.n_q, t = row % a.n_q;
    const int b = u / c.Hkv, h = (u % c.Hkv) * g + hh, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int m = new_rows(a.n_new, b, a.n_q, &g_status_block8_attn);
    const int limit = min(query_limit(c.count[u], m, t), c.max_blocks * c.block);
    const int32_t* list = a.blocks ? a.blocks + (size_t)row * a.n_sel : nullptr;
    int nb = (limit + c.block - 1) / c.block;
    const int held = (min(c.count[u], c.max_blocks * c.block) + c.block - 1) / c.block;
    if (list) nb = limit > 0 ? min(max(a.list_len[row], 0), a.n_sel) : 0;
    const bool mine = lane < D / 4;
    float q[4] = {0, 0, 0, 0}, o[4] = {0, 0, 0, 0}, mx = -INFINITY, l = 0.0f;
    const T* qp = (const T*)a.q + b * a.qs[0] + h * a.qs[1] + t * a.qs[2];
    if (mine && t < m)
        for (int i = 0; i < 4; ++i) q[i] = Elem<T>::to_f(qp[lane * 4 + i]);
    for (int j = warp; j < nb; j += kWarps) {
        const int blk = list ? list[j] : j;
        const int phys = (unsigned)blk < (unsigned)held ? c.table[(size_t)u * c.max_blocks + blk] : -1;
        if ((unsigned)phys >= (unsigned)c.n_blocks) {
            if (lane == 0) atomicOr(&g_status_block8_attn, kDevCheck);
            continue;
        }
        const float ks = c.k_scale[phys] * a.sm_scale * kLog2e, vs = c.v_scale[phys];
        const int n = min(c.block, limit - blk * c.block);
        for (int i = 0; i < n; ++i) {
            const size_t at = ((size_t)phys * c.block + i) * D + lane * 4;
            const float s = logit<CODE>(q, c.k_codes + at, mine) * ks;
            const float nm = fmaxf(mx, s), f0 = mx == nm ? 1.0f : exp2f(mx - nm), p = exp2f(s - nm);
            mx = nm;
            l = l * f0 + p;
            if (mine) {
                float f[4];
                four_codes<CODE>(*reinterpret_cast<const uint32_t*>(c.v_codes + at), f);
                for (int k = 0; k < 4; ++k) o[k] = o[k] * f0 + p * vs * f[k];
            }
        }
    }
    if (mine)
        for (int k = 0; k < 4; ++k) part[warp][lane * 4 + k] = o[k];
    if (lane == 0) {
        part[warp][D] = mx;
        part[warp][D + 1] = l;
    }
    __syncthreads();
    float top = -INFINITY, total = 0.0f;
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, part[w][D]);
    const float ref = top == -INFINITY ? 0.0f : top;
    for (int w = 0; w < kWarps; ++w) total += part[w][D + 1] * exp2f(part[w][D] - ref);
    const size_t orow = ((size_t)b * c.Hq + h) * a.n_q + t;
    for (int d = threadIdx.x; d < D; d += kWarps * 32) {
        float x = 0.0f;
        for (int w = 0; w < kWarps; ++w) x += part[w][d] * exp2f(part[w][D] - ref);
        ((T*)a.o)[orow * D + d] = Elem<T>::from_f(total == 0.0f ? 0.0f : x / total);
    }
    if (threadIdx.x == 0) {
        const float lse2 = total == 0.0f ? -INFINITY : ref + log2f(total);
        if (a.lse) a.lse[orow] = lse2 / kLog2e;
        if (a.accumulate) a.lse2[(size_t)row * g + hh] = lse2;
    }
}

// The blocks' softmax weights, one CTA per unit: queries in turn, warps over blocks.
template <typename T, int D, int CODE>
__global__ void __launch_bounds__(kWarps * 32) weight_kernel(AttnArgs a) {
    const kvq_block8& c = a.c;
    const int g = c.Hq / c.Hkv, u = blockIdx.x, b = u / c.Hkv, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const bool mine = lane < D / 4;
    const int m = new_rows(a.n_new, b, a.n_q, &g_status_block8_attn);
    const int held = (min(c.count[u], c.max_blocks * c.block) + c.block - 1) / c.block;
    for (int t = 0; t < m; ++t) {
        const int row = u * a.n_q + t, limit = min(query_limit(c.count[u], m, t), c.max_blocks * c.block);
        const int32_t* list = a.blocks ? a.blocks + (size_t)row * a.n_sel : nullptr;
        int nb = (limit + c.block - 1) / c.block;
        if (list) nb = limit > 0 ? min(max(a.list_len[row], 0), a.n_sel) : 0;
        for (int j = warp; j < nb; j += kWarps) {
            const int blk = list ? list[j] : j;
            const int phys = (unsigned)blk < (unsigned)held ? c.table[(size_t)u * c.max_blocks + blk] : -1;
            if ((unsigned)phys >= (unsigned)c.n_blocks) continue;
            const float ks = c.k_scale[phys] * a.sm_scale * kLog2e;
            const int n = min(c.block, limit - blk * c.block);
            float weight = 0.0f;
            for (int hh = 0; hh < g; ++hh) {
                float q[4] = {0, 0, 0, 0};
                const T* qp = (const T*)a.q + b * a.qs[0] + ((u % c.Hkv) * g + hh) * a.qs[1] + t * a.qs[2];
                if (mine)
                    for (int i = 0; i < 4; ++i) q[i] = Elem<T>::to_f(qp[lane * 4 + i]);
                const float lse2 = a.lse2[(size_t)row * g + hh];
                for (int i = 0; i < n; ++i)
                    weight += exp2f(logit<CODE>(q, c.k_codes + ((size_t)phys * c.block + i) * D + lane * 4, mine) * ks - lse2);
            }
            if (lane == 0 && n > 0) atomicAdd(&c.acc[phys], weight);
        }
        __syncthreads();
    }
}

}  // namespace

size_t block8_attn_bytes(const kvq_block8& c, int n_q, int, int accumulate) {
    return accumulate ? (size_t)c.B * c.Hq * n_q * sizeof(float) : 0;
}

cudaError_t launch_block8_attn(const void* q, const int64_t* qs, int n_q, const int32_t* n_new, const kvq_block8& c,
                               float sm_scale, const int32_t* blocks, const int32_t* list_len, int n_sel,
                               int accumulate, void* o, float* lse, void* ws, cudaStream_t s) {
    AttnArgs a{c, q, {qs[0], qs[1], qs[2]}, n_q, n_new, sm_scale, blocks, list_len, n_sel, accumulate, o, lse, (float*)ws};
    const unsigned grid = (unsigned)(c.B * c.Hq * n_q);
    auto go = [&](auto t, auto d, auto k) {
        attn_kernel<decltype(t), decltype(d)::value, decltype(k)::value><<<grid, kWarps * 32, 0, s>>>(a);
        if (accumulate)
            weight_kernel<decltype(t), decltype(d)::value, decltype(k)::value>
                <<<(unsigned)(c.B * c.Hkv), kWarps * 32, 0, s>>>(a);
        return cudaGetLastError();
    };
    auto by_code = [&](auto t, auto d) {
        return c.code == KVQ_CODE_E4M3 ? go(t, d, std::integral_constant<int, KVQ_CODE_E4M3>{})
                                       : go(t, d, std::integral_constant<int, KVQ_CODE_INT8>{});
    };
    using D64 = std::integral_constant<int, 64>;
    using D128 = std::integral_constant<int, 128>;
    if (c.dtype == KVQ_F16) return c.D == 64 ? by_code(__half{}, D64{}) : by_code(__half{}, D128{});
    return c.D == 64 ? by_code(__nv_bfloat16{}, D64{}) : by_code(__nv_bfloat16{}, D128{});
}

}  // namespace kvq
