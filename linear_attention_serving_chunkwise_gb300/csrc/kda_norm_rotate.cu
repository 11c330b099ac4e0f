// Norms of queries and keys per head, their rotation by position, and keys and values into the
// slots of a paged cache, in one pass over the three.
//
//     y = x rsqrt(mean(x^2) + eps) w,    (y_a, y_b) <- (y_a cos p f - y_b sin p f, y_a sin p f + y_b cos p f)
//
// with p the token's position, f the pair's frequency (radians a token), and channels (a, b) = (i, i + rot / 2), or
// (2 i, 2 i + 1) when interleaved, for i < rot / 2; channels from rot on are only normed.  fp32 throughout, one
// rounding at the end.
//
// The angle: f / 2 pi as a 64-bit fraction of a turn, times the position as integers, so whole turns
// drop out of the product by themselves and a far position costs no accuracy (fp32 radians are off by 0.06 at a
// million tokens).  A CTA forms its tokens' sines and cosines once, for all heads.
//
// A lane holds two 16-byte chunks of a row that are each other's partners (or lie side by side where nothing is
// rotated), so a rotation needs no exchange and a norm three shuffles.  Bound: HBM.
#include "kda_common.cuh"
#include "kda_prompt_launch.h"

namespace kda {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMostTokens = 8;         // of a CTA

__device__ __forceinline__ void unpack(uint4 u, float (&x)[8])
{
    const uint32_t h[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(h[i] << 16);
        x[2 * i + 1] = __uint_as_float(h[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void unpack(uint4 u, float (&x)[4])
{
    x[0] = __uint_as_float(u.x); x[1] = __uint_as_float(u.y); x[2] = __uint_as_float(u.z); x[3] = __uint_as_float(u.w);
}
__device__ __forceinline__ uint4 pack(const float (&x)[8])
{
    uint32_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 p = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        h[i] = *reinterpret_cast<const uint32_t*>(&p);
    }
    return make_uint4(h[0], h[1], h[2], h[3]);
}
__device__ __forceinline__ uint4 pack(const float (&x)[4])
{
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
}

template <typename T, int D, bool kPairs>
__global__ void __launch_bounds__(kThreads) norm_rotate_kernel(NormRotateArgs a, int per_cta)
{
    constexpr int V = 16 / sizeof(T), CH = D / V, LANES = CH / 2, ROWS = 32 / LANES;   // a row's chunks and lanes, rows of a warp
    constexpr int U = 2;               // groups of rows whose loads are in flight together
    __shared__ float2 s_turn[kMostTokens][D / 2];           // cosine, sine
    __shared__ float s_w[2][D];
    const int t = threadIdx.x, lane = t & 31, w = t >> 5, l = lane % LANES, sub = lane / LANES;
    const int t0 = blockIdx.x * per_cta, tokens = min(per_cta, a.tokens - t0), half = a.rot / 2;

    for (int c = t; c < 2 * D; c += kThreads) {
        const float* src = c < D ? a.q_weight : a.k_weight;
        s_w[c / D][c % D] = src ? src[c % D] : 1.f;
    }
    for (int i = t; i < tokens * half; i += kThreads) {
        const int k = i / half, c = i - k * half;
        double turn = (double)a.inv_freq[c] * 0.15915494309189533577;
        turn -= floor(turn);
        const unsigned long long f = (unsigned long long)(turn * 18446744073709551616.0) * (unsigned long long)(long long)a.positions[t0 + k];
        const float h = (float)(int)(f >> 32) * 4.656612873077393e-10f;   // half turns, from -1 to 1
        s_turn[k][c] = make_float2(cospif(h), sinpif(h));
    }
    __syncthreads();

    // this lane's chunks of a row
    const int turned = a.rot / (2 * V);                     // chunks of each of the halves
    int c0, c1;
    if (kPairs) { c0 = 2 * l; c1 = 2 * l + 1; }
    else if (l < turned) { c0 = l; c1 = l + turned; }
    else { c0 = 2 * l; c1 = 2 * l + 1; }                    // (2 turned + 2 (l - turned))

    const int rows = a.heads + 2 * a.kv_heads, groups = (rows + ROWS - 1) / ROWS, items = tokens * groups;
    for (int i0 = w * U; i0 < items; i0 += kWarps * U) {
        uint4 in[U][2];
        T* dst[U];
        int token[U], kind[U];         // query, key, value; -1: nothing
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k = (i0 + u) / groups, r = (i0 + u - k * groups) * ROWS + sub, tok = t0 + k;
            token[u] = k;
            kind[u] = -1;
            in[u][0] = in[u][1] = make_uint4(0, 0, 0, 0);
            if (i0 + u >= items || r >= rows) continue;
            const T* src;
            if (r < a.heads) {
                kind[u] = 0;
                src = static_cast<const T*>(a.q) + (size_t)tok * a.q_stride + (size_t)r * D;
                dst[u] = static_cast<T*>(a.q_out) + ((size_t)tok * a.heads + r) * D;
            } else {
                const bool value = r >= a.heads + a.kv_heads;
                const int h = r - a.heads - (value ? a.kv_heads : 0);
                const long long slot = a.slots[tok];
                if (slot < 0) continue;
                if (slot >= a.num_slots) {
                    report_status(a.status, kDevBadSeqlens);
                    continue;
                }
                kind[u] = value ? 2 : 1;
                src = static_cast<const T*>(value ? a.v : a.k) + (size_t)tok * (value ? a.v_stride : a.k_stride) + (size_t)h * D;
                const long long page = slot / a.page_size;
                dst[u] = static_cast<T*>(value ? a.v_cache : a.k_cache) + (size_t)page * (value ? a.v_page_stride : a.k_page_stride) +
                         ((size_t)(slot - page * a.page_size) * a.kv_heads + h) * D;
            }
            in[u][0] = *(reinterpret_cast<const uint4*>(src) + c0);
            in[u][1] = *(reinterpret_cast<const uint4*>(src) + c1);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float x[V], y[V];
            unpack(in[u][0], x);
            unpack(in[u][1], y);
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < V; ++i) sum = fmaf(x[i], x[i], fmaf(y[i], y[i], sum));
#pragma unroll
            for (int o = LANES / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            if (kind[u] < 0) continue;
            if (kind[u] != 2) {
                if (a.norm) {
                    const float inv = 1.f / sqrtf(sum * (1.f / D) + a.eps);
                    const float* wt = s_w[kind[u]];
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        x[i] = x[i] * inv * wt[c0 * V + i];
                        y[i] = y[i] * inv * wt[c1 * V + i];
                    }
                }
                const float2* turn = s_turn[token[u]];
                if (kPairs) {
#pragma unroll
                    for (int i = 0; i < V; i += 2) {
                        if (c0 * V < a.rot) {
                            const float2 e = turn[(c0 * V + i) / 2];
                            const float p = x[i], q = x[i + 1];
                            x[i] = p * e.x - q * e.y;
                            x[i + 1] = p * e.y + q * e.x;
                        }
                        if (c1 * V < a.rot) {
                            const float2 e = turn[(c1 * V + i) / 2];
                            const float p = y[i], q = y[i + 1];
                            y[i] = p * e.x - q * e.y;
                            y[i + 1] = p * e.y + q * e.x;
                        }
                    }
                } else if (l < turned) {
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        const float2 e = turn[c0 * V + i];
                        const float p = x[i], q = y[i];
                        x[i] = p * e.x - q * e.y;
                        y[i] = p * e.y + q * e.x;
                    }
                }
                in[u][0] = pack(x);
                in[u][1] = pack(y);
            }
            *(reinterpret_cast<uint4*>(dst[u]) + c0) = in[u][0];
            *(reinterpret_cast<uint4*>(dst[u]) + c1) = in[u][1];
        }
    }
}

template <typename T, int D>
cudaError_t launch(const NormRotateArgs& a, cudaStream_t stream)
{
    // eight tokens to a CTA once that fills the GPU, one before
    const int per = a.tokens >= 152 * kMostTokens ? kMostTokens : 1, grid = (a.tokens + per - 1) / per;
    if (a.interleaved) norm_rotate_kernel<T, D, true><<<grid, kThreads, 0, stream>>>(a, per);
    else norm_rotate_kernel<T, D, false><<<grid, kThreads, 0, stream>>>(a, per);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_norm_rotate(const NormRotateArgs& a, cudaStream_t stream)
{
    if (a.bf16) return a.dim == 128 ? launch<__nv_bfloat16, 128>(a, stream) : launch<__nv_bfloat16, 64>(a, stream);
    return a.dim == 128 ? launch<float, 128>(a, stream) : launch<float, 64>(a, stream);
}

}  // namespace kda
