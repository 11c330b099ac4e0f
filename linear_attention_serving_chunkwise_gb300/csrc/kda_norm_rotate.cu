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
// million tokens).  1 / 2 pi is two doubles, so a high frequency costs none either: the fraction is within 2^-64 for frequencies
// up to 2^40, the angle within 2^-33 of a turn for any position.  A CTA forms its pairs' fractions, then its tokens' sines and
// cosines, once for all heads.
//
// A lane holds two 16-byte chunks of a row that are each other's partners (or lie side by side where nothing is
// rotated), so a rotation needs no exchange and a norm three shuffles.  A warp has one token (or an eighth of one, where
// tokens are few), whose turns and weights stay in registers for all its rows: read from shared memory for every row
// they were what bound it (364 us instead of 300 for 32768 tokens).
// Bound: HBM.  32768 tokens, 96 query and 8 cache heads of 128 channels, bf16: 295 us, 6.4 TB/s (0.94 of a copy); fp32, 32 and 8
// heads: 240 us, 6.7 TB/s; 64 tokens: 6.1 us, the launch and the chain of one row.  Two rows in flight a lane and three CTAs an SM:
// 299 us; four and two 303, one and four 321.
#include "kda_common.cuh"
#include "kda_prompt_launch.h"

namespace kda {
namespace {

constexpr int kThreads = 256;
constexpr int kMostTokens = 8;         // of a CTA: a warp each
constexpr double kPerTurn = 0.15915494309189535, kPerTurnRest = -9.839338337591243e-18;    // 1 / 2 pi, to 2^-110
constexpr double kTwo64 = 18446744073709551616.0;

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
__global__ void __launch_bounds__(kThreads, 3) norm_rotate_kernel(NormRotateArgs a, int per_cta)
{
    constexpr int V = 16 / sizeof(T), CH = D / V, LANES = CH / 2, ROWS = 32 / LANES;   // a row's chunks and lanes, rows of a warp
    constexpr int U = 2;               // groups of rows whose loads are in flight together
    __shared__ float4 s_turn[kMostTokens][V / 2][LANES];    // cosine, sine of a lane's V pairs, two at a time
    __shared__ unsigned long long s_frac[D / 2];            // a pair's turn a token, as a fraction of 2^64
    __shared__ bool s_finite[D / 2];
    __shared__ int s_pos[kMostTokens];
    const int t = threadIdx.x, lane = t & 31, l = lane % LANES, sub = lane / LANES;
    const int t0 = blockIdx.x * per_cta, tokens = min(per_cta, a.tokens - t0), half = a.rot / 2;
    const int turned = a.rot / (2 * V);                     // chunks of each of the halves

    for (int c = t; c < half; c += kThreads) {
        const float freq = a.inv_freq[c];
        const double x = freq, hi = x * kPerTurn, lo = fma(x, kPerTurn, -hi) + x * kPerTurnRest;
        s_frac[c] = (unsigned long long)__double2ll_rn((hi - rint(hi)) * kTwo64) + (unsigned long long)__double2ll_rn((lo - rint(lo)) * kTwo64);
        s_finite[c] = isfinite(freq);                       // (the conversions make some angle of the others too)
    }
    if (half && t >= kThreads - tokens) s_pos[kThreads - 1 - t] = a.positions[t0 + kThreads - 1 - t];
    __syncthreads();
    for (int i = t; i < tokens * half; i += kThreads) {
        const int k = i / half, c = i - k * half;
        const unsigned long long f = s_frac[c] * (unsigned long long)(long long)s_pos[k];
        // The upper 24 bits as half turns from -1 to 1, exact in fp32; the next 24 in radians, b: sin(h + b) = sin h + b cos h to 1e-13.
        const float h = (float)((int)(f >> 32) & ~255) * 4.656612873077393e-10f, b = (float)(int)(f >> 16 & 0xffffff) * (6.2831853f / 281474976710656.f);
        const float co = cospif(h), si = sinpif(h);
        // pair c is the (c % V)-th of lane c / V, in both orders
        reinterpret_cast<float2*>(&s_turn[k][c % V / 2][c / V])[c & 1] = s_finite[c] ? make_float2(fmaf(-si, b, co), fmaf(co, b, si)) : make_float2(NAN, NAN);
    }
    __syncthreads();

    // this warp's token, and its share of the token's rows
    const int each = kThreads / 32 / per_cta, k = (t >> 5) / each, part = (t >> 5) % each, tok = t0 + k;
    if (k >= tokens) return;
    // this lane's chunks of a row, and whether it has pairs to turn
    int c0 = 2 * l, c1 = 2 * l + 1;                         // (of what is not turned: 2 turned + 2 (l - turned))
    if (!kPairs && l < turned) { c0 = l; c1 = l + turned; }
    float2 turn[V];
#pragma unroll
    for (int i = 0; i < V; i += 2) {
        float4 e = make_float4(0.f, 0.f, 0.f, 0.f);
        if (l * V < half) e = s_turn[k][i / 2][l];
        turn[i] = make_float2(e.x, e.y);
        turn[i + 1] = make_float2(e.z, e.w);
    }
    float wx[V], wy[V];
    auto weights = [&](const float* w) {
#pragma unroll
        for (int i = 0; i < V; i += 4) {
            const float4 one = make_float4(1.f, 1.f, 1.f, 1.f);
            const float4 x = w ? make_float4(w[c0 * V + i], w[c0 * V + i + 1], w[c0 * V + i + 2], w[c0 * V + i + 3]) : one;
            const float4 y = w ? make_float4(w[c1 * V + i], w[c1 * V + i + 1], w[c1 * V + i + 2], w[c1 * V + i + 3]) : one;
            wx[i] = x.x; wx[i + 1] = x.y; wx[i + 2] = x.z; wx[i + 3] = x.w;
            wy[i] = y.x; wy[i + 1] = y.y; wy[i + 2] = y.z; wy[i + 3] = y.w;
        }
    };
    // a row's norm and rotation, all lanes of a warp together
    auto apply = [&](uint4 (&in)[2]) {
        float x[V], y[V];
        unpack(in[0], x);
        unpack(in[1], y);
        if (a.norm) {
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < V; ++i) sum = fmaf(x[i], x[i], fmaf(y[i], y[i], sum));
#pragma unroll
            for (int o = LANES / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            const float inv = 1.f / sqrtf(sum * (1.f / D) + a.eps);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                x[i] = x[i] * inv * wx[i];
                y[i] = y[i] * inv * wy[i];
            }
        }
        if (kPairs) {
#pragma unroll
            for (int i = 0; i < V; i += 2) {
                if (l * V < half) {                         // (a lane's pairs are turned together: rot is a multiple of 2 V)
                    const float2 e = turn[i / 2], g = turn[V / 2 + i / 2];
                    float p = x[i], q = x[i + 1];
                    x[i] = p * e.x - q * e.y;
                    x[i + 1] = p * e.y + q * e.x;
                    p = y[i], q = y[i + 1];
                    y[i] = p * g.x - q * g.y;
                    y[i + 1] = p * g.y + q * g.x;
                }
            }
        } else if (l < turned) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float p = x[i], q = y[i];
                x[i] = p * turn[i].x - q * turn[i].y;
                y[i] = p * turn[i].y + q * turn[i].x;
            }
        }
        in[0] = pack(x);
        in[1] = pack(y);
    };

    // queries
    weights(a.q_weight);
    const uint4* src = reinterpret_cast<const uint4*>(static_cast<const T*>(a.q) + (size_t)tok * a.q_stride);
    uint4* dst = reinterpret_cast<uint4*>(static_cast<T*>(a.q_out) + (size_t)tok * a.heads * D);
    for (int r0 = part * U * ROWS; r0 < a.heads; r0 += each * U * ROWS) {
        uint4 in[U][2];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int r = r0 + u * ROWS + sub;
            in[u][0] = in[u][1] = make_uint4(0, 0, 0, 0);
            if (r < a.heads) {
                in[u][0] = src[r * CH + c0];
                in[u][1] = src[r * CH + c1];
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int r = r0 + u * ROWS + sub;
            apply(in[u]);
            if (r < a.heads) {
                dst[r * CH + c0] = in[u][0];
                dst[r * CH + c1] = in[u][1];
            }
        }
    }
    // keys, and the values that go to the same slot
    const long long slot = a.slots[tok];
    if (slot < 0) return;
    if (slot >= a.num_slots) {
        if (part == 0 && lane == 0) report_status(a.status, kDevBadSeqlens);
        return;
    }
    weights(a.k_weight);
    const long long page = slot / a.page_size;
    const size_t in_page = (size_t)(slot - page * a.page_size) * a.kv_heads * D;
    const uint4* ks = reinterpret_cast<const uint4*>(static_cast<const T*>(a.k) + (size_t)tok * a.k_stride);
    const uint4* vs = reinterpret_cast<const uint4*>(static_cast<const T*>(a.v) + (size_t)tok * a.v_stride);
    uint4* kd = reinterpret_cast<uint4*>(static_cast<T*>(a.k_cache) + (size_t)page * a.k_page_stride + in_page);
    uint4* vd = reinterpret_cast<uint4*>(static_cast<T*>(a.v_cache) + (size_t)page * a.v_page_stride + in_page);
    for (int r0 = part * ROWS; r0 < a.kv_heads; r0 += each * ROWS) {
        const int r = r0 + sub;
        const bool there = r < a.kv_heads;
        uint4 x[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)}, y[2];
        if (there) {
            x[0] = ks[r * CH + c0];
            x[1] = ks[r * CH + c1];
            y[0] = vs[r * CH + c0];
            y[1] = vs[r * CH + c1];
        }
        apply(x);
        if (there) {
            kd[r * CH + c0] = x[0];
            kd[r * CH + c1] = x[1];
            vd[r * CH + c0] = y[0];
            vd[r * CH + c1] = y[1];
        }
    }
}

template <typename T, int D>
cudaError_t launch(const NormRotateArgs& a, cudaStream_t stream)
{
    // Fewer warps to a token as tokens fill the GPU (1, 2, 4, 8 tokens to a CTA; us, 32 and 8 heads; turns formed token by token): 256 tokens 6.4, 6.4, 8.4, 10.5;
    // 608 10.5, 8.4, 8.4, 10.4; 1024 14.6, 12.5, 10.5, 10.5; 2432 24.7, 16.7, 16.6, 14.6; 32768 291, 187, 146, 140.
    const int per = a.tokens <= 304 ? 1 : a.tokens <= 608 ? 2 : a.tokens <= 1216 ? 4 : kMostTokens, grid = (a.tokens - 1) / per + 1;
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
