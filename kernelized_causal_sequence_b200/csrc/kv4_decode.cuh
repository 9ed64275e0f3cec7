// kv4_decode.cuh — softmax attention of one query token per sequence over the
// 4-bit cache.
//
// One CTA per query head; its warps take every fourth position and keep a
// running maximum, sum and output each, which are joined at the end.  A lane
// holds one 16-bit field of a row (four channels of one group).
#pragma once
#include "kv4_append.cuh"

namespace la {

struct Kv4DecodeParams {
    const void *q;
    Kv4CacheDev c;
    const int32_t *lens;
    const float *weights_in;
    float *weights_out;
    void *out;
    float *scores;       // [B, H, cap] scale log2(e) q.k, where weights are asked for
    float *lse;          // [B, H] log2 of the softmax's denominator
    int H, group;
    float scale_log2;
};

constexpr int kDecWarps = 4;

template <typename InT, typename OutT, int D>
__global__ void __launch_bounds__(kDecWarps * 32) kv4_decode_kernel(Kv4DecodeParams p) {
    constexpr int G = D / kKv4Group;
    __shared__ float sm[kDecWarps], sl[kDecWarps], so[kDecWarps][D];
    pdl_wait();
    const int h = blockIdx.x, b = blockIdx.y, hk = h / p.group;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int r = lane & 7, g = lane >> 3;
    const bool on = g < G;
    const int n = min(max(p.lens[b], 0), p.c.cap);
    const long row0 = ((long)b * p.c.Hkv + hk) * p.c.cap;
    float q[4] = {};
    if (on) {
        const float4 x = load4<InT>((const InT *)p.q + ((long)b * p.H + h) * D + g * kKv4Group + r * 4);
        q[0] = x.x * p.scale_log2; q[1] = x.y * p.scale_log2; q[2] = x.z * p.scale_log2; q[3] = x.w * p.scale_log2;
    }
    float m = -INFINITY, l = 0.f, o[4] = {};
    for (int t = warp; t < n; t += kDecWarps) {
        const long row = row0 + t;
        float s = 0.f, vv[4] = {};
        if (on) {
            const uint32_t kf = *reinterpret_cast<const uint16_t *>(p.c.k_codes + row * (D / 2) + r * 2 * G + 2 * g);
            const uint32_t vf = *reinterpret_cast<const uint16_t *>(p.c.v_codes + row * (D / 2) + r * 2 * G + 2 * g);
            const uint32_t kw = p.c.k_par[row * G + g], vw = p.c.v_par[row * G + g];
            const float ks = kv4_scale(kw), ko = kv4_offset(kw), vs = kv4_scale(vw), vo = kv4_offset(vw);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                s = fmaf(q[i], ks * ((float)((kf >> (4 * i)) & 15) + ko), s);
                vv[i] = vs * ((float)((vf >> (4 * i)) & 15) + vo);
            }
        }
        s = warp_sum(s);
        if (p.weights_out && lane == 0) p.scores[((long)b * p.H + h) * p.c.cap + t] = s;
        const float mn = fmaxf(m, s), f = exp2f(m - mn), e = exp2f(s - mn);
        m = mn;
        l = l * f + e;
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = o[i] * f + e * vv[i];
    }
    if (on)
#pragma unroll
        for (int i = 0; i < 4; ++i) so[warp][g * kKv4Group + r * 4 + i] = o[i];
    if (lane == 0) { sm[warp] = m; sl[warp] = l; }
    __syncthreads();
    float M = -INFINITY, L = 0.f;
    for (int w = 0; w < kDecWarps; ++w) M = fmaxf(M, sm[w]);
    for (int w = 0; w < kDecWarps; ++w) L += sl[w] > 0.f ? sl[w] * exp2f(sm[w] - M) : 0.f;
    for (int c = threadIdx.x; c < D; c += blockDim.x) {
        float a = 0.f;
        for (int w = 0; w < kDecWarps; ++w) a += sl[w] > 0.f ? so[w][c] * exp2f(sm[w] - M) : 0.f;
        ((OutT *)p.out)[((long)b * p.H + h) * D + c] = from_f32<OutT>(n > 0 ? a / L : 0.f);
    }
    if (p.weights_out && threadIdx.x == 0) p.lse[(long)b * p.H + h] = M + log2f(L);
}

// weights_out = weights_in + the group's heads' softmax weights, for t < lens[b]
__global__ void __launch_bounds__(256) kv4_weights_kernel(Kv4DecodeParams p) {
    pdl_wait();
    const int hk = blockIdx.y, b = blockIdx.z;
    const int n = min(max(p.lens[b], 0), p.c.cap);
    const long row0 = ((long)b * p.c.Hkv + hk) * p.c.cap;
    for (int t = blockIdx.x * 256 + threadIdx.x; t < n; t += gridDim.x * 256) {
        float w = p.weights_in ? p.weights_in[row0 + t] : 0.f;
        float sum = 0.f;
        for (int i = 0; i < p.group; ++i) {
            const long h = (long)b * p.H + hk * p.group + i;
            sum += exp2f(p.scores[h * p.c.cap + t] - p.lse[h]);
        }
        p.weights_out[row0 + t] = w + sum;
    }
}

}  // namespace la
