// softmax_simt.cuh — causal softmax attention over packed sequences on the
// CUDA cores: fp32 inputs (whose 1e-4 class the 16-bit tensor-core operands
// cannot meet) and head dim 32.
//
// One CTA takes 64 queries of one head and walks the keys up to its last
// query in tiles of 64, keeping for each row the running maximum m, the sum l
// and the unnormalised output o (all fp32):
//   m' = max(m, max_j s_j),  l' = l 2^(m - m') + sum_j 2^(s_j - m'),
//   o' = o 2^(m - m') + sum_j 2^(s_j - m') v_j,   s_j = scale log2(e) q.k_j.
// 256 threads as 16 x 16; a thread owns 4 rows x 4 keys of the scores and
// 4 rows x D/16 channels of the output.
#pragma once
#include "common.cuh"
#include "packed.cuh"

namespace la {

struct SoftmaxParams {
    const void *q, *k, *v;
    void *out;
    const int32_t *cu;
    long q_hs, q_ts, k_hs, k_ts, v_hs, v_ts, o_hs, o_ts;   // strides in elements
    int H, group, N, n_seq;                                // group = H / H_kv
    float scale_log2;                                      // scale * log2(e)
    int *status;                                           // the workspace's status word (no wait here can give up)
};

constexpr int kSsTile = 64, kSsThreads = 256, kSsPad = kSsTile + 4;
template <int D> constexpr size_t softmax_simt_smem() {
    return sizeof(float) * (2 * D * kSsPad + kSsTile * D + kSsTile * kSsPad);
}

template <typename T> __device__ __forceinline__ float4 load4(const T *p);
template <> __device__ __forceinline__ float4 load4<float>(const float *p) { return *reinterpret_cast<const float4 *>(p); }
template <> __device__ __forceinline__ float4 load4<bf16>(const bf16 *p) {
    const uint2 u = *reinterpret_cast<const uint2 *>(p);
    return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xFFFF0000u), __uint_as_float(u.y << 16),
                       __uint_as_float(u.y & 0xFFFF0000u));
}
template <> __device__ __forceinline__ float4 load4<f16>(const f16 *p) {
    const uint2 u = *reinterpret_cast<const uint2 *>(p);
    const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&u.x));
    const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&u.y));
    return make_float4(a.x, a.y, b.x, b.y);
}
template <typename T> __device__ __forceinline__ void store4(T *p, float a, float b, float c, float d) {
    p[0] = from_f32<T>(a); p[1] = from_f32<T>(b); p[2] = from_f32<T>(c); p[3] = from_f32<T>(d);
}
template <> __device__ __forceinline__ void store4<float>(float *p, float a, float b, float c, float d) {
    *reinterpret_cast<float4 *>(p) = make_float4(a, b, c, d);
}

// rows [r0, r0 + 64) of a [T][D] matrix to shared memory, rows at or past end as zeros;
// TRANS: [D][kSsPad] (channel-major), else [64][D]
template <typename T, int D, bool TRANS>
__device__ __forceinline__ void load_tile(float *dst, const T *src, long ts, int r0, int end) {
    for (int i = threadIdx.x; i < kSsTile * (D / 4); i += kSsThreads) {
        const int r = i / (D / 4), c = (i % (D / 4)) * 4;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r0 + r < end) x = load4<T>(src + (long)(r0 + r) * ts + c);
        if (TRANS) {
            dst[(c + 0) * kSsPad + r] = x.x;
            dst[(c + 1) * kSsPad + r] = x.y;
            dst[(c + 2) * kSsPad + r] = x.z;
            dst[(c + 3) * kSsPad + r] = x.w;
        } else {
            *reinterpret_cast<float4 *>(dst + r * D + c) = x;
        }
    }
}

template <typename InT, typename OutT, int D>
__global__ void __launch_bounds__(kSsThreads) softmax_simt_kernel(SoftmaxParams p) {
    constexpr int CT = D / 16;   // output channels per thread
    extern __shared__ __align__(16) float ss_smem[];
    float *qs = ss_smem;                   // [D][kSsPad]
    float *ks = qs + D * kSsPad;           // [D][kSsPad]
    float *vs = ks + D * kSsPad;           // [64][D]
    float *ps = vs + kSsTile * D;          // [64 keys][kSsPad]
    pdl_wait();
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x < 2) p.status[threadIdx.x] = 0;
    const SeqTile t = seq_tile<kSsTile>(p.cu, p.n_seq, p.N, blockIdx.x);
    if (t.q0 >= t.end) return;
    const int h = blockIdx.y, hk = h / p.group;
    const InT *Q = (const InT *)p.q + h * p.q_hs;
    const InT *K = (const InT *)p.k + hk * p.k_hs;
    const InT *V = (const InT *)p.v + hk * p.v_hs;
    const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
    load_tile<InT, D, true>(qs, Q, p.q_ts, t.q0, t.end);
    float m[4], l[4], o[4][CT];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.f;
#pragma unroll
        for (int c = 0; c < CT; ++c) o[i][c] = 0.f;
    }
    const int last = min(t.q0 + kSsTile, t.end);   // keys [begin, last)
    for (int j0 = t.begin; j0 < last; j0 += kSsTile) {
        __syncthreads();
        load_tile<InT, D, true>(ks, K, p.k_ts, j0, t.end);
        load_tile<InT, D, false>(vs, V, p.v_ts, j0, t.end);
        __syncthreads();
        float s[4][4] = {};
#pragma unroll 8
        for (int c = 0; c < D; ++c) {
            const float4 a4 = *reinterpret_cast<const float4 *>(qs + c * kSsPad + ty * 4);
            const float4 b4 = *reinterpret_cast<const float4 *>(ks + c * kSsPad + tx * 4);
            const float a[4] = {a4.x, a4.y, a4.z, a4.w}, b[4] = {b4.x, b4.y, b4.z, b4.w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) s[i][j] = fmaf(a[i], b[j], s[i][j]);
        }
        const bool diag = j0 + kSsTile > t.q0 + 1;   // some key of the tile may be hidden
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float mx = -INFINITY;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                s[i][j] *= p.scale_log2;
                // hidden keys; a row past the sequence's end sees the keys that there are
                if (diag && (j0 + tx * 4 + j > t.q0 + ty * 4 + i || j0 + tx * 4 + j >= t.end)) s[i][j] = -INFINITY;
                mx = fmaxf(mx, s[i][j]);
            }
#pragma unroll
            for (int off = 8; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
            const float mn = fmaxf(m[i], mx);
            const float f = exp2f(m[i] - mn);
            m[i] = mn;
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                s[i][j] = exp2f(s[i][j] - mn);
                sum += s[i][j];
                ps[(tx * 4 + j) * kSsPad + ty * 4 + i] = s[i][j];
            }
            l[i] = l[i] * f + sum;   // this thread's four key columns; joined at the end
#pragma unroll
            for (int c = 0; c < CT; ++c) o[i][c] *= f;
        }
        __syncthreads();
        const int n = min(kSsTile, t.end - j0);
        if (!diag) {
#pragma unroll 4
            for (int j = 0; j < kSsTile; ++j) {
                const float4 a4 = *reinterpret_cast<const float4 *>(ps + j * kSsPad + ty * 4);
                const float a[4] = {a4.x, a4.y, a4.z, a4.w};
#pragma unroll
                for (int c = 0; c < CT; ++c) {
                    const float b = vs[j * D + tx + c * 16];
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[i][c] = fmaf(a[i], b, o[i][c]);
                }
            }
        } else {
            // a hidden key's value is left out, not multiplied by 0: it may be NaN or infinite
            for (int j = 0; j < n; ++j) {
                const float4 a4 = *reinterpret_cast<const float4 *>(ps + j * kSsPad + ty * 4);
                const float a[4] = {a4.x, a4.y, a4.z, a4.w};
                const int row = j0 + j - t.q0 - ty * 4;   // first row of this thread's that sees key j
#pragma unroll
                for (int c = 0; c < CT; ++c) {
                    const float b = vs[j * D + tx + c * 16];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (i >= row) o[i][c] = fmaf(a[i], b, o[i][c]);
                }
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int off = 8; off > 0; off >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], off);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = t.q0 + ty * 4 + i;
        if (r < t.end) {
            OutT *dst = (OutT *)p.out + h * p.o_hs + (long)r * p.o_ts + tx;
            const float inv = 1.f / l[i];
#pragma unroll
            for (int c = 0; c < CT; ++c) dst[c * 16] = from_f32<OutT>(o[i][c] * inv);
        }
    }
}

}  // namespace la
