// softmax_simt.cuh — causal softmax attention over packed sequences on the
// CUDA cores, for fp32 inputs (whose 1e-4 class the 16-bit tensor-core operands
// cannot meet).
//
// One CTA takes BM queries of one head (64, or 16 where 64 would leave half of
// the SMs without work) and walks the keys up to its last query in tiles of 64, keeping
// for each row the running maximum m, the sum l and the unnormalised output o
// (all fp32):
//   m' = max(m, max_j s_j),  l' = l 2^(m - m') + sum_j 2^(s_j - m'),
//   o' = o 2^(m - m') + sum_j 2^(s_j - m') v_j,   s_j = scale log2(e) q.k_j.
// 256 threads as 16 x 16; a thread owns BM/16 rows x 4 keys of the scores and
// BM/16 rows x D/16 channels of the output.  The next tile's keys and values
// travel to registers while a tile is computed.  Bound by latency for short prompts
// (four of up to 64 tokens, 8 heads, d 64: 8.3 us with BM 16, 12.4 with 64).
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
template <int D, int BM> constexpr size_t softmax_simt_smem() {
    return sizeof(float) * (D * (BM + 4) + D * kSsPad + kSsTile * D + kSsTile * (BM + 4));
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

template <int N> __device__ __forceinline__ void lds_rows(const float *p, float (&x)[N]) {
    if constexpr (N == 4) {
        const float4 v = *reinterpret_cast<const float4 *>(p);
        x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
    } else {
        x[0] = p[0];
    }
}

template <int D, int BM>
__global__ void __launch_bounds__(kSsThreads) softmax_simt_kernel(SoftmaxParams p) {
    constexpr int CT = D / 16;                           // output channels per thread
    constexpr int RW = BM / 16;                          // rows per thread
    constexpr int QP = BM + 4;                           // row pitch of the channel-major queries and of P
    constexpr int NL = kSsTile * (D / 4) / kSsThreads;   // 4-channel pieces of a tile per thread
    extern __shared__ __align__(16) float ss_smem[];
    float *qs = ss_smem;                   // [D][QP]
    float *ks = qs + D * QP;               // [D][kSsPad]
    float *vs = ks + D * kSsPad;           // [64][D]
    float *ps = vs + kSsTile * D;          // [64 keys][QP]
    pdl_wait();
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x < 2) p.status[threadIdx.x] = 0;
    const SeqTile t = seq_tile<BM>(p.cu, p.n_seq, p.N, blockIdx.x);
    if (t.q0 >= t.end) return;
    const int h = blockIdx.y, hk = h / p.group;
    const float *Q = (const float *)p.q + h * p.q_hs;
    const float *K = (const float *)p.k + hk * p.k_hs;
    const float *V = (const float *)p.v + hk * p.v_hs;
    const int tid = threadIdx.x, ty = tid / 16, tx = tid % 16;
    // keys: thread = row (conflict-free transposed stores); values: thread = piece of a row
    float4 kr[NL], vr[NL];
    auto load = [&](int j0) {
#pragma unroll
        for (int i = 0; i < NL; ++i) {
            const int kj = j0 + tid % kSsTile, kc = (tid / kSsTile + i * (kSsThreads / kSsTile)) * 4;
            const int x = tid + i * kSsThreads, vj = j0 + x / (D / 4), vc = (x % (D / 4)) * 4;
            kr[i] = vr[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (kj < t.end) kr[i] = load4<float>(K + (long)kj * p.k_ts + kc);
            if (vj < t.end) vr[i] = load4<float>(V + (long)vj * p.v_ts + vc);
        }
    };
    load(t.begin);
    for (int x = tid; x < BM * (D / 4); x += kSsThreads) {
        const int r = x % BM, c = (x / BM) * 4;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (t.q0 + r < t.end) v = load4<float>(Q + (long)(t.q0 + r) * p.q_ts + c);
        qs[(c + 0) * QP + r] = v.x;
        qs[(c + 1) * QP + r] = v.y;
        qs[(c + 2) * QP + r] = v.z;
        qs[(c + 3) * QP + r] = v.w;
    }
    float m[RW], l[RW], o[RW][CT];
#pragma unroll
    for (int i = 0; i < RW; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.f;
#pragma unroll
        for (int c = 0; c < CT; ++c) o[i][c] = 0.f;
    }
    const int last = min(t.q0 + BM, t.end);   // keys [begin, last)
    for (int j0 = t.begin; j0 < last; j0 += kSsTile) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < NL; ++i) {
            const int r = tid % kSsTile, kc = (tid / kSsTile + i * (kSsThreads / kSsTile)) * 4, x = tid + i * kSsThreads;
            ks[(kc + 0) * kSsPad + r] = kr[i].x;
            ks[(kc + 1) * kSsPad + r] = kr[i].y;
            ks[(kc + 2) * kSsPad + r] = kr[i].z;
            ks[(kc + 3) * kSsPad + r] = kr[i].w;
            *reinterpret_cast<float4 *>(vs + x * 4) = vr[i];
        }
        __syncthreads();
        if (j0 + kSsTile < last) load(j0 + kSsTile);
        float s[RW][4] = {};
#pragma unroll 8
        for (int c = 0; c < D; ++c) {
            float a[RW], b[4];
            lds_rows(qs + c * QP + ty * RW, a);
            lds_rows(ks + c * kSsPad + tx * 4, b);
#pragma unroll
            for (int i = 0; i < RW; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) s[i][j] = fmaf(a[i], b[j], s[i][j]);
        }
        const bool diag = j0 + kSsTile > t.q0 + 1;   // some key of the tile may be hidden
#pragma unroll
        for (int i = 0; i < RW; ++i) {
            const int row = t.q0 + ty * RW + i;
            float mx = -INFINITY;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                s[i][j] *= p.scale_log2;
                // hidden keys; a row past the sequence's end sees the keys that there are
                if (diag && (j0 + tx * 4 + j > row || j0 + tx * 4 + j >= t.end)) s[i][j] = -INFINITY;
                mx = fmaxf(mx, s[i][j]);
            }
#pragma unroll
            for (int off = 8; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
            const float mn = fmaxf(m[i], mx);
            const float ref = mn == -INFINITY ? 0.f : mn;   // -inf: nothing yet but scores of -inf, whose weights are 0
            const float f = exp2f(m[i] - ref);
            m[i] = mn;
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                s[i][j] = exp2f(s[i][j] - ref);
                sum += s[i][j];
                ps[(tx * 4 + j) * QP + ty * RW + i] = s[i][j];
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
                float a[RW];
                lds_rows(ps + j * QP + ty * RW, a);
#pragma unroll
                for (int c = 0; c < CT; ++c) {
                    const float b = vs[j * D + tx + c * 16];
#pragma unroll
                    for (int i = 0; i < RW; ++i) o[i][c] = fmaf(a[i], b, o[i][c]);
                }
            }
        } else {
            // a hidden key's value is left out, not multiplied by 0: it may be NaN or infinite
#pragma unroll 4
            for (int j = 0; j < n; ++j) {
                float a[RW];
                lds_rows(ps + j * QP + ty * RW, a);
                const int row = j0 + j - t.q0 - ty * RW;   // first row of this thread's that sees key j
#pragma unroll
                for (int c = 0; c < CT; ++c) {
                    const float b = vs[j * D + tx + c * 16];
#pragma unroll
                    for (int i = 0; i < RW; ++i)
                        if (i >= row) o[i][c] = fmaf(a[i], b, o[i][c]);
                }
            }
        }
    }
#pragma unroll
    for (int i = 0; i < RW; ++i)
#pragma unroll
        for (int off = 8; off > 0; off >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], off);
#pragma unroll
    for (int i = 0; i < RW; ++i) {
        const int r = t.q0 + ty * RW + i;
        if (r < t.end) {
            float *dst = (float *)p.out + h * p.o_hs + (long)r * p.o_ts + tx;
            const float inv = 1.f / l[i];
#pragma unroll
            for (int c = 0; c < CT; ++c) dst[c * 16] = o[i][c] * inv;
        }
    }
}

}  // namespace la
