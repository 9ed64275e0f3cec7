// kv4_decode.cuh — softmax attention of one query token per sequence over the
// 4-bit cache, tensor cores (mma.sync) on codes that are never expanded in
// memory.
//
// The cache's bytes are the work: 5 bits per channel and position, each used
// for 2 products per query head.  With the products on the FMA units a group
// of 4 query heads would need 16 instructions per byte, five times what the
// SM issues while its share of the bandwidth delivers one; as m16n8k16
// products with the (up to 8) query heads as the n side it is mostly the
// unpacking of the codes that counts, one shift and one mask for two of them.
//
// A code c becomes the 16-bit number 16 + c by masking it into the mantissa of
// 16.  With scale s and offset o of a (position, group):
//   q.k    = sum_groups s (sum q (16 + c) + (o - 16) sum q)
//   out    = sum_t p s (16 + c) + sum_t p s (o - 16)
// The products take plain numbers 16 + c; s and o enter in fp32 on the scores
// (rows = positions) and on p.  p s is rounded once to the 16-bit type and the
// same rounded number is used in both sums of `out`, so the 16 cancels exactly
// and the rounding counts relative to the value itself.  fp32 queries are
// three bf16 terms and p s two.
//
// A warp takes tiles of 32 positions.  Scores come out with positions as rows;
// the second product needs them as its k index, which movmatrix provides.
// Rows are assigned to positions so that the value loads of a phase fall into
// both halves of the banks (row_pos).  Each warp keeps its own reference
// maximum per head, moved only when exceeded by 2^8 (as in the prompt kernel),
// and its own ring of tiles in shared memory filled by cp.async; the warps of
// a CTA join at the end, CTAs of a long sequence in kv4_finish_kernel.
#pragma once
#include <type_traits>

#include "kv4_append.cuh"
#include "tc_ptx.cuh"

namespace la {

struct Kv4DecodeParams {
    const void *q;
    Kv4CacheDev c;
    const int32_t *lens;
    const float *weights_in;
    float *weights_out;
    void *out;
    float *scores;       // [B, H, cap] scale log2(e) q.k, where weights are asked for
    float2 *part_ml;     // [B, H, n_split] reference maximum (log2), sum; null if no other kernel needs them
    float *part_o;       // [B, H, n_split, D] unnormalised outputs, where n_split > 1
    int H, group, n_split, split_len;
    int head_blocks;     // CTAs over the query heads of a key/value head
    float scale_log2;
};

constexpr int kDecWarps = 4, kDecTile = 32, kDecStages = 3;
constexpr float kDecLazy = 8.f;

// Row i of a 16-row tile holds this position of it: odd pairs are swapped, so
// that rows 0, 2, 4, 6 (one value load of a warp) alternate between even and
// odd positions, whose rows start in different halves of the banks at d 128.
__device__ __forceinline__ int row_pos(int i) { return i ^ ((i >> 1) & 1); }

__device__ __forceinline__ uint32_t movmatrix(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
template <int BYTES> __device__ __forceinline__ void cp_async(void *dst, const void *src, bool ok) {
    const int n = ok ? BYTES : 0;   // 0: zeros
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(tc::smem_u32(dst)), "l"(src), "r"(n) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(tc::smem_u32(dst)), "l"(src), "n"(BYTES), "r"(n) : "memory");
}

// Number types of the products.
template <typename T> struct Mma16;
template <> struct Mma16<bf16> {
    static constexpr uint32_t BASE = 0x41804180u, MASK = 0x00780078u;   // 16; the mantissa bits worth 1 .. 8
    static constexpr int SH = 3;                                        // where those bits begin
    static __device__ __forceinline__ uint32_t pack(float lo, float hi) { return tc::pack_bf16x2(lo, hi); }
    static __device__ __forceinline__ float lo(uint32_t u) { return __uint_as_float(u << 16); }
    static __device__ __forceinline__ float hi(uint32_t u) { return __uint_as_float(u & 0xFFFF0000u); }
    static __device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1) {
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    }
};
template <> struct Mma16<f16> {
    static constexpr uint32_t BASE = 0x4C004C00u, MASK = 0x03C003C0u;
    static constexpr int SH = 6;
    static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
        const __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
    static __device__ __forceinline__ float lo(uint32_t u) { return __low2float(*reinterpret_cast<const __half2 *>(&u)); }
    static __device__ __forceinline__ float hi(uint32_t u) { return __high2float(*reinterpret_cast<const __half2 *>(&u)); }
    static __device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1) {
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    }
};

// W (1, 2 or 4) consecutive words of shared memory, aligned to their size.
template <int W> __device__ __forceinline__ void lds_words(const void *src, uint32_t (&w)[W]) {
    if constexpr (W == 4) {
        const uint4 x = *reinterpret_cast<const uint4 *>(src);
        w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
    } else if constexpr (W == 2) {
        const uint2 x = *reinterpret_cast<const uint2 *>(src);
        w[0] = x.x; w[1] = x.y;
    } else {
        w[0] = *reinterpret_cast<const uint32_t *>(src);
    }
}

// The numbers 16 + c of nibble I of both halves of w.
template <typename M, int I> __device__ __forceinline__ uint32_t code_pair(uint32_t w) {
    constexpr int sh = M::SH - 4 * I;
    const uint32_t x = sh >= 0 ? w << (sh & 31) : w >> ((-sh) & 31);
    return (x & M::MASK) | M::BASE;
}

template <int D> struct DecCfg {
    static constexpr int G = D / kKv4Group;
    static constexpr int OFF_V = kDecTile * D / 2, OFF_KP = 2 * OFF_V, OFF_VP = OFF_KP + kDecTile * G * 4;
    static constexpr int STAGE = OFF_VP + kDecTile * G * 4;
};
template <int D> constexpr size_t kv4_decode_smem(int nt) {
    const size_t ring = (size_t)kDecWarps * kDecStages * DecCfg<D>::STAGE;
    const size_t join = (size_t)kDecWarps * 8 * nt * (D + 4) * sizeof(float);
    return ring > join ? ring : join;
}

template <typename InT, typename OutT, int D, int NT>
__global__ void __launch_bounds__(kDecWarps * 32) kv4_decode_kernel(const Kv4DecodeParams p) {
    using C = DecCfg<D>;
    using MT = typename std::conditional<std::is_same<InT, f16>::value, f16, bf16>::type;
    using M = Mma16<MT>;
    constexpr int G = C::G, HB = 8 * NT;
    constexpr int QT = std::is_same<InT, float>::value ? 3 : 1;   // terms of a query
    constexpr int PT = std::is_same<InT, float>::value ? 2 : 1;   // terms of p s
    extern __shared__ __align__(16) uint8_t dec_smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int r = lane >> 2, cq = lane & 3;
    const int split = blockIdx.x, hk = blockIdx.y / p.head_blocks, hb = blockIdx.y % p.head_blocks, b = blockIdx.z;
    pdl_wait();
    const int n = min(max(p.lens[b], 0), p.c.cap);
    const int t_begin = min(split * p.split_len, n), t_end = min(t_begin + p.split_len, n);
    // (split 0 of an empty sequence writes its zeros)
    if (t_begin >= t_end && split > 0) return;
    const int heads = min(p.group - hb * HB, HB);                 // of this CTA
    const long h0 = (long)b * p.H + (long)hk * p.group + hb * HB;  // its first query head's row
    const long row0 = ((long)b * p.c.Hkv + hk) * p.c.cap;

    // queries as the n side: column r of a group's two products is head r, the
    // k slots of thread cq are the channel pairs (i, i + 4) of chunks 2 cq and 2 cq + 1
    uint32_t qf[NT][QT][G][4];
    float qsum[NT][G][2];   // sum of a group's channels for heads 2 cq, 2 cq + 1 (the scores' columns)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const bool ok = nt * 8 + r < heads;
        const InT *qp = (const InT *)p.q + (h0 + (ok ? nt * 8 + r : 0)) * D;
#pragma unroll
        for (int g = 0; g < G; ++g) {
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
            if (ok) {
                x = load4<InT>(qp + g * kKv4Group + cq * 8);
                y = load4<InT>(qp + g * kKv4Group + cq * 8 + 4);
            }
            float lo[4] = {x.x, x.y, x.z, x.w}, hi[4] = {y.x, y.y, y.z, y.w};
            float s = ((x.x + x.y) + (x.z + x.w)) + ((y.x + y.y) + (y.z + y.w));
            s += __shfl_xor_sync(0xffffffffu, s, 1);
            s += __shfl_xor_sync(0xffffffffu, s, 2);
            qsum[nt][g][0] = __shfl_sync(0xffffffffu, s, 8 * cq);       // head 2 cq sits in lanes 4 (2 cq) ..
            qsum[nt][g][1] = __shfl_sync(0xffffffffu, s, 8 * cq + 4);
#pragma unroll
            for (int t = 0; t < QT; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t u = M::pack(lo[i], hi[i]);
                    qf[nt][t][g][i] = u;
                    lo[i] -= M::lo(u);
                    hi[i] -= M::hi(u);
                }
        }
    }

    uint8_t *ring = dec_smem + warp * kDecStages * C::STAGE;
    const int n_tiles = (t_end - t_begin + kDecTile - 1) / kDecTile;
    auto load = [&](int tile, int stage) {
        uint8_t *dst = ring + stage * C::STAGE;
        const int t0 = t_begin + tile * kDecTile;
        constexpr int CPR = D / 32;   // 16-byte pieces of a row's codes
#pragma unroll
        for (int i = 0; i < CPR; ++i) {
            const int x = lane + 32 * i, t = t0 + x / CPR;
            const bool ok = t < t_end;
            const long off = (row0 + (ok ? t : t_begin)) * (D / 2) + (x % CPR) * 16;
            cp_async<16>(dst + x * 16, p.c.k_codes + off, ok);
            cp_async<16>(dst + C::OFF_V + x * 16, p.c.v_codes + off, ok);
        }
        const bool ok = t0 + lane < t_end;
        const long off = (row0 + (ok ? t0 + lane : t_begin)) * G;
        cp_async<4 * G>(dst + C::OFF_KP + lane * 4 * G, p.c.k_par + off, ok);
        cp_async<4 * G>(dst + C::OFF_VP + lane * 4 * G, p.c.v_par + off, ok);
    };

    float o[NT][2 * G][4];    // rows r, r + 8 = channels 32 g + 4 r + 2 h, + 1; columns = heads 2 cq, 2 cq + 1
    float ob[NT][G][2];       // sum of p s (o - 16) over this thread's positions
    float m[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        m[nt][0] = m[nt][1] = -INFINITY;
        l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
        for (int i = 0; i < 2 * G; ++i) o[nt][i][0] = o[nt][i][1] = o[nt][i][2] = o[nt][i][3] = 0.f;
#pragma unroll
        for (int g = 0; g < G; ++g) ob[nt][g][0] = ob[nt][g][1] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < kDecStages - 1; ++i) {
        if (warp + i * kDecWarps < n_tiles) load(warp + i * kDecWarps, i);
        asm volatile("cp.async.commit_group;" ::: "memory");
    }
    int stage = 0;
    for (int tile = warp; tile < n_tiles; tile += kDecWarps) {
        const int ahead = tile + (kDecStages - 1) * kDecWarps;
        if (ahead < n_tiles) load(ahead, stage == 0 ? kDecStages - 1 : stage - 1);
        asm volatile("cp.async.commit_group;" ::: "memory");
        asm volatile("cp.async.wait_group %0;" ::"n"(kDecStages - 1) : "memory");
        __syncwarp();
        const uint8_t *st = ring + stage * C::STAGE;
        stage = stage == kDecStages - 1 ? 0 : stage + 1;
        const int t0 = t_begin + tile * kDecTile;
        float s[2][NT][4];
        // ---- scores of two 16-position tiles
#pragma unroll
        for (int half = 0; half < 2; ++half) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) s[half][nt][0] = s[half][nt][1] = s[half][nt][2] = s[half][nt][3] = 0.f;
            const int ra = half * 16 + row_pos(r), rb = ra + 8;
            uint32_t ka[G], kb[G], pa[G], pb[G];   // code words (chunks 2 cq | 2 cq + 1) and parameter words of the two rows
            {
                constexpr int W = D / 32;   // 32-bit words of two chunks
                uint32_t xa[W], xb[W];
                lds_words(st + ra * (D / 2) + cq * (D / 8), xa);
                lds_words(st + rb * (D / 2) + cq * (D / 8), xb);
                if constexpr (G == 1) {
                    ka[0] = xa[0]; kb[0] = xb[0];
                } else {
#pragma unroll
                    for (int g = 0; g < G; ++g) {
                        ka[g] = __byte_perm(xa[g / 2], xa[g / 2 + W / 2], (g & 1) ? 0x7632 : 0x5410);
                        kb[g] = __byte_perm(xb[g / 2], xb[g / 2 + W / 2], (g & 1) ? 0x7632 : 0x5410);
                    }
                }
                lds_words(st + C::OFF_KP + ra * G * 4, pa);
                lds_words(st + C::OFF_KP + rb * G * 4, pb);
            }
#pragma unroll
            for (int g = 0; g < G; ++g) {
                const uint32_t a0 = code_pair<M, 0>(ka[g]), a1 = code_pair<M, 0>(kb[g]), a2 = code_pair<M, 1>(ka[g]),
                               a3 = code_pair<M, 1>(kb[g]);
                const uint32_t c0 = code_pair<M, 2>(ka[g]), c1 = code_pair<M, 2>(kb[g]), c2 = code_pair<M, 3>(ka[g]),
                               c3 = code_pair<M, 3>(kb[g]);
                const float sa = kv4_scale(pa[g]), oa = kv4_offset(pa[g]) - 16.f;
                const float sb = kv4_scale(pb[g]), ob_ = kv4_offset(pb[g]) - 16.f;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float d[4] = {oa * qsum[nt][g][0], oa * qsum[nt][g][1], ob_ * qsum[nt][g][0], ob_ * qsum[nt][g][1]};
#pragma unroll
                    for (int t = 0; t < QT; ++t) {
                        M::mma(d, a0, a1, a2, a3, qf[nt][t][g][0], qf[nt][t][g][1]);
                        M::mma(d, c0, c1, c2, c3, qf[nt][t][g][2], qf[nt][t][g][3]);
                    }
                    s[half][nt][0] = fmaf(sa, d[0], s[half][nt][0]);
                    s[half][nt][1] = fmaf(sa, d[1], s[half][nt][1]);
                    s[half][nt][2] = fmaf(sb, d[2], s[half][nt][2]);
                    s[half][nt][3] = fmaf(sb, d[3], s[half][nt][3]);
                }
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i) s[half][nt][i] *= p.scale_log2;
        }
        if (t0 + kDecTile > t_end) {
#pragma unroll
            for (int half = 0; half < 2; ++half)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    if (t0 + half * 16 + row_pos(r) + 8 * i >= t_end)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) s[half][nt][2 * i] = s[half][nt][2 * i + 1] = -INFINITY;
        }
        if (p.scores) {
#pragma unroll
            for (int half = 0; half < 2; ++half)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int t = t0 + half * 16 + row_pos(r) + 8 * (i >> 1), col = nt * 8 + 2 * cq + (i & 1);
                        if (col < heads && t < t_end) p.scores[(h0 + col) * p.c.cap + t] = s[half][nt][i];
                    }
        }
        // ---- running maximum, moved rarely
        float mx[NT][2];
        bool move = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                mx[nt][i] = fmaxf(fmaxf(s[0][nt][i], s[0][nt][i + 2]), fmaxf(s[1][nt][i], s[1][nt][i + 2]));
                move |= mx[nt][i] > m[nt][i] + kDecLazy;
            }
        if (__any_sync(0xffffffffu, move)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float x = fmaxf(m[nt][i], mx[nt][i]);
#pragma unroll
                    for (int off = 4; off < 32; off <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, off));
                    // (x = -inf: nothing yet but -inf scores)
                    const float f = x == -INFINITY ? 1.f : ex2_approx(m[nt][i] - x);
                    m[nt][i] = x;
                    l[nt][i] *= f;
#pragma unroll
                    for (int k = 0; k < 2 * G; ++k) {
                        o[nt][k][i] *= f;
                        o[nt][k][i + 2] *= f;
                    }
#pragma unroll
                    for (int g = 0; g < G; ++g) ob[nt][g][i] *= f;
                }
        }
#pragma unroll
        for (int half = 0; half < 2; ++half) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float mm = m[nt][i & 1] == -INFINITY ? 0.f : m[nt][i & 1];
                    const float e = ex2_approx(s[half][nt][i] - mm);
                    s[half][nt][i] = e;
                    l[nt][i & 1] += e;
                }
            // ---- p s as the k side of the second product, one set per group
            const int ra = half * 16 + row_pos(r), rb = ra + 8;
            uint32_t bf[NT][PT][G][2], pa[G], pb[G];
            lds_words(st + C::OFF_VP + ra * G * 4, pa);
            lds_words(st + C::OFF_VP + rb * G * 4, pb);
#pragma unroll
            for (int g = 0; g < G; ++g) {
                const float sa = kv4_scale(pa[g]), oa = kv4_offset(pa[g]) - 16.f;
                const float sb = kv4_scale(pb[g]), ob_ = kv4_offset(pb[g]) - 16.f;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float x0 = s[half][nt][0] * sa, x1 = s[half][nt][1] * sa, x2 = s[half][nt][2] * sb, x3 = s[half][nt][3] * sb;
#pragma unroll
                    for (int t = 0; t < PT; ++t) {
                        const uint32_t u = M::pack(x0, x1), w = M::pack(x2, x3);
                        const float u0 = M::lo(u), u1 = M::hi(u), w0 = M::lo(w), w1 = M::hi(w);
                        ob[nt][g][0] = fmaf(w0, ob_, fmaf(u0, oa, ob[nt][g][0]));
                        ob[nt][g][1] = fmaf(w1, ob_, fmaf(u1, oa, ob[nt][g][1]));
                        if (t + 1 < PT) { x0 -= u0; x1 -= u1; x2 -= w0; x3 -= w1; }
                        bf[nt][t][g][0] = movmatrix(u);
                        bf[nt][t][g][1] = movmatrix(w);
                    }
                }
            }
            // ---- values: chunk r of positions (rows) 2 cq, 2 cq + 1 and 8 more
            const int va = half * 16 + row_pos(2 * cq), vb = half * 16 + row_pos(2 * cq + 1);
            const uint8_t *vs = st + C::OFF_V + r * (D / 16);
            uint32_t wl[G], wh[G];   // field g of both positions, rows below and above 8
            if constexpr (G == 1) {
                auto f = [&](int row) { return (uint32_t)*reinterpret_cast<const uint16_t *>(vs + row * (D / 2)); };
                wl[0] = f(va) | (f(vb) << 16);
                wh[0] = f(va + 8) | (f(vb + 8) << 16);
            } else {
                constexpr int W = G / 2;
                uint32_t a[W], c[W], e[W], f[W];
                lds_words(vs + va * (D / 2), a);
                lds_words(vs + vb * (D / 2), c);
                lds_words(vs + (va + 8) * (D / 2), e);
                lds_words(vs + (vb + 8) * (D / 2), f);
#pragma unroll
                for (int i = 0; i < W; ++i) {
                    wl[2 * i] = __byte_perm(a[i], c[i], 0x5410);
                    wl[2 * i + 1] = __byte_perm(a[i], c[i], 0x7632);
                    wh[2 * i] = __byte_perm(e[i], f[i], 0x5410);
                    wh[2 * i + 1] = __byte_perm(e[i], f[i], 0x7632);
                }
            }
#pragma unroll
            for (int g = 0; g < G; ++g) {
                const uint32_t a0 = code_pair<M, 0>(wl[g]), a1 = code_pair<M, 1>(wl[g]), a2 = code_pair<M, 0>(wh[g]),
                               a3 = code_pair<M, 1>(wh[g]);
                const uint32_t c0 = code_pair<M, 2>(wl[g]), c1 = code_pair<M, 3>(wl[g]), c2 = code_pair<M, 2>(wh[g]),
                               c3 = code_pair<M, 3>(wh[g]);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int t = 0; t < PT; ++t) {
                        M::mma(o[nt][2 * g], a0, a1, a2, a3, bf[nt][t][g][0], bf[nt][t][g][1]);
                        M::mma(o[nt][2 * g + 1], c0, c1, c2, c3, bf[nt][t][g][0], bf[nt][t][g][1]);
                    }
            }
        }
        __syncwarp();   // the tile has been read: the next turn's load overwrites it
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();    // the rings are done: their memory joins the warps

    // ---- join the warps: [warp][head][D], then [warp][head] (m, l)
    float *jo = reinterpret_cast<float *>(dec_smem);
    float2 *jml = reinterpret_cast<float2 *>(jo + kDecWarps * HB * D);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) {
                l[nt][i] += __shfl_xor_sync(0xffffffffu, l[nt][i], off);
#pragma unroll
                for (int g = 0; g < G; ++g) ob[nt][g][i] += __shfl_xor_sync(0xffffffffu, ob[nt][g][i], off);
            }
            const int col = nt * 8 + 2 * cq + i;
#pragma unroll
            for (int g = 0; g < G; ++g)
                *reinterpret_cast<float4 *>(jo + (warp * HB + col) * D + g * kKv4Group + 4 * r) =
                    make_float4(o[nt][2 * g][i] + ob[nt][g][i], o[nt][2 * g][i + 2] + ob[nt][g][i],
                                o[nt][2 * g + 1][i] + ob[nt][g][i], o[nt][2 * g + 1][i + 2] + ob[nt][g][i]);
            if (r == 0) jml[warp * HB + col] = make_float2(m[nt][i], l[nt][i]);
        }
    __syncthreads();
    const bool whole = n <= p.split_len;   // this CTA's is the final result
    for (int x = threadIdx.x; x < heads * (D / 4); x += kDecWarps * 32) {
        const int col = x / (D / 4), c4 = x % (D / 4);
        float M_ = -INFINITY, L = 0.f;
#pragma unroll
        for (int w = 0; w < kDecWarps; ++w) M_ = fmaxf(M_, jml[w * HB + col].x);
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kDecWarps; ++w) {
            const float2 ml = jml[w * HB + col];
            if (w >= n_tiles) continue;   // a warp without a tile
            const float f = M_ == -INFINITY ? 1.f : ex2_approx(ml.x - M_);
            const float4 v = *reinterpret_cast<const float4 *>(jo + (w * HB + col) * D + c4 * 4);
            L = fmaf(ml.y, f, L);
            a.x = fmaf(v.x, f, a.x); a.y = fmaf(v.y, f, a.y); a.z = fmaf(v.z, f, a.z); a.w = fmaf(v.w, f, a.w);
        }
        const long h = h0 + col;
        if (p.part_ml && c4 == 0) p.part_ml[h * p.n_split + split] = make_float2(M_, L);
        if (whole) {
            const float inv = n > 0 ? 1.f / L : 0.f;
            store4<OutT>((OutT *)p.out + h * D + c4 * 4, a.x * inv, a.y * inv, a.z * inv, a.w * inv);
        } else {
            *reinterpret_cast<float4 *>(p.part_o + (h * p.n_split + split) * D + c4 * 4) = a;
        }
    }
}

// Joins the splits of sequences longer than one, and forms the weights.
// Blocks x < out_blocks of a (head group, sequence): outputs; the others: weights.
constexpr int kFinThreads = 256;
template <typename OutT, int D>
__global__ void __launch_bounds__(kFinThreads) kv4_finish_kernel(const Kv4DecodeParams p, int out_blocks) {
    pdl_wait();
    const int hk = blockIdx.y, b = blockIdx.z;
    const int n = min(max(p.lens[b], 0), p.c.cap);
    const int ns = (n + p.split_len - 1) / p.split_len;
    const long h0 = (long)b * p.H + (long)hk * p.group;
    if ((int)blockIdx.x < out_blocks) {
        if (n <= p.split_len) return;
        constexpr int TPH = D / 4, HPB = kFinThreads / TPH;   // threads of a head, heads of a block
        const int i = blockIdx.x * HPB + threadIdx.x / TPH, c4 = threadIdx.x % TPH;
        if (i >= p.group) return;
        const float2 *ml = p.part_ml + (h0 + i) * p.n_split;
        const float *po = p.part_o + (h0 + i) * p.n_split * D + c4 * 4;
        float M_ = -INFINITY, L = 0.f;
        for (int s = 0; s < ns; ++s) M_ = fmaxf(M_, ml[s].x);
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int s = 0; s < ns; ++s) {
            const float f = M_ == -INFINITY ? 1.f : ex2_approx(ml[s].x - M_);
            const float4 v = *reinterpret_cast<const float4 *>(po + (long)s * D);
            L = fmaf(ml[s].y, f, L);
            a.x = fmaf(v.x, f, a.x); a.y = fmaf(v.y, f, a.y); a.z = fmaf(v.z, f, a.z); a.w = fmaf(v.w, f, a.w);
        }
        const float inv = 1.f / L;
        store4<OutT>((OutT *)p.out + (h0 + i) * D + c4 * 4, a.x * inv, a.y * inv, a.z * inv, a.w * inv);
        return;
    }
    // weights_out[t] = weights_in[t] + sum over the group's heads of 2^(score - lse)
    __shared__ float lse[kFinThreads];
    const long row0 = ((long)b * p.c.Hkv + hk) * p.c.cap;
    const int wb = blockIdx.x - out_blocks, nwb = gridDim.x - out_blocks;
    for (int i0 = 0; i0 < p.group; i0 += kFinThreads) {
        __syncthreads();
        const int gi = min(kFinThreads, p.group - i0);
        if ((int)threadIdx.x < gi) {
            const float2 *ml = p.part_ml + (h0 + i0 + threadIdx.x) * p.n_split;
            float M_ = -INFINITY, L = 0.f;
            for (int s = 0; s < ns; ++s) M_ = fmaxf(M_, ml[s].x);
            for (int s = 0; s < ns; ++s) L += ml[s].y * (M_ == -INFINITY ? 1.f : ex2_approx(ml[s].x - M_));
            lse[threadIdx.x] = M_ + log2f(L);
        }
        __syncthreads();
        for (int t = wb * kFinThreads + threadIdx.x; t < n; t += nwb * kFinThreads) {
            float w = i0 > 0 ? p.weights_out[row0 + t] : p.weights_in ? p.weights_in[row0 + t] : 0.f;
            float sum = 0.f;
#pragma unroll 4
            for (int i = 0; i < gi; ++i) sum += ex2_approx(p.scores[(h0 + i0 + i) * p.c.cap + t] - lse[i]);
            p.weights_out[row0 + t] = w + sum;
        }
    }
}

}  // namespace la
