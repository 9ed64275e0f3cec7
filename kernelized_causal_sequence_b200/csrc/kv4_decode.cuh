// kv4_decode.cuh — softmax attention of one query token per sequence over the
// 4-bit cache, tensor cores (mma.sync) on codes that are never expanded in
// memory.
//
// The cache's bytes are the work: 5 bits per channel and position, each used
// for 2 products per query head.  With the products on the FMA units a group
// of 4 query heads would need 16 instructions per byte, five times what the
// SM issues while its share of the bandwidth delivers one; as m16n8k16
// products with the (up to 8) query heads as the n side it is the unpacking of
// the codes that counts.
//
// Numbers.  A code c enters the products as the fp16 number c - 8: masked into
// the mantissa of 1024, where it counts 1 or, from the upper half of a byte,
// 16, and brought to c - 8 by one fp16 multiply-add, exactly (three integer
// and two half instructions for four codes; the integer pipe, half as wide as
// the others, is what a decode kernel of this kind runs against).  With scale
// s and offset o of a (position, group):
//   q.k    = sum_groups s (sum q (c - 8) + (o + 8) sum q)
//   out    = sum_t p s (c - 8) + sum_t p s (o + 8)
// s and o enter in fp32, on the scores and on p.  Queries are scaled by a power
// of two per head that brings the largest to [2^10, 2^11): 16-bit ones are then
// one fp16 term (bf16: exact down to 2^-35 of the largest), fp32 ones two
// (2^-23 of the largest).  p s is scaled by a power of two, so that fp16 holds
// it whatever the values' magnitude (at most 2^15), and rounded once (16-bit
// queries; 2^-11 of itself) or carried as two terms (fp32); the second sum uses the
// same rounded number.  Products down to 2^-26 of the largest scale (p = 1 at the
// reference) are normal numbers, smaller ones a multiple of 2^-36 of it.  (Held
// 2^6 lower, with a reference moved at 2^8, a position of value 0 with 2^24 of the
// others' weights left those 2^-7 of themselves off.)  With fp32 queries
// tensor-core sums run over one tile of 32 positions only and are joined in
// fp32: the tensor core cuts its sums off instead of rounding, 2^-24 of them
// each time, which over a long cache would be seen at fp32's precision.
//
// A warp takes tiles of 32 positions through a ring of its own in shared
// memory, filled by cp.async.  Each lane first turns one position's parameter
// words into fp32 (so that it happens once, not in every lane that meets the
// row).  The first product's result has positions as rows and heads as
// columns; movmatrix transposes it (fp32 in two halves), and from there on a
// thread has one head and the positions that it must supply as the second
// product's k index: the softmax and p s are formed in that layout.  Rows are
// assigned to positions so that the value loads of a phase fall into both
// halves of the banks (row_pos).  Each warp keeps its own reference maximum per
// head, moved only when exceeded by 2^kDecLazy (as in the prompt kernel).
//
// Work is dealt out by the lengths, which only the device knows: the tiles of
// all rows (a sequence's key/value head, and block of query heads) lie on one
// line that is cut into equal pieces, one per resident CTA (DecLine).  A CTA
// walks its piece row by row, its warps take turns at the tiles and join at
// the row's end; a row cut between CTAs is joined by kv4_finish_kernel.
// Short caches are dealt out by whole rows instead and need no second kernel
// (kDecWhole).
//
// What bounds it.  64 sequences of up to 8192 positions, 16 heads on 4, d 128,
// bf16: 55 us for 168 MB (26 us at the copy rate); the integer pipe is 54% busy
// and the SM issues 2.5 of 4 instructions a cycle, about 1000 per tile of 32
// positions, of which the unpacking of the codes alone is a third.
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
    float2 *part_ml;     // [2 n_cta, 8 NT] reference maximum (log2) and sum of a CTA's first and last row, where cut
    float *part_o;       // [2 n_cta, 8 NT, D] their unnormalised outputs
    float2 *row_ml;      // [B, H] the same of rows that one CTA has whole, where weights are asked for
    int H, group, n_cta;
    int whole;           // one CTA per row
    int head_blocks, head_block;   // blocks of query heads of a key/value head, heads in one
    float scale_log2;
};

constexpr int kDecWarps = 4, kDecTile = 32, kDecStages = 2;
constexpr float kDecLazy = 2.f;     // (8 was no faster: 64 rows x 4, lengths to 8192, 64.3 us for 64.5)
constexpr int kDecCtas = 3;         // CTAs per SM with up to 8 query heads (more: 2)
constexpr int kDecMinTiles = 16;    // places of a CTA at least: three or four tiles a warp, to hide its start
constexpr int kDecRowCost = 8;      // tiles' worth of time (of four warps) that a row's start and join take
                                    // (64 rows x 4, lengths to 8192: 0 66.9 us, 4 64.5, 8 63.9, 12 64.0)
// Positions (of the cache: the lengths are on the device) up to which a row is not cut: always, and where there is a
// row for every SM.  us whole / cut, all rows full (lengths spread evenly), weights in the first two lines:
//   4 rows, d 128, bf16      700: 16 / 18 (10 / 18), 1024: 18 / 18 (16 / 20), 1300: 25 / 18 (12 / 16)
//   120 rows, d 128, fp16    700: 20 / 25 (18 / 23), 1024: 27 / 27 (20 / 25), 1300: 31 / 29 (27 / 25)
//   4 rows, d 128, bf16      2048: 25 / 18 (18 / 18), 4096: 41 / 18 (27 / 18)
//   256 rows, d 64, fp16     1024: 16 / 22 (16 / 20), 2048: 25 / 29 (20 / 23), 4096: 39 / 43 (31 / 25)
//   256 rows, d 128, bf16    1024: 23 / 33 (23 / 29), 2048: 37 / 45 (31 / 34), 4096: 62 / 66 (51 / 43)
constexpr int kDecWhole = 1024, kDecWholeFull = 2048;

// Row i of a 16-row tile holds this position of it: odd pairs are swapped, so
// that rows 0, 2, 4, 6 (one value load of a warp) alternate between even and
// odd positions, whose rows start in different halves of the banks at d 128.
__device__ __forceinline__ int row_pos(int i) { return i ^ ((i >> 1) & 1); }

__device__ __forceinline__ uint32_t movmatrix(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
template <int BYTES> __device__ __forceinline__ void cp_async(uint32_t dst, const void *src) {
    if constexpr (BYTES == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
    else asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(BYTES) : "memory");
}
template <int BYTES> __device__ __forceinline__ void cp_async_or_zero(uint32_t dst, const void *src, bool ok) {
    const int n = ok ? BYTES : 0;
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(BYTES), "r"(n) : "memory");
}

__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ float2 unpack_h2(uint32_t u) { return __half22float2(*reinterpret_cast<const __half2 *>(&u)); }
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// W (1, 2 or 4) consecutive words of shared memory, aligned to their size.
template <int W> __device__ __forceinline__ void lds_words(const void *src, float (&w)[W]) {
    if constexpr (W == 4) {
        const float4 x = *reinterpret_cast<const float4 *>(src);
        w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
    } else if constexpr (W == 2) {
        const float2 x = *reinterpret_cast<const float2 *>(src);
        w[0] = x.x; w[1] = x.y;
    } else {
        w[0] = *reinterpret_cast<const float *>(src);
    }
}
template <int W> __device__ __forceinline__ void sts_words(void *dst, const float (&w)[W]) {
    if constexpr (W == 4) *reinterpret_cast<float4 *>(dst) = make_float4(w[0], w[1], w[2], w[3]);
    else if constexpr (W == 2) *reinterpret_cast<float2 *>(dst) = make_float2(w[0], w[1]);
    else *reinterpret_cast<float *>(dst) = w[0];
}
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

// The product alone (no sum before it).
__device__ __forceinline__ void mma_f16_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
                 : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// The numbers c - 8 of the four codes of both 16-bit fields of w (n[i]: code i of both).
__device__ __forceinline__ void code_numbers(uint32_t w, uint32_t (&n)[4]) {
    constexpr uint32_t B = 0x64006400u;   // 1024
    const uint32_t h = w >> 8;
    n[0] = (w & 0x000F000Fu) | B;         // 1024 + c
    n[1] = (w & 0x00F000F0u) | B;         // 1024 + 16 c
    n[2] = (h & 0x000F000Fu) | B;
    n[3] = (h & 0x00F000F0u) | B;
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
        asm("add.rn.f16x2 %0, %0, %1;" : "+r"(n[i]) : "r"(0xE408E408u));                              // - 1032
        asm("fma.rn.f16x2 %0, %0, %1, %2;" : "+r"(n[i + 1]) : "r"(0x2C002C00u), "r"(0xD480D480u));    // / 16 - 72
    }
}

template <int D> struct DecCfg {
    static constexpr int G = D / kKv4Group;
    // a ring stage: codes of 32 keys, of 32 values, their parameter words
    static constexpr int OFF_V = kDecTile * D / 2, OFF_KP = 2 * OFF_V, OFF_VP = OFF_KP + kDecTile * G * 4;
    static constexpr int STAGE = OFF_VP + kDecTile * G * 4;
    // a tile's parameters in fp32, [kind][position][group]: the keys' scale and offset + 8, the values' scale / unit
    // and (offset + 8) unit, where `unit` is the tile's power of two
    static constexpr int KIND = kDecTile * G * 4, PAR = 4 * KIND;
    static constexpr int WARP = kDecStages * STAGE + PAR;
};
template <int D> constexpr size_t kv4_decode_smem(int nt) {
    const size_t ring = (size_t)kDecWarps * DecCfg<D>::WARP;
    const size_t join = (size_t)kDecWarps * 8 * nt * (D + 2) * sizeof(float) + 8 * nt * sizeof(float);
    return ring > join ? ring : join;
}

// The line: a row takes as many places as it has tiles, and kDecRowCost more for
// its start and join; sequence b begins at rows_per_seq * (places of a row of
// each sequence before it).
struct DecLine {
    int rows;    // rows of a sequence
    int chunk;   // places of a CTA
    long total;
};
__device__ __forceinline__ int dec_len(const int32_t *lens, int b, int cap) { return min(max(lens[b], 0), cap); }
__device__ __forceinline__ int dec_tiles(int n) { return (n + kDecTile - 1) / kDecTile; }
__device__ __forceinline__ int dec_places(int n) { return n > 0 ? dec_tiles(n) + kDecRowCost : 0; }

// Places of a row of each of the sequences [0, b); whole warp.
__device__ __forceinline__ long dec_places_before(const Kv4DecodeParams &p, int b) {
    long sum = 0;
    for (int i = threadIdx.x & 31; i < b; i += 32) sum += dec_places(dec_len(p.lens, i, p.c.cap));
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    return sum;
}
__device__ __forceinline__ DecLine dec_line(const Kv4DecodeParams &p) {
    DecLine d;
    d.rows = p.c.Hkv * p.head_blocks;
    d.total = dec_places_before(p, p.c.B) * d.rows;
    const long c = (d.total + p.n_cta - 1) / p.n_cta;
    d.chunk = (int)max(c, (long)kDecMinTiles);
    return d;
}
// The sequence that holds place `at` < total of the line, and the places of a row of those before it; whole warp.
__device__ __forceinline__ int dec_find(const Kv4DecodeParams &p, const DecLine &d, long at, long *before) {
    const int lane = threadIdx.x & 31;
    long sum = 0;
    for (int b0 = 0;; b0 += 32) {
        const int nt = b0 + lane < p.c.B ? dec_places(dec_len(p.lens, b0 + lane, p.c.cap)) : 0;
        long x = nt;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const long y = __shfl_up_sync(0xffffffffu, x, off);
            if (lane >= off) x += y;
        }
        const uint32_t past = __ballot_sync(0xffffffffu, (sum + x) * d.rows > at);
        if (past || b0 + 32 >= p.c.B) {
            const int l = past ? __ffs(past) - 1 : 31;
            *before = sum + __shfl_sync(0xffffffffu, x - nt, l);
            return min(b0 + l, p.c.B - 1);
        }
        sum += __shfl_sync(0xffffffffu, x, 31);
    }
}

// One row's tiles [tile0, tile0 + count) by one CTA; `slot`: where its partial result goes, -1 if it is the whole row.
template <typename InT, typename OutT, int D, int NT>
__device__ __forceinline__ void decode_row(const Kv4DecodeParams &p, uint8_t *dec_smem, int b, int row, int n, int tile0,
                                           int count, int slot) {
    using C = DecCfg<D>;
    constexpr int G = C::G, HB = 8 * NT;
    constexpr int QT = std::is_same<InT, float>::value ? 2 : 1;   // terms of a query
    constexpr int PT = QT;                                        // terms of p s
    constexpr bool TILE_SUMS = PT > 1;                            // tensor-core sums over one tile only
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int r = lane >> 2, cq = lane & 3;
    const int hk = row / p.head_blocks, hb = row % p.head_blocks;
    const int t_begin = tile0 * kDecTile, t_end = min(t_begin + count * kDecTile, n);
    const int heads = min(p.group - hb * HB, HB);                 // of this row
    const long h0 = (long)b * p.H + (long)hk * p.group + hb * HB;  // its first query head's row
    const long row0 = ((long)b * p.c.Hkv + hk) * p.c.cap;
    const int n_tiles = count;

    uint8_t *ring = dec_smem + warp * C::WARP;
    uint8_t *par = ring + kDecStages * C::STAGE;
    const uint8_t *gk = p.c.k_codes + (row0 + t_begin) * (D / 2) + lane * 16, *gv = p.c.v_codes + (row0 + t_begin) * (D / 2) + lane * 16;
    const uint32_t *gkp = p.c.k_par + (row0 + t_begin + lane) * G, *gvp = p.c.v_par + (row0 + t_begin + lane) * G;
    auto load = [&](int tile, int stage) {
        const uint32_t dst = tc::smem_u32(ring + stage * C::STAGE);
        const int left = t_end - t_begin - tile * kDecTile;   // positions from the tile's first on
        constexpr int CPR = D / 32;                           // 16-byte pieces of a row's codes
        const uint8_t *k = gk + (long)tile * (kDecTile * D / 2), *v = gv + (long)tile * (kDecTile * D / 2);
        const uint32_t *kp = gkp + (long)tile * (kDecTile * G), *vp = gvp + (long)tile * (kDecTile * G);
        if (left >= kDecTile) {
#pragma unroll
            for (int i = 0; i < CPR; ++i) {
                cp_async<16>(dst + (lane + 32 * i) * 16, k + i * 512);
                cp_async<16>(dst + C::OFF_V + (lane + 32 * i) * 16, v + i * 512);
            }
            cp_async<4 * G>(dst + C::OFF_KP + lane * 4 * G, kp);
            cp_async<4 * G>(dst + C::OFF_VP + lane * 4 * G, vp);
        } else {
            // behind the end: zeros (with the tile's first row's address, which is not read)
#pragma unroll
            for (int i = 0; i < CPR; ++i) {
                const bool ok = (lane + 32 * i) / CPR < left;
                cp_async_or_zero<16>(dst + (lane + 32 * i) * 16, ok ? k + i * 512 : k - lane * 16, ok);
                cp_async_or_zero<16>(dst + C::OFF_V + (lane + 32 * i) * 16, ok ? v + i * 512 : v - lane * 16, ok);
            }
            const bool ok = lane < left;
            cp_async_or_zero<4 * G>(dst + C::OFF_KP + lane * 4 * G, ok ? kp : kp - lane * G, ok);
            cp_async_or_zero<4 * G>(dst + C::OFF_VP + lane * 4 * G, ok ? vp : vp - lane * G, ok);
        }
    };
#pragma unroll
    for (int i = 0; i < kDecStages - 1; ++i) {
        if (warp + i * kDecWarps < n_tiles) load(warp + i * kDecWarps, i);
        asm volatile("cp.async.commit_group;" ::: "memory");
    }

    // queries as the n side: column r of a group's two products is head r, the
    // k slots of thread cq are the channel pairs (i, i + 4) of chunks 2 cq and 2 cq + 1
    uint32_t qf[NT][QT][G][4];
    float qsum[NT][G][2];   // sum of a group's (scaled) channels for heads 2 cq, 2 cq + 1 (the scores' columns)
    float qe[NT];           // head r: scale log2(e) over the power of two
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const bool ok = nt * 8 + r < heads;
        const InT *qp = (const InT *)p.q + (h0 + (ok ? nt * 8 + r : 0)) * D;
        float x[G][8], big = 0.f;
#pragma unroll
        for (int g = 0; g < G; ++g) {
            float4 u = make_float4(0.f, 0.f, 0.f, 0.f), v = u;
            if (ok) {
                u = load4<InT>(qp + g * kKv4Group + cq * 8);
                v = load4<InT>(qp + g * kKv4Group + cq * 8 + 4);
            }
            x[g][0] = u.x; x[g][1] = u.y; x[g][2] = u.z; x[g][3] = u.w;
            x[g][4] = v.x; x[g][5] = v.y; x[g][6] = v.z; x[g][7] = v.w;
#pragma unroll
            for (int i = 0; i < 8; ++i) big = fmaxf(big, fabsf(x[g][i]));
        }
        big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
        big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
        const uint32_t e = max(__float_as_uint(big) >> 23, 11u);   // biased exponent
        const float up = __uint_as_float((264u - e) << 23);        // 2^(10 - exponent)
        qe[nt] = __uint_as_float((e - 10u) << 23) * p.scale_log2;
#pragma unroll
        for (int g = 0; g < G; ++g) {
            float s = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                x[g][i] *= up;
                s += x[g][i];
            }
            s += __shfl_xor_sync(0xffffffffu, s, 1);
            s += __shfl_xor_sync(0xffffffffu, s, 2);
            qsum[nt][g][0] = __shfl_sync(0xffffffffu, s, 8 * cq);       // head 2 cq sits in lanes 4 (2 cq) ..
            qsum[nt][g][1] = __shfl_sync(0xffffffffu, s, 8 * cq + 4);
#pragma unroll
            for (int t = 0; t < QT; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t u = pack_h2(x[g][i], x[g][i + 4]);
                    qf[nt][t][g][i] = u;
                    const float2 f = unpack_h2(u);
                    x[g][i] -= f.x;
                    x[g][i + 4] -= f.y;
                }
        }
    }

    float o[NT][2 * G][4];    // rows r, r + 8 = channels 32 g + 4 r + 2 h, + 1; columns = heads 2 cq, 2 cq + 1
    float ob[NT][G];          // head r: sum of p s (o + 8) over this thread's positions
    float m[NT], mm[NT];      // head r: the reference; 0 while that is -inf
    float l[NT];              // head r: sum of p over this thread's positions
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        m[nt] = -INFINITY;
        mm[nt] = 0.f;
        l[nt] = 0.f;
#pragma unroll
        for (int i = 0; i < 2 * G; ++i) o[nt][i][0] = o[nt][i][1] = o[nt][i][2] = o[nt][i][3] = 0.f;
#pragma unroll
        for (int g = 0; g < G; ++g) ob[nt][g] = 0.f;
    }
    // warp-wide: the power of two in which p s is held, and the scale's bits from which it is too small
    float unit = 0.f, per_unit = 0.f;
    uint32_t unit_end = 0u;
    int stage = 0;
#pragma unroll 1
    for (int tile = warp; tile < n_tiles; tile += kDecWarps) {
        const int ahead = tile + (kDecStages - 1) * kDecWarps;
        if (ahead < n_tiles) load(ahead, stage == 0 ? kDecStages - 1 : stage - 1);
        asm volatile("cp.async.commit_group;" ::: "memory");
        asm volatile("cp.async.wait_group %0;" ::"n"(kDecStages - 1) : "memory");
        __syncwarp();
        const uint8_t *st = ring + stage * C::STAGE;
        stage = stage == kDecStages - 1 ? 0 : stage + 1;
        const int t0 = t_begin + tile * kDecTile;
        // ---- parameters: this lane's position
        {
            uint32_t kw[G], vw[G];
            lds_words(st + C::OFF_KP + lane * 4 * G, kw);
            lds_words(st + C::OFF_VP + lane * 4 * G, vw);
            uint32_t big = 0u;
#pragma unroll
            for (int g = 0; g < G; ++g) {
                const uint32_t bits = vw[g] << 16;
                if (bits < 0x7f800000u) big = max(big, bits);   // (a group of NaN is its own: it sets no unit)
            }
            // The unit grows with the largest scale met (in [2^e, 2^(e + 1)): p s < 2^kDecLazy 2^(e + 1) = 2^15 unit);
            // one-term queries sum their products in it from tile to tile.
            if (TILE_SUMS || __any_sync(0xffffffffu, big >= unit_end)) {
                const uint32_t e = max(__reduce_max_sync(0xffffffffu, big) >> 23, 13u);
                const float old = unit;
                unit = __uint_as_float((e - 12u) << 23);
                per_unit = __uint_as_float((266u - e) << 23);
                unit_end = (e + 1u) << 23;
                if (!TILE_SUMS && old > 0.f) {
                    const float f = old / unit;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int k = 0; k < 2 * G; ++k)
#pragma unroll
                            for (int i = 0; i < 4; ++i) o[nt][k][i] *= f;
                }
            }
            float x[4][G];
#pragma unroll
            for (int g = 0; g < G; ++g) {
                x[0][g] = kv4_scale(kw[g]);
                x[1][g] = kv4_offset(kw[g]) + 8.f;
                x[2][g] = kv4_scale(vw[g]) * per_unit;
                x[3][g] = (kv4_offset(vw[g]) + 8.f) * unit;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) sts_words(par + i * C::KIND + lane * G * 4, x[i]);
        }
        __syncwarp();
        float s[2][NT][4];    // head r; positions of rows 2 cq, 2 cq + 1, 2 cq + 8, 2 cq + 9
        // ---- scores of two 16-position tiles
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int ra = half * 16 + row_pos(r), rb = ra + 8;
            uint32_t ka[G], kb[G];   // code words (chunks 2 cq | 2 cq + 1) of the two rows
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
            }
            float sa[G], sb[G], oa[G], ob_[G];
            lds_words(par + ra * G * 4, sa);
            lds_words(par + rb * G * 4, sb);
            lds_words(par + C::KIND + ra * G * 4, oa);
            lds_words(par + C::KIND + rb * G * 4, ob_);
            float sc[NT][4];
#pragma unroll
            for (int g = 0; g < G; ++g) {
                uint32_t na[4], nb[4];
                code_numbers(ka[g], na);
                code_numbers(kb[g], nb);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float d[4] = {oa[g] * qsum[nt][g][0], oa[g] * qsum[nt][g][1], ob_[g] * qsum[nt][g][0], ob_[g] * qsum[nt][g][1]};
#pragma unroll
                    for (int t = 0; t < QT; ++t) {
                        mma_f16(d, na[0], nb[0], na[1], nb[1], qf[nt][t][g][0], qf[nt][t][g][1]);
                        mma_f16(d, na[2], nb[2], na[3], nb[3], qf[nt][t][g][2], qf[nt][t][g][3]);
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        sc[nt][i] = g == 0 ? (i < 2 ? sa[g] : sb[g]) * d[i] : fmaf(i < 2 ? sa[g] : sb[g], d[i], sc[nt][i]);
                }
            }
            // transpose: rows become heads (fp32 as two 16-bit halves)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const float u = sc[nt][2 * x], v = sc[nt][2 * x + 1];
                    const uint32_t lo = movmatrix(__byte_perm(__float_as_uint(u), __float_as_uint(v), 0x5410));
                    const uint32_t hi = movmatrix(__byte_perm(__float_as_uint(u), __float_as_uint(v), 0x7632));
                    s[half][nt][2 * x] = __uint_as_float(__byte_perm(lo, hi, 0x5410)) * qe[nt];
                    s[half][nt][2 * x + 1] = __uint_as_float(__byte_perm(lo, hi, 0x7632)) * qe[nt];
                }
        }
        // position of s[half][nt][i]: t0 + 16 half + 8 (i >> 1) + row_pos(2 cq + (i & 1))
        if (t0 + kDecTile > t_end) {
#pragma unroll
            for (int half = 0; half < 2; ++half)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (t0 + half * 16 + 8 * (i >> 1) + row_pos(2 * cq + (i & 1)) >= t_end)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) s[half][nt][i] = -INFINITY;
        }
        if (p.scores) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
                if (nt * 8 + r < heads) {
                    float *dst = p.scores + (h0 + nt * 8 + r) * p.c.cap + t0;
#pragma unroll
                    for (int half = 0; half < 2; ++half)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int t = half * 16 + 8 * (i >> 1) + row_pos(2 * cq + (i & 1));
                            if (t0 + t < t_end) dst[t] = s[half][nt][i];
                        }
                }
        }
        // ---- reference maximum, moved rarely
        float mx[NT];
        bool move = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            mx[nt] = fmaxf(fmaxf(fmaxf(s[0][nt][0], s[0][nt][1]), fmaxf(s[0][nt][2], s[0][nt][3])),
                           fmaxf(fmaxf(s[1][nt][0], s[1][nt][1]), fmaxf(s[1][nt][2], s[1][nt][3])));
            move |= mx[nt] > m[nt] + kDecLazy;
        }
        if (__any_sync(0xffffffffu, move)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float x = fmaxf(m[nt], mx[nt]);
                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
                // (x = -inf: nothing yet but -inf scores)
                const float f = x == -INFINITY ? 1.f : ex2_approx(m[nt] - x);
                m[nt] = x;
                mm[nt] = x == -INFINITY ? 0.f : x;
                l[nt] *= f;
#pragma unroll
                for (int g = 0; g < G; ++g) ob[nt][g] *= f;
                const float f0 = __shfl_sync(0xffffffffu, f, 8 * cq), f1 = __shfl_sync(0xffffffffu, f, 8 * cq + 4);
#pragma unroll
                for (int k = 0; k < 2 * G; ++k) {
                    o[nt][k][0] *= f0;
                    o[nt][k][1] *= f1;
                    o[nt][k][2] *= f0;
                    o[nt][k][3] *= f1;
                }
            }
        }
        // ---- p, both halves
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
#pragma unroll
                for (int i = 0; i < 4; ++i) s[half][nt][i] = ex2_approx(s[half][nt][i] - mm[nt]);
                l[nt] += (s[half][nt][0] + s[half][nt][1]) + (s[half][nt][2] + s[half][nt][3]);
            }
        // ---- values: chunk r of positions (rows) 2 cq, 2 cq + 1 and 8 more
        uint32_t wl[2][G], wh[2][G];   // field g of both positions, rows below and above 8
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int va = half * 16 + row_pos(2 * cq), vb = half * 16 + row_pos(2 * cq + 1);
            const uint8_t *vs = st + C::OFF_V + r * (D / 16);
            if constexpr (G == 1) {
                auto f = [&](int i) { return (uint32_t)*reinterpret_cast<const uint16_t *>(vs + i * (D / 2)); };
                wl[half][0] = f(va) | (f(vb) << 16);
                wh[half][0] = f(va + 8) | (f(vb + 8) << 16);
            } else {
                constexpr int W = G / 2;
                uint32_t a[W], c[W], e[W], f[W];
                lds_words(vs + va * (D / 2), a);
                lds_words(vs + vb * (D / 2), c);
                lds_words(vs + (va + 8) * (D / 2), e);
                lds_words(vs + (vb + 8) * (D / 2), f);
#pragma unroll
                for (int i = 0; i < W; ++i) {
                    wl[half][2 * i] = __byte_perm(a[i], c[i], 0x5410);
                    wl[half][2 * i + 1] = __byte_perm(a[i], c[i], 0x7632);
                    wh[half][2 * i] = __byte_perm(e[i], f[i], 0x5410);
                    wh[half][2 * i + 1] = __byte_perm(e[i], f[i], 0x7632);
                }
            }
        }
        float tile_sums[TILE_SUMS ? NT : 1][TILE_SUMS ? 2 * G : 1][4];
        auto &ot = [&]() -> auto & {
            if constexpr (TILE_SUMS) return tile_sums;
            else return o;
        }();
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            float vs[4][G], vo[4][G];   // scale / unit, (offset + 8) unit of rows 2 cq, 2 cq + 1, 2 cq + 8, 2 cq + 9
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int at = half * 16 + 8 * (i >> 1) + row_pos(2 * cq + (i & 1));
                lds_words(par + 2 * C::KIND + at * G * 4, vs[i]);
                lds_words(par + 3 * C::KIND + at * G * 4, vo[i]);
            }
#pragma unroll
            for (int g = 0; g < G; ++g) {
                uint32_t nl[4], nh[4];
                code_numbers(wl[half][g], nl);
                code_numbers(wh[half][g], nh);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float x[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) x[i] = s[half][nt][i] * vs[i][g];
#pragma unroll
                    for (int t = 0; t < PT; ++t) {
                        const uint32_t b0 = pack_h2(x[0], x[1]), b1 = pack_h2(x[2], x[3]);
                        const float2 u = unpack_h2(b0), w = unpack_h2(b1);
                        ob[nt][g] = fmaf(u.x, vo[0][g], fmaf(u.y, vo[1][g], fmaf(w.x, vo[2][g], fmaf(w.y, vo[3][g], ob[nt][g]))));
                        if (t + 1 < PT) { x[0] -= u.x; x[1] -= u.y; x[2] -= w.x; x[3] -= w.y; }
                        if (TILE_SUMS && half == 0 && t == 0) {
                            mma_f16_first(ot[nt][2 * g], nl[0], nl[1], nh[0], nh[1], b0, b1);
                            mma_f16_first(ot[nt][2 * g + 1], nl[2], nl[3], nh[2], nh[3], b0, b1);
                        } else {
                            mma_f16(ot[nt][2 * g], nl[0], nl[1], nh[0], nh[1], b0, b1);
                            mma_f16(ot[nt][2 * g + 1], nl[2], nl[3], nh[2], nh[3], b0, b1);
                        }
                    }
                }
            }
        }
        if constexpr (TILE_SUMS) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int k = 0; k < 2 * G; ++k)
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[nt][k][i] = fmaf(ot[nt][k][i], unit, o[nt][k][i]);
        }
        __syncwarp();   // the tile has been read: the next turn's loads and parameters overwrite it
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();    // the rings are done: their memory joins the warps

    if constexpr (!TILE_SUMS) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int k = 0; k < 2 * G; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[nt][k][i] *= unit;
    }
    // ---- join the warps: [warp][head][D], then [warp][head] (m, l)
    float *jo = reinterpret_cast<float *>(dec_smem);
    float2 *jml = reinterpret_cast<float2 *>(jo + kDecWarps * HB * D);
    float *jlse = reinterpret_cast<float *>(jml + kDecWarps * HB);   // [head]
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        float bs[G], ls = l[nt];
        ls += __shfl_xor_sync(0xffffffffu, ls, 1);
        ls += __shfl_xor_sync(0xffffffffu, ls, 2);
        if (cq == 0) jml[warp * HB + nt * 8 + r] = make_float2(m[nt], ls);
#pragma unroll
        for (int g = 0; g < G; ++g) {
            bs[g] = ob[nt][g];
            bs[g] += __shfl_xor_sync(0xffffffffu, bs[g], 1);
            bs[g] += __shfl_xor_sync(0xffffffffu, bs[g], 2);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int g = 0; g < G; ++g) {
                const float add = __shfl_sync(0xffffffffu, bs[g], 8 * cq + 4 * i);   // of head 2 cq + i
                *reinterpret_cast<float4 *>(jo + (warp * HB + nt * 8 + 2 * cq + i) * D + g * kKv4Group + 4 * r) =
                    make_float4(o[nt][2 * g][i] + add, o[nt][2 * g][i + 2] + add, o[nt][2 * g + 1][i] + add,
                                o[nt][2 * g + 1][i + 2] + add);
            }
    }
    __syncthreads();
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
        if (slot < 0) {
            const float inv = 1.f / L;
            store4<OutT>((OutT *)p.out + (h0 + col) * D + c4 * 4, a.x * inv, a.y * inv, a.z * inv, a.w * inv);
            if (p.row_ml && c4 == 0) {
                p.row_ml[h0 + col] = make_float2(M_, L);
                jlse[col] = M_ + log2f(L);
            }
        } else {
            *reinterpret_cast<float4 *>(p.part_o + ((long)slot * HB + col) * D + c4 * 4) = a;
            if (c4 == 0) p.part_ml[slot * HB + col] = make_float2(M_, L);
        }
    }
    __syncthreads();   // the next row's rings take this memory again
    // weights where this CTA has the whole group's row (else: kv4_finish_kernel)
    if (p.weights_out && p.whole && p.head_blocks == 1) {
        for (int t = threadIdx.x; t < n; t += kDecWarps * 32) {
            float sum = 0.f;
            for (int i = 0; i < heads; ++i) sum += ex2_approx(p.scores[(h0 + i) * p.c.cap + t] - jlse[i]);
            p.weights_out[row0 + t] = (p.weights_in ? p.weights_in[row0 + t] : 0.f) + sum;
        }
    }
}

template <typename InT, typename OutT, int D, int NT>
__global__ void __launch_bounds__(kDecWarps * 32, NT == 1 && !std::is_same<InT, float>::value ? kDecCtas : 2)
kv4_decode_kernel(const Kv4DecodeParams p) {
    extern __shared__ __align__(16) uint8_t dec_smem[];
    pdl_wait();
    // sequences without a position: zeros
    for (int b = blockIdx.x; b < p.c.B; b += gridDim.x)
        if (dec_len(p.lens, b, p.c.cap) == 0)
            for (long x = threadIdx.x; x < (long)p.H * D; x += kDecWarps * 32)
                ((OutT *)p.out)[(long)b * p.H * D + x] = from_f32<OutT>(0.f);
    const int rows = p.c.Hkv * p.head_blocks;
    if (p.whole) {
        const int b = blockIdx.x / rows, n = dec_len(p.lens, b, p.c.cap);
        if (n > 0) decode_row<InT, OutT, D, NT>(p, dec_smem, b, blockIdx.x % rows, n, 0, dec_tiles(n), -1);
        return;
    }
    const DecLine d = dec_line(p);
    long at = (long)blockIdx.x * d.chunk;
    const long begin = at, end = min(at + d.chunk, d.total);
    if (at >= end) return;
    long before;
    int b = dec_find(p, d, at, &before);
    int n = dec_len(p.lens, b, p.c.cap), nt = dec_tiles(n);
    const long off = at - before * rows;
    int row = (int)(off / dec_places(n)), tile = (int)(off % dec_places(n));
    while (true) {
        if (tile >= nt) {   // the next row
            at += nt + kDecRowCost - tile;
            if (at >= end) return;
            tile = 0;
            if (++row == rows) {
                row = 0;
                do { n = dec_len(p.lens, ++b, p.c.cap); } while (n == 0);   // (at < total: there is one)
                nt = dec_tiles(n);
            }
        }
        const int count = (int)min((long)(nt - tile), end - at);
        // a cut row: the first of this CTA if it began before, else the last
        const int slot = count == nt ? -1 : 2 * blockIdx.x + (at == begin ? 0 : 1);
        decode_row<InT, OutT, D, NT>(p, dec_smem, b, row, n, tile, count, slot);
        at += count;
        tile += count;
        if (at >= end) return;
    }
}

// Joins the rows that are cut between CTAs, and forms the weights.  Blocks
// x < out_blocks of a (key/value head, sequence): outputs; the others: weights.
constexpr int kFinThreads = 256;

// The pieces of a row that begins at place `start` of the line: the CTAs first
// .. last that have tiles of it; slot of a CTA's piece.
struct DecPieces {
    int first, last;
    long start;
    int chunk;
    __device__ int slot(int cta) const { return 2 * cta + (start <= (long)cta * chunk ? 0 : 1); }
};

template <typename OutT, int D>
__global__ void __launch_bounds__(kFinThreads) kv4_finish_kernel(const Kv4DecodeParams p, int out_blocks) {
    pdl_wait();
    const int hk = blockIdx.y, b = blockIdx.z;
    const int n = dec_len(p.lens, b, p.c.cap), nt = dec_tiles(n);
    const int HB = p.head_block;
    const long h0 = (long)b * p.H + (long)hk * p.group;
    DecLine d{0, 1, 0};
    long before = 0;
    if (!p.whole) {
        d = dec_line(p);
        before = dec_places_before(p, b);
    }
    if (n == 0) return;
    auto pieces = [&](int head) {   // of the row that holds the query head
        DecPieces x{0, 0, 0, d.chunk};
        if (!p.whole) {
            x.start = before * d.rows + (long)(hk * p.head_blocks + head / HB) * (nt + kDecRowCost);
            x.first = (int)(x.start / d.chunk);
            x.last = (int)((x.start + nt - 1) / d.chunk);
        }
        return x;
    };
    // log2 of a row's denominator, and its greatest reference; the pieces over a warp's lanes
    auto join = [&](const DecPieces &x, int head, float *top) {
        const int lane = threadIdx.x & 31;
        float M_ = -INFINITY, L = 0.f;
        for (int c = x.first + lane; c <= x.last; c += 32) {
            const float2 ml = p.part_ml[x.slot(c) * HB + head % HB];
            const float M2 = fmaxf(M_, ml.x);
            if (M2 > -INFINITY) L = L * ex2_approx(M_ - M2) + ml.y * ex2_approx(ml.x - M2);
            else L += ml.y;
            M_ = M2;
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) {
            const float m2 = __shfl_xor_sync(0xffffffffu, M_, off), l2 = __shfl_xor_sync(0xffffffffu, L, off);
            const float M2 = fmaxf(M_, m2);
            if (M2 > -INFINITY) L = L * ex2_approx(M_ - M2) + l2 * ex2_approx(m2 - M2);
            else L += l2;
            M_ = M2;
        }
        *top = M_;
        return L;
    };
    __shared__ float lse[kFinThreads];
    __shared__ float part[kFinThreads * 4];
    if ((int)blockIdx.x < out_blocks) {
        // one head per block: its pieces over the threads' rows, each thread four channels
        constexpr int TPH = D / 4, ROWS = kFinThreads / TPH;
        const int i = blockIdx.x, c4 = threadIdx.x % TPH, k = threadIdx.x / TPH;
        const DecPieces x = pieces(i);
        if (x.first == x.last) return;
        float M_;
        const float L = join(x, i, &M_);
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int c = x.first + k; c <= x.last; c += ROWS) {
            const long at = (long)x.slot(c) * HB + i % HB;
            const float f = M_ == -INFINITY ? 1.f : ex2_approx(p.part_ml[at].x - M_);
            const float4 v = *reinterpret_cast<const float4 *>(p.part_o + at * D + c4 * 4);
            a.x = fmaf(v.x, f, a.x); a.y = fmaf(v.y, f, a.y); a.z = fmaf(v.z, f, a.z); a.w = fmaf(v.w, f, a.w);
        }
        reinterpret_cast<float4 *>(part)[threadIdx.x] = a;
        __syncthreads();
        if (k == 0) {
#pragma unroll
            for (int y = 1; y < ROWS; ++y) {
                const float4 v = reinterpret_cast<const float4 *>(part)[y * TPH + c4];
                a.x += v.x; a.y += v.y; a.z += v.z; a.w += v.w;
            }
            const float inv = 1.f / L;
            store4<OutT>((OutT *)p.out + (h0 + i) * D + c4 * 4, a.x * inv, a.y * inv, a.z * inv, a.w * inv);
        }
        return;
    }
    // weights_out[t] = weights_in[t] + sum over the group's heads of 2^(score - lse)
    const long row0 = ((long)b * p.c.Hkv + hk) * p.c.cap;
    const int wb = blockIdx.x - out_blocks, nwb = gridDim.x - out_blocks;
    for (int i0 = 0; i0 < p.group; i0 += kFinThreads) {
        __syncthreads();
        const int gi = min(kFinThreads, p.group - i0);
        for (int i = threadIdx.x / 32; i < gi; i += kFinThreads / 32) {
            const DecPieces x = pieces(i0 + i);
            float M_, L;
            if (x.first == x.last) {
                const float2 ml = p.row_ml[h0 + i0 + i];
                M_ = ml.x;
                L = ml.y;
            } else {
                L = join(x, i0 + i, &M_);
            }
            if ((threadIdx.x & 31) == 0) lse[i] = M_ + log2f(L);
        }
        __syncthreads();
        // four positions a thread where the rows are aligned for it
        const bool four = (p.c.cap & 3) == 0;
        const int per = four ? 4 : 1;
        for (int t = (wb * kFinThreads + threadIdx.x) * per; t < n; t += nwb * kFinThreads * per) {
            const float *from = i0 > 0 ? p.weights_out : p.weights_in;
            if (four && t + 4 <= n) {
                float4 w = from ? *reinterpret_cast<const float4 *>(from + row0 + t) : make_float4(0.f, 0.f, 0.f, 0.f);
                float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
                for (int i = 0; i < gi; ++i) {
                    const float4 s = *reinterpret_cast<const float4 *>(p.scores + (h0 + i0 + i) * p.c.cap + t);
                    sum.x += ex2_approx(s.x - lse[i]); sum.y += ex2_approx(s.y - lse[i]);
                    sum.z += ex2_approx(s.z - lse[i]); sum.w += ex2_approx(s.w - lse[i]);
                }
                *reinterpret_cast<float4 *>(p.weights_out + row0 + t) =
                    make_float4(w.x + sum.x, w.y + sum.y, w.z + sum.z, w.w + sum.w);
            } else {
                for (int u = t; u < min(t + per, n); ++u) {
                    float sum = 0.f;
                    for (int i = 0; i < gi; ++i) sum += ex2_approx(p.scores[(h0 + i0 + i) * p.c.cap + u] - lse[i]);
                    p.weights_out[row0 + u] = (from ? from[row0 + u] : 0.f) + sum;
                }
            }
        }
    }
}

}  // namespace la
