// kv4_append.cuh — writing tokens into the 4-bit cache and reading them back.
//
// Eight threads per row (a token of one head, keys or values): thread r holds
// channels 4 r .. 4 r + 3 of every group, which are the row's chunk r, so its
// codes are one store of D / 16 bytes, and a group's minimum, maximum and
// largest magnitude take three shuffles.  Each input is read once and each
// cache byte written once.  Appending is bound by instruction issue (9.2k tokens
// x 8 heads, d 128, bf16: 25 us, over 450 instructions per warp and 4 rows at an
// IPC of 3; the bytes alone would be 14 us): exact rounding of scale, offset and code costs
// them, in fp32 with fp64 only where a quotient is near a border (58 us in fp64
// throughout).  Several rows per warp one after the other were slower, as their
// loads then wait for each other.  Reading back is bound by memory (the same rows
// 18 us, 16 x 8 x 2048 of them 54 us, 85% of the copy rate).
#pragma once
#include "kv4_format.cuh"
#include "packed.cuh"
#include "softmax_simt.cuh"

namespace la {

struct Kv4CacheDev {
    uint8_t *k_codes;
    uint32_t *k_par;
    uint8_t *v_codes;
    uint32_t *v_par;
    int B, Hkv, cap;
};

struct Kv4AppendParams {
    const void *k, *v;
    long k_hs, k_ts, v_hs, v_ts;
    const int32_t *cu;      // or null: token t is sequence t's only one
    const int32_t *start;
    Kv4CacheDev c;
    int N;
    void *k_out, *v_out;    // kv4_read
    int per;                // kv4_read: tokens of a warp
};

constexpr int kAppendThreads = 256;

// The cache row of token t, or -1 if it has none.
__device__ __forceinline__ long kv4_row(const Kv4AppendParams &p, int t, int head) {
    int s = t, i = 0;
    if (p.cu) {
        s = seq_of_token(p.cu, p.c.B, p.N, t);
        const int b = seq_start(p.cu, s, p.N);
        i = t - b;
        if (i < 0 || t >= seq_start(p.cu, s + 1, p.N)) return -1;   // of no sequence
    }
    const long pos = (long)p.start[s] + i;
    if (pos < 0 || pos >= p.c.cap) return -1;
    return ((long)s * p.c.Hkv + head) * p.c.cap + pos;
}

// The same for the four tokens of a warp (lane l: token t of its eight lanes), of at most 32 sequences: lane s holds
// sequence s's tokens and start, and a ballot over them finds a token's sequence.  Whole warp; t0 the first token.
// (12 sequences, 9.2k tokens x 8 heads, append and read: 44.5 us, by bisection in each lane, a chain of loads, 46.2.)
__device__ __forceinline__ long kv4_row_of_few(const Kv4AppendParams &p, int t0, int head) {
    const int lane = threadIdx.x & 31, B = p.c.B;
    int begin = 0, end = 0, start = 0;
    if (lane < B) {
        begin = seq_start(p.cu, lane, p.N);
        end = seq_start(p.cu, lane + 1, p.N);
        start = p.start[lane];
    }
    uint32_t at = 0u;   // sequences that begin at or before the token
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t x = __ballot_sync(0xffffffffu, lane < B && begin <= t0 + j);
        if (lane >> 3 == j) at = x;
    }
    const int s = at ? 31 - __clz(at) : 0, t = t0 + (lane >> 3);
    const int i = t - __shfl_sync(0xffffffffu, begin, s);
    end = __shfl_sync(0xffffffffu, end, s);
    const long pos = (long)__shfl_sync(0xffffffffu, start, s) + i;
    if (i < 0 || t >= end || pos < 0 || pos >= p.c.cap) return -1;
    return ((long)s * p.c.Hkv + head) * p.c.cap + pos;
}

template <int D> struct Kv4Chunk;   // a chunk: one 16-bit field per group
template <> struct Kv4Chunk<32> { using type = uint16_t; };
template <> struct Kv4Chunk<64> { using type = uint32_t; };
template <> struct Kv4Chunk<128> { using type = uint64_t; };

template <typename InT, int D>
__global__ void __launch_bounds__(kAppendThreads) kv4_append_kernel(Kv4AppendParams p) {
    constexpr int G = D / kKv4Group;
    using Chunk = typename Kv4Chunk<D>::type;
    pdl_wait();
    const int r = threadIdx.x & 7, head = blockIdx.y;
    const bool keys = blockIdx.z == 0;
    const InT *x = keys ? (const InT *)p.k + head * p.k_hs : (const InT *)p.v + head * p.v_hs;
    const long ts = keys ? p.k_ts : p.v_ts;
    uint8_t *codes = keys ? p.c.k_codes : p.c.v_codes;
    uint32_t *par = keys ? p.c.k_par : p.c.v_par;
    const int t = blockIdx.x * (kAppendThreads / 8) + (threadIdx.x >> 3);
    // the values are on their way while the token's row is found
    float v[G][4], lo[G], hi[G];
#pragma unroll
    for (int g = 0; g < G; ++g) {
        float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
        if (t < p.N) f = load4<InT>(x + (long)t * ts + g * kKv4Group + r * 4);
        v[g][0] = f.x; v[g][1] = f.y; v[g][2] = f.z; v[g][3] = f.w;
    }
    long row;
    if (p.cu && p.c.B <= 32) row = kv4_row_of_few(p, t & ~3, head);
    else row = t < p.N ? kv4_row(p, t, head) : -1;
#pragma unroll
    for (int g = 0; g < G; ++g) {
        lo[g] = min_nan(min_nan(v[g][0], v[g][1]), min_nan(v[g][2], v[g][3]));
        hi[g] = max_nan(max_nan(v[g][0], v[g][1]), max_nan(v[g][2], v[g][3]));
    }
    // over the eight threads; with several groups each step also halves the
    // groups that a thread goes on with (4 groups: 12 shuffles instead of 24),
    // so that thread r ends with group r G / 8
#pragma unroll
    for (int off = 4, n = G; off > 0; off >>= 1) {
        if (n > 1) {
            const bool up = r & off;
            n >>= 1;
#pragma unroll
            for (int g = 0; g < n; ++g) {
                const float l = __shfl_xor_sync(0xffffffffu, up ? lo[g] : lo[g + n], off);
                const float h = __shfl_xor_sync(0xffffffffu, up ? hi[g] : hi[g + n], off);
                lo[g] = min_nan(up ? lo[g + n] : lo[g], l);
                hi[g] = max_nan(up ? hi[g + n] : hi[g], h);
            }
        } else {
            lo[0] = min_nan(lo[0], __shfl_xor_sync(0xffffffffu, lo[0], off));
            hi[0] = max_nan(hi[0], __shfl_xor_sync(0xffffffffu, hi[0], off));
        }
    }
    // the word of that group (NaN in lo and hi if any value was)
    const uint32_t own = kv4_word(lo[0], hi[0], __float_as_uint(max_nan(fabsf(lo[0]), fabsf(hi[0]))) & 0x7fffffffu);
    uint32_t word = 0u;   // group r's, for the store
    Chunk chunk = 0;
#pragma unroll
    for (int g = 0; g < G; ++g) {
        const uint32_t w = __shfl_sync(0xffffffffu, own, g * (8 / G), 8);
        if (r == g) word = w;
        chunk |= (Chunk)((Chunk)kv4_codes(v[g], w) << (16 * g));
    }
    if (row >= 0) {
        reinterpret_cast<Chunk *>(codes)[row * 8 + r] = chunk;
        if (r < G) par[row * G + r] = word;
    }
}

template <typename OutT, int D>
__global__ void __launch_bounds__(kAppendThreads) kv4_read_kernel(Kv4AppendParams p) {
    constexpr int G = D / kKv4Group;
    using Chunk = typename Kv4Chunk<D>::type;
    pdl_wait();
    const int r = threadIdx.x & 7, head = blockIdx.y;
    const bool keys = blockIdx.z == 0;
    const uint8_t *codes = keys ? p.c.k_codes : p.c.v_codes;
    const uint32_t *par = keys ? p.c.k_par : p.c.v_par;
    OutT *out = keys ? (OutT *)p.k_out : (OutT *)p.v_out;
    // a warp takes p.per (4 to 32) tokens: its lanes find a row each, then four tokens at a time
    const int lane = threadIdx.x & 31, w0 = (blockIdx.x * (kAppendThreads / 32) + (threadIdx.x >> 5)) * p.per;
    const long rows = lane < p.per && w0 + lane < p.N ? kv4_row(p, w0 + lane, head) : -1;
#pragma unroll 2
    for (int i = 0; i < p.per; i += 4) {
        const int t = w0 + i + (lane >> 3);
        const long row = __shfl_sync(0xffffffffu, rows, i + (lane >> 3));
        if (t >= p.N) continue;
        Chunk chunk = 0;
        if (row >= 0) chunk = reinterpret_cast<const Chunk *>(codes)[row * 8 + r];
        OutT *dst = out + ((long)head * p.N + t) * D + r * 4;
#pragma unroll
        for (int g = 0; g < G; ++g) {
            const uint32_t w = row >= 0 ? par[row * G + g] : 0u;
            const float sc = kv4_scale(w), of = kv4_offset(w);
            const uint32_t f = (uint32_t)(chunk >> (16 * g)) & 0xffffu;
            store4<OutT>(dst + g * kKv4Group, sc * ((float)(f & 15) + of), sc * ((float)((f >> 4) & 15) + of),
                         sc * ((float)((f >> 8) & 15) + of), sc * ((float)(f >> 12) + of));
        }
    }
}

}  // namespace la
