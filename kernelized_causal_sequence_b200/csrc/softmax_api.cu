// softmax_api.cu — the softmax operators of include/linattn.h: argument
// checks, workspace layout and dispatch.  Everything is checked on the host
// before anything is launched.
#include <cmath>
#include <cstring>

#include "errors.h"
#include "kv4_append.cuh"
#include "kv4_decode.cuh"
#include "kv4_evict.cuh"
#include "launch.h"
#include "linattn.h"
#include "plan.h"
#include "softmax_simt.cuh"
#include "softmax_tc.h"

using namespace la;

namespace {

constexpr size_t kWsAlign = 256;
constexpr int kMaxTokens = 1 << 30;   // N and n_seq: tile numbers and row indexes stay in 32 bits
inline size_t ws_up(size_t x) { return (x + kWsAlign - 1) / kWsAlign * kWsAlign; }
inline bool al16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool al4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
inline bool dt_ok(la_dtype t) { return t == LA_F32 || t == LA_BF16 || t == LA_F16; }
inline bool d_ok(int d) { return d == 32 || d == 64 || d == 128; }
inline int esize(la_dtype t) { return t == LA_F32 ? 4 : 2; }
inline bool ws_ok(const void *ws, size_t have, size_t need) {
    return need == 0 || (ws && have >= need && (reinterpret_cast<uintptr_t>(ws) & (kWsAlign - 1)) == 0);
}

// What the kernels multiply scores by: scale log2(e), a normal number (an infinite one makes a score of 0 NaN, a
// subnormal one is cut short).
inline bool scale_ok(float scale) { return scale > 0.f && std::isnormal(scale * kLog2e); }

la_status check_types(la_dtype in, la_dtype out, int d) {
    if (!dt_ok(in) || !dt_ok(out) || d <= 0) return LA_ERR_INVALID_ARG;
    if (!d_ok(d) || !(out == in || out == LA_F32)) return LA_ERR_UNSUPPORTED;
    return LA_OK;
}

// Query heads over key/value heads.
la_status check_heads(int H, int H_kv) {
    if (H < 0 || H_kv < 0 || (H_kv == 0) != (H == 0)) return LA_ERR_INVALID_ARG;
    if (H == 0) return LA_OK;
    if (H % H_kv) return LA_ERR_INVALID_ARG;
    return H > 65535 ? LA_ERR_UNSUPPORTED : LA_OK;   // heads run along grid y
}

// One tensor's (head, token) strides: given or contiguous.  A stride of an
// extent of at most 1 is never used and is replaced by a valid one.
bool set_strides(const int64_t *s, int heads, int N, int d, int es, long *hs, long *ts) {
    *ts = d;
    *hs = (long)N * d;
    if (!s) return true;
    const int per16 = 16 / es;
    if (N > 1) {
        if (s[1] < d || s[1] % per16 || s[1] >= (1L << 39) / es) return false;
        *ts = s[1];
        *hs = s[1] * N;
    }
    if (heads > 1) {
        if (s[0] < d || s[0] % per16 || s[0] >= (1L << 39) / es) return false;
        *hs = s[0];
    }
    return true;
}

// Bytes from a tensor's first to behind its last element.
inline size_t span(int heads, int N, int d, long hs, long ts, int es) {
    return ((size_t)(heads - 1) * hs + (size_t)(N - 1) * ts + d) * es;
}
inline bool overlap(const void *a, size_t na, const void *b, size_t nb) {
    const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
    return a && b && na && nb && x < y + nb && y < x + na;
}
// The memory of one argument of a call (null or empty: none).
struct Region {
    const void *at;
    size_t bytes;
};
// Whether a call's outputs overlap its inputs or one another: CTAs write while others read.
template <int NO, int NI> bool aliased(const Region (&out)[NO], const Region (&in)[NI]) {
    for (int i = 0; i < NO; ++i) {
        for (int j = 0; j < NI; ++j)
            if (overlap(out[i].at, out[i].bytes, in[j].at, in[j].bytes)) return true;
        for (int j = 0; j < i; ++j)
            if (overlap(out[i].at, out[i].bytes, out[j].at, out[j].bytes)) return true;
    }
    return false;
}

la_status check_cache(const la_kv4_cache *c) {
    if (!c || c->B < 0 || c->H_kv < 0 || c->cap < 0 || c->d <= 0) return LA_ERR_INVALID_ARG;
    if (!d_ok(c->d)) return LA_ERR_UNSUPPORTED;
    if (c->H_kv > 65535 || c->B > 65535 || c->cap > kMaxTokens) return LA_ERR_UNSUPPORTED;
    if ((long)c->B * c->H_kv * c->cap == 0) return LA_OK;
    if (!c->k_codes || !c->k_par || !c->v_codes || !c->v_par || !al16(c->k_codes) || !al16(c->k_par) ||
        !al16(c->v_codes) || !al16(c->v_par))
        return LA_ERR_INVALID_ARG;
    return LA_OK;
}
Kv4CacheDev dev_cache(const la_kv4_cache *c) {
    return Kv4CacheDev{c->k_codes, c->k_par, c->v_codes, c->v_par, c->B, c->H_kv, c->cap};
}
inline size_t code_bytes(const la_kv4_cache *c) { return (size_t)c->B * c->H_kv * c->cap * (c->d / 2); }
inline size_t par_bytes(const la_kv4_cache *c) { return (size_t)c->B * c->H_kv * c->cap * (c->d / 8); }

// Grid x of a kernel that strides over `items` in blocks of `per`: enough
// blocks, over `others` grid rows, for about eight waves of one block per SM.
inline unsigned stride_grid(long items, int per, long others) {
    const long need = (items + per - 1) / per, most = (8L * kNumSMs + others - 1) / others;
    return (unsigned)(need < most ? need : most);
}

#define LA_BY_D(d, CALL)                    \
    switch (d) {                            \
        case 32: { constexpr int D = 32; CALL; }   \
        case 64: { constexpr int D = 64; CALL; }   \
        case 128: { constexpr int D = 128; CALL; } \
        default: return LA_ERR_UNSUPPORTED; \
    }
#define LA_BY_TYPES(in, out, CALL)                                                          \
    if (in == LA_F32) { using InT = float; using OutT = float; CALL; }                      \
    if (in == LA_BF16 && out == LA_BF16) { using InT = bf16; using OutT = bf16; CALL; }     \
    if (in == LA_BF16) { using InT = bf16; using OutT = float; CALL; }                      \
    if (out == LA_F16) { using InT = f16; using OutT = f16; CALL; }                         \
    { using InT = f16; using OutT = float; CALL; }

template <int BM> la_status run_softmax_simt_bm(const SoftmaxParams &p, int d, cudaStream_t st) {
    LA_BY_D(d, return launch_kernel(softmax_simt_kernel<D, BM>,
                                    dim3((unsigned)seq_tiles(p.N, p.n_seq, BM), (unsigned)p.H), dim3(kSsThreads),
                                    softmax_simt_smem<D, BM>(), st, true, "softmax prefill launch", p))
}
la_status run_softmax_simt(const SoftmaxParams &p, int d, cudaStream_t st) {
    // tiles of 64 queries, or of 16 where those leave half of the SMs without one (us 16 / 64, tiles of 64 over all heads:
    //   d 64   1 x 320, 8 heads (48): 37 / 41, 2 x 256, 8 heads (80): 39 / 35, 1 x 1024, 8 heads (136): 162 / 111
    //   d 128  1 x 128, 16 heads (48): 27 / 33, 1 x 256 (80): 66 / 51, 1 x 320 (96): 83 / 61
    // of many sequences shorter than a tile 16 stay faster: 16 x 16 tokens, d 64, 16 heads (320): 14 / 16)
    if (2L * seq_tiles(p.N, p.n_seq, 64) * p.H >= kNumSMs) return run_softmax_simt_bm<64>(p, d, st);
    return run_softmax_simt_bm<16>(p, d, st);
}
template <typename InT> la_status run_append(const Kv4AppendParams &p, int d, cudaStream_t st) {
    const dim3 grid((unsigned)((p.N + kAppendThreads / 8 - 1) / (kAppendThreads / 8)), (unsigned)p.c.Hkv, 2);
    LA_BY_D(d, return launch_kernel(kv4_append_kernel<InT, D>, grid, dim3(kAppendThreads), 0, st, true,
                                    "kv4 append launch", p))
}
template <typename OutT> la_status run_read(Kv4AppendParams p, int d, cudaStream_t st) {
    // as many tokens a warp as leave 40 warps for every SM
    p.per = 4;
    while (p.per < 32 && (long)p.N * p.c.Hkv * 2 / (2 * p.per) >= 40L * kNumSMs) p.per *= 2;
    const int block = kAppendThreads / 32 * p.per;
    const dim3 grid((unsigned)((p.N + block - 1) / block), (unsigned)p.c.Hkv, 2);
    LA_BY_D(d, return launch_kernel(kv4_read_kernel<OutT, D>, grid, dim3(kAppendThreads), 0, st, true,
                                    "kv4 read launch", p))
}
// CTAs of the decode kernel: as many as are resident at once (its launch
// bounds), or one per row for short caches.
struct DecodePlan {
    int nt, head_blocks, n_cta, whole;
    size_t ml_off, o_off, row_off, scores_off, bytes;
};
DecodePlan decode_plan(int B, int H, int H_kv, int cap, int d, int with_weights) {
    DecodePlan w;
    const int group = H / H_kv;
    // up to 16 query heads a row, which unpacks the keys once for them; by 8 where there are not more (us 16 / by 8 of
    // 16 heads a key, d 128, bf16, caches of 8192: 64 x 4 rows 162 / 207, 16 x 2 rows 43 / 41, one row 31 / 18)
    w.nt = group > 8 ? 2 : 1;
    w.head_blocks = (group + 8 * w.nt - 1) / (8 * w.nt);
    const long rows = (long)B * H_kv * w.head_blocks;
    w.whole = cap <= (rows >= kNumSMs ? kDecWholeFull : kDecWhole);
    w.n_cta = w.whole ? (int)rows : kNumSMs * (w.nt == 1 ? kDecCtas : 2);
    size_t at = 0;
    w.ml_off = at;
    if (!w.whole) at += ws_up((size_t)2 * w.n_cta * 8 * w.nt * sizeof(float2));
    w.o_off = at;
    if (!w.whole) at += ws_up((size_t)2 * w.n_cta * 8 * w.nt * d * sizeof(float));
    w.row_off = at;
    if (with_weights) at += ws_up((size_t)B * H * sizeof(float2));
    w.scores_off = at;
    if (with_weights) at += ws_up((size_t)B * H * cap * sizeof(float));
    w.bytes = at;
    return w;
}

template <typename InT, typename OutT, int D, int NT>
la_status run_decode_nt(const Kv4DecodeParams &p, cudaStream_t st) {
    la_status s = launch_kernel(kv4_decode_kernel<InT, OutT, D, NT>, dim3((unsigned)p.n_cta), dim3(kDecWarps * 32),
                                kv4_decode_smem<D>(NT), st, true, "kv4 decode launch", p);
    if (s != LA_OK || (p.whole && (!p.weights_out || p.head_blocks == 1))) return s;
    const unsigned ob = p.whole ? 0u : (unsigned)p.group;
    // (four positions a thread, at most four blocks per SM)
    const unsigned wb = p.weights_out ? stride_grid(p.c.cap, 4 * kFinThreads, 2L * p.c.Hkv * p.c.B) : 0u;
    if (ob + wb == 0) return LA_OK;   // (a cache without positions)
    return launch_kernel(kv4_finish_kernel<OutT, D>, dim3(ob + wb, (unsigned)p.c.Hkv, (unsigned)p.c.B),
                         dim3(kFinThreads), 0, st, true, "kv4 finish launch", p, (int)ob);
}
template <typename InT, typename OutT> la_status run_decode(const Kv4DecodeParams &p, int d, int nt, cudaStream_t st) {
    if (nt == 1) { LA_BY_D(d, return (run_decode_nt<InT, OutT, D, 1>(p, st))) }
    LA_BY_D(d, return (run_decode_nt<InT, OutT, D, 2>(p, st)))
}

template <int THREADS> la_status run_evict(const Kv4EvictParams &p, int d, long rows, int cs, cudaStream_t st) {
    if (rows * cs > 0x7fffffffL) return LA_ERR_UNSUPPORTED;
    LA_BY_D(d, return launch_cluster(kv4_evict_kernel<D, THREADS>, dim3((unsigned)(rows * cs)), dim3(THREADS), 0, st, true, cs,
                                     "kv4 evict launch", p, cs))
}

}  // namespace

extern "C" {

size_t la_softmax_prefill_workspace_size(int H, int H_kv, int N, int d, int n_seq) {
    if (H <= 0 || H_kv <= 0 || H % H_kv || N <= 0 || n_seq <= 0 || !d_ok(d)) return 0;
    return kWsAlign;
}

la_status la_softmax_prefill(const void *q, const void *k, const void *v, la_dtype in_dtype, int H, int H_kv,
                             int N, int d, const int32_t *cu_seqlens, int n_seq, const int64_t *strides,
                             float scale, void *out, la_dtype out_dtype, void *workspace,
                             size_t workspace_bytes, void *stream) {
    la_status s = check_types(in_dtype, out_dtype, d);
    if (s != LA_OK || (s = check_heads(H, H_kv)) != LA_OK) return s;
    if (N < 0 || n_seq < 0 || !scale_ok(scale)) return LA_ERR_INVALID_ARG;
    if (N > kMaxTokens || n_seq > kMaxTokens) return LA_ERR_UNSUPPORTED;
    SoftmaxParams p;
    const int ie = esize(in_dtype), oe = esize(out_dtype);
    if (!set_strides(strides, H, N, d, ie, &p.q_hs, &p.q_ts) ||
        !set_strides(strides ? strides + 2 : nullptr, H_kv, N, d, ie, &p.k_hs, &p.k_ts) ||
        !set_strides(strides ? strides + 4 : nullptr, H_kv, N, d, ie, &p.v_hs, &p.v_ts) ||
        !set_strides(strides ? strides + 6 : nullptr, H, N, d, oe, &p.o_hs, &p.o_ts))
        return LA_ERR_INVALID_ARG;
    if (H == 0 || N == 0 || n_seq == 0) return LA_OK;
    if (!q || !k || !v || !out || !cu_seqlens || !al16(q) || !al16(k) || !al16(v) || !al16(out) || !al4(cu_seqlens))
        return LA_ERR_INVALID_ARG;
    if (!ws_ok(workspace, workspace_bytes, kWsAlign)) return LA_ERR_INVALID_ARG;
    const Region outs[] = {{out, span(H, N, d, p.o_hs, p.o_ts, oe)}, {workspace, kWsAlign}};
    const Region ins[] = {{q, span(H, N, d, p.q_hs, p.q_ts, ie)}, {k, span(H_kv, N, d, p.k_hs, p.k_ts, ie)},
                          {v, span(H_kv, N, d, p.v_hs, p.v_ts, ie)}, {cu_seqlens, sizeof(int32_t) * ((size_t)n_seq + 1)}};
    if (aliased(outs, ins)) return LA_ERR_INVALID_ARG;
    cudaStream_t st = (cudaStream_t)stream;
    p.q = q; p.k = k; p.v = v; p.out = out; p.cu = cu_seqlens;
    p.H = H; p.group = H / H_kv; p.N = N; p.n_seq = n_seq;
    p.scale_log2 = scale * kLog2e;
    p.status = (int *)workspace;
    if (softmax_tc_supported(in_dtype)) {
        // the status word and the tile counter behind it
        if ((s = cuda_check("status memset", cudaMemsetAsync(workspace, 0, 4 * sizeof(int), st))) != LA_OK) return s;
        return softmax_tc(p, in_dtype, out_dtype, d, (int *)workspace, wait_limit_ns(), st);
    }
    return run_softmax_simt(p, d, st);
}

la_status la_kv4_append(const void *k, const void *v, la_dtype in_dtype, int N, const int64_t *strides,
                        const int32_t *cu_seqlens, const int32_t *start, const la_kv4_cache *cache, void *stream) {
    la_status s = check_cache(cache);
    if (s != LA_OK) return s;
    if (!dt_ok(in_dtype) || N < 0 || (!cu_seqlens && N != cache->B)) return LA_ERR_INVALID_ARG;
    if (N > kMaxTokens) return LA_ERR_UNSUPPORTED;
    Kv4AppendParams p;
    std::memset(&p, 0, sizeof(p));
    const int es = esize(in_dtype);
    if (!set_strides(strides, cache->H_kv, N, cache->d, es, &p.k_hs, &p.k_ts) ||
        !set_strides(strides ? strides + 2 : nullptr, cache->H_kv, N, cache->d, es, &p.v_hs, &p.v_ts))
        return LA_ERR_INVALID_ARG;
    if (N == 0 || cache->B == 0 || cache->H_kv == 0 || cache->cap == 0) return LA_OK;
    if (!k || !v || !start || !al16(k) || !al16(v) || !al4(start) || !al4(cu_seqlens)) return LA_ERR_INVALID_ARG;
    const Region outs[] = {{cache->k_codes, code_bytes(cache)}, {cache->k_par, par_bytes(cache)},
                           {cache->v_codes, code_bytes(cache)}, {cache->v_par, par_bytes(cache)}};
    const Region ins[] = {{k, span(cache->H_kv, N, cache->d, p.k_hs, p.k_ts, es)},
                          {v, span(cache->H_kv, N, cache->d, p.v_hs, p.v_ts, es)},
                          {cu_seqlens, sizeof(int32_t) * ((size_t)cache->B + 1)}, {start, sizeof(int32_t) * (size_t)cache->B}};
    if (aliased(outs, ins)) return LA_ERR_INVALID_ARG;
    p.k = k; p.v = v; p.cu = cu_seqlens; p.start = start; p.c = dev_cache(cache); p.N = N;
    cudaStream_t st = (cudaStream_t)stream;
    if (in_dtype == LA_F32) return run_append<float>(p, cache->d, st);
    if (in_dtype == LA_BF16) return run_append<bf16>(p, cache->d, st);
    return run_append<f16>(p, cache->d, st);
}

la_status la_kv4_read(const la_kv4_cache *cache, int N, const int32_t *cu_seqlens, const int32_t *start,
                      void *k_out, void *v_out, la_dtype out_dtype, void *stream) {
    la_status s = check_cache(cache);
    if (s != LA_OK) return s;
    if (!dt_ok(out_dtype) || N < 0 || (!cu_seqlens && N != cache->B)) return LA_ERR_INVALID_ARG;
    if (N > kMaxTokens) return LA_ERR_UNSUPPORTED;
    if (N == 0 || cache->H_kv == 0) return LA_OK;
    if (!k_out || !v_out || !al16(k_out) || !al16(v_out) || (cache->B && !start) || !al4(start) || !al4(cu_seqlens))
        return LA_ERR_INVALID_ARG;
    const size_t n = (size_t)cache->H_kv * N * cache->d * esize(out_dtype);
    const Region outs[] = {{k_out, n}, {v_out, n}};
    const Region ins[] = {{cache->k_codes, code_bytes(cache)}, {cache->k_par, par_bytes(cache)},
                          {cache->v_codes, code_bytes(cache)}, {cache->v_par, par_bytes(cache)},
                          {cu_seqlens, sizeof(int32_t) * ((size_t)cache->B + 1)}, {start, sizeof(int32_t) * (size_t)cache->B}};
    if (aliased(outs, ins)) return LA_ERR_INVALID_ARG;
    if (cache->B == 0) {   // tokens of no sequence
        if ((s = cuda_check("kv4 read", cudaMemsetAsync(k_out, 0, n, (cudaStream_t)stream))) != LA_OK) return s;
        return cuda_check("kv4 read", cudaMemsetAsync(v_out, 0, n, (cudaStream_t)stream));
    }
    Kv4AppendParams p;
    std::memset(&p, 0, sizeof(p));
    p.cu = cu_seqlens; p.start = start; p.c = dev_cache(cache); p.N = N; p.k_out = k_out; p.v_out = v_out;
    cudaStream_t st = (cudaStream_t)stream;
    if (out_dtype == LA_F32) return run_read<float>(p, cache->d, st);
    if (out_dtype == LA_BF16) return run_read<bf16>(p, cache->d, st);
    return run_read<f16>(p, cache->d, st);
}

size_t la_kv4_decode_workspace_size(int B, int H, int H_kv, int cap, int d, int with_weights) {
    if (B <= 0 || H <= 0 || H_kv <= 0 || H % H_kv || cap < 0 || cap > kMaxTokens || !d_ok(d)) return 0;
    return decode_plan(B, H, H_kv, cap, d, with_weights).bytes;
}

la_status la_kv4_decode(const void *q, la_dtype in_dtype, int H, const la_kv4_cache *cache, const int32_t *lens,
                        float scale, const float *weights_in, float *weights_out, void *out, la_dtype out_dtype,
                        void *workspace, size_t workspace_bytes, void *stream) {
    la_status s = check_cache(cache);
    if (s != LA_OK || (s = check_types(in_dtype, out_dtype, cache->d)) != LA_OK ||
        (s = check_heads(H, cache->H_kv)) != LA_OK)
        return s;
    if (!scale_ok(scale) || (weights_in && !weights_out)) return LA_ERR_INVALID_ARG;
    if (H == 0 || cache->B == 0) return LA_OK;
    if (!q || !lens || !out || !al16(q) || !al16(out) || !al4(lens) || !al16(weights_in) || !al16(weights_out))
        return LA_ERR_INVALID_ARG;
    const DecodePlan pl = decode_plan(cache->B, H, cache->H_kv, cache->cap, cache->d, weights_out != nullptr);
    if (!ws_ok(workspace, workspace_bytes, pl.bytes)) return LA_ERR_INVALID_ARG;
    const size_t elems = (size_t)cache->B * H * cache->d, wb = (size_t)cache->B * cache->H_kv * cache->cap * sizeof(float);
    const Region outs[] = {{out, elems * esize(out_dtype)}, {weights_out, wb}, {workspace, pl.bytes}};
    const Region ins[] = {{q, elems * esize(in_dtype)}, {lens, sizeof(int32_t) * (size_t)cache->B},
                          {weights_in == weights_out ? nullptr : weights_in, wb},
                          {cache->k_codes, code_bytes(cache)}, {cache->k_par, par_bytes(cache)},
                          {cache->v_codes, code_bytes(cache)}, {cache->v_par, par_bytes(cache)}};
    if (aliased(outs, ins)) return LA_ERR_INVALID_ARG;
    if ((long)cache->B * cache->H_kv * pl.head_blocks > 0x7fffffffL) return LA_ERR_UNSUPPORTED;
    char *ws = (char *)workspace;
    Kv4DecodeParams p;
    std::memset(&p, 0, sizeof(p));
    p.q = q; p.c = dev_cache(cache); p.lens = lens; p.weights_in = weights_in; p.weights_out = weights_out;
    p.out = out; p.H = H; p.group = H / cache->H_kv; p.scale_log2 = scale * kLog2e;
    p.n_cta = pl.n_cta; p.whole = pl.whole; p.head_blocks = pl.head_blocks; p.head_block = 8 * pl.nt;
    p.part_ml = (float2 *)(ws + pl.ml_off);
    p.part_o = (float *)(ws + pl.o_off);
    if (weights_out) {
        p.row_ml = (float2 *)(ws + pl.row_off);
        p.scores = (float *)(ws + pl.scores_off);
    }
    cudaStream_t st = (cudaStream_t)stream;
    LA_BY_TYPES(in_dtype, out_dtype, return (run_decode<InT, OutT>(p, cache->d, pl.nt, st)))
}

size_t la_kv4_evict_workspace_size(int B, int H_kv, int cap, int keep) {
    if (B <= 0 || H_kv <= 0 || cap < 0 || cap > kMaxTokens || keep < 1) return 0;
    return ws_up((size_t)B * H_kv * keep * sizeof(int32_t));
}

la_status la_kv4_evict(const la_kv4_cache *cache, const float *weights, const int32_t *lens, int keep, int recent,
                       const la_kv4_cache *out, float *out_weights, int32_t *kept, int32_t *out_lens,
                       void *workspace, size_t workspace_bytes, void *stream) {
    la_status s = check_cache(cache);
    if (s != LA_OK || (s = check_cache(out)) != LA_OK) return s;
    if (out->B != cache->B || out->H_kv != cache->H_kv || out->d != cache->d || keep < 1 || recent < 0 ||
        recent > keep || out->cap < keep)
        return LA_ERR_INVALID_ARG;
    if (cache->B == 0) return LA_OK;
    if (cache->H_kv == 0) return out_lens ? LA_ERR_INVALID_ARG : LA_OK;   // (a head's CTA writes them)
    if (!lens || !al4(lens) || !al4(kept) || !al4(out_lens) || !al16(out_weights)) return LA_ERR_INVALID_ARG;
    if (cache->cap > 0 && (!weights || !al16(weights))) return LA_ERR_INVALID_ARG;
    // the list of kept positions: the caller's `kept`, or the workspace
    const size_t need = kept ? 0 : ws_up((size_t)cache->B * cache->H_kv * keep * sizeof(int32_t));
    if (!ws_ok(workspace, workspace_bytes, need)) return LA_ERR_INVALID_ARG;
    const size_t heads = (size_t)cache->B * cache->H_kv, lb = sizeof(int32_t) * (size_t)cache->B;
    const Region outs[] = {{out->k_codes, code_bytes(out)}, {out->k_par, par_bytes(out)}, {out->v_codes, code_bytes(out)},
                           {out->v_par, par_bytes(out)}, {out_weights, heads * out->cap * sizeof(float)},
                           {kept, heads * keep * sizeof(int32_t)}, {out_lens, lb}, {workspace, need}};
    const Region ins[] = {{cache->k_codes, code_bytes(cache)}, {cache->k_par, par_bytes(cache)},
                          {cache->v_codes, code_bytes(cache)}, {cache->v_par, par_bytes(cache)},
                          {weights, heads * cache->cap * sizeof(float)}, {lens, lb}};
    if (aliased(outs, ins)) return LA_ERR_INVALID_ARG;
    Kv4EvictParams p;
    std::memset(&p, 0, sizeof(p));
    p.c = dev_cache(cache); p.o = dev_cache(out); p.weights = weights; p.lens = lens; p.keep = keep;
    p.recent = recent; p.out_weights = out_weights; p.kept = kept; p.out_lens = out_lens;
    p.list = kept ? kept : (int32_t *)workspace;
    cudaStream_t st = (cudaStream_t)stream;
    // Short caches: blocks of 256 threads, whose barriers are cheaper and of which several fit an SM; long ones: of
    // 1024, as many CTAs of a (sequence, head) as its positions fill with 8 keys a thread and the machine has SMs for
    // (us 256 / 1024 threads, cut to half, d 128: 2 rows 12 / 14 at 400 positions, 16 / 16 at 1024, 22 / 22 at 2048;
    // 296 rows 16 / 29, 25 / 35, 39 / 47; d 64, 2 rows 43 / 24 at 4096, 80 / 31 at 8192)
    const long rows = (long)cache->B * cache->H_kv;
    if (cache->cap <= 256 * kEvictKeys) return run_evict<256>(p, cache->d, rows, 1, st);
    int cs = 1;
    while (cs < kEvictMaxCluster && (long)cs * 1024 * kEvictKeys < cache->cap && rows * cs < kNumSMs) cs *= 2;
    return run_evict<1024>(p, cache->d, rows, cs, st);
}

}  // extern "C"
