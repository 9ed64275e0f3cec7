// kv4_evict.cuh — eviction from the 4-bit cache by accumulated weight.
//
// One CTA per (sequence, head).  Of the n - recent older positions the
// keep - recent with the greatest keys are kept; the key of a weight is its
// bits made to order as unsigned integers.  The smallest key that is kept is
// found digit by digit (8 bits at a time, a histogram each); positions are
// then taken in order: those above it, the first few equal to it, and the
// recent ones.
#pragma once
#include "kv4_append.cuh"

namespace la {

struct Kv4EvictParams {
    Kv4CacheDev c, o;
    const float *weights;
    const int32_t *lens;
    int keep, recent;
    float *out_weights;
    int32_t *kept, *out_lens;
    int32_t *list;       // [B, Hkv, keep] workspace
};

constexpr int kEvictThreads = 512;

__device__ __forceinline__ uint32_t weight_key(float w) {
    const uint32_t u = __float_as_uint(w + 0.f);   // -0 becomes 0
    if ((u & 0x7fffffffu) > 0x7f800000u) return 0xffffffffu;
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

// list[0 .. kept) for one (sequence, head), its positions in order
__global__ void __launch_bounds__(kEvictThreads) kv4_select_kernel(Kv4EvictParams p) {
    __shared__ uint32_t hist[256];
    __shared__ uint32_t s_prefix, s_need;
    __shared__ uint32_t warp_gt[kEvictThreads / 32], warp_eq[kEvictThreads / 32], warp_new[kEvictThreads / 32];
    pdl_wait();
    const int hk = blockIdx.x, b = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int n = min(max(p.lens[b], 0), p.c.cap);
    const long bh = (long)b * p.c.Hkv + hk;
    const float *w = p.weights + bh * p.c.cap;
    int32_t *list = p.list + bh * p.keep;
    const int kept = min(n, p.keep);
    if (p.out_lens && hk == 0 && tid == 0) p.out_lens[b] = kept;
    if (p.kept)
        for (int i = kept + tid; i < p.keep; i += kEvictThreads) p.kept[bh * p.keep + i] = -1;
    if (n <= p.keep) {
        for (int i = tid; i < n; i += kEvictThreads) {
            list[i] = i;
            if (p.kept) p.kept[bh * p.keep + i] = i;
        }
        return;
    }
    const int old = n - p.recent;            // > 0: recent <= keep < n
    uint32_t prefix = 0, need = p.keep - p.recent;
    if (need > 0) {
        for (int shift = 24; shift >= 0; shift -= 8) {
            for (int i = tid; i < 256; i += kEvictThreads) hist[i] = 0;
            __syncthreads();
            for (int i = tid; i < old; i += kEvictThreads) {
                const uint32_t key = weight_key(w[i]);
                if (shift == 24 || (key >> (shift + 8)) == (prefix >> (shift + 8))) atomicAdd(&hist[(key >> shift) & 255], 1u);
            }
            __syncthreads();
            if (tid == 0) {
                uint32_t left = need;
                int d = 255;
                while (d > 0 && hist[d] < left) left -= hist[d--];
                s_prefix = prefix | ((uint32_t)d << shift);
                s_need = left;
            }
            __syncthreads();
            prefix = s_prefix;
            need = s_need;      // how many of the keys with this prefix are kept
        }
    }
    // in order: greater keys, the first `need` equal ones (none if recent == keep), the recent positions
    const bool any_old = p.keep > p.recent;
    uint32_t base = 0, base_eq = 0;
    for (int i0 = 0; i0 < n; i0 += kEvictThreads) {
        const int i = i0 + tid;
        bool take = false, eq = false;
        if (i < old && any_old) {
            const uint32_t key = weight_key(w[i]);
            take = key > prefix;
            eq = key == prefix;
        } else if (i >= old && i < n) {
            take = true;
        }
        const uint32_t me = __ballot_sync(0xffffffffu, eq);
        if (lane == 0) warp_eq[warp] = __popc(me);
        __syncthreads();
        uint32_t before_eq = base_eq + __popc(me & ((1u << lane) - 1));
        uint32_t all_eq = 0;
        for (int x = 0; x < kEvictThreads / 32; ++x) {
            if (x < warp) before_eq += warp_eq[x];
            all_eq += warp_eq[x];
        }
        if (eq && before_eq < need) take = true;
        base_eq += all_eq;
        const uint32_t mt = __ballot_sync(0xffffffffu, take);
        if (lane == 0) warp_gt[warp] = __popc(mt);
        __syncthreads();
        uint32_t at = base + __popc(mt & ((1u << lane) - 1)), all = 0;
        for (int x = 0; x < kEvictThreads / 32; ++x) {
            if (x < warp) at += warp_gt[x];
            all += warp_gt[x];
        }
        base += all;
        if (take) {
            list[at] = i;
            if (p.kept) p.kept[bh * p.keep + at] = i;
        }
    }
}

// copies the listed rows and weights; eight threads per row
template <int D> __global__ void __launch_bounds__(256) kv4_gather_kernel(Kv4EvictParams p) {
    constexpr int G = D / kKv4Group;
    using Chunk = typename Kv4Chunk<D>::type;
    pdl_wait();
    const int hk = blockIdx.y, b = blockIdx.z, r = threadIdx.x & 7;
    const int kept = min(min(max(p.lens[b], 0), p.c.cap), p.keep);
    const long bh = (long)b * p.c.Hkv + hk;
    for (int j = blockIdx.x * 32 + (threadIdx.x >> 3); j < kept; j += gridDim.x * 32) {
        const int i = p.list[bh * p.keep + j];
        const long src = bh * p.c.cap + i, dst = bh * p.o.cap + j;
        reinterpret_cast<Chunk *>(p.o.k_codes)[dst * 8 + r] = reinterpret_cast<const Chunk *>(p.c.k_codes)[src * 8 + r];
        reinterpret_cast<Chunk *>(p.o.v_codes)[dst * 8 + r] = reinterpret_cast<const Chunk *>(p.c.v_codes)[src * 8 + r];
        if (r < G) {
            p.o.k_par[dst * G + r] = p.c.k_par[src * G + r];
            p.o.v_par[dst * G + r] = p.c.v_par[src * G + r];
        }
        if (r == 7 && p.out_weights) p.out_weights[dst] = p.weights[bh * p.c.cap + i];
    }
}

}  // namespace la
