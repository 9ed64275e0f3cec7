// kv4_evict.cuh — eviction from the 4-bit cache by accumulated weight.
//
// One thread-block cluster of 1 to 8 CTAs per (sequence, head), each CTA with
// a slice of its positions, whose keys it holds in registers.  Of the
// n - recent older positions the keep - recent with the greatest keys stay (the
// key of a weight is its bits made to order as unsigned integers).  The least
// key that stays is found in at most four steps of eight bits, a histogram
// each, which the CTAs of a cluster add up through distributed shared memory.
// Softmax weights crowd into a few bins, so a warp first joins its equal
// digits (match_any) and adds once for each.  (Bit by bit with a count for each
// the same search took 33 block-wide sums, 21 us for 300 positions.)  16 x 8 rows
// of up to 8192 positions, d 128, cut to 2048: 28 us, a third of the DRAM rate,
// bound by the search's chain of block-wide steps; 300 positions: 12 us (76 and
// 34 as separate kernels for selecting and copying).  Positions
// are then ranked by ballots and two prefix sums (those equal to the least key
// stay from the lowest on), listed, and their rows copied, eight threads each.
#pragma once
#include <cooperative_groups.h>

#include "kv4_append.cuh"

namespace la {

struct Kv4EvictParams {
    Kv4CacheDev c, o;
    const float *weights;
    const int32_t *lens;
    int keep, recent;
    float *out_weights;
    int32_t *kept, *out_lens;
    int32_t *list;       // [B, Hkv, keep]: kept, or the workspace
};

constexpr int kEvictMaxCluster = 8, kEvictKeys = 8;   // CTAs of a cluster, keys of a thread

__device__ __forceinline__ uint32_t weight_key(float w) {
    const uint32_t u = __float_as_uint(w + 0.f);   // -0 becomes 0
    if ((u & 0x7fffffffu) > 0x7f800000u) return 0xffffffffu;
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;   // never 0
}

struct EvictShared {
    uint32_t hist[2][256];              // by turns, as the slots
    uint32_t cells[kEvictKeys * 32];    // ballot counts [key of a thread][warp], then their prefix sums
    uint32_t sums[32];
    uint32_t digit, above, in_digit;    // a step's result: digit, keys in greater ones, keys in it
    uint32_t slots[2][kEvictMaxCluster];   // the CTAs' counts, by turns
};

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }

// The sum of x (a CTA's own number, the same in all threads) over the CTAs of lower rank.  `turn` alternates the
// slots: a CTA can be one exchange ahead of another, not two.
__device__ __forceinline__ uint32_t sum_before(EvictShared &sh, uint32_t x, int cs, int rank, int &turn) {
    auto cl = cooperative_groups::this_cluster();
    if ((int)threadIdx.x < cs) cl.map_shared_rank(&sh.slots[turn][0], threadIdx.x)[rank] = x;
    cl.sync();
    uint32_t sum = 0;
    for (int i = 0; i < rank; ++i) sum += sh.slots[turn][i];
    turn ^= 1;
    return sum;
}

// The sum over the block of a number that each warp's lanes share.  All threads.
template <int NW> __device__ __forceinline__ uint32_t block_sum(EvictShared &sh, uint32_t x) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    __syncthreads();
    if (lane == 0) sh.sums[warp] = x;
    __syncthreads();
    return __reduce_add_sync(0xffffffffu, lane < NW ? sh.sums[lane] : 0u);
}

// Exclusive prefix sums of the first n <= blockDim cells, in place; their total.  All threads.
template <int NW> __device__ __forceinline__ uint32_t scan_cells(EvictShared &sh, int n) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    __syncthreads();
    uint32_t v = (int)threadIdx.x < n ? sh.cells[threadIdx.x] : 0u, x = v;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, x, off);
        if (lane >= off) x += y;
    }
    if (lane == 31) sh.sums[warp] = x;
    __syncthreads();
    const uint32_t s = lane < NW ? sh.sums[lane] : 0u;
    const uint32_t add = __reduce_add_sync(0xffffffffu, lane < warp ? s : 0u);
    const uint32_t total = __reduce_add_sync(0xffffffffu, s);
    if ((int)threadIdx.x < n) sh.cells[threadIdx.x] = x - v + add;
    __syncthreads();
    return total;
}

template <int D, int THREADS> __global__ void __launch_bounds__(THREADS) kv4_evict_kernel(Kv4EvictParams p, int cs) {
    constexpr int G = D / kKv4Group, KPT = kEvictKeys, SPAN = KPT * THREADS, NW = THREADS / 32;
    using Chunk = typename Kv4Chunk<D>::type;
    __shared__ EvictShared sh;
    // A CTA's shared memory may be reached into only once that CTA runs: every CTA of the cluster says so here, and
    // waits for the others below, before its first access to theirs.
    if (cs > 1) cluster_arrive();
    pdl_wait();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = blockIdx.x % cs, bh_i = blockIdx.x / cs;
    const int b = bh_i / p.c.Hkv;
    const long bh = bh_i;
    const int n = min(max(p.lens[b], 0), p.c.cap);
    const float *w = p.weights + bh * p.c.cap;
    int32_t *list = p.list + bh * p.keep;
    const int kept = min(n, p.keep);
    // positions below `old` compete, the others stay
    const int old = n <= p.keep ? 0 : n - p.recent;
    const uint32_t need = n <= p.keep ? 0u : (uint32_t)(p.keep - p.recent);
    const int slice = (n + cs - 1) / cs, s0 = min(rank * slice, n), s1 = min(s0 + slice, n);
    const int spans = (s1 - s0 + SPAN - 1) / SPAN;   // 1, but for slices that do not fit the registers
    int turn = 0;
    uint32_t key[KPT];
    auto load = [&](int span) {
#pragma unroll
        for (int i = 0; i < KPT; ++i) {
            const int at = s0 + span * SPAN + i * THREADS + tid;
            key[i] = at < min(s1, old) ? weight_key(w[at]) : 0u;   // 0: does not compete
        }
    };
    load(0);
    if (cs > 1) cluster_wait();
    // the least key that stays, and how many equal to it do
    uint32_t least = 0xffffffffu, equal = 0;
    if (need > 0) {
        least = 0;
        equal = need;   // of the keys that agree with `least` so far, how many stay
        for (int shift = 24; shift >= 0; shift -= 8) {
            uint32_t *hist = sh.hist[(shift >> 3) & 1];
            for (int i = tid; i < 256; i += THREADS) hist[i] = 0;
            __syncthreads();
            for (int s = 0; s < spans; ++s) {
                if (spans > 1) load(s);
#pragma unroll
                for (int i = 0; i < KPT; ++i) {
                    // (keys of 0 have no place; shift 24: all agree)
                    const bool in = key[i] != 0u && (shift == 24 || (key[i] >> (shift + 8)) == (least >> (shift + 8)));
                    const uint32_t digit = in ? (key[i] >> shift) & 255u : 256u;
                    if (!__any_sync(0xffffffffu, in)) continue;
                    const uint32_t same = __match_any_sync(0xffffffffu, digit);
                    if (in && lane == __ffs(same) - 1) atomicAdd(&hist[digit], (uint32_t)__popc(same));
                }
            }
            if (cs > 1) cooperative_groups::this_cluster().sync();
            else __syncthreads();
            if (warp == 0) {
                // lane l: the digits 255 - 8 l down to 248 - 8 l
                uint32_t c[8], sum = 0;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    c[i] = 0;
                    if (cs > 1) {
                        auto cl = cooperative_groups::this_cluster();
                        for (int k = 0; k < cs; ++k) c[i] += cl.map_shared_rank(hist, k)[255 - 8 * lane - i];
                    } else {
                        c[i] = hist[255 - 8 * lane - i];
                    }
                    sum += c[i];
                }
                uint32_t x = sum;
#pragma unroll
                for (int off = 1; off < 32; off <<= 1) {
                    const uint32_t y = __shfl_up_sync(0xffffffffu, x, off);
                    if (lane >= off) x += y;
                }
                uint32_t above = x - sum;
                if (above < equal && x >= equal) {   // one lane: there are at least `equal` keys
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        if (above < equal && above + c[i] >= equal) {
                            sh.digit = 255 - 8 * lane - i;
                            sh.above = above;
                            sh.in_digit = c[i];
                        }
                        above += c[i];
                    }
                }
            }
            __syncthreads();
            least |= sh.digit << shift;
            equal -= sh.above;
            const bool all = sh.in_digit == equal;   // every key with these digits stays
            __syncthreads();
            if (all) {
                equal = need;
                break;
            }
        }
    }
    // with several CTAs: the equal ones, and the kept ones, in the slices before
    uint32_t eq_before = 0, base = 0;
    if (cs > 1) {
        uint32_t gt = 0, eq = 0;
        for (int s = 0; s < spans; ++s) {
            if (spans > 1) load(s);
#pragma unroll
            for (int i = 0; i < KPT; ++i) {
                const int at = s0 + s * SPAN + i * THREADS + tid;
                gt += (need > 0 && key[i] > least) || (at < s1 && at >= old);
                eq += need > 0 && key[i] == least;
            }
        }
        gt = block_sum<NW>(sh, __reduce_add_sync(0xffffffffu, gt));
        eq = block_sum<NW>(sh, __reduce_add_sync(0xffffffffu, eq));
        eq_before = sum_before(sh, eq, cs, rank, turn);
        base = sum_before(sh, gt + min(eq, equal > eq_before ? equal - eq_before : 0u), cs, rank, turn);
    }
    uint32_t eq_run = eq_before, at_run = base;
    for (int s = 0; s < spans; ++s) {
        if (spans > 1) load(s);
        uint32_t eqm[KPT];
#pragma unroll
        for (int i = 0; i < KPT; ++i) {
            eqm[i] = __ballot_sync(0xffffffffu, need > 0 && key[i] == least);
            if (lane == 0) sh.cells[i * NW + warp] = __popc(eqm[i]);
        }
        const uint32_t eqs = scan_cells<NW>(sh, KPT * NW);
        uint32_t takes = 0;   // bit i: this thread's position i stays
#pragma unroll
        for (int i = 0; i < KPT; ++i) {
            const int at = s0 + s * SPAN + i * THREADS + tid;
            const uint32_t er = eq_run + sh.cells[i * NW + warp] + __popc(eqm[i] & ((1u << lane) - 1));
            const bool t = (need > 0 && (key[i] > least || (key[i] == least && er < equal))) || (at < s1 && at >= old);
            takes |= (uint32_t)t << i;
        }
        __syncthreads();
        uint32_t tm[KPT];
#pragma unroll
        for (int i = 0; i < KPT; ++i) {
            tm[i] = __ballot_sync(0xffffffffu, (takes >> i) & 1);
            if (lane == 0) sh.cells[i * NW + warp] = __popc(tm[i]);
        }
        const uint32_t tks = scan_cells<NW>(sh, KPT * NW);
#pragma unroll
        for (int i = 0; i < KPT; ++i)
            if ((takes >> i) & 1) {
                const int at = s0 + s * SPAN + i * THREADS + tid;
                const uint32_t to = at_run + sh.cells[i * NW + warp] + __popc(tm[i] & ((1u << lane) - 1));
                list[to] = at;
            }
        eq_run += eqs;
        at_run += tks;
        __syncthreads();
    }
    if (rank == 0) {
        if (p.out_lens && bh_i % p.c.Hkv == 0 && tid == 0) p.out_lens[b] = kept;
        if (p.kept)
            for (int i = kept + tid; i < p.keep; i += THREADS) list[i] = -1;
    }
    // the rows of this CTA's part of the list; eight threads a row, four rows in flight each
    const int r = tid & 7, end = (int)at_run;
    const Chunk *kc = reinterpret_cast<const Chunk *>(p.c.k_codes) + bh * p.c.cap * 8 + r;
    const Chunk *vc = reinterpret_cast<const Chunk *>(p.c.v_codes) + bh * p.c.cap * 8 + r;
    Chunk *ko = reinterpret_cast<Chunk *>(p.o.k_codes) + bh * p.o.cap * 8 + r;
    Chunk *vo = reinterpret_cast<Chunk *>(p.o.v_codes) + bh * p.o.cap * 8 + r;
    // threads below 2 G of a row take its parameter words (keys', then values'), the last one its weight
    const bool par = r < 2 * G;
    const uint32_t *ps = (r < G ? p.c.k_par + r : p.c.v_par + (r - G)) + bh * p.c.cap * G;
    uint32_t *pd = (r < G ? p.o.k_par + r : p.o.v_par + (r - G)) + bh * p.o.cap * G;
    constexpr int RP = THREADS / 8, U = 4;
    for (int j0 = (int)base + tid / 8; j0 < end; j0 += RP * U) {
        int src[U];
        Chunk a[U], c[U];
        uint32_t q[U];
        float x[U];
#pragma unroll
        for (int u = 0; u < U; ++u) src[u] = j0 + u * RP < end ? list[j0 + u * RP] : -1;
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (src[u] >= 0) {
                a[u] = kc[(long)src[u] * 8];
                c[u] = vc[(long)src[u] * 8];
                if (par) q[u] = ps[(long)src[u] * G];
                if (r == 7 && p.out_weights) x[u] = w[src[u]];
            }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (src[u] >= 0) {
                const long dst = j0 + u * RP;
                ko[dst * 8] = a[u];
                vo[dst * 8] = c[u];
                if (par) pd[dst * G] = q[u];
                if (r == 7 && p.out_weights) p.out_weights[bh * p.o.cap + dst] = x[u];
            }
    }
    if (cs > 1) cooperative_groups::this_cluster().sync();   // no CTA leaves while another may reach into its memory
}

}  // namespace la
