// softmax_tc.cuh — causal softmax attention over packed sequences on the
// tensor cores (bf16/fp16 inputs, head dim 32 as a padded 64, 64 or 128, fp32
// sums).
//
// A CTA holds one or two tiles ("slots") of 128 queries that read the same keys
// and values (enum Slots), and walks the keys in blocks of 128 from the
// sequence's begin to the tile's diagonal.  Per slot and block j, with
// c = scale log2(e):
//
//   S = Q K_j^T                     tcgen05, fp32 in TMEM
//   m' = max(m, rowmax S)           the reference of the exponents moves only
//                                   where c (m' - m) > kLazy, see below
//   P = 2^(c S - c m + kUp)         rounded once to the input type, in TMEM
//   l += rowsum P                   fp32, unrounded
//   O += P V_j                      tcgen05, fp32 in TMEM
//   out = O / l
//
// Moving the reference multiplies O and l by 2^(c (m - m')).  O lives in TMEM,
// so this is a read and a write of the whole accumulator; a reference that is
// up to 2^kLazy too small costs nothing (bf16 has fp32's exponents; fp16 has room
// for it above kUp), so it is moved only beyond that: after the first blocks almost
// never.
//
// The two slots (or two CTAs of one) alternate on the tensor core: while one
// slot's exponentials run, the products of the other do.
//
// What bounds it.  d 128, 16384 tokens, 16 heads on 2: 917 us, 1.2 PFLOP/s (1058 among
// other calls).  Measured when it took 910: the tensor pipe active 51% of the time; without the
// exponentials 894 us, without maximum and sum too 891, with half the products
// 784, with an eighth of the products and none of that arithmetic 513.  So it is
// neither the products nor the arithmetic alone, but the chain S -> TMEM load ->
// P -> TMEM store -> product, with a barrier at each arrow, of which two per SM
// run by turns and three do not fit TMEM.  Half blocks (S of 64 keys in two
// buffers, so that a slot's next scores are there while it works) shorten the
// chain and were slower, 1156 us for 910: a product with N = 64 reads Q as often
// as one with 128.  P handed over in halves, so that its first product runs under
// the second half's exponentials, was slower too (912 for 896).  d 64, 32 prompts
// up to 700 tokens: 46 us, of which copies and the first products before any
// softmax are a good part; for long prompts the softmax is the bound (226 us with,
// 170 us without it when this was tried: 8192 tokens, 16 heads; 200 us now).
// Computing part of the exponentials on the FMA units gained nothing: a warp's
// issue, not the special-function unit, sets the softmax's pace.
//
// CTAs stay resident and take tiles from one list (a counter in the workspace):
// the copies and the first products of the next tile run during the softmax and
// the output of the last.
//
// Warps (four per slot for the softmax, S in all, then three):
//   0 .. S - 1 softmax: a thread owns one row (TMEM lane)
//   S          the list and the TMA copies (one thread): K_0, Q, V_0, K_1, ...
//   S + 1      TMEM allocation, MMA issue (one thread)
//   S + 2      the values of a diagonal block: rows behind the sequence are
//              zeroed, and NaN or infinities taken out, since P = 0 does not
//              hide them from the product; the rows that see them get them
//              back at the end (restore_nonfinite)
//
// Order on the tensor core: tcgen05 products of one thread run in issue order,
// so S of block j + 1 may overwrite the columns that hold P of block j once
// P V_j has been issued, and a commit after S(j + 1) tells that P V_j is done
// (which the rescaling of O relies on).
#pragma once
#include <type_traits>

#include "packed.cuh"
#include "softmax_simt.cuh"
#include "tc_prefill.cuh"

namespace la {
namespace stc {

using namespace tc;

constexpr int kBlock = 128;   // keys of a block, rows of a slot

// What the slots of a CTA are: one tile of queries (two CTAs per SM), two
// consecutive tiles of one head, or the same tile of two heads.
enum Slots { kOneTile = 0, kTwoTiles = 1, kTwoHeads = 2 };
// kLazy: how far (log2) the maximum may outgrow the reference.  kUp: power of two on P, l and O (O / l drops it).
// bf16 has fp32's range.  fp16's is used up to 2^15: weights down to 2^-25 of the row's greatest are normal numbers,
// rounded relative to themselves, smaller ones to a multiple of 2^-35 of it.  (With 8 and 0 that ended at 2^-14, and
// beside a key with 2^24 of their weight the others were rounded to that step or to nothing.  In fp16, 16384 tokens,
// 16 heads on 2: 920 us with 4 and 11, 923 with 8 and 7, 930 with 2 and 13.)
template <typename InT> constexpr float kLazy = std::is_same<InT, f16>::value ? 4.f : 8.f;
template <typename InT> constexpr float kUp = std::is_same<InT, f16>::value ? 11.f : 0.f;

template <int D, int MODE> struct Cfg {
    static constexpr int SLOTS = MODE == kOneTile ? 1 : 2;
    static constexpr int THREADS = SLOTS == 1 ? 256 : 384;
    static constexpr int TMA_WARP = 4 * SLOTS, MMA_WARP = TMA_WARP + 1, SCRUB_WARP = TMA_WARP + 2;
    static constexpr int KB = D / 64;                  // 128-byte boxes per row
    static constexpr int BOXB = kBlock * 128;
    static constexpr int TILE = kBlock * D * 2;
    // K and V tiles in flight: all the shared memory there is
    static constexpr int NST = SLOTS == 2 ? 5 : D == 128 ? 2 : 5;
    static_assert(D == 128 || SLOTS == 1, "two slots: d 128 only");
    static constexpr int OFF_Q = 0;
    static constexpr int OFF_KV = SLOTS * TILE;
    static constexpr int OFF_BAR = OFF_KV + NST * TILE;
    // barriers: Q of a slot full / empty, ring stages full / empty, S, P, O of a slot full, O of a slot empty
    static constexpr int B_Q = 0, B_Q_EMPTY = 2, B_KV_FULL = 4, B_KV_EMPTY = B_KV_FULL + NST, B_S = B_KV_EMPTY + NST;
    static constexpr int B_P = B_S + 2, B_O = B_P + 2, B_O_EMPTY = B_O + 2;
    // A diagonal block's values have full barriers of their own (by turns; more
    // than can be in the ring at once), as the scrub warp does not follow the
    // ring's phases; and one each for "scrubbed".
    static constexpr int B_VD = B_O_EMPTY + 2, B_CLEAN = B_VD + 4;
    static constexpr int B_WORK = B_CLEAN + 4, B_WORK_EMPTY = B_WORK + 4;   // the list of tiles
    static constexpr int B_DRAIN = B_WORK_EMPTY + 4;
    static constexpr int NBAR = B_DRAIN + 1;
    static constexpr int OFF_TMEM = OFF_BAR + NBAR * 8;
    static constexpr int OFF_ABORT = OFF_TMEM + 4;
    static constexpr int OFF_WORK = (OFF_ABORT + 4 + 15) / 16 * 16;   // [4] Work
    static constexpr int OFF_FLAG = OFF_WORK + 4 * 16;                // [4][2] ints: a diagonal block held NaN or infinities
    static constexpr int SMEM = OFF_FLAG + 4 * 8 + 1024;              // + alignment
    // TMEM: S / P of slot s at 128 s, O behind them (two CTAs of one slot each share the 512 columns)
    static constexpr int T_S = 0, T_O = 128 * SLOTS, TMEM_COLS = 256 * SLOTS;
    static_assert(SMEM <= (SLOTS == 1 ? 115712 : 232448), "shared memory");
};

// One tile of the list: a sequence's tokens, the tile's first, its (first) head; head < 0 ends the list.
struct Work {
    int begin, end, q0, head;
};

struct Params {
    void *out;
    const int32_t *cu;
    long o_hs, o_ts;
    int H, group, N, n_seq, tiles;
    int cols;      // the tensors' head dim (32: the copies fill channels 32 .. 63 of a d 64 tile with zeros)
    float scale_log2;
    int *status;   // [0], [1] the status word, [2] the next tile
    unsigned long long wait_ns;
};

__device__ __forceinline__ uint64_t pack2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float &a, float &b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

template <typename InT> __device__ __forceinline__ uint32_t pack16(float lo, float hi) {
    if constexpr (std::is_same<InT, bf16>::value) return pack_bf16x2(lo, hi);
    else return pack_f16x2(lo, hi);
}

// x * 0 + acc for a packed pair: NaN stays behind for any NaN or infinity.
template <typename InT> __device__ __forceinline__ uint32_t probe2(uint32_t x, uint32_t acc) {
    uint32_t r;
    if constexpr (std::is_same<InT, bf16>::value) asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(x), "r"(0u), "r"(acc));
    else asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(x), "r"(0u), "r"(acc));
    return r;
}
template <typename InT> __device__ __forceinline__ uint32_t finite_or_zero2(uint32_t x) {
    constexpr uint32_t E = std::is_same<InT, bf16>::value ? 0x7F80u : 0x7C00u;
    if ((x & E) == E) x &= 0xFFFF0000u;
    if (((x >> 16) & E) == E) x &= 0x0000FFFFu;
    return x;
}

// A diagonal block's value tile [KB boxes][128 rows][128 B]: rows at or past n
// are zeroed, NaN and infinities become 0 (returns whether there were any).
// One warp.
template <typename InT, int TILE> __device__ __forceinline__ bool scrub_values(uint8_t *tile, int n, int lane) {
    constexpr int CH = TILE / 16;   // 16-byte chunks; chunk i of box b, row r: b * 1024 + r * 8 + i
    uint32_t acc = 0u;
#pragma unroll 8
    for (int i = lane; i < CH; i += 32) {
        uint4 *p = reinterpret_cast<uint4 *>(tile) + i;
        if ((i & 1023) / 8 >= n) {
            *p = make_uint4(0u, 0u, 0u, 0u);
        } else {
            const uint4 x = *p;
            acc = probe2<InT>(x.x, acc);
            acc = probe2<InT>(x.y, acc);
            acc = probe2<InT>(x.z, acc);
            acc = probe2<InT>(x.w, acc);
        }
    }
    constexpr uint32_t E = std::is_same<InT, bf16>::value ? 0x7F80u : 0x7C00u;
    const bool bad = __any_sync(0xffffffffu, (acc & E) == E || ((acc >> 16) & E) == E);
    if (bad) {
        for (int i = lane; i < CH; i += 32) {
            uint4 *p = reinterpret_cast<uint4 *>(tile) + i;
            const uint4 x = *p;
            *p = make_uint4(finite_or_zero2<InT>(x.x), finite_or_zero2<InT>(x.y), finite_or_zero2<InT>(x.z),
                            finite_or_zero2<InT>(x.w));
        }
    }
    return bad;
}

// Adds the NaN and infinities of values j0 .. min(j1, row) to this thread's
// row of O (p > 0 times infinity is infinity).  Rare; whole warp.
template <typename InT, int D>
__device__ __forceinline__ void restore_nonfinite(uint32_t t_o, const InT *v, long ts, int j0, int j1, int row, int cols) {
    for (int cb = 0; cb < cols / 32; ++cb) {
        uint32_t u[32];
        tmem_ld32(t_o + cb * 32, u);
        tmem_ld_wait();
        for (int j = j0; j < j1; ++j) {
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                const float x = to_f32<InT>(v[(long)j * ts + cb * 32 + i]);
                if (j <= row && !isfinite(x)) u[i] = __float_as_uint(__uint_as_float(u[i]) + x);
            }
        }
        tmem_st32(t_o + cb * 32, u);
    }
    tmem_st_wait();
}

// mbar_wait without a call: a kernel that redistributes its registers may not
// call functions.
__device__ __forceinline__ bool wait_bar(uint64_t *bar, uint32_t parity, const AbortCtx &ab, int code) {
    const uint32_t hint = ab.hint();
    if (mbar_try_wait(bar, parity, hint)) return true;
    const uint64_t t0 = globaltimer_ns();
    while (!mbar_try_wait(bar, parity, hint)) {
        if (*ab.flag) return false;
        if (globaltimer_ns() - t0 >= ab.limit_ns) {
            raise_abort(ab, code);
            return false;
        }
    }
    return true;
}

// The same by a whole warp, with one answer for all its lanes.
__device__ __forceinline__ bool wait_warp(uint64_t *bar, uint32_t parity, const AbortCtx &ab, int code) {
    return __all_sync(0xffffffffu, wait_bar(bar, parity, ab, code));
}

// The one thread of a warp that issues for it.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

template <typename InT, typename OutT, int D, int MODE>
__global__ void __launch_bounds__(Cfg<D, MODE>::THREADS, MODE == kOneTile ? 2 : 1)
softmax_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                  const __grid_constant__ CUtensorMap tm_v, const InT *__restrict__ v_gmem, long v_hs, long v_ts,
                  const Params p) {
    using G = Cfg<D, MODE>;
    extern __shared__ uint8_t stc_smem_raw[];
    uint8_t *smem = stc_smem_raw + ((1024u - (smem_u32(stc_smem_raw) & 1023u)) & 1023u);
    uint64_t *bar = reinterpret_cast<uint64_t *>(smem + G::OFF_BAR);
    uint32_t *tmem_addr = reinterpret_cast<uint32_t *>(smem + G::OFF_TMEM);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + G::OFF_ABORT);
    volatile int *flag = reinterpret_cast<volatile int *>(smem + G::OFF_FLAG);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    AbortCtx ab{abort_flag, p.status, p.wait_ns};
    volatile Work *work = reinterpret_cast<volatile Work *>(smem + G::OFF_WORK);
    if (threadIdx.x == 0) {
        *abort_flag = 0;
        for (int i = 0; i < G::NBAR; ++i) {
            const bool soft = (i >= G::B_P && i < G::B_P + 2) || (i >= G::B_O_EMPTY && i < G::B_O_EMPTY + 2);
            const bool list = i >= G::B_WORK_EMPTY && i < G::B_WORK_EMPTY + 4;
            mbar_init(&bar[i], soft ? 4 : list ? 4 * G::SLOTS + 2 : 1);
        }
        fence_mbar_init();
    }
    if (warp == G::MMA_WARP) tmem_alloc(tmem_addr, G::TMEM_COLS);
    if (warp == G::TMA_WARP && lane == 0) {
        prefetch_tmap(&tm_q);
        prefetch_tmap(&tm_k);
        prefetch_tmap(&tm_v);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_addr;

    // blocks of the slots in a tile; the last of each is the diagonal one
    auto blocks0 = [](const Work &w) { return (w.q0 - w.begin) / kBlock + 1; };
    auto blocks1 = [&](const Work &w, int n0) {
        return MODE == kTwoHeads ? n0 : MODE == kTwoTiles && w.q0 + kBlock < w.end ? n0 + 1 : 0;
    };
    // Entry k of the list once its wait is over, or head < 0 (the end, or giving up).
    auto next_work = [&](int k, bool ready) {
        Work w{0, 0, 0, -1};
        if (ready) {
            w.begin = work[k & 3].begin;
            w.end = work[k & 3].end;
            w.q0 = work[k & 3].q0;
            w.head = work[k & 3].head;
        }
        return w;
    };

    // The softmax warps get registers of the others: of the 256 x 128 of a CTA of
    // one slot 128 x 200 + 128 x 56, of the 384 x 168 of two slots 256 x 216 +
    // 128 x 56 (never more than the CTA was launched with: an increase would wait
    // for good).  With 168 for all, two slots took 917 us for 896 (16384 tokens,
    // 16 heads on 2) and 317 for 304 (eight packed prompts) when this was tried.
    if (warp >= G::TMA_WARP) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (warp == G::TMA_WARP) {
        // ================= the list of tiles, and the copies
        if (lane == 0) {
            int it = 0, diag = 0, nq[2] = {0, 0};   // ring items, diagonal blocks, query tiles of a slot so far
            uint32_t kv_phase = 0u, last_vd = 0u;   // per stage: parity of its last ring copy; stages whose last copy was diagonal
            const int nhp = MODE == kTwoHeads ? p.H / 2 : p.H;
            const unsigned total = (unsigned)p.tiles * nhp;
            bool ok = true;
            for (int k = 0; ok; ++k) {
                // heads fastest (CTAs that run together share keys), late tiles,
                // which have the most keys, first
                Work w{0, 0, 0, -1};
                while (true) {
                    const unsigned x = atomicAdd(reinterpret_cast<unsigned *>(p.status) + 2, 1u);
                    if (x >= total) break;
                    const SeqTile t = seq_tile<MODE == kTwoTiles ? 256 : 128>(p.cu, p.n_seq, p.N, p.tiles - 1 - (int)(x / nhp));
                    if (t.q0 < t.end) {
                        w = Work{t.begin, t.end, t.q0, (int)(x % nhp) * (MODE == kTwoHeads ? 2 : 1)};
                        break;
                    }
                }
                if (k >= 4 && !wait_bar(&bar[G::B_WORK_EMPTY + (k & 3)], ((k >> 2) - 1) & 1, ab, 11)) break;
                work[k & 3].begin = w.begin;
                work[k & 3].end = w.end;
                work[k & 3].q0 = w.q0;
                work[k & 3].head = w.head;
                mbar_arrive(&bar[G::B_WORK + (k & 3)]);
                if (w.head < 0) break;
                const int n0 = blocks0(w), n1 = blocks1(w, n0), nb = max(n0, n1), hk = w.head / p.group;
                for (int i = 0; i < 2 * nb; ++i, ++it) {
                    const int st = it % G::NST, use = it / G::NST;
                    if (use > 0 && !(ok = wait_bar(&bar[G::B_KV_EMPTY + st], (use - 1) & 1, ab, 1))) break;
                    const bool vd = (i & 1) && (i >> 1) >= n0 - 1;
                    uint64_t *full = &bar[vd ? G::B_VD + (diag & 3) : G::B_KV_FULL + st];
                    if (vd) {
                        ++diag;
                        last_vd |= 1u << st;
                    } else {
                        kv_phase ^= 1u << st;
                        last_vd &= ~(1u << st);
                    }
                    mbar_expect_tx(full, G::TILE);
                    for (int b = 0; b < G::KB; ++b)
                        tma_load_3d(smem + G::OFF_KV + st * G::TILE + b * G::BOXB, (i & 1) ? &tm_v : &tm_k, full, 64 * b,
                                    w.begin + (i >> 1) * kBlock, hk);
                    if (i > 0) continue;
                    // the queries behind the first keys: their places free later than the ring's
#pragma unroll
                    for (int s = 0; s < G::SLOTS; ++s) {
                        if ((s == 1 && n1 == 0) || !ok) continue;
                        if (nq[s] > 0 && !(ok = wait_bar(&bar[G::B_Q_EMPTY + s], (nq[s] - 1) & 1, ab, 12))) continue;
                        ++nq[s];
                        mbar_expect_tx(&bar[G::B_Q + s], G::TILE);
                        for (int b = 0; b < G::KB; ++b)
                            tma_load_3d(smem + G::OFF_Q + s * G::TILE + b * G::BOXB, &tm_q, &bar[G::B_Q + s], 64 * b,
                                        MODE == kTwoTiles ? w.q0 + s * kBlock : w.q0, MODE == kTwoHeads ? w.head + s : w.head);
                    }
                    if (!ok) { ++it; break; }
                }
            }
            // every copy issued has completed before the CTA exits (each is waited
            // for by its reader too, unless that gave up)
            volatile int never = 0;
            AbortCtx timed{&never, nullptr, kDrainLimitNs};
            for (int s = 0; s < G::SLOTS; ++s)
                if (nq[s] > 0) wait_bar(&bar[G::B_Q + s], (nq[s] - 1) & 1, timed, 0);
            for (int st = 0; st < min(it, G::NST); ++st)
                if (!((last_vd >> st) & 1)) wait_bar(&bar[G::B_KV_FULL + st], ((kv_phase >> st) & 1) ^ 1, timed, 0);
            for (int d = max(0, diag - 4); d < diag; ++d) wait_bar(&bar[G::B_VD + (d & 3)], (d >> 2) & 1, timed, 0);
        }
    } else if (warp == G::MMA_WARP) {
        // The whole warp goes through the waits and the index arithmetic, so that
        // the descriptors are uniform values, ready before the last wait; one
        // thread issues the products and the commits.  Before its commits, which let
        // others go on, a vote makes sure that every lane is through its waits: a lane
        // left behind by two phases would wait for one that has passed.  The vote runs
        // under the products (16384 tokens, 16 heads on 2: 917 us; ahead of them 930, the
        // waits in one thread alone 957).
        constexpr bool BF = std::is_same<InT, bf16>::value;
        constexpr uint32_t ID_S = BF ? idesc_bf16(128, 128, false, false) : idesc_f16(128, 128, false, false);
        constexpr uint32_t ID_O = BF ? idesc_bf16(128, D, false, true) : idesc_f16(128, D, false, true);
        const uint32_t sb = smem_u32(smem);
        const bool leader = elect_one();
        // bits: parity of a stage's next ring copy; of a slot's next tile and block; whether it had a tile
        uint32_t kv_phase = 0u, tile_phase = 0u, block_phase = 0u, had = 0u;
        int it0 = 0, diag = 0;   // ring items, diagonal blocks so far
        bool ok = true;
        auto ring_full = [&](int st) {
            const bool f = wait_bar(&bar[G::B_KV_FULL + st], (kv_phase >> st) & 1, ab, 2);
            kv_phase ^= 1u << st;
            return f;
        };
        for (int k = 0; ok; ++k) {
            const Work w = next_work(k, wait_warp(&bar[G::B_WORK + (k & 3)], (k >> 2) & 1, ab, 10));
            if (w.head < 0) break;
            __syncwarp();   // every lane has read the entry
            if (leader) mbar_arrive(&bar[G::B_WORK_EMPTY + (k & 3)]);
            const int n0 = blocks0(w), n1 = blocks1(w, n0), nb = max(n0, n1);
            // step j: per slot P V_j, then S of block j + 1
            int sv = (it0 + G::NST - 1) % G::NST, sk = it0 % G::NST;   // stages of V_j and K_{j+1}
#pragma unroll 1
            for (int j = -1; j < nb; ++j) {
                if (j >= n0 - 1 && j >= 0) {
                    ok = wait_bar(&bar[G::B_CLEAN + (diag & 3)], (diag >> 2) & 1, ab, 4);
                    ++diag;
                } else if (j >= 0) {
                    ok = ring_full(sv);
                }
                if (ok && j + 1 < nb) ok = ring_full(sk);
                const uint64_t bv = sdesc_sw128(sb + G::OFF_KV + sv * G::TILE, G::BOXB, 1024);
                const uint64_t bk = sdesc_sw128(sb + G::OFF_KV + sk * G::TILE, 16, 1024);
#pragma unroll
                for (int s = 0; s < G::SLOTS; ++s) {
                    const int n = s ? n1 : n0;
                    if (n == 0 || j >= n) continue;   // (one slot at least goes on, to the vote on the waits above)
                    const uint32_t to = tmem + G::T_O + 128 * s, ts = tmem + G::T_S + 128 * s;
                    if (j >= 0) {
                        // (a new tile's first product overwrites O: its last one has been read out)
                        if (j == 0 && ((had >> s) & 1))
                            ok = ok && wait_bar(&bar[G::B_O_EMPTY + s], ((tile_phase >> s) & 1) ^ 1, ab, 13);
                        ok = ok && wait_bar(&bar[G::B_P + s], (block_phase >> s) & 1, ab, 5);
                        block_phase ^= 1u << s;
                    } else {
                        ok = ok && wait_bar(&bar[G::B_Q + s], (tile_phase >> s) & 1, ab, 3);
                    }
                    tc_fence_after();
                    if (leader && ok) {
                        if (j >= 0) {
#pragma unroll
                            for (int kk = 0; kk < kBlock / 16; ++kk)
                                mma_ts(to, ts + kk * 8, bv + (uint64_t)((kk * 2048) >> 4), ID_O, (j > 0 || kk > 0) ? 1u : 0u);
                        }
                        if (j + 1 < n) {
                            const uint64_t a = sdesc_sw128(sb + G::OFF_Q + s * G::TILE, 16, 1024);
#pragma unroll
                            for (int kk = 0; kk < D / 16; ++kk) {
                                const uint32_t off = ((kk >> 2) * G::BOXB + (kk & 3) * 32) >> 4;
                                mma_ss(ts, a + off, bk + off, ID_S, kk > 0);
                            }
                        }
                    }
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    if (leader) {
                        if (j == n - 1) mma_commit(&bar[G::B_O + s]);
                        if (j + 1 < n) {
                            mma_commit(&bar[G::B_S + s]);
                            if (j + 2 == n) mma_commit(&bar[G::B_Q_EMPTY + s]);
                        }
                    }
                    if (j == n - 1) {
                        tile_phase ^= 1u << s;
                        had |= 1u << s;
                    }
                }
                if (!ok) break;
                if (leader) {
                    if (j >= 0) mma_commit(&bar[G::B_KV_EMPTY + sv]);
                    if (j + 1 < nb) mma_commit(&bar[G::B_KV_EMPTY + sk]);
                }
                sv = sk + 1 == G::NST ? 0 : sk + 1;
                sk = sv + 1 == G::NST ? 0 : sv + 1;
            }
            it0 += 2 * nb;
        }
        // every product issued has completed before TMEM is freed
        volatile int never = 0;
        AbortCtx timed{&never, nullptr, kDrainLimitNs};
        __syncwarp();
        if (leader) {
            mma_commit(&bar[G::B_DRAIN]);
            wait_bar(&bar[G::B_DRAIN], 0, timed, 0);
        }
        __syncwarp();
    } else if (warp == G::SCRUB_WARP) {
        int it0 = 0, diag = 0;
        bool ok = true;
        for (int k = 0; ok; ++k) {
            const Work w = next_work(k, wait_warp(&bar[G::B_WORK + (k & 3)], (k >> 2) & 1, ab, 10));
            if (w.head < 0) break;
            const int n0 = blocks0(w), n1 = blocks1(w, n0);
            for (int b = 0; b < (n1 > n0 ? 2 : 1); ++b, ++diag) {
                const int j = n0 - 1 + b, i = it0 + 2 * j + 1;
                ok = wait_warp(&bar[G::B_VD + (diag & 3)], (diag >> 2) & 1, ab, 6);
                if (!ok) break;
                const int n = w.end - (w.begin + j * kBlock);   // rows of the sequence
                const bool bad = scrub_values<InT, G::TILE>(smem + G::OFF_KV + (i % G::NST) * G::TILE, n, lane);
                if (lane == 0) flag[(k & 3) * 2 + b] = bad;
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar[G::B_CLEAN + (diag & 3)]);
            }
            it0 += 2 * max(n0, n1);
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar[G::B_WORK_EMPTY + (k & 3)]);
        }
    }
    } else {
        if constexpr (G::SLOTS == 1) asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
        else asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
        // softmax of slot s: thread = row
        const int s = warp >> 2, q = warp & 3;
        const uint32_t lane_base = (uint32_t)(q * 32) << 16;
        const uint32_t t_s = tmem + lane_base + G::T_S + 128 * s, t_o = tmem + lane_base + G::T_O + 128 * s;
        const int r = q * 32 + lane;
        const float c = p.scale_log2;
        int nt = 0, np = 0;   // this slot's tiles and blocks so far
        bool ok = true;
        for (int k = 0; ok; ++k) {
            const Work w = next_work(k, wait_warp(&bar[G::B_WORK + (k & 3)], (k >> 2) & 1, ab, 10));
            if (w.head < 0) break;
            const int n0 = blocks0(w), n1 = blocks1(w, n0), n = s ? n1 : n0;
            const int q0 = MODE == kTwoTiles ? w.q0 + s * kBlock : w.q0;
            float m = -INFINITY, l = 0.f;
            for (int j = 0; j < n; ++j, ++np) {
                ok = wait_warp(&bar[G::B_S + s], np & 1, ab, 7);
                if (!ok) break;
                tc_fence_after();
                uint32_t u[4][32];
#pragma unroll
                for (int i = 0; i < 4; ++i) tmem_ld32(t_s + 32 * i, u[i]);
                tmem_ld_wait();
                if (j == n - 1) {
                    // diagonal block: keys up to the row's own and within the sequence
                    // (rows behind the sequence see its last key: their results are dropped)
                    const int last = min(r, w.end - 1 - q0);
#pragma unroll
                    for (int i = 0; i < 128; ++i)
                        if (i > last) u[i / 32][i % 32] = 0xff800000u;
                }
                float mx[4] = {m, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int i = 0; i < 128; ++i) mx[i & 3] = fmaxf(mx[i & 3], __uint_as_float(u[i / 32][i % 32]));
                const float mn = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                if (j == 0) {
                    m = mn;
                } else {
                    const bool move = (mn - m) * c > kLazy<InT>;   // (m = -inf: infinite; mn = -inf: NaN, false)
                    if (__any_sync(0xffffffffu, move)) {
                        const float f = move ? ex2_approx((m - mn) * c) : 1.f;
#pragma unroll 1
                        for (int cb = 0; cb < D / 32; ++cb) {
                            uint32_t o[32];
                            tmem_ld32(t_o + cb * 32, o);
                            tmem_ld_wait();
#pragma unroll
                            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                            tmem_st32(t_o + cb * 32, o);
                        }
                        l *= f;
                        m = move ? mn : m;
                    }
                }
                const float neg = m == -INFINITY ? 0.f : fmaf(-m, c, kUp<InT>);
                const uint64_t c2 = pack2(c, c), n2 = pack2(neg, neg);
                uint64_t sum[2] = {0ull, 0ull};
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    uint32_t pw[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        const int e = g * 64 + 2 * i;
                        float a, b;
                        unpack2(fma2(pack2(__uint_as_float(u[e / 32][e % 32]), __uint_as_float(u[e / 32][e % 32 + 1])), c2, n2), a, b);
                        a = ex2_approx(a);
                        b = ex2_approx(b);
                        sum[i & 1] = add2(sum[i & 1], pack2(a, b));
                        pw[i] = pack16<InT>(a, b);
                    }
                    tmem_st32(t_s + 32 * g, pw);
                }
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar[G::B_P + s]);
                float s0, s1, s2, s3;
                unpack2(sum[0], s0, s1);
                unpack2(sum[1], s2, s3);
                l += (s0 + s1) + (s2 + s3);
            }
            if (!ok) break;
            if (n > 0) {
                ok = wait_warp(&bar[G::B_O + s], nt & 1, ab, 8);
                if (!ok) break;
                ++nt;
                tc_fence_after();
                const int row = q0 + r;
                for (int b = 0; b < (n1 > n0 ? 2 : 1); ++b)
                    if (flag[(k & 3) * 2 + b]) {
                        const int j0 = w.begin + (n0 - 1 + b) * kBlock;
                        restore_nonfinite<InT, D>(t_o, v_gmem + (w.head / p.group) * v_hs, v_ts, j0, min(j0 + kBlock, w.end), row,
                                                  p.cols);
                    }
                // O / l, from the registers to the thread's own row (whole 32-byte
                // sectors; the query tile is already being filled for the next tile)
                const float inv = 1.f / l;
                OutT *out = (OutT *)p.out + (long)(MODE == kTwoHeads ? w.head + s : w.head) * p.o_hs + (long)row * p.o_ts;
#pragma unroll
                for (int cb = 0; cb < D / 32; ++cb) {
                    uint32_t o[32];
                    __syncwarp();
                    tmem_ld32(t_o + cb * 32, o);
                    tmem_ld_wait();
                    if (cb == D / 32 - 1) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&bar[G::B_O_EMPTY + s]);
                    }
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * inv);
                    if (row >= w.end || cb * 32 >= p.cols) {
                        // behind the sequence: not a row of it; behind the channels
                    } else if constexpr (sizeof(OutT) == 2) {
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            uint4 v;
                            uint32_t *vp = reinterpret_cast<uint32_t *>(&v);
#pragma unroll
                            for (int y = 0; y < 4; ++y)
                                vp[y] = pack16<InT>(__uint_as_float(o[8 * x + 2 * y]), __uint_as_float(o[8 * x + 2 * y + 1]));
                            reinterpret_cast<uint4 *>(out + cb * 32)[x] = v;
                        }
                    } else {
#pragma unroll
                        for (int x = 0; x < 8; ++x)
                            reinterpret_cast<uint4 *>(out + cb * 32)[x] = make_uint4(o[4 * x], o[4 * x + 1], o[4 * x + 2], o[4 * x + 3]);
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar[G::B_WORK_EMPTY + (k & 3)]);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == G::MMA_WARP) {
        tc_fence_after();
        tmem_dealloc(tmem, G::TMEM_COLS);
    }
}

}  // namespace stc
}  // namespace la
