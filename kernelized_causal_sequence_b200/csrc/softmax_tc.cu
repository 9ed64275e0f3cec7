// softmax_tc.cu — tensor maps and launch of the tensor-core softmax prefill.
#include <cudaTypedefs.h>

#include <mutex>

#include "launch.h"
#include "plan.h"
#include "softmax_tc.cuh"
#include "softmax_tc.h"

namespace la {

namespace {

PFN_cuTensorMapEncodeTiled_v12000 encode() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    });
    return fn;
}

// [heads][N][d] with strides, boxes of 64 channels x 128 rows, 128-byte
// swizzle, zeros past N and past d
bool map16(CUtensorMap *m, const void *base, la_dtype dt, int heads, int N, int d, long hs, long ts) {
    auto enc = encode();
    if (!enc) return false;
    cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)N, (cuuint64_t)heads};
    cuuint64_t strides[2] = {(cuuint64_t)ts * 2, (cuuint64_t)hs * 2};
    cuuint32_t box[3] = {64, 128, 1};
    cuuint32_t one[3] = {1, 1, 1};
    return enc(m, dt == LA_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
               const_cast<void *>(base), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename InT, typename OutT, int D, int MODE>
la_status run(const SoftmaxParams &sp, la_dtype dt, int d, int *status, unsigned long long wait_ns, cudaStream_t st) {
    CUtensorMap mq, mk, mv;
    const int Hk = sp.H / sp.group;
    if (!map16(&mq, sp.q, dt, sp.H, sp.N, d, sp.q_hs, sp.q_ts) || !map16(&mk, sp.k, dt, Hk, sp.N, d, sp.k_hs, sp.k_ts) ||
        !map16(&mv, sp.v, dt, Hk, sp.N, d, sp.v_hs, sp.v_ts))
        return cuda_fail_msg("cuTensorMapEncodeTiled", "tensor map encoding failed");
    stc::Params p;
    p.out = sp.out; p.cu = sp.cu; p.o_hs = sp.o_hs; p.o_ts = sp.o_ts;
    p.H = sp.H; p.group = sp.group; p.N = sp.N; p.n_seq = sp.n_seq;
    p.tiles = seq_tiles(sp.N, sp.n_seq, MODE == stc::kTwoTiles ? 256 : 128);
    p.cols = d; p.scale_log2 = sp.scale_log2; p.status = status; p.wait_ns = wait_ns;
    const long tiles = (long)p.tiles * (MODE == stc::kTwoHeads ? sp.H / 2 : sp.H);
    if (tiles > 0x7fffffffL) return LA_ERR_UNSUPPORTED;
    using G = stc::Cfg<D, MODE>;
    const long resident = kNumSMs * (G::SLOTS == 1 ? 2 : 1);
    const long grid = tiles < resident ? tiles : resident;
    return launch_kernel(stc::softmax_tc_kernel<InT, OutT, D, MODE>, dim3((unsigned)grid), dim3(G::THREADS), G::SMEM, st,
                         false, "softmax tensor-core launch", mq, mk, mv, (const InT *)sp.v, sp.v_hs, sp.v_ts, p);
}

// Which slots (us, 16 query heads; one tile / two slots; S sequences of L tokens):
//   d 128, 4 key heads   64 x 200: 66 / 62, 32 x 512: 84 / 80, 16 x 1000: 112 / 105, 8 x 2048: 168 / 155, 1 x 8192: 266 / 251
//   d 128, 16 key heads  64 x 200: 64 / 66, 32 x 512: 86 / 85, 16 x 1000: 117 / 110, 8 x 2048: 175 / 160, 1 x 8192: 275 / 258
//   d 128, 1 x 4096      80 / 78 and 82 / 80; 1 x 2048: 41 / 43 and 41 / 45 (too few tiles of two slots)
//   d 64                 one tile up to 8192 tokens (1 x 8192: 200 / 209 when two were built): the softmax bounds it there
// (N stands for the lengths, which are on the device; a buffer longer than its batch counts as longer sequences.)  Two slots read a key and value tile once for both, which counts where the
// products' operands bound it; one tile leaves less empty and more to overlap.
template <typename InT, typename OutT, int D>
la_status by_slots(const SoftmaxParams &sp, la_dtype dt, int d, int *status, unsigned long long wait_ns, cudaStream_t st) {
    if constexpr (D == 128) {
        if ((long)sp.N > 256L * sp.n_seq && 2L * seq_tiles(sp.N, sp.n_seq, 256) * sp.H >= 3L * kNumSMs) {
            if (sp.group % 2 == 0) return run<InT, OutT, D, stc::kTwoHeads>(sp, dt, d, status, wait_ns, st);
            return run<InT, OutT, D, stc::kTwoTiles>(sp, dt, d, status, wait_ns, st);
        }
    }
    return run<InT, OutT, D, stc::kOneTile>(sp, dt, d, status, wait_ns, st);
}

template <typename InT, typename OutT>
la_status by_shape(const SoftmaxParams &sp, la_dtype dt, int d, int *status, unsigned long long wait_ns, cudaStream_t st) {
    return d == 128 ? by_slots<InT, OutT, 128>(sp, dt, d, status, wait_ns, st)
                    : by_slots<InT, OutT, 64>(sp, dt, d, status, wait_ns, st);
}

}  // namespace

la_status softmax_tc(const SoftmaxParams &sp, la_dtype in, la_dtype out, int d, int *status,
                     unsigned long long wait_ns, cudaStream_t st) {
    if (in == LA_BF16)
        return out == LA_F32 ? by_shape<bf16, float>(sp, in, d, status, wait_ns, st)
                             : by_shape<bf16, bf16>(sp, in, d, status, wait_ns, st);
    return out == LA_F32 ? by_shape<f16, float>(sp, in, d, status, wait_ns, st)
                         : by_shape<f16, f16>(sp, in, d, status, wait_ns, st);
}

}  // namespace la
