// bwd_main.cu -- the launch of the gradient kernels: the CTAs of dk and dv and those of dq, which
// need nothing of each other; the kind that goes out second fills the SMs as the first
// runs out of work.
#include "bwd_kv.cuh"
#include "bwd_q.cuh"

namespace skv {
namespace bwd {

// PARTS: fp16 numbers that hold p and ds: one each, two of dq's ds, two of all.
template <int D, int PARTS>
__global__ void __launch_bounds__(kThreads, 1)
    splitkv_bwd_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap to,
                       const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                       const __grid_constant__ MainArgs kv_args, const __grid_constant__ MainArgs q_args, int kv_ctas, int q_first)
{
    extern __shared__ uint8_t smem_raw[];
    const int q_ctas = gridDim.x - kv_ctas, first = q_first ? q_ctas : kv_ctas;
    const bool second = blockIdx.x >= first;
    const int b = second ? blockIdx.x - first : blockIdx.x;
    if (second != (q_first != 0)) {
        const int units = q_ctas / q_args.pieces;
        q::run<D, PARTS != kOnePart>(tq, to, tk, tv, q_args, b % units, b / units, smem_raw);
    } else {
        const int units = kv_ctas / kv_args.pieces;
        kv::run<D, PARTS == kTwoParts>(tq, to, tk, tv, kv_args, b % units, b / units, smem_raw);
    }
}

template <int D, int PARTS>
static int launch_t(skv_handle *h, const CUtensorMap &mq, const CUtensorMap &mo, const CUtensorMap &mk, const CUtensorMap &mv,
                    const MainArgs &kv_args, const MainArgs &q_args, bool q_first, cudaStream_t st)
{
    static KernelAttrCache attr;
    constexpr int kStatic = 1792;                          // at most, of both: 1.7 KB as built
    static_assert(q::Lay<128>::kBytes + kStatic <= 227 * 1024 && kv::Lay<128>::kBytes + kStatic <= 227 * 1024, "shared memory per CTA");
    constexpr int smem = kv::Lay<D>::kBytes > q::Lay<D>::kBytes ? kv::Lay<D>::kBytes : q::Lay<D>::kBytes;
    const cudaError_t e = kernel_smem_optin(attr, reinterpret_cast<const void *>(splitkv_bwd_kernel<D, PARTS>), smem, kThreads, nullptr);
    if (e != cudaSuccess) return cuda_fail(h, e, "cudaFuncSetAttribute(gradients)");
    const int64_t units = static_cast<int64_t>(kv_args.g.Hk) * kv_args.g.groups;
    const int64_t kv_ctas = kv_args.out0 ? units * kv_args.g.KT * kv_args.pieces : 0;
    const int64_t q_ctas = q_args.out0 ? units * q_args.g.QT * q_args.pieces : 0;
    if (kv_ctas + q_ctas > INT32_MAX) return fail(h, SKV_EUNSUPPORTED, "too many tiles for one launch");
    splitkv_bwd_kernel<D, PARTS><<<static_cast<unsigned>(kv_ctas + q_ctas), kThreads, smem, st>>>(mq, mo, mk, mv, kv_args, q_args,
                                                                                           static_cast<int>(kv_ctas), q_first);
    return cuda_fail(h, cudaGetLastError(), "gradient kernel launch");
}

template <int D>
static int launch_d(skv_handle *h, const CUtensorMap &mq, const CUtensorMap &mo, const CUtensorMap &mk, const CUtensorMap &mv,
                    const MainArgs &kv_args, const MainArgs &q_args, bool q_first, int parts, cudaStream_t st)
{
    if (parts == kOnePart) return launch_t<D, kOnePart>(h, mq, mo, mk, mv, kv_args, q_args, q_first, st);
    if (parts == kTwoOfDq) return launch_t<D, kTwoOfDq>(h, mq, mo, mk, mv, kv_args, q_args, q_first, st);
    return launch_t<D, kTwoParts>(h, mq, mo, mk, mv, kv_args, q_args, q_first, st);
}

int launch_main(skv_handle *h, const CUtensorMap &mq, const CUtensorMap &mo, const CUtensorMap &mk, const CUtensorMap &mv,
                const MainArgs &kv_args, const MainArgs &q_args, bool q_first, int parts, cudaStream_t st)
{
    return kv_args.g.D == 64 ? launch_d<64>(h, mq, mo, mk, mv, kv_args, q_args, q_first, parts, st)
                             : launch_d<128>(h, mq, mo, mk, mv, kv_args, q_args, q_first, parts, st);
}

}  // namespace bwd
}  // namespace skv
