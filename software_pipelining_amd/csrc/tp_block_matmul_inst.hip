// The product's kernels for one pair of 8-bit types (one compilation each).
#include "tp_block_matmul.hpp"

namespace tp {
namespace {

using Fn = void (*)(MatmulParams);

int launch(Fn fn, dim3 grid, int threads, int lds, const MatmulParams &p, void *stream)
{
    MatmulParams args = p;
    void *kargs[] = {&args};
    return (int)hipLaunchKernel(reinterpret_cast<const void *>(fn), grid, dim3((uint32_t)threads), kargs,
                                (size_t)lds, (hipStream_t)stream);
}

template <bool Wide, bool Square, int Shape, int BM, int BN, int GM, int GN>
int launch_tile(const MatmulPlan &plan, const MatmulParams &p, void *stream)
{
    constexpr int Stages = matmul_stages(Shape);
    using S = dev::Tile<BM, BN, GM, GN, Stages, Wide ? 4 : 8>;
    return launch(&dev::block_matmul_kernel<TP_INST_FA, TP_INST_FB, Wide, Square, BM, BN, GM, GN, Stages>,
                  dim3((uint32_t)plan.grid), S::threads, S::lds_bytes, p, stream);
}

template <bool Wide, bool Square, int MT, int Slots>
int launch_skinny(const MatmulParams &p, void *stream)
{
    return launch(&dev::block_matmul_skinny_kernel<TP_INST_FA, TP_INST_FB, Wide, Square, MT, Slots>,
                  dim3((uint32_t)p.tiles_n, (uint32_t)p.splits), 64 * kSkinnyWaves,
                  dev::Skinny<MT, Slots>::lds_bytes, p, stream);
}

template <bool Wide, bool Square>
int launch_shape(const MatmulPlan &plan, const MatmulParams &p, void *stream)
{
    switch (plan.shape) {
    case kMatmulSkinny:
        switch (plan.tile_m) {
        case 16:
            return plan.stages == 2 ? launch_skinny<Wide, Square, 1, 2>(p, stream)
                                    : launch_skinny<Wide, Square, 1, 1>(p, stream);
        case 32: return launch_skinny<Wide, Square, 2, 1>(p, stream);
        case 48: return launch_skinny<Wide, Square, 3, 1>(p, stream);
        default: return launch_skinny<Wide, Square, 4, 1>(p, stream);
        }
    case kMatmul64:
        return launch_tile<Wide, Square, kMatmul64, 64, 64, 1, 2>(plan, p, stream);
    case kMatmul128:
        return launch_tile<Wide, Square, kMatmul128, 128, 128, 2, 2>(plan, p, stream);
    case kMatmul128x256:
        return launch_tile<Wide, Square, kMatmul128x256, 128, 256, 2, 4>(plan, p, stream);
    default:
        if constexpr (Wide)
            return (int)hipErrorInvalidValue;    // matmul_plan has no such plan
        else
            return launch_tile<Wide, Square, kMatmul256, 256, 256, 4, 2>(plan, p, stream);
    }
}

}  // namespace

int TP_INST_FN(const MatmulPlan &plan, const MatmulParams &p, int square, void *stream)
{
    if (matmul_wide(p.out_type))
        return square ? launch_shape<true, true>(plan, p, stream) : launch_shape<true, false>(plan, p, stream);
    return square ? launch_shape<false, true>(plan, p, stream) : launch_shape<false, false>(plan, p, stream);
}

}  // namespace tp
