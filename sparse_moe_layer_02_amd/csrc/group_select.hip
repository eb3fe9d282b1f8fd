// group_select.hip - top-k selection with expert groups and softmax scores
// (group_dev.h), one wavefront per token.
#include "common.h"
#include "group_dev.h"
#include "kernels.h"

#pragma clang fp contract(off)

namespace moe {

template <int KPL>
__global__ __launch_bounds__(256) void group_topk_kernel(SelectArgs a, GroupArgs g) {
    __shared__ uint32_t keys[4][KPL * WAVE];
    const int wave = wave_index(), t = blockIdx.x * 4 + wave;
    if (t >= a.T) return;
    group_topk_token<KPL>(a.logits + (size_t)t * a.E, a.bias, a.E, a.k, a.score, a.route_scale, g, keys[wave],
                          a.topk_idx + (size_t)t * a.k, a.topk_w + (size_t)t * a.k);
}

hipError_t launch_group_topk(const SelectArgs& a, const GroupArgs& g, hipStream_t st, const KTime& kt) {
    const int kpl = (a.E + WAVE - 1) / WAVE;
    const dim3 grid((a.T + 3) / 4);
    if (kpl <= 1) launch_kernel(group_topk_kernel<1>, grid, 256, st, kt, a, g);
    else if (kpl <= 2) launch_kernel(group_topk_kernel<2>, grid, 256, st, kt, a, g);
    else if (kpl <= 3) launch_kernel(group_topk_kernel<3>, grid, 256, st, kt, a, g);
    else if (kpl <= 4) launch_kernel(group_topk_kernel<4>, grid, 256, st, kt, a, g);
    else if (kpl <= 8) launch_kernel(group_topk_kernel<8>, grid, 256, st, kt, a, g);
    else launch_kernel(group_topk_kernel<16>, grid, 256, st, kt, a, g);
    return hipGetLastError();
}

}  // namespace moe
