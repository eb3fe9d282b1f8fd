// quantize.hip - rows of fp32 or bf16 to e4m3 codes (quantize_dev.h).
#include "common.h"
#include "kernels.h"
#include "quantize_dev.h"

namespace moe {

template <int XF>
__global__ __launch_bounds__(256) void quantize_rows_kernel(QuantArgs a) {
    quantize_blocks<XF>(a, (int64_t)blockIdx.x * 16 + threadIdx.x / 16, (int64_t)gridDim.x * 16);
}

hipError_t launch_quantize_rows(const QuantArgs& a, hipStream_t st, const KTime& kt) {
    const int64_t blocks = ((int64_t)a.rows * f8_scale_ld(a.cols) + 15) / 16;
    const int grid = (int)(blocks < 65536 ? blocks : 65536);
    if (a.xdt == MOE_DT_BF16) launch_kernel(quantize_rows_kernel<MOE_DT_BF16>, grid, 256, st, kt, a);
    else launch_kernel(quantize_rows_kernel<MOE_DT_F32>, grid, 256, st, kt, a);
    return hipGetLastError();
}

}  // namespace moe
