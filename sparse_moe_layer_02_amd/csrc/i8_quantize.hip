// i8_quantize.hip - rows of fp32 or bf16 to int8 codes with one fp32 scale per
// row (i8_quantize_dev.h).
#include "common.h"
#include "i8_quantize_dev.h"
#include "kernels.h"

namespace moe {
namespace {

constexpr int QT = 256;  // threads per row

template <int XF>
__global__ __launch_bounds__(QT) void quantize_tokens_kernel(TokenQuantArgs a) {
    quantize_token_rows<XF, QT>(a, blockIdx.x, gridDim.x);
}

}  // namespace

hipError_t launch_quantize_tokens(const TokenQuantArgs& a, hipStream_t st, const KTime& kt) {
    const int grid = (int)(a.rows < 65536 ? a.rows : 65536);
    if (a.xdt == MOE_DT_BF16) launch_kernel(quantize_tokens_kernel<MOE_DT_BF16>, grid, QT, st, kt, a);
    else launch_kernel(quantize_tokens_kernel<MOE_DT_F32>, grid, QT, st, kt, a);
    return hipGetLastError();
}

}  // namespace moe
