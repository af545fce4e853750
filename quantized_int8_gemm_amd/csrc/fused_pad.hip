// Operands whose rows are not whole 16-byte pieces, laid out once more so that they are, zeros
// behind each row: what the tiled kernels load directly to LDS.  Bound by memory (rows of 4095
// bytes of a 4095 x 4095 weight: 33.5 MB read and written).
#include "fused_common.h"
#include "fused_load.h"

namespace qg {
namespace {

constexpr int NT = 256;

__global__ __launch_bounds__(NT) void fused_pad_kernel(PadArgs a) {
    const int h = blockIdx.y;
    const int64_t t = (int64_t)blockIdx.x * NT + threadIdx.x;
    const int per = (int)(a.ldd[h] / 16);
    const int64_t row = t / per;
    if (row >= a.rows[h]) return;
    const int c = (int)(t - row * per) * 16;
    *reinterpret_cast<u32x4*>(a.dst[h] + row * a.ldd[h] + c) = load16_any(a.src[h] + row * a.ld[h], c, (int)a.cols[h]);
}

}  // namespace

hipError_t launch_fused_pad(const PadArgs& a, hipStream_t s) {
    int64_t most = 0;
    for (int h = 0; h < a.count; ++h) most = a.rows[h] * (a.ldd[h] / 16) > most ? a.rows[h] * (a.ldd[h] / 16) : most;
    if (most >= (int64_t)1 << 32) return hipErrorInvalidValue;
    hipLaunchKernelGGL(fused_pad_kernel, dim3((unsigned)((most + NT - 1) / NT), a.count), dim3(NT), 0, s, a);
    return hipGetLastError();
}

}  // namespace qg
