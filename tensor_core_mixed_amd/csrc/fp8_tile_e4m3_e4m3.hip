#include "fp8_tile.h"

namespace tcm {
int launch_fp8_tile_e4m3_e4m3(int cfg, const Fp8Args& a, void* stream) {
    return fp8t::launch_types<false, false>(cfg, a, (hipStream_t)stream);
}

// the sum of a split launch's partial tiles (the operands' types play no part)
namespace fp8t {
template <int CFG>
__global__ __launch_bounds__(256) void fp8_tile_sum_kernel(Fp8Args a) {
    Tile<CFG, false, false, false, false>::run_sum(a);
}
template <int CFG>
int launch_sum(const Fp8Args& a, hipStream_t s) {
    using T = Tile<CFG, false, false, false, false>;
    hipLaunchKernelGGL((fp8_tile_sum_kernel<CFG>), dim3((unsigned)(a.tiles_m * a.tiles_n * T::NW * T::FM)), dim3(256), 0, s, a);
    return (int)hipGetLastError();
}
}  // namespace fp8t
int launch_fp8_tile_sum(int cfg, const Fp8Args& a, void* stream) {
    hipStream_t s = (hipStream_t)stream;
    switch (cfg) {
    case 0: return fp8t::launch_sum<0>(a, s);
    case 1: return fp8t::launch_sum<1>(a, s);
    case 2: return fp8t::launch_sum<2>(a, s);
    default: return fp8t::launch_sum<3>(a, s);
    }
}
}  // namespace tcm
