#include "fp8_tile.h"

namespace tcm {
int launch_fp8_tile_e4m3_e5m2(int cfg, const Fp8Args& a, void* stream) {
    return fp8t::launch_types<false, true>(cfg, a, (hipStream_t)stream);
}
}  // namespace tcm
