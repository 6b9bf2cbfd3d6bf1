// Tiled kernel of the block-scaled 4-bit product,
//
//     C[m][n] = epi(init + sum over blocks b of 32 k of 2^(ea[b, m] + eb[b, n]) P_b[m][n]),
//     P_b[m][n] = sum over the block's k of A[m][k] * B[n][k],
//
// on the main loop of pair_tile.h: the matrix instruction's block scales are
// the format's, so a K-step is nothing but copies, LDS reads and products.
//
// 8192^3 takes 254 to 268 us (4.2 PFLOP/s) on 256 x 256 tiles: the products
// alone 157, the copies alone 196, all but the copies 173, all but the scales'
// copies 250, all but the LDS reads 232; so the copies bound it, and with them
// the two stages that fit (four of 64-byte rows, half lines: 276).  4096 x
// 4096 x 5003 with binary32 C 62 us (2.7 PFLOP/s), one round of 256 tiles.
// 37 x 5120 x 8192 on 64 x 128 tiles: 10 us and 4.0 for the sum (9 and 2.8 at
// least), 160 workgroups on 256 CUs.  Eight waves
// and three stages on 128 x 128 tiles gain where a tile is all a CU has
// (300 x 5120 x 8192 22.5 us for 28.3, where 64 x 128 tiles take 17.1) and
// lose where it has more (4096^3 58 for 47).
#include <hip/hip_runtime.h>

#include "fp8_util.h"
#include "lowp.h"
#include "pair_tile.h"

namespace tcm {
namespace fp4t {

using pair::f4;

template <int CFG, bool WIDE>
struct Tile : pair::Loop<kFp4Tiles[CFG].bm, kFp4Tiles[CFG].bn, kFp4Tiles[CFG].wm, kFp4Tiles[CFG].wn, kFp4Tiles[CFG].stages, true, WIDE> {
    using L = pair::Loop<kFp4Tiles[CFG].bm, kFp4Tiles[CFG].bn, kFp4Tiles[CFG].wm, kFp4Tiles[CFG].wn, kFp4Tiles[CFG].stages, true, WIDE>;
    static constexpr int FM = L::FM;

    __device__ __forceinline__ static void run(const Fp4Args& a) {
        __shared__ __attribute__((aligned(1024))) char smem_raw[L::LDS];
        pair::lds_char* smem = (pair::lds_char*)smem_raw;
        const int tid = threadIdx.x, lane = tid & 63;
        const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
        const int wm = wave / L::WN, wn = wave % L::WN;
        const int T = a.tiles_m * a.tiles_n;
        const int nidx = xcd_order(blockIdx.x, T * a.split);
        const int share = nidx / T, t = nidx - share * T;
        int tm, tn;
        super_order(t, a.tiles_m, a.tiles_n, a.group_m, a.super_m, a.super_n, &tm, &tn);
        const int64_t m0 = (int64_t)tm * L::BM, n0 = (int64_t)tn * L::BN;
        const int64_t steps = (a.K + 255) / 256;
        const int k_lo = (int)(share * steps / a.split), k_hi = (int)((share + 1) * steps / a.split);
        f4 acc[FM][4];
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] = f4{0.f, 0.f, 0.f, 0.f};
        const pair::Operands o{a.A, a.B, a.M, a.N, a.lda, a.ldb, mx_bytes(a.K), a.K, a.sa, a.sb, a.ldsa, a.ldsb};
        if (k_lo < k_hi) L::run(acc, o, smem, m0, n0, k_lo, k_hi, k_hi - k_lo, wave, lane);
        if (a.split > 1) {
            f4* w = (f4*)a.ws + ((int64_t)nidx * L::NW + wave) * FM * 4 * 64 + lane;
#pragma unroll
            for (int i = 0; i < FM; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) w[(i * 4 + j) * 64] = acc[i][j];
            return;
        }
        store_tile(acc, a, m0 + wm * L::TM + (lane & 15), n0 + wn * 64 + L::n_row(4 * (lane >> 4)));
    }
    // accumulators to C: row m of row tile 0, column n of tile 0
    __device__ __forceinline__ static void store_tile(const f4 (&acc)[FM][4], const Fp4Args& a, int64_t m, int64_t n) {
        constexpr int E = WIDE ? 4 : 16;  // consecutive columns a lane has
#pragma unroll
        for (int q = 0; q < 16 / E; ++q) {
            const int64_t nq = n + L::n_tile(q);
            if (nq >= a.N) continue;
            const Epilogue<E, Fp4Args> epi(a, nq);
#pragma unroll
            for (int i = 0; i < FM; ++i) {
                if (m + 16 * i >= a.M) continue;
                float v[E];
#pragma unroll
                for (int e = 0; e < E; ++e) v[e] = acc[i][(q * E + e) >> 2][e & 3];
                epi.store(v, m + 16 * i);
            }
        }
    }
    // Sum of a split launch: a wave takes one accumulator tile (16 rows by four columns a lane) and has up to eight
    // shares' partials of it in flight; they are added in order.
    __device__ __forceinline__ static void run_sum(const Fp4Args& a) {
        const int lane = threadIdx.x & 63, j = threadIdx.x >> 6;
        const int64_t T = (int64_t)a.tiles_m * a.tiles_n;
        int64_t b = blockIdx.x;
        const int i = (int)(b % FM);
        b /= FM;
        const int wave = (int)(b % L::NW);
        const int t = (int)(b / L::NW);
        int tm, tn;
        super_order(t, a.tiles_m, a.tiles_n, a.group_m, a.super_m, a.super_n, &tm, &tn);
        const int wm = wave / L::WN, wn = wave % L::WN;
        const int64_t m = (int64_t)tm * L::BM + wm * L::TM + 16 * i + (lane & 15);
        const int64_t n = (int64_t)tn * L::BN + wn * 64 + L::n_row(4 * (lane >> 4)) + L::n_tile(j);
        if (m >= a.M || n >= a.N) return;
        const f4* p = (const f4*)a.ws + ((((int64_t)t * L::NW + wave) * FM + i) * 4 + j) * 64 + lane;
        const int64_t step = T * L::NW * FM * 4 * 64;
        f4 s = {0.f, 0.f, 0.f, 0.f};
        for (int k = 0; k < a.split; k += 8) {
            f4 x[8];
#pragma unroll
            for (int u = 0; u < 8; ++u)
                if (k + u < a.split) x[u] = p[(k + u) * step];
#pragma unroll
            for (int u = 0; u < 8; ++u)
                if (k + u < a.split) s += x[u];
        }
        const Epilogue<4, Fp4Args> epi(a, n);
        float v[4] = {s[0], s[1], s[2], s[3]};
        epi.store(v, m);
    }
};

template <int CFG, bool WIDE>
__global__ __launch_bounds__((Tile<CFG, WIDE>::L::NT)) __attribute__((amdgpu_waves_per_eu(2))) void fp4_tile_kernel(Fp4Args a) {
    Tile<CFG, WIDE>::run(a);
}
template <int CFG, bool WIDE>
__global__ __launch_bounds__(256) void fp4_sum_kernel(Fp4Args a) {
    Tile<CFG, WIDE>::run_sum(a);
}

template <int CFG, bool WIDE>
int launch(const Fp4Args& a, hipStream_t s) {
    using X = Tile<CFG, WIDE>;
    const unsigned tiles = (unsigned)(a.tiles_m * a.tiles_n);
    hipLaunchKernelGGL((fp4_tile_kernel<CFG, WIDE>), dim3(tiles * a.split), dim3(X::L::NT), 0, s, a);
    if (a.split > 1) hipLaunchKernelGGL((fp4_sum_kernel<CFG, WIDE>), dim3(tiles * X::L::NW * X::FM), dim3(256), 0, s, a);
    return (int)hipGetLastError();
}
template <int CFG>
int launch_width(const Fp4Args& a, hipStream_t s) {
    return a.c_type == C_ACC ? launch<CFG, true>(a, s) : launch<CFG, false>(a, s);
}

}  // namespace fp4t

int launch_fp4_tile(int cfg, const Fp4Args& a, void* stream) {
    hipStream_t s = (hipStream_t)stream;
    static_assert(kNumFp4Tiles == 4, "one case a config");
    switch (cfg) {
    case 0: return fp4t::launch_width<0>(a, s);
    case 1: return fp4t::launch_width<1>(a, s);
    case 2: return fp4t::launch_width<2>(a, s);
    default: return fp4t::launch_width<3>(a, s);
    }
}

}  // namespace tcm
