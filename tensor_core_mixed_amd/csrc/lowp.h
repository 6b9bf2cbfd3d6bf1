// Arguments and launchers of the block-scaled 8-bit product, its quantiser,
// the expert router and the mixture-of-experts layer (tcm_gemm_fp8,
// tcm_quantize_fp8, tcm_moe_route, tcm_moe), shared by the C ABI and the
// kernels.
#pragma once
#include <cstddef>
#include <cstdint>
#include <initializer_list>
#include <mutex>

namespace tcm {

// One scale covers kScaleBlock values of a row, or a kScaleBlock-square tile.
constexpr int kScaleBlock = 128;
constexpr int64_t scale_blocks(int64_t n) { return (n + kScaleBlock - 1) / kScaleBlock; }
// The largest values of the two 8-bit formats, and the least scale: a block
// of zeros keeps a normal, finite one.
constexpr float kE4M3Max = 448.f, kE5M2Max = 57344.f;
constexpr float kScaleMin = 0x1p-126f;

struct QuantArgs {
    const void* x;
    int64_t rows, cols, ldx;
    unsigned char* q;      // [rows][cols] as x lies, or null
    int64_t ldq;
    float* s;              // its scales
    int64_t lds;
    unsigned char* qt;     // [cols][rows], or null
    int64_t ldqt;
    float* st;
    int64_t ldst;
};
// x_type: F16, BF16 or F32
int launch_quantize(int x_type, bool e5m2, bool tile, const QuantArgs& a, void* stream);

struct Fp8Args {
    const unsigned char* A;  // [M][K]
    const unsigned char* B;  // [N][K]
    void* C;                 // [M][N]
    const float* sa;         // [k block][row of A]
    const float* sb;         // [row tile of B][k block], or with b_row [k block][row of B]
    const float* bias;
    int64_t M, N, K, lda, ldb, ldc, ldsa, ldsb;
    int a_e5m2, b_e5m2, b_row;
    int has_bias, relu, accum, c_type;
    // the tiled kernels
    int c_vec;                       // C's rows at multiples of 16 bytes
    int tiles_m, tiles_n;
    int group_m, super_m, super_n;   // tile order (tile_coords)
    int split;                       // k ranges of a tile, summed by a second launch
    float* ws;                       // their partial tiles
};
// any alignment, leading dimension and size
int launch_fp8_generic(const Fp8Args& a, void* stream);
// Macro tiles of the tiled kernel: waves WM x WN of (BM/WM) x 64 outputs, LDS stages of 128 k.
struct Fp8Tile {
    int bm, bn, wm, wn, stages;
    bool wide;  // serves binary32 C (products on 16-bit operands, which take more registers)
};
constexpr int kNumFp8Tiles = 4;
constexpr Fp8Tile kFp8Tiles[kNumFp8Tiles] = {
    {256, 256, 2, 4, 2, false},  // large products: 128 x 64 a wave, two waves a SIMD
    {256, 128, 4, 2, 3, true},  // half as many columns, three stages
    {128, 128, 2, 2, 2, true},  // two workgroups a CU
    {64, 128, 2, 2, 3, true},   // few rows
};
// A, B and sizes as fp8_tiles_fit accepts; the operand types pick the instance
int launch_fp8_tile_e4m3_e4m3(int cfg, const Fp8Args& a, void* stream);
int launch_fp8_tile_e5m2_e4m3(int cfg, const Fp8Args& a, void* stream);
int launch_fp8_tile_e4m3_e5m2(int cfg, const Fp8Args& a, void* stream);
int launch_fp8_tile_e5m2_e5m2(int cfg, const Fp8Args& a, void* stream);
int launch_fp8_tile_sum(int cfg, const Fp8Args& a, void* stream);
// A few rows: workgroups of kFp8SkinnyCols columns by up to kFp8SkinnyRows
// rows (`rows`, a row block; a.tiles_m of them), a.split k ranges.
constexpr int kFp8SkinnyCols = 16, kFp8SkinnyRows = 64;
int launch_fp8_skinny(int rows, const Fp8Args& a, void* stream);

struct RouteArgs {
    const void* x;         // [tokens][experts]
    int64_t tokens, ldx;
    int experts, topk;
    int sigmoid, norm;
    const float* bias;     // [experts], added to the scores for the choice only, or null
    float scale;
    int* ids;              // [tokens][topk]
    float* weights;        // [tokens][topk]
};
constexpr int kRouteMaxExperts = 1024, kRouteMaxTopk = 64;
int launch_route(int x_type, const RouteArgs& a, void* stream);

struct MoeArgs {
    const void* x;         // [tokens][hidden], 16-bit
    int64_t ldx;
    const int* ids;        // [tokens][topk]
    const float* weights;
    const void* w1;        // [experts][gate, up][inter][hidden]
    const float* s1;       // [experts][gate, up][inter tile][hidden tile] (8-bit weights)
    const void* w2;        // [experts][hidden][inter]
    const float* s2;
    void* out;             // [tokens][hidden], x's type
    int64_t ldo;
    int tokens, hidden, inter, experts, topk;
    void* ws;              // h, the products between the matrices: [pair][inter] binary32,
                           // or [pair][upper, lower][inter] bfloat16 parts
    // the tiled kernels
    float* y;              // [pair][hidden]
    unsigned* hmax;        // float16 weights: |h|'s largest of each 16, [pair][inter / 16]
};
// Tiled kernels: rows of x, w1 and w2 at multiples of 4 bytes, at most
// kMoePairs pairs a call.
constexpr int kMoePairs = 1024;
int launch_moe_tile(int x_type, bool w_e4m3, const MoeArgs& a, void* stream);
int launch_moe_generic(int x_type, bool w_e4m3, const MoeArgs& a, void* stream);

// Process-wide switches of tcm_gemm_fp8 (tcm_set_option): the kernel, -1 the
// planner's choice, else a row of kFp8Tiles, kFp8Skinny or kFp8Generic; and
// the k ranges of a tile, 0 the planner's choice.
constexpr int kFp8Skinny = kNumFp8Tiles, kFp8Generic = kNumFp8Tiles + 1, kFp8MaxSplit = 64;
struct LowpOpts {
    int fp8_config = -1, fp8_split = 0;
};
LowpOpts lowp_opts();
// Shared with the C ABI's other entry points (tcm_api.cpp): the stream's
// workspace, grown to `bytes` (a tcm_status), with the lock to hold until the
// last launch that uses it, and the text of tcm_last_plan.
int workspace_for(void* stream, int64_t bytes, void** out, std::unique_lock<std::mutex>* order);
void set_last_plan(const char* text);
// (formatted when it is asked for)
constexpr int kPlanValues = 10;
using PlanFormat = void (*)(char* buf, size_t n, const int64_t* v);
void set_last_plan(PlanFormat format, std::initializer_list<int64_t> v);

}  // namespace tcm
