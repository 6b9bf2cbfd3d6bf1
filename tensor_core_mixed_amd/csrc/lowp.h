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

struct BalanceArgs {
    const void* x;         // [tokens][experts]
    int64_t tokens, ldx;
    int experts, topk;
    int sigmoid;
    const int* ids;        // [tokens][topk]
    const unsigned char* mask;  // [tokens], 0: the token does not count; or null
    int* counts;           // [experts + 1], the last the tokens that count
    float* losses;         // [2]
    // several workgroups: each one's partial sums, and what the second launch's hand on
    int groups;
    float* p;              // [groups][experts]
    int* n;                // [groups][experts + 1]
    double* z;             // [groups]
    unsigned long long* arrived;
};
// a workgroup's waves in the two ways to run, and the most workgroups of the second
constexpr int kBalanceWaves = 8, kBalanceOneWaves = 16, kBalanceGroups = 256, kBalanceOneTokens = 128;
// a lane's tokens whose shares are added in binary32
constexpr int kBalanceRun = 32;
int launch_balance(int x_type, const BalanceArgs& a, void* stream);

struct RouteGradArgs {
    const void* x;
    int64_t tokens, ldx;
    int experts, topk;
    int sigmoid, norm, d_type;
    float scale;
    const int* ids;
    const unsigned char* mask;
    const float* dweights; // [tokens][topk] or null
    const int* counts;     // BalanceArgs::counts, with dlosses
    const float* dlosses;  // [2] or null
    void* d;               // [tokens][experts]
    int64_t ldd;
};
int launch_route_grad(int x_type, const RouteGradArgs& a, void* stream);

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

// ---- 4-bit floats (e2m1) with a power of two for each block of 32 (MXFP4)

// Four scales of a row's consecutive blocks lie in one word, the first lowest.
constexpr int kMxBlock = 32, kMxWord = 4 * kMxBlock;
constexpr int64_t mx_words(int64_t n) { return (n + kMxWord - 1) / kMxWord; }
constexpr int64_t mx_bytes(int64_t n) { return (n + 1) / 2; }

struct MxQuantArgs {
    const void* x;
    int64_t rows, cols, ldx;
    unsigned char* q;      // [rows][cols / 2] as x lies, or null
    int64_t ldq;           // bytes
    unsigned* s;           // [cols / 128][rows]
    int64_t lds;
    unsigned char* qt;     // [cols][rows / 2], or null
    int64_t ldqt;
    unsigned* st;          // [rows / 128][cols]
    int64_t ldst;
};
// x_type: F16, BF16 or F32
int launch_mx_quantize(int x_type, const MxQuantArgs& a, void* stream);
// x from (q, s)
int launch_mx_dequantize(int x_type, const MxQuantArgs& a, void* stream);

struct Fp4Args {
    const unsigned char* A;  // [M][K / 2]
    const unsigned char* B;  // [N][K / 2]
    void* C;                 // [M][N]
    const unsigned* sa;      // [k / 128][row of A]
    const unsigned* sb;
    const float* bias;
    int64_t M, N, K, lda, ldb, ldc, ldsa, ldsb;  // lda and ldb in bytes
    int has_bias, relu, accum, c_type;
    // the fast kernels
    int c_vec;                       // C's rows at multiples of 16 bytes
    int tiles_m, tiles_n;
    int group_m, super_m, super_n;   // tile order (tile_coords)
    int split;                       // k ranges of a tile, summed by a second launch
    float* ws;                       // their partial tiles
};
// any alignment, leading dimension and size
int launch_fp4_generic(const Fp4Args& a, void* stream);
// Macro tiles of the tiled kernel: waves WM x WN of (BM/WM) x 64 outputs, LDS stages of 256 k.
struct Fp4Tile {
    int bm, bn, wm, wn, stages;
};
constexpr int kNumFp4Tiles = 4;
constexpr Fp4Tile kFp4Tiles[kNumFp4Tiles] = {
    {256, 256, 2, 4, 2},  // large products: 128 x 64 a wave, two waves a SIMD
    {256, 128, 4, 2, 3},  // half as many columns, three stages
    {128, 128, 2, 2, 2},  // two workgroups a CU
    {64, 128, 2, 2, 3},   // few rows
};
// A, B and sizes as fp4_tiles_fit accepts
int launch_fp4_tile(int cfg, const Fp4Args& a, void* stream);
// A few rows: workgroups of kFp4SkinnyCols columns by up to kFp4SkinnyRows
// rows (`rows`, a row block; a.tiles_m of them), a.split k ranges.
constexpr int kFp4SkinnyCols = 16, kFp4SkinnyRows = 64;
int launch_fp4_skinny(int rows, const Fp4Args& a, void* stream);

// ---- Newton-Schulz steps (tcm_orthogonalize)

// Macro tiles of its products: `parts` times waves WM x WN of (BM/WM) x 64 outputs, each part with its own share of k and
// LDS stages of 32 k in two parts.
struct OrthoTile {
    int bm, bn, wm, wn, stages, parts;
};
constexpr int kNumOrthoTiles = 3;
constexpr OrthoTile kOrthoTiles[kNumOrthoTiles] = {
    {256, 256, 2, 4, 2, 1},  // large products
    {128, 128, 4, 2, 3, 1},  // few tiles
    {64, 64, 2, 1, 3, 2},    // fewer: two halves of k, added in LDS
};
// sizes up to 2^20 - 32 (a tile's rows stay within a buffer descriptor's range), workspace of the entries of a launch, slices
// of a sum of squares
constexpr int64_t kOrthoMaxSize = ((int64_t)1 << 20) - 32, kOrthoWorkspace = (int64_t)2 << 30, kOrthoSlices = 256;
struct OrthoArgs {
    const void* g;         // [rows][cols]
    int64_t batch, rows, cols, ldg, stride_g;
    void* o;
    int64_t ldo, stride_o;
    int o_type;
    float eps;
    int64_t rows_pad, cols_pad;  // to whole pieces of 32
    int64_t slices;        // of an entry's sum of squares
    double* squares;       // [batch][slices]; null: the launch sums them itself (launch_ortho_small of one chunk)
    char* as_is;           // parts of G over its norm [rows][cols_pad], entry_bytes apart
    char* across;          // and transposed [cols][rows_pad]
    int64_t entry_bytes;
    int64_t first_tile;    // of a launch
};
int launch_ortho_norm(int x_type, const OrthoArgs& a, void* stream);
// factor * G / (norm + eps): its parts, or with `out` O
int launch_ortho_start(int x_type, const OrthoArgs& a, float factor, bool out, void* stream);

// alpha * A B^T + beta * P of every entry, in parts: A [M][k_pad], B [N][k_pad], P and D [M][n_pad], E [N][m_pad]
// transposed; or to out.
struct OrthoMul {
    const char *A, *B, *P;
    char *D, *E;
    int64_t entry_bytes, M, N, k_pad, n_pad, m_pad;
    float alpha, beta;
    char* out;             // [M][N], or with out_across [N][M], of out_type; or null
    int64_t ld_out, stride_out;
    int out_type, out_across;
    int batch, symmetric;
    int tiles, tiles_m, tiles_n, group_m, super_m, super_n, split;
    float* ws;             // partial tiles
};
int launch_ortho_mul(int cfg, const OrthoMul& p, void* stream);

// Shorter sides up to 128: chunks of kOrthoSmallElems values of an entry's X (64 or 128 rows of it), a workgroup each.
constexpr int kOrthoSmallMax = 128, kOrthoSmallElems = 16384, kOrthoSmallSteps = 16;
inline int ortho_small_rows(int64_t n) { return n <= 64 ? 64 : 128; }
// Every workgroup of an entry reads all its chunks' shares of S: up to half a MiB of them (64 x 8192: 88 us, 126 by
// ortho.hip's kernels; 128 x 1024: 112, 117).  Of 128 rows they are 64 KiB a chunk, which pays in one round of workgroups
// only (16 of 128 x 1024: 150, 174; 300 of 100 x 1000: 1800, 1153).
inline bool ortho_small_fits(int64_t batch, int64_t n, int64_t m) {
    const int64_t np = ortho_small_rows(n), cw = kOrthoSmallElems / np, chunks = (m + cw - 1) / cw;
    return n <= kOrthoSmallMax && chunks * np * np * 4 <= (1 << 19) && (np == 64 || chunks == 1 || batch * chunks <= 256);
}
struct OrthoStep {
    float s_alpha, t_alpha, t_beta, x_alpha, x_beta;  // S's factor, and those of T and X as OrthoMul's
};
struct OrthoSmallArgs {
    OrthoArgs g;               // G, O and the norm
    int64_t m;                 // the longer side
    int n, tall, chunks;
    int first, last, steps;    // G becomes X first; O comes out last; steps in between
    float factor;              // of the first X
    char* state;               // the chunks' X between launches
    const float* shares_in;    // the chunks' S of the launch before
    float* shares_out;
    OrthoStep step[kOrthoSmallSteps];
};
int launch_ortho_small(int x_type, const OrthoSmallArgs& p, void* stream);

// Process-wide switches of tcm_gemm_fp8 (tcm_set_option): the kernel, -1 the
// planner's choice, else a row of kFp8Tiles, kFp8Skinny or kFp8Generic; and
// the k ranges of a tile, 0 the planner's choice.
constexpr int kFp8Skinny = kNumFp8Tiles, kFp8Generic = kNumFp8Tiles + 1, kFp8MaxSplit = 64;
// and the same of tcm_gemm_mxfp4
constexpr int kFp4Skinny = kNumFp4Tiles, kFp4Generic = kNumFp4Tiles + 1, kFp4MaxSplit = 64;
struct LowpOpts {
    int fp8_config = -1, fp8_split = 0;
    int fp4_config = -1, fp4_split = 0;
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
