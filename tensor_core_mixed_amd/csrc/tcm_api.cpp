// C ABI of the engine (declared in include/tcm.h): argument checks, the
// per-(device, stream) Stream-K workspace, and dispatch to the kernels.
#include <hip/hip_runtime.h>

#include <dlfcn.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <fstream>
#include <map>
#include <mutex>
#include <sstream>
#include <string>
#include <utility>
#include <vector>

#include "../../include/tcm.h"
#include "lowp.h"
#include "planner.h"
#include "tcm_internal.h"

namespace tcm {
TileLauncher tile_launcher_f16(int config, bool b_kmajor);
TileLauncher tile_launcher_bf16(int config, bool b_kmajor);
TileLauncher tile_launcher_f32(int config, bool b_kmajor);
TileLauncher tile_launcher_i8(int config, bool b_kmajor);
TileLauncher tile_acol_launcher_f16(int config, bool b_kmajor);
TileLauncher tile_acol_launcher_bf16(int config, bool b_kmajor);
TileLauncher tile_acol_launcher_f32(int config, bool b_kmajor);
TileLauncher tile_acol_launcher_i8(int config, bool b_kmajor);
int tile_sk_occupancy_f16(int config, bool b_kmajor);
int tile_sk_occupancy_bf16(int config, bool b_kmajor);
int tile_sk_occupancy_f32(int config, bool b_kmajor);
int tile_sk_occupancy_i8(int config, bool b_kmajor);
TileLauncher conv_launcher_f16(int config);
TileLauncher conv_launcher_bf16(int config);
TileLauncher conv_launcher_f32(int config);
TileLauncher conv_launcher_i8(int config);
int conv_sk_occupancy_f16(int config);
int conv_sk_occupancy_bf16(int config);
int conv_sk_occupancy_f32(int config);
int conv_sk_occupancy_i8(int config);

GroupLauncher group_launcher_f16(int config, bool b_kmajor);
GroupLauncher group_launcher_bf16(int config, bool b_kmajor);
GroupLauncher group_launcher_f32(int config, bool b_kmajor);
GroupLauncher group_launcher_i8(int config, bool b_kmajor);

GroupLauncher group_launcher(int config, int dtype, bool b_kmajor) {
    switch (dtype) {
    case F16: return group_launcher_f16(config, b_kmajor);
    case BF16: return group_launcher_bf16(config, b_kmajor);
    case F32: return group_launcher_f32(config, b_kmajor);
    case I8: return group_launcher_i8(config, b_kmajor);
    default: return nullptr;
    }
}

TileLauncher conv_launcher(int config, int dtype) {
    switch (dtype) {
    case F16: return conv_launcher_f16(config);
    case BF16: return conv_launcher_bf16(config);
    case F32: return conv_launcher_f32(config);
    case I8: return conv_launcher_i8(config);
    default: return nullptr;
    }
}

int conv_sk_occupancy(int config, int dtype) {
    switch (dtype) {
    case F16: return conv_sk_occupancy_f16(config);
    case BF16: return conv_sk_occupancy_bf16(config);
    case F32: return conv_sk_occupancy_f32(config);
    case I8: return conv_sk_occupancy_i8(config);
    default: return 0;
    }
}

int tile_sk_occupancy(int config, int dtype, bool b_kmajor) {
    switch (dtype) {
    case F16: return tile_sk_occupancy_f16(config, b_kmajor);
    case BF16: return tile_sk_occupancy_bf16(config, b_kmajor);
    case F32: return tile_sk_occupancy_f32(config, b_kmajor);
    case I8: return tile_sk_occupancy_i8(config, b_kmajor);
    default: return 0;
    }
}

TileLauncher tile_launcher(int config, int dtype, bool b_kmajor, bool a_mmajor) {
    if (a_mmajor) {
        switch (dtype) {
        case F16: return tile_acol_launcher_f16(config, b_kmajor);
        case BF16: return tile_acol_launcher_bf16(config, b_kmajor);
        case F32: return tile_acol_launcher_f32(config, b_kmajor);
        case I8: return tile_acol_launcher_i8(config, b_kmajor);
        default: return nullptr;
        }
    }
    switch (dtype) {
    case F16: return tile_launcher_f16(config, b_kmajor);
    case BF16: return tile_launcher_bf16(config, b_kmajor);
    case F32: return tile_launcher_f32(config, b_kmajor);
    case I8: return tile_launcher_i8(config, b_kmajor);
    default: return nullptr;
    }
}

namespace {

std::mutex g_mu;
Options g_opts;
int g_use_tuned = 1;  // option "tuned"

// Auto-tuned choices by shape class.  Problems of one element type, operand
// layout, output type, epilogue, alignment and batching whose M, N and K
// each fall in the same half octave (floor(2 log2 x)) form a class; a class
// entry holds the plan parameters that measured fastest on the shape it was
// tuned on: tile config and mode, Stream-K grid policy, split-tile fix-up,
// tile-order group rows.
struct TuneKey {
    int dtype, a_col, b_col, c_type, epilogue, aligned, batched;
    int mc, nc, kc;
    bool operator<(const TuneKey& o) const {
        const int x[10] = {dtype, a_col, b_col, c_type, epilogue, aligned, batched, mc, nc, kc};
        const int y[10] = {o.dtype, o.a_col, o.b_col, o.c_type, o.epilogue, o.aligned, o.batched, o.mc, o.nc, o.kc};
        return std::lexicographical_compare(x, x + 10, y, y + 10);
    }
};
// One point of the tuning space.
struct Cand {
    int config = -1, mode = 0;
    int grid_kind = 0, grid_param = 0;  // Stream-K grid: 0 the planner's, 1 grid_param/8 per CU, 2 grid_param per tile
    int fixup = 0;                      // 0 the planner's, 1 last arrival, 2 fix-up kernel
    int group_m = 0;                    // 0 the planner's (4)
};
struct TuneEntry {
    Cand c;
    double us;           // measured time per call
    int64_t M, N, K;     // the shape it was tuned on
};
std::map<TuneKey, TuneEntry> g_tune;
int half_octave(int64_t x) { return x <= 0 ? -1 : (int)std::floor(2.0 * std::log2((double)x) + 1e-9); }
TuneKey tune_key(const Problem& p) {
    return TuneKey{p.dtype, (int)p.a_col, (int)p.b_col, p.c_type, p.epilogue, (int)p.aligned, p.batch > 1 ? 1 : 0,
                   half_octave(p.M), half_octave(p.N), half_octave(p.K)};
}
// The split-k GEMV kernels as candidates: configs outside the tile table's
// index range, mode 1, no other parameter (their k ranges are the
// planner's).  kGemvCand: the 4x4x4 row-major-B kernel or the column-major-B
// one; kGemvWideCand: the 16x16x32 row-major-B kernel.
constexpr int kGemvCand = 100, kGemvWideCand = 101;
bool gemv_cand(int config) { return config == kGemvCand || config == kGemvWideCand; }
bool valid_cand(const Cand& c) {
    if (gemv_cand(c.config))
        return c.mode == 1 && c.grid_kind == 0 && c.grid_param == 0 && c.fixup == 0 && c.group_m == 0;
    return c.config >= 0 && c.config < kNumConfigs && (c.mode == 1 || c.mode == 2) && c.grid_kind >= 0 &&
           c.grid_kind <= 2 && c.grid_param >= 0 && c.grid_param <= 64 && (c.grid_kind == 0 || c.grid_param > 0) &&
           c.fixup >= 0 && c.fixup <= 2 && c.group_m >= 0 && c.group_m <= 16;
}
// Apply candidate c to options o.
void apply_cand(const Cand& c, Options* o) {
    o->sk_grid = 0;
    if (gemv_cand(c.config)) {
        o->force_config = -1;
        o->force_mode = 0;
        o->gemv = 2;
        o->gemv_wide = c.config == kGemvWideCand ? 2 : 1;
        return;
    }
    o->force_config = c.config;
    o->force_mode = c.mode;
    o->grid_per_cu8 = c.grid_kind == 1 ? c.grid_param : 0;
    o->grid_shares = c.grid_kind == 2 ? c.grid_param : 0;
    if (c.fixup) o->sk_fixup = c.fixup;
    if (c.group_m) o->group_m = c.group_m;
}
// The candidate tcm_tune is timing on this thread (null: none).
thread_local const Cand* t_cand = nullptr;
// The class entry the last plan_options call on this thread applied (for tcm_last_plan).
thread_local std::string t_tuned_note;

struct Workspace {
    void* partial = nullptr;
    int64_t partial_bytes = 0;
    int* counters = nullptr;
    int64_t n_counters = 0;
};
std::map<std::pair<int, void*>, Workspace> g_ws;  // (device, stream_key) -> workspace
// The stream's handle; but hipStreamPerThread is one handle for a stream of
// every thread, so there a number of the thread's own (odd, as no other
// handle but hipStreamLegacy's 1 is).
void* stream_key(void* stream) {
    if (stream != (void*)hipStreamPerThread) return stream;
    static std::atomic<uintptr_t> next{3};
    thread_local const uintptr_t mine = next.fetch_add(2);
    return (void*)mine;
}
// Held from the look-up of a stream's workspace (or of the fixed scratch) to
// the last launch of the call: a call of several launches hands its partial
// results on through it, so another host thread's launches on the same stream
// must not come between them.  Streams have locks of their own: one stream's
// full queue holds no other up.  (Taken before g_mu, never after it.)
std::map<std::pair<int, void*>, std::mutex> g_enqueue;  // (device, stream_key) -> lock
std::unique_lock<std::mutex> enqueue_order(int dev, void* stream) {
    std::mutex* m;
    {
        std::lock_guard<std::mutex> lk(g_mu);
        m = &g_enqueue[{dev, stream_key(stream)}];
    }
    return std::unique_lock<std::mutex>(*m);
}
// Buffers a workspace outgrew.  A graph captured before the growth still
// points at them, and kernels enqueued before it may still run on them, so
// they live until tcm_release_workspace (no free, and no synchronisation, on
// the calling path).
std::vector<std::pair<int, void*>> g_retired;  // (device, pointer)

// The text of tcm_last_plan: assigned, or (the short calls, which would spend
// more on it than on their checks) values that are formatted when asked for,
// in place: asking allocates nothing, so it throws nothing.
struct PlanText {
    std::string s;
    char formatted[256];
    PlanFormat format = nullptr;
    int64_t v[kPlanValues];
    PlanText& operator=(std::string t) {
        s = std::move(t);
        format = nullptr;
        return *this;
    }
    const char* text() {
        if (!format) return s.c_str();
        format(formatted, sizeof formatted, v);
        return formatted;
    }
};
thread_local PlanText t_last_plan;

// Scratch of tcm_gemm_noalloc: the Stream-K partial tiles (two slots per
// workgroup of the grid) and the split tiles' arrival counters, in one
// fixed device array instead of the per-stream workspace.  Each device the
// library runs on holds its own copy, at its own address, until the process
// ends.  Host code never uses the array's name as an address (on the host it
// is only a stand-in): the address of each device's copy comes from
// hipGetSymbolAddress, called once per device with that device current.
constexpr int64_t kScratchPartialBytes = (int64_t)64 << 20;
constexpr int64_t kScratchCounters = (int64_t)1 << 16;
constexpr int64_t kScratchBytes = kScratchPartialBytes + kScratchCounters * (int64_t)sizeof(int);
static __device__ __align__(256) unsigned char scratch[kScratchBytes];
std::map<int, char*> g_scratch;  // device -> address of its copy of `scratch`

// Address of the current device `dev`'s scratch (looked up on its first use).
int scratch_of(int dev, char** out) {
    std::lock_guard<std::mutex> lk(g_mu);
    auto it = g_scratch.find(dev);
    if (it == g_scratch.end()) {
        void* p = nullptr;
        if (hipGetSymbolAddress(&p, HIP_SYMBOL(scratch)) != hipSuccess || p == nullptr) {
            (void)hipGetLastError();
            return TCM_ERR_HIP;
        }
        it = g_scratch.emplace(dev, (char*)p).first;
    }
    *out = it->second;
    return TCM_OK;
}
bool scratch_fits(const Plan& pl) {
    return pl.ws_partial_bytes <= kScratchPartialBytes && pl.ws_counters <= kScratchCounters;
}

int device_cus(int dev) {
    static std::map<int, int> cache;
    std::lock_guard<std::mutex> lk(g_mu);
    auto it = cache.find(dev);
    if (it != cache.end()) return it->second;
    int n = 0;
    if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || n <= 0) n = kDefaultCUs;
    cache[dev] = n;
    return n;
}

Options current_options() {
    std::lock_guard<std::mutex> lk(g_mu);
    return g_opts;
}

int parse_table(const char* text, std::vector<std::pair<TuneKey, TuneEntry>>* rows);
void load_shipped_table();
int current_cus();

// Wave regime of T tiles on `slots` co-resident workgroups: the number of
// waves (the last one full or not) when the tiles fill the GPU at least
// once, else whether the tiles fit it two or more times over (a split-k grid
// can give every tile equal shares) or not.
int64_t wave_regime(int64_t T, int64_t slots) {
    if (T <= 0 || slots <= 0) return 0;
    if (T >= slots) return (T + slots - 1) / slots;
    return slots / T >= 2 ? -2 : -1;
}
// A class entry applies to problem p only if p's tiles, on the entry's tile
// config, quantise onto the CUs as the tuned shape's did.  A split-k entry
// needs the same wave regime (2048^2 x 8192 on 128x128 units: 256 tiles,
// exactly two shares per workgroup slot, split-k wins; 2304^2 x 9216, the
// same class: 324 tiles, split-k at 209 us against 140 us data-parallel).
// A data-parallel entry carries over to problems of as many waves or fewer,
// not to ones that need more (2048^3 on 64x64 units fills one wave; 2816^3,
// one class up, needs two, and runs at 78 us on them against 54 us on
// 128x128 tiles).
bool same_regime(const Problem& p, const TuneEntry& e, int cus) {
    const TileConfig& c = kConfigs[e.c.config];
    const int64_t occ = e.c.mode == 2 ? tile_sk_wg_per_cu(c) : tile_wg_per_cu(c);
    const int64_t nb = std::max<int64_t>(p.batch, 1);
    const int64_t tq = ((p.M + c.bm - 1) / c.bm) * ((p.N + c.bn - 1) / c.bn) * nb;
    const int64_t tt = ((e.M + c.bm - 1) / c.bm) * ((e.N + c.bn - 1) / c.bn) * nb;
    const int64_t rq = wave_regime(tq, cus * occ), rt = wave_regime(tt, cus * occ);
    if (e.c.mode == 2 || rq == rt) return rq == rt;
    // (negative codes: under one wave; -2 under half of one, where the
    // GPU would sit mostly idle on the entry's tiles: 2048^2 x 4096 on the
    // 256x256 tiles tuned for 3840^2 x 4096 took 84 us against 51 us)
    return rq != -2 && rq <= rt;
}

// The entry for problem p: its own class's, else the nearest class of the
// same type, layouts, output, epilogue, alignment and batching whose M, N
// and K classes each lie within one half octave (smallest summed distance;
// the first in key order on a tie); in both cases only an entry whose tiles
// quantise onto the CUs as the tuned shape's did (same_regime).
// g_tune.end() if none.  Caller holds g_mu.
std::map<TuneKey, TuneEntry>::iterator entry_for(const Problem& p, const TuneKey& k, int cus) {
    auto best = g_tune.end();
    int best_d = 1 << 30;
    for (auto it = g_tune.begin(); it != g_tune.end(); ++it) {
        const TuneKey& e = it->first;
        if (e.dtype != k.dtype || e.a_col != k.a_col || e.b_col != k.b_col || e.c_type != k.c_type ||
            e.epilogue != k.epilogue || e.aligned != k.aligned || e.batched != k.batched)
            continue;
        const int dm = std::abs(e.mc - k.mc), dn = std::abs(e.nc - k.nc), dk = std::abs(e.kc - k.kc);
        if (dm > 1 || dn > 1 || dk > 1) continue;
        if (dm + dn + dk < best_d && same_regime(p, it->second, cus)) {
            best_d = dm + dn + dk;
            best = it;
        }
    }
    return best;
}

// Options for planning problem p: the global switches, then the tuned class
// entry for p (unless a switch already forces config or mode; switches the
// caller set keep their values), then a candidate tcm_tune is timing on this
// thread.
Options plan_options(const Problem& p) {
    static std::once_flag shipped;
    std::call_once(shipped, load_shipped_table);
    const int cus = current_cus();  // (takes the lock itself)
    Options o;
    t_tuned_note.clear();
    {
        std::lock_guard<std::mutex> lk(g_mu);
        o = g_opts;
        // tuned entries describe single GEMM calls; a convolution or a group is planned afresh
        // (option gemv = 2 asks for the GEMV wherever it can serve: the table is not consulted there)
        if (g_use_tuned && !p.conv && !p.group && o.force_config < 0 && o.force_mode == 0 && o.sk_grid == 0 &&
            !(o.gemv == 2 && gemv_eligible(p))) {
            const TuneKey k = tune_key(p);
            auto it = entry_for(p, k, cus);
            // a GEMV entry does not apply with option gemv = 1 (never), nor
            // against option gemv_wide's choice of kernel
            const bool skip = it != g_tune.end() && gemv_cand(it->second.c.config) &&
                              (o.gemv == 1 || (it->second.c.config == kGemvWideCand ? o.gemv_wide == 1 : o.gemv_wide == 2));
            if (it != g_tune.end() && !skip) {
                const Cand& c = it->second.c;
                if (gemv_cand(c.config)) {
                    o.gemv = 2;  // (a problem it cannot serve is planned as if untuned)
                    o.gemv_wide = c.config == kGemvWideCand ? 2 : 1;
                } else {
                    o.force_config = c.config;
                    o.force_mode = c.mode;
                    o.grid_per_cu8 = c.grid_kind == 1 ? c.grid_param : 0;
                    o.grid_shares = c.grid_kind == 2 ? c.grid_param : 0;
                    if (c.fixup && o.sk_fixup == 0) o.sk_fixup = c.fixup;
                    if (c.group_m && o.group_m == 0) o.group_m = c.group_m;
                }
                char buf[96];
                snprintf(buf, sizeof buf, " tuned=%d,%d,%d", it->first.mc, it->first.nc, it->first.kc);
                t_tuned_note = buf;
            }
        }
    }
    if (t_cand) apply_cand(*t_cand, &o);
    return o;
}

// Workgroups per CU of the Stream-K kernels of p's (dtype, B layout, GEMM or
// convolution), as the runtime reports them for the compiled kernels (queried
// once per kind); a runtime that cannot answer (no device) leaves the
// planner's static estimate.
void fill_sk_occupancy(const Problem& p, Options* o) {
    static std::map<int, std::vector<int>> occ_cache;
    std::lock_guard<std::mutex> lk(g_mu);
    const int key = p.dtype * 4 + (p.b_col ? 1 : 0) + (p.conv ? 2 : 0);
    auto it = occ_cache.find(key);
    if (it == occ_cache.end()) {
        std::vector<int> v(kNumConfigs);
        for (int c = 0; c < kNumConfigs; ++c)
            v[c] = p.conv ? conv_sk_occupancy(c, p.dtype) : tile_sk_occupancy(c, p.dtype, p.b_col);
        (void)hipGetLastError();
        it = occ_cache.emplace(key, v).first;
    }
    for (int c = 0; c < kNumConfigs; ++c) o->sk_occ[c] = it->second[c];
}

// CUs of the current device, or the default without one.
int current_cus() {
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess) {
        (void)hipGetLastError();
        return kDefaultCUs;
    }
    return device_cus(dev);
}

// Grow (never shrink) the workspace of (dev, stream); counters start at zero
// and every split tile's last arrival resets its counter, so they stay zero
// between calls.  A buffer that is outgrown is retired, not freed (see
// g_retired); growth rounds up to a power of two, so a stream retires at most
// a few dozen buffers however its calls grow.  Growth while the stream is
// being captured into a graph is refused (TCM_ERR_NOT_SUPPORTED): the
// allocation would not be part of the graph.
int64_t round_pow2(int64_t x) {
    int64_t r = 1;
    while (r < x) r <<= 1;
    return r;
}
int get_workspace(int dev, void* stream, int64_t partial_bytes, int64_t n_counters, Workspace* out) {
    std::lock_guard<std::mutex> lk(g_mu);
    Workspace& w = g_ws[{dev, stream_key(stream)}];
    const bool grow_p = w.partial_bytes < partial_bytes, grow_c = w.n_counters < n_counters;
    if (grow_p || grow_c) {
        hipStreamCaptureStatus cs = hipStreamCaptureStatusNone;
        if (hipStreamIsCapturing((hipStream_t)stream, &cs) != hipSuccess) {
            (void)hipGetLastError();
            return TCM_ERR_HIP;
        }
        if (cs != hipStreamCaptureStatusNone) return TCM_ERR_NOT_SUPPORTED;
    }
    if (grow_p) {
        const int64_t bytes = round_pow2(partial_bytes);
        void* p = nullptr;
        if (hipMalloc(&p, (size_t)bytes) != hipSuccess) {
            (void)hipGetLastError();
            return TCM_ERR_ALLOC;
        }
        if (w.partial) g_retired.emplace_back(dev, w.partial);
        w.partial = p;
        w.partial_bytes = bytes;
    }
    if (grow_c) {
        const int64_t n = round_pow2(n_counters);
        int* c = nullptr;
        if (hipMalloc((void**)&c, (size_t)n * sizeof(int)) != hipSuccess) {
            (void)hipGetLastError();
            return TCM_ERR_ALLOC;
        }
        if (launch_fill_zero(c, n, stream) != 0) {
            (void)hipFree(c);
            return TCM_ERR_HIP;
        }
        if (w.counters) g_retired.emplace_back(dev, (void*)w.counters);
        w.counters = c;
        w.n_counters = n;
    }
    *out = w;
    return TCM_OK;
}

bool overlaps(const void* a, int64_t abytes, const void* b, int64_t bbytes) {
    if (!a || !b || abytes <= 0 || bbytes <= 0) return false;
    const char* x = (const char*)a;
    const char* y = (const char*)b;
    return x < y + bbytes && y < x + abytes;
}

// extent in elements of a rows x cols matrix with leading dimension ld
int64_t extent(int64_t rows, int64_t cols, int64_t ld) { return rows == 0 || cols == 0 ? 0 : (rows - 1) * ld + cols; }

std::string describe(const Plan& pl, const Problem& p) {
    char buf[320];
    if (pl.kernel == 0) {
        snprintf(buf, sizeof buf, "empty problem M=%lld N=%lld", (long long)p.M, (long long)p.N);
    } else if (pl.kernel == 3) {
        snprintf(buf, sizeof buf,
                 "kernel=gemv rows=%d cols_per_wg=%d k_per_wg=%d splits=%lld grid=%d M=%lld N=%lld K=%lld dtype=%d b_col=%d "
                 "mfma=%s%s",
                 pl.bm, pl.bn, pl.bk, (long long)pl.iters, pl.grid, (long long)p.M, (long long)p.N, (long long)p.K, p.dtype,
                 (int)p.b_col, p.b_col || pl.gemv_wide ? "16x16x32" : "4x4x4", pl.fixup_kernel ? " fixup=kernel" : "");
    } else if (pl.kernel == 1) {
        snprintf(buf, sizeof buf, "kernel=generic tile=64x64 tiles=%lld iters=%lld M=%lld N=%lld K=%lld dtype=%d batch=%lld%s",
                 (long long)pl.tiles, (long long)pl.iters, (long long)p.M, (long long)p.N, (long long)p.K, p.dtype,
                 (long long)p.batch, p.conv ? " conv=1" : "");
    } else {
        snprintf(buf, sizeof buf,
                 "kernel=%s config=%d tile=%dx%dx%d mode=%s grid=%d tiles=%lld iters=%lld dp_tiles=%lld sk_tiles=%lld "
                 "M=%lld N=%lld K=%lld dtype=%d b_col=%d batch=%lld est_cycles=%.0f%s%s%s",
                 p.conv ? "conv" : "tile", pl.config, pl.bm, pl.bn, pl.bk, pl.mode == 1 ? "dp" : "streamk", pl.grid, (long long)pl.tiles,
                 (long long)pl.iters, (long long)pl.dp_tiles, (long long)pl.sk_tiles, (long long)p.M, (long long)p.N,
                 (long long)p.K, p.dtype, (int)p.b_col, (long long)p.batch, pl.est_cycles,
                 pl.fixup_kernel ? " fixup=kernel" : "", p.a_col ? " a_col=1" : "",
                 pl.split > 1 ? (" split=" + std::to_string(pl.split)).c_str() : "");
    }
    return buf;
}

int check_problem(int64_t M, int64_t N, int64_t K, int64_t lda, int64_t ldb, int64_t ldc, int dtype, int epilogue,
                  Problem* p) {
    const int dt = dtype & 0xff;
    const int flags = dtype & ~0xff;
    if (dt < F16 || dt > I8) return TCM_ERR_INVALID_VALUE;
    if (flags & ~(TCM_A_COLMAJOR | TCM_B_COLMAJOR | TCM_C_F16 | TCM_C_BF16)) return TCM_ERR_INVALID_VALUE;
    const int c_type = (flags & TCM_C_F16) ? C_F16 : ((flags & TCM_C_BF16) ? C_BF16 : C_ACC);
    if ((flags & TCM_C_F16) && (flags & TCM_C_BF16)) return TCM_ERR_INVALID_VALUE;
    if (c_type != C_ACC && dt == I8) return TCM_ERR_INVALID_VALUE;
    if (epilogue < 0 || epilogue > (TCM_EPI_BIAS | TCM_EPI_RELU | TCM_EPI_ACCUM)) return TCM_ERR_INVALID_VALUE;
    if (M < 0 || N < 0 || K < 0) return TCM_ERR_INVALID_VALUE;
    const bool a_col = flags & TCM_A_COLMAJOR, b_col = flags & TCM_B_COLMAJOR;
    if (lda < 1 || lda < (a_col ? M : K)) return TCM_ERR_INVALID_VALUE;
    if (ldb < 1 || ldb < (b_col ? K : N)) return TCM_ERR_INVALID_VALUE;
    if (ldc < 1 || ldc < N) return TCM_ERR_INVALID_VALUE;
    p->M = M;
    p->N = N;
    p->K = K;
    p->lda = lda;
    p->ldb = ldb;
    p->ldc = ldc;
    p->dtype = dt;
    p->a_col = a_col;
    p->b_col = b_col;
    p->epilogue = epilogue;
    p->c_type = c_type;
    p->aligned = true;
    return TCM_OK;
}

}  // namespace

namespace {
LowpOpts g_lowp;  // (guarded by g_mu)
}
LowpOpts lowp_opts() {
    std::lock_guard<std::mutex> lk(g_mu);
    return g_lowp;
}
int workspace_for(void* stream, int64_t bytes, void** out, std::unique_lock<std::mutex>* order) {
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess) {
        (void)hipGetLastError();
        return TCM_ERR_HIP;
    }
    Workspace w;
    *order = enqueue_order(dev, stream);
    const int st = get_workspace(dev, stream, bytes, 0, &w);
    if (st == TCM_OK) *out = w.partial;
    return st;
}
void set_last_plan(const char* text) { t_last_plan = text; }
void set_last_plan(PlanFormat format, std::initializer_list<int64_t> v) {
    std::copy(v.begin(), v.begin() + std::min<size_t>(v.size(), kPlanValues), t_last_plan.v);
    t_last_plan.format = format;
}

}  // namespace tcm

using namespace tcm;

extern "C" {

const char* tcm_version(void) { return "tcm 0.1 (gfx950)"; }

const char* tcm_status_string(int status) {
    switch (status) {
    case TCM_OK: return "TCM_OK";
    case TCM_ERR_INVALID_VALUE: return "TCM_ERR_INVALID_VALUE: invalid argument";
    case TCM_ERR_NOT_SUPPORTED: return "TCM_ERR_NOT_SUPPORTED: request not supported";
    case TCM_ERR_HIP: return "TCM_ERR_HIP: HIP runtime error";
    case TCM_ERR_ALLOC: return "TCM_ERR_ALLOC: workspace allocation failed";
    default: return "unknown tcm status";
    }
}

int tcm_set_option(const char* key, int64_t value) {
    if (!key) return TCM_ERR_INVALID_VALUE;
    std::lock_guard<std::mutex> lk(g_mu);
    if (!strcmp(key, "force_mode")) {
        if (value < 0 || value > 2) return TCM_ERR_INVALID_VALUE;
        g_opts.force_mode = (int)value;
    } else if (!strcmp(key, "force_config")) {
        if (value < -1 || value >= kNumConfigs) return TCM_ERR_INVALID_VALUE;
        g_opts.force_config = (int)value;
    } else if (!strcmp(key, "sk_grid")) {
        if (value < 0 || value > (1 << 20)) return TCM_ERR_INVALID_VALUE;
        g_opts.sk_grid = (int)value;
    } else if (!strcmp(key, "generic")) {
        if (value < 0 || value > 1) return TCM_ERR_INVALID_VALUE;
        g_opts.generic = (int)value;
    } else if (!strcmp(key, "sk_fixup")) {
        if (value < 0 || value > 2) return TCM_ERR_INVALID_VALUE;
        g_opts.sk_fixup = (int)value;
    } else if (!strcmp(key, "group_m")) {
        if (value < 0 || value > 16) return TCM_ERR_INVALID_VALUE;
        g_opts.group_m = (int)value;
    } else if (!strcmp(key, "grid_per_cu8")) {
        if (value < 0 || value > 64) return TCM_ERR_INVALID_VALUE;
        g_opts.grid_per_cu8 = (int)value;
    } else if (!strcmp(key, "grid_shares")) {
        if (value < 0 || value > 64) return TCM_ERR_INVALID_VALUE;
        g_opts.grid_shares = (int)value;
    } else if (!strcmp(key, "tuned")) {
        if (value < 0 || value > 1) return TCM_ERR_INVALID_VALUE;
        g_use_tuned = (int)value;
    } else if (!strcmp(key, "gemv")) {
        if (value < 0 || value > 2) return TCM_ERR_INVALID_VALUE;
        g_opts.gemv = (int)value;
    } else if (!strcmp(key, "gemv_splits")) {
        if (value < 0 || value > 4096) return TCM_ERR_INVALID_VALUE;
        g_opts.gemv_splits = (int)value;
    } else if (!strcmp(key, "gemv_wide")) {
        if (value < 0 || value > 2) return TCM_ERR_INVALID_VALUE;
        g_opts.gemv_wide = (int)value;
    } else if (!strcmp(key, "fp8_config")) {
        if (value < -1 || value > kFp8Generic) return TCM_ERR_INVALID_VALUE;
        g_lowp.fp8_config = (int)value;
    } else if (!strcmp(key, "fp8_split")) {
        if (value < 0 || value > kFp8MaxSplit) return TCM_ERR_INVALID_VALUE;
        g_lowp.fp8_split = (int)value;
    } else {
        return TCM_ERR_INVALID_VALUE;
    }
    return TCM_OK;
}

int64_t tcm_get_option(const char* key) {
    if (!key) return -2;
    std::lock_guard<std::mutex> lk(g_mu);
    if (!strcmp(key, "force_mode")) return g_opts.force_mode;
    if (!strcmp(key, "force_config")) return g_opts.force_config;
    if (!strcmp(key, "sk_grid")) return g_opts.sk_grid;
    if (!strcmp(key, "generic")) return g_opts.generic;
    if (!strcmp(key, "sk_fixup")) return g_opts.sk_fixup;
    if (!strcmp(key, "group_m")) return g_opts.group_m;
    if (!strcmp(key, "grid_per_cu8")) return g_opts.grid_per_cu8;
    if (!strcmp(key, "grid_shares")) return g_opts.grid_shares;
    if (!strcmp(key, "tuned")) return g_use_tuned;
    if (!strcmp(key, "gemv")) return g_opts.gemv;
    if (!strcmp(key, "gemv_splits")) return g_opts.gemv_splits;
    if (!strcmp(key, "gemv_wide")) return g_opts.gemv_wide;
    if (!strcmp(key, "fp8_config")) return g_lowp.fp8_config;
    if (!strcmp(key, "fp8_split")) return g_lowp.fp8_split;
    return -2;
}

int tcm_config_count(void) { return kNumConfigs; }

int tcm_config_info(int index, int dtype, int32_t* bm, int32_t* bn, int32_t* bk, int32_t* waves) {
    const int dt = dtype & 0xff;
    if (index < 0 || index >= kNumConfigs || dt < F16 || dt > I8) return TCM_ERR_INVALID_VALUE;
    if (bm) *bm = kConfigs[index].bm;
    if (bn) *bn = kConfigs[index].bn;
    if (bk) *bk = bk_elems(dt);
    if (waves) *waves = kConfigs[index].wm * kConfigs[index].wn;
    return TCM_OK;
}

int tcm_streamk_range(int64_t sk_tiles, int64_t iters_per_tile, int32_t grid, int32_t wg, int64_t* begin, int64_t* end) {
    if (sk_tiles < 0 || iters_per_tile < 1 || grid < 1 || wg < 0 || wg >= grid || !begin || !end) return TCM_ERR_INVALID_VALUE;
    streamk_range(sk_tiles, iters_per_tile, grid, wg, begin, end);
    return TCM_OK;
}

int tcm_plan_batched(int64_t batch, int64_t M, int64_t N, int64_t K, int64_t lda, int64_t ldb, int64_t ldc, int dtype,
                     int epilogue, int aligned, tcm_plan_info* out) {
    if (!out || batch < 1 || batch >= ((int64_t)1 << 31)) return TCM_ERR_INVALID_VALUE;
    Problem p;
    int st = check_problem(M, N, K, lda, ldb, ldc, dtype, epilogue, &p);
    if (st != TCM_OK) return st;
    p.aligned = aligned != 0;
    p.batch = batch;
    Options o = plan_options(p);
    fill_sk_occupancy(p, &o);
    Plan pl;
    if (!make_plan(p, o, current_cus(), &pl)) return TCM_ERR_INVALID_VALUE;
    out->kernel = pl.kernel == 2 ? 1 : (pl.kernel == 3 ? 2 : 0);
    out->config = pl.config;
    out->bm = pl.bm;
    out->bn = pl.bn;
    out->bk = pl.bk;
    out->mode = pl.mode;
    out->grid = pl.grid;
    out->tiles = pl.tiles;
    out->iters_per_tile = pl.iters;
    out->dp_tiles = pl.dp_tiles;
    out->sk_tiles = pl.sk_tiles;
    out->workspace_bytes = pl.ws_partial_bytes + pl.ws_counters * (int64_t)sizeof(int);
    out->fixup_kernel = pl.fixup_kernel ? 1 : 0;
    out->split = pl.split > 1 ? pl.split : 0;
    return TCM_OK;
}

int tcm_plan(int64_t M, int64_t N, int64_t K, int64_t lda, int64_t ldb, int64_t ldc, int dtype, int epilogue, int aligned,
             tcm_plan_info* out) {
    return tcm_plan_batched(1, M, N, K, lda, ldb, ldc, dtype, epilogue, aligned, out);
}

int tcm_tile_order(int32_t t, int32_t tiles_m, int32_t tiles_n, int32_t* tm, int32_t* tn) {
    if (tiles_m < 1 || tiles_n < 1 || (int64_t)tiles_m * tiles_n >= (1LL << 31) || t < 0 ||
        (int64_t)t >= (int64_t)tiles_m * tiles_n || !tm || !tn)
        return TCM_ERR_INVALID_VALUE;
    int sm, sn;
    const int gm = 4;
    tile_order_shape(tiles_m, tiles_n, gm, &sm, &sn);
    tile_coords(t, tiles_m, tiles_n, gm, sm, sn, tm, tn);
    return TCM_OK;
}

int tcm_last_plan(char* buf, int64_t len) {
    const char* s = t_last_plan.text();
    const int64_t size = (int64_t)strlen(s);
    if (buf && len > 0) {
        int64_t n = std::min<int64_t>(len - 1, size);
        memcpy(buf, s, (size_t)n);
        buf[n] = 0;
    }
    return (int)size;
}

void tcm_release_workspace(void) {
    std::lock_guard<std::mutex> lk(g_mu);
    int cur = 0;
    (void)hipGetDevice(&cur);
    std::vector<std::pair<int, void*>> all = g_retired;
    for (auto& kv : g_ws) {
        if (kv.second.partial) all.emplace_back(kv.first.first, kv.second.partial);
        if (kv.second.counters) all.emplace_back(kv.first.first, (void*)kv.second.counters);
    }
    // every device that holds a buffer finishes its work first (the streams
    // themselves may have been destroyed by now)
    std::vector<int> devs;
    for (auto& x : all)
        if (std::find(devs.begin(), devs.end(), x.first) == devs.end()) devs.push_back(x.first);
    for (int d : devs) {
        (void)hipSetDevice(d);
        (void)hipDeviceSynchronize();
    }
    for (auto& x : all) {
        (void)hipSetDevice(x.first);
        (void)hipFree(x.second);
    }
    (void)hipSetDevice(cur);
    g_ws.clear();
    g_enqueue.clear();
    g_retired.clear();
}

}  // extern "C"

namespace tcm {
namespace {

// Bytes spanned by `batch` entries of `ext` bytes placed `stride_bytes` apart.
int64_t batch_extent(int64_t batch, int64_t stride_bytes, int64_t ext) {
    return ext > 0 ? (batch - 1) * stride_bytes + ext : 0;
}

int launch_tiled(const Problem& p, const Plan& pl, TileArgs& a, int dev, void* stream, bool noalloc = false);

// noalloc: the Stream-K partials and counters live in the fixed `scratch`
// array; a plan that needs more is replaced by the data-parallel one, or
// refused (TCM_ERR_NOT_SUPPORTED) when Stream-K is forced.
int gemm_impl(int64_t batch, int64_t M, int64_t N, int64_t K, const void* A, int64_t lda, int64_t sa, const void* B,
              int64_t ldb, int64_t sb, void* C, int64_t ldc, int64_t sc, int dtype, const void* bias, int64_t sbias,
              int epilogue, void* stream, bool noalloc = false) {
    Problem p;
    int st = check_problem(M, N, K, lda, ldb, ldc, dtype, epilogue, &p);
    if (st != TCM_OK) return st;
    if (batch < 0 || sa < 0 || sb < 0 || sc < 0 || sbias < 0) return TCM_ERR_INVALID_VALUE;
    // keep every byte offset of the batch inside int64 (and the tile count inside int32 below)
    const int64_t kStrideLimit = (int64_t)1 << 40;
    if (batch >= ((int64_t)1 << 31) || sa >= kStrideLimit || sb >= kStrideLimit || sc >= kStrideLimit ||
        sbias >= kStrideLimit)
        return TCM_ERR_INVALID_VALUE;
    p.batch = batch;
    if (M == 0 || N == 0 || batch == 0) {
        t_last_plan = "empty problem";
        return TCM_OK;
    }
    const int es = elem_bytes(p.dtype);
    const int cs = c_elem_bytes(p.c_type);
    const int64_t a_one = extent(p.a_col ? K : M, p.a_col ? M : K, lda) * es;
    const int64_t b_one = extent(p.b_col ? N : K, p.b_col ? K : N, ldb) * es;
    const int64_t c_one = extent(M, N, ldc) * cs;
    // entries of C are written: they must not overlap one another
    if (batch > 1 && sc * cs < c_one) return TCM_ERR_INVALID_VALUE;
    const int64_t a_ext = batch_extent(batch, sa * es, a_one);
    const int64_t b_ext = batch_extent(batch, sb * es, b_one);
    const int64_t c_ext = batch_extent(batch, sc * cs, c_one);
    const bool use_bias = epilogue & TCM_EPI_BIAS;
    const int64_t bias_ext = use_bias ? batch_extent(batch, sbias * 4, N * 4) : 0;
    if (!C) return TCM_ERR_INVALID_VALUE;
    if (a_ext > 0 && !A) return TCM_ERR_INVALID_VALUE;
    if (b_ext > 0 && !B) return TCM_ERR_INVALID_VALUE;
    if (use_bias && !bias) return TCM_ERR_INVALID_VALUE;
    // pointers (and batch strides in bytes) that are not multiples of their
    // element size are served by the generic kernel with single-byte accesses
    const bool bytewise = ((uintptr_t)A % es) || ((uintptr_t)B % es) || ((uintptr_t)C % cs) ||
                          (use_bias && ((uintptr_t)bias % 4));
    if (overlaps(C, c_ext, A, a_ext) || overlaps(C, c_ext, B, b_ext) || (use_bias && overlaps(C, c_ext, bias, bias_ext)))
        return TCM_ERR_INVALID_VALUE;
    // the fast path wants every entry 16-byte aligned
    p.aligned = ((uintptr_t)A % 16 == 0) && ((uintptr_t)B % 16 == 0) && ((uintptr_t)C % 16 == 0) &&
                (!use_bias || (uintptr_t)bias % 16 == 0) &&
                (batch == 1 || ((sa * es) % 16 == 0 && (sb * es) % 16 == 0 && (sc * cs) % 16 == 0 &&
                                (!use_bias || (sbias * 4) % 16 == 0)));

    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess) {
        (void)hipGetLastError();
        return TCM_ERR_HIP;
    }
    Options o = plan_options(p);
    fill_sk_occupancy(p, &o);
    Plan pl;
    if (!make_plan(p, o, device_cus(dev), &pl)) return TCM_ERR_INVALID_VALUE;
    if (noalloc && pl.kernel == 3 && !scratch_fits(pl)) {
        o.gemv = 1;  // its partial sums do not fit the fixed scratch: the tiled kernel serves the call
        if (!make_plan(p, o, device_cus(dev), &pl)) return TCM_ERR_INVALID_VALUE;
    }
    if (noalloc && pl.kernel == 2 && pl.mode == 2 && !scratch_fits(pl)) {
        if (current_options().force_mode == 2) {
            t_last_plan = describe(pl, p) + " (split-k workspace beyond the fixed scratch)";
            return TCM_ERR_NOT_SUPPORTED;
        }
        o.force_mode = 1;
        if (!make_plan(p, o, device_cus(dev), &pl)) return TCM_ERR_INVALID_VALUE;
    }
    t_last_plan = describe(pl, p) + t_tuned_note + (noalloc ? " scratch=static" : "");

    if (pl.kernel == 1) {
        GenericArgs g{};
        g.A = A;
        g.B = B;
        g.C = C;
        g.bias = use_bias ? bias : nullptr;
        g.M = M;
        g.N = N;
        g.K = K;
        g.lda = lda;
        g.ldb = ldb;
        g.ldc = ldc;
        g.a_col = p.a_col;
        g.b_col = p.b_col;
        g.relu = (epilogue & TCM_EPI_RELU) != 0;
        g.has_bias = use_bias;
        g.accum = (epilogue & TCM_EPI_ACCUM) != 0;
        g.c_type = p.c_type;
        g.bytewise = bytewise ? 1 : 0;
        g.batch = (int)batch;
        g.stride_a = sa;
        g.stride_b = sb;
        g.stride_c = sc;
        g.stride_bias = sbias;
        g.tiles_m = (int)((M + 63) / 64);
        g.tiles_n = (int)((N + 63) / 64);
        return launch_generic(p.dtype, g, stream) == 0 ? TCM_OK : TCM_ERR_HIP;
    }

    if (pl.kernel == 3) {
        GemvArgs v{};
        v.A = A;
        v.B = B;
        v.C = C;
        v.bias = use_bias ? bias : nullptr;
        v.M = (int)M;
        v.N = (int)N;
        v.K = (int)K;
        v.lda = (int)lda;
        v.ldb = (int)ldb;
        v.ldc = (int)ldc;
        v.relu = (epilogue & TCM_EPI_RELU) != 0;
        v.has_bias = use_bias;
        v.accum = (epilogue & TCM_EPI_ACCUM) != 0;
        v.c_type = p.c_type;
        v.splits = (int)pl.iters;
        v.kw = pl.bk;
        v.b_bytes = b_one;
        v.a_bytes = a_one;
        v.b_col = p.b_col ? 1 : 0;
        v.wide = pl.gemv_wide ? 1 : 0;
        std::unique_lock<std::mutex> order;
        if (pl.ws_partial_bytes > 0) {
            order = enqueue_order(dev, stream);
            if (noalloc) {
                char* base = nullptr;
                int st2 = scratch_of(dev, &base);
                if (st2 != TCM_OK) return st2;
                v.partial = (float*)base;
            } else {
                Workspace w;
                int ws = get_workspace(dev, stream, pl.ws_partial_bytes, 0, &w);
                if (ws != TCM_OK) return ws;
                v.partial = (float*)w.partial;
            }
        }
        return launch_gemv(p.dtype, v, stream) == 0 ? TCM_OK : TCM_ERR_HIP;
    }

    TileArgs a{};
    a.A = A;
    a.B = B;
    a.C = C;
    a.bias = use_bias ? bias : nullptr;
    a.lda = (int)lda;
    a.ldb = (int)ldb;
    a.ldc = (int)ldc;
    a.batch = (int)batch;
    a.stride_a = sa;
    a.stride_b = sb;
    a.stride_c = sc;
    a.stride_bias = sbias;
    return launch_tiled(p, pl, a, dev, stream, noalloc);
}

// Fills the plan-dependent fields of `a` (sizes, epilogue, tile schedule,
// Stream-K workspace) and launches the tiled kernel the plan names.
int launch_tiled(const Problem& p, const Plan& pl, TileArgs& a, int dev, void* stream, bool noalloc) {
    a.M = (int)p.M;
    a.N = (int)p.N;
    a.K = (int)p.K;
    a.relu = (p.epilogue & TCM_EPI_RELU) != 0;
    a.has_bias = (p.epilogue & TCM_EPI_BIAS) != 0;
    a.accum = (p.epilogue & TCM_EPI_ACCUM) != 0;
    a.c_type = p.c_type;
    a.tiles_m = (int)((p.M + pl.bm - 1) / pl.bm);
    a.tiles_n = (int)((p.N + pl.bn - 1) / pl.bn);
    a.iters = (int)pl.iters;
    a.dp_tiles = (int)pl.dp_tiles;
    a.sk_tiles = (int)pl.sk_tiles;
    a.grid = pl.grid;
    a.group_m = pl.group_m;
    tile_order_shape(a.tiles_m, a.tiles_n, a.group_m, &a.super_m, &a.super_n);
    a.ws_partial = nullptr;
    a.ws_counter = nullptr;
    a.sk_fixup_kernel = pl.fixup_kernel ? 1 : 0;
    a.split = pl.split;
    if (pl.split > kMaxSplit) return TCM_ERR_INVALID_VALUE;  // the sum kernel holds at most kMaxSplit partials a block
    std::unique_lock<std::mutex> order;
    if (pl.mode == 2 && pl.sk_tiles > 0) order = enqueue_order(dev, stream);
    if (pl.mode == 2 && pl.sk_tiles > 0 && noalloc) {
        char* base = nullptr;
        int st = scratch_of(dev, &base);
        if (st != TCM_OK) return st;
        a.ws_partial = (float*)base;
        a.ws_counter = (int*)(base + kScratchPartialBytes);
        // the arrival counters must start at zero; a previous call on this
        // device leaves them so, but clear them anyway (a fill kernel, so the
        // call stays capturable into a graph)
        if (!pl.fixup_kernel && launch_fill_zero(a.ws_counter, pl.sk_tiles, stream) != 0) return TCM_ERR_HIP;
    } else if (pl.mode == 2 && pl.sk_tiles > 0) {
        Workspace w;
        int ws = get_workspace(dev, stream, pl.ws_partial_bytes, pl.ws_counters, &w);
        if (ws != TCM_OK) return ws;
        a.ws_partial = (float*)w.partial;
        a.ws_counter = w.counters;
    }
    TileLauncher launch = p.conv ? conv_launcher(pl.config, p.dtype) : tile_launcher(pl.config, p.dtype, p.b_col, p.a_col);
    if (!launch) return TCM_ERR_NOT_SUPPORTED;
    return launch(a, stream) == 0 ? TCM_OK : TCM_ERR_HIP;
}

// a * b for non-negative a, b; -1 once the product passes 2^62
int64_t mul_cap(int64_t a, int64_t b) {
    if (a < 0 || b < 0) return -1;
    if (a != 0 && b > ((int64_t)1 << 62) / a) return -1;
    return a * b;
}

// Convolution of an NHWC input with a KRSC filter as the GEMM
// y[(n,p,q), k] = sum over (r,s,c) of x[n, p*sh - ph + r*dh, q*sw - pw + s*dw, c] * f[k, r, s, c]
// with zero padding (the implicit-GEMM reading of a 2-D convolution).
int conv_impl(int64_t N, int64_t H, int64_t W, int64_t C, int64_t K, int64_t R, int64_t S, int64_t pad_h, int64_t pad_w,
              int64_t stride_h, int64_t stride_w, int64_t dil_h, int64_t dil_w, const void* x, const void* f, void* y,
              int dtype, const void* bias, int epilogue, void* stream) {
    const int64_t kDimLimit = (int64_t)1 << 31;
    const int64_t dims[13] = {N, H, W, C, K, R, S, pad_h, pad_w, stride_h, stride_w, dil_h, dil_w};
    for (int64_t d : dims)
        if (d < 0 || d >= kDimLimit) return TCM_ERR_INVALID_VALUE;
    if (R < 1 || S < 1 || stride_h < 1 || stride_w < 1 || dil_h < 1 || dil_w < 1) return TCM_ERR_INVALID_VALUE;
    if (dtype & (TCM_A_COLMAJOR | TCM_B_COLMAJOR)) return TCM_ERR_INVALID_VALUE;  // layouts are fixed
    if (epilogue & TCM_EPI_ACCUM) return TCM_ERR_INVALID_VALUE;
    const int64_t eh = H + 2 * pad_h - dil_h * (R - 1) - 1, ew = W + 2 * pad_w - dil_w * (S - 1) - 1;
    if (eh < 0 || ew < 0) return TCM_ERR_INVALID_VALUE;  // the dilated filter is larger than the padded image
    const int64_t P = eh / stride_h + 1, Q = ew / stride_w + 1;
    const int64_t M = mul_cap(mul_cap(N, P), Q), Kg = mul_cap(mul_cap(R, S), C);
    const int64_t x_elems = mul_cap(mul_cap(mul_cap(N, H), W), C);
    if (M < 0 || Kg < 0 || x_elems < 0 || mul_cap(M, K) < 0 || mul_cap(K, Kg) < 0) return TCM_ERR_INVALID_VALUE;
    Problem p;
    int st = check_problem(M, K, Kg, std::max<int64_t>(Kg, 1), std::max<int64_t>(Kg, 1), std::max<int64_t>(K, 1),
                           dtype | TCM_B_COLMAJOR, epilogue, &p);
    if (st != TCM_OK) return st;
    p.conv = true;
    p.conv_c = C;
    const int es = elem_bytes(p.dtype);
    const int cs = c_elem_bytes(p.c_type);
    p.conv_x_bytes = x_elems * es;
    // the tiled gather keeps its pixel offsets in int: bound them by the
    // padded image (one image past the last, for rows beyond M)
    const double span = (double)(N + 1) * (double)(H + 2 * pad_h + 1) * (double)(W + 2 * pad_w + 1) * (double)C * es;
    if (span >= (double)kDimLimit) p.conv_x_bytes = kDimLimit;  // too large for the tiled gather
    if (M == 0 || K == 0) {
        t_last_plan = "empty problem";
        return TCM_OK;
    }
    const bool use_bias = epilogue & TCM_EPI_BIAS;
    const int64_t x_ext = Kg > 0 ? x_elems * es : 0, f_ext = K * Kg * es, y_ext = M * K * cs;
    if (!y) return TCM_ERR_INVALID_VALUE;
    if (x_ext > 0 && !x) return TCM_ERR_INVALID_VALUE;
    if (f_ext > 0 && !f) return TCM_ERR_INVALID_VALUE;
    if (use_bias && !bias) return TCM_ERR_INVALID_VALUE;
    const bool bytewise = ((uintptr_t)x % es) || ((uintptr_t)f % es) || ((uintptr_t)y % cs) ||
                          (use_bias && ((uintptr_t)bias % 4));
    if (overlaps(y, y_ext, x, x_ext) || overlaps(y, y_ext, f, f_ext) || (use_bias && overlaps(y, y_ext, bias, K * 4)))
        return TCM_ERR_INVALID_VALUE;
    p.aligned = ((uintptr_t)x % 16 == 0) && ((uintptr_t)f % 16 == 0) && ((uintptr_t)y % 16 == 0) &&
                (!use_bias || (uintptr_t)bias % 16 == 0);

    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess) {
        (void)hipGetLastError();
        return TCM_ERR_HIP;
    }
    Options o = plan_options(p);
    fill_sk_occupancy(p, &o);
    Plan pl;
    if (!make_plan(p, o, device_cus(dev), &pl)) return TCM_ERR_INVALID_VALUE;
    t_last_plan = describe(pl, p);

    if (pl.kernel == 1) {
        GenericArgs g{};
        g.A = x;
        g.B = f;
        g.C = y;
        g.bias = use_bias ? bias : nullptr;
        g.M = M;
        g.N = K;
        g.K = Kg;
        g.lda = Kg;
        g.ldb = Kg;
        g.ldc = K;
        g.a_col = 0;
        g.b_col = 1;
        g.relu = (epilogue & TCM_EPI_RELU) != 0;
        g.has_bias = use_bias;
        g.accum = 0;
        g.c_type = p.c_type;
        g.bytewise = bytewise ? 1 : 0;
        g.batch = 1;
        g.tiles_m = (int)((M + 63) / 64);
        g.tiles_n = (int)((K + 63) / 64);
        g.conv = 1;
        g.cv_H = H;
        g.cv_W = W;
        g.cv_C = C;
        g.cv_P = P;
        g.cv_Q = Q;
        g.cv_R = R;
        g.cv_S = S;
        g.cv_pad_h = pad_h;
        g.cv_pad_w = pad_w;
        g.cv_stride_h = stride_h;
        g.cv_stride_w = stride_w;
        g.cv_dil_h = dil_h;
        g.cv_dil_w = dil_w;
        return launch_generic(p.dtype, g, stream) == 0 ? TCM_OK : TCM_ERR_HIP;
    }

    TileArgs a{};
    a.A = x;
    a.B = f;
    a.C = y;
    a.bias = use_bias ? bias : nullptr;
    a.lda = (int)Kg;
    a.ldb = (int)Kg;
    a.ldc = (int)K;
    a.batch = 1;
    a.cv_H = (int)H;
    a.cv_W = (int)W;
    a.cv_C = (int)C;
    a.cv_P = (int)P;
    a.cv_Q = (int)Q;
    a.cv_S = (int)S;
    a.cv_pad_h = (int)pad_h;
    a.cv_pad_w = (int)pad_w;
    a.cv_stride_h = (int)stride_h;
    a.cv_stride_w = (int)stride_w;
    a.cv_dil_h = (int)dil_h;
    a.cv_dil_w = (int)dil_w;
    a.cv_x_bytes = (int)p.conv_x_bytes;
    return launch_tiled(p, pl, a, dev, stream);
}

// A group of products sharing K, dtype and epilogue (tcm_gemm_grouped).
static_assert(kMaxGroup == TCM_MAX_GROUP, "the header's group limit is the kernel's");
int grouped_impl(int64_t count, const tcm_group_entry* ent, int64_t K, int dtype, int epilogue, void* stream) {
    if (count < 0 || count > kMaxGroup || (count > 0 && !ent)) return TCM_ERR_INVALID_VALUE;
    Problem pe[kMaxGroup];
    int64_t a_ext[kMaxGroup], b_ext[kMaxGroup], c_ext[kMaxGroup];
    const bool use_bias = epilogue & TCM_EPI_BIAS;
    int64_t M_total = 0, N_max = 0;
    bool aligned = true, work = false;
    for (int64_t i = 0; i < count; ++i) {
        const tcm_group_entry& x = ent[i];
        int st = check_problem(x.M, x.N, K, x.lda, x.ldb, x.ldc, dtype, epilogue, &pe[i]);
        if (st != TCM_OK) return st;
        const Problem& p = pe[i];
        const int es = elem_bytes(p.dtype), cs = c_elem_bytes(p.c_type);
        a_ext[i] = extent(p.a_col ? K : x.M, p.a_col ? x.M : K, x.lda) * es;
        b_ext[i] = extent(p.b_col ? x.N : K, p.b_col ? K : x.N, x.ldb) * es;
        c_ext[i] = extent(x.M, x.N, x.ldc) * cs;
        if (x.M == 0 || x.N == 0) continue;  // nothing read or written
        work = true;
        if (!x.C || (a_ext[i] > 0 && !x.A) || (b_ext[i] > 0 && !x.B) || (use_bias && !x.bias)) return TCM_ERR_INVALID_VALUE;
        aligned = aligned && (uintptr_t)x.A % 16 == 0 && (uintptr_t)x.B % 16 == 0 && (uintptr_t)x.C % 16 == 0 &&
                  (!use_bias || (uintptr_t)x.bias % 16 == 0);
        M_total += x.M;
        N_max = std::max(N_max, x.N);
    }
    // every C is written: it must not overlap any entry's inputs or another C
    for (int64_t i = 0; i < count; ++i) {
        if (ent[i].M == 0 || ent[i].N == 0) continue;
        for (int64_t j = 0; j < count; ++j) {
            if (ent[j].M == 0 || ent[j].N == 0) continue;
            if (overlaps(ent[i].C, c_ext[i], ent[j].A, a_ext[j]) || overlaps(ent[i].C, c_ext[i], ent[j].B, b_ext[j]) ||
                (use_bias && overlaps(ent[i].C, c_ext[i], ent[j].bias, ent[j].N * 4)) ||
                (i != j && overlaps(ent[i].C, c_ext[i], ent[j].C, c_ext[j])))
                return TCM_ERR_INVALID_VALUE;
        }
    }
    if (!work) {
        t_last_plan = "empty problem";
        return TCM_OK;
    }
    // plan over the whole work list: exact tile counts and eligibility per config
    Problem p = pe[0];
    p.M = M_total;
    p.N = N_max;
    p.lda = p.ldb = p.ldc = 1;  // per entry; the group fields below decide
    p.aligned = aligned;
    p.group = true;
    const double es = elem_bytes(p.dtype);
    for (int64_t i = 0; i < count; ++i) {
        if (ent[i].M == 0 || ent[i].N == 0) continue;
        p.group_a_bytes += (double)ent[i].M * K * es;
        p.group_b_bytes += (double)K * ent[i].N * es;
        p.group_c_bytes += (double)ent[i].M * ent[i].N * 4;
    }
    for (int c = 0; c < kNumConfigs; ++c) {
        int64_t tiles = 0;
        bool ok = aligned && !p.a_col;  // the grouped kernels stage k-contiguous A only
        for (int64_t i = 0; i < count && ok; ++i) {
            if (ent[i].M == 0 || ent[i].N == 0) continue;
            Problem q = pe[i];
            q.aligned = aligned;
            ok = tile_eligible(q, kConfigs[c]);
            const int64_t tm = (ent[i].M + kConfigs[c].bm - 1) / kConfigs[c].bm, tn = (ent[i].N + kConfigs[c].bn - 1) / kConfigs[c].bn;
            tiles += tm * tn;
            p.group_a_reads[c] += (double)ent[i].M * K * es * tn;
            p.group_b_reads[c] += (double)K * ent[i].N * es * tm;
        }
        p.group_ok[c] = ok && tiles < ((int64_t)1 << 31);
        p.group_tiles[c] = tiles;
    }
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess) {
        (void)hipGetLastError();
        return TCM_ERR_HIP;
    }
    Options o = plan_options(p);
    fill_sk_occupancy(p, &o);
    Plan pl;
    if (!make_plan(p, o, device_cus(dev), &pl)) return TCM_ERR_INVALID_VALUE;
    if (pl.kernel != 2) {
        // no tile config serves every entry: each runs on its own (the
        // generic kernel where the tiled one cannot take it)
        for (int64_t i = 0; i < count; ++i) {
            const tcm_group_entry& x = ent[i];
            int st = gemm_impl(1, x.M, x.N, K, x.A, x.lda, 0, x.B, x.ldb, 0, x.C, x.ldc, 0, dtype, x.bias, 0, epilogue,
                               stream);
            if (st != TCM_OK) return st;
        }
        t_last_plan = "kernel=generic group=" + std::to_string(count) + " (entries one by one)";
        return TCM_OK;
    }
    t_last_plan = describe(pl, p) + " group=" + std::to_string(count);

    GroupArgs g{};
    TileArgs& a = g.t;
    a.K = (int)K;
    a.relu = (epilogue & TCM_EPI_RELU) != 0;
    a.has_bias = use_bias;
    a.accum = (epilogue & TCM_EPI_ACCUM) != 0;
    a.c_type = p.c_type;
    a.batch = 1;
    a.iters = (int)pl.iters;
    a.dp_tiles = (int)pl.dp_tiles;
    a.sk_tiles = (int)pl.sk_tiles;
    a.grid = pl.grid;
    a.group_m = pl.group_m;
    a.sk_fixup_kernel = pl.fixup_kernel ? 1 : 0;
    int64_t tile0 = 0;
    for (int64_t i = 0; i < count; ++i) {
        const tcm_group_entry& x = ent[i];
        if (x.M == 0 || x.N == 0) continue;
        GroupEntry& y = g.e[g.count++];
        y.A = x.A;
        y.B = x.B;
        y.C = x.C;
        y.bias = use_bias ? x.bias : nullptr;
        y.M = (int)x.M;
        y.N = (int)x.N;
        y.lda = (int)x.lda;
        y.ldb = (int)x.ldb;
        y.ldc = (int)x.ldc;
        y.tiles_m = (int)((x.M + pl.bm - 1) / pl.bm);
        y.tiles_n = (int)((x.N + pl.bn - 1) / pl.bn);
        tile_order_shape(y.tiles_m, y.tiles_n, pl.group_m, &y.super_m, &y.super_n);
        y.tile0 = (int)tile0;
        tile0 += (int64_t)y.tiles_m * y.tiles_n;
    }
    if (tile0 != pl.tiles) return TCM_ERR_INVALID_VALUE;  // the plan and the table disagree (cannot happen)
    std::unique_lock<std::mutex> order;
    if (pl.mode == 2 && pl.sk_tiles > 0) {
        Workspace w;
        order = enqueue_order(dev, stream);
        int ws = get_workspace(dev, stream, pl.ws_partial_bytes, pl.ws_counters, &w);
        if (ws != TCM_OK) return ws;
        a.ws_partial = (float*)w.partial;
        a.ws_counter = w.counters;
    }
    GroupLauncher launch = group_launcher(pl.config, p.dtype, p.b_col);
    if (!launch) return TCM_ERR_NOT_SUPPORTED;
    return launch(g, stream) == 0 ? TCM_OK : TCM_ERR_HIP;
}

// Tuning table text, one class per line (blank lines and lines starting
// with '#' are skipped): "tcm-tune-2" then dtype a_col b_col c_type epilogue
// aligned batched, the half-octave classes of M N K, then config mode
// grid_kind grid_param fixup group_m, the measured microseconds and the
// tuned shape M N K.  All or nothing: any malformed line rejects the text.
int parse_table(const char* text, std::vector<std::pair<TuneKey, TuneEntry>>* rows) {
    const char* q = text;
    while (*q) {
        const char* eol = strchr(q, '\n');
        std::string line(q, eol ? (size_t)(eol - q) : strlen(q));
        q = eol ? eol + 1 : q + strlen(q);
        const size_t first = line.find_first_not_of(" \t\r");
        if (first == std::string::npos || line[first] == '#') continue;
        int d[16];
        long long m = 0, n = 0, k = 0;
        double us = 0;
        char tag[16];
        int used = 0;
        const int got = sscanf(line.c_str(), "%15s %d %d %d %d %d %d %d %d %d %d %d %d %d %d %d %d %lf %lld %lld %lld %n", tag,
                               &d[0], &d[1], &d[2], &d[3], &d[4], &d[5], &d[6], &d[7], &d[8], &d[9], &d[10], &d[11], &d[12],
                               &d[13], &d[14], &d[15], &us, &m, &n, &k, &used);
        if (got != 21 || strcmp(tag, "tcm-tune-2") || line.find_first_not_of(" \t\r", (size_t)used) != std::string::npos)
            return TCM_ERR_INVALID_VALUE;
        const TuneKey key{d[0], d[1], d[2], d[3], d[4], d[5], d[6], d[7], d[8], d[9]};
        Cand c;
        c.config = d[10];
        c.mode = d[11];
        c.grid_kind = d[12];
        c.grid_param = d[13];
        c.fixup = d[14];
        c.group_m = d[15];
        const bool flags_ok = (key.a_col | key.b_col | key.aligned | key.batched) >= 0 && key.a_col <= 1 && key.b_col <= 1 &&
                              key.aligned <= 1 && key.batched <= 1 && key.c_type >= 0 && key.c_type <= 2 &&
                              key.epilogue >= 0 && key.epilogue <= 7;
        if (key.dtype < F16 || key.dtype > I8 || !flags_ok || key.mc < 0 || key.nc < 0 || key.kc < 0 || !valid_cand(c) ||
            !(us >= 0) || m < 1 || n < 1 || k < 1)
            return TCM_ERR_INVALID_VALUE;
        rows->emplace_back(key, TuneEntry{c, us, m, n, k});
    }
    return TCM_OK;
}

// The tuning table shipped with the library: tuned/mi355x.txt next to the
// directory that holds libtcm.so (or the file TCM_TUNE_FILE names; an empty
// TCM_TUNE_FILE ships nothing).  Loaded once, before the first plan; a
// missing file leaves the table empty, a malformed one is ignored whole.
void load_shipped_table() {
    std::string path;
    const char* env = getenv("TCM_TUNE_FILE");
    if (env) {
        path = env;
    } else {
        Dl_info info;
        if (dladdr((void*)&load_shipped_table, &info) && info.dli_fname) {
            std::string so = info.dli_fname;
            const size_t slash = so.rfind('/');
            const std::string dir = slash == std::string::npos ? "." : so.substr(0, slash);
            path = dir + "/../tuned/mi355x.txt";
        }
    }
    if (path.empty()) return;
    std::ifstream f(path);
    if (!f) return;
    std::stringstream ss;
    ss << f.rdbuf();
    std::vector<std::pair<TuneKey, TuneEntry>> rows;
    if (parse_table(ss.str().c_str(), &rows) != TCM_OK) return;
    std::lock_guard<std::mutex> lk(g_mu);
    for (const auto& r : rows) g_tune.emplace(r.first, r.second);  // entries loaded or tuned first stay
}

}  // namespace
}  // namespace tcm

extern "C" {

int tcm_gemm(int64_t M, int64_t N, int64_t K, const void* A, int64_t lda, const void* B, int64_t ldb, void* C, int64_t ldc,
             int dtype, const void* bias, int epilogue, void* stream) {
    return gemm_impl(1, M, N, K, A, lda, 0, B, ldb, 0, C, ldc, 0, dtype, bias, 0, epilogue, stream);
}

int tcm_gemm_noalloc(int64_t M, int64_t N, int64_t K, const void* A, int64_t lda, const void* B, int64_t ldb, void* C,
                     int64_t ldc, int dtype, const void* bias, int epilogue, void* stream) {
    return gemm_impl(1, M, N, K, A, lda, 0, B, ldb, 0, C, ldc, 0, dtype, bias, 0, epilogue, stream, true);
}

int64_t tcm_noalloc_scratch_bytes(void) { return kScratchBytes; }

int tcm_gemm_grouped(int64_t count, const tcm_group_entry* entries, int64_t K, int dtype, int epilogue, void* stream) {
    return grouped_impl(count, entries, K, dtype, epilogue, stream);
}

int tcm_conv2d(int64_t N, int64_t H, int64_t W, int64_t C, int64_t K, int64_t R, int64_t S, int64_t pad_h, int64_t pad_w,
               int64_t stride_h, int64_t stride_w, int64_t dil_h, int64_t dil_w, const void* x, const void* f, void* y,
               int dtype, const void* bias, int epilogue, void* stream) {
    return conv_impl(N, H, W, C, K, R, S, pad_h, pad_w, stride_h, stride_w, dil_h, dil_w, x, f, y, dtype, bias, epilogue,
                     stream);
}

int tcm_gemm_batched(int64_t batch, int64_t M, int64_t N, int64_t K, const void* A, int64_t lda, int64_t stride_a,
                     const void* B, int64_t ldb, int64_t stride_b, void* C, int64_t ldc, int64_t stride_c, int dtype,
                     const void* bias, int64_t stride_bias, int epilogue, void* stream) {
    return gemm_impl(batch, M, N, K, A, lda, stride_a, B, ldb, stride_b, C, ldc, stride_c, dtype, bias, stride_bias, epilogue,
                     stream);
}

int tcm_tune(int64_t M, int64_t N, int64_t K, const void* A, int64_t lda, const void* B, int64_t ldb, void* C, int64_t ldc,
             int dtype, const void* bias, int epilogue, int iters, void* stream, tcm_plan_info* best) {
    if (iters < 1 || iters > 10000) return TCM_ERR_INVALID_VALUE;
    // the model's own choice first: it validates the call and names the key
    int st = gemm_impl(1, M, N, K, A, lda, 0, B, ldb, 0, C, ldc, 0, dtype, bias, 0, epilogue, stream);
    if (st != TCM_OK) return st;
    if (M == 0 || N == 0) return TCM_OK;
    Problem p;
    check_problem(M, N, K, lda, ldb, ldc, dtype, epilogue, &p);
    const bool use_bias = epilogue & TCM_EPI_BIAS;
    const int cs = c_elem_bytes(p.c_type);
    p.aligned = ((uintptr_t)A % 16 == 0) && ((uintptr_t)B % 16 == 0) && ((uintptr_t)C % 16 == 0) &&
                (!use_bias || (uintptr_t)bias % 16 == 0) && ((uintptr_t)C % cs == 0);
    if (strstr(t_last_plan.text(), "kernel=generic")) return TCM_OK;  // the generic kernel: nothing to choose
    hipStream_t s = (hipStream_t)stream;
    hipEvent_t e0, e1;
    if (hipEventCreate(&e0) != hipSuccess) return TCM_ERR_HIP;
    if (hipEventCreate(&e1) != hipSuccess) {
        (void)hipEventDestroy(e0);
        return TCM_ERR_HIP;
    }
    auto run = [&]() { return gemm_impl(1, M, N, K, A, lda, 0, B, ldb, 0, C, ldc, 0, dtype, bias, 0, epilogue, stream); };
    auto field = [](const std::string& plan, const char* key) {
        const char* q = strstr(plan.c_str(), key);
        return q ? atoll(q + strlen(key)) : -1LL;
    };
    // Time candidate c (`iters` calls); false if it cannot run as asked (an
    // ineligible config falls back to another plan).
    auto time_cand = [&](const Cand& c, double* us, int64_t* tiles) -> bool {
        t_cand = &c;
        st = run();  // warm-up, and the plan this candidate really gets
        const std::string plan = t_last_plan.text();
        const int pm = strstr(plan.c_str(), "mode=streamk") ? 2 : 1;
        const bool wide = strstr(plan.c_str(), "kernel=gemv") && strstr(plan.c_str(), " b_col=0 mfma=16x16x32");
        const bool as_asked = c.config == kGemvCand       ? strstr(plan.c_str(), "kernel=gemv") && !wide
                              : c.config == kGemvWideCand ? wide
                                                          : strstr(plan.c_str(), "kernel=tile") && field(plan, " config=") == c.config;
        if (st != TCM_OK || !as_asked || pm != c.mode) {
            t_cand = nullptr;
            return false;
        }
        if (tiles) *tiles = field(plan, " tiles=");
        if (hipEventRecord(e0, s) != hipSuccess) st = TCM_ERR_HIP;
        for (int i = 0; i < iters && st == TCM_OK; ++i) st = run();
        float ms = 0;
        if (st == TCM_OK && (hipEventRecord(e1, s) != hipSuccess || hipEventSynchronize(e1) != hipSuccess ||
                             hipEventElapsedTime(&ms, e0, e1) != hipSuccess))
            st = TCM_ERR_HIP;
        t_cand = nullptr;
        if (st != TCM_OK) return false;
        *us = (double)ms * 1e3 / iters;
        return true;
    };
    // The shader clock needs tens of milliseconds of load to settle: keep the
    // model's plan running for at least 50 ms (measured on the stream) first.
    {
        float warm_ms = 0;
        while (st == TCM_OK && warm_ms < 50.0f) {
            if (hipEventRecord(e0, s) != hipSuccess) st = TCM_ERR_HIP;
            for (int i = 0; i < 8 && st == TCM_OK; ++i) st = run();
            float ms = 0;
            if (st == TCM_OK && (hipEventRecord(e1, s) != hipSuccess || hipEventSynchronize(e1) != hipSuccess ||
                                 hipEventElapsedTime(&ms, e0, e1) != hipSuccess))
                st = TCM_ERR_HIP;
            warm_ms += ms;
            if (ms <= 0 && st == TCM_OK) break;
        }
    }
    // Stage 1: every tile config in both modes with the planner's other
    // parameters, and the split-k GEMV where it can serve the call; two
    // sweeps, each candidate keeping its better time.
    struct Timed {
        Cand c;
        double us;
        int64_t tiles;
    };
    std::vector<Timed> stage1;
    for (int c = 0; c < kNumConfigs; ++c)
        for (int mode = 1; mode <= 2; ++mode) {
            Cand x;
            x.config = c;
            x.mode = mode;
            stage1.push_back({x, 1e300, 0});
        }
    for (int gc : {kGemvCand, kGemvWideCand})
        if (gc == kGemvCand ? gemv_narrow_eligible(p) : gemv_wide_eligible(p)) {
            Cand x;
            x.config = gc;
            x.mode = 1;
            stage1.push_back({x, 1e300, 0});
        }
    std::vector<char> valid(stage1.size(), 1);
    for (int sweep = 0; sweep < 2 && st == TCM_OK; ++sweep)
        for (size_t i = 0; i < stage1.size() && st == TCM_OK; ++i) {
            if (!valid[i]) continue;
            double us = 0;
            if (!time_cand(stage1[i].c, &us, &stage1[i].tiles)) {
                valid[i] = 0;
                continue;
            }
            stage1[i].us = std::min(stage1[i].us, us);
        }
    std::vector<Timed> ranked;
    for (size_t i = 0; i < stage1.size(); ++i)
        if (valid[i]) ranked.push_back(stage1[i]);
    std::sort(ranked.begin(), ranked.end(), [](const Timed& x, const Timed& y) { return x.us < y.us; });
    // A data-parallel point within 2% of a faster Stream-K one ranks first:
    // within timing noise the plan without split tiles carries better to the
    // other shapes of its class (f32 768^3: Stream-K 17.42 against 17.50 us
    // data-parallel; on 1024^3, which uses that entry, 26.1 against 22.8 us).
    if (!ranked.empty() && ranked[0].c.mode == 2 && !gemv_cand(ranked[0].c.config))
        for (size_t i = 1; i < ranked.size(); ++i)
            if (ranked[i].c.mode == 1 && !gemv_cand(ranked[i].c.config) && ranked[i].us <= 1.02 * ranked[0].us) {
                std::rotate(ranked.begin(), ranked.begin() + i, ranked.begin() + i + 1);
                break;
            }
    // Stage 2: around the three fastest, the parameters the table leaves to
    // the planner: tile-order group rows; for Stream-K also the grid (per-CU
    // sizes, equal shares of every tile) and the way split tiles are summed.
    std::vector<Timed> stage2;
    const int cus = current_cus();
    for (size_t r = 0; r < ranked.size() && r < 3; ++r) {
        const Cand b = ranked[r].c;
        if (gemv_cand(b.config)) continue;  // nothing of the tile schedule applies
        const int64_t T = ranked[r].tiles;
        for (int gm : {1, 2, 8}) {
            Cand x = b;
            x.group_m = gm;
            stage2.push_back({x, 1e300, 0});
        }
        if (b.mode == 2 && split_config(b.config)) {
            // the eight-wave config's Stream-K is equal shares: their count
            // (per-CU grids would run its persistent kernel, and the shares
            // are always summed by the second kernel)
            for (int sh = 2; sh <= kMaxSplit; ++sh)
                if (T > 0 && T * sh <= cus) {  // (the planner caps the shares at one wave)
                    Cand x = b;
                    x.grid_kind = 2;
                    x.grid_param = sh;
                    stage2.push_back({x, 1e300, 0});
                }
        } else if (b.mode == 2) {
            for (int g8 : {4, 8, 12, 16}) {
                Cand x = b;
                x.grid_kind = 1;
                x.grid_param = g8;
                stage2.push_back({x, 1e300, 0});
            }
            for (int sh = 1; sh <= 4; ++sh)
                if (T > 0 && T * sh <= 4LL * cus) {
                    Cand x = b;
                    x.grid_kind = 2;
                    x.grid_param = sh;
                    stage2.push_back({x, 1e300, 0});
                }
            for (int fx : {1, 2}) {
                Cand x = b;
                x.fixup = fx;
                stage2.push_back({x, 1e300, 0});
            }
        }
    }
    std::vector<char> valid2(stage2.size(), 1);
    for (int sweep = 0; sweep < 2 && st == TCM_OK; ++sweep)
        for (size_t i = 0; i < stage2.size() && st == TCM_OK; ++i) {
            if (!valid2[i]) continue;
            double us = 0;
            if (!time_cand(stage2[i].c, &us, nullptr)) {
                valid2[i] = 0;
                continue;
            }
            stage2[i].us = std::min(stage2[i].us, us);
        }
    (void)hipEventDestroy(e0);
    (void)hipEventDestroy(e1);
    if (st != TCM_OK) return st;
    // A stage-2 variant must beat the best stage-1 point (the planner's own
    // grid, fix-up and group rows) by 2% to be kept: within timing noise the
    // planner's parameters win, since they adapt to other shapes of the
    // class and a fixed variant may not (three shares per tile, tuned on
    // 144 tiles, is the planner's own grid there but not on 100 tiles).
    const Timed* win = ranked.empty() ? nullptr : &ranked[0];
    const double bar = win ? 0.98 * win->us : 0.0;
    for (size_t i = 0; i < stage2.size(); ++i)
        if (valid2[i] && win && stage2[i].us < bar && stage2[i].us < win->us) win = &stage2[i];
    if (win) {
        std::lock_guard<std::mutex> lk(g_mu);
        g_tune[tune_key(p)] = TuneEntry{win->c, win->us, M, N, K};
    }
    if (best) return tcm_plan(M, N, K, lda, ldb, ldc, dtype, epilogue, p.aligned ? 1 : 0, best);
    return TCM_OK;
}

int tcm_tune_table(char* buf, int64_t len) {
    std::string out;
    {
        std::lock_guard<std::mutex> lk(g_mu);
        char line[320];
        for (const auto& kv : g_tune) {
            const TuneKey& k = kv.first;
            const TuneEntry& e = kv.second;
            snprintf(line, sizeof line, "tcm-tune-2 %d %d %d %d %d %d %d %d %d %d %d %d %d %d %d %d %.3f %lld %lld %lld\n",
                     k.dtype, k.a_col, k.b_col, k.c_type, k.epilogue, k.aligned, k.batched, k.mc, k.nc, k.kc, e.c.config,
                     e.c.mode, e.c.grid_kind, e.c.grid_param, e.c.fixup, e.c.group_m, e.us, (long long)e.M, (long long)e.N,
                     (long long)e.K);
            out += line;
        }
    }
    if (buf && len > 0) {
        const int64_t n = std::min<int64_t>(len - 1, (int64_t)out.size());
        memcpy(buf, out.data(), (size_t)n);
        buf[n] = 0;
    }
    return (int)out.size();
}

int tcm_tune_load(const char* text) {
    if (!text) return TCM_ERR_INVALID_VALUE;
    std::vector<std::pair<TuneKey, TuneEntry>> rows;
    if (parse_table(text, &rows) != TCM_OK) return TCM_ERR_INVALID_VALUE;
    std::lock_guard<std::mutex> lk(g_mu);
    for (const auto& r : rows) g_tune[r.first] = r.second;
    return TCM_OK;
}

void tcm_tune_clear(void) {
    std::lock_guard<std::mutex> lk(g_mu);
    g_tune.clear();
}

}  // extern "C"
