// Host-side declarations shared between the C ABI layer and the kernel
// launchers.  Launchers assume validated arguments and report launch errors
// through their hipError_t return value.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "vla.h"

namespace vla {

// ---------------------------------------------------------------- codec
hipError_t launch_quantize_pack(const float* W, void* Wq, float* scales, int64_t N, int64_t K,
                                int wfmt, int layout, hipStream_t s);
// MXFP4 block-scale bytes per weight row: K/32 rounded up to 8.
constexpr int64_t mxfp4_scale_row_bytes(int64_t K) { return ((K >> 5) + 7) & ~int64_t(7); }
hipError_t launch_mxfp4_quantize_pack(const float* W, uint8_t* Wq, int64_t N, int64_t K, hipStream_t s);
hipError_t launch_pack_fp8(const uint8_t* q, uint8_t* qp, int64_t N, int64_t K, hipStream_t s);
hipError_t launch_reencode(const uint8_t* q, const float* sc, uint8_t* q2, float* sc2, int64_t N,
                           int64_t K, int layout, hipStream_t s);
size_t quantize_act_ws_bytes(int64_t M, int64_t K);
hipError_t launch_quantize_act(const uint16_t* A, uint8_t* qa, float* s_a, void* ws, int64_t M,
                               int64_t K, hipStream_t s);
hipError_t launch_quantize_tokens_int8(const uint16_t* A, int8_t* qa, float* s_a, int64_t M, int64_t K, hipStream_t s);
hipError_t launch_gate_residual_ada_norm(const uint16_t* resid, const uint16_t* out, const uint16_t* gate,
                                         const uint16_t* style, int style_per_row, float eps, uint16_t* r_out,
                                         uint16_t* h_out, uint16_t* ng_out, int64_t M, int64_t D, hipStream_t s);
bool boundary_width_ok(int64_t D);   // D a positive multiple of 4, at most 8192

// ------------------------------------------------------------ attention
constexpr int kMostAxes = 4;                   // positions per token
struct RopeArgs {
    const uint16_t *q, *k, *v;
    const uint16_t *q_weight, *k_weight;       // nullable
    const float* inv_freq;
    const int32_t* positions;                  // axes rows of T
    const uint8_t* axis_of;                    // nullable: one axis
    const int64_t* slots;                      // nullable with the caches
    uint16_t *q_out, *k_out, *k_cache, *v_cache;   // k_out, caches nullable
    int64_t T, q_stride, k_stride, v_stride, q_out_stride, k_out_stride, num_slots;
    int Hq, Hkv, D, rot, interleaved, axes;
    float rot_scale, eps;
    int gw, gw_log2, chunks, steps;            // set by the launcher
};
hipError_t launch_qk_norm_rope_append(RopeArgs a, hipStream_t s);

// Division of 32-bit numbers by a number that the launch knows, in three
// instructions (Granlund and Montgomery, "Division by invariant integers using
// multiplication", 1994: the unsigned form, right for every numerator).  The
// compiler's own division takes about 25, and one that starts a workgroup is
// bound by its length.
struct Divisor {
    uint32_t d, mul, sh1, sh2;
    Divisor() = default;
    explicit Divisor(int64_t by) : d(static_cast<uint32_t>(by > 0 ? by : 1)) {
        uint32_t l = 0;
        while ((uint64_t(1) << l) < d) ++l;
        mul = static_cast<uint32_t>(((((uint64_t(1) << l) - d) << 32) / d) + 1);
        sh1 = l ? 1 : 0;
        sh2 = l ? l - 1 : 0;
    }
#ifdef __HIPCC__
    __device__ __forceinline__ int divide(int n, int& rest) const {   // n >= 0
        const uint32_t t = __umulhi(mul, static_cast<uint32_t>(n));
        const uint32_t q = (t + ((static_cast<uint32_t>(n) - t) >> sh1)) >> sh2;
        rest = n - static_cast<int>(q * d);
        return static_cast<int>(q);
    }
#endif
};

// Workgroups of one launch of the attention kernels: a launch dimension holds
// fewer than 2^32 threads, 256 to a workgroup.
constexpr int64_t kMostWorkgroups = (int64_t(1) << 24) - 1;

struct AppendArgs {
    const uint16_t *k, *v;
    const int32_t *cu_rows;                    // nullable: L rows per sequence
    const int32_t *block_table, *seq_lens;
    uint8_t *k_cache, *v_cache, *k_scales, *v_scales;
    int64_t k_stride, v_stride;
    int B, L, total, Hkv, D, page_log2, block_log2, pages_per_seq, capacity;
    uint32_t num_pages;
    // set by the launcher
    int dense, items, gw, gw_log2;
    Divisor by_most, by_heads2;
};
// Work items of an append, from its host sizes alone.
struct AppendPlan {
    bool dense;          // `most` items per sequence, else as many as it has blocks
    int64_t most, items; // items with the heads, keys and values apart
};
AppendPlan plan_kv_append(int64_t B, int64_t L, int64_t total, int64_t Hkv, int64_t block);
hipError_t launch_kv_append_e4m3(AppendArgs a, const AppendPlan& p, hipStream_t s);

struct PromptArgs {
    const uint16_t *q, *k, *v;
    const int32_t *cu_q, *cu_k;
    uint16_t* out;
    int64_t q_stride, k_stride, v_stride, out_stride;
    int B, total_q, total_k, Hq, Hkv, D, causal;
    float c;                                   // scale * log2(e)
    // set by the launcher
    int tiles;                                 // most row tiles per key/value head
    Divisor by_group, by_heads;                // query heads per key/value head; key/value heads, or the tiles
};
// Launch plan of a prompt call, from its host sizes alone.
struct PromptPlan {
    int tm;              // query rows per workgroup
    int64_t tiles;       // most row tiles per key/value head
};
PromptPlan plan_attn_prompt(int64_t B, int64_t total_q, int64_t Hq, int64_t Hkv, int64_t D, bool causal);
hipError_t launch_attn_prompt(PromptArgs a, const PromptPlan& p, hipStream_t s);

struct SharedArgs {
    const uint16_t *q, *k_cache, *v_cache;
    const int32_t *prefix_pages, *prefix_len;  // nullable: no prefix
    const int32_t *block_table, *seq_lens;     // nullable: no suffix
    uint16_t* out;
    int64_t q_stride, out_stride;
    int B, L, Hq, Hkv, D, causal;
    float c;
    int page_log2, pages_per_seq, prefix_cap, suffix_cap;   // capacities in keys
    uint32_t num_pages;
    // set by the launcher
    int merged, prefix_items, prefix_splits, suffix_splits, suffix_tiles, parts;
    Divisor by_group, by_q_heads, by_prefix_pairs, by_prefix_splits, by_suffix_pairs, by_suffix_splits, by_suffix_tiles;
    float *part_ml, *part_o;
    // a cache in codes alone
    const uint8_t *k_scales, *v_scales;
    int block_log2;
};
// Launch plan of a shared-prefix call, from its host sizes alone.
struct SharedPlan {
    bool merged;         // prefix and suffix are one range of keys
    int prefix_tm, suffix_tm;   // query rows per workgroup
    int64_t prefix_splits, suffix_splits, suffix_tiles, prefix_items, suffix_items, parts;
    int join_waves;      // per row, where its parts are joined
    int64_t ml_bytes, ws_bytes;
    int64_t workgroups;  // of the call's largest launch
};
SharedPlan plan_attn_shared(int64_t B, int64_t L, int64_t Hq, int64_t Hkv, int64_t D, int64_t prefix_cap,
                            int64_t suffix_cap, bool codes);
hipError_t launch_attn_shared(SharedArgs a, const SharedPlan& p, void* ws, hipStream_t s);
// The same over a cache in E4M3 codes (k_cache and v_cache point to bytes).
hipError_t launch_attn_shared_e4m3(SharedArgs a, const SharedPlan& p, void* ws, hipStream_t s);
void prepare_attn_shared(SharedArgs& a, const SharedPlan& p, void* ws);     // the launcher's fields
hipError_t launch_attn_join(const SharedArgs& a, const SharedPlan& p, hipStream_t s);

hipError_t launch_stream_read(const void* src, size_t bytes, uint32_t* sink, int blocks, hipStream_t s);
hipError_t launch_mfma_rate(int form, const uint32_t* src, int iters, float* out, uint64_t* clocks, int blocks,
                            hipStream_t s);
hipError_t launch_quantize_act_static(const uint16_t* A, const float* s_a, uint8_t* qa, int64_t M, int64_t K,
                                      hipStream_t s);

// ----------------------------------------------------------------- GEMM
enum class AType { BF16 = 0, FP8 = 1, INT8 = 2 };
enum class WType { BF16 = 0, FP8 = 1, FP4 = 2, INT8 = 3 };   // FP4: MXFP4 (E2M1 + E8M0 per 32 K); INT8 with INT8 A only
// The longest sum of 8-bit products that any codes keep inside 32 bits:
// K (2^7)^2 < 2^31 with K a multiple of 32.
constexpr int64_t kMostInt8K = 131040;
enum class Epi { PLAIN = 0, GELU_MUL = 1 };

struct GemmProblem {
    const void* A;
    const float* s_a;       // device scalar for FP8 A, M values for INT8 A, else nullptr
    const void* W;          // packed weights
    const float* s_w;       // per-row scales (FP8 and INT8 weights), else nullptr
    const uint16_t* bias;   // nullable
    const uint16_t* resid;  // nullable
    uint16_t* Y;            // PLAIN: M x N; GELU_MUL: M x N/2
    uint16_t* gu;           // GELU_MUL debug output M x N, nullable
    uint16_t* ypre;         // PLAIN: output before the residual add, M x N, nullable
    void* ws;
    int64_t M, N, K;        // N = weight rows
    AType atype;
    WType wtype;
    Epi epi;
};

// Launch plan chosen for a problem (host-side, deterministic per shape).
struct GemmPlan {
    int kernel;     // 0 = skinny (M <= 64), 1 = wide (above; 8-bit integers: also above 16 rows, large weights)
    int nt;         // skinny: 16-column tiles per workgroup; wide: tile width BN
    int steps;      // K steps (of 32) per wave per workgroup chunk (skinny)
    int waves;      // wavefronts per workgroup
    int wnw;        // wide: wavefronts along N (the rest are along M)
    int ksplit;     // number of K chunks across workgroups
    int groups;     // N groups (grid x)
    int mblocks;    // M blocks (wide: grid y of 192 rows; skinny: grid z of mt 16-row tiles)
    int mt;         // skinny: 16-row activation tiles per workgroup
    bool alds;      // skinny: stage activations through LDS
    bool ok;        // false when the shape exceeds the split-K counter or partial space
};

// The first kCounterBytes of every GEMM workspace hold the split-K arrival
// counters (one uint32 per skinny output group, kWideCounters per wide output
// tile: workgroups started, arrivals with handed-over slices, workgroups done),
// at the same place for every shape, so one zero-filled workspace can serve
// calls of different shapes.  Its last 4 KiB are not used.
constexpr size_t kCounterBytes = 65536;
constexpr size_t kZeroPageOffset = kCounterBytes - 4096;
constexpr int kMaxCounters = static_cast<int>(kZeroPageOffset / 4);
constexpr int kWideCounters = 4;   // three used, one pad
// The status word: the first 4 bytes of the page after the counters.  Zero
// until a bounded in-kernel wait gives up; each cause sets one bit.
constexpr size_t kStatusOffset = kZeroPageOffset;
constexpr uint32_t kStatusWideSplitK = 1u;   // wide split-K owner gave up waiting for partials
constexpr uint32_t kStatusChainBarrier = 2u;   // fused chain: a phase barrier gave up
// Split-K partial regions are addressed with 32-bit offsets.
constexpr uint64_t kMaxPartBytes = uint64_t(1) << 32;
// Default bound of every in-kernel wait, in polls (about 2 s of polling on
// MI355X; never reached by a grid that is resident).
constexpr uint32_t kDefaultWaitPolls = 1u << 22;
uint32_t wait_polls();                  // current bound (vla_set_wait_limit)

// vla_gemm_fp8w_noalloc's workspace: counters (64 KiB) + up to 32 MiB of
// split-K partials, enough for the encoder GEMMs at 768 rows.
constexpr size_t kNoAllocWorkspaceBytes = kCounterBytes + (size_t(32) << 20);
// Device address of the library's workspace on the current device (set up
// on first use per device; its counters are cleared by a kernel on `s`).
hipError_t noalloc_workspace(hipStream_t s, void** ptr);

// ------------------------------------------------------------ fused chain
// One persistent launch of kChainGrid workgroups runs every layer of the
// gated-MLP chain (chain.hip); the weight pointers travel in the kernel
// arguments, so at most kMaxChainLayers layers.
constexpr int kChainGrid = 256;
constexpr int kMaxChainLayers = 32;
// Barrier words of the fused chain (34 lines of 128 bytes), zero between
// launches; the chain scratch holds them after its GEMM workspace.
constexpr size_t kChainSyncBytes = 8192;

struct ChainLaunch {
    const uint8_t* const* wgu;     // host arrays of L device pointers
    const float* const* sgu;
    const uint8_t* const* wd;
    const float* const* sd;
    const uint16_t* x_in;
    uint16_t* x_out;
    uint16_t* xbuf;                // x after layers 0..L-2, xstride elements apart
    uint16_t* actbuf;              // act of layers 0..L-1, M * I elements apart
    uint16_t* gu_out;              // nullable per-layer stage outputs
    uint16_t* down_out;
    uint16_t* xlast;               // nullable second copy of the final x
    uint32_t* sync;
    uint32_t* err;
    int64_t xstride;
    int L;
    int64_t M, H, I;
    // decoder-block chain (style != nullptr): the boundary closes every layer
    const uint16_t* const* style = nullptr;   // host array of L device pointers
    int style_per_row = 0;
    float eps = 0.0f;
    const uint16_t* h_in = nullptr;
    const uint16_t* g_in = nullptr;
    uint16_t* h_out = nullptr;
    uint16_t* g_out = nullptr;
    uint16_t* hbuf = nullptr;                 // nullable per-layer stage output
    double* sspart = nullptr;                 // L x M x H/16 partial sums of squares
};
// Whether a compiled fused configuration covers (M, H, I, L); npa receives
// the gate/up pairs per workgroup.
bool chain_fused_plan(int64_t M, int64_t H, int64_t I, int L, int* npa);
// Whether the fused grid can be resident at once on the current device.
bool chain_fused_resident(int64_t H, int64_t I, int npa);
hipError_t launch_mlp_chain_fused(const ChainLaunch& c, hipStream_t s);

GemmPlan plan_gemm(int64_t M, int64_t N, int64_t K, AType at, WType wt, Epi epi);
size_t gemm_ws_bytes(const GemmPlan& p, int64_t M, int64_t N);
hipError_t launch_gemm(const GemmProblem& pr, hipStream_t s);
// Whether the plan names a compiled kernel configuration (host only).
bool plan_dispatchable(const GemmPlan& p, AType at, WType wt, Epi epi);

}  // namespace vla
