// Attention over packed prompts and over a paged key/value cache.
//
// One core serves both: a workgroup of four waves takes 128, 64 or 32 query
// rows of one key/value head and walks a range of keys in steps, with the
// running maximum and sum of a softmax per row, so scores never leave the
// registers.  The G = Hq / Hkv query heads that read one key/value head are
// rows of the same tile (row = token * G + g): keys are read once for all of
// them, and short sequences still fill the tiles.
//
//   S^T = K Q^T      v_mfma_f32_32x32x16_bf16, A = 32 keys, B = 32 query rows
//   P^T = exp2(c S^T - c m)      c = scale * log2(e), m = running row maximum
//   O^T += V^T P^T   the same instruction, A = 32 channels, B = P^T
//
// With the scores transposed a lane holds 16 keys of ONE row, so the row
// maximum and sum are 15 in-lane operations and one exchange between the wave
// halves, the rescaling factor is one value per lane, and P^T in accumulator
// layout already is the next product's B operand: lane half h holds keys
// 8 a + 4 h + (0..3), and because a product's keys may come in any order, V^T
// is read in that same order by LDS transpose reads (ds_read_b64_tr_b16: four
// keys of one channel per lane).  P never passes through LDS.
//
// P is rounded to bf16 (to nearest) for the second product, the form the
// matrix instruction takes; its relative error of at most 2^-8 per weight is
// that of the output's own rounding and averages over the keys.  Scores,
// maxima, sums and O are fp32; the sum is that of the unrounded weights.
//
// K and V rows go global -> LDS with 16-byte loads that write LDS directly.
// The 16-byte chunks of a row are XOR-swizzled so that the operand reads of K
// (32 rows, one chunk) and the transpose reads of V (4 keys x 64 bytes) are
// free of bank conflicts.  A row that is no key (past the range, on a page
// that does not exist) and channels past D load zeros, so nothing outside the
// tensors is read and no stale value meets a zero weight.
//
// What bounds it, and what it measured (a large bf16 matrix product reaches
// 1276 TFLOP/s here, a copy 5.14 TB/s): long prompts run at 1070 TFLOP/s of 128
// channels (16384 causal tokens, 32 heads on 8: 2.06 ms), 1060 of 256 (8192 x
// 8192, 8 heads on 1: 0.52 ms) and 800 of 64 (8192 x 8192, 16 heads on 2: 0.34
// ms); head sizes between these do the work of the next one (4000 x 4000, 16
// heads on 16 of 72: 134 us, of 80 131, of 128 141); a sub-tile's exponentials
// and the exchange of maxima stand between its two products and are covered by
// the other wave of the SIMD (up to 128 channels) or not at all (256).  One token
// over 131071 keys streams the cache at 5.0 TB/s.  Small calls (50 rows 6.3 us,
// 10 rows over 778 cached keys 10.6 us) are bound by the chain of a workgroup:
// its arguments and lengths, its first loads, one step, its results.  Two figures
// beside a rule below were measured side by side when the rule was made.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "attention_core.h"

namespace vla {
namespace {

// ------------------------------------------------------------------ prompt

// Workgroup -> (key/value head, rank of its row tile).  Workgroups go to the 8
// XCDs round robin: workgroups of one XCD share key/value heads, so a head's
// keys are fetched into one L2 (or into 8 / Hkv of them).
__device__ __forceinline__ void head_rank(const PromptArgs& a, int id, int& hk, int& rank) {
    if (a.Hkv % 8 == 0) {
        hk = a.by_heads.divide(id >> 3, rank) * 8 + (id & 7);         // by the tiles
    } else {
        rank = a.by_heads.divide(id, hk);                             // by the key/value heads
    }
}

// Sum over the wave, the same in every lane.
__device__ __forceinline__ uint32_t wave_sum(uint32_t x) {
    auto from = [&](auto ctrl, auto rows) __attribute__((always_inline)) {
        return static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(x), ctrl(), rows(), 0xF, false));
    };
    x += from(std::integral_constant<int, 0x111>{}, std::integral_constant<int, 0xF>{});   // row_shr:1
    x += from(std::integral_constant<int, 0x112>{}, std::integral_constant<int, 0xF>{});   // row_shr:2
    x += from(std::integral_constant<int, 0x114>{}, std::integral_constant<int, 0xF>{});   // row_shr:4
    x += from(std::integral_constant<int, 0x118>{}, std::integral_constant<int, 0xF>{});   // row_shr:8
    x += from(std::integral_constant<int, 0x142>{}, std::integral_constant<int, 0xA>{});   // row_bcast:15
    x += from(std::integral_constant<int, 0x143>{}, std::integral_constant<int, 0xC>{});   // row_bcast:31
    return __builtin_amdgcn_readlane(x, 63);
}

// One sequence's rows and keys, bounded to the tensors: no value in the
// offsets can lead outside.
struct Range {
    int q0, nq, k0, nk;
    __device__ __forceinline__ Range(const PromptArgs& a, int b) {
        bounded_rows(a.cu_q[b], a.cu_q[b + 1], a.total_q, q0, nq);
        bounded_rows(a.cu_k[b], a.cu_k[b + 1], a.total_k, k0, nk);
    }
    __device__ __forceinline__ Range() : q0(0), nq(0), k0(0), nk(0) {}
    __device__ __forceinline__ uint32_t tiles(int G, int tm) const {
        return (static_cast<uint32_t>(nq) * G + tm - 1) / tm;
    }
    __device__ __forceinline__ void from_lane(int lane) {
        q0 = __builtin_amdgcn_readlane(q0, lane);
        nq = __builtin_amdgcn_readlane(nq, lane);
        k0 = __builtin_amdgcn_readlane(k0, lane);
        nk = __builtin_amdgcn_readlane(nk, lane);
    }
};

// The row tile of rank `rank`: its sequence's range, and its place there as
// the result, or -1 if there are fewer tiles.
template <int TM>
__device__ __forceinline__ int find_tile(const PromptArgs& a, int G, int rank, Range& r) {
    const int lane = threadIdx.x & 63;
    if (a.B == 1) {
        r = Range(a, 0);
        r.from_lane(0);
        const uint32_t n = r.tiles(G, TM);
        return static_cast<uint32_t>(rank) < n ? static_cast<int>(n) - 1 - rank : -1;
    }
    if (a.B <= 64) {
        // One sequence per lane.  Tiles with most keys first, so that none of
        // them starts last: tile t of a sequence is on level t + `base`, base
        // being its keys ahead of its first row in units of a tile's rows (16
        // causal prompts of 1 to 1814 tokens, 28 heads on 4 of 128: 151 us, in
        // the sequences' order 154).  The level of rank `rank` is the highest
        // x with more than `rank` tiles on x and above.
        r = lane < a.B ? Range(a, lane) : Range();
        const uint32_t n = r.tiles(G, TM);
        const int64_t ahead = a.causal ? static_cast<int64_t>(r.nk) - r.nq : r.nk;
        const uint32_t base = n ? static_cast<uint32_t>(min(max(ahead, int64_t(0)) * G / TM, int64_t(1) << 20)) : 0;
        auto above = [&](uint32_t x) __attribute__((always_inline)) {   // tiles on level x and above
            return wave_sum(x <= base ? n : (x < base + n ? base + n - x : 0));
        };
        if (above(0) <= static_cast<uint32_t>(rank)) return -1;
        uint32_t lo = 0, size = 1;
        while (size < 0x80000000u && __any(base + n > size)) size *= 2;
        for (size /= 2; size; size /= 2)
            if (above(lo + size) > static_cast<uint32_t>(rank)) lo += size;
        // the level's tiles, one per sequence, in the sequences' order
        const uint64_t on = __ballot(lo >= base && lo < base + n);
        const uint32_t nth = static_cast<uint32_t>(rank) - above(lo + 1);
        const uint32_t mine = __builtin_amdgcn_mbcnt_hi(static_cast<uint32_t>(on >> 32), __builtin_amdgcn_mbcnt_lo(static_cast<uint32_t>(on), 0));
        const uint64_t hit = __ballot((on >> lane & 1) && mine == nth);
        const int src = __builtin_ctzll(hit);
        r.from_lane(src);
        return static_cast<int>(lo - __builtin_amdgcn_readlane(base, src));
    }
    // Many sequences: a scan over their tile counts, 64 at a time, the last
    // tiles of the batch first.
    const uint32_t tile = a.tiles - 1 - rank;
    uint32_t first = 0;
    for (int b0 = 0; b0 < a.B; b0 += 64) {
        r = b0 + lane < a.B ? Range(a, b0 + lane) : Range();
        const uint32_t n = r.tiles(G, TM);
        uint32_t incl = n;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const uint32_t up = __shfl_up(incl, o, 64);
            if (lane >= o) incl += up;
        }
        const uint64_t hit = __ballot(tile >= first + incl - n && tile < first + incl);
        if (hit) {
            const int src = __builtin_ctzll(hit);
            r.from_lane(src);
            return static_cast<int>(tile - __builtin_amdgcn_readlane(first + incl - n, src));
        }
        first += __builtin_amdgcn_readlane(incl, 63);
    }
    return -1;
}

template <class C>
__global__ __launch_bounds__(kAThreads) __attribute__((amdgpu_waves_per_eu(C::WAVES, C::WAVES)))
void attn_prompt_kernel(PromptArgs a) {
    ATTN_LDS;
    const int lane = threadIdx.x & 63;
    int hk, rank;
    head_rank(a, blockIdx.x, hk, rank);
    const int G = a.Hq / a.Hkv;
    Range at;
    const int rt = __builtin_amdgcn_readfirstlane(find_tile<C::TM>(a, G, rank, at));
    if (rt < 0) return;
    at.from_lane(0);
    const int q0 = at.q0, nq = at.nq, k0 = at.k0, nk = at.nk;

    const int rows = nq * G, r = rt * C::TM + wave_row<C>() + (lane & 31);
    const bool live = r < rows;
    int g;
    const int i = a.by_group.divide(r, g);
    const uint16_t* q = live ? a.q + static_cast<int64_t>(q0 + i) * a.q_stride + static_cast<int64_t>(hk * G + g) * a.D : nullptr;
    // ends aligned: row i sees key j <= i + nk - nq
    const int klim = a.causal ? min(max(i + 1 + nk - nq, 0), nk) : nk;
    int kend = nk;
    if (a.causal) {
        int rest;
        kend = min(max(a.by_group.divide(min((rt + 1) * C::TM, rows) - 1, rest) + 1 + nk - nq, 0), nk);
    }
    PackedKeys keys;
    keys.k = a.k + static_cast<int64_t>(k0) * a.k_stride + static_cast<int64_t>(hk) * a.D;
    keys.v = a.v + static_cast<int64_t>(k0) * a.v_stride + static_cast<int64_t>(hk) * a.D;
    keys.k_stride = static_cast<int>(a.k_stride) * 2;
    keys.v_stride = static_cast<int>(a.v_stride) * 2;
    keys.n = nk;
    State<C> st;
    attend<C>(keys, q, klim, 0, kend, a.D, a.c, b0, b1, b2, b3, st);
    uint16_t* const out = a.out + static_cast<int64_t>(q0 + i) * a.out_stride + static_cast<int64_t>(hk * G + g) * a.D;
    write_rows<C, false>(st, live ? reinterpret_cast<uint64_t>(out) : 0, nullptr, nullptr, a.D, b0, b1, b2, b3, ml, row_at);
}

// Joins a row's parts.  WPR waves per row (1 or 4) take every WPR-th part,
// eight parts' channels in flight at once (four channels per lane), and meet
// in LDS.
template <int WPR>
__global__ __launch_bounds__(kAThreads) void attn_join_kernel(SharedArgs a) {
    __shared__ f32x4_t o_all[4][64];
    __shared__ float l_all[4];
    const int lane = threadIdx.x & 63, ch = 4 * lane;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t row = static_cast<int64_t>(blockIdx.x) * (4 / WPR) + (WPR == 1 ? wave : 0);
    if (row >= static_cast<int64_t>(a.B) * a.L * a.Hq) return;    // WPR == 1 alone: no barrier follows
    const int w0 = WPR == 1 ? 0 : wave;
    const float* const ml = a.part_ml + 2 * row * a.parts;
    const float* const po = a.part_o + row * a.parts * a.D + ch;
    float m = -__builtin_inff();
    for (int p = lane; p < a.parts; p += 64) m = fmaxf(m, ml[2 * p]);
    m = wave_max(m);
    float l = 0.0f;
    f32x4_t o = f32x4_t{};
    const bool live = ch < a.D;
    // the wave's parts p = w0 + WPR i; lane i holds the weight of part i of a
    // group of 64
    for (int base = w0; base < a.parts; base += 64 * WPR) {
        const int pl = base + WPR * lane;
        float w = 0.0f;
        bool has = false;                                         // part pl saw a key
        if (pl < a.parts) {
            const float2 x = *reinterpret_cast<const float2*>(ml + 2 * pl);
            has = x.x != -__builtin_inff();
            w = x.x == -__builtin_inff() ? 0.0f : (x.x == m ? 1.0f : __builtin_amdgcn_exp2f(x.x - m));
            // a part without keys has sum 0, or NaN where every score was NaN
            l += x.x == -__builtin_inff() ? x.y : x.y * w;
        }
        const uint64_t there = __ballot(has);
        const int n = min(64, (a.parts - base + WPR - 1) / WPR);
        for (int i = 0; i < n; i += 8) {
            f32x4_t x[8];
            float wi[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                wi[j] = i + j < n ? __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(w), i + j)) : 0.0f;
                // a part without keys has nothing to add; one whose weight is
                // 0 in fp32 has its infinities and NaN
                x[j] = f32x4_t{};
                if ((there >> (i + j) & 1) && live) x[j] = *reinterpret_cast<const f32x4_t*>(po + static_cast<int64_t>(base + WPR * (i + j)) * a.D);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) o += x[j] * wi[j];
        }
    }
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) l += __shfl_xor(l, off, 64);
    if constexpr (WPR == 4) {
        o_all[wave][lane] = o;
        if (lane == 0) l_all[wave] = l;
        __syncthreads();
        if (wave != 0) return;
        l = l_all[0] + l_all[1] + l_all[2] + l_all[3];
        o = o_all[0][lane] + o_all[1][lane] + o_all[2][lane] + o_all[3][lane];
    }
    if (!live) return;
    const float inv = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);
    uint2 w;
    w.x = f32x2_to_bf16x2(o.x * inv, o.y * inv);
    w.y = f32x2_to_bf16x2(o.z * inv, o.w * inv);
    int head;
    const int token = a.by_q_heads.divide(static_cast<int>(row), head);
    *reinterpret_cast<uint2*>(a.out + token * a.out_stride + head * a.D + ch) = w;
}

constexpr int kComputeUnits = 256;

// Keys of a workgroup's step.
int step_keys(int64_t D, int tm, bool codes) { return (D <= 128 && tm == 32) || (codes && tm <= 32) ? 128 : 64; }

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

}  // namespace

PromptPlan plan_attn_prompt(int64_t B, int64_t total_q, int64_t Hq, int64_t Hkv, int64_t D, bool causal) {
    PromptPlan p{};
    const int64_t rows = total_q * (Hq / Hkv);
    // Narrow tiles where the GPU runs them all at once, wide ones, which load
    // less, where not: two workgroups per compute unit, one with 256 channels.
    // Of a causal prompt's tiles, half as long on average, up to one and a
    // half (64 rows: two) times as many.  Measured with 128 / 64 / 32 rows:
    //   32 heads on 8 of 128, all keys: 450 tokens 18.5 / 13.3 / 12.0 us, 1024
    //   tokens 30 / 27 / 34, 1500 tokens 54 / 55 / 63; causal: 1024 tokens 30 /
    //   21 / 25, 1500 tokens 42 / 36 / 40, 8191 tokens 575 / 640
    //   8 heads on 1 of 256, all keys: 800 tokens 36 / 25 / 21, 2048 tokens 71 /
    //   50 / 76, 2500 tokens 85 / 104 / 129; causal: 1500 tokens 56 / 37 / 31,
    //   3900 tokens 124 / 89 / 140
    // And no tile that the average sequence would not half fill.
    const int64_t slots = (D > 128 ? 1 : 2) * kComputeUnits;
    auto fits = [&](int tm) { return Hkv * ceil_div(rows, tm) <= (causal ? (tm == 64 ? 2 * slots : 3 * slots / 2) : slots); };
    p.tm = 128;
    while (p.tm > 32 && (2 * rows <= B * p.tm || fits(p.tm / 2))) p.tm /= 2;
    // every sequence ends in at most one partial tile
    p.tiles = rows / p.tm + (B < rows ? B : rows);
    return p;
}

hipError_t launch_attn_prompt(PromptArgs a, const PromptPlan& p, hipStream_t s) {
    a.tiles = static_cast<int>(p.tiles);
    a.by_group = Divisor(a.Hq / a.Hkv);
    a.by_heads = Divisor(a.Hkv % 8 == 0 ? a.tiles : a.Hkv);
    auto run = [&](auto cfg) {
        attn_prompt_kernel<decltype(cfg)><<<a.tiles * a.Hkv, kAThreads, 0, s>>>(a);
        return hipGetLastError();
    };
    return p.tm == 128 ? by_size<128>(a.D, run) : (p.tm == 64 ? by_size<64>(a.D, run) : by_size<32>(a.D, run));
}

SharedPlan plan_attn_shared(int64_t B, int64_t L, int64_t Hq, int64_t Hkv, int64_t D, int64_t prefix_cap,
                            int64_t suffix_cap, bool codes) {
    SharedPlan p{};
    const int64_t G = Hq / Hkv, rows_s = L * G, rows_p = B * rows_s;
    // As for prompts: narrow tiles where all of them run at once, and none that
    // one sequence's rows would not half fill (32 sequences of 50 tokens over
    // 850 keys, 8 heads on 1 of 256: 31 us with 64 rows, 43 with 128 rows and
    // the keys in two parts; 100 single tokens behind 4000 keys, 32 heads on 8
    // of 128: 33 us with 32 rows, 50 with 128).
    const int64_t slots = (D > 128 ? 1 : 2) * kComputeUnits;
    // Over a cache in codes, 16 rows where those tiles run at once too, three
    // workgroups per compute unit (16 chunks of 10 rows over 850 keys, 32 heads
    // on 8 of 128: 17.6 us, with 32 rows 24.0), and no taller few-row tile above
    // 128 channels, where 32 rows would not fit the registers.
    auto tile = [&](int64_t batches, int64_t rows) {
        int tm = 128;
        while (tm > 32 && (2 * rows <= tm || Hkv * batches * ceil_div(rows, tm / 2) <= slots)) tm /= 2;
        if (codes && tm == 32 && (rows <= 16 || D > 128 || Hkv * batches * ceil_div(rows, 16) <= 3 * kComputeUnits)) tm = 16;
        return tm;
    };
    p.prefix_tm = tile(1, rows_p);
    // A long prefix is worth 32 rows, which bring its codes half as often (64
    // single tokens of 32 heads on 8 of 128 with 300 keys of their own behind
    // 8000: 37.6 us, with 16 rows 47.6; behind 2051 with up to 3000 of their own
    // 71.5, with 16 rows 61.6).  The border lies between these two, unmeasured
    // there, and goes by the table's capacity, which is what the host knows.
    if (codes && p.prefix_tm == 16 && rows_p > 16 && D <= 128 && prefix_cap > 4096) p.prefix_tm = 32;
    p.suffix_tm = tile(B, rows_s);
    // A sequence whose rows fill its tiles reads the prefix no more often by
    // itself than a tile of the whole batch does: then the prefix is the head
    // of every sequence's range of keys and nothing has to be joined (32
    // sequences of 50 tokens over 800 shared keys: 31 us, apart 50; 64 single
    // tokens behind 8195 shared keys: apart 34 us, merged 114).
    p.merged = B == 1 || prefix_cap == 0 ||
               2 * B * ceil_div(rows_s, p.suffix_tm) * p.suffix_tm <= 3 * ceil_div(rows_p, p.prefix_tm) * p.prefix_tm;
    // 64-row tiles for the prefix take the suffixes into their launch, 128-row
    // ones would leave too much of theirs empty (single tokens behind a shared
    // prefix: 600 of 32 heads on 8 of 128, 64 rows: 87 us, two launches 98;
    // 2000, 128 rows: 287 us, two launches 241; 600 with 64 shared and up to
    // 1500 own keys, 64 rows: 403 us, two launches 396).
    if (!p.merged && p.prefix_tm == 64) p.suffix_tm = 64;
    // one launch for both as well where both are few
    if (codes && !p.merged && p.prefix_tm <= 32 && p.suffix_tm <= 32) p.suffix_tm = p.prefix_tm = std::max(p.prefix_tm, p.suffix_tm);
    const int64_t keys_s = suffix_cap + (p.merged ? prefix_cap : 0);
    const int64_t steps_p = p.merged ? 0 : ceil_div(prefix_cap, step_keys(D, p.prefix_tm, codes));
    const int64_t steps_s = ceil_div(keys_s, step_keys(D, p.suffix_tm, codes));
    const int64_t tiles_p = p.merged ? 0 : ceil_div(rows_p, p.prefix_tm);
    p.suffix_tiles = ceil_div(rows_s, p.suffix_tm);
    // Keys are split as often as the workgroups fit the compute units once (32
    // heads on 8 of 128: one token over 131071 keys 108 us, unsplit 1350; 8 and
    // 16 single tokens over up to 32768 own keys 138 and 249 us, unsplit 343
    // and 389; 64 behind 8195 shared and 300 own 31 us, unsplit 72).  Twice as
    // often, two workgroups to a compute unit, takes 112, 135, 256 and 39 us
    // for those, but from 129 to 256 workgroups, where this rule does not
    // split, it is ahead: 20 such tokens 436 us, halved 323, the bytes' time
    // 312.  With 64 of them the sequences fill the GPU (891 us, the bytes' 860).
    auto splits = [&](int64_t tiles, int64_t steps, int tm) {
        if (tiles == 0 || steps == 0) return int64_t(0);
        int64_t most = kComputeUnits / tiles;
        if (codes && tm <= 32) {
            // Few rows over codes take twice as many workgroups, whose loads
            // overlap (one token over 131071 keys: 65 us, with 256 workgroups
            // 69), and sequences, whose lengths differ, six times as many while
            // a part keeps 1024 keys: the long ones' parts then even out (32
            // heads on 8 of 128: 20 tokens over up to 20000 keys 114 us, with
            // 512 workgroups 125; 64 over up to 3000 58, with 512 61; 64 over
            // 1500 each 46, with parts of 512 keys 50).
            most = 2 * kComputeUnits / tiles;
            if (B > 1) most = std::max(most, std::min(6 * kComputeUnits / tiles, steps / 8));
        }
        return most <= 1 ? int64_t(1) : ceil_div(steps, ceil_div(steps, most));
    };
    p.prefix_splits = splits(Hkv * tiles_p, steps_p, 64);
    p.suffix_splits = splits(Hkv * B * p.suffix_tiles, steps_s, p.suffix_tm);
    p.prefix_items = Hkv * tiles_p * p.prefix_splits;
    p.suffix_items = Hkv * B * p.suffix_tiles * p.suffix_splits;
    p.parts = p.prefix_splits + p.suffix_splits;
    const int64_t rows = B * L * Hq;
    p.ml_bytes = p.parts > 1 ? ceil_div(rows * p.parts * 8, 256) * 256 : 0;
    p.ws_bytes = p.parts > 1 ? p.ml_bytes + rows * p.parts * D * 4 : 256;
    // four waves per row where the parts are many (80 rows of 13 parts, the
    // whole call: 11.5 us, with one wave 12.6), one where they are few (3200
    // rows of 2 parts: 22 us, with four waves 26)
    p.join_waves = p.parts > 8 ? 4 : 1;
    const int64_t join = p.parts > 1 ? ceil_div(rows * p.join_waves, 4) : 0;
    p.workgroups = std::max(p.prefix_tm == p.suffix_tm ? p.prefix_items + p.suffix_items
                                                       : std::max(p.prefix_items, p.suffix_items), join);
    return p;
}

void prepare_attn_shared(SharedArgs& a, const SharedPlan& p, void* ws) {
    a.merged = p.merged;
    a.prefix_splits = static_cast<int>(p.prefix_splits);
    a.suffix_splits = static_cast<int>(p.suffix_splits);
    a.suffix_tiles = static_cast<int>(p.suffix_tiles);
    a.parts = static_cast<int>(p.parts);
    a.by_group = Divisor(a.Hq / a.Hkv);
    a.by_q_heads = Divisor(a.Hq);
    a.by_prefix_pairs = Divisor(a.Hkv * p.prefix_splits);
    a.by_prefix_splits = Divisor(p.prefix_splits);
    a.by_suffix_pairs = Divisor(a.Hkv * p.suffix_splits);
    a.by_suffix_splits = Divisor(p.suffix_splits);
    a.by_suffix_tiles = Divisor(p.suffix_tiles);
    uint8_t* w = static_cast<uint8_t*>(ws);
    a.part_ml = reinterpret_cast<float*>(w);
    a.part_o = reinterpret_cast<float*>(w + p.ml_bytes);
}

hipError_t launch_attn_join(const SharedArgs& a, const SharedPlan& p, hipStream_t s) {
    const int64_t rows = static_cast<int64_t>(a.B) * a.L * a.Hq;
    if (p.join_waves == 4) attn_join_kernel<4><<<static_cast<unsigned>(rows), kAThreads, 0, s>>>(a);
    else attn_join_kernel<1><<<static_cast<unsigned>((rows + 3) / 4), kAThreads, 0, s>>>(a);
    return hipGetLastError();
}

hipError_t launch_attn_shared(SharedArgs a, const SharedPlan& p, void* ws, hipStream_t s) {
    prepare_attn_shared(a, p, ws);
    const bool wide = (static_cast<uint64_t>(a.num_pages) << a.page_log2) * a.Hkv * a.D * 2 > kNoOffset;
    const hipError_t e = launch_walks<PagedKeys>(a, p, wide, s);
    return e != hipSuccess || a.parts == 1 ? e : launch_attn_join(a, p, s);
}

}  // namespace vla
