// Attention over a paged key/value cache held in OCP E4M3 with a power-of-two
// scale per block of tokens and head.
//
// Tall tiles (64 and 128 query rows) take the walks over bf16 rows
// (attention.hip tells their mathematics): a row's codes are fetched into
// registers and enter LDS as the bf16 values they stand for, code times scale in
// one instruction per pair (exact: three fraction bits, and the scale only moves
// the exponent).
//
// Few rows (16 or 32 per key/value head: single tokens, short chunks) have a
// kernel of their own.  Its waves share no keys: each walks every fourth 32-key
// sub-tile by itself, with 16x16x32 products that waste less of a tile on rows
// that are not there, and what a wave does per key is kept small, since a byte
// of cache brings twice the keys that it does in bf16:
//
//   S^T = K Q^T      A = 16 keys: lane = key, 8 channels, read from the codes in
//                    LDS 16 at a time (Q is loaded in the same order of
//                    channels); codes become bf16 with the key's scale
//   P^T = exp2(c S^T - c m), times the values' scales relative to `ref`
//   O^T += V^T P^T   A = 16 channels x 32 keys, read from the codes in LDS by
//                    8-bit transpose reads whose rows are named in the order
//                    in which the scores' layout holds the keys; B = P^T as it is
//
// The values' scales go onto the weights, because a transpose read pairs keys
// that may lie in different blocks.  `ref` is a running scale, raised when a
// sub-tile brings one 2^20 times larger, so that weights times scales stay far
// from bf16's limits wherever the scales lie: keys whose scale is 2^100 below
// the largest that a wave has met lose precision, others do not.
//
// Measured, captured calls one behind another on caches of their own, 32 heads
// on 8 of 128 unless another is said (in parentheses the same keys in bf16): one
// token over 131071 keys 60-63 us, 4.25-4.5 TB/s (112); 64 single tokens behind
// 2051 shared and up to 3000 own keys 58-60 us, 3.5 TB/s (116); over 1500 own keys each
// 46 (79); 8 heads on 1 of 256, 10 rows over 778 keys 11.5 (11.1), one token over
// 30000 21.5 (23).  Bound by the loads of the cache, which three waves per SIMD
// keep in flight with one sub-tile each (128 channels; two need more registers
// than three waves have), and where the rows are few by the way through a
// launch, a part and its join.  Tall tiles are bound as the bf16 ones are, by the
// matrix pipes and the exponentials, and pay for the codes' conversion: 2048 rows
// over 8192 keys 320 us (282); of 256 channels, one workgroup of one wave per
// SIMD, whose accumulators leave the conversion no registers, 258 (170).
#include <hip/hip_runtime.h>

#include "attention_core.h"

namespace vla {
namespace {

// ------------------------------------------------------------- few rows

// DP padded channels, NR groups of 16 query rows.
template <int DP_, int NR_>
struct FCfg {
    static constexpr int DP = DP_, NR = NR_, TM = 16 * NR;
    static constexpr int NQ = DP / 32;           // products of K Q^T
    static constexpr int ND = DP / 16;           // 16-channel blocks of O^T
    static constexpr int CPR = DP / 16;          // 16-byte chunks of a row of codes
    static constexpr int RPI = 64 / CPR;         // rows per load instruction
    static constexpr int NI = 32 / RPI;          // loads of 32 rows
    static constexpr int ST = 128;               // keys per workgroup step
    static constexpr int BYTES = 32 * DP;        // codes of 32 rows
    static constexpr int O_BYTES = TM * DP * 4;  // a wave's part of the results
    static constexpr int LDS = 4 * O_BYTES;      // which take the codes' place, and more, at the end
    static_assert(O_BYTES >= 2 * BYTES, "a wave's keys and values fit its part");
    static constexpr int WAVES = DP > 128 || NR > 1 ? 2 : 3;   // per SIMD
    static constexpr int AHEAD = DP > 64 ? 1 : 2;   // sub-tiles on their way
};

// Position of a row's 16-byte chunks in LDS: chunk ^ swizzle.  One chunk of 16
// rows in a line (the keys' reads) and of rows 0-7 and 16-23, or 8-15 and 24-31
// (a half wave's transpose read), lies in as many places of the banks.  (The
// conflicts that counters show are the results' exchange at the end: 128 cycles a
// workgroup of 256 channels over 128 keys and over 512.)
template <int DP>
__device__ __forceinline__ int swz_codes(int row) {
    if constexpr (DP == 64) return (row >> 2 & 3) ^ (row >> 4) << 1;
    else if constexpr (DP == 128) return (row >> 1 & 7) ^ (row >> 4) << 2;
    else return (row & 15) ^ (row >> 4) << 3;
}

// Largest / sum over the four lanes of a row (lane l, l ^ 16, l ^ 32, l ^ 48).
__device__ __forceinline__ float row_max(float x) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return half_max(fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1])));
}
__device__ __forceinline__ float row_sum(float x) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return half_sum(__uint_as_float(r[0]) + __uint_as_float(r[1]));
}

// The top bit of each byte of a dword that is a NaN code.
__device__ __forceinline__ uint32_t nan_codes(uint32_t w) { return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u; }

// One workgroup, one work item, as in attn_shared_kernel.  ODD: head sizes that
// are no multiple of 16, whose rows start and end on 8 bytes.
template <class C, bool WIDE, bool ODD>
__global__ __launch_bounds__(kAThreads) __attribute__((amdgpu_waves_per_eu(C::WAVES, C::WAVES)))
void attn_few_codes_kernel(SharedArgs a) {
    __shared__ __attribute__((aligned(256))) uint8_t lds[C::LDS];
    __shared__ __attribute__((aligned(16))) float v_factor[4][32];
    __shared__ float ml[4][2][C::TM];
    __shared__ int refs[4];
    int id = blockIdx.x;
    const bool prefix = id < a.prefix_items;
    if (!prefix) id -= a.prefix_items;
    const int splits = prefix ? a.prefix_splits : a.suffix_splits;
    int pair, split, tile, b = 0;
    const int rest = (prefix ? a.by_prefix_pairs : a.by_suffix_pairs).divide(id, pair);
    const int hk = (prefix ? a.by_prefix_splits : a.by_suffix_splits).divide(pair, split);
    if (prefix) tile = rest;
    else b = a.by_suffix_tiles.divide(rest, tile);

    const int lane = threadIdx.x & 63, n16 = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int G = a.Hq / a.Hkv;
    const int np = a.prefix_pages ? min(max(a.prefix_len[0], 0), a.prefix_cap) : 0;
    int ns = 0;
    if (!prefix && a.block_table) ns = min(max(a.seq_lens[b], 0), a.suffix_cap);
    PagedCodes<WIDE> keys;
    keys.init(a, hk);
    keys.prefix = a.prefix_pages;
    keys.suffix = a.block_table ? a.block_table + static_cast<int64_t>(b) * a.pages_per_seq : nullptr;
    keys.n_prefix = (prefix || a.merged) ? np : 0;
    keys.n = keys.n_prefix + ns;
    keys.page_log2 = a.page_log2;
    keys.num_pages = a.num_pages;

    // the lane's rows, one of each group of 16
    const int rows = (prefix ? a.B : 1) * a.L * G, row0 = tile * C::TM;
    auto limit = [&](int row) __attribute__((always_inline)) {     // keys that a row of the item sees
        int unused;
        const int tok = a.by_group.divide(row, unused);
        return a.causal && !prefix ? keys.n_prefix + min(max(tok + 1 + ns - a.L, 0), ns) : keys.n;
    };
    int klim[C::NR];
    bf16x8_t qf[C::NR][C::NQ];
#pragma unroll
    for (int r = 0; r < C::NR; ++r) {
        const int row = row0 + 16 * r + n16;
        const bool live = row < rows;
        int h;
        const int64_t token = static_cast<int64_t>(b) * a.L + a.by_group.divide(row, h);
        const uint16_t* const q = a.q + token * a.q_stride + static_cast<int64_t>(hk * G + h) * a.D;
        klim[r] = limit(live ? row : rows - 1);
#pragma unroll
        for (int i = 0; i < C::NQ; ++i) {
            const int ch = 64 * (i / 2) + 16 * g + 8 * (i & 1);
            u32x4_t w = {0, 0, 0, 0};
            if (live && ch < a.D) w = *reinterpret_cast<const u32x4_t*>(q + ch);
            qf[r][i] = as_bf16x8(w);
        }
    }
    // every row sees keys below kfull
    const int kfull = __builtin_amdgcn_readfirstlane(limit(row0));

    const int steps = (keys.n + C::ST - 1) / C::ST;
    int unused;
    const int per = (prefix ? a.by_prefix_splits : a.by_suffix_splits).divide(steps + splits - 1, unused);
    // steps first: the last part's end in keys could pass 32 bits
    const int s0 = split * per, s1 = s0 + per;
    const int k0 = s0 >= steps ? keys.n : s0 * C::ST, k1 = s1 >= steps ? keys.n : s1 * C::ST;
    const int first = k0 + wave * 32;
    const int n = k1 > first ? (k1 - first + 127) / 128 : 0;

    // ---- fetches.  The lane's keys of a sub-tile are n16 and 16 + n16; it loads
    //      16 codes of rows i RPI + lane / CPR, for keys and values alike
    __amdgpu_buffer_rsrc_t rk, rv;
    if constexpr (!WIDE) {
        rk = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(keys.k), 0, keys.bytes, kBufferWord3);
        rv = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(keys.v), 0, keys.bytes, kBufferWord3);
    }
    // 16 codes from channel ch of the row at `at` (a byte offset past the cache
    // where there is none; WIDE: its slot)
    auto codes16 = [&](bool v, uint32_t at, int ch) __attribute__((always_inline)) -> u32x4_t {
        if constexpr (!WIDE) {
            const uint32_t off = ch < a.D ? at + ch : kNoOffset;
            if constexpr (!ODD) {
                return __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(v ? rv : rk, off, 0, 0));
            } else {
                const uint32_t off2 = ch + 8 < a.D ? at + ch + 8 : kNoOffset;
                const u32x2_t x = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_raw_buffer_load_b64(v ? rv : rk, off, 0, 0));
                const u32x2_t y = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_raw_buffer_load_b64(v ? rv : rk, off2, 0, 0));
                return u32x4_t{x.x, x.y, y.x, y.y};
            }
        } else {
            const uint8_t* const row = (v ? keys.v : keys.k) + static_cast<uint64_t>(at) * keys.stride + ch;
            const uint8_t* const none = reinterpret_cast<const uint8_t*>(kZeroChunk);
            const bool there = static_cast<int>(at) >= 0;
            if constexpr (!ODD) {
                return *reinterpret_cast<const u32x4_t*>(there && ch < a.D ? row : none);
            } else {
                const u32x2_t x = *reinterpret_cast<const u32x2_t*>(there && ch < a.D ? row : none);
                const u32x2_t y = *reinterpret_cast<const u32x2_t*>(there && ch + 8 < a.D ? row + 8 : none);
                return u32x4_t{x.x, x.y, y.x, y.y};
            }
        }
    };
    struct Stage {
        u32x4_t kc[C::NI], vc[C::NI];
        int slot[2];
        typename PagedCodes<WIDE>::Bytes bytes[2];
    };
    int32_t page[2] = {0, 0};                     // of the next sub-tile to fetch
    auto entries = [&](int t) __attribute__((always_inline)) {
#pragma unroll
        for (int h = 0; h < 2; ++h) page[h] = keys.entry(min(first + t * 128 + 16 * h + n16, k1 - 1));
    };
    auto fetch = [&](Stage& st, int t) __attribute__((always_inline)) {
        uint32_t at[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int key = first + t * 128 + 16 * h + n16;
            st.slot[h] = key < k1 ? keys.slot(key, page[h]) : -1;
            at[h] = WIDE ? static_cast<uint32_t>(st.slot[h])
                         : (st.slot[h] >= 0 ? static_cast<uint32_t>(st.slot[h]) * keys.stride : kNoOffset);
            st.bytes[h] = keys.bytes_of(st.slot[h]);
        }
        uint32_t from[C::NI];
#pragma unroll
        for (int i = 0; i < C::NI; ++i)
            from[i] = static_cast<uint32_t>(__shfl(static_cast<int>(at[i >= C::NI / 2]), (i * C::RPI + lane / C::CPR) & 15, 64));
#pragma unroll
        for (int i = 0; i < C::NI; ++i) st.kc[i] = codes16(false, from[i], 16 * ((lane % C::CPR) ^ swz_codes<C::DP>(i * C::RPI + lane / C::CPR)));
#pragma unroll
        for (int i = 0; i < C::NI; ++i) st.vc[i] = codes16(true, from[i], 16 * ((lane % C::CPR) ^ swz_codes<C::DP>(i * C::RPI + lane / C::CPR)));
        entries(t + 1);
    };
    Stage stages[C::AHEAD];
    if (n > 0) {
        entries(0);
#pragma unroll
        for (int i = 0; i < C::AHEAD; ++i)
            if (i < n) fetch(stages[i], i);
    }

    // ---- state: lane = row n16 of each group, channels 16 d + 4 g .. + 3
    f32x4_t acc[C::NR][C::ND];
    float m[C::NR], l[C::NR];
#pragma unroll
    for (int r = 0; r < C::NR; ++r) {
        m[r] = -__builtin_inff();
        l[r] = 0.0f;
#pragma unroll
        for (int d = 0; d < C::ND; ++d) acc[r][d] = f32x4_t{};
    }
    int ref = -4096;                              // the running scale's byte; none yet
    uint8_t* const kt = lds + wave * C::O_BYTES;
    uint8_t* const vt = kt + C::BYTES;
    // the keys' reads: row n16 (+ 16), chunk 4 j + g
    const int kaddr = n16 * C::DP + ((swz_codes<C::DP>(n16) ^ g) << 4);
    const int kaddr2 = (16 + n16) * C::DP + ((swz_codes<C::DP>(16 + n16) ^ g) << 4);
    // transpose read: rows 4 g + (0..3), 16 + 4 g + (0..3), two lanes each
    const int vrow = 4 * g + (n16 >> 1 & 3) + 16 * (n16 >> 3);
    const int vaddr = vrow * C::DP + (n16 & 1) * 8 + (swz_codes<C::DP>(vrow) << 4);
    auto v_frag = [&](int d) __attribute__((always_inline)) {
        typedef __attribute__((ext_vector_type(2))) int i32x2_t;
        const i32x2_t w = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
            (__attribute__((address_space(3))) i32x2_t*)(vt + (vaddr ^ (d << 4))));
        return __builtin_bit_cast(u32x2_t, w);
    };

    auto step = [&](Stage& st, int t) __attribute__((always_inline)) {
        const int key0 = first + t * 128;
        // the values' scales relative to the running one
        int e[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) e[h] = static_cast<int>(st.bytes[h].v) & ~(st.slot[h] >> 31);
        const int most = max(e[0] == 255 ? 0 : e[0], e[1] == 255 ? 0 : e[1]);   // a NaN scale is no measure
        if (__any(most > ref + 20)) {
            int top = most;
#pragma unroll
            for (int off = 8; off >= 1; off >>= 1) top = max(top, __shfl_xor(top, off, 64));   // the 16 lanes hold all 32 keys
            top = __builtin_amdgcn_readfirstlane(top);
            if (top > ref) {
                const float by = __uint_as_float(static_cast<uint32_t>(max(ref - top + 127, 0)) << 23);   // 2^-127 as 0
#pragma unroll
                for (int r = 0; r < C::NR; ++r)
#pragma unroll
                    for (int d = 0; d < C::ND; ++d) acc[r][d] *= by;
                ref = top;
            }
        }
        float f[2], ks[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            f[h] = e[h] == 255 ? 0.0f : __uint_as_float(static_cast<uint32_t>(max(e[h] - ref + 127, 0)) << 23);
            // 0 where there is no slot, so that the zeros loaded there stay zeros
            ks[h] = __uint_as_float(PagedCodes<WIDE>::scale_bits(st.bytes[h].k) << 16 & ~(st.slot[h] >> 31));
        }
        if (g < 2) v_factor[wave][lane] = g ? f[1] : f[0];
        // values whose scale is NaN: they count as 0 in the weights, so that unseen
        // ones stay out, and reach the rows that see them after the product's weights
        const uint32_t nan_scales = static_cast<uint32_t>(__ballot(e[0] == 255) & 0xFFFFu) |
                                    static_cast<uint32_t>(__ballot(e[1] == 255) & 0xFFFFu) << 16;
        bool bad = false;                          // a NaN code that some row may not see
        if (key0 + 32 > kfull) {
            uint32_t any = 0;
#pragma unroll
            for (int i = 0; i < C::NI; ++i) any |= nan_codes(st.vc[i].x) | nan_codes(st.vc[i].y) | nan_codes(st.vc[i].z) | nan_codes(st.vc[i].w);
            bad = __any(any != 0);
        }
#pragma unroll
        for (int i = 0; i < C::NI; ++i) {
            *reinterpret_cast<u32x4_t*>(kt + i * 1024 + lane * 16) = st.kc[i];
            *reinterpret_cast<u32x4_t*>(vt + i * 1024 + lane * 16) = st.vc[i];
        }
        const uint32_t vm = static_cast<uint32_t>(__ballot(st.slot[0] >= 0) & 0xFFFFu) |
                            static_cast<uint32_t>(__ballot(st.slot[1] >= 0) & 0xFFFFu) << 16;

        if (t + C::AHEAD < n) fetch(st, t + C::AHEAD);

        __builtin_amdgcn_sched_barrier(0);
        // ---- scores: lane = row n16, keys 16 h + 4 g + i
        f32x4_t s[C::NR][2];
#pragma unroll
        for (int r = 0; r < C::NR; ++r)
#pragma unroll
            for (int h = 0; h < 2; ++h) s[r][h] = f32x4_t{};
        u32x4_t kw[2][C::NQ / 2];
#pragma unroll
        for (int j = 0; j < C::NQ / 2; ++j)
#pragma unroll
            for (int h = 0; h < 2; ++h) kw[h][j] = *reinterpret_cast<const u32x4_t*>(kt + ((h ? kaddr2 : kaddr) ^ (j << 6)));
#pragma unroll
        for (int i = 0; i < C::NQ; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const u32x4_t w = kw[h][i / 2];
                const bf16x8_t kf = as_bf16x8(ocp8_to_bf16x8_scaled(i & 1 ? u32x2_t{w.z, w.w} : u32x2_t{w.x, w.y}, ks[h]));
#pragma unroll
                for (int r = 0; r < C::NR; ++r) s[r][h] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf, qf[r][i], s[r][h], 0, 0, 0);
            }

        __builtin_amdgcn_sched_barrier(0);
        // ---- weights
        const f32x4_t vf0 = *reinterpret_cast<const f32x4_t*>(&v_factor[wave][4 * g]);
        const f32x4_t vf1 = *reinterpret_cast<const f32x4_t*>(&v_factor[wave][16 + 4 * g]);
        u32x4_t pw[C::NR];
        float mx[C::NR];
        bool moves = false;
#pragma unroll
        for (int r = 0; r < C::NR; ++r) {
#pragma unroll
            for (int h = 0; h < 2; ++h) s[r][h] *= a.c;
            if (key0 + 32 > kfull || vm != 0xFFFFFFFFu) {
                const int lim = klim[r] - key0 - 4 * g;
                const uint32_t seen = vm >> (4 * g);
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        s[r][h][i] = 16 * h + i < lim && (seen >> (16 * h + i) & 1u) ? s[r][h][i] : -__builtin_inff();
            }
            mx[r] = fmaxf(fmaxf(fmaxf(s[r][0][0], s[r][0][1]), fmaxf(s[r][0][2], s[r][0][3])),
                          fmaxf(fmaxf(s[r][1][0], s[r][1][1]), fmaxf(s[r][1][2], s[r][1][3])));
            moves |= mx[r] > m[r] + kLag;
        }
        if (__any(moves)) {
#pragma unroll
            for (int r = 0; r < C::NR; ++r) {
                const float mn = fmaxf(m[r], row_max(mx[r]));
                const float al = mn == m[r] ? 1.0f : __builtin_amdgcn_exp2f(m[r] - mn);
                m[r] = mn;
                l[r] *= al;
#pragma unroll
                for (int d = 0; d < C::ND; ++d) acc[r][d] *= al;
            }
        }
#pragma unroll
        for (int r = 0; r < C::NR; ++r) {
            const float m0 = m[r] == -__builtin_inff() ? 0.0f : m[r];      // a row that has seen no key: exp2(-inf) = 0
            float p[8], sum[2];
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float w = __builtin_amdgcn_exp2f(s[r][h][i] - m0);
                    sum[h] = i ? sum[h] + w : w;
                    p[4 * h + i] = w * (h ? vf1[i] : vf0[i]);
                }
            l[r] += sum[0] + sum[1];
            pw[r] = u32x4_t{f32x2_to_bf16x2(p[0], p[1]), f32x2_to_bf16x2(p[2], p[3]), f32x2_to_bf16x2(p[4], p[5]), f32x2_to_bf16x2(p[6], p[7])};
        }
        if (bad) {
            // A zero weight times NaN is not zero: NaN codes go to the rows that
            // see them by hand, and leave LDS before the product.
            for (int j = 0; j < 32; ++j) {
                if (!(vm >> j & 1u)) continue;
#pragma unroll
                for (int r = 0; r < C::NR; ++r) {
                    const float sees = key0 + j < klim[r] ? __builtin_nanf("") : 0.0f;
#pragma unroll
                    for (int d = 0; d < C::ND; ++d) {
                        const uint32_t c4 = *reinterpret_cast<const uint32_t*>(vt + j * C::DP + ((d ^ swz_codes<C::DP>(j)) << 4) + 4 * g);
#pragma unroll
                        for (int i = 0; i < 4; ++i) acc[r][d][i] += (c4 >> (8 * i) & 0x7Fu) == 0x7Fu ? sees : 0.0f;
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < C::NI; ++i) {
                u32x4_t* const at = reinterpret_cast<u32x4_t*>(vt + i * 1024 + lane * 16);
                u32x4_t w = *at;
#pragma unroll
                for (int x = 0; x < 4; ++x) w[x] &= ~((nan_codes(w[x]) >> 7) * 0xFFu);
                *at = w;
            }
        }
        if (nan_scales != 0) {
            // every channel of the rows that see the first of them, also where its
            // weight is 0 (a score of -inf)
#pragma unroll
            for (int r = 0; r < C::NR; ++r) {
                const float sees = key0 + __builtin_ctz(nan_scales) < klim[r] ? __builtin_nanf("") : 0.0f;
#pragma unroll
                for (int d = 0; d < C::ND; ++d) acc[r][d] += sees;
            }
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int d = 0; d < C::ND; ++d) {
            const bf16x8_t vf = ocp8_to_bf16x8(v_frag(d));
#pragma unroll
            for (int r = 0; r < C::NR; ++r) acc[r][d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vf, as_bf16x8(pw[r]), acc[r][d], 0, 0, 0);
        }
    };
    for (int t = 0; t < n; t += C::AHEAD)
#pragma unroll
        for (int i = 0; i < C::AHEAD; ++i)
            if (i == 0 || t + i < n) step(stages[i], t + i);

    // ---- the waves' parts, scaled to their common maximum, meet in LDS
#pragma unroll
    for (int r = 0; r < C::NR; ++r) {
        l[r] = row_sum(l[r]);
        if (g == 0) {
            ml[wave][0][16 * r + n16] = m[r];
            ml[wave][1][16 * r + n16] = l[r];
        }
    }
    if (lane == 0) refs[wave] = ref;
    __syncthreads();                              // every wave is past its codes, too
    const int top = max(max(refs[0], refs[1]), max(refs[2], refs[3]));
    const bool direct = a.parts == 1;
#pragma unroll
    for (int r = 0; r < C::NR; ++r) {
        const int row = 16 * r + n16;
        float mk[4], mm = -__builtin_inff();
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            mk[k] = ml[k][0][row];
            mm = fmaxf(mm, mk[k]);
        }
        float ll = 0.0f;
#pragma unroll
        for (int k = 0; k < 4; ++k) ll += ml[k][1][row] * (mk[k] == mm ? 1.0f : __builtin_amdgcn_exp2f(mk[k] - mm));
        float by = m[r] == mm ? 1.0f : __builtin_amdgcn_exp2f(m[r] - mm);
        by *= __uint_as_float(static_cast<uint32_t>(max(ref - top + 127, 0)) << 23);
        if (direct) by *= ll > 0.0f ? 1.0f / ll : (ll == 0.0f ? 0.0f : ll);       // NaN stays NaN
        else if (wave == 0 && g == 0 && row0 + row < rows) {
            int h;
            const int64_t token = static_cast<int64_t>(b) * a.L + a.by_group.divide(row0 + row, h);
            const int64_t at = (token * a.Hq + hk * G + h) * a.parts + (prefix ? 0 : a.prefix_splits) + split;
            *reinterpret_cast<float2*>(a.part_ml + 2 * at) = make_float2(klim[r] > k0 ? fmaxf(mm, kSeen) : mm, ll);
        }
        uint8_t* const mine = lds + wave * C::O_BYTES + row * C::DP * 4;
#pragma unroll
        for (int d = 0; d < C::ND; ++d)
            *reinterpret_cast<f32x4_t*>(mine + (((4 * d + g) ^ n16) & (C::DP / 4 - 1)) * 16) = acc[r][d] * by;
    }
    __syncthreads();
    // 8 channels per thread and pass; real values are the running scale's multiple
    const float up = top > 0 ? e8m0_to_f32(static_cast<uint32_t>(top)) : (top == 0 ? 0x1p-127f : 1.0f);
    constexpr int CG = C::DP / 8;
#pragma unroll 1
    for (int x = threadIdx.x; x < C::TM * CG; x += kAThreads) {
        const int row = x / CG, cg = x % CG;
        if (row0 + row >= rows || cg * 8 >= a.D) continue;
        f32x4_t o[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint8_t* const at = lds + row * C::DP * 4 + (((2 * cg + i) ^ (row & 15)) & (C::DP / 4 - 1)) * 16;
            o[i] = *reinterpret_cast<const f32x4_t*>(at);
#pragma unroll
            for (int k = 1; k < 4; ++k) o[i] += *reinterpret_cast<const f32x4_t*>(at + k * C::O_BYTES);
            o[i] *= up;
        }
        int h;
        const int64_t token = static_cast<int64_t>(b) * a.L + a.by_group.divide(row0 + row, h);
        if (direct) {
            const u32x4_t w = {f32x2_to_bf16x2(o[0].x, o[0].y), f32x2_to_bf16x2(o[0].z, o[0].w),
                               f32x2_to_bf16x2(o[1].x, o[1].y), f32x2_to_bf16x2(o[1].z, o[1].w)};
            *reinterpret_cast<u32x4_t*>(a.out + token * a.out_stride + static_cast<int64_t>(hk * G + h) * a.D + cg * 8) = w;
        } else {
            const int64_t at = (token * a.Hq + hk * G + h) * a.parts + (prefix ? 0 : a.prefix_splits) + split;
            f32x4_t* const p = reinterpret_cast<f32x4_t*>(a.part_o + at * a.D + cg * 8);
            p[0] = o[0];
            p[1] = o[1];
        }
    }
}

template <int DP, int NR>
hipError_t launch_few(const SharedArgs& a, int grid, bool wide, hipStream_t s) {
    using C = FCfg<DP, NR>;
    if (a.D % 16) {
        if (wide) attn_few_codes_kernel<C, true, true><<<grid, kAThreads, 0, s>>>(a);
        else attn_few_codes_kernel<C, false, true><<<grid, kAThreads, 0, s>>>(a);
    } else {
        if (wide) attn_few_codes_kernel<C, true, false><<<grid, kAThreads, 0, s>>>(a);
        else attn_few_codes_kernel<C, false, false><<<grid, kAThreads, 0, s>>>(a);
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_attn_shared_e4m3(SharedArgs a, const SharedPlan& p, void* ws, hipStream_t s) {
    prepare_attn_shared(a, p, ws);
    const bool wide = (static_cast<uint64_t>(a.num_pages) << a.page_log2) * a.Hkv * a.D > kNoOffset;
    auto run = [&](int tm, int64_t prefix_items, int64_t suffix_items) {
        a.prefix_items = static_cast<int>(prefix_items);
        const int grid = static_cast<int>(prefix_items + suffix_items);
        if (grid == 0) return hipSuccess;
        auto tall = [&](auto cfg) {
            if (wide) attn_shared_kernel<decltype(cfg), PagedCodes<true>><<<grid, kAThreads, 0, s>>>(a);
            else attn_shared_kernel<decltype(cfg), PagedCodes<false>><<<grid, kAThreads, 0, s>>>(a);
            return hipGetLastError();
        };
        if (tm == 128) return by_size<128>(a.D, tall);
        if (tm == 64) return by_size<64>(a.D, tall);
        if (a.D > 128) return launch_few<256, 1>(a, grid, wide, s);
        if (tm == 32) return a.D > 64 ? launch_few<128, 2>(a, grid, wide, s) : launch_few<64, 2>(a, grid, wide, s);
        return a.D > 64 ? launch_few<128, 1>(a, grid, wide, s) : launch_few<64, 1>(a, grid, wide, s);
    };
    hipError_t e;
    if (p.prefix_tm == p.suffix_tm) {
        e = run(p.prefix_tm, p.prefix_items, p.suffix_items);
    } else {
        e = run(p.prefix_tm, p.prefix_items, 0);
        if (e == hipSuccess) e = run(p.suffix_tm, 0, p.suffix_items);
    }
    return e != hipSuccess || a.parts == 1 ? e : launch_attn_join(a, p, s);
}

}  // namespace vla
