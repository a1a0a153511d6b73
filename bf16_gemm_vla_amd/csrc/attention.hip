// Attention over packed prompts and over a paged key/value cache.
//
// One core serves both: a workgroup of four waves takes QW x 32 query rows of
// one key/value head and walks a range of keys in stages of ST, with the
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
// K and V rows go global -> LDS with 16-byte loads that write LDS directly,
// double-buffered, one barrier per stage.  The 16-byte chunks of a row are
// XOR-swizzled so that the operand reads of K (32 rows, one chunk) and the
// transpose reads of V (4 keys x 64 bytes) spread over the banks.  A row that is no key (past the
// range, on a page that does not exist) and channels past D load zeros from a
// constant instead, so nothing outside the tensors is read and no stale value
// meets a zero weight.
#include <hip/hip_runtime.h>

#include <climits>
#include <cstdint>
#include <type_traits>

#include "vla_device.h"
#include "vla_internal.h"

namespace vla {
namespace {

typedef __attribute__((ext_vector_type(16))) float f32x16_t;
typedef __attribute__((ext_vector_type(4))) short s16x4_t;

constexpr int kAThreads = 256;

__device__ __attribute__((aligned(16))) const uint32_t kZeroChunk[4] = {0, 0, 0, 0};

// QW waves along the rows x KW waves along the keys of a stage.
template <int DP_, int QW_, int KW_>
struct ACfg {
    static constexpr int DP = DP_, QW = QW_, KW = KW_;
    static_assert(QW * KW * 64 == kAThreads, "four waves");
    static constexpr int TM = 32 * QW;                       // query rows per workgroup
    static constexpr int WK = KW == 1 ? 64 : 32;             // keys per wave per stage
    static constexpr int ST = WK * KW;                       // keys per stage
    static constexpr int SUB = WK / 32;                      // 32-key sub-tiles per wave per stage
    static constexpr int CH = DP / 8;                        // 16-byte chunks per row
    static constexpr int RB = DP * 2;                        // bytes per row
    static constexpr int R = WK / QW;                        // rows a wave loads per stage (of K and of V)
    static constexpr int RPI = 1024 / RB;                    // rows per load instruction
    static constexpr int NI = R / RPI;
    static constexpr int HALF = ST * RB;                     // bytes of K (and of V) per stage
    static constexpr int STAGE = 2 * HALF;
    static constexpr int NK = DP / 16;                       // MFMA steps of K Q^T
    static constexpr int ND = DP / 32;                       // 32-channel blocks of O^T
    static_assert(R % RPI == 0, "whole load instructions");
    static_assert((KW - 1) * QW * 64 * (ND * 16 + 2) * 4 <= 2 * STAGE, "the key waves join through the stage buffers");
};

// Position of a row's 16-byte chunks in LDS: chunk ^ swizzle.
template <int DP>
__device__ __forceinline__ int swz_k(int row) { return DP == 64 ? (row >> 1) & 7 : row & 15; }
template <int DP>
__device__ __forceinline__ int swz_v(int row) { return DP == 64 ? ((row >> 1) & 1) << 2 : (row & 3) << 2; }

// Keys 0 .. n-1 of one key/value head: rows of packed tensors, or rows of the
// cache named by the page tables (first the prefix's keys, then the suffix's).
struct PackedKeys {
    const uint16_t *k, *v;     // row 0 of this head
    int64_t k_stride, v_stride;
    int n;
};
struct PagedKeys {
    const uint16_t *k, *v;     // slot 0 of this head
    int64_t stride;
    const int32_t *prefix, *suffix;
    int n_prefix, n;           // prefix keys, all keys
    int page_log2;
    uint32_t num_pages;
};

template <class C>
struct State {
    f32x16_t acc[C::ND];
    float m, l;
};

// Exchange between the wave halves: the value of lane ^ 32 combined by max / +.
__device__ __forceinline__ float half_max(float x) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float half_sum(float x) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// Whether 32 rows of V in a stage buffer hold an infinity or NaN (any chunk
// order: all of them are looked at).
template <class C>
__device__ __forceinline__ bool has_nonfinite(const uint8_t* buf, int row) {
    const uint8_t* v = buf + C::HALF + row * C::RB + (threadIdx.x & 63) * 16;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 32 * C::RB / 1024; ++i) {
        const u32x4_t w = *reinterpret_cast<const u32x4_t*>(v + i * 1024);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            bad |= (w[j] & 0x7F80u) == 0x7F80u || (w[j] & 0x7F800000u) == 0x7F800000u;
    }
    return __any(bad);
}

// O += P V for 32 keys of the stage, one key after another, leaving out the
// keys the lane's row does not see (key >= limit, or not in vm).  Slow and
// rare: only values that are infinite or NaN need it.
template <class C>
__device__ __forceinline__ void add_by_key(const uint8_t* buf, int row, int limit, uint32_t vm, const uint32_t* pw,
                                           State<C>& st) {
    const int lane = threadIdx.x & 63, l32 = lane & 31, g2 = lane >> 5;
#pragma unroll 1
    for (int r = 0; r < 32; ++r) {
        // weight of key r: accumulator value 4 (r / 8) + r % 4 of half (r / 4) % 2
        const int wi = 2 * (r >> 3) + ((r & 3) >> 1);
        uint32_t w = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) w = wi == i ? pw[i] : w;
        w = __shfl(w, l32 + 32 * ((r >> 2) & 1), 64);
        const float p = __uint_as_float((r & 1) ? (w & 0xFFFF0000u) : (w << 16));
        const bool seen = r < limit && ((vm >> r) & 1u);
        const uint8_t* v = buf + C::HALF + (row + r) * C::RB + g2 * 8;
        const int sw = swz_v<C::DP>(r);
#pragma unroll
        for (int d = 0; d < C::ND; ++d)
#pragma unroll
            for (int a = 0; a < 4; ++a) {
                const uint2 x = *reinterpret_cast<const uint2*>(v + ((4 * d + a) ^ sw) * 16);
                const float f[4] = {__uint_as_float(x.x << 16), __uint_as_float(x.x & 0xFFFF0000u),
                                    __uint_as_float(x.y << 16), __uint_as_float(x.y & 0xFFFF0000u)};
#pragma unroll
                for (int j = 0; j < 4; ++j) st.acc[d][4 * a + j] += seen ? p * f[j] : 0.0f;
            }
    }
}

// Walks keys k0 .. k1-1 (a uniform range) for this wave's 32 rows.  q: the
// lane's query row or nullptr; klim: keys the lane's row may see (its first
// klim keys); D channels.  Leaves the row's partial result of this wave's
// keys in st.
template <class C, class Keys>
__device__ __forceinline__ void attend(const Keys& keys, const uint16_t* q, int klim, int k0, int k1, int D, float c,
                                       uint8_t* buf0, uint8_t* buf1, State<C>& st) {
    constexpr bool PAGED = std::is_same<Keys, PagedKeys>::value;
    constexpr int DP = C::DP;
    const int lane = threadIdx.x & 63, l32 = lane & 31, g2 = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int qw = wave % C::QW, kw = wave / C::QW;

    // query fragments: B operand, lane = row l32, channels 16 kk + 8 g2 .. +7
    bf16x8_t qf[C::NK];
#pragma unroll
    for (int kk = 0; kk < C::NK; ++kk) {
        const int d = 16 * kk + 8 * g2;
        u32x4_t w = {0, 0, 0, 0};
        if (q && d < D) w = *reinterpret_cast<const u32x4_t*>(q + d);
        qf[kk] = as_bf16x8(w);
    }
    // bounds of the rows this wave holds: all rows see keys below kfull, none
    // sees a key at or past kmax
    int kfull = q ? klim : INT_MAX, kmax = q ? klim : 0;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
        kfull = min(kfull, __shfl_xor(kfull, o, 64));
        kmax = max(kmax, __shfl_xor(kmax, o, 64));
    }
    kfull = __builtin_amdgcn_readfirstlane(kfull);
    kmax = __builtin_amdgcn_readfirstlane(kmax);

#pragma unroll
    for (int i = 0; i < C::ND; ++i) st.acc[i] = f32x16_t{};
    st.m = -__builtin_inff();
    st.l = 0.0f;

    const int n_stages = (k1 - k0 + C::ST - 1) / C::ST;
    if (n_stages <= 0) return;

    // ---- loads of a stage.  Wave (qw, kw) loads R rows of K and of V of key
    //      window kw; lane l keeps the slot of window key l % WK.
    const int row0 = kw * C::WK + qw * C::R;                      // first stage row this wave loads
    const int lrow = lane / C::CH, lpos = lane % C::CH;
    auto table_entry = [&](int s) __attribute__((always_inline)) -> int {
        if constexpr (!PAGED) {
            return 0;
        } else {
            const int key = k0 + s * C::ST + kw * C::WK + (lane & (C::WK - 1));
            if (key >= k1) return -1;
            const bool pre = key < keys.n_prefix;
            const int j = pre ? key : key - keys.n_prefix;
            const int32_t* t = pre ? keys.prefix : keys.suffix;
            const uint32_t page = static_cast<uint32_t>(t[j >> keys.page_log2]);
            if (page >= keys.num_pages) return -1;
            return static_cast<int>((page << keys.page_log2) | (j & ((1 << keys.page_log2) - 1)));
        }
    };
    auto issue = [&](uint8_t* buf, int s, int slot) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < C::NI; ++i) {
            const int rr = i * C::RPI + lrow;                     // row among this wave's R
            const int sr = row0 + rr;                             // row of the stage
            const int ck = lpos ^ swz_k<DP>(sr), cv = lpos ^ swz_v<DP>(sr);
            const uint16_t *pk, *pv;
            bool ok;
            if constexpr (PAGED) {
                const int sl = __shfl(slot, qw * C::R + rr, 64);
                ok = sl >= 0;
                const int64_t off = static_cast<int64_t>(sl) * keys.stride;
                pk = keys.k + off;
                pv = keys.v + off;
            } else {
                const int key = k0 + s * C::ST + sr;
                ok = key < k1;
                pk = keys.k + key * keys.k_stride;
                pv = keys.v + key * keys.v_stride;
            }
            const uint16_t* zero = reinterpret_cast<const uint16_t*>(kZeroChunk);
            const uint16_t* sk = ok && ck * 8 < D ? pk + ck * 8 : zero;
            const uint16_t* sv = ok && cv * 8 < D ? pv + cv * 8 : zero;
            uint8_t* dst = buf + (row0 + i * C::RPI) * C::RB;
            __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)sk,
                                             (__attribute__((address_space(3))) void*)dst, 16, 0, 0);
            __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)sv,
                                             (__attribute__((address_space(3))) void*)(dst + C::HALF), 16, 0, 0);
        }
    };

    // ---- LDS operand addresses within a stage
    const int kbase = (kw * C::WK + l32) * C::RB + ((swz_k<DP>(l32) ^ g2) << 4);      // ^ (kk << 5)
    const int i16 = lane & 15, g16 = (lane >> 4) & 1;
    // transpose read: key 4 g2 + i16/4 of an 8-key group, channels 16 g16 + 4 (i16 % 4)
    const int vrow = 4 * g2 + (i16 >> 2);
    const int vbase = C::HALF + (kw * C::WK + vrow) * C::RB + (i16 & 1) * 8;
    const int vchunk = 2 * g16 + ((i16 & 3) >> 1), vswz = swz_v<DP>(i16 >> 2);

    auto compute = [&](const uint8_t* buf, int s, uint64_t vmask) __attribute__((always_inline)) {
#pragma unroll
        for (int sub = 0; sub < C::SUB; ++sub) {
            const int key0 = k0 + s * C::ST + kw * C::WK + sub * 32;
            if (key0 >= kmax) break;
            f32x16_t sc = f32x16_t{};
#pragma unroll
            for (int kk = 0; kk < C::NK; ++kk) {
                const u32x4_t kf = *reinterpret_cast<const u32x4_t*>(buf + ((kbase ^ (kk << 5)) + sub * 32 * C::RB));
                sc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(as_bf16x8(kf), qf[kk], sc, 0, 0, 0);
            }
            // masks: rows that end inside the tile, rows of missing pages
            const uint32_t vm = static_cast<uint32_t>(vmask >> (32 * sub));
            const bool ragged = key0 + 32 > kfull;                // some row does not see every key here
            if (ragged || vm != 0xFFFFFFFFu) {
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int r = 8 * (i / 4) + 4 * g2 + (i % 4);
                    sc[i] = (key0 + r < klim && ((vm >> r) & 1u)) ? sc[i] : -__builtin_inff();
                }
            }
            float mx = sc[0];
#pragma unroll
            for (int i = 1; i < 16; ++i) mx = fmaxf(mx, sc[i]);
            mx = half_max(mx);
            if (__any(mx > st.m)) {
                const float mn = fmaxf(st.m, mx);
                const float al = mn == st.m ? 1.0f : __builtin_amdgcn_exp2f((st.m - mn) * c);
                st.m = mn;
                st.l *= al;
#pragma unroll
                for (int d = 0; d < C::ND; ++d)
#pragma unroll
                    for (int i = 0; i < 16; ++i) st.acc[d][i] *= al;
            }
            // a row that has seen no key yet: weights exp2(-inf) = 0
            const float mc = st.m == -__builtin_inff() ? 0.0f : st.m * c;
            float sum = 0.0f;
            uint32_t pw[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float p0 = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[2 * i], c, -mc));
                const float p1 = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[2 * i + 1], c, -mc));
                sum += p0 + p1;
                pw[i] = f32x2_to_bf16x2(p0, p1);
            }
            st.l += sum;
            // a product with a zero weight is not zero where V is infinite or
            // NaN: such a tile that some row sees in part goes key by key
            if (ragged && has_nonfinite<C>(buf, kw * C::WK + sub * 32)) {
                add_by_key<C>(buf, kw * C::WK + sub * 32, klim - key0, vm, pw, st);
                continue;
            }
            // O^T += V^T P^T, 16 keys per step
#pragma unroll
            for (int k2 = 0; k2 < 2; ++k2) {
                const u32x4_t pv = {pw[4 * k2], pw[4 * k2 + 1], pw[4 * k2 + 2], pw[4 * k2 + 3]};
                const bf16x8_t pf = as_bf16x8(pv);
#pragma unroll
                for (int d = 0; d < C::ND; ++d) {
                    const uint8_t* va = buf + vbase + (((d * 4) ^ vswz) + vchunk) * 16 + (sub * 32 + 16 * k2) * C::RB;
                    const s16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4_t*)va);
                    const s16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                        (__attribute__((address_space(3))) s16x4_t*)(va + 8 * C::RB));
                    const u32x2_t a = __builtin_bit_cast(u32x2_t, lo), b = __builtin_bit_cast(u32x2_t, hi);
                    const u32x4_t vf = {a.x, a.y, b.x, b.y};
                    st.acc[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(as_bf16x8(vf), pf, st.acc[d], 0, 0, 0);
                }
            }
        }
    };

    auto valid = [&](int slot) __attribute__((always_inline)) -> uint64_t {
        if constexpr (PAGED) return __ballot(slot >= 0);
        else return ~uint64_t(0);
    };
    // stage s lives in buffer s % 2; its loads are issued while stage s-1 is
    // computed, its table entries are read one stage earlier still
    int slot = table_entry(0);
    issue(buf0, 0, slot);
    uint64_t vcur = valid(slot);
    slot = n_stages > 1 ? table_entry(1) : 0;
    auto step = [&](const uint8_t* cur, uint8_t* next, int s) __attribute__((always_inline)) {
        // this wave's loads of stage s have landed and its reads of stage s-1
        // are done (vmcnt 0, lgkmcnt 0); the barrier says so for every wave
        __builtin_amdgcn_sched_barrier(0);
        __atomic_signal_fence(__ATOMIC_SEQ_CST);
        __builtin_amdgcn_s_waitcnt(0x0070);
        __builtin_amdgcn_s_barrier();
        __atomic_signal_fence(__ATOMIC_SEQ_CST);
        __builtin_amdgcn_sched_barrier(0);
        uint64_t vnext = 0;
        if (s + 1 < n_stages) {
            issue(next, s + 1, slot);
            vnext = valid(slot);
            if (s + 2 < n_stages) slot = table_entry(s + 2);
        }
        compute(cur, s, vcur);
        vcur = vnext;
    };
    for (int s = 0; s < n_stages; s += 2) {
        step(buf0, buf1, s);
        if (s + 1 < n_stages) step(buf1, buf0, s + 1);
    }
    st.l = half_sum(st.l);
}

// Joins the key waves' partial results into the waves with kw = 0.
template <class C>
__device__ __forceinline__ void join_key_waves(uint8_t* buf0, uint8_t* buf1, float c, State<C>& st) {
    if constexpr (C::KW > 1) {
        const int lane = threadIdx.x & 63;
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        const int qw = wave % C::QW, kw = wave / C::QW;
        constexpr int PER = 64 * (C::ND * 16 + 2);                // floats per wave
        constexpr int PERBUF = C::STAGE / (PER * 4);              // waves' states per buffer
        static_assert(PERBUF >= 1 && 2 * PERBUF >= (C::KW - 1) * C::QW, "room for every joining wave");
        auto area = [&](int k) -> float* {
            const int at = (k - 1) * C::QW + qw;
            return reinterpret_cast<float*>(at < PERBUF ? buf0 : buf1) + (at % PERBUF) * PER + lane;
        };
        __syncthreads();                                          // every wave is past its last stage
        if (kw > 0) {
            float* a = area(kw);
#pragma unroll
            for (int d = 0; d < C::ND; ++d)
#pragma unroll
                for (int i = 0; i < 16; ++i) a[(d * 16 + i) * 64] = st.acc[d][i];
            a[C::ND * 16 * 64] = st.m;
            a[(C::ND * 16 + 1) * 64] = st.l;
        }
        __syncthreads();
        if (kw == 0) {
#pragma unroll
            for (int k = 1; k < C::KW; ++k) {
                const float* a = area(k);
                const float m2 = a[C::ND * 16 * 64], l2 = a[(C::ND * 16 + 1) * 64];
                const float mn = fmaxf(st.m, m2);
                const float s1 = st.m == mn ? 1.0f : __builtin_amdgcn_exp2f((st.m - mn) * c);
                const float s2 = m2 == mn ? 1.0f : __builtin_amdgcn_exp2f((m2 - mn) * c);
                st.m = mn;
                st.l = st.l * s1 + l2 * s2;
#pragma unroll
                for (int d = 0; d < C::ND; ++d)
#pragma unroll
                    for (int i = 0; i < 16; ++i) st.acc[d][i] = st.acc[d][i] * s1 + a[(d * 16 + i) * 64] * s2;
            }
        }
    }
}

// The row's result, O / l rounded to bf16; a row without keys is 0.
template <class C>
__device__ __forceinline__ void store_row(const State<C>& st, uint16_t* out, int D) {
    const int g2 = (threadIdx.x >> 5) & 1;
    const float inv = st.l > 0.0f ? 1.0f / st.l : (st.l == 0.0f ? 0.0f : st.l);   // NaN stays NaN
#pragma unroll
    for (int d = 0; d < C::ND; ++d)
#pragma unroll
        for (int a = 0; a < 4; ++a) {
            const int ch = 32 * d + 8 * a + 4 * g2;
            if (ch < D) {
                uint2 w;
                w.x = f32x2_to_bf16x2(st.acc[d][4 * a] * inv, st.acc[d][4 * a + 1] * inv);
                w.y = f32x2_to_bf16x2(st.acc[d][4 * a + 2] * inv, st.acc[d][4 * a + 3] * inv);
                *reinterpret_cast<uint2*>(out + ch) = w;
            }
        }
}

// ------------------------------------------------------------------ prompt

// Workgroup -> (key/value head, row tile).  Workgroups go to the 8 XCDs round
// robin: workgroups of one XCD share key/value heads, so a head's keys are
// fetched into one L2 (or into 8 / Hkv of them), and row tiles come last rows
// first, so the longest causal tiles do not start last.
__device__ __forceinline__ void head_tile(int id, int Hkv, int tiles, int& hk, int& tile) {
    if (Hkv % 8 == 0) {
        const int x = id & 7, j = id >> 3;
        hk = (j / tiles) * 8 + x;
        tile = j % tiles;
    } else {
        hk = id % Hkv;
        tile = id / Hkv;
    }
    tile = tiles - 1 - tile;
}

template <class C>
__global__ __launch_bounds__(kAThreads) void attn_prompt_kernel(PromptArgs a) {
    __shared__ __attribute__((aligned(16))) uint8_t buf0[C::STAGE];
    __shared__ __attribute__((aligned(16))) uint8_t buf1[C::STAGE];
    const int lane = threadIdx.x & 63;
    int hk, tile;
    head_tile(blockIdx.x, a.Hkv, a.tiles, hk, tile);

    // which sequence holds row tile `tile`: a scan over the sequences' tile
    // counts, 64 at a time.  Offsets are bounded to the tensors here, so no
    // value in them can lead outside.
    const int G = a.Hq / a.Hkv;
    int q0 = 0, nq = 0, k0 = 0, nk = 0, first = 0, found = 0;
    for (int base = 0; base < a.B && !found; base += 64) {
        const int b = base + lane;
        int s = 0, n = 0, t = 0;
        if (b < a.B) {
            s = min(max(a.cu_q[b], 0), a.total_q);
            n = max(min(a.cu_q[b + 1], a.total_q) - s, 0);
            t = static_cast<int>((static_cast<int64_t>(n) * G + C::TM - 1) / C::TM);
        }
        int incl = t;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int up = __shfl_up(incl, o, 64);
            if (lane >= o) incl += up;
        }
        const bool here = t > 0 && tile >= first + incl - t && tile < first + incl;
        const uint64_t hit = __ballot(here);
        if (hit) {
            const int src = __builtin_ctzll(hit);
            q0 = __shfl(s, src, 64);
            nq = __shfl(n, src, 64);
            const int bb = base + src;
            k0 = min(max(a.cu_k[bb], 0), a.total_k);
            nk = max(min(a.cu_k[bb + 1], a.total_k) - k0, 0);
            first = __shfl(first + incl - t, src, 64);
            found = 1;
        } else {
            first += __shfl(incl, 63, 64);
        }
    }
    if (!found) return;
    q0 = __builtin_amdgcn_readfirstlane(q0);
    nq = __builtin_amdgcn_readfirstlane(nq);
    k0 = __builtin_amdgcn_readfirstlane(k0);
    nk = __builtin_amdgcn_readfirstlane(nk);
    const int rt = tile - __builtin_amdgcn_readfirstlane(first);

    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t rows = static_cast<int64_t>(nq) * G;
    const int64_t r = static_cast<int64_t>(rt) * C::TM + (wave % C::QW) * 32 + (lane & 31);
    const bool live = r < rows;
    const int i = static_cast<int>(r / G), g = static_cast<int>(r - static_cast<int64_t>(i) * G);
    const uint16_t* q = live ? a.q + static_cast<int64_t>(q0 + i) * a.q_stride + static_cast<int64_t>(hk * G + g) * a.D : nullptr;
    // ends aligned: row i sees key j <= i + nk - nq
    const int klim = a.causal ? min(max(i + 1 + nk - nq, 0), nk) : nk;
    int kend = nk;
    if (a.causal) {
        const int64_t lastr = min(static_cast<int64_t>(rt + 1) * C::TM, rows) - 1;
        kend = min(max(static_cast<int>(lastr / G) + 1 + nk - nq, 0), nk);
    }
    PackedKeys keys;
    keys.k = a.k + static_cast<int64_t>(k0) * a.k_stride + static_cast<int64_t>(hk) * a.D;
    keys.v = a.v + static_cast<int64_t>(k0) * a.v_stride + static_cast<int64_t>(hk) * a.D;
    keys.k_stride = a.k_stride;
    keys.v_stride = a.v_stride;
    keys.n = nk;
    State<C> st;
    attend<C>(keys, q, klim, 0, kend, a.D, a.c, buf0, buf1, st);
    join_key_waves<C>(buf0, buf1, a.c, st);
    if (wave / C::QW == 0 && live)
        store_row<C>(st, a.out + static_cast<int64_t>(q0 + i) * a.out_stride + static_cast<int64_t>(hk * G + g) * a.D, a.D);
}

// ----------------------------------------------------------- shared prefix

// One work item: a row tile of one key/value head against one split of the
// shared prefix (rows of the whole batch) or of one sequence's suffix.  With
// one sequence both are one range of keys.  More than one part per row: the
// parts' unnormalised O, maximum and sum go to the workspace.
template <class C>
__device__ __forceinline__ void shared_item(const SharedArgs& a, int hk, int tile, int split, int splits, int part,
                                            int b, bool prefix, uint8_t* buf0, uint8_t* buf1) {
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int G = a.Hq / a.Hkv;
    const int np = a.prefix_pages ? min(max(a.prefix_len[0], 0), a.prefix_cap) : 0;
    int ns = 0;
    if (!prefix && a.block_table) ns = min(max(a.seq_lens[b], 0), a.suffix_cap);
    PagedKeys keys;
    keys.stride = static_cast<int64_t>(a.Hkv) * a.D;
    keys.k = a.k_cache + static_cast<int64_t>(hk) * a.D;
    keys.v = a.v_cache + static_cast<int64_t>(hk) * a.D;
    keys.prefix = a.prefix_pages;
    keys.suffix = a.block_table ? a.block_table + static_cast<int64_t>(b) * a.pages_per_seq : nullptr;
    keys.n_prefix = (prefix || a.merged) ? np : 0;
    keys.n = keys.n_prefix + ns;
    keys.page_log2 = a.page_log2;
    keys.num_pages = a.num_pages;

    // rows: of the whole batch for the prefix, else of sequence b
    const int rows = (prefix ? a.B : 1) * a.L * G;
    const int r = tile * C::TM + (wave % C::QW) * 32 + (lane & 31);
    const bool live = r < rows;
    const int tok = r / G, g = r - tok * G;
    const int64_t token = static_cast<int64_t>(prefix ? 0 : b) * a.L + tok;       // of B * L
    const int head = hk * G + g;
    const uint16_t* q = live ? a.q + token * a.q_stride + static_cast<int64_t>(head) * a.D : nullptr;
    int klim = keys.n;
    if (a.causal && !prefix) klim = keys.n_prefix + min(max(tok + 1 + ns - a.L, 0), ns);
    const int stages = (keys.n + C::ST - 1) / C::ST, per = (stages + splits - 1) / splits;
    const int k0 = min(split * per * C::ST, keys.n), k1 = min((split + 1) * per * C::ST, keys.n);
    State<C> st;
    attend<C>(keys, q, klim, k0, k1, a.D, a.c, buf0, buf1, st);
    join_key_waves<C>(buf0, buf1, a.c, st);
    if (wave / C::QW != 0 || !live) return;
    if (a.parts == 1) {
        store_row<C>(st, a.out + token * a.out_stride + static_cast<int64_t>(head) * a.D, a.D);
        return;
    }
    const int64_t at = (token * a.Hq + head) * a.parts + part;
    const int g2 = lane >> 5;
    if (g2 == 0) *reinterpret_cast<float2*>(a.part_ml + 2 * at) = make_float2(st.m, st.l);
    if (st.m == -__builtin_inff()) return;
    float* o = a.part_o + at * a.D;
#pragma unroll
    for (int d = 0; d < C::ND; ++d)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const int ch = 32 * d + 8 * x + 4 * g2;
            if (ch < a.D)
                *reinterpret_cast<float4*>(o + ch) =
                    make_float4(st.acc[d][4 * x], st.acc[d][4 * x + 1], st.acc[d][4 * x + 2], st.acc[d][4 * x + 3]);
        }
}

template <class CP, class CS>
__global__ __launch_bounds__(kAThreads) void attn_shared_kernel(SharedArgs a) {
    constexpr int STAGE = CP::STAGE > CS::STAGE ? CP::STAGE : CS::STAGE;
    __shared__ __attribute__((aligned(16))) uint8_t buf0[STAGE];
    __shared__ __attribute__((aligned(16))) uint8_t buf1[STAGE];
    int id = blockIdx.x;
    // (head, split) fastest: the row tiles that read the same keys are Hkv *
    // splits apart, on one XCD when that is a multiple of 8
    if (id < a.prefix_items) {
        const int pair = id % (a.Hkv * a.prefix_splits);
        shared_item<CP>(a, pair / a.prefix_splits, id / (a.Hkv * a.prefix_splits), pair % a.prefix_splits,
                        a.prefix_splits, pair % a.prefix_splits, 0, true, buf0, buf1);
    } else {
        id -= a.prefix_items;
        const int pair = id % (a.Hkv * a.suffix_splits);
        const int rest = id / (a.Hkv * a.suffix_splits);
        const int split = pair % a.suffix_splits;
        shared_item<CS>(a, pair / a.suffix_splits, rest % a.suffix_tiles, split, a.suffix_splits,
                        (a.prefix_items ? a.prefix_splits : 0) + split, rest / a.suffix_tiles, false, buf0, buf1);
    }
}

// Joins a row's parts: one wave per row, four channels per lane.
__global__ __launch_bounds__(kAThreads) void attn_join_kernel(SharedArgs a) {
    const int lane = threadIdx.x & 63;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * (kAThreads / 64) + (threadIdx.x >> 6);
    if (row >= static_cast<int64_t>(a.B) * a.L * a.Hq) return;
    const float* ml = a.part_ml + 2 * row * a.parts;
    float m = -__builtin_inff();
    for (int p = lane; p < a.parts; p += 64) m = fmaxf(m, ml[2 * p]);
    m = wave_max(m);
    const int ch = 4 * lane;
    float l = 0.0f;
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    const float* po = a.part_o + row * a.parts * a.D + ch;
    for (int p = 0; p < a.parts; ++p) {
        const float mp = ml[2 * p];
        if (mp == -__builtin_inff()) {
            l += ml[2 * p + 1];                                   // 0, or NaN where every score was NaN
            continue;
        }
        const float w = mp == m ? 1.0f : __builtin_amdgcn_exp2f((mp - m) * a.c);
        l += ml[2 * p + 1] * w;
        if (ch < a.D) {
            const float4 x = *reinterpret_cast<const float4*>(po + static_cast<int64_t>(p) * a.D);
            o.x += x.x * w; o.y += x.y * w; o.z += x.z * w; o.w += x.w * w;
        }
    }
    if (ch >= a.D) return;
    const float inv = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);
    uint2 w;
    w.x = f32x2_to_bf16x2(o.x * inv, o.y * inv);
    w.y = f32x2_to_bf16x2(o.z * inv, o.w * inv);
    const int64_t token = row / a.Hq;
    *reinterpret_cast<uint2*>(a.out + token * a.out_stride + (row - token * a.Hq) * a.D + ch) = w;
}

// Tiles by padded head size: many rows (128 x 64 keys a stage) and few rows
// (32 x 128, or 64 x 64 where 128 keys of 256 channels would not fit LDS twice).
template <int DP> using Many = ACfg<DP, 4, 1>;
template <int DP> struct FewOf { using type = ACfg<DP, 1, 4>; };
template <> struct FewOf<256> { using type = ACfg<256, 2, 2>; };
template <int DP> using Few = typename FewOf<DP>::type;

int pad_d(int D) { return D <= 64 ? 64 : (D <= 128 ? 128 : 256); }
int few_rows(int D) { return pad_d(D) == 256 ? 64 : 32; }
int stage_keys(int D, bool many) { return many || pad_d(D) == 256 ? 64 : 128; }

constexpr int kComputeUnits = 256;

template <int DP>
hipError_t prompt_dispatch(const PromptArgs& a, bool many, int grid, hipStream_t s) {
    if (many) attn_prompt_kernel<Many<DP>><<<grid, kAThreads, 0, s>>>(a);
    else attn_prompt_kernel<Few<DP>><<<grid, kAThreads, 0, s>>>(a);
    return hipGetLastError();
}

template <int DP>
hipError_t shared_dispatch(const SharedArgs& a, bool pm, bool sm, int grid, hipStream_t s) {
    if (pm && sm) attn_shared_kernel<Many<DP>, Many<DP>><<<grid, kAThreads, 0, s>>>(a);
    else if (pm) attn_shared_kernel<Many<DP>, Few<DP>><<<grid, kAThreads, 0, s>>>(a);
    else if (sm) attn_shared_kernel<Few<DP>, Many<DP>><<<grid, kAThreads, 0, s>>>(a);
    else attn_shared_kernel<Few<DP>, Few<DP>><<<grid, kAThreads, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_attn_prompt(PromptArgs a, hipStream_t s) {
    // wide tiles once they fill the compute units, else more and narrower ones
    const int64_t rows = static_cast<int64_t>(a.total_q) * (a.Hq / a.Hkv);
    const bool many = a.Hkv * ((rows + 127) / 128) >= kComputeUnits;
    const int tm = many ? 128 : few_rows(a.D);
    // every sequence ends in at most one partial tile
    a.tiles = static_cast<int>(rows / tm + (a.B < rows ? a.B : rows));
    if (a.tiles == 0) return hipSuccess;
    const int grid = a.tiles * a.Hkv;
    switch (pad_d(a.D)) {
        case 64: return prompt_dispatch<64>(a, many, grid, s);
        case 128: return prompt_dispatch<128>(a, many, grid, s);
        default: return prompt_dispatch<256>(a, many, grid, s);
    }
}

SharedPlan plan_attn_shared(int64_t B, int64_t L, int64_t Hq, int64_t Hkv, int64_t D, int64_t prefix_cap,
                            int64_t suffix_cap) {
    SharedPlan p{};
    const int64_t G = Hq / Hkv;
    p.merged = B == 1 || prefix_cap == 0;
    const int64_t rows_p = B * L * G, rows_s = L * G;
    p.prefix_many = rows_p > 64;
    p.suffix_many = rows_s > 64;
    const int64_t tm_p = p.prefix_many ? 128 : few_rows(static_cast<int>(D));
    const int64_t tm_s = p.suffix_many ? 128 : few_rows(static_cast<int>(D));
    const int64_t st_p = stage_keys(static_cast<int>(D), p.prefix_many), st_s = stage_keys(static_cast<int>(D), p.suffix_many);
    const int64_t keys_s = suffix_cap + (p.merged ? prefix_cap : 0);
    const int64_t stages_p = p.merged ? 0 : (prefix_cap + st_p - 1) / st_p;
    const int64_t stages_s = keys_s > 0 ? (keys_s + st_s - 1) / st_s : 0;
    const int64_t tiles_p = p.merged ? 0 : (rows_p + tm_p - 1) / tm_p;
    p.suffix_tiles = (rows_s + tm_s - 1) / tm_s;
    // stages per work item such that the items of both kinds fill the compute
    // units once
    const int64_t all = Hkv * (tiles_p * stages_p + B * p.suffix_tiles * stages_s);
    int64_t per = (all + kComputeUnits - 1) / kComputeUnits;
    if (per < 1) per = 1;
    p.prefix_splits = stages_p ? (stages_p + per - 1) / per : 0;
    p.suffix_splits = stages_s ? (stages_s + per - 1) / per : 0;
    p.prefix_items = Hkv * tiles_p * p.prefix_splits;
    p.suffix_items = Hkv * B * p.suffix_tiles * p.suffix_splits;
    p.parts = p.prefix_splits + p.suffix_splits;
    const int64_t rows = B * L * Hq;
    p.ml_bytes = p.parts > 1 ? (rows * p.parts * 8 + 255) / 256 * 256 : 0;
    p.ws_bytes = 256 + p.ml_bytes + (p.parts > 1 ? rows * p.parts * D * 4 : 0);
    return p;
}

hipError_t launch_attn_shared(SharedArgs a, const SharedPlan& p, void* ws, hipStream_t s) {
    a.merged = p.merged;
    a.prefix_items = static_cast<int>(p.prefix_items);
    a.prefix_splits = static_cast<int>(p.prefix_splits);
    a.suffix_splits = static_cast<int>(p.suffix_splits);
    a.suffix_tiles = static_cast<int>(p.suffix_tiles);
    a.parts = static_cast<int>(p.parts);
    uint8_t* w = static_cast<uint8_t*>(ws) + 256;
    a.part_ml = reinterpret_cast<float*>(w);
    a.part_o = reinterpret_cast<float*>(w + p.ml_bytes);
    const int grid = static_cast<int>(p.prefix_items + p.suffix_items);
    hipError_t e;
    switch (pad_d(a.D)) {
        case 64: e = shared_dispatch<64>(a, p.prefix_many, p.suffix_many, grid, s); break;
        case 128: e = shared_dispatch<128>(a, p.prefix_many, p.suffix_many, grid, s); break;
        default: e = shared_dispatch<256>(a, p.prefix_many, p.suffix_many, grid, s); break;
    }
    if (e != hipSuccess || a.parts == 1) return e;
    const int64_t rows = static_cast<int64_t>(a.B) * a.L * a.Hq;
    attn_join_kernel<<<static_cast<unsigned>((rows + 3) / 4), kAThreads, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace vla
