// The attention kernels' core: walks of 32 query rows over keys in packed tensors
// or in a paged cache of bf16 rows or of E4M3 codes, and the results' way out.
// The mathematics and the layout are told in attention.hip.
#pragma once

#include <hip/hip_runtime.h>

#include <algorithm>
#include <climits>
#include <cstdint>
#include <type_traits>

#include "bounded.h"
#include "vla_device.h"
#include "vla_internal.h"

namespace vla {
namespace {

typedef __attribute__((ext_vector_type(16))) float f32x16_t;
typedef __attribute__((ext_vector_type(4))) short s16x4_t;

constexpr int kAThreads = 256;
constexpr float kLag = 8.0f;                     // log2 of the largest weight, see weights()
// The maximum of a part whose keys a row sees and whose scores are all -inf: the
// join reads it, for the NaN among its values, and a part without keys it does not.
constexpr float kSeen = -3.402823466e38f;
constexpr uint32_t kNoOffset = 0xFFFFF000u;      // a buffer offset past every cache that takes 32-bit ones
constexpr int kBufferWord3 = 0x00020000;          // raw buffer, 32-bit data format

__device__ __attribute__((aligned(16))) const uint32_t kZeroChunk[4] = {0, 0, 0, 0};

// How a workgroup's four waves share its work: QG groups of 32 query rows x HV
// parts of the output channels x KG parts of the keys.
//   128 rows (QG 4) and 64 rows (QG 2, KG 2): all waves load and share stages
//     of 64 keys; a wave takes both 32-key sub-tiles of a stage, or one of them.
//   Up to 128 channels, 32 rows (KG 4): each wave walks every fourth 32-key
//     sub-tile through LDS of its own, so that no wave waits for another
//     before the end.
//   256 channels: 128 and 64 rows alike; 32 rows (HV 2, KG 2): shared stages
//     of 64 keys, one sub-tile per key part.  Queries and output of 32 rows
//     would need more than 256 registers; with half of the output channels a
//     wave fits, at the price of forming its scores twice (10 rows over 778
//     keys: 11.7 us; with private sub-tiles of all channels 13.9).
template <int DP_, int TM_>
struct ACfg {
    static constexpr int DP = DP_, TM = TM_;                 // padded channels, query rows per workgroup
    static constexpr int QG = TM / 32, HV = DP > 128 && TM < 64 ? 2 : 1, KG = 4 / (QG * HV);
    static_assert(QG * HV * KG == 4, "four waves");
    static constexpr bool SHARE = KG < 4;                    // stages shared by all waves
    static constexpr int SUBS = SHARE && QG == 4 ? 2 : 1;    // sub-tiles per wave and stage
    static constexpr int ST = 32 * KG * SUBS;                // keys per workgroup step
    static constexpr int CH = DP / 8;                        // 16-byte chunks per row
    static constexpr int RB = DP * 2;                        // bytes per row
    static constexpr int R = SHARE ? ST / 4 : 32;            // rows of K (and V) a wave loads at once
    static constexpr int RPI = 1024 / RB;                    // rows per load instruction
    static constexpr int NI = R / RPI;                       // load instructions for R rows
    static constexpr int NK = DP / 16;                       // MFMA steps of K Q^T
    static constexpr int ND = DP / 32 / HV;                  // 32-channel blocks of O^T per wave
    // LDS buffers: K and V of two shared stages, or of one sub-tile per wave,
    // each an object of its own: the compiler orders LDS reads after the
    // loads that write the same object
    static constexpr int BUF = ST * RB;
    static constexpr int WAVES = (SHARE ? 4 : 2) * BUF > 80 * 1024 ? 1 : 2;   // workgroups per compute unit
    static_assert(R % RPI == 0, "whole load instructions");
};

// The calling wave's parts.
template <class C>
struct Part {
    int wave, qg, kg, hv;
    __device__ __forceinline__ Part() {
        wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        qg = wave % C::QG;
        kg = wave / C::QG % C::KG;
        hv = wave / (C::QG * C::KG);
    }
};

// Position of a row's 16-byte chunks in LDS: chunk ^ swizzle.
template <int DP>
__device__ __forceinline__ int swz_k(int row) { return DP == 64 ? (row >> 1) & 7 : row & 15; }
template <int DP>
__device__ __forceinline__ int swz_v(int row) { return DP == 64 ? ((row >> 1) & 1) << 2 : (row & 3) << 2; }

// Keys 0 .. n-1 of one key/value head: rows of packed tensors, or rows of the
// cache named by the page tables (first the prefix's keys, then the suffix's).
struct PackedKeys {
    static constexpr bool CODES = false;
    const uint16_t *k, *v;     // row 0 of this head
    int k_stride, v_stride;    // bytes
    int n;
};
struct PageTable {
    const int32_t *prefix, *suffix;
    int n_prefix, n;           // prefix keys, all keys
    int page_log2;
    uint32_t num_pages;
    // A key's slot in two steps, so that the table is read well before its
    // entry is needed: the entry (of key 0 <= key < n), then the slot, -1
    // where the page does not exist.
    __device__ __forceinline__ int32_t entry(int key) const {
        const bool pre = key < n_prefix;
        return (pre ? prefix : suffix)[(pre ? key : key - n_prefix) >> page_log2];
    }
    __device__ __forceinline__ int slot(int key, int32_t page) const {
        const int j = key < n_prefix ? key : key - n_prefix;
        const int at = static_cast<int>((static_cast<uint32_t>(page) << page_log2) | (j & ((1 << page_log2) - 1)));
        return static_cast<uint32_t>(page) < num_pages ? at : -1;
    }
};
template <bool WIDE_>
struct PagedKeys : PageTable {
    static constexpr bool WIDE = WIDE_;   // byte offsets past 32 bits
    static constexpr bool CODES = false;
    const uint16_t *k, *v;     // slot 0 of this head
    uint32_t bytes;            // to the end of the last slot's D channels (not WIDE)
    uint32_t stride;           // bytes
    __device__ __forceinline__ void init(const SharedArgs& a, int hk) {
        stride = static_cast<uint32_t>(a.Hkv * a.D * 2);
        bytes = static_cast<uint32_t>(((static_cast<uint64_t>(a.num_pages) << a.page_log2) - 1) * stride + a.D * 2);
        k = a.k_cache + static_cast<int64_t>(hk) * a.D;
        v = a.v_cache + static_cast<int64_t>(hk) * a.D;
    }
};
// The cache in E4M3 codes, a scale per block of tokens and head.
template <bool WIDE_>
struct PagedCodes : PageTable {
    static constexpr bool WIDE = WIDE_;
    static constexpr bool CODES = true;
    const uint8_t *k, *v;      // slot 0 of this head
    const uint8_t *k_scales, *v_scales;   // block 0 of this head
    uint32_t bytes, stride;
    int Hkv, block_log2;
    __device__ __forceinline__ void init(const SharedArgs& a, int hk) {
        stride = static_cast<uint32_t>(a.Hkv * a.D);
        bytes = static_cast<uint32_t>(((static_cast<uint64_t>(a.num_pages) << a.page_log2) - 1) * stride + a.D);
        k = reinterpret_cast<const uint8_t*>(a.k_cache) + static_cast<int64_t>(hk) * a.D;
        v = reinterpret_cast<const uint8_t*>(a.v_cache) + static_cast<int64_t>(hk) * a.D;
        k_scales = a.k_scales + hk;
        v_scales = a.v_scales + hk;
        Hkv = a.Hkv;
        block_log2 = a.block_log2;
    }
    // A slot's two scale bytes (of slot 0 where there is none: a load that no
    // branch holds back)
    struct Bytes {
        uint32_t k, v;
    };
    __device__ __forceinline__ Bytes bytes_of(int slot) const {
        const int64_t at = static_cast<int64_t>(max(slot, 0) >> block_log2) * Hkv;
        return {k_scales[at], v_scales[at]};
    }
    // Both scales as bf16 bits, the keys' in the high half: a power of two with
    // eight exponent bits is a bf16 number.  0 where there is no slot, so that
    // the zeros loaded there stay zeros.
    static __device__ __forceinline__ uint32_t scales(Bytes b, int slot) {
        return slot >= 0 ? scale_bits(b.k) << 16 | scale_bits(b.v) : 0;
    }
    // 2^(byte - 127): 2^-127 is subnormal, 255 is NaN
    static __device__ __forceinline__ uint32_t scale_bits(uint32_t byte) { return (byte << 7) + (byte == 0 || byte == 255 ? 0x0040u : 0u); }
};

// A wave's partial result for its 32 rows: lane = row l % 32, O^T unnormalised,
// m the running maximum in log2 units, l the sum of weights (of this lane's
// keys until the walk's end).
template <class C>
struct State {
    f32x16_t acc[C::ND];
    float m, l;
    uint32_t late;     // sub-tiles left to add_late
};

__device__ __forceinline__ float half_max(float x) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float half_sum(float x) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// Whether 32 rows of V in LDS hold an infinity or NaN (in any chunk order:
// all of them are looked at).
template <class C>
__device__ __forceinline__ bool has_nonfinite(const uint8_t* v) {
    const int lane16 = (threadIdx.x & 63) * 16;
    uint32_t top = 0;
#pragma unroll 4
    for (int i = 0; i < 32 * C::RB / 1024; ++i) {
        const u32x4_t w = *reinterpret_cast<const u32x4_t*>(v + (lane16 + i * 1024));
        // an exponent of all ones plus one carries into the sign's place
#pragma unroll
        for (int j = 0; j < 4; ++j) top |= (w[j] & 0x7F807F80u) + 0x00800080u;
    }
    return __any((top & 0x80008000u) != 0);
}

// What one wave needs to walk keys for its 32 rows.
template <class C, class Keys>
struct Walk {
    static constexpr bool PAGED = !std::is_same<Keys, PackedKeys>::value;
    const Keys& keys;
    int klim;                  // the lane's row sees keys below this
    int kfull, kmax;           // every row sees keys below kfull, none one at or past kmax
    int D;
    float c;                   // scale * log2(e)
    int l32, g2;
    // the swizzle of V works within 128 channels; the next 128 are 256 bytes on
    static constexpr int NV = C::ND < 4 ? C::ND : 4;
    int kaddr, vaddr[NV];      // LDS operand addresses within 32 rows
    int ch0;                   // first of the wave's output channels
    int lrow, lpos;            // row and chunk position this lane loads, within one instruction
    bf16x8_t qf[C::NK];
    State<C>& st;

    // live: the lane has a row
    __device__ __forceinline__ Walk(const Keys& keys_, int klim_, int D_, float c_, State<C>& st_, bool live)
        : keys(keys_), klim(klim_), D(D_), c(c_), st(st_) {
        const int lane = threadIdx.x & 63;
        l32 = lane & 31;
        g2 = lane >> 5;
        // live rows come first, and no row sees fewer keys than the one before
        const int rows = __builtin_popcount(static_cast<uint32_t>(__ballot(live)));
        kfull = rows ? __builtin_amdgcn_readlane(klim, 0) : INT_MAX;
        kmax = rows ? __builtin_amdgcn_readlane(klim, rows - 1) : 0;
#pragma unroll
        for (int i = 0; i < C::ND; ++i) st.acc[i] = f32x16_t{};
        st.m = -__builtin_inff();
        st.l = 0.0f;
        st.late = 0;
        // A operand of K Q^T: row l32, chunk (2 kk + g2) ^ swizzle = kaddr ^ (kk << 5)
        kaddr = l32 * C::RB + ((swz_k<C::DP>(l32) ^ g2) << 4);
        // transpose read: key 4 g2 + i16/4 of an 8-key group, channels 16 g16 + 4 (i16 % 4)
        const int i16 = lane & 15, g16 = (lane >> 4) & 1;
        const int v0 = (4 * g2 + (i16 >> 2)) * C::RB + (2 * g16 + ((i16 & 3) >> 1)) * 16 + (i16 & 1) * 8;
#pragma unroll
        for (int d = 0; d < NV; ++d) vaddr[d] = v0 + ((d * 4) ^ swz_v<C::DP>(i16 >> 2)) * 16;
        lrow = lane / C::CH;
        lpos = lane % C::CH;
    }
    // Query rows r0 .. r0 + N * RPI - 1 into LDS like rows of K (q: the lane's
    // row, or nullptr; lane r holds row r): whole rows per instruction, where
    // operand reads from memory would touch 32 rows each.
    template <int N>
    __device__ __forceinline__ void stage_q(const uint16_t* q, uint8_t* dst, int r0) const {
        const uint64_t mine = reinterpret_cast<uint64_t>(q);
        const int lo = static_cast<int>(mine), hi = static_cast<int>(mine >> 32);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int row = r0 + i * C::RPI + lrow;
            const int ch = lpos ^ swz_k<C::DP>(row);
            const uint64_t p = static_cast<uint32_t>(__shfl(lo, row, 64)) | static_cast<uint64_t>(static_cast<uint32_t>(__shfl(hi, row, 64))) << 32;
            const uint64_t src = (p != 0 && ch * 8 < D) ? p + ch * 16 : reinterpret_cast<uint64_t>(kZeroChunk);
            __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)src,
                                             (__attribute__((address_space(3))) void*)(dst + (r0 + i * C::RPI) * C::RB), 16, 0, 0);
        }
        // the waits for these rows count the loads of keys that go out after
        // them, and the compiler may reorder loads into different LDS objects
        __atomic_signal_fence(__ATOMIC_SEQ_CST);
        __builtin_amdgcn_sched_barrier(0);
    }
    // Operand addresses from the buffers' starts, `first` bytes on.  They are
    // made opaque: the compiler follows an address to its LDS object over a few
    // steps only, and before a read of an object it does not know it waits for
    // every load into LDS, the next keys' among them.
    __device__ __forceinline__ void address(int first, int hv) {
        kaddr += first;
        ch0 = hv * C::ND * 32;
#pragma unroll
        for (int d = 0; d < NV; ++d) {
            vaddr[d] += first + ch0 * 2;
            asm volatile("" : "+v"(vaddr[d]));
        }
    }
    // query fragments: B operand, lane = row l32, channels 16 kk + 8 g2 .. +7
    __device__ __forceinline__ void read_q(const uint8_t* qt) {
#pragma unroll
        for (int kk = 0; kk < C::NK; ++kk) qf[kk] = as_bf16x8(*reinterpret_cast<const u32x4_t*>(qt + (kaddr ^ (kk << 5))));
    }

    // ---- loads of R rows of K or V into LDS, one instruction (i < C::NI) at a
    //      time.  row0: the rows' place in the buffer modulo 32 (for the
    //      swizzle); Source holds what is common to the instructions.
    struct Source {
        __amdgpu_buffer_rsrc_t rs;   // packed: ends with the last key, rows past it load zeros; paged: the cache
        int stride;
    };
    // Paged: the rows that this lane loads, taken from the lanes that read the
    // table (lane l: window key l; from: the window row of instruction 0).
    // Byte offsets in the cache, past its end where there is no row; WIDE: slots.
    struct Slots {
        uint32_t at[PAGED ? C::NI : 1];
    };
    __device__ __forceinline__ Slots slots_of(int slot, int from) const {
        Slots s;
        if constexpr (PAGED) {
            int mine = slot;
            if constexpr (!Keys::WIDE) mine = static_cast<int>(slot >= 0 ? static_cast<uint32_t>(slot) * keys.stride : kNoOffset);
#pragma unroll
            for (int i = 0; i < C::NI; ++i) s.at[i] = static_cast<uint32_t>(__shfl(mine, from + i * C::RPI + lrow, 64));
        }
        return s;
    }
    template <bool V>
    __device__ __forceinline__ Source source(int key0, int k1) const {
        Source s;
        if constexpr (!PAGED) {
            s.stride = V ? keys.v_stride : keys.k_stride;
            const int left = min(k1 - key0, C::R);
            s.rs = __builtin_amdgcn_make_buffer_rsrc(
                const_cast<uint8_t*>(reinterpret_cast<const uint8_t*>(V ? keys.v : keys.k) + static_cast<int64_t>(key0) * s.stride), 0,
                left > 0 ? (left - 1) * s.stride + D * 2 : 0, kBufferWord3);
        } else if constexpr (!Keys::WIDE) {
            s.rs = __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(static_cast<const void*>(V ? keys.v : keys.k)), 0, keys.bytes, kBufferWord3);
        }
        return s;
    }
    template <bool V>
    __device__ __forceinline__ void load(const Source& s, const Slots& sl, uint8_t* dst, int row0, int i) const {
        const int row = row0 + i * C::RPI + lrow;
        const int ch = lpos ^ (V ? swz_v<C::DP>(row) : swz_k<C::DP>(row));
        __attribute__((address_space(3))) void* const to = (__attribute__((address_space(3))) void*)(dst + i * 1024);
        if constexpr (!PAGED) {
            const uint32_t off = ch * 8 < D ? static_cast<uint32_t>(lrow * s.stride + ch * 16) : 0x80000000u;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(s.rs, to, 16, off, i * C::RPI * s.stride, 0, 0);
        } else if constexpr (!Keys::WIDE) {
            __builtin_amdgcn_raw_ptr_buffer_load_lds(s.rs, to, 16, ch * 8 < D ? sl.at[i] + ch * 16 : kNoOffset, 0, 0, 0);
        } else {
            const uint64_t at = reinterpret_cast<uint64_t>(V ? keys.v : keys.k) + static_cast<uint64_t>(sl.at[i]) * keys.stride + ch * 16;
            const uint64_t src = (static_cast<int>(sl.at[i]) >= 0 && ch * 8 < D) ? at : reinterpret_cast<uint64_t>(kZeroChunk);
            __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)src, to, 16, 0, 0);
        }
    }

    // ---- one 32-key sub-tile in LDS
    //      N loads, load_one(0 .. N-1), go out between the matrix instructions:
    //      issued in a block they would hold the wave until the load path has
    //      taken them all
    template <int N, class F>
    __device__ __forceinline__ f32x16_t scores(const uint8_t* kt, F&& load_one) const {
        u32x4_t kf[C::NK];
#pragma unroll
        for (int kk = 0; kk < C::NK; ++kk) kf[kk] = *reinterpret_cast<const u32x4_t*>(kt + (kaddr ^ (kk << 5)));
        if constexpr (Keys::CODES) __builtin_amdgcn_sched_barrier(0);   // all reads on their way before the first product
        f32x16_t sc = f32x16_t{};
#pragma unroll
        for (int kk = 0; kk < C::NK; ++kk) {
            sc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(as_bf16x8(kf[kk]), qf[kk], sc, 0, 0, 0);
            if (kk < N) load_one(kk);
        }
        // LDS reads stay a few steps ahead of the products
        constexpr int AHEAD = C::NK < 6 ? C::NK : 6;
        __builtin_amdgcn_sched_group_barrier(0x100, AHEAD, 0);                        // DS reads
#pragma unroll
        for (int kk = 0; kk < C::NK; ++kk) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);                        // MFMA
            if (kk < N) __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);            // VMEM loads
            if (kk + AHEAD < C::NK) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        }
        return sc;
    }
    // Scores in log2 units; those a row does not see become -inf.
    __device__ __forceinline__ void scale_and_mask(f32x16_t& sc, int key0, uint32_t vm) const {
#pragma unroll
        for (int i = 0; i < 16; ++i) sc[i] *= c;
        if (key0 + 32 > kfull) {
            const int lim = klim - key0 - 4 * g2;
#pragma unroll
            for (int i = 0; i < 16; ++i) sc[i] = 8 * (i / 4) + (i % 4) < lim ? sc[i] : -__builtin_inff();
        }
        if (vm != 0xFFFFFFFFu) {
            const uint32_t w = vm >> (4 * g2);
#pragma unroll
            for (int i = 0; i < 16; ++i) sc[i] = (w >> (8 * (i / 4) + (i % 4))) & 1u ? sc[i] : -__builtin_inff();
        }
    }
    // Weights, as bf16 pairs in accumulator order; moves the running maximum.
    // N loads go out among the exponentials.
    template <int N, class F>
    __device__ __forceinline__ void weights(const f32x16_t& sc, uint32_t* pw, F&& load_one) const {
        float mx = fmaxf(sc[0], sc[1]);
#pragma unroll
        for (int i = 2; i < 16; i += 2) mx = fmaxf(fmaxf(sc[i], sc[i + 1]), mx);
        mx = half_max(mx);
        // the running maximum follows once a row's scores pass it by kLag:
        // until then weights are at most 2^kLag and lose no precision
        if (__any(mx > st.m + kLag)) {
            const float mn = fmaxf(st.m, mx);
            const float al = mn == st.m ? 1.0f : __builtin_amdgcn_exp2f(st.m - mn);
            st.m = mn;
            st.l *= al;
#pragma unroll
            for (int d = 0; d < C::ND; ++d)
#pragma unroll
                for (int i = 0; i < 16; ++i) st.acc[d][i] *= al;
        }
        // a row that has seen no key yet: weights exp2(-inf) = 0
        const float m0 = st.m == -__builtin_inff() ? 0.0f : st.m;
        float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float p0 = __builtin_amdgcn_exp2f(sc[2 * i] - m0);
            const float p1 = __builtin_amdgcn_exp2f(sc[2 * i + 1] - m0);
            s0 += p0;
            s1 += p1;
            pw[i] = f32x2_to_bf16x2(p0, p1);
#pragma unroll
            for (int j = i * N / 8; j < (i + 1) * N / 8; ++j) load_one(j);
        }
        st.l += s0 + s1;
        if constexpr (N > 0) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                __builtin_amdgcn_sched_group_barrier(0x402, 48 / N, 0);                       // VALU, exponentials
                __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);                            // VMEM loads
            }
        }
    }
    // V^T fragments: 16 keys (step k2) x 32 channels (block d)
    __device__ __forceinline__ bf16x8_t v_frag(const uint8_t* vt, int k2, int d) const {
        const int at = vaddr[d & 3] + (d >> 2) * 256 + 16 * k2 * C::RB;
        const s16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4_t*)(vt + at));
        const s16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4_t*)(vt + (at + 8 * C::RB)));
        const u32x2_t a = __builtin_bit_cast(u32x2_t, lo), b = __builtin_bit_cast(u32x2_t, hi);
        const u32x4_t vf = {a.x, a.y, b.x, b.y};
        return as_bf16x8(vf);
    }
    __device__ __forceinline__ void add(const uint8_t* vt, const uint32_t* pw) const {
        bf16x8_t vf[2][C::ND];
#pragma unroll
        for (int k2 = 0; k2 < 2; ++k2)
#pragma unroll
            for (int d = 0; d < C::ND; ++d) vf[k2][d] = v_frag(vt, k2, d);
#pragma unroll
        for (int k2 = 0; k2 < 2; ++k2) {
            const u32x4_t pv = {pw[4 * k2], pw[4 * k2 + 1], pw[4 * k2 + 2], pw[4 * k2 + 3]};
#pragma unroll
            for (int d = 0; d < C::ND; ++d)
                st.acc[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vf[k2][d], as_bf16x8(pv), st.acc[d], 0, 0, 0);
        }
        constexpr int AHEAD = 2 * C::ND < 4 ? 2 * C::ND : 4;                          // fragments of two reads each
        __builtin_amdgcn_sched_group_barrier(0x100, 2 * AHEAD, 0);
#pragma unroll
        for (int i = 0; i < 2 * C::ND; ++i) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
            if (i + AHEAD < 2 * C::ND) __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
        }
    }
    // A zero weight times an infinity or NaN is not zero: a sub-tile that
    // some row sees only in part and whose V holds one is left out of the
    // product and added at the end, key by key.  So is one that no row sees
    // (the walk goes on for other waves' rows): there is nothing to add.  Bit b
    // of `late` is the sub-tile that ends 32 b to 32 b + 31 keys past the last
    // key that every row sees; 32 rows see at most 31 keys more than that, and
    // a sub-tile that one of them sees ends at most 31 past those.  k1: the end
    // of the walk's keys; past it V holds zeros.
    __device__ __forceinline__ bool put_off(const uint8_t* vt, int key0, int k1) const {
        if (key0 >= kmax) return true;
        if (key0 + 32 <= kfull || k1 <= kfull || !has_nonfinite<C>(vt)) return false;
        st.late |= 1u << ((key0 + 32 - kfull) >> 5);
        return true;
    }
    // weights() for one score (of a row whose scores are all -inf: 0)
    __device__ __forceinline__ float late_weight(float s) const {
        return bf16_to_f32(f32_to_bf16(__builtin_amdgcn_exp2f(s * c - (st.m == -__builtin_inff() ? 0.0f : st.m))));
    }
    // key0_of: first key of this wave's sub-tile that holds a key, or -1 (another wave's)
    template <class F>
    __device__ __forceinline__ void add_late(const uint16_t* q, int k1, F&& key0_of) const {
        if (!st.late) return;
        for (int key = max(kfull - 31, 0); key < min(kmax, k1); ++key) {
            const int key0 = key0_of(key);
            if (key0 < 0 || key0 + 32 <= kfull || !((st.late >> ((key0 + 32 - kfull) >> 5)) & 1u)) continue;
            if constexpr (Keys::CODES) {
                add_late_code(q, key);
            } else {
                const uint16_t *kr, *vr;
                if constexpr (PAGED) {
                    const int sl = keys.slot(key, keys.entry(key));
                    if (sl < 0) continue;
                    const int64_t at = static_cast<int64_t>(sl) * (keys.stride / 2);
                    kr = keys.k + at;
                    vr = keys.v + at;
                } else {
                    kr = keys.k + static_cast<int64_t>(key) * (keys.k_stride / 2);
                    vr = keys.v + static_cast<int64_t>(key) * (keys.v_stride / 2);
                }
                if (!q || key >= klim) continue;
                float s = 0.0f;
                for (int d = 0; d < D; ++d) s += bf16_to_f32(q[d]) * bf16_to_f32(kr[d]);
                const float p = late_weight(s);
#pragma unroll
                for (int d = 0; d < C::ND; ++d)
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const int ch = ch0 + 32 * d + 8 * x + 4 * g2;
                        uint2 v = make_uint2(0, 0);
                        if (ch < D) v = *reinterpret_cast<const uint2*>(vr + ch);
                        st.acc[d][4 * x] += p * __uint_as_float(v.x << 16);
                        st.acc[d][4 * x + 1] += p * __uint_as_float(v.x & 0xFFFF0000u);
                        st.acc[d][4 * x + 2] += p * __uint_as_float(v.y << 16);
                        st.acc[d][4 * x + 3] += p * __uint_as_float(v.y & 0xFFFF0000u);
                    }
            }
        }
    }
    __device__ __forceinline__ void add_late_code(const uint16_t* q, int key) const {
        const int sl = keys.slot(key, keys.entry(key));
        if (sl < 0 || !q || key >= klim) return;
        const uint8_t* const kr = keys.k + static_cast<int64_t>(sl) * keys.stride;
        const uint8_t* const vr = keys.v + static_cast<int64_t>(sl) * keys.stride;
        const uint32_t sw = Keys::scales(keys.bytes_of(sl), sl);
        const float ks = __uint_as_float(sw & 0xFFFF0000u), vs = __uint_as_float(sw << 16);
        float s = 0.0f;
        for (int d = 0; d < D; ++d) s += bf16_to_f32(q[d]) * (decode_e4m3<false>(kr[d]) * ks);
        const float p = late_weight(s);
#pragma unroll
        for (int d = 0; d < C::ND; ++d)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const int ch = ch0 + 32 * d + 8 * x + 4 * g2;
                uint32_t v = 0;
                if (ch < D) v = *reinterpret_cast<const uint32_t*>(vr + ch);
#pragma unroll
                for (int i = 0; i < 4; ++i) st.acc[d][4 * x + i] += p * (decode_e4m3<false>(v >> (8 * i) & 0xFFu) * vs);
            }
    }

    // ---- a cache in codes: rows pass through registers and enter LDS as the
    //      bf16 values they stand for, in the places that loads of bf16 rows
    //      would have written.
    struct Codes {
        u32x2_t x[C::NI];
    };
    struct Exponents {
        uint32_t x[C::NI];     // the rows' scales (PagedCodes::scales)
    };
    __device__ __forceinline__ Exponents exponents_of(uint32_t scales, int from) const {
        Exponents e;
#pragma unroll
        for (int i = 0; i < C::NI; ++i) e.x[i] = static_cast<uint32_t>(__shfl(static_cast<int>(scales), from + i * C::RPI + lrow, 64));
        return e;
    }
    template <bool V>
    __device__ __forceinline__ void fetch(const Source& s, const Slots& sl, int row0, Codes& x) const {
#pragma unroll
        for (int i = 0; i < C::NI; ++i) {
            const int row = row0 + i * C::RPI + lrow;
            const int ch = lpos ^ (V ? swz_v<C::DP>(row) : swz_k<C::DP>(row));
            if constexpr (!Keys::WIDE) {
                x.x[i] = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_raw_buffer_load_b64(s.rs, ch * 8 < D ? sl.at[i] + ch * 8 : kNoOffset, 0, 0));
            } else {
                const uint64_t at = reinterpret_cast<uint64_t>(V ? keys.v : keys.k) + static_cast<uint64_t>(sl.at[i]) * keys.stride + ch * 8;
                const uint64_t src = (static_cast<int>(sl.at[i]) >= 0 && ch * 8 < D) ? at : reinterpret_cast<uint64_t>(kZeroChunk);
                x.x[i] = *reinterpret_cast<const u32x2_t*>(src);
            }
        }
    }
    // dst: the rows' first place in LDS
    template <bool V>
    __device__ __forceinline__ void put(const Codes& x, const Exponents& e, uint8_t* dst) const {
        const int lane16 = (threadIdx.x & 63) * 16;
#pragma unroll
        for (int i = 0; i < C::NI; ++i) {
            const float by = __uint_as_float(V ? e.x[i] << 16 : e.x[i] & 0xFFFF0000u);
            *reinterpret_cast<u32x4_t*>(dst + i * 1024 + lane16) = ocp8_to_bf16x8_scaled(x.x[i], by);
        }
    }
};

// s_waitcnt immediates: at most n vector-memory operations outstanding, LDS
// unconstrained; and all vector-memory and LDS operations done.
constexpr int wait_vm(int n) { return (n & 15) | ((n >> 4) << 14) | 0x0F70; }
constexpr int kWaitAll = 0x0070;
constexpr int kWaitLds = 0xC07F;

// A point that no memory operation or instruction moves across.
template <int IMM>
__device__ __forceinline__ void wait_here() {
    __builtin_amdgcn_sched_barrier(0);
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    __builtin_amdgcn_s_waitcnt(IMM);
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    __builtin_amdgcn_sched_barrier(0);
}

// Keys k0 .. k1-1 (a uniform range) for the wave's 32 rows, the workgroup's
// four waves sharing each stage of C::ST keys.
template <class C, class Keys>
__device__ __forceinline__ void attend_stages(const Keys& keys, const uint16_t* q, int klim, int k0, int k1, int D, float c,
                                              uint8_t* kb0, uint8_t* vb0, uint8_t* kb1, uint8_t* vb1, State<C>& st) {
    using W = Walk<C, Keys>;
    using Source = typename W::Source;
    using Slots = typename W::Slots;
    const Part<C> part;
    const int n_stages = (k1 - k0 + C::ST - 1) / C::ST;
    const int row0 = part.wave * C::R;                            // rows of a stage this wave loads
    // the lane's key of a stage: its table entry (of the last key past the
    // range), then its slot, for the loads and the masks
    const int mine = k0 + static_cast<int>(threadIdx.x & (C::ST - 1));
    auto entry = [&](int s) __attribute__((always_inline)) -> int32_t {
        if constexpr (W::PAGED) return keys.entry(min(mine + s * C::ST, k1 - 1));
        else return 0;
    };
    auto slot_of = [&](int s, int32_t page) __attribute__((always_inline)) -> int {
        const int key = mine + s * C::ST;
        if constexpr (W::PAGED) return key < k1 ? keys.slot(key, page) : -1;
        else return 0;
    };
    int32_t page = n_stages > 0 ? entry(0) : 0;
    W w(keys, klim, D, c, st, q != nullptr);
    auto valid = [&](int sl) __attribute__((always_inline)) -> uint64_t {
        if constexpr (W::PAGED) return __ballot(sl >= 0);
        else return ~uint64_t(0);
    };
    if (n_stages <= 0) return;
    // stage s lives in buffers s % 2; its loads are issued while stage s-1 is
    // computed, its table entries are read one stage earlier still.  The
    // query rows come through the buffers of stage 1, each row group's from
    // the waves that share it.
    constexpr int PER = C::BUF / (32 * C::RB), WPG = 4 / C::QG;   // row groups per buffer, waves per row group
    uint8_t* const qt = (part.qg < PER ? kb1 : vb1) + (part.qg % PER) * 32 * C::RB;
    w.template stage_q<32 / WPG / C::RPI>(q, qt, part.wave / C::QG * (32 / WPG));
    int slot = slot_of(0, page);
    uint64_t vcur = valid(slot);
    {
        const Source k = w.template source<false>(k0 + row0, k1), v = w.template source<true>(k0 + row0, k1);
        const Slots sl = w.slots_of(slot, row0);
#pragma unroll
        for (int i = 0; i < C::NI; ++i) w.template load<false>(k, sl, kb0 + row0 * C::RB, row0, i);
#pragma unroll
        for (int i = 0; i < C::NI; ++i) w.template load<true>(v, sl, vb0 + row0 * C::RB, row0, i);
    }
    wait_here<wait_vm(2 * C::NI)>();
    if constexpr (WPG > 1) {
        __builtin_amdgcn_s_barrier();
        __atomic_signal_fence(__ATOMIC_SEQ_CST);
    }
    w.read_q(qt);
    w.address(0, part.hv);
    page = entry(1);
    auto sub_tile = [&](const uint8_t* kt, const uint8_t* vt, int key0, uint32_t vm, auto&& load_one, auto&& load_more) __attribute__((always_inline)) {
        f32x16_t sc = w.template scores<C::NI>(kt, load_one);
        w.scale_and_mask(sc, key0, vm);
        uint32_t pw[8];
        w.template weights<C::SUBS == 2 ? 0 : C::NI>(sc, pw, load_more);
        if (!w.put_off(vt, key0, k1)) w.add(vt, pw);
    };
    auto step = [&](uint8_t* kc, uint8_t* vc, uint8_t* kn, uint8_t* vn, int s, auto more) __attribute__((always_inline)) {
        // this wave's loads of stage s have landed and its reads of stage s-1
        // are done; the barrier says so for every wave
        wait_here<kWaitAll>();
        __builtin_amdgcn_s_barrier();
        __atomic_signal_fence(__ATOMIC_SEQ_CST);
        __builtin_amdgcn_sched_barrier(0);
        const int key0 = k0 + s * C::ST;
        // the next stage's loads go out among this one's scores and, with one
        // sub-tile per stage, its weights
        Source k, v;
        Slots sl;
        uint64_t vnext = 0;
        if constexpr (more()) {
            k = w.template source<false>(key0 + C::ST + row0, k1);
            v = w.template source<true>(key0 + C::ST + row0, k1);
            slot = slot_of(s + 1, page);
            sl = w.slots_of(slot, row0);
            if constexpr (W::PAGED) __builtin_amdgcn_sched_barrier(0);   // the exchanges together, not one wait among the products each
            vnext = valid(slot);
            page = entry(s + 2);
        }
        auto load_k = [&](int i) __attribute__((always_inline)) { if constexpr (more()) w.template load<false>(k, sl, kn + row0 * C::RB, row0, i); };
        auto load_v = [&](int i) __attribute__((always_inline)) { if constexpr (more()) w.template load<true>(v, sl, vn + row0 * C::RB, row0, i); };
        if constexpr (C::SUBS == 2) {
            sub_tile(kc, vc, key0, static_cast<uint32_t>(vcur), load_k, [](int) {});
            sub_tile(kc + 32 * C::RB, vc + 32 * C::RB, key0 + 32, static_cast<uint32_t>(vcur >> 32), load_v, [](int) {});
        } else {
            const int at = part.kg * 32;
            sub_tile(kc + at * C::RB, vc + at * C::RB, key0 + at, static_cast<uint32_t>(vcur >> at), load_k, load_v);
        }
        vcur = vnext;
    };
    for (int s = 0; s + 1 < n_stages; s += 2) {
        step(kb0, vb0, kb1, vb1, s, std::true_type{});
        if (s + 2 < n_stages) step(kb1, vb1, kb0, vb0, s + 1, std::true_type{});
    }
    step(n_stages % 2 ? kb0 : kb1, n_stages % 2 ? vb0 : vb1, nullptr, nullptr, n_stages - 1, std::false_type{});
    st.l = half_sum(st.l);
    w.add_late(q, k1, [&](int key) {
        const int t = key - k0;
        return (t >> 5 & (C::KG - 1)) == part.kg ? k0 + (t & ~31) : -1;
    });
}

// Keys k0 .. k1-1 for 32 rows that the four waves share: wave w takes
// sub-tiles w, w + 4, ...  Each wave's K and V have one place in LDS: K of
// the next sub-tile goes out before this one's weights are formed, its V among
// its scores, so up to 16 (D <= 64: 8) KiB per wave are in flight.
template <class C, class Keys>
__device__ __forceinline__ void attend_streams(const Keys& keys, const uint16_t* q, int klim, int k0, int k1, int D, float c,
                                           uint8_t* kb_all, uint8_t* vb_all, State<C>& st) {
    using W = Walk<C, Keys>;
    using Source = typename W::Source;
    using Slots = typename W::Slots;
    constexpr bool PAGED = W::PAGED;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    uint8_t* const kb = kb_all + wave * 32 * C::RB;
    uint8_t* const vb = vb_all + wave * 32 * C::RB;
    const int first = k0 + wave * 32;
    const int n = k1 > first ? (k1 - first + 127) / 128 : 0;
    auto entry = [&](int t) __attribute__((always_inline)) -> int32_t {
        if constexpr (PAGED) return keys.entry(min(first + t * 128 + static_cast<int>(threadIdx.x & 31), k1 - 1));
        else return 0;
    };
    auto slot_of = [&](int t, int32_t page) __attribute__((always_inline)) -> int {
        const int key = first + t * 128 + (threadIdx.x & 31);
        if constexpr (PAGED) return key < k1 ? keys.slot(key, page) : -1;
        else return 0;
    };
    int32_t page = n > 0 ? entry(0) : 0;
    W w(keys, klim, D, c, st, q != nullptr);
    // the query rows come through the place of wave 0's V, eight from each wave
    w.template stage_q<8 / C::RPI>(q, vb_all, wave * 8);
    Slots sl = {};
    int slot = -1;
    if (n > 0) {
        const Source k = w.template source<false>(first, k1);
        slot = slot_of(0, page);
        sl = w.slots_of(slot, 0);
#pragma unroll
        for (int i = 0; i < C::NI; ++i) w.template load<false>(k, sl, kb, 0, i);
        wait_here<wait_vm(C::NI)>();
    } else {
        wait_here<wait_vm(0)>();
    }
    __builtin_amdgcn_s_barrier();
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    w.read_q(vb_all);
    w.address(wave * 32 * C::RB, 0);
    wait_here<kWaitLds>();
    __builtin_amdgcn_s_barrier();
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    if (n <= 0) return;
    page = entry(1);
    for (int t = 0; t < n; ++t) {
        const int key0 = first + t * 128;
        const bool more = t + 1 < n;
        wait_here<wait_vm(0)>();                                  // K(t), and the entry of t + 1
        const Source v = w.template source<true>(key0, k1);
        f32x16_t sc = w.template scores<C::NI>(kb_all, [&](int i) __attribute__((always_inline)) { w.template load<true>(v, sl, vb, 0, i); });
        const uint32_t vm = PAGED ? static_cast<uint32_t>(__ballot(slot >= 0)) : 0xFFFFFFFFu;
        wait_here<kWaitLds>();                                    // K(t) has been read
        if (more) {
            slot = slot_of(t + 1, page);
            const Source k = w.template source<false>(key0 + 128, k1);
            sl = w.slots_of(slot, 0);
#pragma unroll
            for (int i = 0; i < C::NI; ++i) w.template load<false>(k, sl, kb, 0, i);
            page = entry(t + 2);
        }
        w.scale_and_mask(sc, key0, vm);
        uint32_t pw[8];
        w.template weights<0>(sc, pw, [](int) {});
        if (more) wait_here<wait_vm(C::NI)>();                    // V(t); K(t+1) may be on its way
        else wait_here<wait_vm(0)>();
        if (!w.put_off(vb, key0, k1)) w.add(vb_all, pw);
        wait_here<kWaitLds>();                                    // V(t) has been read
    }
    st.l = half_sum(st.l);
    w.add_late(q, k1, [&](int key) {
        const int t = key - k0;
        return (t >> 5 & 3) == wave ? k0 + (t & ~31) : -1;
    });
}

// The walk of shared stages over a cache in codes.  A stage's codes are fetched
// two steps ahead, two registers to eight values, and enter LDS a step ahead:
// the conversions go out among the products of the stage before, each half of a
// step taking the keys' or the values'.
template <class C, class Keys>
__device__ __forceinline__ void attend_code_stages(const Keys& keys, const uint16_t* q, int klim, int k0, int k1, int D, float c,
                                                   uint8_t* kb0, uint8_t* vb0, uint8_t* kb1, uint8_t* vb1, State<C>& st) {
    using W = Walk<C, Keys>;
    const Part<C> part;
    const int n_stages = (k1 - k0 + C::ST - 1) / C::ST;
    const int row0 = part.wave * C::R;                            // rows of a stage this wave brings
    const int mine = k0 + static_cast<int>(threadIdx.x & (C::ST - 1));
    auto entry = [&](int s) __attribute__((always_inline)) { return keys.entry(min(mine + s * C::ST, k1 - 1)); };
    auto slot_of = [&](int s, int32_t page) __attribute__((always_inline)) {
        const int key = mine + s * C::ST;
        return key < k1 ? keys.slot(key, page) : -1;
    };
    int32_t page = n_stages > 0 ? entry(0) : 0;
    W w(keys, klim, D, c, st, q != nullptr);
    if (n_stages <= 0) return;
    constexpr int PER = C::BUF / (32 * C::RB), WPG = 4 / C::QG;   // row groups per buffer, waves per row group
    uint8_t* const qt = (part.qg < PER ? kb1 : vb1) + (part.qg % PER) * 32 * C::RB;
    w.template stage_q<32 / WPG / C::RPI>(q, qt, part.wave / C::QG * (32 / WPG));
    typename W::Codes ck, cv;
    typename W::Slots sl;
    int slot;
    typename Keys::Bytes bytes;
    const typename W::Source ks = w.template source<false>(0, 0), vs = w.template source<true>(0, 0);
    auto locate = [&](int s) __attribute__((always_inline)) {
        slot = slot_of(s, page);
        bytes = keys.bytes_of(slot);
        sl = w.slots_of(slot, row0);
        page = entry(s + 1);
    };
    locate(0);
    w.template fetch<false>(ks, sl, row0, ck);
    w.template fetch<true>(vs, sl, row0, cv);
    wait_here<wait_vm(0)>();
    if constexpr (WPG > 1) {
        __builtin_amdgcn_s_barrier();
        __atomic_signal_fence(__ATOMIC_SEQ_CST);
    }
    w.read_q(qt);
    w.address(0, part.hv);
    uint64_t vcur = __ballot(slot >= 0);
    {
        const typename W::Exponents e = w.exponents_of(Keys::scales(bytes, slot), row0);
        w.template put<false>(ck, e, kb0 + row0 * C::RB);
        w.template put<true>(cv, e, vb0 + row0 * C::RB);
    }
    if (n_stages > 1) {
        locate(1);
        w.template fetch<false>(ks, sl, row0, ck);
        w.template fetch<true>(vs, sl, row0, cv);
    }
    auto sub_tile = [&](const uint8_t* kt, const uint8_t* vt, int key0, uint32_t vm, auto&& first, auto&& then) __attribute__((always_inline)) {
        f32x16_t sc = w.template scores<0>(kt, [](int) {});
        first();
        w.scale_and_mask(sc, key0, vm);
        uint32_t pw[8];
        w.template weights<0>(sc, pw, [](int) {});
        then();
        if (!w.put_off(vt, key0, k1)) w.add(vt, pw);
    };
    auto step = [&](uint8_t* kc, uint8_t* vc, uint8_t* kn, uint8_t* vn, int s, auto more) __attribute__((always_inline)) {
        // stage s is in its buffers and every wave is done with those of stage s - 1
        wait_here<kWaitLds>();
        __builtin_amdgcn_s_barrier();
        __atomic_signal_fence(__ATOMIC_SEQ_CST);
        const int key0 = k0 + s * C::ST;
        typename W::Exponents e;
        uint64_t vnext = 0;
        if constexpr (more()) {
            e = w.exponents_of(Keys::scales(bytes, slot), row0);
            vnext = __ballot(slot >= 0);
        }
        auto move_k = [&]() __attribute__((always_inline)) {
            if constexpr (more()) {
                w.template put<false>(ck, e, kn + row0 * C::RB);
                locate(s + 2);                                    // past the end: zeros
                w.template fetch<false>(ks, sl, row0, ck);
            }
        };
        auto move_v = [&]() __attribute__((always_inline)) {
            if constexpr (more()) {
                w.template put<true>(cv, e, vn + row0 * C::RB);
                w.template fetch<true>(vs, sl, row0, cv);
            }
        };
        if constexpr (C::SUBS == 2) {
            sub_tile(kc, vc, key0, static_cast<uint32_t>(vcur), move_k, [] {});
            sub_tile(kc + 32 * C::RB, vc + 32 * C::RB, key0 + 32, static_cast<uint32_t>(vcur >> 32), move_v, [] {});
        } else {
            const int at = part.kg * 32;
            sub_tile(kc + at * C::RB, vc + at * C::RB, key0 + at, static_cast<uint32_t>(vcur >> at), move_k, move_v);
        }
        vcur = vnext;
    };
    for (int s = 0; s + 1 < n_stages; s += 2) {
        step(kb0, vb0, kb1, vb1, s, std::true_type{});
        if (s + 2 < n_stages) step(kb1, vb1, kb0, vb0, s + 1, std::true_type{});
    }
    step(n_stages % 2 ? kb0 : kb1, n_stages % 2 ? vb0 : vb1, nullptr, nullptr, n_stages - 1, std::false_type{});
    st.l = half_sum(st.l);
    w.add_late(q, k1, [&](int key) {
        const int t = key - k0;
        return (t >> 5 & (C::KG - 1)) == part.kg ? k0 + (t & ~31) : -1;
    });
}

// ------------------------------------------------------------- results

// LDS of one workgroup.
#define ATTN_LDS                                                                                       \
    __shared__ __attribute__((aligned(16))) uint8_t b0[C::BUF], b1[C::BUF];                            \
    __shared__ __attribute__((aligned(16))) uint8_t b2[C::SHARE ? C::BUF : 16], b3[C::SHARE ? C::BUF : 16]; \
    __shared__ float ml[4][2][32];                                                                     \
    __shared__ uint64_t row_at[4][32]

// First of this wave's 32 rows in the workgroup's tile.
template <class C>
__device__ __forceinline__ int wave_row() {
    return Part<C>().qg * 32;
}

// Writes the workgroup's rows: through LDS, so that a row goes out as one run
// of 16-byte words.  The KG key parts' results for the same rows are scaled to
// their common maximum first and only added on the way.  PART false: O / l
// rounded to bf16 (0 for a row without keys) at address `to` of the lane's
// row; PART true: row number to - 1 of part_ml (maximum, sum) and part_o (O,
// fp32).  to 0: the lane has no row.
template <class C, bool PART>
__device__ __forceinline__ void write_rows(const State<C>& st, uint64_t to, float* part_ml, float* part_o, int D,
                                           uint8_t* b0, uint8_t* b1, uint8_t* b2, uint8_t* b3, float (*ml)[2][32],
                                           uint64_t (*row_at)[32]) {
    const int lane = threadIdx.x & 63, l32 = lane & 31, g2 = lane >> 5;
    const Part<C> part;
    constexpr int ROW = C::DP * 4;                                // bytes; 16-byte chunk c of row r at c ^ r
    // row r of (row group, key part) a; a buffer holds PER such sets of 32 rows
    constexpr int PER = C::BUF / (32 * ROW);
    static_assert(PER > 0, "whole sets");
    auto place = [&](int a, int r) __attribute__((always_inline)) -> uint8_t* {
        const int at = a / PER;
        return (at == 0 ? b0 : (at == 1 ? b1 : (at == 2 ? b2 : b3))) + (a % PER * 32 + r) * ROW;
    };
    const int set = part.qg + part.kg * C::QG;
    if (g2 == 0 && part.hv == 0) {
        if constexpr (C::KG > 1) {
            ml[set][0][l32] = st.m;
            ml[set][1][l32] = st.l;
        }
        if (part.kg == 0) row_at[part.qg][l32] = to;
    }
    wait_here<kWaitAll>();
    __syncthreads();                                              // every wave is past its last keys
    float m = st.m, l = st.l, f = 1.0f;
    if constexpr (C::KG > 1) {
        float mk[C::KG];
#pragma unroll
        for (int k = 0; k < C::KG; ++k) {
            mk[k] = ml[part.qg + k * C::QG][0][l32];
            m = fmaxf(m, mk[k]);
        }
        l = 0.0f;
#pragma unroll
        for (int k = 0; k < C::KG; ++k) l += ml[part.qg + k * C::QG][1][l32] * (mk[k] == m ? 1.0f : __builtin_amdgcn_exp2f(mk[k] - m));
        f = st.m == m ? 1.0f : __builtin_amdgcn_exp2f(st.m - m);
    }
    if constexpr (PART) {
        if (g2 == 0 && part.hv == 0 && part.kg == 0 && to != 0)
            *reinterpret_cast<float2*>(part_ml + 2 * static_cast<int64_t>(to - 1)) = make_float2(m, l);
    } else {
        f *= l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);        // NaN stays NaN
    }
    uint8_t* const mine = place(set, l32);
#pragma unroll
    for (int d = 0; d < C::ND; ++d)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const f32x4_t v = {st.acc[d][4 * x], st.acc[d][4 * x + 1], st.acc[d][4 * x + 2], st.acc[d][4 * x + 3]};
            *reinterpret_cast<f32x4_t*>(mine + (((8 * (d + part.hv * C::ND) + 2 * x + g2) ^ l32) & (C::DP / 4 - 1)) * 16) = v * f;
        }
    __syncthreads();
    // the waves of a row group write its 32 rows, 8 channels per lane.  Many
    // passes stay a loop: code that runs once per workgroup is bound by its
    // length.
    constexpr int GROUPS = C::DP / 8, RPW = 64 / GROUPS;          // rows per wave and pass
    constexpr int WPG = 4 / C::QG, PASSES = 32 / (WPG * RPW), UNROLL = WPG == 4 ? PASSES : 2;
    const int cg = lane % GROUPS;
#pragma unroll UNROLL
    for (int pass = 0; pass < PASSES; ++pass) {
        const int row = (pass * WPG + part.wave / C::QG) * RPW + lane / GROUPS;
        const uint64_t dst = row_at[part.qg][row];
        f32x4_t o[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int at = (((2 * cg + x) ^ row) & (C::DP / 4 - 1)) * 16;
            o[x] = *reinterpret_cast<const f32x4_t*>(place(part.qg, row) + at);
#pragma unroll
            for (int k = 1; k < C::KG; ++k) o[x] += *reinterpret_cast<const f32x4_t*>(place(part.qg + k * C::QG, row) + at);
        }
        if (dst == 0 || cg * 8 >= D) continue;
        if constexpr (PART) {
            f32x4_t* const p = reinterpret_cast<f32x4_t*>(part_o + static_cast<int64_t>(dst - 1) * D + cg * 8);
            p[0] = o[0];
            p[1] = o[1];
        } else {
            const u32x4_t w = {f32x2_to_bf16x2(o[0].x, o[0].y), f32x2_to_bf16x2(o[0].z, o[0].w),
                               f32x2_to_bf16x2(o[1].x, o[1].y), f32x2_to_bf16x2(o[1].z, o[1].w)};
            *reinterpret_cast<u32x4_t*>(reinterpret_cast<uint16_t*>(dst) + cg * 8) = w;
        }
    }
}

template <class C, class Keys>
__device__ __forceinline__ void attend(const Keys& keys, const uint16_t* q, int klim, int k0, int k1, int D, float c,
                                       uint8_t* b0, uint8_t* b1, uint8_t* b2, uint8_t* b3, State<C>& st) {
    if constexpr (Keys::CODES) attend_code_stages<C>(keys, q, klim, k0, k1, D, c, b0, b1, b2, b3, st);   // tall tiles alone
    else if constexpr (C::SHARE) attend_stages<C>(keys, q, klim, k0, k1, D, c, b0, b1, b2, b3, st);
    else attend_streams<C>(keys, q, klim, k0, k1, D, c, b0, b1, st);
}

// ----------------------------------------------------------- shared prefix

// One workgroup, one work item: a row tile of one key/value head against one
// split of the shared prefix (rows of the whole batch) or of one sequence's
// suffix.  With one sequence both are one range of keys.  More than one part
// per row: the parts' unnormalised O, maximum and sum go to the workspace.
template <class C, class Keys>
__global__ __launch_bounds__(kAThreads) __attribute__((amdgpu_waves_per_eu(C::WAVES, C::WAVES)))
void attn_shared_kernel(SharedArgs a) {
    ATTN_LDS;
    int id = blockIdx.x;
    const bool prefix = id < a.prefix_items;
    if (!prefix) id -= a.prefix_items;
    // (head, split) fastest: the row tiles that read the same keys are Hkv *
    // splits apart, on one XCD when that is a multiple of 8
    const int splits = prefix ? a.prefix_splits : a.suffix_splits;
    int pair, split, tile, b = 0;
    const int rest = (prefix ? a.by_prefix_pairs : a.by_suffix_pairs).divide(id, pair);
    const int hk = (prefix ? a.by_prefix_splits : a.by_suffix_splits).divide(pair, split);
    if (prefix) tile = rest;
    else b = a.by_suffix_tiles.divide(rest, tile);

    const int lane = threadIdx.x & 63;
    const int G = a.Hq / a.Hkv;
    const int np = a.prefix_pages ? min(max(a.prefix_len[0], 0), a.prefix_cap) : 0;
    int ns = 0;
    if (!prefix && a.block_table) ns = min(max(a.seq_lens[b], 0), a.suffix_cap);
    Keys keys;
    keys.init(a, hk);
    keys.prefix = a.prefix_pages;
    keys.suffix = a.block_table ? a.block_table + static_cast<int64_t>(b) * a.pages_per_seq : nullptr;
    keys.n_prefix = (prefix || a.merged) ? np : 0;
    keys.n = keys.n_prefix + ns;
    keys.page_log2 = a.page_log2;
    keys.num_pages = a.num_pages;

    const int rows = (prefix ? a.B : 1) * a.L * G;
    const int r = tile * C::TM + wave_row<C>() + (lane & 31);
    const bool live = r < rows;
    int g;
    const int tok = a.by_group.divide(r, g);
    const int64_t token = static_cast<int64_t>(b) * a.L + tok;    // of B * L
    const int head = hk * G + g;
    const uint16_t* q = live ? a.q + token * a.q_stride + static_cast<int64_t>(head) * a.D : nullptr;
    int klim = keys.n;
    if (a.causal && !prefix) klim = keys.n_prefix + min(max(tok + 1 + ns - a.L, 0), ns);
    int unused;
    const int steps = (keys.n + C::ST - 1) / C::ST;
    const int per = (prefix ? a.by_prefix_splits : a.by_suffix_splits).divide(steps + splits - 1, unused);
    const int k0 = min(split * per * C::ST, keys.n), k1 = min((split + 1) * per * C::ST, keys.n);
    State<C> st;
    attend<C>(keys, q, klim, k0, k1, a.D, a.c, b0, b1, b2, b3, st);
    if (klim > k0) st.m = fmaxf(st.m, kSeen);
    if (a.parts == 1) {
        uint16_t* const out = a.out + token * a.out_stride + static_cast<int64_t>(head) * a.D;
        write_rows<C, false>(st, live ? reinterpret_cast<uint64_t>(out) : 0, nullptr, nullptr, a.D, b0, b1, b2, b3, ml, row_at);
    } else {
        const int64_t at = (token * a.Hq + head) * a.parts + (prefix ? 0 : a.prefix_splits) + split;
        write_rows<C, true>(st, live ? static_cast<uint64_t>(at) + 1 : 0, a.part_ml, a.part_o, a.D, b0, b1, b2, b3, ml, row_at);
    }
}

// D channels run in the kernels of the next padded size.
template <int TM, class F>
hipError_t by_size(int D, F&& launch) {
    if (D <= 64) return launch(ACfg<64, TM>{});
    return D <= 128 ? launch(ACfg<128, TM>{}) : launch(ACfg<256, TM>{});
}

// The walks of a planned call (the parts' join apart).  wide: the cache takes
// byte offsets past 32 bits.
template <template <bool> class Keys>
hipError_t launch_walks(SharedArgs& a, const SharedPlan& p, bool wide, hipStream_t s) {
    auto run = [&](int tm, int64_t prefix_items, int64_t suffix_items) {
        a.prefix_items = static_cast<int>(prefix_items);
        const int grid = static_cast<int>(prefix_items + suffix_items);
        if (grid == 0) return hipSuccess;
        auto kernel = [&](auto cfg) {
            // caches below 4 GiB take one 32-bit offset per row and load, where
            // 64-bit addresses with a select for missing rows take five
            // instructions more each (32 sequences of 50 tokens over 850 keys:
            // 31 us against 35)
            if (wide) attn_shared_kernel<decltype(cfg), Keys<true>><<<grid, kAThreads, 0, s>>>(a);
            else attn_shared_kernel<decltype(cfg), Keys<false>><<<grid, kAThreads, 0, s>>>(a);
            return hipGetLastError();
        };
        return tm == 128 ? by_size<128>(a.D, kernel) : (tm == 64 ? by_size<64>(a.D, kernel) : by_size<32>(a.D, kernel));
    };
    hipError_t e;
    if (p.prefix_tm == p.suffix_tm) {
        e = run(p.prefix_tm, p.prefix_items, p.suffix_items);
    } else {
        e = run(p.prefix_tm, p.prefix_items, 0);
        if (e == hipSuccess) e = run(p.suffix_tm, 0, p.suffix_items);
    }
    return e;
}

}  // namespace
}  // namespace vla
