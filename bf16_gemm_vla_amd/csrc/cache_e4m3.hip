// Rows appended to a paged key/value cache held in OCP E4M3, a scale for each
// block of tokens and head.
//
//   scale of (block, head) = 2^e, the least with max |x| <= 448 2^e over the
//   rows that the block holds; code = e4m3(x / 2^e)
//
// Powers of two, held as E8M0 bytes, lose nothing against other scales (the
// codes are floating-point: their relative step is the same wherever in its
// binade the maximum lies) and make both steps exact: the division, and the
// change of scale when a later row has a larger maximum than the block had
// (codes only move to another exponent, but for those that fall below the
// smallest normal and round once more).  So a block's codes are those of its
// rows under its final scale whatever calls brought them, up to that.
//
// One work item is one block of one sequence, one head, keys or values: a wave
// or, where the block is large, a workgroup owns all of it, so a scale that
// grows and the earlier rows that move with it need no atomics.  Rows stay in
// registers between their maximum and their codes.
//
// Bound by HBM on prompts and by latency on single tokens.  Measured, captured
// calls one behind another, 8 heads of 128: 16 prompts of 9001 rows together in
// blocks of 32 14.6 us (3.8 TB/s; a copy's rate would take 10.8, an empty launch
// takes 2.8), 64 single tokens in blocks of 16 4.9 us.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "bounded.h"
#include "vla_device.h"
#include "vla_internal.h"

namespace vla {
namespace {

constexpr int kCThreads = 256;
constexpr int kKeep = 8;            // wave steps of rows kept in registers

// Four codes times 2^k, k <= 0, encoded again; NaN codes stay as they are.
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float by) {
    typedef __attribute__((ext_vector_type(2))) float f32x2_t;
    const f32x2_t lo = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(w), false);
    const f32x2_t hi = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(w), true);
    int c = __builtin_amdgcn_cvt_pk_fp8_f32(lo.x * by, lo.y * by, 0, false);
    c = __builtin_amdgcn_cvt_pk_fp8_f32(hi.x * by, hi.y * by, c, true);
    // bytes whose low seven bits are all ones
    const uint32_t nan = (((w & 0x7F7F7F7Fu) + 0x01010101u) >> 7 & 0x01010101u) * 0xFFu;
    return (w & nan) | (static_cast<uint32_t>(c) & ~nan);
}

// Eight bf16 values times 2^-e (exact) as codes; what is not finite becomes
// the code 0x7F.
__device__ __forceinline__ uint2 encode8(uint4 v, float by) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t o[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t a = w[2 * h], b = w[2 * h + 1];
        int c = __builtin_amdgcn_cvt_pk_fp8_f32(__uint_as_float(a << 16) * by, __uint_as_float(a & 0xFFFF0000u) * by, 0, false);
        c = __builtin_amdgcn_cvt_pk_fp8_f32(__uint_as_float(b << 16) * by, __uint_as_float(b & 0xFFFF0000u) * by, c, true);
        o[h] = static_cast<uint32_t>(c);
        // an exponent of all ones plus one carries into the sign's place
        const uint32_t x = (a & 0x7F807F80u) + 0x00800080u, y = (b & 0x7F807F80u) + 0x00800080u;
        if (__builtin_expect(((x | y) & 0x80008000u) != 0, 0)) {
            const uint32_t bad = (x >> 15 & 1u) | (x >> 23 & 0x100u) | (y << 1 & 0x10000u) | (y >> 7 & 0x1000000u);
            o[h] = (o[h] & ~(bad * 0xFFu)) | bad * 0x7Fu;
        }
    }
    return make_uint2(o[0], o[1]);
}

// Largest finite magnitude of eight bf16 values, as bits.
__device__ __forceinline__ uint32_t top8(uint4 v) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t lo = w[i] & 0x7FFFu, hi = w[i] >> 16 & 0x7FFFu;
        top = max(top, max(lo < 0x7F80u ? lo : 0u, hi < 0x7F80u ? hi : 0u));
    }
    return top;
}

// E8M0 byte of the least 2^e, e >= -127, with m <= 448 2^e, m given as bf16
// bits: 448 = 1.75 2^8, so e is m's exponent - 8, one more where its fraction
// is past 1.75; subnormal m are below 448 2^-127 by far.
__device__ __forceinline__ int scale_byte(uint32_t m) {
    const int e = static_cast<int>(m >> 7) - 8 + ((m & 0x7Fu) > 0x60u ? 1 : 0);
    return e > 0 ? e : 0;
}

// The item's sequence and its block, counted from the first one that the
// sequence's new rows touch: dense, every sequence has `most` items, or packed
// one sequence after another (a scan over the sequences, 64 at a time).
struct Rows {
    int first, m, n;       // first row of k and v, how many, the sequence's length with them
    __device__ __forceinline__ Rows(const AppendArgs& a, int b) {
        n = bounded(a.seq_lens[b], 0, a.capacity);
        if (a.cu_rows) {
            bounded_rows(a.cu_rows[b], a.cu_rows[b + 1], a.total, first, m);
            m = min(m, a.L);
        } else {
            first = b * a.L;
            m = a.L;
        }
    }
    // positions n - m .. n - 1, those below 0 left out
    __device__ __forceinline__ int from() const { return max(n - m, 0); }
    __device__ __forceinline__ int blocks(int log2) const { return m > 0 && n > 0 ? ((n - 1) >> log2) - (from() >> log2) + 1 : 0; }
};

template <int WPI>
__global__ __launch_bounds__(kCThreads) void kv_append_e4m3_kernel(AppendArgs a) {
    __shared__ uint32_t tops[kCThreads / kWave];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int part = wave % WPI;
    const int id = static_cast<int>(blockIdx.x) * (4 / WPI) + wave / WPI;
    // (head, keys or values) fastest: neighbours read neighbouring parts of a row
    int hv;
    const int item = a.by_heads2.divide(id, hv);
    const bool values = hv >= a.Hkv;
    const int h = values ? hv - a.Hkv : hv;
    int b = -1, nth = 0;
    if (id < a.items) {
        if (a.dense) {
            b = a.by_most.divide(item, nth);
        } else {
            int before = 0;
            for (int b0 = 0; b0 < a.B; b0 += 64) {
                const int c = b0 + lane < a.B ? Rows(a, b0 + lane).blocks(a.block_log2) : 0;
                int incl = c;
#pragma unroll
                for (int o = 1; o < 64; o <<= 1) {
                    const int up = __shfl_up(incl, o, 64);
                    if (lane >= o) incl += up;
                }
                const uint64_t hit = __ballot(item >= before + incl - c && item < before + incl);
                if (hit) {
                    const int src = __builtin_ctzll(hit);
                    b = b0 + src;
                    nth = item - __builtin_amdgcn_readlane(before + incl - c, src);
                    break;
                }
                before += __builtin_amdgcn_readlane(incl, 63);
            }
        }
    }
    int lo = 0, hi = 0, p0 = 0, first = 0, page = -1, start = 0;
    if (b >= 0) {
        const Rows r(a, b);
        if (static_cast<uint32_t>(nth) < static_cast<uint32_t>(r.blocks(a.block_log2))) {
            start = ((r.from() >> a.block_log2) + nth) << a.block_log2;
            p0 = r.n - r.m;
            first = r.first;
            lo = max(start, r.from());
            hi = min(start + (1 << a.block_log2), r.n);
            page = a.block_table[static_cast<int64_t>(b) * a.pages_per_seq + (start >> a.page_log2)];
        }
    }
    if (static_cast<uint32_t>(page) >= a.num_pages) hi = lo;       // nothing to do, but the barrier
    // rows of 8 gw channels, 64 / gw rows per wave step
    const int u = lane & (a.gw - 1), rps = 64 >> a.gw_log2, step = rps * WPI;
    const bool live = u * 8 < a.D;
    const int row0 = lo + part * rps + (lane >> a.gw_log2);
    const int64_t stride = values ? a.v_stride : a.k_stride;
    const uint16_t* const src = (values ? a.v : a.k) + static_cast<int64_t>(h) * a.D + u * 8;
    auto fetch = [&](int p) __attribute__((always_inline)) {
        return *reinterpret_cast<const uint4*>(src + (first + static_cast<int64_t>(p - p0)) * stride);
    };
    const int64_t slot = (static_cast<int64_t>(page) << a.page_log2) + (start & ((1 << a.page_log2) - 1));
    uint8_t* const scale = (values ? a.v_scales : a.k_scales) + (slot >> a.block_log2) * a.Hkv + h;
    const int old = lo - start;                                   // rows that the block held before
    int was = 0;
    if (old > 0 && lo < hi) was = min(static_cast<int>(*scale), 254);   // a NaN scale counts as the largest
    uint4 x[kKeep];
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < kKeep; ++i) {
        const int p = row0 + i * step;
        x[i] = make_uint4(0, 0, 0, 0);
        if (live && p < hi) x[i] = fetch(p);
    }
#pragma unroll
    for (int i = 0; i < kKeep; ++i) top = max(top, top8(x[i]));
    for (int p = row0 + kKeep * step; p < hi; p += step)
        if (live) top = max(top, top8(fetch(p)));
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), off, kWave)));
    if constexpr (WPI > 1) {
        if (lane == 0) tops[wave] = top;
        __syncthreads();                                          // and every wave has read the old scale
#pragma unroll
        for (int i = 0; i < WPI; ++i) top = max(top, tops[i]);
    }
    if (lo >= hi) return;
    const int byte = max(scale_byte(top), was);
    uint8_t* const dst = (values ? a.v_cache : a.k_cache) + (slot * a.Hkv + h) * a.D + u * 8;
    const int64_t row_bytes = static_cast<int64_t>(a.Hkv) * a.D;
    if (byte != was && live) {
        // 448 2^-19 rounds to 0: what moves further is 0 as well
        const float by = __uint_as_float(static_cast<uint32_t>(max(was - byte, -30) + 127) << 23);
        // kKeep steps' codes on their way at a time (64 single tokens, each behind
        // 63 rows of its block that all move: 6.6 us, by four waves 7.6; behind
        // 127: 9.6, 9.5)
        for (int r = part * rps + (lane >> a.gw_log2); r < old; r += kKeep * step) {
            uint2 w[kKeep];
#pragma unroll
            for (int i = 0; i < kKeep; ++i)
                if (r + i * step < old) w[i] = *reinterpret_cast<const uint2*>(dst + (r + i * step) * row_bytes);
#pragma unroll
            for (int i = 0; i < kKeep; ++i)
                if (r + i * step < old)
                    *reinterpret_cast<uint2*>(dst + (r + i * step) * row_bytes) = make_uint2(rescale4(w[i].x, by), rescale4(w[i].y, by));
        }
    }
    const float by = e8m0_to_f32(254 - byte);                     // 2^-e
    auto put = [&](int p, uint4 v) __attribute__((always_inline)) {
        *reinterpret_cast<uint2*>(dst + (p - start) * row_bytes) = encode8(v, by);
    };
#pragma unroll
    for (int i = 0; i < kKeep; ++i) {
        const int p = row0 + i * step;
        if (live && p < hi) put(p, x[i]);
    }
    for (int p = row0 + kKeep * step; p < hi; p += step)
        if (live) put(p, fetch(p));
    if (lane == 0 && part == 0) *scale = static_cast<uint8_t>(byte);
}

}  // namespace

AppendPlan plan_kv_append(int64_t B, int64_t L, int64_t total, int64_t Hkv, int64_t block) {
    AppendPlan p{};
    // L rows in a line touch at most this many blocks
    p.most = (L + block - 2) / block + 1;
    // all rows together: a sequence's rows fill blocks but for two (and rows are
    // one sequence's each: offsets that fall could ask for more)
    const int64_t packed = total / block + 2 * B < total ? total / block + 2 * B : total;
    p.dense = B * p.most <= packed;
    p.items = (p.dense ? B * p.most : packed) * Hkv * 2;
    return p;
}

hipError_t launch_kv_append_e4m3(AppendArgs a, const AppendPlan& p, hipStream_t s) {
    a.dense = p.dense;
    a.items = static_cast<int>(p.items);
    a.by_most = Divisor(p.most);
    a.by_heads2 = Divisor(2 * a.Hkv);
    a.gw_log2 = 0;
    while ((8 << a.gw_log2) < a.D) ++a.gw_log2;
    a.gw = 1 << a.gw_log2;
    // One wave where it holds all of a block's new rows in its registers, four
    // where not: with one wave, rows that do not fit are read twice (8192 rows
    // of 8 heads of 128, blocks of 64: 15.5 us, with four waves 12.5; of 128:
    // 25.1, 12.5), with four, waves have little or nothing to do (blocks of 16:
    // 22.6 us, with one 12.5; of 32: 15.3, 12.4; 64 single tokens, blocks of
    // 64: 6.2, 4.5).
    const int rows = a.L < (1 << a.block_log2) ? a.L : 1 << a.block_log2;
    const int steps = (rows * a.gw + 63) / 64;                    // wave steps of them
    if (steps > kKeep) kv_append_e4m3_kernel<4><<<static_cast<unsigned>(p.items), kCThreads, 0, s>>>(a);
    else kv_append_e4m3_kernel<1><<<static_cast<unsigned>((p.items + 3) / 4), kCThreads, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace vla
