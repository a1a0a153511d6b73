// Per-head RMS norm, rotary positions and the append to a paged key/value
// cache in one pass over the rows of a QKV GEMM:
//   n = x * w / sqrt(mean(x^2) + eps)                  (q and k, with a weight)
//   (a, b) -> (a c - b s, b c + a s),  c, s = rot_scale * (cos, sin)(position * inv_freq[j])
// with (a, b) = (n_j, n_{j + rot/2}) or (n_2j, n_2j+1); channels rot .. D-1
// pass.  The rotated k row and the v row also go to their cache slot.  With
// AXES a token has a position on each of up to four axes (time, height, width)
// and pair j turns by the one that axis_of[j] names.
//
// A head is cut into units of 2 VEC channels that hold whole pairs: in the
// rotated part of the half layout VEC channels and their VEC partners rot/2
// further on, elsewhere 2 VEC consecutive channels.  A lane keeps one unit
// position for every head it handles, so its VEC angles are computed once per
// token and a wave reads 64 units (64 / GW heads of GW lanes) per step.  The
// norm's sum of squares runs over the GW lanes of a head.
//
// The angle is formed in fp64 revolutions and reduced before it is rounded:
// at position 2^20 an fp32 product alone would be off by 2^-5 radians.  The
// sine and cosine instructions take revolutions and are within 2^-22.9 of the
// exact values over one turn (measured at 2^24 points), 2^-13 of a bf16 step.
// Mean squares are fp32; heads whose sum of squares leaves its range (1e-30 ..
// 1e30) take it and the normed values in fp64, with the root on the mantissa, so
// the largest and smallest bf16 values neither overflow nor vanish.  Each output
// is rounded to bf16 once, from fp32.
// The kernel is bound by HBM on prompts and by latency on single tokens: a
// wave's loads of a head go out before the angles, and before the previous
// head's arithmetic.  Measured, captured calls one behind another: 16387 tokens
// of 32 heads on 8 of 128, appended and kept, 91 us (4.8 TB/s, where a copy
// reaches 5.14); 2049 tokens of 28 on 4 of 128, normed, 12.1 us (3.3 TB/s); 50
// tokens of 8 on 1 of 256 3.0 us and one token 2.8 us, the time of a launch.
// Positions on three axes cost a byte load per pair and a select: 12601 tokens of
// 32 on 8 of 128, normed, 71 us (4.7 TB/s), 256 patches of 16 on 16 of 72 4.2 us.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "vla_device.h"
#include "vla_internal.h"

namespace vla {
namespace {

constexpr int kRThreads = 256;

template <int VEC>
struct Words;   // VEC bf16 values as loaded
template <>
struct Words<8> { using type = uint4; };
template <>
struct Words<4> { using type = uint2; };

template <int VEC>
struct Axes;    // the axis bytes of VEC pairs
template <>
struct Axes<8> { using type = uint64_t; };
template <>
struct Axes<4> { using type = uint32_t; };

template <int VEC>
__device__ __forceinline__ void to_f32(typename Words<VEC>::type w, float* x) {
    uint32_t u[VEC / 2];
    __builtin_memcpy(u, &w, sizeof(w));
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) {
        x[2 * i] = __uint_as_float(u[i] << 16);
        x[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
    }
}

template <int VEC>
__device__ __forceinline__ typename Words<VEC>::type to_words(const float* x) {
    using W = typename Words<VEC>::type;
    uint32_t u[VEC / 2];
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) u[i] = f32x2_to_bf16x2(x[2 * i], x[2 * i + 1]);
    W w;
    __builtin_memcpy(&w, u, sizeof(w));
    return w;
}

template <int VEC, bool AXES>
__global__ __launch_bounds__(kRThreads) void qk_norm_rope_append_kernel(RopeArgs a) {
    using W = typename Words<VEC>::type;
    const int lane = threadIdx.x & 63;
    const int64_t wave = static_cast<int64_t>(blockIdx.x) * (kRThreads / 64) + (threadIdx.x >> 6);
    const int64_t t = wave / a.chunks;
    if (t >= a.T) return;
    const int chunk = static_cast<int>(wave - t * a.chunks);
    const int u = lane & (a.gw - 1), hs = lane >> a.gw_log2;
    const int hpw = 64 >> a.gw_log2;                     // heads per wave step
    const int units = a.D / (2 * VEC), rot_units = a.rot / (2 * VEC);
    const bool live = u < units, turned = u < rot_units;
    const int lo = (turned && !a.interleaved) ? u * VEC : 2 * VEC * u;
    const int hi = (turned && !a.interleaved) ? a.rot / 2 + u * VEC : 2 * VEC * u + VEC;

    const int heads = a.Hq + (a.v ? 2 : 1) * a.Hkv;
    const int first = chunk * a.steps * hpw, last = min(heads, first + a.steps * hpw);
    // q, k, v heads in one order: 0, 1, 2
    auto kind_of = [&](int h) { return h < a.Hq ? 0 : (h < a.Hq + a.Hkv ? 1 : 2); };
    W rx = {}, ry = {};
    auto fetch = [&](int h) __attribute__((always_inline)) {
        if (!live || h >= last) return;
        const int kind = kind_of(h);
        const uint16_t* src = kind == 0 ? a.q + t * a.q_stride + static_cast<int64_t>(h) * a.D
                              : kind == 1 ? a.k + t * a.k_stride + static_cast<int64_t>(h - a.Hq) * a.D
                                          : a.v + t * a.v_stride + static_cast<int64_t>(h - a.Hq - a.Hkv) * a.D;
        rx = *reinterpret_cast<const W*>(src + lo);
        ry = *reinterpret_cast<const W*>(src + hi);
    };
    const int64_t slot = a.slots ? a.slots[t] : -1;
    fetch(first + hs);

    float c[VEC], s[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) { c[e] = 1.0f; s[e] = 0.0f; }
    if (turned) {
        constexpr double kPerTurn = 0.15915494309189533577;   // 1 / (2 pi)
        int at[AXES ? kMostAxes : 1] = {};                    // the token's positions
        typename Axes<VEC>::type axis = 0;                    // one byte per pair
        if constexpr (AXES) {
            // the pairs' axes and every axis's position in flight together,
            // then a choice: an indexed load would wait for the first
            axis = *reinterpret_cast<const typename Axes<VEC>::type*>(a.axis_of + u * VEC);
#pragma unroll
            for (int x = 0; x < kMostAxes; ++x)
                if (x < a.axes) at[x] = a.positions[x * a.T + t];
        } else {
            at[0] = a.positions[t];
        }
        const double first = static_cast<double>(at[0]) * kPerTurn;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            double pos = first;
            if constexpr (AXES) {
                const uint32_t x = static_cast<uint32_t>(axis >> (8 * e)) & 0xFFu;
                int p = 0;                                    // an axis that the token does not have
#pragma unroll
                for (int i = 0; i < kMostAxes; ++i) p = x == static_cast<uint32_t>(i) ? at[i] : p;
                pos = static_cast<double>(p) * kPerTurn;
            }
            const double rev = pos * static_cast<double>(a.inv_freq[u * VEC + e]);
            const float f = static_cast<float>(rev - __builtin_rint(rev));
            s[e] = __builtin_amdgcn_sinf(f) * a.rot_scale;
            c[e] = __builtin_amdgcn_cosf(f) * a.rot_scale;
        }
    }
    const bool append = slot >= 0 && slot < a.num_slots;

    for (int h = first + hs; h < last; h += hpw) {
        const int kind = kind_of(h);
        const int hh = kind == 0 ? h : (kind == 1 ? h - a.Hq : h - a.Hq - a.Hkv);
        const int64_t at = (slot * a.Hkv + hh) * a.D;                 // in the caches
        const W vx = rx, vy = ry;
        fetch(h + hpw);
        if (kind == 2) {
            if (live && append) {
                *reinterpret_cast<W*>(a.v_cache + at + lo) = vx;
                *reinterpret_cast<W*>(a.v_cache + at + hi) = vy;
            }
            continue;
        }
        float x[VEC], y[VEC];
        to_f32<VEC>(vx, x);
        to_f32<VEC>(vy, y);
        const uint16_t* w = kind == 0 ? a.q_weight : a.k_weight;
        if (w) {
            auto weights = [&](float* wl, float* wh) __attribute__((always_inline)) {
                to_f32<VEC>(*reinterpret_cast<const W*>(w + lo), wl);
                to_f32<VEC>(*reinterpret_cast<const W*>(w + hi), wh);
            };
            // the lanes of one head share `kind`: the whole group is here
            float ss = 0.0f;
            if (live) {
#pragma unroll
                for (int e = 0; e < VEC; ++e) ss += x[e] * x[e] + y[e] * y[e];
            }
            for (int o = a.gw >> 1; o > 0; o >>= 1) ss += __shfl_xor(ss, o, 64);
            const float r = __builtin_amdgcn_rsqf(ss / static_cast<float>(a.D) + a.eps);
            if (!(ss > 1e-30f && ss < 1e30f)) {
                double sd = 0.0;
                if (live) {
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        sd += static_cast<double>(x[e]) * x[e];
                        sd += static_cast<double>(y[e]) * y[e];
                    }
                }
                for (int o = a.gw >> 1; o > 0; o >>= 1) sd += __shfl_xor(sd, o, 64);
                // 1 / sqrt(m 2^(2k)) = rsq(m) 2^-k with m in [1/2, 2); the
                // products too are fp64: x r alone can leave fp32 on either
                // side where x r w does not
                int ex;
                const double m = frexp(sd / a.D + static_cast<double>(a.eps), &ex);
                const int odd = ex & 1;
                const double rd = ldexp(static_cast<double>(__builtin_amdgcn_rsqf(static_cast<float>(odd ? 2.0 * m : m))),
                                        -((ex - odd) / 2));
                if (live) {
                    float wl[VEC], wh[VEC];
                    weights(wl, wh);
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        x[e] = static_cast<float>(x[e] * rd * wl[e]);
                        y[e] = static_cast<float>(y[e] * rd * wh[e]);
                    }
                }
            } else if (live) {
                float wl[VEC], wh[VEC];
                weights(wl, wh);
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    x[e] = x[e] * r * wl[e];
                    y[e] = y[e] * r * wh[e];
                }
            }
        }
        if (turned) {
            if (a.interleaved) {
#pragma unroll
                for (int e = 0; e < VEC / 2; ++e) {
                    const float p = x[2 * e], q = x[2 * e + 1];
                    x[2 * e] = p * c[e] - q * s[e];
                    x[2 * e + 1] = q * c[e] + p * s[e];
                    const float p2 = y[2 * e], q2 = y[2 * e + 1];
                    y[2 * e] = p2 * c[VEC / 2 + e] - q2 * s[VEC / 2 + e];
                    y[2 * e + 1] = q2 * c[VEC / 2 + e] + p2 * s[VEC / 2 + e];
                }
            } else {
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const float p = x[e], q = y[e];
                    x[e] = p * c[e] - q * s[e];
                    y[e] = q * c[e] + p * s[e];
                }
            }
        }
        if (!live) continue;
        const W wx = to_words<VEC>(x), wy = to_words<VEC>(y);
        if (kind == 0) {
            uint16_t* o = a.q_out + t * a.q_out_stride + static_cast<int64_t>(hh) * a.D;
            *reinterpret_cast<W*>(o + lo) = wx;
            *reinterpret_cast<W*>(o + hi) = wy;
        } else {
            if (a.k_out) {
                uint16_t* o = a.k_out + t * a.k_out_stride + static_cast<int64_t>(hh) * a.D;
                *reinterpret_cast<W*>(o + lo) = wx;
                *reinterpret_cast<W*>(o + hi) = wy;
            }
            if (append) {
                *reinterpret_cast<W*>(a.k_cache + at + lo) = wx;
                *reinterpret_cast<W*>(a.k_cache + at + hi) = wy;
            }
        }
    }
}

}  // namespace

hipError_t launch_qk_norm_rope_append(RopeArgs a, hipStream_t s) {
    // 16-byte words where whole pairs of them fit the head and its rotated
    // part (16387 tokens as above: 90 us, 8-byte words 97)
    const int vec = (a.D % 16 == 0 && a.rot % 16 == 0) ? 8 : 4;
    const int units = a.D / (2 * vec);
    a.gw_log2 = 0;
    while ((1 << a.gw_log2) < units) ++a.gw_log2;
    a.gw = 1 << a.gw_log2;
    const int hpw = 64 >> a.gw_log2;
    const int steps = (a.Hq + (a.v ? 2 : 1) * a.Hkv + hpw - 1) / hpw;    // wave steps of one token
    // one wave per step while that fills the GPU's 1024 SIMDs some 8 times
    // over, then one wave per token, which computes its angles once (300
    // tokens of 8 heads on 1 of 256: 3.8 us, one wave per token 5.0; 16387
    // tokens as above: 90 us, one wave per step 94).  Between the two the rule
    // is a compromise: 2049 tokens as above take 12.1 us in its three waves per
    // token, 11.1 in two, 11.9 in one, 11.7 in one per step
    int64_t chunks = (8192 + a.T - 1) / a.T;
    if (chunks > steps) chunks = steps;
    a.steps = static_cast<int>((steps + chunks - 1) / chunks);
    a.chunks = (steps + a.steps - 1) / a.steps;
    const int64_t blocks = (a.T * a.chunks + kRThreads / 64 - 1) / (kRThreads / 64);
    const dim3 grid(static_cast<unsigned>(blocks));
    if (a.axis_of) {
        if (vec == 8) qk_norm_rope_append_kernel<8, true><<<grid, kRThreads, 0, s>>>(a);
        else qk_norm_rope_append_kernel<4, true><<<grid, kRThreads, 0, s>>>(a);
    } else {
        if (vec == 8) qk_norm_rope_append_kernel<8, false><<<grid, kRThreads, 0, s>>>(a);
        else qk_norm_rope_append_kernel<4, false><<<grid, kRThreads, 0, s>>>(a);
    }
    return hipGetLastError();
}

}  // namespace vla
