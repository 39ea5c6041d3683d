// Row pieces shared by the residual-stream norms and the 8-bit activation
// checkpoints: how a warp's lanes hold 256 channels of a row, and the
// checkpoint's code and scale.
//
// A warp covers a chunk of 256 channels, 8 a lane.  With rows that 16-byte
// loads can take (VEC) lane l holds channels 8l .. 8l+7; otherwise it holds
// l, l+32, .. l+224, so that single-element loads stay coalesced.
#pragma once

#include "common.cuh"

namespace mom {

constexpr int kChunk = 256;                   // channels of a warp's chunk
constexpr int kActGroup = MOM_ACT8_GROUP;     // channels that share a scale
static_assert(kChunk == 2 * kActGroup, "a chunk holds two groups");

// channel of element i of lane l, from the chunk's first channel
template <bool VEC> __device__ __forceinline__ int chunk_col(int lane, int i) {
    return VEC ? lane * 8 + i : i * 32 + lane;
}

// 8 channels of a row from channel c0 of the chunk on; channels >= d give 0.
// With VEC, d is a multiple of 8 and a lane's 8 channels are all in or all out.
template <bool VEC, typename T>
__device__ __forceinline__ void load8(const T* row, int c0, int d, int lane, float* out) {
    if constexpr (VEC) {
        const int c = c0 + lane * 8;
        if (c < d) {
            load_vec<8>(row + c, out);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) out[i] = 0.f;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int c = c0 + i * 32 + lane;
            out[i] = c < d ? to_f(row[c]) : 0.f;
        }
    }
}
template <bool VEC, typename T>
__device__ __forceinline__ void store8(T* row, int c0, int d, int lane, const float* v) {
    if constexpr (VEC) {
        const int c = c0 + lane * 8;
        if (c < d) store_vec<8>(row + c, v);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int c = c0 + i * 32 + lane;
            if (c < d) row[c] = from_f<T>(v[i]);
        }
    }
}

// --------------------------------------------------- 8-bit checkpoints --
// A group of 128 channels of a row keeps scale = fl32(max|x| / 127) and the
// codes round_half_even(x / scale), exactly: the quotient is never formed, a
// rounded product with 1/scale gives a first code and the remainder
// x - code * scale (one fused multiply-add; it is a multiple of half an ulp
// of the scale below 2^24 of them, so it is exact) moves it by one where the
// product fell on the other side of a border.  A group whose largest
// magnitude is below 2^-100 is stored as zeros; a group that holds an
// infinity or a NaN gets a NaN scale, so that all of it restores to NaN.
__device__ __forceinline__ float act8_scale(uint32_t amax_bits) {
    if (amax_bits >= 0x7f800000u) return __uint_as_float(0x7fc00000u);
    const float a = __uint_as_float(amax_bits);
    return a < 7.888609052210118e-31f ? 0.f : a / 127.f;      // 2^-100
}
__device__ __forceinline__ int act8_code(float x, float s, float inv) {
    if (!(s > 0.f)) return 0;
    float q = rintf(x * inv);
    const float r = fmaf(-q, s, x), half = 0.5f * s;
    const bool odd = (static_cast<int>(q) & 1) != 0;
    if (r > half || (r == half && odd)) q += 1.f;
    if (r < -half || (r == -half && odd)) q -= 1.f;
    return static_cast<int>(q);
}

// The two groups' scales of a chunk held in v (lane layout above): every lane
// gets the scale of its element i in s[i >= 4] (VEC: both entries are its own
// group's).
template <bool VEC> __device__ __forceinline__ void act8_scales(const float* v, float (&s)[2]) {
    uint32_t m[2] = {0u, 0u};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t b = __float_as_uint(v[i]) & 0x7fffffffu;
        if constexpr (VEC) m[0] = m[0] > b ? m[0] : b;
        else m[i >> 2] = m[i >> 2] > b ? m[i >> 2] : b;
    }
    if constexpr (VEC) {
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) {
            const uint32_t b = __shfl_xor_sync(0xffffffffu, m[0], o);
            m[0] = m[0] > b ? m[0] : b;
        }
        s[0] = s[1] = act8_scale(m[0]);
    } else {
        s[0] = act8_scale(__reduce_max_sync(0xffffffffu, m[0]));
        s[1] = act8_scale(__reduce_max_sync(0xffffffffu, m[1]));
    }
}

// Codes and scales of a chunk out: codes_row [d], scales_row [ceil(d / 128)].
template <bool VEC>
__device__ __forceinline__ void act8_store(const float* v, int c0, int d, int lane, int8_t* codes_row,
                                           float* scales_row) {
    float s[2];
    act8_scales<VEC>(v, s);
    const float inv[2] = {s[0] > 0.f ? 1.f / s[0] : 0.f, s[1] > 0.f ? 1.f / s[1] : 0.f};
    const int g0 = c0 / kActGroup;
    if constexpr (VEC) {
        const int c = c0 + lane * 8;
        if (c < d) {
            uint32_t w[2] = {0u, 0u};
#pragma unroll
            for (int i = 0; i < 8; ++i)
                w[i >> 2] |= (static_cast<uint32_t>(act8_code(v[i], s[0], inv[0])) & 0xffu) << (8 * (i & 3));
            *reinterpret_cast<uint2*>(codes_row + c) = make_uint2(w[0], w[1]);
            if ((lane & 15) == 0) scales_row[g0 + (lane >> 4)] = s[0];
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int c = c0 + i * 32 + lane;
            if (c < d) codes_row[c] = static_cast<int8_t>(act8_code(v[i], s[i >> 2], inv[i >> 2]));
        }
        if (lane == 0 && c0 < d) scales_row[g0] = s[0];
        if (lane == 0 && c0 + kActGroup < d) scales_row[g0 + 1] = s[1];
    }
}

// The restored values of a chunk: code * scale (one rounding to float32).
template <bool VEC>
__device__ __forceinline__ void act8_load(const int8_t* codes_row, const float* scales_row, int c0, int d, int lane,
                                          float* out) {
    const int g0 = c0 / kActGroup;
    if constexpr (VEC) {
        const int c = c0 + lane * 8;
        if (c < d) {
            const uint2 u = *reinterpret_cast<const uint2*>(codes_row + c);
            const float s = scales_row[g0 + (lane >> 4)];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t w = i < 4 ? u.x : u.y;
                out[i] = static_cast<float>(static_cast<int8_t>(w >> (8 * (i & 3)))) * s;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) out[i] = 0.f;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int c = c0 + i * 32 + lane;
            out[i] = c < d ? static_cast<float>(codes_row[c]) * scales_row[g0 + (i >> 2)] : 0.f;
        }
    }
}

}  // namespace mom
