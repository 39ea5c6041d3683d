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

// Two float32 in a register pair: one instruction for both, rounded as two.
// These row kernels are bound by issuing instructions as much as by memory.
typedef unsigned long long f2;
__device__ __forceinline__ f2 make_f2(float a, float b) {
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ f2 both(float a) { return make_f2(a, a); }
__device__ __forceinline__ void split(f2 v, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ float sum2(f2 v) {
    float a, b;
    split(v, a, b);
    return a + b;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
    f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
    f2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
    f2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ void get_f2(const float* v, f2 (&o)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = make_f2(v[2 * i], v[2 * i + 1]);
}
__device__ __forceinline__ void put_f2(const f2 (&v)[4], float* o) {
#pragma unroll
    for (int i = 0; i < 4; ++i) split(v[i], o[2 * i], o[2 * i + 1]);
}

// 16-byte pieces that a thread keeps for itself in shared memory while their
// copies are in flight: piece p of a slot at slot + p * pitch, pitch = threads * 16.
__device__ __forceinline__ void piece_copy16(uint32_t dst, const void* src, bool in) {      // else zeros
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}
__device__ __forceinline__ uint4 piece_read(uint32_t at) {
    uint4 u;
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w) : "r"(at) : "memory");
    return u;
}

constexpr int kChunk = 256;                   // channels of a warp's chunk
constexpr int kActGroup = MOM_ACT8_GROUP;     // channels that share a scale
static_assert(kChunk == 2 * kActGroup, "a chunk holds two groups");

// The hardware reciprocal and exponential (one and two ulps; tiny results are
// flushed to 0): a rounded division took 15 of an element's 50 instructions.
__device__ __forceinline__ float fast_rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float fast_ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// A lane's 8 channels of a row as they lie in memory (channels >= d give 0):
// held packed between the load and the use, so that several rows' worth can be
// in flight.  With VEC, d is a multiple of 8 and a lane's 8 channels are all in
// or all out.
template <typename T, bool VEC> struct Raw8 {
    static constexpr int PIECES = 0;
    float v[8];
    __device__ __forceinline__ void load(const T* row, int c0, int d, int lane) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int c = c0 + i * 32 + lane;
            v[i] = c < d ? to_f(row[c]) : 0.f;
        }
    }
    __device__ __forceinline__ void get(float* out) const {
#pragma unroll
        for (int i = 0; i < 8; ++i) out[i] = v[i];
    }
    // largest magnitude's bits of the lane's elements of each group
    __device__ __forceinline__ void amax(uint32_t (&m)[2]) const {
        m[0] = m[1] = 0u;
#pragma unroll
        for (int i = 0; i < 8; ++i) m[i >> 2] = max(m[i >> 2], __float_as_uint(v[i]) & 0x7fffffffu);
    }
};
template <> struct Raw8<bf16, true> {
    static constexpr int PIECES = 1;
    uint4 u;
    __device__ __forceinline__ void load(const bf16* row, int c0, int d, int lane) {
        const int c = c0 + lane * 8;
        u = c < d ? *reinterpret_cast<const uint4*>(row + c) : make_uint4(0u, 0u, 0u, 0u);
    }
    static __device__ __forceinline__ void copy(uint32_t slot, uint32_t, const bf16* row, int c0, int d, int lane) {
        const int c = c0 + lane * 8;
        piece_copy16(slot, row + (c < d ? c : 0), c < d);
    }
    __device__ __forceinline__ void take(uint32_t slot, uint32_t) { u = piece_read(slot); }
    __device__ __forceinline__ void get(float* out) const {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            out[2 * i] = __uint_as_float(w[i] << 16);
            out[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    __device__ __forceinline__ void amax(uint32_t (&m)[2]) const {      // two elements an instruction
        const uint32_t a = 0x7fff7fffu;
        const uint32_t t = __vmaxu2(__vmaxu2(u.x & a, u.y & a), __vmaxu2(u.z & a, u.w & a));
        m[0] = m[1] = max(t << 16, t & 0xffff0000u);
    }
};
template <> struct Raw8<float, true> {
    static constexpr int PIECES = 2;
    float4 a, b;
    static __device__ __forceinline__ void copy(uint32_t slot, uint32_t pitch, const float* row, int c0, int d, int lane) {
        const int c = c0 + lane * 8;
        piece_copy16(slot, row + (c < d ? c : 0), c < d);
        piece_copy16(slot + pitch, row + (c < d ? c + 4 : 0), c < d);
    }
    __device__ __forceinline__ void take(uint32_t slot, uint32_t pitch) {
        const uint4 u = piece_read(slot), v = piece_read(slot + pitch);
        a = make_float4(__uint_as_float(u.x), __uint_as_float(u.y), __uint_as_float(u.z), __uint_as_float(u.w));
        b = make_float4(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z), __uint_as_float(v.w));
    }
    __device__ __forceinline__ void load(const float* row, int c0, int d, int lane) {
        const int c = c0 + lane * 8;
        a = c < d ? *reinterpret_cast<const float4*>(row + c) : make_float4(0.f, 0.f, 0.f, 0.f);
        b = c < d ? *reinterpret_cast<const float4*>(row + c + 4) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    __device__ __forceinline__ void get(float* out) const {
        out[0] = a.x; out[1] = a.y; out[2] = a.z; out[3] = a.w;
        out[4] = b.x; out[5] = b.y; out[6] = b.z; out[7] = b.w;
    }
    __device__ __forceinline__ void amax(uint32_t (&m)[2]) const {
        float v[8];
        get(v);
        m[0] = 0u;
#pragma unroll
        for (int i = 0; i < 8; ++i) m[0] = max(m[0], __float_as_uint(v[i]) & 0x7fffffffu);
        m[1] = m[0];
    }
};

template <bool VEC, typename T>
__device__ __forceinline__ void load8(const T* row, int c0, int d, int lane, float* out) {
    Raw8<T, VEC> r;
    r.load(row, c0, d, lane);
    r.get(out);
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
// codes round_half_even(x / scale), exactly: the quotient is never formed.  A
// first code is the rounded product with 1/scale (the addition of 1.5 * 2^23
// leaves the integer in the low bits); the remainder x - code * scale, one
// fused multiply-add, is a multiple of half an ulp of the scale below 2^24 of
// them, so it is exact, and where it reaches half a scale the code moves by one
// (another code is nearer, or a tie goes to the even one).  That is rare: one
// test covers a lane's 8 elements.  A group whose largest magnitude is below
// 2^-100 is stored as zeros; a group that holds an infinity or a NaN gets a NaN
// scale, so that all of it restores to NaN.
constexpr float kRoundMagic = 12582912.f;                     // 1.5 * 2^23

// fl32(a / 127): the product with 1/127 and one correction by its remainder,
// which gives the rounded quotient of every float a >= 2^-100 (all mantissas
// were compared with the division).
__device__ __forceinline__ float act8_scale(uint32_t amax_bits) {
    if (amax_bits >= 0x7f800000u) return __uint_as_float(0x7fc00000u);
    const float a = __uint_as_float(amax_bits), r = 1.f / 127.f, q = a * r;
    return a < 7.888609052210118e-31f ? 0.f : fmaf(fmaf(-127.f, q, a), r, q);      // 2^-100
}

// The two groups' scales of a chunk from the lanes' maxima: the scale of
// element i in s[i >= 4] (VEC: both entries are the lane's own group's).
template <bool VEC> __device__ __forceinline__ void act8_scales(uint32_t (&m)[2], float (&s)[2]) {
    if constexpr (VEC) {
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) m[0] = max(m[0], __shfl_xor_sync(0xffffffffu, m[0], o));
        s[0] = s[1] = act8_scale(m[0]);
    } else {
        s[0] = act8_scale(__reduce_max_sync(0xffffffffu, m[0]));
        s[1] = act8_scale(__reduce_max_sync(0xffffffffu, m[1]));
    }
}

// The codes of a lane's 8 elements, in the low byte of q[i].
__device__ __forceinline__ void act8_codes(const float* v, const float (&s)[2], uint32_t* q) {
    // 1 / scale: an ulp off, which the remainder puts right (scale 0: the product is not used)
    const float inv[2] = {fast_rcp(s[0]), fast_rcp(s[1])};
    bool fix = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float f = fmaf(v[i], inv[i >> 2], kRoundMagic);
        const float r = fmaf(kRoundMagic - f, s[i >> 2], v[i]);
        q[i] = __float_as_uint(f);
        fix |= !(fabsf(r) < 0.5f * s[i >> 2]);                // also where the scale is 0 or NaN
    }
    if (fix) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float sc = s[i >> 2], half = 0.5f * sc;
            if (!(sc > 0.f)) { q[i] = 0u; continue; }
            const float r = fmaf(kRoundMagic - __uint_as_float(q[i]), sc, v[i]);
            const bool odd = (q[i] & 1u) != 0u;
            if (r > half || (r == half && odd)) q[i] += 1u;
            else if (r < -half || (r == -half && odd)) q[i] -= 1u;
        }
    }
}

// Codes and scales of a chunk out: codes_row [d], scales_row [ceil(d / 128)].
// v: the lane's elements, m: their groups' maxima (Raw8::amax).
template <bool VEC>
__device__ __forceinline__ void act8_store(const float* v, uint32_t (&m)[2], int c0, int d, int lane,
                                           int8_t* codes_row, float* scales_row) {
    float s[2];
    uint32_t q[8];
    act8_scales<VEC>(m, s);
    act8_codes(v, s, q);
    const int g0 = c0 / kActGroup;
    if constexpr (VEC) {
        const int c = c0 + lane * 8;
        if (c < d) {
            const uint32_t lo = __byte_perm(__byte_perm(q[0], q[1], 0x0040), __byte_perm(q[2], q[3], 0x0040), 0x5410);
            const uint32_t hi = __byte_perm(__byte_perm(q[4], q[5], 0x0040), __byte_perm(q[6], q[7], 0x0040), 0x5410);
            *reinterpret_cast<uint2*>(codes_row + c) = make_uint2(lo, hi);
            if ((lane & 15) == 0) scales_row[g0 + (lane >> 4)] = s[0];
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int c = c0 + i * 32 + lane;
            if (c < d) codes_row[c] = static_cast<int8_t>(q[i]);
        }
        if (lane == 0 && c0 < d) scales_row[g0] = s[0];
        if (lane == 0 && c0 + kActGroup < d) scales_row[g0 + 1] = s[1];
    }
}

// A lane's 8 restored values, code * scale (one rounding to float32), held
// packed until they are used.
struct Q8 {};                  // the stream's type tag where it is a checkpoint
template <bool VEC> struct Raw8Q;
template <> struct Raw8Q<true> {
    // a piece: all threads' codes, 8 bytes each, then a scale for 16 threads,
    // which lanes 0 and 16 copy for their half warps
    static constexpr int PIECES = 1;
    uint2 u;
    float s;
    static __device__ __forceinline__ void copy(uint32_t slot, uint32_t pitch, const int8_t* codes_row,
                                                const float* scales_row, int c0, int d, int lane) {
        const int c = c0 + lane * 8;
        const uint32_t at = slot - threadIdx.x * 8;
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;"
                     ::"r"(at), "l"(codes_row + (c < d ? c : 0)), "r"(c < d ? 8 : 0) : "memory");
        if ((lane & 15) == 0)
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;"
                         ::"r"(slot - threadIdx.x * 16 + pitch / 2 + (threadIdx.x >> 4) * 4),
                           "l"(scales_row + (c < d ? c / kActGroup : 0)), "r"(c < d ? 4 : 0) : "memory");
    }
    __device__ __forceinline__ void take(uint32_t slot, uint32_t pitch) {
        __syncwarp();
        asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(u.x), "=r"(u.y) : "r"(slot - threadIdx.x * 8) : "memory");
        asm volatile("ld.shared.f32 %0, [%1];"
                     : "=f"(s) : "r"(slot - threadIdx.x * 16 + pitch / 2 + (threadIdx.x >> 4) * 4) : "memory");
    }
    __device__ __forceinline__ void load(const int8_t* codes_row, const float* scales_row, int c0, int d, int lane) {
        const int c = c0 + lane * 8;
        u = make_uint2(0u, 0u);
        s = 0.f;
        if (c < d) {
            u = *reinterpret_cast<const uint2*>(codes_row + c);
            s = scales_row[c0 / kActGroup + (lane >> 4)];
        }
    }
    __device__ __forceinline__ void get(float* out) const {
        // byte + 128 in the low mantissa of 2^23: an exact float of the code
        const uint32_t w[2] = {u.x ^ 0x80808080u, u.y ^ 0x80808080u};
#pragma unroll
        for (int i = 0; i < 8; ++i)
            out[i] = (__uint_as_float(__byte_perm(w[i >> 2], 0x4b000000u, 0x7440 + (i & 3))) - 8388736.f) * s;
    }
};
template <> struct Raw8Q<false> {
    static constexpr int PIECES = 0;
    float v[8];
    __device__ __forceinline__ void load(const int8_t* codes_row, const float* scales_row, int c0, int d, int lane) {
        const int g0 = c0 / kActGroup;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int c = c0 + i * 32 + lane;
            v[i] = c < d ? static_cast<float>(codes_row[c]) * scales_row[g0 + (i >> 2)] : 0.f;
        }
    }
    __device__ __forceinline__ void get(float* out) const {
#pragma unroll
        for (int i = 0; i < 8; ++i) out[i] = v[i];
    }
};

}  // namespace mom
