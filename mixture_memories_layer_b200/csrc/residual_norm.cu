// The residual stream between blocks: the norm after a block, its gate and
// residual scale, the addition to the stream and the next block's norm in one
// pass over a row, and the adjoint.
//
//   x' = x + s sigma(gate) n_y w_post,  n_y = y / rms(y)     rms(a)^2 = mean(a^2) + eps
//   h  = n_x w_pre,                     n_x = x' / rms(x')
//
// Adjoint, from D' = dL/dx' and dh = dL/dh:
//   D    = D' + (dn - n_x mean(dn n_x)) / rms(x'),  dn = dh w_pre,   dx = D
//   u    = D s sigma w_post,  dy = (u - n_y mean(u n_y)) / rms(y)
//   dgate = D s w_post n_y sigma (1 - sigma)        (its row's sum for one gate a token)
//   A    = sum_t D sigma n_y,  dw_post = s A,  ds = w_post A,  dw_pre = sum_t dh n_x
//
// Bound by memory and, with the 16 warps an SM that the registers leave, by each
// warp's own latencies (56 % of the issue slots forward, 62 % in the adjoint).
// A row is spread over the W warps of a CTA, C chunks of 256 channels a warp;
// every operand is read from memory once and later rows' operands are on their
// way while one is worked on.  Sums, norms and the whole arithmetic are float32;
// each output is rounded once, as it is stored.  16384 x 1024 bf16 with an
// element gate: forward 35 us, 4.8 TB/s; adjoint with float32 gradients and the
// stream from its checkpoint 72 us, 4.9 TB/s (a plain copy of 4 GB: 6.6).
#include <type_traits>

#include "rows8.cuh"
#include "kernels.h"

namespace mom {
namespace {

// The stream's operand: a type's elements or an 8-bit checkpoint.
template <typename XT, bool VEC> struct RawX : Raw8<XT, VEC> {
    typedef Raw8<XT, VEC> R;
    __device__ __forceinline__ void load(const ResNormArgs& a, int64_t row, int c0, int lane) {
        R::load(reinterpret_cast<const XT*>(a.x) + row * a.d, c0, a.d, lane);
    }
    static __device__ __forceinline__ void copy(uint32_t slot, uint32_t pitch, const ResNormArgs& a, int64_t row, int c0,
                                                int lane) {
        R::copy(slot, pitch, reinterpret_cast<const XT*>(a.x) + row * a.d, c0, a.d, lane);
    }
};
template <bool VEC> struct RawX<Q8, VEC> : Raw8Q<VEC> {
    typedef Raw8Q<VEC> R;
    __device__ __forceinline__ void load(const ResNormArgs& a, int64_t row, int c0, int lane) {
        R::load(a.x_codes + row * a.d, a.x_scales + row * a.groups, c0, a.d, lane);
    }
    static __device__ __forceinline__ void copy(uint32_t slot, uint32_t pitch, const ResNormArgs& a, int64_t row, int c0,
                                                int lane) {
        R::copy(slot, pitch, a.x_codes + row * a.d, a.x_scales + row * a.groups, c0, a.d, lane);
    }
};

// sigma(z) = 1 / (1 + e), e = exp(-z), by the hardware exponential and
// reciprocal.  Its relative error is at most 1.22 |z| + 4 + 1 + 2 in 2^-24: the
// exponent's two roundings, the exponential, the sum, the reciprocal; 2^-19.9
// for |z| < 8, 2^-17.6 at 60, where sigma or 1 - sigma is 1e-26.  1 - sigma
// without cancellation: e sigma for z > 0.
__device__ __forceinline__ float sigmoid(float z, float& rest) {
    const float e = fast_ex2(z * -1.4426950408889634f), s = fast_rcp(1.f + e);
    rest = z > 0.f ? e * s : 1.f - s;
    return s;
}
__device__ __forceinline__ void sigmoid(f2 (&v)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float a, b;
        split(mul2(v[i], both(-1.4426950408889634f)), a, b);
        split(add2(make_f2(fast_ex2(a), fast_ex2(b)), both(1.f)), a, b);
        v[i] = make_f2(fast_rcp(a), fast_rcp(b));
    }
}

constexpr int kMaxWarps = 16;      // of a row

// Sums of K values over the W warps of a row (every thread gets them), in warp
// order; one warp a row needs no barrier.  buf [K][kMaxWarps] holds zeros past
// warp W.
template <int K> __device__ __forceinline__ void row_sum(float (&v)[K], float* buf, int W, int warp, int lane) {
    warp_sum_n<K>(v);
    if (W == 1) return;
    if (lane == 0)
#pragma unroll
        for (int k = 0; k < K; ++k) buf[k * kMaxWarps + warp] = v[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = 0.f;
    for (int i = 0; i < W; i += 4)
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const float4 p = *reinterpret_cast<const float4*>(buf + k * kMaxWarps + i);
            v[k] += (p.x + p.y) + (p.z + p.w);
        }
}

// The column weights of a thread's channels, res_scale * w_post and w_pre: in
// registers for all of a CTA's rows with one chunk a warp, else read again
// (from L1) at each use.
template <bool VEC, int C> struct Weights {
    static constexpr bool KEEP = C == 1;
    f2 post[KEEP ? 4 : 1], pre[KEEP ? 4 : 1];
    static __device__ __forceinline__ void read(const float* from, const ResNormArgs& a, int c0, int lane, f2 (&w)[4]) {
        float v[8];
        load8<VEC>(from, c0, a.d, lane, v);
        get_f2(v, w);
    }
    static __device__ __forceinline__ void read_post(const ResNormArgs& a, int c0, int lane, f2 (&w)[4]) {
        read(a.w_post, a, c0, lane, w);
        if (a.res_scale) {
            f2 s[4];
            read(a.res_scale, a, c0, lane, s);
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = mul2(w[i], s[i]);
        }
    }
    __device__ __forceinline__ Weights(const ResNormArgs& a, bool has_pre, int c0, int lane) {
        if constexpr (KEEP) {
#pragma unroll
            for (int i = 0; i < 4; ++i) post[i] = pre[i] = 0ull;
            if (a.y) read_post(a, c0, lane, post);
            if (has_pre) read(a.w_pre, a, c0, lane, pre);
        }
    }
    __device__ __forceinline__ void get_post(const ResNormArgs& a, int c0, int lane, f2 (&w)[4]) const {
        if constexpr (KEEP) {
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = post[i];
        } else {
            read_post(a, c0, lane, w);
        }
    }
    __device__ __forceinline__ void get_pre(const ResNormArgs& a, int c0, int lane, f2 (&w)[4]) const {
        if constexpr (KEEP) {
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = pre[i];
        } else {
            read(a.w_pre, a, c0, lane, w);
        }
    }
};

// Where the rows' operands come from.
//   RING    the forward's rows of up to 8192 channels that 16-byte copies take:
//           copies in flight to slots in shared memory, the slots but one rows
//           ahead (more without a block's output, when a row is short); each
//           thread reads only what it copied itself (no barrier), into
//           registers, and a slot is filled again one row after it was read
//   REGS    loads into registers one row ahead, one chunk a warp
//   DIRECT  loads when the row's turn comes, its lines asked into L2 one row
//           ahead: the adjoint's rows that 16-byte loads cannot take, and wide
//           rows, which are read again at each use, from L1
// 16 M elements bf16, d 8192, forward: 49 us by RING, 64 us by DIRECT; 3001 x
// 1021 float32, adjoint: 23 us by DIRECT, 31 us by REGS, which spill.
enum Source { RING, REGS, DIRECT };

template <typename R> __device__ __forceinline__ void take_f2(const R& r, f2 (&v)[4]) {
    float f[8];
    r.get(f);
    get_f2(f, v);
}
template <bool VEC, typename T>
__device__ __forceinline__ void store_f2(T* row, int c0, int d, int lane, const f2 (&v)[4]) {
    float f[8];
    put_f2(v, f);
    store8<VEC>(row, c0, d, lane, f);
}

__device__ __forceinline__ void ask_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// HAS_Y: whether there is a block's output (the adjoint asks at run time)
template <typename XT, typename T, typename G, bool VEC, int C, bool HAS_Y, bool BWD, int SRC> struct Rows {
    static constexpr bool HOLD = C == 1 || SRC == RING;      // the registers hold a row
    static_assert(SRC != REGS || C == 1, "");
    enum { SLOTS = C == 2 ? (HAS_Y ? 2 : 4) : HAS_Y ? 3 : 5 };
    typedef RawX<XT, VEC> X;
    typedef Raw8<T, VEC> Y;
    typedef Raw8<G, VEC> D;
    struct Held {
        X x;
        Y y, g;
        D d, h;
    };
    const ResNormArgs& a;
    const ResNormBwdArgs& b;
    int W, warp, lane;
    int64_t row, step;
    Held cur[HOLD ? C : 1], next;            // REGS: the next row's
    uint32_t base, pitch, bytes;             // RING
    int in, out;

    static __host__ __device__ __forceinline__ int pieces(const ResNormArgs& a) {
        return X::PIECES + (HAS_Y ? (a.gate_mode == MOM_GATE_ELEMENT ? 2 : 1) * Y::PIECES : 0);
    }
    __device__ __forceinline__ bool has_y() const { return HAS_Y && (!BWD || a.y); }
    __device__ __forceinline__ int c0(int j) const { return (warp + j * W) * kChunk; }
    __device__ __forceinline__ const T* at_y(int64_t r) const { return reinterpret_cast<const T*>(a.y) + r * a.d; }
    __device__ __forceinline__ const T* at_g(int64_t r) const { return reinterpret_cast<const T*>(a.gate) + r * a.d; }
    __device__ __forceinline__ const G* at_d(int64_t r) const { return reinterpret_cast<const G*>(b.dx_out) + r * a.d; }
    __device__ __forceinline__ const G* at_h(int64_t r) const { return reinterpret_cast<const G*>(b.dh) + r * a.d; }
    __device__ __forceinline__ bool elem() const { return HAS_Y && a.gate_mode == MOM_GATE_ELEMENT; }

    __device__ __forceinline__ Rows(const ResNormArgs& a_, const ResNormBwdArgs& b_, void* smem, int W_,
                                    int warp_, int lane_, int64_t first, int64_t step_)
        : a(a_), b(b_), W(W_), warp(warp_), lane(lane_), row(first), step(step_) {
        if constexpr (SRC == RING) {
            pitch = blockDim.x * 16;
            base = (uint32_t)__cvta_generic_to_shared(smem) + threadIdx.x * 16;
            bytes = C * pieces(a) * pitch;
            in = out = 0;
#pragma unroll
            for (int i = 0; i < SLOTS - 1; ++i) put(row + i * step);
        } else if constexpr (SRC == REGS) {
            load(next, first, 0);
        }
    }
    __device__ __forceinline__ void load(Held& o, int64_t r, int j) {
        if (r >= a.n_rows) return;
        if (has_y()) o.y.load(at_y(r), c0(j), a.d, lane);
        o.x.load(a, r, c0(j), lane);
        if (elem()) o.g.load(at_g(r), c0(j), a.d, lane);
        if (BWD && b.dh) o.h.load(at_h(r), c0(j), a.d, lane);
        if (BWD && b.dx_out) o.d.load(at_d(r), c0(j), a.d, lane);
    }
    __device__ __forceinline__ void put(int64_t r) {
        if (r < a.n_rows) {
            uint32_t at = base + in * bytes;
#pragma unroll
            for (int j = 0; j < C; ++j) {
                X::copy(at, pitch, a, r, c0(j), lane);
                at += X::PIECES * pitch;
                if (HAS_Y) {
                    Y::copy(at, pitch, at_y(r), c0(j), a.d, lane);
                    at += Y::PIECES * pitch;
                }
                if (elem()) {
                    Y::copy(at, pitch, at_g(r), c0(j), a.d, lane);
                    at += Y::PIECES * pitch;
                }
            }
        }
        in = in + 1 == SLOTS ? 0 : in + 1;
        asm volatile("cp.async.commit_group;" ::: "memory");
    }
    __device__ __forceinline__ void take() {
        asm volatile("cp.async.wait_group %0;" ::"n"(SLOTS - 2) : "memory");      // all but the youngest
        uint32_t at = base + out * bytes;
#pragma unroll
        for (int j = 0; j < C; ++j) {
            cur[j].x.take(at, pitch);
            at += X::PIECES * pitch;
            if (HAS_Y) {
                cur[j].y.take(at, pitch);
                at += Y::PIECES * pitch;
            }
            if (elem()) {
                cur[j].g.take(at, pitch);
                at += Y::PIECES * pitch;
            }
        }
        out = out + 1 == SLOTS ? 0 : out + 1;
    }
    __device__ __forceinline__ void ask(int64_t r) const {
        if (r >= a.n_rows) return;
#pragma unroll
        for (int j = 0; j < C; ++j) {
            const int c = c0(j) + lane * 8;
            if (c >= a.d) continue;
            if (a.x) ask_l2(reinterpret_cast<const char*>(a.x) + (r * a.d + c) * (std::is_same<XT, bf16>::value ? 2 : 4));
            else ask_l2(a.x_codes + r * a.d + c);
            if (has_y()) ask_l2(at_y(r) + c);
            if (elem()) ask_l2(at_g(r) + c);
            if (BWD && b.dh) ask_l2(at_h(r) + c);
            if (BWD && b.dx_out) ask_l2(at_d(r) + c);
        }
    }
    // the row at work is there, and a later one is on its way
    __device__ __forceinline__ void begin() {
        if constexpr (SRC == RING) {
            take();
            put(row + (SLOTS - 1) * step);
        } else if constexpr (SRC == REGS) {
            cur[0] = next;
            load(next, row + step, 0);
        } else {
            if constexpr (HOLD) {
#pragma unroll
                for (int j = 0; j < C; ++j) load(cur[j], row, j);
            }
            ask(row + step);
        }
    }
    __device__ __forceinline__ void x(int j, X& o) const {
        if constexpr (HOLD) o = cur[j].x;
        else o.load(a, row, c0(j), lane);
    }
    __device__ __forceinline__ void y(int j, f2 (&v)[4]) const {
        if constexpr (HOLD) { take_f2(cur[j].y, v); return; }
        Y o;
        o.load(at_y(row), c0(j), a.d, lane);
        take_f2(o, v);
    }
    __device__ __forceinline__ void g(int j, f2 (&v)[4]) const {
        if constexpr (HOLD) { take_f2(cur[j].g, v); return; }
        Y o;
        o.load(at_g(row), c0(j), a.d, lane);
        take_f2(o, v);
    }
    __device__ __forceinline__ void h(int j, f2 (&v)[4]) const {
        if constexpr (HOLD) { take_f2(cur[j].h, v); return; }
        D o;
        o.load(at_h(row), c0(j), a.d, lane);
        take_f2(o, v);
    }
    __device__ __forceinline__ void d(int j, f2 (&v)[4]) const {
        if constexpr (HOLD) { take_f2(cur[j].d, v); return; }
        D o;
        o.load(at_d(row), c0(j), a.d, lane);
        take_f2(o, v);
    }
};

// CTAs (warps, with one warp a row) walk the rows.  `red` alternates between
// two rows, so that one barrier a sum is enough.
template <typename XT, typename T, bool VEC, int C, bool HAS_Y, int SRC, int MAXT>
__global__ void __launch_bounds__(MAXT, MAXT > 256 ? 1 : SRC == RING && !HAS_Y ? 4 : 2)
residual_norm_kernel(const ResNormArgs a) {
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ __align__(16) float red[2][2][kMaxWarps];
    if (threadIdx.x < 4 * kMaxWarps) (&red[0][0][0])[threadIdx.x] = 0.f;
    const int lane = threadIdx.x & 31, W = a.warps_per_row, warp = W > 1 ? threadIdx.x >> 5 : 0;
    const int rows_cta = W > 1 ? 1 : blockDim.x >> 5;
    const int64_t step = (int64_t)gridDim.x * rows_cta;
    const int64_t first = (int64_t)blockIdx.x * rows_cta + (W > 1 ? 0 : threadIdx.x >> 5);
    const int d = a.d;
    const float inv_d = 1.f / (float)d;
    const ResNormBwdArgs none{};
    Rows<XT, T, T, VEC, C, HAS_Y, false, SRC> in(a, none, smem, W, warp, lane, first, step);
    T gate_next = from_f<T>(0.f);
    if (a.gate_mode == MOM_GATE_TOKEN && first < a.n_rows) gate_next = reinterpret_cast<const T*>(a.gate)[first];
    const Weights<VEC, C> wt(a, a.h != nullptr, warp * kChunk, lane);
    __syncthreads();
    for (int buf = 0; in.row < a.n_rows; in.row += in.step, buf ^= 1) {      // the same count in all warps of a row
        const int64_t row = in.row, at = row * d;
        in.begin();
        const T gate = gate_next;
        if (a.gate_mode == MOM_GATE_TOKEN && row + step < a.n_rows)
            gate_next = reinterpret_cast<const T*>(a.gate)[row + step];
        f2 xv[C][4];
        float ry = 0.f, ss[1];
        if (HAS_Y) {
            f2 q = 0ull;
#pragma unroll
            for (int j = 0; j < C; ++j) {
                f2 y[4];
                in.y(j, y);
#pragma unroll
                for (int i = 0; i < 4; ++i) q = fma2(y[i], y[i], q);
            }
            ss[0] = sum2(q);
            row_sum<1>(ss, red[buf][0], W, warp, lane);
            ry = rsqrtf(ss[0] * inv_d + a.eps);                     // 1 / rms(y), times a token's gate
            if (a.gate_mode == MOM_GATE_TOKEN) {
                float rest;
                ry *= sigmoid(to_f(gate), rest);
            }
        }
        f2 q = 0ull;
#pragma unroll
        for (int j = 0; j < C; ++j) {
            const int c0 = in.c0(j);
            RawX<XT, VEC> x;
            in.x(j, x);
            take_f2(x, xv[j]);
            if constexpr (!std::is_same<XT, Q8>::value) {
                if (a.codes_out) {
                    uint32_t m[2];
                    float f[8];
                    x.amax(m);
                    put_f2(xv[j], f);
                    act8_store<VEC>(f, m, c0, d, lane, a.codes_out + at, a.scales_out + row * a.groups);
                }
            }
            if (HAS_Y) {
                f2 y[4], w[4];
                in.y(j, y);
                wt.get_post(a, c0, lane, w);
#pragma unroll
                for (int i = 0; i < 4; ++i) y[i] = mul2(y[i], both(ry));
                if (a.gate_mode == MOM_GATE_ELEMENT) {
                    f2 g[4];
                    in.g(j, g);
                    sigmoid(g);
#pragma unroll
                    for (int i = 0; i < 4; ++i) y[i] = mul2(y[i], g[i]);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) xv[j][i] = fma2(y[i], w[i], xv[j][i]);
            }
            if (a.x_out) {
                if (a.x_out_f32) store_f2<VEC>(reinterpret_cast<float*>(a.x_out) + at, c0, d, lane, xv[j]);
                else store_f2<VEC>(reinterpret_cast<bf16*>(a.x_out) + at, c0, d, lane, xv[j]);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) q = fma2(xv[j][i], xv[j][i], q);
        }
        if (a.h) {
            ss[0] = sum2(q);
            row_sum<1>(ss, red[buf][1], W, warp, lane);
            const f2 rx = both(rsqrtf(ss[0] * inv_d + a.eps));
#pragma unroll
            for (int j = 0; j < C; ++j) {
                f2 w[4];
                wt.get_pre(a, in.c0(j), lane, w);
#pragma unroll
                for (int i = 0; i < 4; ++i) xv[j][i] = mul2(mul2(xv[j][i], rx), w[i]);
                store_f2<VEC>(reinterpret_cast<T*>(a.h) + at, in.c0(j), d, lane, xv[j]);
            }
        }
    }
}

// The adjoint.  Threads keep the two column sums (A and dw_pre) of their
// channels in registers over all of a CTA's rows and write them once as a
// partial, which cols_reduce_kernel adds up in CTA order: no atomics, the same
// sums every time on the same device.  With one chunk a warp n_y and sigma stay
// in registers between the passes over a row, else they are formed again.
template <typename XT, typename T, typename G, bool VEC, int C, int SRC, int MAXT>
__global__ void __launch_bounds__(MAXT, MAXT > 256 ? 1 : 2)
residual_norm_bwd_kernel(const ResNormArgs a, const ResNormBwdArgs b) {
    __shared__ __align__(16) float red[2][4][kMaxWarps];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    for (int i = threadIdx.x; i < 8 * kMaxWarps; i += blockDim.x) (&red[0][0][0])[i] = 0.f;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, W = blockDim.x >> 5;
    const int d = a.d;
    const float inv_d = 1.f / (float)d;
    f2 accA[C][4], accP[C][4];
#pragma unroll
    for (int j = 0; j < C; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) accA[j][i] = accP[j][i] = 0ull;
    Rows<XT, T, G, VEC, C, true, true, SRC> in(a, b, nullptr, W, warp, lane, blockIdx.x, gridDim.x);
    T gate_next = from_f<T>(0.f);
    if (a.gate_mode == MOM_GATE_TOKEN && in.row < a.n_rows) gate_next = reinterpret_cast<const T*>(a.gate)[in.row];
    const Weights<VEC, C> wt(a, b.dh != nullptr, warp * kChunk, lane);
    __syncthreads();
    for (int buf = 0; in.row < a.n_rows; in.row += in.step, buf ^= 1) {
        const int64_t row = in.row, at = row * d;
        in.begin();
        const T gate = gate_next;
        if (a.gate_mode == MOM_GATE_TOKEN && row + in.step < a.n_rows)
            gate_next = reinterpret_cast<const T*>(a.gate)[row + in.step];
        f2 yk[C == 1 ? 4 : 1], gk[C == 1 ? 4 : 1], dv[C][4];
        float gt = 1.f, rest = 0.f, ry = 0.f;
        if (a.gate_mode == MOM_GATE_TOKEN) gt = sigmoid(to_f(gate), rest);
        // n_y and sigma of chunk j
        auto form = [&](int j, f2 (&y)[4], f2 (&g)[4]) {
            in.y(j, y);
#pragma unroll
            for (int i = 0; i < 4; ++i) y[i] = mul2(y[i], both(ry));
            if (a.gate_mode == MOM_GATE_ELEMENT) {
                in.g(j, g);
                sigmoid(g);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) g[i] = both(gt);
            }
        };
        auto again = [&](int j, f2 (&y)[4], f2 (&g)[4]) {
            if constexpr (C == 1) {
#pragma unroll
                for (int i = 0; i < 4; ++i) { y[i] = yk[i]; g[i] = gk[i]; }
            } else {
                form(j, y, g);
            }
        };
        if (a.y) {
            f2 q = 0ull;
#pragma unroll
            for (int j = 0; j < C; ++j) {
                f2 y[4];
                in.y(j, y);
#pragma unroll
                for (int i = 0; i < 4; ++i) q = fma2(y[i], y[i], q);
            }
            float ss[1] = {sum2(q)};
            row_sum<1>(ss, red[buf][0], W, warp, lane);
            ry = rsqrtf(ss[0] * inv_d + a.eps);
            if constexpr (C == 1) form(0, yk, gk);
        }
        if (b.dh) {
            f2 qx = 0ull, qh = 0ull;
#pragma unroll
            for (int j = 0; j < C; ++j) {                                     // dv: x' for now
                f2 h[4], w[4];
                RawX<XT, VEC> x;
                in.x(j, x);
                take_f2(x, dv[j]);
                if (a.y) {
                    f2 y[4], g[4];
                    again(j, y, g);
                    wt.get_post(a, in.c0(j), lane, w);
#pragma unroll
                    for (int i = 0; i < 4; ++i) dv[j][i] = fma2(mul2(y[i], g[i]), w[i], dv[j][i]);
                }
                in.h(j, h);
                wt.get_pre(a, in.c0(j), lane, w);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    qx = fma2(dv[j][i], dv[j][i], qx);
                    qh = fma2(dv[j][i], mul2(h[i], w[i]), qh);
                }
            }
            float ss[2] = {sum2(qx), sum2(qh)};
            row_sum<2>(ss, red[buf][1], W, warp, lane);
            const float r = rsqrtf(ss[0] * inv_d + a.eps);
            const f2 rx = both(r), mk = both(-ss[1] * inv_d * r * r * r);     // - mean(dn n_x) / rms / rms
#pragma unroll
            for (int j = 0; j < C; ++j) {
                f2 h[4], w[4], o[4];
                in.h(j, h);
                wt.get_pre(a, in.c0(j), lane, w);
                if (b.dx_out) {
                    in.d(j, o);
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[i] = 0ull;
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const f2 hr = mul2(h[i], rx);
                    accP[j][i] = fma2(hr, dv[j][i], accP[j][i]);
                    dv[j][i] = fma2(hr, w[i], fma2(dv[j][i], mk, o[i]));      // D
                }
            }
        } else {
#pragma unroll
            for (int j = 0; j < C; ++j) in.d(j, dv[j]);
        }
#pragma unroll
        for (int j = 0; j < C; ++j) store_f2<VEC>(reinterpret_cast<G*>(b.dx) + at, in.c0(j), d, lane, dv[j]);
        if (a.y) {
            f2 q = 0ull;
#pragma unroll
            for (int j = 0; j < C; ++j) {
                f2 y[4], g[4], w[4];
                again(j, y, g);
                wt.get_post(a, in.c0(j), lane, w);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const f2 t = mul2(dv[j][i], g[i]);
                    accA[j][i] = fma2(t, y[i], accA[j][i]);
                    dv[j][i] = mul2(t, w[i]);                                 // u = D s sigma w_post
                    q = fma2(dv[j][i], y[i], q);
                }
            }
            float ss[1] = {sum2(q)};
            row_sum<1>(ss, red[buf][3], W, warp, lane);
            const f2 m = both(-ss[0] * inv_d * ry);
            if (a.gate_mode == MOM_GATE_TOKEN && b.dgate && threadIdx.x == 0)
                reinterpret_cast<T*>(b.dgate)[row] = from_f<T>(ss[0] * rest);
#pragma unroll
            for (int j = 0; j < C; ++j) {
                f2 y[4];
                if constexpr (C == 1) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) y[i] = yk[i];
                } else {
                    in.y(j, y);
#pragma unroll
                    for (int i = 0; i < 4; ++i) y[i] = mul2(y[i], both(ry));
                }
                if (a.gate_mode == MOM_GATE_ELEMENT && b.dgate) {
                    f2 z[4], o[4];
                    in.g(j, z);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float z0, z1, r0, r1;
                        split(z[i], z0, z1);
                        sigmoid(z0, r0);
                        sigmoid(z1, r1);
                        o[i] = mul2(mul2(dv[j][i], y[i]), make_f2(r0, r1));
                    }
                    store_f2<VEC>(reinterpret_cast<T*>(b.dgate) + at, in.c0(j), d, lane, o);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) dv[j][i] = fma2(dv[j][i], both(ry), mul2(y[i], m));
                store_f2<VEC>(reinterpret_cast<T*>(b.dy) + at, in.c0(j), d, lane, dv[j]);
            }
        }
    }
    float* pa = b.partial + (int64_t)blockIdx.x * 2 * d;
#pragma unroll
    for (int j = 0; j < C; ++j) {
        store_f2<VEC>(pa, in.c0(j), d, lane, accA[j]);
        store_f2<VEC>(pa + d, in.c0(j), d, lane, accP[j]);
    }
}

// Column sums of the CTAs' partials: a CTA sums 32 channels of one of the two
// (blockIdx.y), its 32 warps a strided part of the partials each, joined in
// warp order.
__global__ void __launch_bounds__(1024) cols_reduce_kernel(const float* partial, int n_part, int d, const float* w_post,
                                                           const float* res_scale, float* dw_post, float* dres_scale,
                                                           float* dw_pre) {
    __shared__ float sh[32][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane, which = blockIdx.y;
    float v = 0.f;
    asm volatile("griddepcontrol.wait;" ::: "memory");      // launched as the adjoint's CTAs leave
    if (c < d) {
        const float* at = partial + (int64_t)which * d + c;
#pragma unroll 8
        for (int p = warp; p < n_part; p += 32) v += at[(int64_t)p * 2 * d];
    }
    sh[warp][lane] = v;
    __syncthreads();
    if (warp != 0 || c >= d) return;
#pragma unroll
    for (int w = 1; w < 32; ++w) v += sh[w][lane];
    if (which) {
        if (dw_pre) dw_pre[c] = v;
    } else {
        if (dw_post) dw_post[c] = res_scale ? v * res_scale[c] : v;
        if (dres_scale) dres_scale[c] = v * w_post[c];
    }
}

int sm_count() {
    int dev = 0, sms = 148;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    return sms;
}

// Chunks a warp and warps of a row.
struct Shape {
    int C, warps;
};
Shape shape_for(int d) {
    const int chunks = (int)cdiv(d, kChunk), C = chunks <= 16 ? 1 : chunks <= 32 ? 2 : 4;
    return {C, (int)cdiv(chunks, C)};
}

// Warps an SM that the registers leave (__launch_bounds__): without a block's
// output the ring needs 64 with up to 8 warps a row, everything else 128.  (24
// warps with a block's output, 80 registers, spill: 37 us instead of 35 for
// 16384 x 1024.)
constexpr int kShortWarps = 32, kWarps = 16;
constexpr int kSmemSM = 220 * 1024;

template <typename XT, typename T, bool VEC, int C, bool HAS_Y, int MAXT>
cudaError_t run_fwd(ResNormArgs a, cudaStream_t st) {
    constexpr int SRC = C <= 2 && VEC ? RING : C == 1 ? REGS : DIRECT;
    auto* kernel = residual_norm_kernel<XT, T, VEC, C, HAS_Y, SRC, MAXT>;
    const int W = shape_for(a.d).warps, threads = W == 1 ? 128 : 32 * W;
    a.warps_per_row = W;
    const int ctas = (SRC == RING && !HAS_Y && MAXT <= 256 ? kShortWarps : kWarps) / (threads / 32);
    size_t smem = 0;
    if (SRC == RING) {
        typedef Rows<XT, T, T, VEC, C, HAS_Y, false, SRC> R;
        // at most 16 warps x 12 pieces x 2 slots, or 32 x 2 x 5: 192 KB an SM
        smem = (size_t)R::SLOTS * R::pieces(a) * C * threads * 16;
        static unsigned long long optin_done = 0;
        const cudaError_t e = smem_optin((const void*)kernel, kSmemSM, &optin_done);
        if (e != cudaSuccess) return e;
    }
    const int64_t units = W == 1 ? cdiv(a.n_rows, threads / 32) : a.n_rows, most = (int64_t)sm_count() * ctas;
    kernel<<<(unsigned)(units < most ? units : most), threads, smem, st>>>(a);
    return cudaGetLastError();
}

template <typename XT, typename T, typename G, bool VEC, int C, int MAXT>
cudaError_t run_bwd(ResNormArgs a, const ResNormBwdArgs& b, int parts, cudaStream_t st) {
    constexpr int SRC = C > 1 || !VEC ? DIRECT : REGS;
    a.warps_per_row = shape_for(a.d).warps;
    residual_norm_bwd_kernel<XT, T, G, VEC, C, SRC, MAXT><<<parts, 32 * a.warps_per_row, 0, st>>>(a, b);
    return cudaGetLastError();
}

template <typename XT, typename T, bool VEC, bool HAS_Y> cudaError_t shape_fwd(const ResNormArgs& a, cudaStream_t st) {
    const Shape s = shape_for(a.d);
    if (s.C == 1) return s.warps <= 8 ? run_fwd<XT, T, VEC, 1, HAS_Y, 256>(a, st) : run_fwd<XT, T, VEC, 1, HAS_Y, 512>(a, st);
    return s.C == 2 ? run_fwd<XT, T, VEC, 2, HAS_Y, 512>(a, st) : run_fwd<XT, T, VEC, 4, HAS_Y, 512>(a, st);
}
template <typename XT, typename T, bool VEC> cudaError_t pick_fwd(const ResNormArgs& a, cudaStream_t st) {
    return a.y ? shape_fwd<XT, T, VEC, true>(a, st) : shape_fwd<XT, T, VEC, false>(a, st);
}
template <typename XT, typename T, typename G, bool VEC>
cudaError_t pick_bwd(const ResNormArgs& a, const ResNormBwdArgs& b, int parts, cudaStream_t st) {
    const Shape s = shape_for(a.d);
    if (s.C == 1) return s.warps <= 8 ? run_bwd<XT, T, G, VEC, 1, 256>(a, b, parts, st) : run_bwd<XT, T, G, VEC, 1, 512>(a, b, parts, st);
    return s.C == 2 ? run_bwd<XT, T, G, VEC, 2, 512>(a, b, parts, st) : run_bwd<XT, T, G, VEC, 4, 512>(a, b, parts, st);
}

}  // namespace

// rows of partial column sums the adjoint writes
int residual_norm_bwd_parts(int64_t n_rows, int d) {
    const int64_t most = (int64_t)sm_count() * (kWarps / shape_for(d).warps);
    return (int)(n_rows < most ? n_rows : most);
}

cudaError_t launch_residual_norm(const ResNormArgs& a, int x_kind, int dt, bool vec, cudaStream_t st) {
    cudaError_t e;
#define MOM_RN(XT, T) e = vec ? pick_fwd<XT, T, true>(a, st) : pick_fwd<XT, T, false>(a, st)
    if (x_kind == RN_X_BF16) MOM_RN(bf16, bf16);
    else if (x_kind == RN_X_F32) { if (dt == MOM_BF16) MOM_RN(float, bf16); else MOM_RN(float, float); }
    else { if (dt == MOM_BF16) MOM_RN(Q8, bf16); else MOM_RN(Q8, float); }
#undef MOM_RN
    count_launches(1);
    return e;
}

cudaError_t launch_residual_norm_bwd(const ResNormArgs& a, const ResNormBwdArgs& b, int x_kind, int dt, int g_dt,
                                     bool vec, cudaStream_t st) {
    const int parts = residual_norm_bwd_parts(a.n_rows, a.d);
    if (parts > 0) {
        cudaError_t e;
#define MOM_RNB(XT, T, G) e = vec ? pick_bwd<XT, T, G, true>(a, b, parts, st) : pick_bwd<XT, T, G, false>(a, b, parts, st)
#define MOM_RNG(XT, T) do { if (g_dt == MOM_BF16) { MOM_RNB(XT, T, bf16); } else { MOM_RNB(XT, T, float); } } while (0)
        if (x_kind == RN_X_BF16) MOM_RNG(bf16, bf16);
        else if (x_kind == RN_X_F32) { if (dt == MOM_BF16) MOM_RNG(float, bf16); else MOM_RNG(float, float); }
        else { if (dt == MOM_BF16) MOM_RNG(Q8, bf16); else MOM_RNG(Q8, float); }
#undef MOM_RNG
#undef MOM_RNB
        count_launches(1);
        if (e != cudaSuccess) return e;
    }
    if (b.dw_post || b.dres_scale || b.dw_pre) {
        cudaLaunchAttribute at;
        at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
        at.val.programmaticStreamSerializationAllowed = 1;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)cdiv(a.d, 32), 2);
        cfg.blockDim = dim3(1024);
        cfg.stream = st;
        cfg.attrs = &at;
        cfg.numAttrs = parts > 0 ? 1 : 0;
        count_launches(1);
        return cudaLaunchKernelEx(&cfg, cols_reduce_kernel, (const float*)b.partial, parts, a.d, a.w_post, a.res_scale,
                                  b.dw_post, b.dres_scale, b.dw_pre);
    }
    return cudaSuccess;
}

}  // namespace mom
