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
// Bound by memory.  A row lives in the registers of W warps (C chunks of 256
// channels each), every operand is read once and all of a row's loads are
// issued before its first reduction.  Sums, norms and the whole arithmetic
// are float32; each output is rounded once, as it is stored.
#include <type_traits>

#include "rows8.cuh"
#include "kernels.h"

namespace mom {
namespace {

template <typename XT, bool VEC> struct RawX {
    Raw8<XT, VEC> r;
    __device__ __forceinline__ void load(const ResNormArgs& a, int64_t row, int c0, int lane) {
        r.load(reinterpret_cast<const XT*>(a.x) + row * a.d, c0, a.d, lane);
    }
    __device__ __forceinline__ void get(float* out) const { r.get(out); }
};
template <bool VEC> struct RawX<Q8, VEC> {
    Raw8Q<VEC> r;
    __device__ __forceinline__ void load(const ResNormArgs& a, int64_t row, int c0, int lane) {
        r.load(a.x_codes + row * a.d, a.x_scales + row * a.groups, c0, a.d, lane);
    }
    __device__ __forceinline__ void get(float* out) const { r.get(out); }
};

// sigma(z): the hardware exponential and reciprocal, below 2^-21 relative for
// |z| < 8 (2^-18 at |z| = 60, where sigma or 1 - sigma is 1e-26); a correctly
// rounded division cost 15 of the 50 instructions an element took.
__device__ __forceinline__ float fast_sigmoid(float z) { return __fdividef(1.f, 1.f + __expf(-z)); }

// Sums of K values over the W = blockDim / 32 warps of a row (every thread
// gets them); one warp a row needs no barrier.  `buf` alternates so that one
// barrier is enough.
template <int K> __device__ __forceinline__ void row_sum(float (&v)[K], float* buf, int W, int warp, int lane) {
    warp_sum_n<K>(v);
    if (W > 1) {
        if (lane == 0)
#pragma unroll
            for (int k = 0; k < K; ++k) buf[warp * K + k] = v[k];
        __syncthreads();
#pragma unroll
        for (int k = 0; k < K; ++k) v[k] = 0.f;
        for (int w = 0; w < W; ++w)
#pragma unroll
            for (int k = 0; k < K; ++k) v[k] += buf[w * K + k];
    }
}

constexpr int kMaxWarps = 16;

// W > 1: a CTA of W warps holds one row.  W == 1: each warp holds its own.
template <typename XT, typename T, bool VEC, int C, int MAXW>
__global__ void __launch_bounds__(32 * MAXW) residual_norm_kernel(const ResNormArgs a) {
    __shared__ float red[2][kMaxWarps];
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, nw = blockDim.x >> 5;
    const int W = a.warps_per_row, warp = W > 1 ? wid : 0;
    const int64_t row = W > 1 ? (int64_t)blockIdx.x : (int64_t)blockIdx.x * nw + wid;
    if (row >= a.n_rows) return;      // whole CTAs (W > 1) or whole warps (W == 1)
    const int d = a.d;
    const float inv_d = 1.f / (float)d;
    RawX<XT, VEC> xr[C];
    float xv[C][8];
    if (a.y) {
        Raw8<T, VEC> yr[C], gr[C];
#pragma unroll
        for (int j = 0; j < C; ++j)
            yr[j].load(reinterpret_cast<const T*>(a.y) + row * d, (warp + j * W) * kChunk, d, lane);
#pragma unroll
        for (int j = 0; j < C; ++j) xr[j].load(a, row, (warp + j * W) * kChunk, lane);
        if (a.gate_mode == MOM_GATE_ELEMENT) {
#pragma unroll
            for (int j = 0; j < C; ++j)
                gr[j].load(reinterpret_cast<const T*>(a.gate) + row * d, (warp + j * W) * kChunk, d, lane);
        }
        float gt = 1.f;
        if (a.gate_mode == MOM_GATE_TOKEN) gt = fast_sigmoid(to_f(reinterpret_cast<const T*>(a.gate)[row]));
        float ss[1] = {0.f};
#pragma unroll
        for (int j = 0; j < C; ++j) {
            float y[8];
            yr[j].get(y);
#pragma unroll
            for (int i = 0; i < 8; ++i) ss[0] = fmaf(y[i], y[i], ss[0]);
        }
        row_sum<1>(ss, red[0], W, warp, lane);
        const float ry = gt / sqrtf(ss[0] * inv_d + a.eps);      // 1 / rms(y), times a token's gate
#pragma unroll
        for (int j = 0; j < C; ++j) {
            const int c0 = (warp + j * W) * kChunk;
            float y[8], w[8];
            yr[j].get(y);
            xr[j].get(xv[j]);
            if (a.codes_out)
                act8_store<VEC>(xv[j], c0, d, lane, a.codes_out + row * d, a.scales_out + row * a.groups);
            load8<VEC>(a.w_post, c0, d, lane, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] *= y[i] * ry;
            if (a.gate_mode == MOM_GATE_ELEMENT) {
                gr[j].get(y);
#pragma unroll
                for (int i = 0; i < 8; ++i) w[i] *= fast_sigmoid(y[i]);
            }
            if (a.res_scale) {
                load8<VEC>(a.res_scale, c0, d, lane, y);
#pragma unroll
                for (int i = 0; i < 8; ++i) xv[j][i] = fmaf(w[i], y[i], xv[j][i]);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) xv[j][i] += w[i];
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < C; ++j) xr[j].load(a, row, (warp + j * W) * kChunk, lane);
#pragma unroll
        for (int j = 0; j < C; ++j) {
            xr[j].get(xv[j]);
            if (a.codes_out)
                act8_store<VEC>(xv[j], (warp + j * W) * kChunk, d, lane, a.codes_out + row * d,
                                a.scales_out + row * a.groups);
        }
    }
    if (a.x_out) {
#pragma unroll
        for (int j = 0; j < C; ++j) {
            const int c0 = (warp + j * W) * kChunk;
            if (a.x_out_f32) store8<VEC>(reinterpret_cast<float*>(a.x_out) + row * d, c0, d, lane, xv[j]);
            else store8<VEC>(reinterpret_cast<bf16*>(a.x_out) + row * d, c0, d, lane, xv[j]);
        }
    }
    if (a.h) {
        float ss[1] = {0.f};
#pragma unroll
        for (int j = 0; j < C; ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i) ss[0] = fmaf(xv[j][i], xv[j][i], ss[0]);
        row_sum<1>(ss, red[1], W, warp, lane);
        const float rx = 1.f / sqrtf(ss[0] * inv_d + a.eps);
#pragma unroll
        for (int j = 0; j < C; ++j) {
            const int c0 = (warp + j * W) * kChunk;
            float w[8];
            load8<VEC>(a.w_pre, c0, d, lane, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] *= xv[j][i] * rx;
            store8<VEC>(reinterpret_cast<T*>(a.h) + row * d, c0, d, lane, w);
        }
    }
}

// A row's operands of the adjoint, as they lie in memory.
template <typename XT, typename T, typename G, bool VEC, int C> struct BwdRow {
    RawX<XT, VEC> x[C];
    Raw8<T, VEC> y[C], g[C];
    Raw8<G, VEC> d[C], h[C];
    T gate;
    __device__ __forceinline__ void load(const ResNormArgs& a, const ResNormBwdArgs& b, int64_t row, int warp, int W,
                                         int lane) {
        if (row >= a.n_rows) return;
        const int n = a.d;
#pragma unroll
        for (int j = 0; j < C; ++j) {
            const int c0 = (warp + j * W) * kChunk;
            if (a.y) y[j].load(reinterpret_cast<const T*>(a.y) + row * n, c0, n, lane);
            x[j].load(a, row, c0, lane);
            if (a.gate_mode == MOM_GATE_ELEMENT) g[j].load(reinterpret_cast<const T*>(a.gate) + row * n, c0, n, lane);
            if (b.dh) h[j].load(reinterpret_cast<const G*>(b.dh) + row * n, c0, n, lane);
            if (b.dx_out) d[j].load(reinterpret_cast<const G*>(b.dx_out) + row * n, c0, n, lane);
        }
        if (a.gate_mode == MOM_GATE_TOKEN) gate = reinterpret_cast<const T*>(a.gate)[row];
    }
};

// The adjoint.  A CTA walks rows blockIdx.x, + gridDim.x, ..; the next row's
// operands are loaded (packed) before this row's arithmetic, so that loads are
// in flight through its three reductions.  Its threads keep the two column
// sums (A and dw_pre) of their channels in registers and write them once as
// the CTA's partial, which cols_reduce_kernel adds up in CTA order: no
// atomics, the same sums every time on the same device.
template <typename XT, typename T, typename G, bool VEC, int C, int MAXW>
__global__ void __launch_bounds__(32 * MAXW) residual_norm_bwd_kernel(const ResNormArgs a, const ResNormBwdArgs b) {
    __shared__ float red[3][2 * kMaxWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, W = blockDim.x >> 5;
    const int d = a.d;
    const float inv_d = 1.f / (float)d;
    float accA[C][8], accP[C][8];
#pragma unroll
    for (int j = 0; j < C; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) accA[j][i] = accP[j][i] = 0.f;
    BwdRow<XT, T, G, VEC, C> next;
    next.load(a, b, blockIdx.x, warp, W, lane);
    for (int64_t row = blockIdx.x; row < a.n_rows; row += gridDim.x) {
        const BwdRow<XT, T, G, VEC, C> r = next;
        next.load(a, b, row + gridDim.x, warp, W, lane);
        float xv[C][8], yv[C][8], gv[C][8], dv[C][8], hv[C][8];
        float gt = 1.f;
        if (a.gate_mode == MOM_GATE_TOKEN) gt = fast_sigmoid(to_f(r.gate));
        float ry = 0.f;
        if (a.y) {
            float ss[1] = {0.f};
#pragma unroll
            for (int j = 0; j < C; ++j) {
                r.y[j].get(yv[j]);
#pragma unroll
                for (int i = 0; i < 8; ++i) ss[0] = fmaf(yv[j][i], yv[j][i], ss[0]);
            }
            row_sum<1>(ss, red[0], W, warp, lane);
            ry = 1.f / sqrtf(ss[0] * inv_d + a.eps);
#pragma unroll
            for (int j = 0; j < C; ++j) {
                if (a.gate_mode == MOM_GATE_ELEMENT) r.g[j].get(gv[j]);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    yv[j][i] *= ry;                                       // n_y
                    gv[j][i] = a.gate_mode == MOM_GATE_ELEMENT ? fast_sigmoid(gv[j][i]) : gt;
                }
            }
        }
#pragma unroll
        for (int j = 0; j < C; ++j) {
            if (b.dx_out) {
                r.d[j].get(dv[j]);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) dv[j][i] = 0.f;
            }
        }
        if (b.dh) {
            float ss[2] = {0.f, 0.f};
#pragma unroll
            for (int j = 0; j < C; ++j) {
                const int c0 = (warp + j * W) * kChunk;
                float w[8];
                r.x[j].get(xv[j]);
                r.h[j].get(hv[j]);
                if (a.y) {
                    load8<VEC>(a.w_post, c0, d, lane, w);
                    if (a.res_scale) {
                        float s[8];
                        load8<VEC>(a.res_scale, c0, d, lane, s);
#pragma unroll
                        for (int i = 0; i < 8; ++i) w[i] *= s[i];
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i) xv[j][i] = fmaf(yv[j][i] * gv[j][i], w[i], xv[j][i]);   // x'
                }
                load8<VEC>(a.w_pre, c0, d, lane, w);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    ss[0] = fmaf(xv[j][i], xv[j][i], ss[0]);
                    ss[1] = fmaf(xv[j][i], hv[j][i] * w[i], ss[1]);
                }
            }
            row_sum<2>(ss, red[1], W, warp, lane);
            const float rx = 1.f / sqrtf(ss[0] * inv_d + a.eps);
            const float k = ss[1] * inv_d * rx * rx;                      // mean(dn n_x) / rms
#pragma unroll
            for (int j = 0; j < C; ++j) {
                float w[8];
                load8<VEC>(a.w_pre, (warp + j * W) * kChunk, d, lane, w);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    accP[j][i] = fmaf(hv[j][i], xv[j][i] * rx, accP[j][i]);
                    dv[j][i] = fmaf(fmaf(hv[j][i], w[i], -xv[j][i] * k), rx, dv[j][i]);
                }
            }
        }
#pragma unroll
        for (int j = 0; j < C; ++j)
            store8<VEC>(reinterpret_cast<G*>(b.dx) + row * d, (warp + j * W) * kChunk, d, lane, dv[j]);
        if (a.y) {
            float ss[1] = {0.f};
#pragma unroll
            for (int j = 0; j < C; ++j) {
                const int c0 = (warp + j * W) * kChunk;
                float w[8];
                load8<VEC>(a.w_post, c0, d, lane, w);
                if (a.res_scale) {
                    float s[8];
                    load8<VEC>(a.res_scale, c0, d, lane, s);
#pragma unroll
                    for (int i = 0; i < 8; ++i) w[i] *= s[i];
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float t = dv[j][i] * gv[j][i];
                    accA[j][i] = fmaf(t, yv[j][i], accA[j][i]);
                    dv[j][i] = t * w[i];                                  // u = D s sigma w_post
                    ss[0] = fmaf(dv[j][i], yv[j][i], ss[0]);
                }
            }
            row_sum<1>(ss, red[2], W, warp, lane);
            const float m = ss[0] * inv_d;
            if (a.gate_mode == MOM_GATE_TOKEN && b.dgate && threadIdx.x == 0)
                reinterpret_cast<T*>(b.dgate)[row] = from_f<T>(ss[0] * (1.f - gt));
#pragma unroll
            for (int j = 0; j < C; ++j) {
                const int c0 = (warp + j * W) * kChunk;
                float o[8];
                if (a.gate_mode == MOM_GATE_ELEMENT && b.dgate) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) o[i] = dv[j][i] * yv[j][i] * (1.f - gv[j][i]);
                    store8<VEC>(reinterpret_cast<T*>(b.dgate) + row * d, c0, d, lane, o);
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) o[i] = (dv[j][i] - yv[j][i] * m) * ry;
                store8<VEC>(reinterpret_cast<T*>(b.dy) + row * d, c0, d, lane, o);
            }
        }
        // the next row's sums reuse `red`
        if (W > 1) __syncthreads();
    }
    float* pa = b.partial + (int64_t)blockIdx.x * 2 * d;
#pragma unroll
    for (int j = 0; j < C; ++j) {
        const int c0 = (warp + j * W) * kChunk;
        store8<VEC>(pa, c0, d, lane, accA[j]);
        store8<VEC>(pa + d, c0, d, lane, accP[j]);
    }
}

// Column sums of the CTAs' partials: a CTA sums 32 channels, its 8 warps a
// strided eighth of the partials each, joined in warp order.
__global__ void __launch_bounds__(256) cols_reduce_kernel(const float* partial, int n_part, int d, const float* w_post,
                                                          const float* res_scale, float* dw_post, float* dres_scale,
                                                          float* dw_pre) {
    __shared__ float sA[8][32], sP[8][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    float A = 0.f, P = 0.f;
    if (c < d) {
#pragma unroll 4
        for (int p = warp; p < n_part; p += 8) {
            A += partial[(int64_t)p * 2 * d + c];
            P += partial[(int64_t)p * 2 * d + d + c];
        }
    }
    sA[warp][lane] = A;
    sP[warp][lane] = P;
    __syncthreads();
    if (warp == 0 && c < d) {
#pragma unroll
        for (int w = 1; w < 8; ++w) { A += sA[w][lane]; P += sP[w][lane]; }
        if (dw_post) dw_post[c] = res_scale ? A * res_scale[c] : A;
        if (dres_scale) dres_scale[c] = A * w_post[c];
        if (dw_pre) dw_pre[c] = P;
    }
}

int sm_count() {
    int dev = 0, sms = 148;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    return sms;
}

// Chunks of 256 channels a warp holds.  Forward: two up to 4096 channels (16384
// rows of 1024, bf16, an element gate: 44 us; one 49 us, four 47 us), four
// above, so that a row stays within 16 warps.  Adjoint, which holds five
// operands and two column sums: one up to 2048 channels (104 us; two 122 us),
// 16 warps an SM (32: 124 us, by spilling its registers).
constexpr int kFwdC = 2, kBwdC = 1, kBwdWarps = 16;
template <typename XT, typename T, bool VEC>
void run_fwd(ResNormArgs a, cudaStream_t st) {
    const int chunks = (int)cdiv(a.d, kChunk);
    const int C = chunks <= 1 ? 1 : chunks <= 8 * kFwdC ? kFwdC : 4;
    const int W = (int)cdiv(chunks, C);
    a.warps_per_row = W;
    const int threads = W > 1 ? 32 * W : 128;
    const int64_t grid = W > 1 ? a.n_rows : cdiv(a.n_rows, threads / 32);
    if (C == 1) residual_norm_kernel<XT, T, VEC, 1, 8><<<(unsigned)grid, threads, 0, st>>>(a);
    else if (C == kFwdC) residual_norm_kernel<XT, T, VEC, kFwdC, 8><<<(unsigned)grid, threads, 0, st>>>(a);
    else residual_norm_kernel<XT, T, VEC, 4, 16><<<(unsigned)grid, threads, 0, st>>>(a);
}

template <typename XT, typename T, typename G, bool VEC>
void run_bwd(const ResNormArgs& a, const ResNormBwdArgs& b, int grid, cudaStream_t st) {
    const int chunks = (int)cdiv(a.d, kChunk);
    const int C = chunks <= 8 * kBwdC ? kBwdC : chunks <= 16 ? 2 : 4;
    const int threads = 32 * (int)cdiv(chunks, C);
    if (C == kBwdC) residual_norm_bwd_kernel<XT, T, G, VEC, kBwdC, 8><<<grid, threads, 0, st>>>(a, b);
    else if (C == 2) residual_norm_bwd_kernel<XT, T, G, VEC, 2, 8><<<grid, threads, 0, st>>>(a, b);
    else residual_norm_bwd_kernel<XT, T, G, VEC, 4, 16><<<grid, threads, 0, st>>>(a, b);
}

}  // namespace

// rows of partial column sums the adjoint writes
int residual_norm_bwd_parts(int64_t n_rows, int d) {
    const int chunks = (int)cdiv(d, kChunk);
    const int warps = (int)cdiv(chunks, chunks <= 8 * kBwdC ? kBwdC : chunks <= 16 ? 2 : 4);
    const int64_t most = (int64_t)sm_count() * (warps <= kBwdWarps ? kBwdWarps / warps : 1);
    return (int)(n_rows < most ? n_rows : most);
}

cudaError_t launch_residual_norm(const ResNormArgs& a, int x_kind, int dt, bool vec, cudaStream_t st) {
#define MOM_RN(XT, T) do { if (vec) run_fwd<XT, T, true>(a, st); else run_fwd<XT, T, false>(a, st); } while (0)
    if (x_kind == RN_X_BF16) MOM_RN(bf16, bf16);
    else if (x_kind == RN_X_F32) { if (dt == MOM_BF16) MOM_RN(float, bf16); else MOM_RN(float, float); }
    else { if (dt == MOM_BF16) MOM_RN(Q8, bf16); else MOM_RN(Q8, float); }
#undef MOM_RN
    count_launches(1);
    return cudaGetLastError();
}

cudaError_t launch_residual_norm_bwd(const ResNormArgs& a, const ResNormBwdArgs& b, int x_kind, int dt, int g_dt,
                                     bool vec, cudaStream_t st) {
    const int parts = residual_norm_bwd_parts(a.n_rows, a.d);
    if (parts > 0) {
#define MOM_RNB(XT, T, G) do { if (vec) run_bwd<XT, T, G, true>(a, b, parts, st); else run_bwd<XT, T, G, false>(a, b, parts, st); } while (0)
#define MOM_RNG(XT, T) do { if (g_dt == MOM_BF16) MOM_RNB(XT, T, bf16); else MOM_RNB(XT, T, float); } while (0)
        if (x_kind == RN_X_BF16) MOM_RNG(bf16, bf16);
        else if (x_kind == RN_X_F32) { if (dt == MOM_BF16) MOM_RNG(float, bf16); else MOM_RNG(float, float); }
        else { if (dt == MOM_BF16) MOM_RNG(Q8, bf16); else MOM_RNG(Q8, float); }
#undef MOM_RNG
#undef MOM_RNB
        count_launches(1);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    if (b.dw_post || b.dres_scale || b.dw_pre) {
        cols_reduce_kernel<<<(unsigned)cdiv(a.d, 32), 256, 0, st>>>(b.partial, parts, a.d, a.w_post, a.res_scale,
                                                                    b.dw_post, b.dres_scale, b.dw_pre);
        count_launches(1);
    }
    return cudaGetLastError();
}

}  // namespace mom
