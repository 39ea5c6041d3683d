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

struct Q8 {};      // tag: the stream comes from an 8-bit checkpoint

template <typename XT, bool VEC>
__device__ __forceinline__ void load_x(const ResNormArgs& a, int64_t row, int c0, int lane, float* out) {
    if constexpr (std::is_same<XT, Q8>::value)
        act8_load<VEC>(a.x_codes + row * a.d, a.x_scales + row * a.groups, c0, a.d, lane, out);
    else
        load8<VEC>(reinterpret_cast<const XT*>(a.x) + row * a.d, c0, a.d, lane, out);
}

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
template <typename XT, typename T, bool VEC, int C>
__global__ void __launch_bounds__(32 * kMaxWarps) residual_norm_kernel(const ResNormArgs a) {
    __shared__ float red[2][kMaxWarps];
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, nw = blockDim.x >> 5;
    const int W = a.warps_per_row, warp = W > 1 ? wid : 0;
    const int64_t row = W > 1 ? (int64_t)blockIdx.x : (int64_t)blockIdx.x * nw + wid;
    if (row >= a.n_rows) return;      // whole CTAs (W > 1) or whole warps (W == 1)
    const int d = a.d;
    const float inv_d = 1.f / (float)d;
    float xv[C][8], yv[C][8], gv[C][8];
#pragma unroll
    for (int j = 0; j < C; ++j) load_x<XT, VEC>(a, row, (warp + j * W) * kChunk, lane, xv[j]);
    if (a.y) {
        const T* y = reinterpret_cast<const T*>(a.y) + row * d;
#pragma unroll
        for (int j = 0; j < C; ++j) load8<VEC>(y, (warp + j * W) * kChunk, d, lane, yv[j]);
        if (a.gate_mode == MOM_GATE_ELEMENT) {
            const T* g = reinterpret_cast<const T*>(a.gate) + row * d;
#pragma unroll
            for (int j = 0; j < C; ++j) load8<VEC>(g, (warp + j * W) * kChunk, d, lane, gv[j]);
        }
        const float gt = a.gate_mode == MOM_GATE_TOKEN ? sigmoidf_(to_f(reinterpret_cast<const T*>(a.gate)[row])) : 1.f;
        if (a.codes_out) {
#pragma unroll
            for (int j = 0; j < C; ++j)
                act8_store<VEC>(xv[j], (warp + j * W) * kChunk, d, lane, a.codes_out + row * d,
                                a.scales_out + row * a.groups);
        }
        float ss[1] = {0.f};
#pragma unroll
        for (int j = 0; j < C; ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i) ss[0] = fmaf(yv[j][i], yv[j][i], ss[0]);
        row_sum<1>(ss, red[0], W, warp, lane);
        const float ry = 1.f / sqrtf(ss[0] * inv_d + a.eps);
#pragma unroll
        for (int j = 0; j < C; ++j) {
            const int c0 = (warp + j * W) * kChunk;
            float w[8], s[8];
            load8<VEC>(a.w_post, c0, d, lane, w);
            if (a.res_scale) load8<VEC>(a.res_scale, c0, d, lane, s);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float u = yv[j][i] * ry * w[i];
                u *= a.gate_mode == MOM_GATE_ELEMENT ? sigmoidf_(gv[j][i]) : gt;
                if (a.res_scale) u *= s[i];
                xv[j][i] += u;
            }
        }
    } else if (a.codes_out) {
#pragma unroll
        for (int j = 0; j < C; ++j)
            act8_store<VEC>(xv[j], (warp + j * W) * kChunk, d, lane, a.codes_out + row * d,
                            a.scales_out + row * a.groups);
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

// The adjoint.  A CTA walks rows blockIdx.x, + gridDim.x, ..; its threads keep
// the two column sums (A and dw_pre) of their channels in registers and write
// them once as the CTA's partial, which cols_reduce_kernel adds up in CTA
// order: no atomics, the same sums every time on the same device.
template <typename XT, typename T, typename G, bool VEC, int C>
__global__ void __launch_bounds__(32 * kMaxWarps) residual_norm_bwd_kernel(const ResNormArgs a, const ResNormBwdArgs b) {
    __shared__ float red[3][2 * kMaxWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, W = blockDim.x >> 5;
    const int d = a.d;
    const float inv_d = 1.f / (float)d;
    float accA[C][8], accP[C][8];
#pragma unroll
    for (int j = 0; j < C; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) accA[j][i] = accP[j][i] = 0.f;
    for (int64_t row = blockIdx.x; row < a.n_rows; row += gridDim.x) {
        float xv[C][8], yv[C][8], gv[C][8], dv[C][8], hv[C][8];
#pragma unroll
        for (int j = 0; j < C; ++j) {
            const int c0 = (warp + j * W) * kChunk;
            load_x<XT, VEC>(a, row, c0, lane, xv[j]);
            if (a.y) load8<VEC>(reinterpret_cast<const T*>(a.y) + row * d, c0, d, lane, yv[j]);
            if (a.gate_mode == MOM_GATE_ELEMENT)
                load8<VEC>(reinterpret_cast<const T*>(a.gate) + row * d, c0, d, lane, gv[j]);
            if (b.dx_out) {
                load8<VEC>(reinterpret_cast<const G*>(b.dx_out) + row * d, c0, d, lane, dv[j]);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) dv[j][i] = 0.f;
            }
            if (b.dh) load8<VEC>(reinterpret_cast<const G*>(b.dh) + row * d, c0, d, lane, hv[j]);
        }
        const float gt = a.gate_mode == MOM_GATE_TOKEN ? sigmoidf_(to_f(reinterpret_cast<const T*>(a.gate)[row])) : 1.f;
        float ry = 0.f;
        if (a.y) {
            float ss[1] = {0.f};
#pragma unroll
            for (int j = 0; j < C; ++j)
#pragma unroll
                for (int i = 0; i < 8; ++i) ss[0] = fmaf(yv[j][i], yv[j][i], ss[0]);
            row_sum<1>(ss, red[0], W, warp, lane);
            ry = 1.f / sqrtf(ss[0] * inv_d + a.eps);
#pragma unroll
            for (int j = 0; j < C; ++j)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    yv[j][i] *= ry;                                       // n_y
                    gv[j][i] = a.gate_mode == MOM_GATE_ELEMENT ? sigmoidf_(gv[j][i]) : gt;
                }
        }
        if (b.dh) {
            float ss[2] = {0.f, 0.f};
            float dn[C][8];
#pragma unroll
            for (int j = 0; j < C; ++j) {
                const int c0 = (warp + j * W) * kChunk;
                float w[8];
                if (a.y) {
                    float s[8];
                    load8<VEC>(a.w_post, c0, d, lane, w);
                    if (a.res_scale) load8<VEC>(a.res_scale, c0, d, lane, s);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float coef = a.res_scale ? w[i] * s[i] : w[i];
                        xv[j][i] = fmaf(yv[j][i] * gv[j][i], coef, xv[j][i]);   // x'
                    }
                }
                load8<VEC>(a.w_pre, c0, d, lane, w);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    dn[j][i] = hv[j][i] * w[i];
                    ss[0] = fmaf(xv[j][i], xv[j][i], ss[0]);
                    ss[1] = fmaf(xv[j][i], dn[j][i], ss[1]);
                }
            }
            row_sum<2>(ss, red[1], W, warp, lane);
            const float rx = 1.f / sqrtf(ss[0] * inv_d + a.eps);
            const float k = ss[1] * inv_d * rx * rx * rx;                 // mean(dn n_x) / rms^2
#pragma unroll
            for (int j = 0; j < C; ++j)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    accP[j][i] = fmaf(hv[j][i], xv[j][i] * rx, accP[j][i]);
                    dv[j][i] += dn[j][i] * rx - xv[j][i] * k;
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
                float w[8], s[8];
                load8<VEC>(a.w_post, c0, d, lane, w);
                if (a.res_scale) load8<VEC>(a.res_scale, c0, d, lane, s);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float coef = a.res_scale ? w[i] * s[i] : w[i];
                    accA[j][i] = fmaf(dv[j][i] * gv[j][i], yv[j][i], accA[j][i]);
                    dv[j][i] *= coef;                                     // D s w_post
                    ss[0] = fmaf(dv[j][i] * gv[j][i], yv[j][i], ss[0]);
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
                    for (int i = 0; i < 8; ++i) o[i] = dv[j][i] * yv[j][i] * gv[j][i] * (1.f - gv[j][i]);
                    store8<VEC>(reinterpret_cast<T*>(b.dgate) + row * d, c0, d, lane, o);
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) o[i] = (dv[j][i] * gv[j][i] - yv[j][i] * m) * ry;
                store8<VEC>(reinterpret_cast<T*>(b.dy) + row * d, c0, d, lane, o);
            }
        }
        // the next row's sums reuse `red`: with three buffers a warp can be at
        // most one row_sum ahead of the slowest reader of the buffer it writes
        if (W > 1) __syncthreads();
    }
    float* pa = b.partial + (int64_t)blockIdx.x * 2 * d;
#pragma unroll
    for (int j = 0; j < C; ++j) {
        const int c0 = (warp + j * W) * kChunk;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int c = c0 + chunk_col<VEC>(lane, i);
            if (c < d) {
                pa[c] = accA[j][i];
                pa[d + c] = accP[j][i];
            }
        }
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

template <typename XT, typename T, bool VEC>
void run_fwd(ResNormArgs a, cudaStream_t st) {
    const int chunks = (int)cdiv(a.d, kChunk);
    const int C = chunks <= 1 ? 1 : chunks <= 2 ? 2 : 4;
    const int W = (int)cdiv(chunks, C);
    a.warps_per_row = W;
    const int threads = W > 1 ? 32 * W : 128;
    const int64_t grid = W > 1 ? a.n_rows : cdiv(a.n_rows, threads / 32);
    if (C == 1) residual_norm_kernel<XT, T, VEC, 1><<<(unsigned)grid, threads, 0, st>>>(a);
    else if (C == 2) residual_norm_kernel<XT, T, VEC, 2><<<(unsigned)grid, threads, 0, st>>>(a);
    else residual_norm_kernel<XT, T, VEC, 4><<<(unsigned)grid, threads, 0, st>>>(a);
}

template <typename XT, typename T, typename G, bool VEC>
void run_bwd(const ResNormArgs& a, const ResNormBwdArgs& b, int grid, cudaStream_t st) {
    const int chunks = (int)cdiv(a.d, kChunk);
    const int C = chunks <= 16 ? 1 : chunks <= 32 ? 2 : 4;
    const int threads = 32 * (int)cdiv(chunks, C);
    if (C == 1) residual_norm_bwd_kernel<XT, T, G, VEC, 1><<<grid, threads, 0, st>>>(a, b);
    else if (C == 2) residual_norm_bwd_kernel<XT, T, G, VEC, 2><<<grid, threads, 0, st>>>(a, b);
    else residual_norm_bwd_kernel<XT, T, G, VEC, 4><<<grid, threads, 0, st>>>(a, b);
}

}  // namespace

// rows of partial column sums the adjoint writes
int residual_norm_bwd_parts(int64_t n_rows, int d) {
    const int warps = (int)cdiv(cdiv(d, kChunk), d <= 4096 ? 1 : d <= 8192 ? 2 : 4);
    const int64_t most = (int64_t)sm_count() * (warps <= 4 ? 16 / warps : warps <= 8 ? 2 : 1);
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
