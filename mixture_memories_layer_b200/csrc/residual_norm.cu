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
    typedef Raw8<XT, VEC> R;
    R r;
    static __device__ __forceinline__ void copy(uint32_t slot, uint32_t pitch, const ResNormArgs& a, int64_t row, int c0, int lane) {
        R::copy(slot, pitch, reinterpret_cast<const XT*>(a.x) + row * a.d, c0, a.d, lane);
    }
    __device__ __forceinline__ void load(const ResNormArgs& a, int64_t row, int c0, int lane) {
        r.load(reinterpret_cast<const XT*>(a.x) + row * a.d, c0, a.d, lane);
    }
    __device__ __forceinline__ void get(float* out) const { r.get(out); }
};
template <bool VEC> struct RawX<Q8, VEC> {
    typedef Raw8Q<VEC> R;
    R r;
    static __device__ __forceinline__ void copy(uint32_t slot, uint32_t pitch, const ResNormArgs& a, int64_t row, int c0, int lane) {
        R::copy(slot, pitch, a.x_codes + row * a.d, a.x_scales + row * a.groups, c0, a.d, lane);
    }
    __device__ __forceinline__ void load(const ResNormArgs& a, int64_t row, int c0, int lane) {
        r.load(a.x_codes + row * a.d, a.x_scales + row * a.groups, c0, a.d, lane);
    }
    __device__ __forceinline__ void get(float* out) const { r.get(out); }
};

// sigma(z) = 1 / (1 + e), e = exp(-z), by the hardware exponential and
// reciprocal: below 2^-21 relative for |z| < 8 (2^-18 at |z| = 60, where sigma
// or 1 - sigma is 1e-26).  1 - sigma without cancellation: e sigma for z > 0.
__device__ __forceinline__ float sigmoid(float z, float& rest) {
    const float e = fast_ex2(z * -1.4426950408889634f), s = fast_rcp(1.f + e);
    rest = z > 0.f ? e * s : 1.f - s;
    return s;
}
__device__ __forceinline__ float sigmoid(float z) { return fast_rcp(1.f + fast_ex2(z * -1.4426950408889634f)); }

constexpr int kWarps = 8;        // warps of a row's CTA; wider rows take a cluster of CTAs
constexpr int kMaxCluster = 8;
static_assert(kMaxCluster * kWarps * kChunk >= MOM_NORM_MAX_D, "a cluster holds a row");

// Who holds what of a row: W warps a CTA with one chunk of 256 channels each,
// in `cl` CTAs.  One warp a row: every warp of the CTA has its own.
struct Place {
    int lane, W, warp, cl, rank, c0;
    __device__ __forceinline__ Place(const ResNormArgs& a) {
        lane = threadIdx.x & 31;
        W = a.warps_per_row;
        warp = W > 1 ? threadIdx.x >> 5 : 0;
        cl = a.cluster;
        asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
        c0 = (rank * W + warp) * kChunk;
    }
};
__device__ __forceinline__ void cluster_barrier() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Sums of K values over a row (every thread gets them), in warp order.  One
// warp a row needs no barrier; in a cluster each warp writes its sums to every
// CTA's shared memory and one cluster barrier takes the place of the CTA's.
template <int K> __device__ __forceinline__ void row_sum(float (&v)[K], float* buf, const Place& w) {
    warp_sum_n<K>(v);
    if (w.W * w.cl == 1) return;
    if (w.cl > 1) {
        if (w.lane < w.cl) {
            uint32_t at;
            asm("mapa.shared::cluster.u32 %0, %1, %2;"
                : "=r"(at) : "r"((uint32_t)__cvta_generic_to_shared(buf)), "r"(w.lane));
#pragma unroll
            for (int k = 0; k < K; ++k)
                asm volatile("st.shared::cluster.f32 [%0], %1;"
                             ::"r"(at + 4 * ((w.rank * w.W + w.warp) * K + k)), "f"(v[k]) : "memory");
        }
        cluster_barrier();
    } else {
        if (w.lane == 0)
#pragma unroll
            for (int k = 0; k < K; ++k) buf[w.warp * K + k] = v[k];
        __syncthreads();
    }
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = 0.f;
    for (int i = 0; i < w.W * w.cl; ++i)
#pragma unroll
        for (int k = 0; k < K; ++k) v[k] += buf[i * K + k];
}

// The column weights of a thread's channels, res_scale * w_post and w_pre, in
// registers for all of a CTA's rows.
template <bool VEC> struct Weights {
    float post[8], pre[8];
    __device__ __forceinline__ Weights(const ResNormArgs& a, bool has_pre, const Place& w) {
#pragma unroll
        for (int i = 0; i < 8; ++i) post[i] = pre[i] = 0.f;
        if (a.y) load8<VEC>(a.w_post, w.c0, a.d, w.lane, post);
        if (a.y && a.res_scale) {
            float s[8];
            load8<VEC>(a.res_scale, w.c0, a.d, w.lane, s);
#pragma unroll
            for (int i = 0; i < 8; ++i) post[i] *= s[i];
        }
        if (has_pre) load8<VEC>(a.w_pre, w.c0, a.d, w.lane, pre);
    }
};

// A row's operands of the forward, as they lie in memory.
template <typename XT, typename T, bool VEC, bool HAS_Y> struct FwdRow {
    RawX<XT, VEC> x;
    Raw8<T, VEC> y, g;
    __device__ __forceinline__ void load(const ResNormArgs& a, int64_t row, const Place& w) {
        if (row >= a.n_rows) return;
        if (HAS_Y) y.load(reinterpret_cast<const T*>(a.y) + row * a.d, w.c0, a.d, w.lane);
        x.load(a, row, w.c0, w.lane);
        if (HAS_Y && a.gate_mode == MOM_GATE_ELEMENT)
            g.load(reinterpret_cast<const T*>(a.gate) + row * a.d, w.c0, a.d, w.lane);
    }
};

// Rows of the forward ahead of the one at work: copies in flight to a ring of
// slots in shared memory, of which each thread reads only what it copied (no
// barrier).  A slot is filled again one row after it was read.  Without a
// block's output a row is short, so more rows are ahead.  Rows that 16-byte
// copies cannot take are loaded one ahead into registers.
template <typename XT, typename T, bool VEC, bool HAS_Y> struct FwdRing {
    static constexpr int AHEAD = HAS_Y ? 2 : 6, SLOTS = AHEAD + 1;
    typedef FwdRow<XT, T, VEC, HAS_Y> Row;
    uint32_t base, pitch, bytes;
    int in, out;
    static __host__ __device__ constexpr int pieces(bool elem) {
        return RawX<XT, true>::R::PIECES + (HAS_Y ? (elem ? 2 : 1) * Raw8<T, true>::PIECES : 0);
    }
    __device__ __forceinline__ FwdRing(const ResNormArgs& a, void* smem) {
        pitch = blockDim.x * 16;
        base = (uint32_t)__cvta_generic_to_shared(smem) + threadIdx.x * 16;
        bytes = pieces(a.gate_mode == MOM_GATE_ELEMENT) * pitch;
        in = out = 0;
    }
    __device__ __forceinline__ void put(const ResNormArgs& a, int64_t row, const Place& w) {
        if (row < a.n_rows) {
            uint32_t at = base + in * bytes;
            RawX<XT, VEC>::copy(at, pitch, a, row, w.c0, w.lane);
            at += RawX<XT, VEC>::R::PIECES * pitch;
            if (HAS_Y) Raw8<T, VEC>::copy(at, pitch, reinterpret_cast<const T*>(a.y) + row * a.d, w.c0, a.d, w.lane);
            at += Raw8<T, VEC>::PIECES * pitch;
            if (HAS_Y && a.gate_mode == MOM_GATE_ELEMENT)
                Raw8<T, VEC>::copy(at, pitch, reinterpret_cast<const T*>(a.gate) + row * a.d, w.c0, a.d, w.lane);
        }
        in = in + 1 == SLOTS ? 0 : in + 1;
        asm volatile("cp.async.commit_group;" ::: "memory");
    }
    __device__ __forceinline__ void take(const ResNormArgs& a, Row& r) {
        asm volatile("cp.async.wait_group %0;" ::"n"(AHEAD - 1) : "memory");
        uint32_t at = base + out * bytes;
        r.x.r.take(at, pitch);
        at += RawX<XT, VEC>::R::PIECES * pitch;
        if (HAS_Y) r.y.take(at, pitch);
        at += Raw8<T, VEC>::PIECES * pitch;
        if (HAS_Y && a.gate_mode == MOM_GATE_ELEMENT) r.g.take(at, pitch);
        out = out + 1 == SLOTS ? 0 : out + 1;
    }
};
template <typename XT, typename T, bool HAS_Y> struct FwdRing<XT, T, false, HAS_Y> {
    typedef FwdRow<XT, T, false, HAS_Y> Row;
    static constexpr int AHEAD = 1, SLOTS = 0;
    Row next;
    static constexpr int pieces(bool) { return 0; }
    __device__ __forceinline__ FwdRing(const ResNormArgs&, void*) {}
    __device__ __forceinline__ void put(const ResNormArgs& a, int64_t row, const Place& w) { next.load(a, row, w); }
    __device__ __forceinline__ void take(const ResNormArgs&, Row& r) { r = next; }
};

// CTAs (clusters; warps, with one warp a row) walk the rows.  `red` alternates
// between two rows, so that one barrier a sum is enough.
template <typename XT, typename T, bool VEC, bool HAS_Y>
__global__ void __launch_bounds__(32 * kWarps, VEC ? 3 : 2) residual_norm_kernel(const ResNormArgs a) {
    extern __shared__ __align__(16) unsigned char slots[];
    __shared__ float red[2][2][kMaxCluster * kWarps];
    typedef FwdRing<XT, T, VEC, HAS_Y> Ring;
    const Place w(a);
    const int rows_cta = w.W > 1 ? 1 : blockDim.x >> 5;
    const int64_t step = (int64_t)gridDim.x / w.cl * rows_cta;
    int64_t row = (int64_t)(blockIdx.x / w.cl) * rows_cta + (w.W > 1 ? 0 : threadIdx.x >> 5);
    const int d = a.d;
    const float inv_d = 1.f / (float)d;
    Ring ring(a, slots);
#pragma unroll
    for (int i = 0; i < Ring::AHEAD; ++i) ring.put(a, row + i * step, w);
    T gate_next = from_f<T>(0.f);
    if (a.gate_mode == MOM_GATE_TOKEN && row < a.n_rows) gate_next = reinterpret_cast<const T*>(a.gate)[row];
    const Weights<VEC> wt(a, a.h != nullptr, w);
    if (w.cl > 1) cluster_barrier();          // the other CTAs' shared memory is there
    for (int buf = 0; row < a.n_rows; row += step, buf ^= 1) {      // the same count in all warps of a row
        FwdRow<XT, T, VEC, HAS_Y> r;
        ring.take(a, r);
        ring.put(a, row + Ring::AHEAD * step, w);
        const T gate = gate_next;
        if (a.gate_mode == MOM_GATE_TOKEN && row + step < a.n_rows)
            gate_next = reinterpret_cast<const T*>(a.gate)[row + step];
        float xv[8], ry = 0.f;
        if (HAS_Y) {
            float ss[1] = {0.f}, y[8];
            r.y.get(y);
#pragma unroll
            for (int i = 0; i < 8; ++i) ss[0] = fmaf(y[i], y[i], ss[0]);
            row_sum<1>(ss, red[buf][0], w);
            ry = rsqrtf(ss[0] * inv_d + a.eps);                     // 1 / rms(y), times a token's gate
            if (a.gate_mode == MOM_GATE_TOKEN) ry *= sigmoid(to_f(gate));
        }
        r.x.get(xv);
        if constexpr (!std::is_same<XT, Q8>::value) {
            if (a.codes_out) {
                uint32_t m[2];
                r.x.r.amax(m);
                act8_store<VEC>(xv, m, w.c0, d, w.lane, a.codes_out + row * d, a.scales_out + row * a.groups);
            }
        }
        if (HAS_Y) {
            float y[8];
            r.y.get(y);
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] *= ry;
            if (a.gate_mode == MOM_GATE_ELEMENT) {
                float g[8];
                r.g.get(g);
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] *= sigmoid(g[i]);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) xv[i] = fmaf(y[i], wt.post[i], xv[i]);
        }
        if (a.x_out) {
            if (a.x_out_f32) store8<VEC>(reinterpret_cast<float*>(a.x_out) + row * d, w.c0, d, w.lane, xv);
            else store8<VEC>(reinterpret_cast<bf16*>(a.x_out) + row * d, w.c0, d, w.lane, xv);
        }
        if (a.h) {
            float ss[1] = {0.f};
#pragma unroll
            for (int i = 0; i < 8; ++i) ss[0] = fmaf(xv[i], xv[i], ss[0]);
            row_sum<1>(ss, red[buf][1], w);
            const float rx = rsqrtf(ss[0] * inv_d + a.eps);
#pragma unroll
            for (int i = 0; i < 8; ++i) xv[i] *= rx * wt.pre[i];
            store8<VEC>(reinterpret_cast<T*>(a.h) + row * d, w.c0, d, w.lane, xv);
        }
    }
}

// A row's operands of the adjoint, as they lie in memory.
template <typename XT, typename T, typename G, bool VEC> struct BwdRow {
    RawX<XT, VEC> x;
    Raw8<T, VEC> y, g;
    Raw8<G, VEC> d, h;
    T gate;
    __device__ __forceinline__ void load(const ResNormArgs& a, const ResNormBwdArgs& b, int64_t row, const Place& w) {
        if (row >= a.n_rows) return;
        const int n = a.d;
        if (a.y) y.load(reinterpret_cast<const T*>(a.y) + row * n, w.c0, n, w.lane);
        x.load(a, row, w.c0, w.lane);
        if (a.gate_mode == MOM_GATE_ELEMENT) g.load(reinterpret_cast<const T*>(a.gate) + row * n, w.c0, n, w.lane);
        if (b.dh) h.load(reinterpret_cast<const G*>(b.dh) + row * n, w.c0, n, w.lane);
        if (b.dx_out) d.load(reinterpret_cast<const G*>(b.dx_out) + row * n, w.c0, n, w.lane);
        if (a.gate_mode == MOM_GATE_TOKEN) gate = reinterpret_cast<const T*>(a.gate)[row];
    }
};

// The adjoint.  CTAs (clusters) walk the rows; the next row's operands are
// loaded (packed) before this row's arithmetic, so that loads are in flight
// through its three reductions.  Threads keep the two column sums (A and
// dw_pre) of their channels in registers and write them once as a partial,
// which cols_reduce_kernel adds up in order: no atomics, the same sums every
// time on the same device.
template <typename XT, typename T, typename G, bool VEC>
__global__ void __launch_bounds__(32 * kWarps, 2) residual_norm_bwd_kernel(const ResNormArgs a,
                                                                           const ResNormBwdArgs b) {
    __shared__ float red[2][4][kMaxCluster * kWarps];
    const Place w(a);
    const int d = a.d;
    const int64_t step = gridDim.x / w.cl, first = blockIdx.x / w.cl;
    const float inv_d = 1.f / (float)d;
    float accA[8], accP[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) accA[i] = accP[i] = 0.f;
    BwdRow<XT, T, G, VEC> next;
    next.load(a, b, first, w);
    const Weights<VEC> wt(a, b.dh != nullptr, w);
    if (w.cl > 1) cluster_barrier();          // the other CTAs' shared memory is there
    int buf = 0;
    for (int64_t row = first; row < a.n_rows; row += step, buf ^= 1) {
        const BwdRow<XT, T, G, VEC> r = next;
        next.load(a, b, row + step, w);
        float yv[8], gv[8], dv[8];
        float gt = 1.f, rest = 0.f, ry = 0.f;
        if (a.gate_mode == MOM_GATE_TOKEN) gt = sigmoid(to_f(r.gate), rest);
        if (a.y) {
            float ss[1] = {0.f};
            r.y.get(yv);
#pragma unroll
            for (int i = 0; i < 8; ++i) ss[0] = fmaf(yv[i], yv[i], ss[0]);
            row_sum<1>(ss, red[buf][0], w);
            ry = rsqrtf(ss[0] * inv_d + a.eps);
#pragma unroll
            for (int i = 0; i < 8; ++i) yv[i] *= ry;                          // n_y
            if (a.gate_mode == MOM_GATE_ELEMENT) {
                r.g.get(gv);
#pragma unroll
                for (int i = 0; i < 8; ++i) gv[i] = sigmoid(gv[i]);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) gv[i] = gt;
            }
        }
        if (b.dx_out) {
            r.d.get(dv);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) dv[i] = 0.f;
        }
        if (b.dh) {
            float ss[2] = {0.f, 0.f}, xv[8], hv[8];
            r.x.get(xv);
            r.h.get(hv);
            if (a.y) {
#pragma unroll
                for (int i = 0; i < 8; ++i) xv[i] = fmaf(yv[i] * gv[i], wt.post[i], xv[i]);      // x'
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                ss[0] = fmaf(xv[i], xv[i], ss[0]);
                ss[1] = fmaf(xv[i], hv[i] * wt.pre[i], ss[1]);
            }
            row_sum<2>(ss, red[buf][1], w);
            const float rx = rsqrtf(ss[0] * inv_d + a.eps);
            const float k = ss[1] * inv_d * rx * rx * rx;                     // mean(dn n_x) / rms / rms
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float hr = hv[i] * rx;
                accP[i] = fmaf(hr, xv[i], accP[i]);
                dv[i] = fmaf(hr, wt.pre[i], fmaf(xv[i], -k, dv[i]));
            }
        }
        store8<VEC>(reinterpret_cast<G*>(b.dx) + row * d, w.c0, d, w.lane, dv);
        if (a.y) {
            float ss[1] = {0.f}, o[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float t = dv[i] * gv[i];
                accA[i] = fmaf(t, yv[i], accA[i]);
                dv[i] = t * wt.post[i];                                       // u = D s sigma w_post
                ss[0] = fmaf(dv[i], yv[i], ss[0]);
            }
            row_sum<1>(ss, red[buf][3], w);
            const float m = ss[0] * inv_d * ry;
            if (a.gate_mode == MOM_GATE_TOKEN && b.dgate && threadIdx.x == 0 && w.rank == 0)
                reinterpret_cast<T*>(b.dgate)[row] = from_f<T>(ss[0] * rest);
            if (a.gate_mode == MOM_GATE_ELEMENT && b.dgate) {
                r.g.get(o);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    float q;
                    sigmoid(o[i], q);
                    o[i] = dv[i] * yv[i] * q;
                }
                store8<VEC>(reinterpret_cast<T*>(b.dgate) + row * d, w.c0, d, w.lane, o);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = fmaf(dv[i], ry, -yv[i] * m);
            store8<VEC>(reinterpret_cast<T*>(b.dy) + row * d, w.c0, d, w.lane, o);
        }
    }
    float* pa = b.partial + first * 2 * d;
    store8<VEC>(pa, w.c0, d, w.lane, accA);
    store8<VEC>(pa + d, w.c0, d, w.lane, accP);
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

// CTAs of a row's cluster and warps of a CTA.
struct Shape {
    int cluster, warps;
};
Shape shape_for(int d) {
    const int chunks = (int)cdiv(d, kChunk);
    int cl = 1;
    while (cl * kWarps < chunks) cl *= 2;
    return {cl, (int)cdiv(chunks, cl)};
}

template <typename... P, typename... A>
cudaError_t launch(void (*kernel)(P...), int64_t ctas, int threads, size_t smem, int cluster, cudaStream_t st,
                   const A&... args) {
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = cluster;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = &at;
    cfg.numAttrs = cluster > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Warps an SM that the registers leave (__launch_bounds__).
constexpr int kFwdWarps = 24, kWarpsSM = 16;
constexpr int kSmemSM = 220 * 1024;

template <typename XT, typename T, bool VEC, bool HAS_Y> cudaError_t run_fwd(ResNormArgs a, cudaStream_t st) {
    typedef FwdRing<XT, T, VEC, HAS_Y> Ring;
    auto* kernel = residual_norm_kernel<XT, T, VEC, HAS_Y>;
    const Shape s = shape_for(a.d);
    a.cluster = s.cluster;
    a.warps_per_row = s.warps;
    const bool own = s.warps * s.cluster == 1;                 // a row a warp
    const int threads = own ? 128 : 32 * s.warps;
    const size_t smem = (size_t)Ring::SLOTS * Ring::pieces(a.gate_mode == MOM_GATE_ELEMENT) * threads * 16;
    static unsigned long long optin_done = 0;
    const cudaError_t e = smem_optin((const void*)kernel, Ring::SLOTS * Ring::pieces(true) * 32 * kWarps * 16, &optin_done);
    if (e != cudaSuccess) return e;
    int ctas = (VEC ? kFwdWarps : kWarpsSM) / (threads / 32);
    if (smem * ctas > kSmemSM) ctas = (int)(kSmemSM / smem);
    const int64_t units = own ? cdiv(a.n_rows, threads / 32) : a.n_rows;
    const int64_t most = (int64_t)sm_count() * ctas / s.cluster;
    return launch(kernel, (units < most ? units : most) * s.cluster, threads, smem, s.cluster, st, a);
}

template <typename XT, typename T, typename G, bool VEC>
cudaError_t run_bwd(ResNormArgs a, const ResNormBwdArgs& b, int parts, cudaStream_t st) {
    const Shape s = shape_for(a.d);
    a.cluster = s.cluster;
    a.warps_per_row = s.warps;
    return launch(residual_norm_bwd_kernel<XT, T, G, VEC>, (int64_t)parts * s.cluster, 32 * s.warps, 0, s.cluster, st, a, b);
}

}  // namespace

// rows of partial column sums the adjoint writes
int residual_norm_bwd_parts(int64_t n_rows, int d) {
    const Shape s = shape_for(d);
    const int64_t most = (int64_t)sm_count() * (kWarpsSM / s.warps) / s.cluster;
    return (int)(n_rows < most ? n_rows : most);
}

cudaError_t launch_residual_norm(const ResNormArgs& a, int x_kind, int dt, bool vec, cudaStream_t st) {
    cudaError_t e;
#define MOM_RN(XT, T) e = a.y ? (vec ? run_fwd<XT, T, true, true>(a, st) : run_fwd<XT, T, false, true>(a, st)) \
                        : (vec ? run_fwd<XT, T, true, false>(a, st) : run_fwd<XT, T, false, false>(a, st))
    if (x_kind == RN_X_BF16) MOM_RN(bf16, bf16);
    else if (x_kind == RN_X_F32) { if (dt == MOM_BF16) MOM_RN(float, bf16); else MOM_RN(float, float); }
    else { if (dt == MOM_BF16) MOM_RN(Q8, bf16); else MOM_RN(Q8, float); }
#undef MOM_RN
    count_launches(1);
    return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_residual_norm_bwd(const ResNormArgs& a, const ResNormBwdArgs& b, int x_kind, int dt, int g_dt,
                                     bool vec, cudaStream_t st) {
    const int parts = residual_norm_bwd_parts(a.n_rows, a.d);
    if (parts > 0) {
        cudaError_t e;
#define MOM_RNB(XT, T, G) e = vec ? run_bwd<XT, T, G, true>(a, b, parts, st) : run_bwd<XT, T, G, false>(a, b, parts, st)
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
        cols_reduce_kernel<<<dim3((unsigned)cdiv(a.d, 32), 2), 1024, 0, st>>>(b.partial, parts, a.d, a.w_post, a.res_scale,
                                                                    b.dw_post, b.dres_scale, b.dw_pre);
        count_launches(1);
    }
    return cudaGetLastError();
}

}  // namespace mom
