// 8-bit activation checkpoints: a stored activation [n_rows, d] as int8 codes
// with one float32 scale for 128 channels of a row (rows8.cuh has the rule),
// and back.  Training keeps a block's input this way between its forward and
// its backward pass.
//
// Bound by memory: 2 or 4 bytes an element one way, 1 + 4/128 the other.  A
// warp owns chunks of 256 channels, which hold two whole groups, so the
// maxima never leave the warp; each lane reads 16 or 32 bytes at once.
#include "rows8.cuh"
#include "kernels.h"

namespace mom {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;       // chunks of a warp in flight

// Row and first channel of chunk u.  Where d is a multiple of 256 (FLAT in the
// kernels) the array is taken as rows of one chunk and nothing is divided.
struct Where {
    int64_t row;
    int c0;
};
__device__ __forceinline__ Where where(int64_t u, int chunks) {
    Where w;
    w.row = u < 0x7fffffffLL ? (int64_t)((uint32_t)u / (uint32_t)chunks) : u / chunks;
    w.c0 = (int)(u - w.row * chunks) * kChunk;
    return w;
}

// Rows that 16-byte copies can take: kAhead chunks of a warp are in flight to
// slots in shared memory, of which each thread reads what it copied itself.
constexpr int kAhead = 5, kSlots = kAhead + 1;
template <typename T, bool FLAT>
__global__ void __launch_bounds__(kThreads, 4) act8_pack_kernel(const T* __restrict__ x, int64_t total, int d, int chunks,
                                                                int groups, int8_t* __restrict__ codes,
                                                                float* __restrict__ scales) {
    typedef Raw8<T, true> R;
    extern __shared__ __align__(16) unsigned char smem[];
    const int lane = threadIdx.x & 31;
    const uint32_t pitch = kThreads * 16, base = (uint32_t)__cvta_generic_to_shared(smem) + threadIdx.x * 16;
    const int64_t step = (int64_t)gridDim.x * (kThreads / 32);
    int64_t u = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    const int dd = FLAT ? kChunk : d;
    auto put = [&](int64_t v, int slot) {
        if (v < total) {
            const Where w = FLAT ? Where{v, 0} : where(v, chunks);
            R::copy(base + slot * R::PIECES * pitch, pitch, x + w.row * dd, w.c0, dd, lane);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int k = 0; k < kAhead; ++k) put(u + k * step, k);
    int in = kAhead, out = 0;
    for (; u < total; u += step) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
        R r;
        r.take(base + out * R::PIECES * pitch, pitch);
        put(u + kAhead * step, in);
        in = in + 1 == kSlots ? 0 : in + 1;
        out = out + 1 == kSlots ? 0 : out + 1;
        const Where w = FLAT ? Where{u, 0} : where(u, chunks);
        float f[8];
        uint32_t m[2];
        r.get(f);
        r.amax(m);
        act8_store<true>(f, m, w.c0, dd, lane, codes + w.row * dd, scales + w.row * (FLAT ? 2 : groups));
    }
}

// Other rows: kUnroll chunks of a warp loaded at a time.
template <typename T>
__global__ void __launch_bounds__(kThreads) act8_pack_odd_kernel(const T* __restrict__ x, int64_t total, int d, int chunks,
                                                                 int groups, int8_t* __restrict__ codes,
                                                                 float* __restrict__ scales) {
    const int lane = threadIdx.x & 31;
    const int64_t step = (int64_t)gridDim.x * (kThreads / 32);
    for (int64_t u = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); u < total; u += step * kUnroll) {
        Raw8<T, false> r[kUnroll];
        Where w[kUnroll];
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) {
            const int64_t v = u + k * step;
            if (v < total) {
                w[k] = where(v, chunks);
                r[k].load(x + w[k].row * d, w[k].c0, d, lane);
            }
        }
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) {
            if (u + k * step < total) {
                float f[8];
                uint32_t m[2];
                r[k].get(f);
                r[k].amax(m);
                act8_store<false>(f, m, w[k].c0, d, lane, codes + w[k].row * d, scales + w[k].row * groups);
            }
        }
    }
}

template <typename T, bool VEC, bool FLAT>
__global__ void __launch_bounds__(kThreads) act8_unpack_kernel(const int8_t* __restrict__ codes,
                                                               const float* __restrict__ scales, int64_t total, int d,
                                                               int chunks, int groups, T* __restrict__ x) {
    const int lane = threadIdx.x & 31;
    const int64_t step = (int64_t)gridDim.x * (kThreads / 32);
    for (int64_t u = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); u < total; u += step * kUnroll) {
        Raw8Q<VEC> r[kUnroll];
        Where w[kUnroll];
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) {
            const int64_t v = u + k * step;
            if (v < total) {
                w[k] = FLAT ? Where{v, 0} : where(v, chunks);
                r[k].load(codes + w[k].row * (FLAT ? kChunk : d), scales + w[k].row * (FLAT ? 2 : groups), w[k].c0,
                          FLAT ? kChunk : d, lane);
            }
        }
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) {
            if (u + k * step < total) {
                float f[8];
                r[k].get(f);
                store8<VEC>(x + w[k].row * (FLAT ? kChunk : d), w[k].c0, FLAT ? kChunk : d, lane, f);
            }
        }
    }
}

// `ctas` an SM at most
unsigned grid_for(int64_t units, int ctas) {
    int dev = 0, sms = 148;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    const int64_t want = cdiv(units, kThreads / 32), most = (int64_t)sms * ctas;
    return (unsigned)(want < most ? want : most);
}

template <typename T, bool FLAT>
cudaError_t run_pack(const void* x, int64_t total, int d, int chunks, int groups, int8_t* codes, float* scales,
                     cudaStream_t st) {
    constexpr int SMEM = kSlots * Raw8<T, true>::PIECES * kThreads * 16;
    auto* kernel = act8_pack_kernel<T, FLAT>;
    static unsigned long long optin_done = 0;
    const cudaError_t e = smem_optin((const void*)kernel, SMEM, &optin_done);
    if (e != cudaSuccess) return e;
    kernel<<<grid_for(total, 4), kThreads, SMEM, st>>>(reinterpret_cast<const T*>(x), total, d, chunks, groups, codes, scales);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_act8_pack(const void* x, int dt, int64_t n_rows, int d, int8_t* codes, float* scales, bool vec,
                             cudaStream_t st) {
    const int chunks = (int)cdiv(d, kChunk), groups = (int)cdiv(d, kActGroup);
    const int64_t total = n_rows * chunks;
    const bool flat = vec && d % kChunk == 0;
    count_launches(1);
    if (dt == MOM_BF16) {
        if (flat) return run_pack<bf16, true>(x, total, d, chunks, groups, codes, scales, st);
        if (vec) return run_pack<bf16, false>(x, total, d, chunks, groups, codes, scales, st);
        act8_pack_odd_kernel<bf16><<<grid_for(total, 8), kThreads, 0, st>>>(reinterpret_cast<const bf16*>(x), total, d, chunks, groups, codes, scales);
    } else {
        if (flat) return run_pack<float, true>(x, total, d, chunks, groups, codes, scales, st);
        if (vec) return run_pack<float, false>(x, total, d, chunks, groups, codes, scales, st);
        act8_pack_odd_kernel<float><<<grid_for(total, 8), kThreads, 0, st>>>(reinterpret_cast<const float*>(x), total, d, chunks, groups, codes, scales);
    }
    return cudaGetLastError();
}

cudaError_t launch_act8_unpack(const int8_t* codes, const float* scales, int64_t n_rows, int d, void* x, int dt,
                               bool vec, cudaStream_t st) {
    const int chunks = (int)cdiv(d, kChunk), groups = (int)cdiv(d, kActGroup);
    const int64_t total = n_rows * chunks;
    const unsigned grid = grid_for(total, 8);
    const bool flat = vec && d % kChunk == 0;
#define MOM_UNPACK(T, V, F) \
    act8_unpack_kernel<T, V, F><<<grid, kThreads, 0, st>>>(codes, scales, total, d, chunks, groups, reinterpret_cast<T*>(x))
#define MOM_UNPACK_T(T) do { if (flat) MOM_UNPACK(T, true, true); else if (vec) MOM_UNPACK(T, true, false); else MOM_UNPACK(T, false, false); } while (0)
    if (dt == MOM_BF16) MOM_UNPACK_T(bf16);
    else MOM_UNPACK_T(float);
#undef MOM_UNPACK_T
#undef MOM_UNPACK
    count_launches(1);
    return cudaGetLastError();
}

}  // namespace mom
