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

template <typename T, bool VEC, bool FLAT>
__global__ void __launch_bounds__(kThreads) act8_pack_kernel(const T* __restrict__ x, int64_t total, int d, int chunks,
                                                             int groups, int8_t* __restrict__ codes,
                                                             float* __restrict__ scales) {
    const int lane = threadIdx.x & 31;
    const int64_t step = (int64_t)gridDim.x * (kThreads / 32);
    for (int64_t u = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); u < total; u += step * kUnroll) {
        Raw8<T, VEC> r[kUnroll];
        Where w[kUnroll];
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) {
            const int64_t v = u + k * step;
            if (v < total) {
                w[k] = FLAT ? Where{v, 0} : where(v, chunks);
                r[k].load(x + w[k].row * (FLAT ? kChunk : d), w[k].c0, FLAT ? kChunk : d, lane);
            }
        }
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) {
            if (u + k * step < total) {
                float f[8];
                uint32_t m[2];
                r[k].get(f);
                r[k].amax(m);
                act8_store<VEC>(f, m, w[k].c0, FLAT ? kChunk : d, lane, codes + w[k].row * (FLAT ? kChunk : d),
                                scales + w[k].row * (FLAT ? 2 : groups));
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

unsigned grid_for(int64_t units) {
    int dev = 0, sms = 148;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    const int64_t want = cdiv(units, kThreads / 32), most = (int64_t)sms * 8;
    return (unsigned)(want < most ? want : most);
}

}  // namespace

cudaError_t launch_act8_pack(const void* x, int dt, int64_t n_rows, int d, int8_t* codes, float* scales, bool vec,
                             cudaStream_t st) {
    const int chunks = (int)cdiv(d, kChunk), groups = (int)cdiv(d, kActGroup);
    const int64_t total = n_rows * chunks;
    const unsigned grid = grid_for(total);
    const bool flat = vec && d % kChunk == 0;
#define MOM_PACK(T, V, F) \
    act8_pack_kernel<T, V, F><<<grid, kThreads, 0, st>>>(reinterpret_cast<const T*>(x), total, d, chunks, groups, codes, scales)
#define MOM_PACK_T(T) do { if (flat) MOM_PACK(T, true, true); else if (vec) MOM_PACK(T, true, false); else MOM_PACK(T, false, false); } while (0)
    if (dt == MOM_BF16) MOM_PACK_T(bf16);
    else MOM_PACK_T(float);
#undef MOM_PACK_T
#undef MOM_PACK
    count_launches(1);
    return cudaGetLastError();
}

cudaError_t launch_act8_unpack(const int8_t* codes, const float* scales, int64_t n_rows, int d, void* x, int dt,
                               bool vec, cudaStream_t st) {
    const int chunks = (int)cdiv(d, kChunk), groups = (int)cdiv(d, kActGroup);
    const int64_t total = n_rows * chunks;
    const unsigned grid = grid_for(total);
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
