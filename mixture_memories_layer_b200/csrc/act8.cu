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

// One warp per (row, chunk), grid-strided.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads) act8_pack_kernel(const T* __restrict__ x, int64_t n_rows, int d,
                                                             int chunks, int groups, int8_t* __restrict__ codes,
                                                             float* __restrict__ scales) {
    const int lane = threadIdx.x & 31;
    const int64_t total = n_rows * chunks, step = (int64_t)gridDim.x * (kThreads / 32);
    for (int64_t u = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); u < total; u += step) {
        const int64_t row = u / chunks;
        const int c0 = (int)(u - row * chunks) * kChunk;
        float v[8];
        load8<VEC>(x + row * d, c0, d, lane, v);
        act8_store<VEC>(v, c0, d, lane, codes + row * d, scales + row * groups);
    }
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads) act8_unpack_kernel(const int8_t* __restrict__ codes,
                                                               const float* __restrict__ scales, int64_t n_rows, int d,
                                                               int chunks, int groups, T* __restrict__ x) {
    const int lane = threadIdx.x & 31;
    const int64_t total = n_rows * chunks, step = (int64_t)gridDim.x * (kThreads / 32);
    for (int64_t u = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); u < total; u += step) {
        const int64_t row = u / chunks;
        const int c0 = (int)(u - row * chunks) * kChunk;
        float v[8];
        act8_load<VEC>(codes + row * d, scales + row * groups, c0, d, lane, v);
        store8<VEC>(x + row * d, c0, d, lane, v);
    }
}

unsigned grid_for(int64_t units) {
    int dev = 0, sms = 148;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    const int64_t want = cdiv(units, kThreads / 32), most = (int64_t)sms * 16;
    return (unsigned)(want < most ? want : most);
}

}  // namespace

cudaError_t launch_act8_pack(const void* x, int dt, int64_t n_rows, int d, int8_t* codes, float* scales, bool vec,
                             cudaStream_t st) {
    const int chunks = (int)cdiv(d, kChunk), groups = (int)cdiv(d, kActGroup);
    const unsigned grid = grid_for(n_rows * chunks);
#define MOM_PACK(T, V) \
    act8_pack_kernel<T, V><<<grid, kThreads, 0, st>>>(reinterpret_cast<const T*>(x), n_rows, d, chunks, groups, codes, scales)
    if (dt == MOM_BF16) { if (vec) MOM_PACK(bf16, true); else MOM_PACK(bf16, false); }
    else { if (vec) MOM_PACK(float, true); else MOM_PACK(float, false); }
#undef MOM_PACK
    count_launches(1);
    return cudaGetLastError();
}

cudaError_t launch_act8_unpack(const int8_t* codes, const float* scales, int64_t n_rows, int d, void* x, int dt,
                               bool vec, cudaStream_t st) {
    const int chunks = (int)cdiv(d, kChunk), groups = (int)cdiv(d, kActGroup);
    const unsigned grid = grid_for(n_rows * chunks);
#define MOM_UNPACK(T, V) \
    act8_unpack_kernel<T, V><<<grid, kThreads, 0, st>>>(codes, scales, n_rows, d, chunks, groups, reinterpret_cast<T*>(x))
    if (dt == MOM_BF16) { if (vec) MOM_UNPACK(bf16, true); else MOM_UNPACK(bf16, false); }
    else { if (vec) MOM_UNPACK(float, true); else MOM_UNPACK(float, false); }
#undef MOM_UNPACK
    count_launches(1);
    return cudaGetLastError();
}

}  // namespace mom
