// Softmax cross entropy of the logits z = x W^T over a large vocabulary, and
// its gradient, on the tcgen05 tensor cores without storing the logits.
//
//   forward   lse_t = log sum_v exp(z_tv),  loss_t = lse_t - z_t,target
//   backward  g_tv = r_t (exp(z_tv - lse_t) - [v = target_t]),
//             dx = g W,  dW = g^T x
//
// One persistent GEMM kernel runs all four products; they differ in the
// operands' majors and in what happens to an accumulator tile:
//   stats  x W^T      each row's running maximum and sum of exponentials over
//                     the tile's columns (float32, one pass over TMEM), and
//                     the target's logit; logsumexp_kernel joins the tiles
//   grad   x W^T      the logits of one piece of the vocabulary again, made
//                     into g and stored as bf16
//   store / add       dx += g W over the pieces (float32, added in L2 by the
//                     copy engine, in piece order), dW = g^T x
// Bound by the tensor cores (2 n d v operations a product) except for few
// rows, where reading W once bounds it; then the long vocabulary axis of dx
// (or the long token axis of dW) is split over CTAs and the slots are summed
// in a fixed order.  There are no atomics on floats: results repeat.
//
// float32 operands: every value is split exactly into three bf16 parts, a =
// a0 + a1 + a2 (8 bits each), and the six products a_i b_j with i + j <= 2 run
// as one longer K loop into the same accumulator, smallest first; the rest is
// below 2^-24 of a product.
//
// Roles (320 threads, one CTA per SM, persistent over tiles): warp 0 issues
// the TMA loads of both operands (4 stages of 128 x 64 and 256 x 64), warp 1
// the MMAs (M 128, N 256, K 16) into one of two TMEM accumulators, warps 2-9
// are the epilogue (two warps a TMEM lane quarter) and overlap the next
// tile's main loop.  Every wait is bounded (sm100.cuh).
#include "common.cuh"
#include "kernels.h"
#include "sm100.cuh"

namespace mom {

namespace {

using namespace sm100;

constexpr int BM = 128, BN = 256, BK = 64, STAGES = 4;
constexpr int A_BYTES = BM * BK * 2, B_BYTES = BN * BK * 2;
constexpr int MN_GROUP = 64 * BK * 2;                // an MN-major box: 64 MN x 64 K, bf16
constexpr int NEPI = 256, THREADS = 64 + NEPI;
constexpr int PIECE = 32 * 128;                      // an epilogue warp's staging: 32 rows x 128 bytes
constexpr size_t SMEM_BYTES = 1024 + (size_t)STAGES * (A_BYTES + B_BYTES) + (size_t)(NEPI / 32) * PIECE + 256;
constexpr uint32_t TMEM_COLS = 2 * BN;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

enum Epi { EPI_STATS, EPI_GRAD, EPI_BF16, EPI_F32 };

struct GemmArgs {
    int64_t m_tiles, n_tiles, tiles;     // output tiles; tiles = m_tiles * n_tiles * k_splits
    int kb_total, kb_split;              // K blocks of 64 in all and of one split
    int n_pairs;                         // products of operand parts
    uint8_t pa[6], pb[6];
    int b_row0;                          // K-major B: first row; MN-major B: first K row
    int64_t m, n;                        // valid output rows and columns
    // stats / grad
    const int32_t* targets;
    int64_t v0, vocab;                   // the piece's first class
    float2* partials;                    // [column half tiles][m]
    float* zt;                           // the targets' logits
    const float *lse, *dloss, *dscale;
    int n_parts;                         // bf16 parts of g
    int add;                             // EPI_F32: add to what is there
    void* ws;
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, uint32_t src, int c0, int c1, int c2) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];"
                 ::"l"(reinterpret_cast<uint64_t>(map)), "r"(src), "r"(c0), "r"(c1), "r"(c2)
                 : "memory");
}
__device__ __forceinline__ void tma_add_3d(const CUtensorMap* map, uint32_t src, int c0, int c1, int c2) {
    asm volatile("cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.bulk_group [%0, {%2, %3, %4}], [%1];"
                 ::"l"(reinterpret_cast<uint64_t>(map)), "r"(src), "r"(c0), "r"(c1), "r"(c2)
                 : "memory");
}
__device__ __forceinline__ void st_shared_v4(uint32_t dst, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(dst), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&h);
}
// part p of the exact split of v into bf16 parts
__device__ __forceinline__ float bf16_part(float v, int p) {
    for (int i = 0; i < p; ++i) v -= __bfloat162float(__float2bfloat16_rn(v));
    return v;
}

struct Tile {
    int64_t mt, nt;
    int ks, kb0, kb1;
};
// rows fastest: the CTAs of one wave share few column tiles of B
__device__ __forceinline__ Tile tile_at(const GemmArgs& p, int64_t t) {
    Tile T;
    T.mt = t % p.m_tiles;
    const int64_t r = t / p.m_tiles;
    T.nt = r % p.n_tiles;
    T.ks = (int)(r / p.n_tiles);
    T.kb0 = T.ks * p.kb_split;
    T.kb1 = T.kb0 + p.kb_split < p.kb_total ? T.kb0 + p.kb_split : p.kb_total;
    return T;
}

template <int EPI, bool A_MN, bool B_MN>
__global__ void __launch_bounds__(THREADS, 1)
ce_gemm_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
               const __grid_constant__ CUtensorMap tm_out, const GemmArgs p) {
    extern __shared__ unsigned char smem_raw[];
    unsigned char* smem = align1024_shared(smem_raw);
    unsigned char* sA = smem;
    unsigned char* sB = smem + STAGES * A_BYTES;
    unsigned char* sOut = sB + STAGES * B_BYTES;
    uint64_t* bars = reinterpret_cast<uint64_t*>(sOut + (NEPI / 32) * PIECE);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * STAGES + 5);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t full0 = smem_u32(bars), empty0 = smem_u32(bars + STAGES);
    const uint32_t tfull0 = smem_u32(bars + 2 * STAGES), tempty0 = smem_u32(bars + 2 * STAGES + 2);
    const uint32_t done_bar = smem_u32(bars + 2 * STAGES + 4);
    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(full0 + 8 * s, 1);
            mbar_init(empty0 + 8 * s, 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(tfull0 + 8 * a, 1);
            mbar_init(tempty0 + 8 * a, NEPI);
        }
        mbar_init(done_bar, 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(tmem_slot), TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;

    if (warp == 0) {
        if (lane == 0) {
            // ---------------------------------------------------- TMA loads
            uint32_t it = 0;
            bool ok = true;
            for (int64_t t = blockIdx.x; t < p.tiles && ok; t += gridDim.x) {
                const Tile T = tile_at(p, t);
                const int m0 = (int)(T.mt * BM), n0 = (int)(T.nt * BN);
                for (int pr = 0; pr < p.n_pairs && ok; ++pr) {
                    const int qa = p.pa[pr], qb = p.pb[pr];
                    for (int kb = T.kb0; kb < T.kb1; ++kb, ++it) {
                        const uint32_t s = it % STAGES, ph = (it / STAGES) & 1;
                        if (!mbar_wait(empty0 + 8 * s, ph ^ 1, abort_flag, p.ws, 1)) { ok = false; break; }
                        const uint32_t bar = full0 + 8 * s;
                        const uint32_t a0 = smem_u32(sA + s * A_BYTES), b0 = smem_u32(sB + s * B_BYTES);
                        mbar_arrive_expect_tx(bar, A_BYTES + B_BYTES);
                        if constexpr (A_MN) {
#pragma unroll
                            for (int g = 0; g < BM / 64; ++g)
                                tma_load_3d(a0 + g * MN_GROUP, &tm_a, bar, m0 + 64 * g, kb * BK, qa);
                        } else {
                            tma_load_3d(a0, &tm_a, bar, kb * BK, m0, qa);
                        }
                        if constexpr (B_MN) {
#pragma unroll
                            for (int g = 0; g < BN / 64; ++g)
                                tma_load_3d(b0 + g * MN_GROUP, &tm_b, bar, n0 + 64 * g, p.b_row0 + kb * BK, qb);
                        } else {
                            tma_load_3d(b0, &tm_b, bar, kb * BK, p.b_row0 + n0, qb);
                        }
                    }
                }
            }
            if (!ok)      // loads still in flight must land before the CTA exits
                for (uint32_t j = it >= STAGES ? it - STAGES : 0; j < it; ++j)
                    mbar_wait_drain(full0 + 8 * (j % STAGES), (j / STAGES) & 1);
        }
    } else if (warp == 1) {
        if (lane == 0) {
            // --------------------------------------------------- MMA issuer
            constexpr uint32_t IDESC = idesc_bf16_f32(BM, BN, A_MN, B_MN);
            uint32_t it = 0, tc = 0;
            bool ok = true;
            for (int64_t t = blockIdx.x; t < p.tiles && ok; t += gridDim.x, ++tc) {
                const Tile T = tile_at(p, t);
                const uint32_t acc = tc & 1, aph = (tc >> 1) & 1;
                if (!mbar_wait(tempty0 + 8 * acc, aph ^ 1, abort_flag, p.ws, 2)) break;
                tc_fence_after();
                const uint32_t d_tmem = tmem_base + acc * BN;
                const int steps = (T.kb1 - T.kb0) * p.n_pairs;
                for (int k = 0; k < steps; ++k, ++it) {
                    const uint32_t s = it % STAGES, ph = (it / STAGES) & 1;
                    if (!mbar_wait(full0 + 8 * s, ph, abort_flag, p.ws, 3)) { ok = false; break; }
                    tc_fence_after();
                    const uint32_t a0 = smem_u32(sA + s * A_BYTES), b0 = smem_u32(sB + s * B_BYTES);
#pragma unroll
                    for (int j = 0; j < BK / 16; ++j) {
                        const uint64_t da = A_MN ? desc_mnmajor_sw128(a0 + 2048 * j, MN_GROUP)
                                                 : desc_kmajor_sw128(a0 + 32 * j);
                        const uint64_t db = B_MN ? desc_mnmajor_sw128(b0 + 2048 * j, MN_GROUP)
                                                 : desc_kmajor_sw128(b0 + 32 * j);
                        umma_f16(d_tmem, da, db, IDESC, (k | j) != 0);
                    }
                    umma_commit(empty0 + 8 * s);
                }
                if (!ok) break;
                umma_commit(tfull0 + 8 * acc);
            }
            // every MMA this CTA issued has finished before TMEM is released
            umma_commit(done_bar);
            mbar_wait_drain(done_bar, 0);
        }
    } else {
        // ------------------------------------------------------- epilogue
        // warp 2 + e: TMEM lanes 32 (warp % 4) .. + 31, columns [128 (e / 4), + 128)
        const int e = warp - 2, qd = warp & 3, hf = e >> 2;
        constexpr int HALF = BN / 2;
        const uint32_t piece = smem_u32(sOut + e * PIECE);
        float gscale = 1.f;
        if constexpr (EPI == EPI_GRAD) gscale = p.dscale ? *p.dscale : 1.f;
        uint32_t tc = 0;
        for (int64_t t = blockIdx.x; t < p.tiles; t += gridDim.x, ++tc) {
            const Tile T = tile_at(p, t);
            const uint32_t acc = tc & 1, aph = (tc >> 1) & 1;
            const int64_t row = T.mt * BM + 32 * qd + lane;
            const bool live = row < p.m;
            const int64_t col0 = T.nt * BN + hf * HALF;
            // the target's column inside this half tile (< 0: not here)
            int tl = -1;
            float lse2 = 0.f, wt = 0.f;
            if constexpr (EPI == EPI_STATS || EPI == EPI_GRAD) {
                if (live) {
                    const int64_t tg = p.targets[row];
                    const bool in = tg >= 0 && tg < p.vocab;
                    const int64_t rel = tg - p.v0 - col0;
                    if (in && rel >= 0 && rel < HALF) tl = (int)rel;
                    if constexpr (EPI == EPI_GRAD) {
                        if (in) wt = (p.dloss ? p.dloss[row] : 1.f) * gscale;
                        lse2 = in ? p.lse[row] * kLog2e : INFINITY;      // padding: every exponential is 0
                    }
                }
            }
            if (!mbar_wait(tfull0 + 8 * acc, aph, abort_flag, p.ws, 4)) break;
            tc_fence_after();
            const uint32_t taddr = tmem_base + ((uint32_t)(32 * qd) << 16) + acc * BN + hf * HALF;
            const int64_t left = p.n - col0;
            const int nv = left < 0 ? 0 : left < HALF ? (int)left : HALF;      // valid columns of the half tile
            if constexpr (EPI == EPI_STATS) {
                float m = -INFINITY, s = 0.f, zt = 0.f;
#pragma unroll
                for (int c = 0; c < HALF; c += 32) {
                    uint32_t r[32];
                    tmem_ld_x32(taddr + c, r);
                    tmem_ld_wait();
                    if (c + 32 > nv) {
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (c + i >= nv) r[i] = 0xff800000u;               // -inf
                    }
                    float mx = m;
#pragma unroll
                    for (int i = 0; i < 32; ++i) mx = fmaxf(mx, __uint_as_float(r[i]));
                    // all -inf so far: exponentials of (-inf - 0) are 0, not NaN
                    const float sub = mx == -INFINITY ? 0.f : mx * kLog2e;
                    s *= ex2(fmaf(m, kLog2e, -sub));
#pragma unroll
                    for (int i = 0; i < 32; ++i) s += ex2(fmaf(__uint_as_float(r[i]), kLog2e, -sub));
                    m = mx;
                    if (tl >= c && tl < c + 32) {
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (tl == c + i) zt = __uint_as_float(r[i]);
                    }
                }
                if (live) {
                    p.partials[(T.nt * 2 + hf) * p.m + row] = make_float2(m, s);
                    if (tl >= 0) p.zt[row] = zt;
                }
            } else if constexpr (EPI == EPI_F32) {
#pragma unroll
                for (int c = 0; c < HALF; c += 32) {
                    if (c >= nv) break;
                    if (lane == 0) bulk_wait_read0();          // the previous piece has left shared memory
                    __syncwarp();
                    uint32_t r[32];
                    tmem_ld_x32(taddr + c, r);
                    tmem_ld_wait();
#pragma unroll
                    for (int q = 0; q < 8; ++q)
                        st_shared_v4(piece + lane * 128 + ((q ^ (lane & 7)) << 4), r[4 * q], r[4 * q + 1], r[4 * q + 2],
                                     r[4 * q + 3]);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0 && T.mt * BM + 32 * qd < p.m) {
                        if (p.add) tma_add_3d(&tm_out, piece, (int)col0 + c, (int)(T.mt * BM) + 32 * qd, T.ks);
                        else tma_store_3d(&tm_out, piece, (int)col0 + c, (int)(T.mt * BM) + 32 * qd, T.ks);
                        bulk_commit();
                    }
                }
            } else {
                const int parts = EPI == EPI_GRAD ? p.n_parts : 1;
                // g is stored over whole tiles (0 past the vocabulary); a bf16
                // output only where it has columns
                const int ncol = EPI == EPI_GRAD ? HALF : nv;
                for (int part = 0; part < parts; ++part) {
#pragma unroll
                    for (int pc = 0; pc < HALF / 64; ++pc) {
                        if (pc * 64 >= ncol) break;
                        if (lane == 0) bulk_wait_read0();
                        __syncwarp();
#pragma unroll
                        for (int hh = 0; hh < 2; ++hh) {
                            const int c = pc * 64 + hh * 32;
                            uint32_t r[32], w[16];
                            tmem_ld_x32(taddr + c, r);
                            tmem_ld_wait();
                            if constexpr (EPI == EPI_GRAD) {
                                float g[32];
#pragma unroll
                                for (int i = 0; i < 32; ++i) {
                                    const float pv = ex2(fmaf(__uint_as_float(r[i]), kLog2e, -lse2));
                                    g[i] = c + i < nv ? wt * (tl == c + i ? pv - 1.f : pv) : 0.f;
                                }
                                if (lse2 == INFINITY) {        // padding, whatever its logits are
#pragma unroll
                                    for (int i = 0; i < 32; ++i) g[i] = 0.f;
                                }
                                if (part > 0) {
#pragma unroll
                                    for (int i = 0; i < 32; ++i) g[i] = bf16_part(g[i], part);
                                }
#pragma unroll
                                for (int i = 0; i < 16; ++i) w[i] = pack2(g[2 * i], g[2 * i + 1]);
                            } else {
#pragma unroll
                                for (int i = 0; i < 16; ++i)
                                    w[i] = pack2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
                            }
#pragma unroll
                            for (int q = 0; q < 4; ++q)
                                st_shared_v4(piece + lane * 128 + (((hh * 4 + q) ^ (lane & 7)) << 4), w[4 * q],
                                             w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
                        }
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0 && T.mt * BM + 32 * qd < p.m) {
                            tma_store_3d(&tm_out, piece, (int)col0 + 64 * pc, (int)(T.mt * BM) + 32 * qd, part);
                            bulk_commit();
                        }
                    }
                }
            }
            tc_fence_before();
            mbar_arrive(tempty0 + 8 * acc);
        }
        if (lane == 0) bulk_wait0();
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem_base, TMEM_COLS);
    }
}

// ------------------------------------------------------------ small kernels
// Joins the half tiles' (maximum, sum) of 32 rows: 8 warps take a strided
// eighth of the tiles each (lane = row), then the eight are joined in order.
__device__ __forceinline__ void lse_join(float& m, float& s, float m2, float s2) {
    if (s2 == 0.f) return;                        // nothing but -inf
    const float mx = fmaxf(m, m2);
    s = s * (m == mx ? 1.f : ex2((m - mx) * kLog2e)) + s2 * (m2 == mx ? 1.f : ex2((m2 - mx) * kLog2e));
    m = mx;
}
__global__ void __launch_bounds__(256) logsumexp_kernel(const float2* partials, int n_part, int64_t rows, int64_t row0,
                                                        const float* zt, const int32_t* targets, int64_t vocab,
                                                        float* loss, float* lse, float2* sums, void* ws) {
    __shared__ float2 sh[8][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t row = (int64_t)blockIdx.x * 32 + lane;
    float m = -INFINITY, s = 0.f;
    if (row < rows) {
#pragma unroll 4
        for (int q = warp; q < n_part; q += 8) {
            const float2 v = partials[(int64_t)q * rows + row];
            lse_join(m, s, v.x, v.y);
        }
    }
    sh[warp][lane] = make_float2(m, s);
    __syncthreads();
    if (warp != 0) return;
#pragma unroll
    for (int w = 1; w < 8; ++w) lse_join(m, s, sh[w][lane].x, sh[w][lane].y);
    float l = 0.f, n = 0.f;
    if (row < rows) {
        const float ls = m + log2f(s) * kLn2;
        const int64_t tg = targets[row];
        if (tg >= vocab) record_error(ws, MOM_DEVERR_TARGET, row0 + row);
        if (tg >= 0 && tg < vocab) {
            l = ls - zt[row];
            n = 1.f;
        }
        lse[row] = ls;
        loss[row] = l;
    }
    l = warp_sum(l);
    n = warp_sum(n);
    if (lane == 0) sums[row0 / 32 + blockIdx.x] = make_float2(l, n);
}
// mean[0] = sum of losses / rows counted, mean[1] = 1 / rows counted
__global__ void __launch_bounds__(1024) mean_loss_kernel(const float2* sums, int64_t n, float* mean) {
    __shared__ double sl[32], sn[32];
    double l = 0.0, c = 0.0;
    for (int64_t i = threadIdx.x; i < n; i += 1024) {
        const float2 v = sums[i];
        l += v.x;
        c += v.y;
    }
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        l += __shfl_xor_sync(0xffffffffu, l, o);
        c += __shfl_xor_sync(0xffffffffu, c, o);
    }
    if (lane == 0) { sl[warp] = l; sn[warp] = c; }
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < 32; ++w) { l += sl[w]; c += sn[w]; }
        mean[0] = c > 0.0 ? (float)(l / c) : 0.f;
        mean[1] = c > 0.0 ? (float)(1.0 / c) : 0.f;
    }
}

// [rows, d] -> bf16 parts [parts][rows, pitch]: rows that TMA can stride over
// (a pitch that is a multiple of 8), float32 split into its three parts.
template <typename T, int PARTS>
__global__ void __launch_bounds__(256) parts_kernel(const T* src, int64_t rows, int d, int pitch, bf16* dst) {
    const int64_t n = rows * (int64_t)d, step = (int64_t)gridDim.x * 256, part = rows * (int64_t)pitch;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += step) {
        const int64_t r = i / d;
        bf16* o = dst + r * pitch + (i - r * d);
        if constexpr (PARTS == 1) {
            *o = src[i];
        } else {
            float v = to_f(src[i]);
#pragma unroll
            for (int q = 0; q < PARTS; ++q) {
                const bf16 b = __float2bfloat16_rn(v);
                o[q * part] = b;
                v -= __bfloat162float(b);
            }
        }
    }
}
// out [rows, d] = sum over slots of in [slots][rows, pitch], in slot order
template <typename TI, typename TO>
__global__ void __launch_bounds__(256) join_kernel(const TI* in, int slots, int64_t rows, int d, int pitch, TO* out) {
    const int64_t n = rows * (int64_t)d, step = (int64_t)gridDim.x * 256, slot = rows * (int64_t)pitch;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += step) {
        const int64_t r = i / d;
        const TI* p = in + r * pitch + (i - r * d);
        float v = to_f(*p);
        for (int s = 1; s < slots; ++s) v += to_f(p[s * slot]);
        out[i] = from_f<TO>(v);
    }
}

// ------------------------------------------------------------------- host
inline int64_t up(int64_t x, int64_t a) { return (x + a - 1) / a * a; }
inline size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

int sm_count() {
    int dev = 0, sms = 148;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    return sms;
}

constexpr int64_t kRowChunk = 32768;             // rows of a forward sweep (bounds its partial sums)
constexpr int64_t kPieceBytes = 512LL << 20;     // of g, and of a split or padded piece of W

struct Plan {
    int parts;             // bf16 parts of an operand
    bool direct;           // x, w, dx, dw are read and written in place by TMA
    int pitch;             // row pitch of copied operands and staged outputs (elements)
    int64_t piece;         // classes of a piece (a multiple of 256)
    int sx, sw;            // K slots of dx and dw
    bool dx_direct, dw_direct;
    size_t zt, partials, sums, xbuf, wbuf, g, dxs, dws, bytes;
};

int slots_for(int64_t tiles, int64_t kb, int sms) {
    if (2 * tiles > sms) return 1;
    int64_t s = sms / tiles;
    if (s > kb / 8) s = kb / 8;                  // at least 512 of K a slot
    if (s < 1) s = 1;
    const int64_t per = cdiv(kb, s);
    return (int)cdiv(kb, per);
}

Plan plan_for(int64_t n, int d, int64_t v, int dt, bool bwd) {
    Plan L{};
    const int sms = sm_count();
    const bool b16 = dt == MOM_BF16;
    L.parts = b16 ? 1 : 3;
    L.direct = b16 && d % 8 == 0;
    L.pitch = (int)up(d, 8);
    int64_t piece = kPieceBytes / (2 * L.parts * (n > L.pitch ? n : L.pitch)) / 256 * 256;
    if (piece < 256) piece = 256;
    const int64_t np = cdiv(v, piece);
    L.piece = up(cdiv(v, np), 256);
    size_t o = MOM_WS_HEADER_BYTES;
    auto take = [&](size_t b) { const size_t at = o; o += up256(b); return at; };
    if (!L.direct) {
        L.xbuf = take((size_t)L.parts * n * L.pitch * 2);
        L.wbuf = take((size_t)L.parts * L.piece * L.pitch * 2);
    }
    if (!bwd) {
        const int64_t rows = n < kRowChunk ? n : kRowChunk;
        L.zt = take(rows * 4);
        L.partials = take((size_t)rows * 2 * cdiv(v, BN) * 8);
        L.sums = take((size_t)cdiv(n, 32) * 8);
    } else {
        const int64_t kb = cdiv(v < L.piece ? v : L.piece, BK), tiles = cdiv(n, BM) * cdiv(d, BN);
        L.sx = slots_for(tiles, kb, sms);
        L.sw = slots_for(cdiv(L.piece, BM) * cdiv(d, BN), cdiv(n, BK), sms);
        L.dx_direct = L.sx == 1 && L.piece >= v && (b16 ? d % 8 == 0 : d % 4 == 0);
        L.dw_direct = L.sw == 1 && (b16 ? d % 8 == 0 : d % 4 == 0);
        L.g = take((size_t)L.parts * n * L.piece * 2);
        if (!L.dx_direct) L.dxs = take((size_t)L.sx * n * L.pitch * 4);
        if (!L.dw_direct) L.dws = take((size_t)L.sw * L.piece * L.pitch * 4);
    }
    L.bytes = o;
    return L;
}

template <int EPI, bool A_MN, bool B_MN>
cudaError_t run_gemm(const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& out, GemmArgs p, int splits,
                     int parts, cudaStream_t st) {
    p.m_tiles = cdiv(p.m, BM);
    p.n_tiles = cdiv(p.n, BN);
    p.kb_split = (int)cdiv(p.kb_total, splits);
    p.tiles = p.m_tiles * p.n_tiles * splits;
    if (parts == 1) {
        p.n_pairs = 1;
        p.pa[0] = p.pb[0] = 0;
    } else {
        static const uint8_t A6[6] = {2, 1, 0, 1, 0, 0}, B6[6] = {0, 1, 2, 0, 1, 0};
        p.n_pairs = 6;
        for (int i = 0; i < 6; ++i) { p.pa[i] = A6[i]; p.pb[i] = B6[i]; }
    }
    static unsigned long long optin_done = 0;
    auto* k = ce_gemm_kernel<EPI, A_MN, B_MN>;
    cudaError_t e = smem_optin((const void*)k, (int)SMEM_BYTES, &optin_done);
    if (e != cudaSuccess) return e;
    const int sms = sm_count();
    k<<<(unsigned)(p.tiles < sms ? p.tiles : sms), THREADS, SMEM_BYTES, st>>>(a, b, out, p);
    count_launches(1);
    return cudaGetLastError();
}

unsigned ew_grid(int64_t n) {
    const int64_t b = cdiv(n, 256), most = (int64_t)sm_count() * 16;
    return (unsigned)(b < most ? b : most);
}

cudaError_t to_parts(const void* src, int dt, int64_t rows, int d, int pitch, void* dst, cudaStream_t st) {
    bf16* o = reinterpret_cast<bf16*>(dst);
    if (dt == MOM_BF16) parts_kernel<bf16, 1><<<ew_grid(rows * d), 256, 0, st>>>(reinterpret_cast<const bf16*>(src), rows, d, pitch, o);
    else parts_kernel<float, 3><<<ew_grid(rows * d), 256, 0, st>>>(reinterpret_cast<const float*>(src), rows, d, pitch, o);
    count_launches(1);
    return cudaGetLastError();
}

// the piece of W from class v0 on as a TMA operand: in place, or copied
struct WPiece {
    const void* base;
    uint64_t rows, pitch;
    int row0;
};
cudaError_t w_piece(const LinearCeArgs& a, const Plan& L, int64_t v0, int64_t pw, WPiece& w, cudaStream_t st) {
    if (L.direct) {
        w = WPiece{a.w, (uint64_t)a.v, (uint64_t)a.d, (int)v0};
        return cudaSuccess;
    }
    char* buf = reinterpret_cast<char*>(a.ws) + L.wbuf;
    w = WPiece{buf, (uint64_t)pw, (uint64_t)L.pitch, 0};
    const size_t es = a.dt == MOM_BF16 ? 2 : 4;
    return to_parts(reinterpret_cast<const char*>(a.w) + (size_t)v0 * a.d * es, a.dt, pw, a.d, L.pitch, buf, st);
}

#define MOM_TRY(x) do { const cudaError_t e_ = (x); if (e_ != cudaSuccess) return e_; } while (0)
#define MOM_MAP(x) do { if (!(x)) return cudaErrorInvalidValue; } while (0)

}  // namespace

size_t linear_ce_workspace_bytes(int64_t n, int d, int64_t v, int dt, bool bwd) {
    return plan_for(n > 0 ? n : 1, d, v, dt, bwd).bytes;
}

cudaError_t launch_linear_ce_fwd(const LinearCeArgs& a, cudaStream_t st) {
    const Plan L = plan_for(a.n, a.d, a.v, a.dt, false);
    char* ws = reinterpret_cast<char*>(a.ws);
    if (!L.direct) MOM_TRY(to_parts(a.x, a.dt, a.n, a.d, L.pitch, ws + L.xbuf, st));
    const void* xb = L.direct ? a.x : ws + L.xbuf;
    const int n_part = (int)(2 * cdiv(a.v, BN));
    float2* partials = reinterpret_cast<float2*>(ws + L.partials);
    float* zt = reinterpret_cast<float*>(ws + L.zt);
    for (int64_t r0 = 0; r0 < a.n; r0 += kRowChunk) {
        const int64_t rows = a.n - r0 < kRowChunk ? a.n - r0 : kRowChunk;
        CUtensorMap ma, mb;
        // the chunk's rows: a map that starts at r0; the parts lie n rows apart
        MOM_MAP(make_tma_3d(&ma, reinterpret_cast<const bf16*>(xb) + r0 * L.pitch, false, a.d, rows, L.parts, L.pitch,
                            BM, a.n));
        for (int64_t v0 = 0; v0 < a.v; v0 += L.direct ? a.v : L.piece) {
            const int64_t pw = L.direct ? a.v : a.v - v0 < L.piece ? a.v - v0 : L.piece;
            WPiece w;
            MOM_TRY(w_piece(a, L, v0, pw, w, st));
            MOM_MAP(make_tma_3d(&mb, w.base, false, a.d, w.rows, L.parts, w.pitch, BN));
            GemmArgs p{};
            p.m = rows;
            p.n = pw;
            p.kb_total = (int)cdiv(a.d, BK);
            p.b_row0 = w.row0;
            p.targets = a.targets + r0;
            p.v0 = v0;
            p.vocab = a.v;
            p.partials = partials + v0 / BN * 2 * rows;
            p.zt = zt;
            p.ws = a.ws;
            MOM_TRY((run_gemm<EPI_STATS, false, false>(ma, mb, ma, p, 1, L.parts, st)));
        }
        logsumexp_kernel<<<(unsigned)cdiv(rows, 32), 256, 0, st>>>(partials, n_part, rows, r0, zt, a.targets + r0, a.v,
                                                                   a.loss + r0, a.lse + r0,
                                                                   reinterpret_cast<float2*>(ws + L.sums), a.ws);
        count_launches(1);
        MOM_TRY(cudaGetLastError());
    }
    if (a.mean) {
        mean_loss_kernel<<<1, 1024, 0, st>>>(reinterpret_cast<const float2*>(ws + L.sums), cdiv(a.n, 32), a.mean);
        count_launches(1);
    }
    return cudaGetLastError();
}

cudaError_t launch_linear_ce_bwd(const LinearCeArgs& a, cudaStream_t st) {
    const Plan L = plan_for(a.n, a.d, a.v, a.dt, true);
    const bool b16 = a.dt == MOM_BF16;
    const size_t es = b16 ? 2 : 4;
    char* ws = reinterpret_cast<char*>(a.ws);
    if (!L.direct) MOM_TRY(to_parts(a.x, a.dt, a.n, a.d, L.pitch, ws + L.xbuf, st));
    const void* xb = L.direct ? a.x : ws + L.xbuf;
    CUtensorMap mx_k, mx_mn;       // x: K-major rows of the logits; MN-major rows (K = tokens) of dw
    MOM_MAP(make_tma_3d(&mx_k, xb, false, a.d, a.n, L.parts, L.pitch, BM));
    MOM_MAP(make_tma_3d(&mx_mn, xb, false, a.d, a.n, L.parts, L.pitch, BK));
    for (int64_t v0 = 0; v0 < a.v; v0 += L.piece) {
        const int64_t pw = a.v - v0 < L.piece ? a.v - v0 : L.piece;
        WPiece w;
        MOM_TRY(w_piece(a, L, v0, pw, w, st));
        CUtensorMap mw_k, mw_mn, mg_st, mg_k, mg_mn, mo;
        MOM_MAP(make_tma_3d(&mw_k, w.base, false, a.d, w.rows, L.parts, w.pitch, BN));
        MOM_MAP(make_tma_3d(&mw_mn, w.base, false, a.d, w.rows, L.parts, w.pitch, BK));
        MOM_MAP(make_tma_3d(&mg_st, ws + L.g, false, L.piece, a.n, L.parts, L.piece, 32));
        MOM_MAP(make_tma_3d(&mg_k, ws + L.g, false, L.piece, a.n, L.parts, L.piece, BM));
        MOM_MAP(make_tma_3d(&mg_mn, ws + L.g, false, L.piece, a.n, L.parts, L.piece, BK));
        {   // g of the piece
            GemmArgs p{};
            p.m = a.n;
            p.n = pw;
            p.kb_total = (int)cdiv(a.d, BK);
            p.b_row0 = w.row0;
            p.targets = a.targets;
            p.v0 = v0;
            p.vocab = a.v;
            p.lse = a.lse;
            p.dloss = a.dloss;
            p.dscale = a.dscale;
            p.n_parts = L.parts;
            p.ws = a.ws;
            MOM_TRY((run_gemm<EPI_GRAD, false, false>(mx_k, mw_k, mg_st, p, 1, L.parts, st)));
        }
        {   // dx (+)= g W
            GemmArgs p{};
            p.m = a.n;
            p.n = a.d;
            p.kb_total = (int)cdiv(pw, BK);
            p.b_row0 = w.row0;
            p.add = v0 > 0;
            p.ws = a.ws;
            const int64_t per = cdiv(p.kb_total, L.sx);
            const int splits = (int)cdiv(p.kb_total, per);       // a short last piece may fill fewer slots
            if (L.dx_direct && b16) {
                MOM_MAP(make_tma_3d(&mo, a.dx, false, a.d, a.n, 1, a.d, 32));
                MOM_TRY((run_gemm<EPI_BF16, false, true>(mg_k, mw_mn, mo, p, 1, L.parts, st)));
            } else {
                void* out = L.dx_direct ? a.dx : ws + L.dxs;
                MOM_MAP(make_tma_3d(&mo, out, true, a.d, a.n, L.sx, L.dx_direct ? a.d : L.pitch, 32));
                MOM_TRY((run_gemm<EPI_F32, false, true>(mg_k, mw_mn, mo, p, splits, L.parts, st)));
            }
        }
        {   // dw = g^T x
            GemmArgs p{};
            p.m = pw;
            p.n = a.d;
            p.kb_total = (int)cdiv(a.n, BK);
            p.ws = a.ws;
            char* dw = reinterpret_cast<char*>(a.dw) + (size_t)v0 * a.d * es;
            if (L.dw_direct && b16) {
                MOM_MAP(make_tma_3d(&mo, dw, false, a.d, pw, 1, a.d, 32));
                MOM_TRY((run_gemm<EPI_BF16, true, true>(mg_mn, mx_mn, mo, p, 1, L.parts, st)));
            } else {
                void* out = L.dw_direct ? dw : ws + L.dws;
                MOM_MAP(make_tma_3d(&mo, out, true, a.d, pw, L.sw, L.dw_direct ? a.d : L.pitch, 32));
                MOM_TRY((run_gemm<EPI_F32, true, true>(mg_mn, mx_mn, mo, p, L.sw, L.parts, st)));
                if (!L.dw_direct) {
                    const float* in = reinterpret_cast<const float*>(ws + L.dws);
                    if (b16) join_kernel<float, bf16><<<ew_grid(pw * a.d), 256, 0, st>>>(in, L.sw, pw, a.d, L.pitch, reinterpret_cast<bf16*>(dw));
                    else join_kernel<float, float><<<ew_grid(pw * a.d), 256, 0, st>>>(in, L.sw, pw, a.d, L.pitch, reinterpret_cast<float*>(dw));
                    count_launches(1);
                    MOM_TRY(cudaGetLastError());
                }
            }
        }
    }
    if (!L.dx_direct) {
        const float* in = reinterpret_cast<const float*>(ws + L.dxs);
        if (b16) join_kernel<float, bf16><<<ew_grid(a.n * a.d), 256, 0, st>>>(in, L.sx, a.n, a.d, L.pitch, reinterpret_cast<bf16*>(a.dx));
        else join_kernel<float, float><<<ew_grid(a.n * a.d), 256, 0, st>>>(in, L.sx, a.n, a.d, L.pitch, reinterpret_cast<float*>(a.dx));
        count_launches(1);
    }
    return cudaGetLastError();
}

}  // namespace mom
