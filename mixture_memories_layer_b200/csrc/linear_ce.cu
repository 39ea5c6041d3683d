// Softmax cross entropy of the logits z = x W^T over a large vocabulary, and
// its gradient, on the tcgen05 tensor cores without storing the logits.
//
//   forward   m_t = max_v z_tv,  lse_t = m_t + log sum_v exp(z_tv - m_t),
//             loss_t = (m_t - z_t,target) + log sum_v exp(z_tv - m_t)
//   backward  g_tv = exp(z_tv - lse_t) - [v = target_t],
//             (times the row's weight),  dx = r g W,  dW = r g^T x
//
// One persistent GEMM kernel runs all four products; they differ in the
// operands' majors and in what happens to an accumulator tile:
//   STATS  x W^T      each row's running maximum and sum of exponentials over
//                     the tile's columns (float32, one pass over TMEM), and
//                     the target's logit; logsumexp_kernel joins the tiles
//   GRAD   x W^T      the logits of one piece of the vocabulary again, made
//                     into g and stored as bf16
//   OUT    g W, g^T x both products of a piece in one launch
// Rows without a target take no part in the gradient: gather_kernel packs the
// rows that have one, in order, and the later kernels read their number on the
// device, so a batch that is mostly padding costs what its targets cost.
//
// The common factor r (1 / rows for the mean loss) multiplies the sums, in
// float32, as they are stored: in a bf16 g it would give every -1 of g the
// same relative error, up to 2^-8 of the whole gradient (16384 rows, 32000
// classes: 0.0030 of the gradient's norm, and 0.0017, the output's own
// rounding, without).  Weights that differ from row to row are in g.
//
// Bound by the tensor cores (2 n d v operations a product) except for few
// rows, where reading W once bounds it.  dx and dW of a piece have few, long
// tiles; schedule() deals them out so that the clusters finish together, and
// an axis so long that one tile would outlast the rest is split into slots
// that join_kernel adds in order.  No atomics on floats: results repeat.
//
// float32 operands: every finite value is split exactly into three bf16 parts, a
// = a0 + a1 + a2 (8 bits each), and the six products a_i b_j with i + j <= 2 run
// into the same accumulator, smallest first; the rest is below 2^-24 of a
// product.  The tensor core truncates as it accumulates, so a float32 tile's
// sum leaves TMEM every 128 of K and is continued in registers, rounded.
//
// Two CTAs of a cluster share a 256 x 256 tile (cta_group::2, K 16 an
// instruction): each loads its 128 rows of A and half of B, 64 bytes from L2
// for each tensor-core cycle where a CTA by itself (128 x 256) needs 96.
// Roles (320 threads): warp 0 issues the TMA loads (6 stages of K 64; float32
// 2 stages of all three parts), warp 1 of the first CTA the MMAs into one of
// two TMEM accumulators, warps 2-9 are the epilogue (two warps a TMEM lane
// quarter) and overlap the next tile's main loop.  Every wait is bounded
// (sm100.cuh).
#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "rows8.cuh"
#include "sm100.cuh"

namespace mom {

namespace {

using namespace sm100;

constexpr int BM = 256, BN_MAX = 256, BK = 64;       // a cluster's tile (columns: 256 or 128)
constexpr int HM = BM / 2;                           // a CTA's rows of A, and of B
constexpr int OP_BYTES = HM * BK * 2;                // one operand part of a stage
constexpr int MN_GROUP = 64 * BK * 2;                // an MN-major box: 64 MN x 64 K, bf16
constexpr int NEPI = 256, THREADS = 64 + NEPI;
constexpr int EPI_ARRIVE = 2 * NEPI / 32;            // warps of both CTAs that free an accumulator
constexpr int PIECE = 32 * 128;                      // an epilogue warp's staging: 32 rows x 128 bytes
constexpr uint32_t TMEM_COLS = 2 * BN_MAX;
constexpr int SEG_KB = 2;                            // float32: K blocks between two reads of the accumulator
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
template <int PARTS> struct Stages { static constexpr int N = PARTS == 1 ? 6 : 2, BYTES = 2 * PARTS * OP_BYTES; };
template <int PARTS> constexpr size_t smem_bytes() {
    return 1024 + (size_t)Stages<PARTS>::N * Stages<PARTS>::BYTES + (size_t)(NEPI / 32) * PIECE + 256;
}

enum Epi { EPI_STATS, EPI_GRAD, EPI_OUT };

// One of OUT's products: [rows, d] over kb blocks of K, its slots, and where
// the result goes.
struct Prod {
    int64_t rows, row0;                  // output rows of the piece, the first one's place in `out`
    int kb, slots;
    void* out;
    int64_t ld;                          // out's row pitch, a multiple of 16 bytes (join_kernel: d)
    const int32_t* row_of;               // row -> output row (null: row0 + row)
    const float* scale;                  // r (null: 1)
    float* partial;                      // [slots][up(rows, 32) / 32][up(d, 32)][32], null: none
    int add, last;                       // add to what the partial holds; this is the last piece
};

struct GemmArgs {
    int64_t rows, cols;                  // STATS, GRAD: rows of x, classes of the piece
    int kb;                              // K blocks of d
    int b_row0;                          // W's first row
    const int32_t* live;                 // GRAD, OUT: number of packed rows (device)
    const int32_t* targets;
    int64_t v0, vocab;                   // the piece's first class
    float2* partials;                    // [column half tiles][rows]
    float* zt;                           // the targets' logits
    bf16* g;                             // GRAD: [parts][.., g_pitch], the parts g_part elements apart
    int64_t g_pitch, g_part;
    const float *lse, *weight;           // GRAD: lse of the packed rows, their weights (null: 1)
    int32_t* ticket;                     // STATS: set to 0 for logsumexp_kernel
    // OUT: dx (rows and K of dw follow `live`), dw
    Prod dx, dw;
    int d;
    void* ws;
};

__device__ __forceinline__ void st_shared_v4(uint32_t dst, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(dst), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&h);
}
// one 32-byte sector
__device__ __forceinline__ void st_global_32(bf16* dst, const uint32_t* v) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
                 ::"l"(dst), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

// The launches of one call follow each other with programmatic stream
// serialization: a kernel's launch and prologue overlap the end of the one
// before, and everything that touches memory comes after this (TMA reads what
// that kernel wrote by plain stores, hence the fence).  Letting the next kernel
// in from the start of this one gains 0.5 % on large calls and loses 3 us of 50
// on small ones.
__device__ __forceinline__ void after_previous() {
    asm volatile("griddepcontrol.wait;\n\tfence.proxy.async.global;" ::: "memory");
}

// ------------------------------------------------------- CTA pairs --
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// the address of this CTA's `addr` in the cluster's first CTA
__device__ __forceinline__ uint32_t leader_addr(uint32_t addr) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(addr));
    return r;
}
// An accumulator is free: what is passed on is the end of reads from TMEM, which
// tcgen05.wait::ld and the fence before this order.  A release of cluster scope
// would wait for the warp's global stores as well (OUT's tiles with one token:
// 6400 cycles each instead of 5100).
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t addr) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}
// a box of this CTA's shared memory, counted on a barrier of either CTA
__device__ __forceinline__ void pair_load_3d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0, int c1,
                                             int c2) {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%3, %4, %5}], [%2];"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
        : "memory");
}
__device__ __forceinline__ void pair_tmem_alloc(uint32_t dst_smem, uint32_t ncols) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem), "r"(ncols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void pair_tmem_dealloc(uint32_t taddr, uint32_t ncols) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
__device__ __forceinline__ void pair_umma(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                          uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}"
        ::"r"(d_tmem), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// arrives on the barrier at this offset in both CTAs when the MMAs so far are done
__device__ __forceinline__ void pair_commit(uint32_t bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
        ::"r"(bar), "h"((uint16_t)3)
        : "memory");
}

// ---------------------------------------------------------- scheduling --
struct Tile {
    int dw;                              // OUT: the product
    int mt, nt, ks, kb0, kb1;
};

// Tile j of cluster c among n; false past its last one.  OUT: the product with
// the longer tiles first, round robin; the clusters that got one fewer take
// the head start of as many of the other's tiles as last as long as one, and
// the rest goes round robin, those clusters first.  Closed form, so that every
// role walks the same list, in 32 bits: 64-bit divisions for each tile cost 2-3 %
// (a call by itself: 2047 tokens, d 1024, 65003 classes 738 us, 722 without; 4096
// tokens, d 64, 30000 classes 237 and 230).
struct Schedule {
    uint32_t c, n, m1, m2, n_tiles, na, nb, head, first, own;
    int kb1, kb2, k1, k2, dw_first;
    __device__ __forceinline__ Schedule(const GemmArgs& p, int epi, int parts, int bn) {
        c = blockIdx.x >> 1;
        n = gridDim.x >> 1;
        const uint32_t live = (uint32_t)(p.live ? *p.live : p.rows);
        m1 = (live + BM - 1) / BM;
        dw_first = 0;
        if (epi != EPI_OUT) {
            n_tiles = (uint32_t)cdiv(p.cols, bn);
            na = m1 * n_tiles;
            k1 = p.kb;
            return;
        }
        n_tiles = ((uint32_t)p.d + bn - 1) / bn;
        m2 = (uint32_t)cdiv(p.dw.rows, BM);
        kb1 = p.dx.kb;
        kb2 = (int)((live + BK - 1) / BK);
        k1 = (kb1 + p.dx.slots - 1) / p.dx.slots;
        k2 = (kb2 + p.dw.slots - 1) / p.dw.slots;
        dw_first = k2 > k1;
        const uint32_t n1 = m1 * n_tiles * p.dx.slots, n2 = m2 * n_tiles * p.dw.slots;
        na = dw_first ? n2 : n1;
        nb = dw_first ? n1 : n2;
        first = na % n;                            // clusters that get one more
        own = na / n + (c < first ? 1 : 0);        // this one's tiles of the first product
        // (an epilogue lasts about 4 K blocks, or one of six products each)
        const int e = parts == 1 ? 4 : 1;
        head = first ? (dw_first ? (k2 + e) / (k1 + e) : (k1 + e) / (k2 + e)) : 0;
    }
    __device__ __forceinline__ bool at(int epi, uint32_t j, Tile& T) const {
        uint32_t t = c + j * n;
        if (epi != EPI_OUT) {
            if (t >= na) return false;
            T.dw = 0;
            T.ks = 0;
            T.kb0 = 0;
            T.kb1 = k1;
            T.nt = t / m1;
            T.mt = t - T.nt * m1;                  // rows fastest: a wave shares few column tiles of W
            return true;
        }
        T.dw = dw_first;
        if (j >= own) {
            T.dw = 1 - dw_first;
            const uint32_t light = n - first, i = j - own;
            if (c >= first && i < head) t = i * light + (c - first);
            else t = head * light + (c >= first ? (i - head) * n + (c - first) : i * n + light + c);
            if (t >= nb) return false;
        }
        const uint32_t r = t / n_tiles, m = T.dw ? m2 : m1;
        T.nt = t - r * n_tiles;
        const int k = T.dw ? k2 : k1, kb = T.dw ? kb2 : kb1;
        T.ks = r / m;
        T.mt = r - T.ks * m;
        T.kb0 = T.ks * k;
        T.kb1 = T.kb0 + k < kb ? T.kb0 + k : kb;
        return true;
    }
};

// ------------------------------------------------------------- outputs --
// Tiles' rows go to memory through the warp's staging, 32 columns of 32 rows at
// a time, so that a store covers whole sectors: a row is 2 sizeof(T) chunks of
// 16 bytes, and lane l moves chunk l % Q of rows l / Q, + 32 / Q, ..
template <typename T> struct Emit {
    static constexpr int Q = 2 * sizeof(T), E = 16 / sizeof(T), RI = 32 / Q;
    int32_t to[Q];                                 // output rows of the lane's chunks (< 0: none)
    __device__ __forceinline__ void rows(int32_t row, int lane) {      // row: lane's row of the tile
#pragma unroll
        for (int it = 0; it < Q; ++it) to[it] = __shfl_sync(0xffffffffu, row, it * RI + lane / Q);
    }
    static __device__ __forceinline__ uint32_t at(uint32_t piece, int r, int q) {
        return piece + r * (16 * Q) + ((sizeof(T) == 4 ? q ^ (r & 7) : q ^ ((r >> 1) & 3)) << 4);
    }
    // v: lane's row's columns from `col` on, into out [.., ld], up to the last
    // 16 bytes that hold a column below d
    __device__ __forceinline__ void put(T* out, int64_t ld, int d, int64_t col, const float* v, uint32_t piece,
                                        int lane) const {
        __syncwarp();
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            if constexpr (sizeof(T) == 4)
                st_shared_v4(at(piece, lane, q), __float_as_uint(v[4 * q]), __float_as_uint(v[4 * q + 1]),
                             __float_as_uint(v[4 * q + 2]), __float_as_uint(v[4 * q + 3]));
            else
                st_shared_v4(at(piece, lane, q), pack2(v[8 * q], v[8 * q + 1]), pack2(v[8 * q + 2], v[8 * q + 3]),
                             pack2(v[8 * q + 4], v[8 * q + 5]), pack2(v[8 * q + 6], v[8 * q + 7]));
        }
        __syncwarp();
        const int q = lane % Q;
        uint4 u[Q];
#pragma unroll
        for (int it = 0; it < Q; ++it)
            asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                         : "=r"(u[it].x), "=r"(u[it].y), "=r"(u[it].z), "=r"(u[it].w)
                         : "r"(at(piece, it * RI + lane / Q, q)));
        if (col + q * E >= d) return;
        T* o = out + col + q * E;
#pragma unroll
        for (int it = 0; it < Q; ++it)
            if (to[it] >= 0) *reinterpret_cast<uint4*>(o + to[it] * ld) = u[it];
    }
};

// A partial's element of row block rb, column col, lane 0.
__device__ __forceinline__ float* partial_at(const Prod& q, int d, int slot, int64_t rb, int64_t col) {
    const int64_t blocks = cdiv(q.rows, 32), dp = cdiv(d, 32) * 32;
    return q.partial + ((slot * blocks + rb) * dp + col) * 32;
}

template <int PARTS, int EPI, int BN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS, 1)
ce_gemm_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
               const __grid_constant__ CUtensorMap tm_a2, const __grid_constant__ CUtensorMap tm_b2,
               const GemmArgs p) {
    constexpr int STAGES = Stages<PARTS>::N, STAGE_BYTES = Stages<PARTS>::BYTES;
    constexpr bool SEG = PARTS == 3;
    typedef typename std::conditional<PARTS == 1, bf16, float>::type OT;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* smem = align1024_shared(smem_raw);
    unsigned char* sOut = smem + STAGES * STAGE_BYTES;
    uint64_t* bars = reinterpret_cast<uint64_t*>(sOut + (NEPI / 32) * PIECE);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * STAGES + 5);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const uint32_t full0 = smem_u32(bars), empty0 = smem_u32(bars + STAGES);
    const uint32_t tfull0 = smem_u32(bars + 2 * STAGES), tempty0 = smem_u32(bars + 2 * STAGES + 2);
    const uint32_t done_bar = smem_u32(bars + 2 * STAGES + 4);
    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(full0 + 8 * s, 1);           // of the first CTA: both CTAs' loads
            mbar_init(empty0 + 8 * s, 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(tfull0 + 8 * a, 1);
            mbar_init(tempty0 + 8 * a, EPI_ARRIVE);      // of the first CTA: both epilogues
        }
        mbar_init(done_bar, 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 1) pair_tmem_alloc(smem_u32(tmem_slot), TMEM_COLS);
    tc_fence_before();
    __syncthreads();
    cluster_sync();                                // the other CTA's barriers are ready
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    after_previous();
    if (EPI == EPI_STATS && p.ticket && blockIdx.x == 0 && threadIdx.x == 0) *p.ticket = 0;
    const Schedule S(p, EPI, PARTS, BN);
    Tile T;

    if (warp == 0) {
        if (lane == 0) {
            // ---------------------------------------------------- TMA loads
            const uint32_t full_lead = leader_addr(full0);
            constexpr int groups = BN / 128;
            constexpr uint32_t stage_tx = 2 * PARTS * (OP_BYTES + BN / 2 * BK * 2);
            uint32_t it = 0;
            bool ok = true;
            for (uint32_t j = 0; ok && S.at(EPI, j, T); ++j) {
                const int m0 = T.mt * BM + HM * (int)rank;
                const int n0 = T.nt * BN + BN / 2 * (int)rank;
                for (int kb = T.kb0; kb < T.kb1; ++kb, ++it) {
                    const uint32_t s = it % STAGES, ph = (it / STAGES) & 1;
                    if (!mbar_wait(empty0 + 8 * s, ph ^ 1, abort_flag, p.ws, 1)) { ok = false; break; }
                    if (rank == 0) mbar_arrive_expect_tx(full0 + 8 * s, stage_tx);
                    const uint32_t bar = full_lead + 8 * s;
                    const uint32_t a0 = smem_u32(smem + s * STAGE_BYTES), b0 = a0 + PARTS * OP_BYTES;
#pragma unroll
                    for (int q = 0; q < PARTS; ++q) {
                        if constexpr (EPI == EPI_OUT) {
                            if (T.dw) {
                                pair_load_3d(a0 + q * OP_BYTES, &tm_a2, bar, m0, kb * BK, q);
                                pair_load_3d(a0 + q * OP_BYTES + MN_GROUP, &tm_a2, bar, m0 + 64, kb * BK, q);
                                for (int g = 0; g < groups; ++g)
                                    pair_load_3d(b0 + q * OP_BYTES + g * MN_GROUP, &tm_b2, bar, n0 + 64 * g, kb * BK, q);
                            } else {
                                pair_load_3d(a0 + q * OP_BYTES, &tm_a, bar, kb * BK, m0, q);
                                for (int g = 0; g < groups; ++g)
                                    pair_load_3d(b0 + q * OP_BYTES + g * MN_GROUP, &tm_b, bar, n0 + 64 * g,
                                                 p.b_row0 + kb * BK, q);
                            }
                        } else {
                            pair_load_3d(a0 + q * OP_BYTES, &tm_a, bar, kb * BK, m0, q);
                            pair_load_3d(b0 + q * OP_BYTES, &tm_b, bar, kb * BK, p.b_row0 + n0, q);
                        }
                    }
                }
            }
            if (!ok && rank == 0)      // loads still in flight must land before the CTAs exit
                for (uint32_t j = it >= STAGES ? it - STAGES : 0; j < it; ++j)
                    mbar_wait_drain(full0 + 8 * (j % STAGES), (j / STAGES) & 1);
        }
    } else if (warp == 1) {
        if (lane == 0 && rank == 0) {
            // --------------------------------------------------- MMA issuer
            uint32_t it = 0, tc = 0;
            bool ok = true;
            for (uint32_t j = 0; ok && S.at(EPI, j, T); ++j) {
                const bool a_mn = EPI == EPI_OUT && T.dw;
                const uint32_t idesc = idesc_bf16_f32(BM, BN, a_mn, EPI == EPI_OUT);
                const int seg = SEG ? SEG_KB : T.kb1 - T.kb0;
                for (int k0 = T.kb0; ok && k0 < T.kb1; k0 += seg, ++tc) {
                    const uint32_t acc = tc & 1, aph = (tc >> 1) & 1;
                    if (!mbar_wait(tempty0 + 8 * acc, aph ^ 1, abort_flag, p.ws, 2)) { ok = false; break; }
                    tc_fence_after();
                    const uint32_t d_tmem = tmem_base + acc * BN_MAX;
                    const int k1 = k0 + seg < T.kb1 ? k0 + seg : T.kb1;
                    for (int kb = k0; kb < k1; ++kb, ++it) {
                        const uint32_t s = it % STAGES, ph = (it / STAGES) & 1;
                        if (!mbar_wait(full0 + 8 * s, ph, abort_flag, p.ws, 3)) { ok = false; break; }
                        tc_fence_after();
                        const uint32_t a0 = smem_u32(smem + s * STAGE_BYTES), b0 = a0 + PARTS * OP_BYTES;
                        constexpr int PAIRS = PARTS == 1 ? 1 : 6;
                        constexpr int PA[6] = {PARTS == 1 ? 0 : 2, 1, 0, 1, 0, 0}, PB[6] = {0, 1, 2, 0, 1, 0};
#pragma unroll
                        for (int pr = 0; pr < PAIRS; ++pr) {
#pragma unroll
                            for (int i = 0; i < BK / 16; ++i) {
                                const uint32_t a = a0 + PA[pr] * OP_BYTES, b = b0 + PB[pr] * OP_BYTES;
                                const uint64_t da = a_mn ? desc_mnmajor_sw128(a + 2048 * i, MN_GROUP)
                                                         : desc_kmajor_sw128(a + 32 * i);
                                const uint64_t db = EPI == EPI_OUT ? desc_mnmajor_sw128(b + 2048 * i, MN_GROUP)
                                                                   : desc_kmajor_sw128(b + 32 * i);
                                pair_umma(d_tmem, da, db, idesc, kb != k0 || (pr | i) != 0);
                            }
                        }
                        pair_commit(empty0 + 8 * s);
                    }
                    if (ok) pair_commit(tfull0 + 8 * acc);
                }
            }
            // every MMA of the pair has finished before TMEM is released
            pair_commit(done_bar);
            mbar_wait_drain(done_bar, 0);
        }
    } else {
        // ------------------------------------------------------- epilogue
        // warp 2 + e: TMEM lanes 32 (warp % 4) .. + 31, half e / 4 of the tile's columns
        const int e = warp - 2, qd = warp & 3, hf = e >> 2;
        constexpr int half = BN / 2;
        const uint32_t piece = smem_u32(sOut + e * PIECE);
        const uint32_t lead_tempty = leader_addr(tempty0);
        const int64_t live = p.live ? *p.live : p.rows;
        const float scale = EPI == EPI_OUT && p.dx.scale ? *p.dx.scale : 1.f;      // (of dw as well)
        uint32_t tc = 0;
        bool ok = true;
        for (uint32_t j = 0; S.at(EPI, j, T); ++j) {
            const int64_t row = (int64_t)T.mt * BM + HM * rank + 32 * qd + lane;
            const int64_t col0 = (int64_t)T.nt * BN + hf * half;
            int tl = -1;                           // the target's column inside this half tile (< 0: not here)
            float lse = 0.f, wt = 1.f;
            if constexpr (EPI != EPI_OUT) {
                if (row < live) {
                    const int64_t tg = p.targets[row], rel = tg - p.v0 - col0;
                    if (tg >= 0 && tg < p.vocab && rel >= 0 && rel < half) tl = (int)rel;
                    if constexpr (EPI == EPI_GRAD) {
                        lse = p.lse[row];
                        if (p.weight) wt = p.weight[row];
                    }
                }
            }
            // float32: the tile's sum, continued in registers
            float sum[SEG ? half : 1];
            uint32_t acc = tc & 1;
            if constexpr (SEG) {
#pragma unroll
                for (int i = 0; i < half; ++i) sum[i] = 0.f;
                for (int k0 = T.kb0; k0 < T.kb1; k0 += SEG_KB, ++tc) {
                    acc = tc & 1;
                    if (!mbar_wait(tfull0 + 8 * acc, (tc >> 1) & 1, abort_flag, p.ws, 4)) { ok = false; break; }
                    tc_fence_after();
                    const uint32_t ta = tmem_base + ((uint32_t)(32 * qd) << 16) + acc * BN_MAX + hf * half;
#pragma unroll
                    for (int c = 0; c < half; c += 32) {
                        uint32_t r[32];
                        tmem_ld_x32(ta + c, r);
                        tmem_ld_wait();
#pragma unroll
                        for (int i = 0; i < 32; ++i) sum[c + i] += __uint_as_float(r[i]);
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_cluster(lead_tempty + 8 * acc);
                }
            } else if (T.kb0 < T.kb1) {
                ok = mbar_wait(tfull0 + 8 * acc, (tc >> 1) & 1, abort_flag, p.ws, 4);
                tc_fence_after();
            }
            if (!ok) break;
            const uint32_t taddr = tmem_base + ((uint32_t)(32 * qd) << 16) + acc * BN_MAX + hf * half;
            // columns c .. c + 31 of the half tile (an empty K range: zeros)
            auto chunk = [&](int c, float* v) {
                if constexpr (SEG) {
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] = sum[c + i];
                } else {
                    uint32_t r[32];
                    tmem_ld_x32(taddr + c, r);
                    tmem_ld_wait();
                    const bool any = T.kb0 < T.kb1;
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] = EPI != EPI_OUT || any ? __uint_as_float(r[i]) : 0.f;
                }
            };
            if constexpr (EPI == EPI_OUT) {
                const Prod& q = T.dw ? p.dw : p.dx;
                const int64_t rows = T.dw ? q.rows : live;
                const bool final = q.last && q.slots == 1;
                Emit<OT> emit;
                if (final) {
                    int32_t to = -1;
                    if (row < rows) to = q.row_of ? q.row_of[row] : (int32_t)(q.row0 + row);
                    emit.rows(to, lane);
                }
                const int64_t rb = (int64_t)T.mt * (BM / 32) + (HM / 32) * rank + qd;
#pragma unroll
                for (int c = 0; c < half; c += 32) {
                    if (col0 + c < p.d && rb * 32 < rows) {
                        float v[32];
                        chunk(c, v);
                        if (q.partial) {
                            float* at = partial_at(q, p.d, T.ks, rb, col0 + c) + lane;
                            if (q.add) {
#pragma unroll
                                for (int i = 0; i < 32; ++i) v[i] += at[i * 32];
                            }
                            if (!final) {
#pragma unroll
                                for (int i = 0; i < 32; ++i) at[i * 32] = v[i];
                            }
                        }
                        if (final) {
#pragma unroll
                            for (int i = 0; i < 32; ++i) v[i] *= scale;
                            emit.put(reinterpret_cast<OT*>(q.out), q.ld, p.d, col0 + c, v, piece, lane);
                        }
                    }
                }
            } else {
                const int64_t left = p.cols - col0;
                const int nv = left < 0 ? 0 : left < half ? (int)left : half;      // valid columns of the half tile
                if constexpr (EPI == EPI_STATS) {
                    float m = -INFINITY, s = 0.f, zt = 0.f;
                    // 64 columns at a time where registers allow it, two loads in flight
                    // (16384 rows, d 64, 8000 classes: 62 us, 66 with 32)
                    constexpr int CW = SEG ? 32 : 64;
#pragma unroll
                    for (int c = 0; c < half; c += CW) {
                        float v[CW];
                        if constexpr (SEG) {
                            chunk(c, v);
                        } else {
                            uint32_t r0[32], r1[32];
                            tmem_ld_x32(taddr + c, r0);
                            tmem_ld_x32(taddr + c + 32, r1);
                            tmem_ld_wait();
#pragma unroll
                            for (int i = 0; i < 32; ++i) {
                                v[i] = __uint_as_float(r0[i]);
                                v[32 + i] = __uint_as_float(r1[i]);
                            }
                        }
                        if (c + CW > nv) {
#pragma unroll
                            for (int i = 0; i < CW; ++i)
                                if (c + i >= nv) v[i] = -INFINITY;
                        }
                        float mx = m;
#pragma unroll
                        for (int i = 0; i < CW; ++i) mx = fmaxf(mx, v[i]);
                        // The difference first: exact at the maximum, whose exponential is
                        // 1 however large it is, and never above 0.  (v log2e - round(mx
                        // log2e) is off by 2^-24 |mx|: inf for classes masked by -1e10.)
                        // All -inf so far: exponentials of (-inf - 0) are 0, not NaN.
                        const float sub = mx == -INFINITY ? 0.f : mx;
                        const f2 nsub = both(-sub), l2e = both(kLog2e);
                        s *= fast_ex2((m - sub) * kLog2e);
                        float s2 = 0.f;
#pragma unroll
                        for (int i = 0; i < CW; i += 2) {
                            float e0, e1;
                            split(mul2(add2(make_f2(v[i], v[i + 1]), nsub), l2e), e0, e1);
                            s += fast_ex2(e0);
                            s2 += fast_ex2(e1);
                        }
                        s += s2;
                        m = mx;
                        if (tl >= c && tl < c + CW) {
#pragma unroll
                            for (int i = 0; i < CW; ++i)
                                if (tl == c + i) zt = v[i];
                        }
                    }
                    if (row < live) {
                        p.partials[((int64_t)T.nt * 2 + hf) * p.rows + row] = make_float2(m, s);
                        if (tl >= 0) p.zt[row] = zt;
                    }
                } else {
                    // g is 0 past the vocabulary and past the packed rows, up to whole
                    // K blocks of dW (or n, past which TMA fills in zeros).  A lane
                    // writes its row in 32-byte sectors, past shared memory: the MMAs'
                    // operands and the copies that bring them take all of its bandwidth.
                    const int nvr = row < live ? nv : 0;
                    const f2 nlse = both(-lse);
                    bf16* out = p.g + row * p.g_pitch + col0;
                    const bool some = row < cdiv(live, BK) * BK && row < p.rows;
#pragma unroll
                    for (int c = 0; c < half; c += 32) {
                        float g[32];
                        chunk(c, g);
#pragma unroll
                        for (int i = 0; i < 32; i += 2) {      // (the difference first, as in STATS)
                            float e[2];
                            split(mul2(add2(make_f2(g[i], g[i + 1]), nlse), both(kLog2e)), e[0], e[1]);
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                const float pv = fast_ex2(e[k]);
                                g[i + k] = c + i + k < nvr ? wt * (tl == c + i + k ? pv - 1.f : pv) : 0.f;
                            }
                        }
#pragma unroll
                        for (int part = 0; part < PARTS; ++part) {
                            uint32_t u[16];
#pragma unroll
                            for (int i = 0; i < 16; ++i) {
                                u[i] = pack2(g[2 * i], g[2 * i + 1]);
                                if (part + 1 < PARTS) {
                                    g[2 * i] -= __uint_as_float(u[i] << 16);
                                    g[2 * i + 1] -= __uint_as_float(u[i] & 0xffff0000u);
                                }
                            }
                            if (some) {
                                st_global_32(out + part * p.g_part + c, u);
                                st_global_32(out + part * p.g_part + c + 16, u + 8);
                            }
                        }
                    }
                }
            }
            if (!SEG && T.kb0 < T.kb1) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(lead_tempty + 8 * acc);
                ++tc;
            }
        }
    }

    __syncwarp();
    if (*abort_flag) {           // the other CTA's copies into this one end in microseconds; give them a millisecond
        const long long t0 = clock64();
        while (clock64() - t0 < 2000000) {}
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();              // no CTA leaves while the other one's MMAs or arrivals need it
    if (warp == 1) {
        tc_fence_after();
        pair_tmem_dealloc(tmem_base, TMEM_COLS);
    }
}

// ------------------------------------------------------------ small kernels
// The sum of a product's slots as its rows of the output: a block for 32 rows
// x 32 columns.  A warp sums 8 columns of every fourth slot, in order and four
// at a time; the four sums are added in order.
template <typename T>
__global__ void __launch_bounds__(512) join_kernel(const Prod q, const int32_t* live, int d) {
    __shared__ float tile[4][32][33];
    after_previous();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, cw = warp & 3, sg = warp >> 2;
    const int64_t rows = live ? *live : q.rows, cb = cdiv(d, 32), total = cdiv(rows, 32) * cb;
    const float f = q.scale ? *q.scale : 1.f;
    for (int64_t u = blockIdx.x; u < total; u += gridDim.x) {
        const int64_t rb = u / cb, col = (u - rb * cb) * 32;
        const int64_t stride = partial_at(q, d, 1, 0, 0) - q.partial;
        const float* at = partial_at(q, d, 0, rb, col + 8 * cw) + lane;
        float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        for (int s = sg; s < q.slots; s += 16) {
            float w[4][8];
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int i = 0; i < 8; ++i) w[k][i] = s + 4 * k < q.slots ? at[(s + 4 * k) * stride + i * 32] : 0.f;
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] += w[k][i];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) tile[sg][lane][8 * cw + i] = v[i];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = 2 * warp + i;
            const int64_t row = rb * 32 + r;
            if (row < rows && col + lane < d) {
                const int64_t to = q.row_of ? q.row_of[row] : q.row0 + row;
                const float sum = (tile[0][r][lane] + tile[1][r][lane]) + (tile[2][r][lane] + tile[3][r][lane]);
                reinterpret_cast<T*>(q.out)[to * d + col + lane] = from_f<T>(sum * f);
            }
        }
        __syncthreads();
    }
}

// Joins the half tiles' (maximum, sum) of 32 rows: 32 warps take a strided
// part of the tiles each (lane = row), then theirs are joined in order.  The
// last block to finish (a ticket) adds up all blocks' losses, in block order.
__device__ __forceinline__ void lse_join(float& m, float& s, float m2, float s2) {
    if (s2 == 0.f) return;                        // nothing but -inf
    const float mx = fmaxf(m, m2);
    s = s * (m == mx ? 1.f : fast_ex2((m - mx) * kLog2e)) + s2 * (m2 == mx ? 1.f : fast_ex2((m2 - mx) * kLog2e));
    m = mx;
}
__global__ void __launch_bounds__(1024) logsumexp_kernel(const float2* partials, int n_part, int64_t rows, int64_t row0,
                                                         const float* zt, const int32_t* targets, int64_t vocab,
                                                         float* loss, float* lse, float2* sums, int32_t* ticket,
                                                         int64_t blocks, float* mean, void* ws) {
    __shared__ float2 sh[32][33];
    __shared__ double sl[32], sn[32];
    __shared__ bool last;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t row = (int64_t)blockIdx.x * 32 + lane;
    float m = -INFINITY, s = 0.f, z = 0.f;
    int64_t tg = -1;
    after_previous();
    if (row < rows) {
        if (warp == 0) {
            tg = targets[row];
            if (tg >= 0 && tg < vocab) z = zt[row];
        }
        for (int q = warp; q < n_part; q += 32 * 8) {
            float2 v[8];
#pragma unroll
            for (int u = 0; u < 8; ++u)
                v[u] = q + 32 * u < n_part ? partials[(int64_t)(q + 32 * u) * rows + row] : make_float2(-INFINITY, 0.f);
#pragma unroll
            for (int u = 0; u < 8; ++u) lse_join(m, s, v[u].x, v[u].y);
        }
    }
    sh[warp][lane] = make_float2(m, s);
    __syncthreads();
    // warp w joins row w's 32 parts, a fixed tree
    {
        const float2 v = sh[lane][warp];
        m = v.x;
        s = v.y;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const float m2 = __shfl_xor_sync(0xffffffffu, m, o), s2 = __shfl_xor_sync(0xffffffffu, s, o);
            float ma = (lane & o) ? m2 : m, sa = (lane & o) ? s2 : s;      // lower lane's part first, on both sides
            lse_join(ma, sa, (lane & o) ? m : m2, (lane & o) ? s : s2);
            m = ma;
            s = sa;
        }
    }
    __syncthreads();
    if (lane == 0) sh[0][warp] = make_float2(m, s);
    __syncthreads();
    if (warp == 0) {
        m = sh[0][lane].x;
        s = sh[0][lane].y;
        float l = 0.f, n = 0.f;
        if (row < rows) {
            const float ls0 = log2f(s) * kLn2, ls = m + ls0;
            if (tg >= vocab) record_error(ws, MOM_DEVERR_TARGET, row0 + row);
            if (tg >= 0 && tg < vocab) {
                l = (m - z) + ls0;        // not lse - z: far from 0 that keeps 2^-24 of the logits only
                n = 1.f;
            }
            lse[row] = ls;
            loss[row] = l;
        }
        l = warp_sum(l);
        n = warp_sum(n);
        if (lane == 0) {
            sums[row0 / 32 + blockIdx.x] = make_float2(l, n);
            __threadfence();
            last = mean && atomicAdd(ticket, 1) == blocks - 1;
        }
    }
    __syncthreads();
    if (!last) return;
    __threadfence();
    // mean[0] = sum of losses / rows counted, mean[1] = 1 / rows counted
    double l = 0.0, c = 0.0;
    for (int64_t i = threadIdx.x; i < blocks; i += 1024) {
        const float2 v = __ldcg(sums + i);
        l += v.x;
        c += v.y;
    }
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

// The first part of a float32 value is held to bf16's largest: from 3.396e38 on
// rounding would make it infinite and the rest of the value NaN.  So every
// finite value is the sum of its parts; an infinity or a NaN leaves a NaN in
// the second or third.  W: a -inf (a masked class) counts as the lowest float32
// value, since products of an infinity with the other operand's parts, of
// either sign or 0, are no longer its product with that operand.
template <bool W> __device__ __forceinline__ float split_value(float v) {
    return W && v == -INFINITY ? -3.402823466e38f : v;
}
__device__ __forceinline__ float split_first(float v) {
    constexpr float big = 3.3895313892515355e38f;      // 0x7f7f
    return fminf(fmaxf(v, -big), big);
}

// A row of d elements as its bf16 parts (each `part` elements after the one
// before) by one warp, several loads in flight.  `vec`: both rows take 16-byte
// accesses (bf16); W: a row of W.
template <typename T, int PARTS, bool W>
__device__ __forceinline__ void copy_row(const T* __restrict__ src, int d, bf16* __restrict__ dst, int64_t part, bool vec,
                                         int lane) {
    if (PARTS == 1 && vec) {
        for (int c0 = lane * 8; c0 < d; c0 += 1024) {
            uint4 v[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (c0 + 256 * k < d) v[k] = *reinterpret_cast<const uint4*>(src + c0 + 256 * k);
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (c0 + 256 * k < d) *reinterpret_cast<uint4*>(dst + c0 + 256 * k) = v[k];
        }
        return;
    }
    constexpr int U = 8;
    for (int c0 = lane * 2; c0 < d; c0 += 64 * U) {      // (pairs stay inside the pitch, which is even)
        float v[U][2];
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int c = c0 + 64 * k;
            v[k][0] = c < d ? to_f(src[c]) : 0.f;
            v[k][1] = c + 1 < d ? to_f(src[c + 1]) : 0.f;
            if constexpr (PARTS > 1) {
                v[k][0] = split_value<W>(v[k][0]);
                v[k][1] = split_value<W>(v[k][1]);
            }
        }
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int c = c0 + 64 * k;
            if (c >= d) break;
#pragma unroll
            for (int q = 0; q < PARTS; ++q) {
                const bool first = PARTS > 1 && q == 0;
                const __nv_bfloat162 b = __floats2bfloat162_rn(first ? split_first(v[k][0]) : v[k][0],
                                                               first ? split_first(v[k][1]) : v[k][1]);
                *reinterpret_cast<__nv_bfloat162*>(dst + q * part + c) = b;
                v[k][0] -= __bfloat162float(b.x);
                v[k][1] -= __bfloat162float(b.y);
            }
        }
    }
}

// [rows, d] -> bf16 parts [parts][rows, pitch]: rows that TMA can stride over
// (a pitch that is a multiple of 8), float32 split into its three parts.
template <typename T, int PARTS, bool W>
__global__ void __launch_bounds__(256) parts_kernel(const T* src, int64_t rows, int d, int pitch, bf16* dst) {
    after_previous();
    const int64_t step = (int64_t)gridDim.x * 8;
    for (int64_t r = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); r < rows; r += step)
        copy_row<T, PARTS, W>(src + r * d, d, dst + r * pitch, rows * pitch, false, threadIdx.x & 31);
}

// The rows that have a target, packed in order.  A block takes 8 rows, one a
// warp; it counts the targets before them itself (kCountRows at most; where
// there are more, count_kernel has counted whole chunks of kCountRows).
constexpr int kGatherRows = 8, kCountRows = 16384;
struct GatherArgs {
    const void* x;
    const int32_t* targets;
    const float *lse, *dloss;
    const int32_t* counts;               // null: n <= kCountRows
    int64_t n, vocab;
    int d, pitch;
    int64_t part;                        // elements between the parts
    bf16* xc;                            // the packed rows
    int32_t *targets_c, *row_of, *live;
    float *lse_c, *weight;               // lse, dloss
    void* dx;
    int64_t dx_ld;
    int vec;                             // x, xc and dx take 16-byte accesses
    void* ws;
};
__device__ __forceinline__ bool has_target(int32_t t, int64_t vocab) { return t >= 0 && t < vocab; }
__device__ __forceinline__ int block_sum(int v) {
    __shared__ int sh[8];
    v = __reduce_add_sync(0xffffffffu, v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
    __syncthreads();
    int s = 0;
#pragma unroll
    for (int w = 0; w < 8; ++w) s += sh[w];
    return s;
}
__global__ void __launch_bounds__(256) count_kernel(const int32_t* targets, int64_t n, int64_t vocab, int32_t* counts) {
    after_previous();
    const int64_t r0 = (int64_t)blockIdx.x * kCountRows, r1 = r0 + kCountRows < n ? r0 + kCountRows : n;
    int v = 0;
    for (int64_t r = r0 + threadIdx.x; r < r1; r += 256) v += has_target(targets[r], vocab);
    v = block_sum(v);
    if (threadIdx.x == 0) counts[blockIdx.x] = v;
}
template <typename T, int PARTS>
__global__ void __launch_bounds__(256) gather_kernel(const GatherArgs a) {
    after_previous();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t r0 = (int64_t)blockIdx.x * kGatherRows, chunk = r0 / kCountRows, row = r0 + warp;
    int before = 0;
    for (int64_t i = threadIdx.x; i < chunk; i += 256) before += a.counts[i];
#pragma unroll 8
    for (int64_t r = chunk * kCountRows + threadIdx.x; r < r0; r += 256) before += has_target(a.targets[r], a.vocab);
    const int32_t mine = lane < kGatherRows && r0 + lane < a.n ? a.targets[r0 + lane] : -1;
    const uint32_t in = __ballot_sync(0xffffffffu, has_target(mine, a.vocab));
    before = block_sum(before);
    const int64_t to = before + __popc(in & ((1u << warp) - 1u));
    if (row < a.n) {
        if (!((in >> warp) & 1u)) {                // dx of padding is 0
            if (lane == 0 && a.targets[row] >= 0) record_error(a.ws, MOM_DEVERR_TARGET, row);      // (>= vocab)
            T* o = reinterpret_cast<T*>(a.dx) + row * a.dx_ld;
            const float z[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            if (a.vec) for (int c = lane * 8; c < a.d; c += 256) store_vec<8>(o + c, z);
            else for (int c = lane; c < a.d; c += 32) o[c] = from_f<T>(0.f);
        } else {
            if (lane == 0) {
                a.targets_c[to] = a.targets[row];
                a.row_of[to] = (int32_t)row;
                a.lse_c[to] = a.lse[row];
                if (a.dloss) a.weight[to] = a.dloss[row];
            }
            copy_row<T, PARTS, false>(reinterpret_cast<const T*>(a.x) + row * a.d, a.d, a.xc + to * a.pitch, a.part,
                                      a.vec != 0, lane);
        }
    }
    if (r0 + kGatherRows < a.n) return;
    // the last block: the number of rows, and zeros up to whole K blocks of dW (or n)
    const int64_t live = before + __popc(in);
    if (threadIdx.x == 0) *a.live = (int32_t)live;
    for (int64_t r = live + warp; r < cdiv(live, BK) * BK && r < a.n; r += 8)
        for (int q = 0; q < PARTS; ++q)
            for (int c = lane * 2; c < a.d; c += 64)
                *reinterpret_cast<__nv_bfloat162*>(a.xc + q * a.part + r * a.pitch + c) = __floats2bfloat162_rn(0.f, 0.f);
}

// [rows, pitch] -> dense [rows, d], 16 bytes a store whatever d is: two aligned
// 16-byte loads, shifted to the elements between them (pitch is a multiple of
// 8), or single elements where a row ends.  Storing elements one by one from
// the GEMM's tiles, 64 bytes of a row at a time, wrote parts of sectors: 79 us
// for dW of 10608 x 1452 bf16 with one token, 42 us this way.
template <typename T>
__global__ void __launch_bounds__(256) flatten_kernel(const T* __restrict__ src, int64_t rows, int d, int pitch,
                                                      T* __restrict__ dst) {
    after_previous();
    constexpr int E = 16 / sizeof(T);
    const int64_t n = rows * d, step = (int64_t)gridDim.x * 256 * E;
    for (int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * E; i < n; i += step) {
        int64_t r = n <= 0xffffffffLL ? (uint32_t)i / (uint32_t)d : i / d;
        int c = (int)(i - r * d);
        const int64_t at = r * pitch + c;
        if (c + E <= d) {
            const uint4* p = reinterpret_cast<const uint4*>(src + at / E * E);
            const int off = (int)(at % E), o = off * (int)sizeof(T) / 4;      // whole words
            const uint4 a = p[0], b = off ? p[1] : a;
            const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
            uint32_t x[5];
#pragma unroll
            for (int k = 0; k < 5; ++k) x[k] = o == 0 ? w[k] : o == 1 ? w[k + 1] : o == 2 ? w[k + 2] : w[k + 3];
            if (sizeof(T) == 2 && (off & 1)) {
#pragma unroll
                for (int k = 0; k < 4; ++k) x[k] = __funnelshift_r(x[k], x[k + 1], 16);
            }
            *reinterpret_cast<uint4*>(dst + i) = make_uint4(x[0], x[1], x[2], x[3]);
        } else {
            T v[E];
#pragma unroll
            for (int e = 0; e < E; ++e) {
                if (i + e < n) v[e] = src[r * pitch + c];
                if (++c == d) { c = 0; ++r; }
            }
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (i + e < n) dst[i + e] = v[e];
        }
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
    bool direct;           // x (forward) and w are read in place by TMA
    int pitch;             // row pitch of copied operands (elements)
    int64_t piece;         // classes of a piece (a multiple of 256)
    int bn, bn_logits;     // columns of a tile: OUT; STATS or GRAD
    int sx, sw;            // K slots of dx and dw
    bool dx_partial, dw_partial;
    bool stage;            // dx and dw leave the GEMM in rows of the pitch (d's are not multiples of 16 bytes)
    size_t zt, partials, sums, ticket, xbuf, wbuf, g, dxp, dwp, dx_stage, dw_stage, targets, row_of, lse_c, weight, live, counts, bytes;
};

// Columns of the logits' tiles, 256, or 128 where the clusters then finish
// first: by the instructions' cycles (512 for 256 columns of a K block) and
// 1500 for a tile's rest.  200 tokens of 8000 classes, d 360, float32: 95 us
// with 256 (32 tiles for 74 clusters), 82 us with 128.
int columns_for(int64_t rows, int64_t cols, int d, int parts, int clusters) {
    const int64_t kb = cdiv(d, BK) * (parts == 1 ? 1 : 6), m = cdiv(rows, BM);
    auto cost = [&](int bn) { return cdiv(m * cdiv(cols, bn), clusters) * (kb * 2 * bn + 1500); };
    return cost(128) < cost(256) ? 128 : 256;
}

Plan plan_for(int64_t n, int d, int64_t v, int dt, bool bwd) {
    Plan L{};
    const int clusters = sm_count() / 2;
    const bool b16 = dt == MOM_BF16;
    L.parts = b16 ? 1 : 3;
    L.direct = b16 && d % 8 == 0;
    L.pitch = (int)up(d, 8);
    int64_t piece = kPieceBytes / (2 * L.parts * (n > L.pitch ? n : L.pitch)) / 256 * 256;
    if (piece < 256) piece = 256;
    const int64_t np = cdiv(v, piece);
    L.piece = up(cdiv(v, np), 256);
    size_t o = MOM_WS_HEADER_BYTES;      // from the workspace's first 256-byte boundary on (ws_base)
    auto take = [&](size_t b) { const size_t at = o; o += up256(b); return at; };
    if (!L.direct) L.wbuf = take((size_t)L.parts * L.piece * L.pitch * 2);
    if (!L.direct || bwd) L.xbuf = take((size_t)L.parts * n * L.pitch * 2);
    if (!bwd) {
        const int64_t rows = n < kRowChunk ? n : kRowChunk;
        L.zt = take(rows * 4);
        L.bn_logits = columns_for(rows, L.direct ? v : L.piece, d, L.parts, clusters);
        const int64_t cols = L.direct ? v : L.piece;           // (a copied W comes in pieces)
        L.partials = take((size_t)rows * 2 * (v / cols * cdiv(cols, L.bn_logits) + cdiv(v % cols, L.bn_logits)) * 8);
        L.sums = take((size_t)cdiv(n, 32) * 8);
        L.ticket = take(4);
    } else {
        // 128 columns where 256 would leave a quarter or more of them empty;
        // float32, whose six products need fewer bytes each, a tenth.  float32,
        // 256 -> 128 columns, us: 1001 x 515 x 8009 244 -> 240, 1001 x 1100 x
        // 8009 387 -> 377, 4000 x 1100 x 4000 701 -> 643.  Below a tenth it goes
        // either way: 1001 x 1300 x 8009 459 -> 451, 4000 x 1300 x 4000 775 ->
        // 786, 200 x 1660 x 16000 356 -> 364.
        const int64_t narrow = up(d, 128), wide = up(d, 256);
        L.bn = (b16 ? narrow * 4 <= wide * 3 : narrow * 11 < wide * 10) ? 128 : 256;
        L.bn_logits = columns_for(n, L.piece < v ? L.piece : v, d, L.parts, clusters);
        // K blocks of a tile, and of a cluster's share of a piece, each tile's
        // epilogue counted as 4 of them (float32, six products a block: as 1)
        const int64_t nt = cdiv(d, L.bn), k1 = cdiv(v < L.piece ? v : L.piece, BK), k2 = cdiv(n, BK);
        const int64_t t1 = cdiv(n, BM) * nt, t2 = cdiv(L.piece, BM) * nt;
        const int64_t e = b16 ? 4 : 1;
        int64_t share = cdiv(t1 * (k1 + e) + t2 * (k2 + e), clusters);
        if (share < 4 * e) share = 4 * e;
        L.sx = (int)cdiv(k1, share);
        L.sw = (int)cdiv(k2, share);
        L.dx_partial = L.sx > 1 || L.piece < v;
        L.dw_partial = L.sw > 1;
        L.g = take((size_t)L.parts * n * L.piece * 2);
        if (L.dx_partial) L.dxp = take((size_t)L.sx * up(n, 32) * up(d, 32) * 4);
        if (L.dw_partial) L.dwp = take((size_t)L.sw * up(L.piece, 32) * up(d, 32) * 4);
        const size_t es = b16 ? 2 : 4;
        L.stage = d * es % 16 != 0;
        if (L.stage && L.sx == 1) L.dx_stage = take((size_t)n * L.pitch * es);
        if (L.stage && L.sw == 1) L.dw_stage = take((size_t)L.piece * L.pitch * es);
        L.targets = take(n * 4);
        L.row_of = take(n * 4);
        L.lse_c = take(n * 4);
        L.weight = take(n * 4);
        L.live = take(4);
        L.counts = take(cdiv(n, kCountRows) * 4);
    }
    L.bytes = o + 240;
    return L;
}

// A launch that follows another one of the same call (`next`) may begin before that one's end.
template <typename... P, typename... A>
cudaError_t launch(void (*kernel)(P...), int64_t blocks, int threads, size_t smem, bool next, cudaStream_t st, const A&... args) {
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = &at;
    cfg.numAttrs = next ? 1 : 0;
    count_launches(1);
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <int PARTS, int EPI, int BN>
cudaError_t run_tiles(const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& a2, const CUtensorMap& b2,
                      const GemmArgs& p, int64_t tiles, bool next, cudaStream_t st) {
    static unsigned long long optin_done = 0;
    auto* k = ce_gemm_kernel<PARTS, EPI, BN>;
    const cudaError_t e = smem_optin((const void*)k, (int)smem_bytes<PARTS>(), &optin_done);
    if (e != cudaSuccess) return e;
    const int64_t clusters = sm_count() / 2;
    return launch(k, 2 * (tiles < clusters ? tiles : clusters), THREADS, smem_bytes<PARTS>(), next, st, a, b, a2, b2, p);
}
template <int PARTS, int EPI>
cudaError_t run_gemm(int bn, const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& a2, const CUtensorMap& b2,
                     const GemmArgs& p, int64_t tiles, bool next, cudaStream_t st) {
    return bn == 128 ? run_tiles<PARTS, EPI, 128>(a, b, a2, b2, p, tiles, next, st)
                     : run_tiles<PARTS, EPI, 256>(a, b, a2, b2, p, tiles, next, st);
}

unsigned warps_grid(int64_t warps) {
    const int64_t b = cdiv(warps, 8), most = (int64_t)sm_count() * 16;
    return (unsigned)(b < most ? b : most);
}

cudaError_t to_parts(const void* src, int dt, bool w, int64_t rows, int d, int pitch, void* dst, bool next, cudaStream_t st) {
    bf16* o = reinterpret_cast<bf16*>(dst);
    if (dt == MOM_BF16)
        return launch(parts_kernel<bf16, 1, false>, warps_grid(rows), 256, 0, next, st, reinterpret_cast<const bf16*>(src), rows, d, pitch, o);
    return launch(w ? parts_kernel<float, 3, true> : parts_kernel<float, 3, false>, warps_grid(rows), 256, 0, next, st,
                  reinterpret_cast<const float*>(src), rows, d, pitch, o);
}

template <typename T>
cudaError_t flatten(const void* src, int64_t rows, int d, int pitch, T* dst, cudaStream_t st) {
    const int64_t b = cdiv(rows * d, 256 * (16 / (int)sizeof(T))), most = (int64_t)sm_count() * 16;
    return launch(flatten_kernel<T>, b < most ? b : most, 256, 0, true, st, reinterpret_cast<const T*>(src), rows, d, pitch, dst);
}

int64_t join_grid(int64_t rows, int d) {
    const int64_t b = cdiv(rows, 32) * cdiv(d, 32), most = (int64_t)sm_count() * 4;
    return b < most ? b : most;
}

// A workspace is 16-byte aligned; its arrays start at multiples of 256 (g's rows take 32-byte stores).
inline char* ws_base(void* ws) { return reinterpret_cast<char*>(up(static_cast<int64_t>(reinterpret_cast<uintptr_t>(ws)), 256)); }

// the piece of W from class v0 on as a TMA operand: in place, or copied
struct WPiece {
    const void* base;
    uint64_t rows, pitch;
    int row0;
};
cudaError_t w_piece(const LinearCeArgs& a, const Plan& L, int64_t v0, int64_t pw, WPiece& w, bool next, cudaStream_t st) {
    if (L.direct) {
        w = WPiece{a.w, (uint64_t)a.v, (uint64_t)a.d, (int)v0};
        return cudaSuccess;
    }
    char* buf = ws_base(a.ws) + L.wbuf;
    w = WPiece{buf, (uint64_t)pw, (uint64_t)L.pitch, 0};
    const size_t es = a.dt == MOM_BF16 ? 2 : 4;
    return to_parts(reinterpret_cast<const char*>(a.w) + (size_t)v0 * a.d * es, a.dt, true, pw, a.d, L.pitch, buf, next, st);
}

#define MOM_TRY(x) do { const cudaError_t e_ = (x); if (e_ != cudaSuccess) return e_; } while (0)
#define MOM_MAP(x) do { if (!(x)) return cudaErrorInvalidValue; } while (0)

template <int PARTS> cudaError_t fwd(const LinearCeArgs& a, cudaStream_t st) {
    const Plan L = plan_for(a.n, a.d, a.v, a.dt, false);
    char* ws = ws_base(a.ws);
    if (!L.direct) MOM_TRY(to_parts(a.x, a.dt, false, a.n, a.d, L.pitch, ws + L.xbuf, false, st));
    const void* xb = L.direct ? a.x : ws + L.xbuf;
    int n_part = 0;
    float2* partials = reinterpret_cast<float2*>(ws + L.partials);
    float* zt = reinterpret_cast<float*>(ws + L.zt);
    int32_t* ticket = reinterpret_cast<int32_t*>(ws + L.ticket);
    for (int64_t r0 = 0; r0 < a.n; r0 += kRowChunk) {
        const int64_t rows = a.n - r0 < kRowChunk ? a.n - r0 : kRowChunk;
        n_part = 0;
        CUtensorMap ma, mb;
        // the chunk's rows: a map that starts at r0; the parts lie n rows apart
        MOM_MAP(make_tma_3d(&ma, reinterpret_cast<const bf16*>(xb) + r0 * L.pitch, false, a.d, rows, PARTS, L.pitch,
                            HM, a.n));
        for (int64_t v0 = 0; v0 < a.v; v0 += L.direct ? a.v : L.piece) {
            const int64_t pw = L.direct ? a.v : a.v - v0 < L.piece ? a.v - v0 : L.piece;
            WPiece w;
            MOM_TRY(w_piece(a, L, v0, pw, w, true, st));
            MOM_MAP(make_tma_3d(&mb, w.base, false, a.d, w.rows, PARTS, w.pitch, L.bn_logits / 2));
            GemmArgs p{};
            p.rows = rows;
            p.cols = pw;
            p.kb = (int)cdiv(a.d, BK);
            p.b_row0 = w.row0;
            p.targets = a.targets + r0;
            p.v0 = v0;
            p.vocab = a.v;
            p.partials = partials + n_part * rows;
            n_part += (int)(2 * cdiv(pw, L.bn_logits));
            p.zt = zt;
            p.ticket = r0 == 0 ? ticket : nullptr;
            p.ws = a.ws;
            MOM_TRY((run_gemm<PARTS, EPI_STATS>(L.bn_logits, ma, mb, ma, mb, p, cdiv(rows, BM) * cdiv(pw, L.bn_logits), !L.direct || r0 > 0, st)));
        }
        MOM_TRY(launch(logsumexp_kernel, cdiv(rows, 32), 1024, 0, true, st, (const float2*)partials, n_part, rows, r0,
                       (const float*)zt, a.targets + r0, a.v, a.loss + r0, a.lse + r0,
                       reinterpret_cast<float2*>(ws + L.sums), ticket, cdiv(a.n, 32), a.mean, a.ws));
    }
    return cudaSuccess;
}

template <int PARTS> cudaError_t bwd(const LinearCeArgs& a, cudaStream_t st) {
    typedef typename std::conditional<PARTS == 1, bf16, float>::type T;
    const Plan L = plan_for(a.n, a.d, a.v, a.dt, true);
    char* ws = ws_base(a.ws);
    auto i32 = [&](size_t at) { return reinterpret_cast<int32_t*>(ws + at); };
    auto f32 = [&](size_t at) { return reinterpret_cast<float*>(ws + at); };
    // where the GEMM's tiles go; a split axis' sums go from its slots to their place
    const bool sdx = L.stage && L.sx == 1, sdw = L.stage && L.sw == 1;
    T* dx = sdx ? reinterpret_cast<T*>(ws + L.dx_stage) : reinterpret_cast<T*>(a.dx);
    bf16* xc = reinterpret_cast<bf16*>(ws + L.xbuf);
    const int32_t* live = i32(L.live);
    {
        GatherArgs g{};
        g.x = a.x;
        g.targets = a.targets;
        g.lse = a.lse;
        g.dloss = a.dloss;
        g.counts = i32(L.counts);
        g.n = a.n;
        g.vocab = a.v;
        g.d = a.d;
        g.pitch = L.pitch;
        g.part = a.n * L.pitch;
        g.xc = xc;
        g.targets_c = i32(L.targets);
        g.row_of = i32(L.row_of);
        g.live = i32(L.live);
        g.lse_c = f32(L.lse_c);
        g.weight = f32(L.weight);
        g.dx = dx;
        g.dx_ld = sdx ? L.pitch : a.d;
        g.vec = a.d % 8 == 0;
        g.ws = a.ws;
        if (a.n > kCountRows) {
            MOM_TRY(launch(count_kernel, cdiv(a.n, kCountRows), 256, 0, false, st, a.targets, a.n, a.v, i32(L.counts)));
        }
        MOM_TRY(launch(gather_kernel<T, PARTS>, cdiv(a.n, kGatherRows), 256, 0, a.n > kCountRows, st, g));
    }
    CUtensorMap mx_k, mx_mn;       // x: K-major rows of the logits; MN-major rows (K = tokens) of dw
    MOM_MAP(make_tma_3d(&mx_k, xc, false, a.d, a.n, PARTS, L.pitch, HM));
    MOM_MAP(make_tma_3d(&mx_mn, xc, false, a.d, a.n, PARTS, L.pitch, BK));
    const int64_t mt = cdiv(a.n, BM);
    for (int64_t v0 = 0; v0 < a.v; v0 += L.piece) {
        const int64_t pw = a.v - v0 < L.piece ? a.v - v0 : L.piece;
        WPiece w;
        MOM_TRY(w_piece(a, L, v0, pw, w, true, st));
        CUtensorMap mw_k, mw_mn, mg_k, mg_mn;
        MOM_MAP(make_tma_3d(&mw_k, w.base, false, a.d, w.rows, PARTS, w.pitch, L.bn_logits / 2));
        MOM_MAP(make_tma_3d(&mw_mn, w.base, false, a.d, w.rows, PARTS, w.pitch, BK));
        MOM_MAP(make_tma_3d(&mg_k, ws + L.g, false, L.piece, a.n, PARTS, L.piece, HM));
        MOM_MAP(make_tma_3d(&mg_mn, ws + L.g, false, L.piece, a.n, PARTS, L.piece, BK));
        GemmArgs p{};
        p.rows = a.n;
        p.cols = pw;
        p.kb = (int)cdiv(a.d, BK);
        p.b_row0 = w.row0;
        p.live = live;
        p.targets = i32(L.targets);
        p.v0 = v0;
        p.vocab = a.v;
        p.g = reinterpret_cast<bf16*>(ws + L.g);
        p.g_pitch = L.piece;
        p.g_part = a.n * L.piece;
        p.lse = f32(L.lse_c);
        p.weight = a.dloss ? f32(L.weight) : nullptr;
        p.ws = a.ws;
        MOM_TRY((run_gemm<PARTS, EPI_GRAD>(L.bn_logits, mx_k, mw_k, mx_k, mw_k, p, mt * cdiv(pw, L.bn_logits), true, st)));
        p.d = a.d;
        p.dx.rows = a.n;
        p.dx.kb = (int)cdiv(pw, BK);
        p.dx.slots = L.sx;
        p.dx.out = dx;
        p.dx.ld = sdx ? L.pitch : a.d;
        p.dx.row_of = i32(L.row_of);
        p.dx.scale = a.dscale;
        p.dx.partial = L.dx_partial ? f32(L.dxp) : nullptr;
        p.dx.add = v0 > 0;
        p.dx.last = v0 + L.piece >= a.v;
        p.dw.rows = pw;
        p.dw.row0 = sdw ? 0 : v0;
        p.dw.kb = (int)cdiv(a.n, BK);
        p.dw.slots = L.sw;
        p.dw.out = sdw ? ws + L.dw_stage : reinterpret_cast<char*>(a.dw);
        p.dw.ld = sdw ? L.pitch : a.d;
        p.dw.scale = a.dscale;
        p.dw.partial = L.dw_partial ? f32(L.dwp) : nullptr;
        p.dw.last = 1;
        const int64_t nt = cdiv(a.d, L.bn), tiles = mt * nt * L.sx + cdiv(pw, BM) * nt * L.sw;
        MOM_TRY((run_gemm<PARTS, EPI_OUT>(L.bn, mg_k, mw_mn, mg_mn, mx_mn, p, tiles, true, st)));
        if (L.sx > 1 && p.dx.last)
            MOM_TRY(launch(join_kernel<T>, join_grid(a.n, a.d), 512, 0, true, st, p.dx, live, a.d));
        if (L.sw > 1) MOM_TRY(launch(join_kernel<T>, join_grid(pw, a.d), 512, 0, true, st, p.dw, (const int32_t*)nullptr, a.d));
        if (sdw) MOM_TRY(flatten<T>(p.dw.out, pw, a.d, L.pitch, reinterpret_cast<T*>(a.dw) + v0 * a.d, st));
        if (sdx && p.dx.last) MOM_TRY(flatten<T>(dx, a.n, a.d, L.pitch, reinterpret_cast<T*>(a.dx), st));
    }
    return cudaSuccess;
}

}  // namespace

size_t linear_ce_workspace_bytes(int64_t n, int d, int64_t v, int dt, bool bwd) {
    return plan_for(n > 0 ? n : 1, d, v, dt, bwd).bytes;
}

cudaError_t launch_linear_ce_fwd(const LinearCeArgs& a, cudaStream_t st) {
    return a.dt == MOM_BF16 ? fwd<1>(a, st) : fwd<3>(a, st);
}

cudaError_t launch_linear_ce_bwd(const LinearCeArgs& a, cudaStream_t st) {
    return a.dt == MOM_BF16 ? bwd<1>(a, st) : bwd<3>(a, st);
}

}  // namespace mom
