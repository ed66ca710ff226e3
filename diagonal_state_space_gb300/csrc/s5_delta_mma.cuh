// s5_delta_mma.cuh -- what the tensor-core kernels of the gated delta rule
// share: the image of a chunk, splits of 32-bit values, operand descriptors,
// copies and bounded waits.
#pragma once
#include <cuda.h>
#include <cudaTypedefs.h>

#include "s5_delta.cuh"
#include "s5_sm100.cuh"

namespace s5 {
namespace delta {

cudaError_t tc_prepare(const Args &a, bool transposed, cudaStream_t st);   // s5_delta_prep.cu
int prep_fault_take();
int scan_fault_take();                                                     // s5_delta_scan.cu
int adjoint_fault_take();                                                  // s5_delta_adjoint.cu

namespace {
using namespace sm100;

constexpr int C = CHUNK;
constexpr uint32_t M2_BYTES = 128 * 128;              // one part of a 128 x 64 bf16 matrix
constexpr unsigned long long WAIT_NS = 2000000000ull;

// The image of one chunk and value head: [E; P beta E] (or [T; P T]) in three
// parts, 128-byte swizzled rows of 64 values, then the chunk's factors.
struct Meta {
    float up[C];         // e^{G_i}
    float down[C];       // e^{G_64 - G_i}
    float beta[C];
    float hi[C], lo[C];  // G_i as a pair of floats
    float last;          // e^{G_64}
    float pad[3];
};
constexpr uint32_t MAT_BYTES = 3 * M2_BYTES;
constexpr uint32_t META_BYTES = sizeof(Meta);
constexpr uint32_t IMG_BYTES = MAT_BYTES + META_BYTES;
static_assert(IMG_BYTES % 16 == 0, "bulk copies");

__device__ int g_fault = 0;   // a bounded wait of this file's kernels ran out

inline int fault_take() {
    int v = 0, zero = 0;
    if (cudaMemcpyFromSymbol(&v, g_fault, sizeof(int)) != cudaSuccess) return -1;
    if (v && cudaMemcpyToSymbol(g_fault, &zero, sizeof(int)) != cudaSuccess) return -1;
    return v;
}

// ---------------------------------------------------------------------------
// bf16 pairs and parts.
// ---------------------------------------------------------------------------
__device__ __forceinline__ float lo16(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float hi16(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }
// Two floats rounded to bf16.
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// Parts.  x = h + m + l with bf16 h, m, l: 8 significant bits each, cut off and
// not rounded, so that three parts hold all 24 bits of a normal x and the
// differences are exact.  Eleven instructions a pair, the least of the forms
// measured (seven of them integer, at half rate: 15 cycles a pair and warp;
// packed f32x2 differences need 24).
__device__ __forceinline__ uint32_t tops(float a, float b) { return __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632); }
__device__ __forceinline__ float rest(float a) { return a - __uint_as_float(__float_as_uint(a) & 0xffff0000u); }
__device__ __forceinline__ void split3(float a, float b, uint32_t &h, uint32_t &m, uint32_t &l) {
    h = tops(a, b);
    a = rest(a), b = rest(b);
    m = tops(a, b);
    l = tops(rest(a), rest(b));
}
// Two parts, both rounded: off by at most 2^-17 of the value, to either side.  Two
// cut-off parts would be off by 2^-15 towards zero, and the product of two second
// parts, which is left out, would have the values' sign: 7e-6 of them each.
__device__ __forceinline__ void split2(float a, float b, uint32_t &h, uint32_t &m) {
    h = pack2(a, b);
    m = pack2(a - lo16(h), b - hi16(h));
}
// Three parts whose first two are split2's: where they are used by themselves
// too.  What the second leaves has 7 bits at most, so that all 24 are held.
__device__ __forceinline__ void split3_rounded(float a, float b, uint32_t &h, uint32_t &m, uint32_t &l) {
    h = pack2(a, b);
    a -= lo16(h), b -= hi16(h);
    m = pack2(a, b);
    l = tops(a - lo16(m), b - hi16(m));
}

// ---------------------------------------------------------------------------
// Shared memory: rows of 128 bytes, 16-byte piece j of row r at j ^ (r & 7)
// (the 128-byte swizzle of the copies and of the operand descriptors).
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t piece(uint32_t base, int row, int j) {
    return base + (uint32_t)row * 128u + (uint32_t)((j ^ (row & 7)) << 4);
}
__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}
// W values of a row from column c0 on, as three parts.  An operand of 64
// columns is an image for each part, `stride` bytes apart; of 32 columns
// (NARROW) the first two parts share an image's rows.  ROUNDED: split3_rounded.
template <int W, bool NARROW = false, bool ROUNDED = false>
__device__ __forceinline__ void put3(uint32_t img, uint32_t stride, int row, int c0, const float *v) {
#pragma unroll
    for (int j = 0; j < W / 8; ++j) {
        uint32_t h[4], m[4], l[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if constexpr (ROUNDED)
                split3_rounded(v[8 * j + 2 * i], v[8 * j + 2 * i + 1], h[i], m[i], l[i]);
            else
                split3(v[8 * j + 2 * i], v[8 * j + 2 * i + 1], h[i], m[i], l[i]);
        const uint32_t to = piece(img, row, c0 / 8 + j);
        sts128(to, h[0], h[1], h[2], h[3]);
        sts128(NARROW ? piece(img, row, c0 / 8 + j + 4) : to + stride, m[0], m[1], m[2], m[3]);
        sts128(to + (NARROW ? 1 : 2) * stride, l[0], l[1], l[2], l[3]);
    }
}
// 32 floats as the 128-byte row of a staged tile.
__device__ __forceinline__ void put_row(uint32_t tile, int row, const float *v) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
        sts128(piece(tile, row, j), __float_as_uint(v[4 * j]), __float_as_uint(v[4 * j + 1]), __float_as_uint(v[4 * j + 2]),
               __float_as_uint(v[4 * j + 3]));
}

// ---------------------------------------------------------------------------
// Fragments: 16 rows x 2 F columns over a warp (F values a thread, 16 or 8),
// f[4 j + 2 i + k] = row lane / 4 + 8 i, column 8 j + 2 (lane % 4) + k: what
// the 16-lane TMEM loads give and the 8 x 8 matrix stores and loads take.  The
// tokens of a chunk lie 16 to a warp's 32 TMEM lanes, so that all warps share
// their conversion.
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t frag_addr(uint32_t img, int row0, int c0, int j, int lane) {
    return piece(img, row0 + (lane & 15), c0 / 8 + j + (lane >> 4));
}
// The same in a tile of 64-byte rows (64-byte swizzle).
__device__ __forceinline__ uint32_t frag_addr64(uint32_t tile, int row0, int c0, int j, int lane) {
    const int r = row0 + (lane & 15), k = c0 / 8 + j + (lane >> 4);
    return tile + (uint32_t)r * 64u + (uint32_t)((k ^ ((r >> 1) & 3)) << 4);
}
__device__ __forceinline__ void stmatrix4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d)
                 : "memory");
}
__device__ __forceinline__ void ldmatrix4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
// Rows row0 .. row0 + 15, columns c0 on as three parts (F = 8: NARROW).  Blocks
// of 16 columns past `last` are zeros.
template <int F>
__device__ __forceinline__ void frag_put3(uint32_t img, uint32_t stride, int row0, int c0, int lane, const float (&f)[F], int last = 3) {
#pragma unroll
    for (int j = 0; j < F / 4; j += 2) {
        uint32_t h[4] = {}, m[4] = {}, l[4] = {};
        if (c0 / 16 + j / 2 <= last)
#pragma unroll
            for (int i = 0; i < 4; ++i) split3(f[4 * j + 2 * i], f[4 * j + 2 * i + 1], h[i], m[i], l[i]);
        const uint32_t to = frag_addr(img, row0, c0, j, lane);
        stmatrix4(to, h[0], h[1], h[2], h[3]);
        stmatrix4(F == 8 ? frag_addr(img, row0, c0 + 32, j, lane) : to + stride, m[0], m[1], m[2], m[3]);
        stmatrix4(to + (F == 8 ? 1 : 2) * stride, l[0], l[1], l[2], l[3]);
    }
}
// The same rows and columns of a bf16 tile (4 F columns wide), as floats; and
// rounded to one.
template <int F> __device__ __forceinline__ void frag_get(uint32_t tile, int row0, int c0, int lane, float (&f)[F]) {
#pragma unroll
    for (int j = 0; j < F / 4; j += 2) {
        uint32_t r[4];
        ldmatrix4(F == 8 ? frag_addr64(tile, row0, c0, j, lane) : frag_addr(tile, row0, c0, j, lane), r);
#pragma unroll
        for (int i = 0; i < 4; ++i) f[4 * j + 2 * i] = lo16(r[i]), f[4 * j + 2 * i + 1] = hi16(r[i]);
    }
}
template <int F> __device__ __forceinline__ void frag_round(uint32_t tile, int row0, int c0, int lane, const float (&f)[F]) {
#pragma unroll
    for (int j = 0; j < F / 4; j += 2)
        stmatrix4(F == 8 ? frag_addr64(tile, row0, c0, j, lane) : frag_addr(tile, row0, c0, j, lane), pack2(f[4 * j], f[4 * j + 1]),
                  pack2(f[4 * j + 2], f[4 * j + 3]), pack2(f[4 * j + 4], f[4 * j + 5]), pack2(f[4 * j + 6], f[4 * j + 7]));
}
// In 32 bits: 32 columns are the tile's whole row.
__device__ __forceinline__ void frag_put_rows(uint32_t tile, int row0, int lane, const float (&f)[16]) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < 2; ++i)
            asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(piece(tile, row0 + lane / 4 + 8 * i, 2 * j + lane % 4 / 2) +
                                                                 (lane & 1) * 8u),
                         "f"(f[4 * j + 2 * i]), "f"(f[4 * j + 2 * i + 1])
                         : "memory");
}
// f's rows times a (lane / 4) and b (lane / 4 + 8).
template <int F> __device__ __forceinline__ void frag_scale(float (&f)[F], float a, float b) {
#pragma unroll
    for (int i = 0; i < F; ++i) f[i] *= (i & 2) ? b : a;
}

// ---------------------------------------------------------------------------
// Accumulators.
// ---------------------------------------------------------------------------
constexpr int NV = 64;                       // value columns of a slice

__device__ __forceinline__ void tmem_ldw(uint32_t addr, uint32_t (&r)[16]) { tmem_ld16(addr, r); }
__device__ __forceinline__ void tmem_ldw(uint32_t addr, uint32_t (&r)[32]) { tmem_ld32(addr, r); }
// W columns of this thread's lane: the sum of P column blocks, STRIDE apart,
// one for each part of a split operand.
template <int P, int W, int STRIDE = NV> __device__ __forceinline__ void load_parts(uint32_t addr, float *v) {
    uint32_t r[P][W];
#pragma unroll
    for (int p = 0; p < P; ++p) tmem_ldw(addr + p * STRIDE, r[p]);
    tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < W; ++i) {
        v[i] = __uint_as_float(r[P - 1][i]);
#pragma unroll
        for (int p = P - 2; p >= 0; --p) v[i] += __uint_as_float(r[p][i]);
    }
}
// 16 lanes x 32 or 16 columns as a fragment.
__device__ __forceinline__ void tmem_ld_frag(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
          "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld_frag(uint32_t taddr, uint32_t (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
}
// The sum of P column blocks, 4 F apart.
template <int P, int F> __device__ __forceinline__ void frag_load(uint32_t addr, float (&f)[F]) {
    uint32_t r[P][F];
#pragma unroll
    for (int p = 0; p < P; ++p) tmem_ld_frag(addr + p * 4 * F, r[p]);
    tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < F; ++i) {
        f[i] = __uint_as_float(r[P - 1][i]);
#pragma unroll
        for (int p = P - 2; p >= 0; --p) f[i] += __uint_as_float(r[p][i]);
    }
}
constexpr uint32_t QUERY_LANES = 16u << 16;   // the query rows' lanes, past the key rows'

// ---------------------------------------------------------------------------
// Operand descriptors.
// K-major: 128-byte rows of 64 K values; a step of 16 is 32 bytes on.
// MN-major: 128-byte rows of 64 M or N values, one row per K value; a step of
// 16 is 2048 bytes on, the next 64 values of M or N are `far` on.
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint64_t desc128(uint32_t addr, uint32_t lbo) {
    uint64_t d = 0;
    d |= (uint64_t)((addr >> 4) & 0x3FFFu);
    d |= (uint64_t)((lbo >> 4) & 0x3FFFu) << 16;
    d |= (uint64_t)(1024u >> 4) << 32;
    d |= (uint64_t)1u << 46;
    d |= (uint64_t)2u << 61;
    return d;
}
__device__ __forceinline__ uint64_t desc_k(uint32_t base) { return desc128(base, 16u); }
__device__ __forceinline__ uint64_t desc_mn(uint32_t base, uint32_t far) { return desc128(base, far); }
// The same operand `bytes` on (the address field cannot carry: shared memory
// ends below its 256 KB).
__device__ __forceinline__ uint64_t on(uint64_t desc, uint32_t bytes) { return desc + (bytes >> 4); }
constexpr uint32_t K_STEP = 32, MN_STEP = 2048;
constexpr uint32_t A_MN = 1u << 15, B_MN = 1u << 16;
// 128 rows of 64 values: 16 keys, 16 queries, 16 keys, ...; a chunk's matrix
// [E; P beta E] has its rows in the same order.
constexpr uint32_t KQ_BOX = 128 * 128;
constexpr uint32_t KQ_GROUP = 16 * 128;      // 16 of those rows
constexpr uint32_t RU_IMG = 64 * 128;        // one part of a 64 x 64 operand

// ---------------------------------------------------------------------------
// Copies and waits.
// ---------------------------------------------------------------------------
__device__ __forceinline__ void bulk_store(void *dst, const void *src, uint32_t bytes) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(smem_addr(src)), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void tma_load_4d(void *dst, const void *tmap, int c0, int c1, int c2, int c3, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_addr(dst)),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(smem_addr(bar))
        : "memory");
}
__device__ __forceinline__ void tma_store_4d(const void *tmap, const void *src, int c0, int c1, int c2, int c3) {
    asm volatile("cp.async.bulk.tensor.4d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3, %4}], [%5];" ::"l"(
                     reinterpret_cast<uint64_t>(tmap)),
                 "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(smem_addr(src))
                 : "memory");
}
// The keys and queries of a chunk, as DK / 64 boxes of interleaved rows.
template <int DK>
__device__ __forceinline__ void load_chunk_rows(unsigned char *to, const void *k, const void *q, int hk, int t0, int b,
                                                uint64_t *bar) {
    mbar_arrive_tx(bar, DK / 64 * KQ_BOX);
#pragma unroll 1
    for (int x = 0; x < DK / 64; ++x)
#pragma unroll 1
        for (int i = 0; i < C / 16; ++i) {
            tma_load_4d(to + x * KQ_BOX + 2 * i * KQ_GROUP, k, 64 * x, hk, t0 + 16 * i, b, bar);
            tma_load_4d(to + x * KQ_BOX + (2 * i + 1) * KQ_GROUP, q, 64 * x, hk, t0 + 16 * i, b, bar);
        }
}
// True once the phase is over; false once a wait of the block has run out
// (2 s): the block then ends without waiting further, and the host is told.
__device__ __forceinline__ bool bounded_wait(uint64_t *bar, uint32_t parity, volatile int *abort) {
    if (mbar_try_wait(bar, parity)) return true;
    const unsigned long long t0 = global_ns();
    for (;;) {
        if (mbar_try_wait_sleep(bar, parity, 100000)) return true;
        if (*abort) return false;
        if (global_ns() - t0 > WAIT_NS) {
            *abort = 1;
            atomicExch(&g_fault, 1);
            return false;
        }
    }
}
// After a wait that ran out: copies in flight land (microseconds) before the
// block gives its memory back.
__device__ __forceinline__ void settle_copies() {
    const unsigned long long t0 = global_ns();
    while (global_ns() - t0 < 2000000ull) __nanosleep(1000);
}
// Every MMA that this thread issued has completed, or 0.2 s have passed.
__device__ __forceinline__ void drain_products(uint64_t *bar) {
    mma_commit(bar);
    const unsigned long long t0 = global_ns();
    while (!mbar_try_wait_sleep(bar, 0, 100000))
        if (global_ns() - t0 > 200000000ull) break;
}
// What a warp wrote to shared memory and read from TMEM is done before the
// waiting thread goes on.
__device__ __forceinline__ void hand_over(uint64_t *bar, int lane) {
    fence_proxy_async_smem();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
}

// ---------------------------------------------------------------------------
// Tensor maps.  Rows [B][L][H][D] with a pitch between tokens, in boxes of 64
// (or fewer) tokens x 128 (or 64) bytes of one head; tokens past L read as
// zeros and are not written.
// ---------------------------------------------------------------------------
inline cudaError_t encode(CUtensorMap *m, bool f32, int rank, const void *p, const cuuint64_t *dims, const cuuint64_t *strides,
                          const cuuint32_t *box) {
    const bool half = box[0] * (f32 ? 4 : 2) == 64;
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    if (!fn) {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            return cudaErrorNotSupported;
        fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
    }
    const cuuint32_t es[4] = {1, 1, 1, 1};
    return fn(m, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void *>(p), dims,
              strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, half ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? cudaSuccess
               : cudaErrorInvalidValue;
}
inline cudaError_t encode_rows(CUtensorMap *m, bool f32, const void *p, long long ld, int B, int L, int H, int D,
                               int tokens = C, int values = 0) {
    const cuuint64_t e = f32 ? 4 : 2;
    const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)H, (cuuint64_t)L, (cuuint64_t)B};
    const cuuint64_t strides[3] = {(cuuint64_t)D * e, (cuuint64_t)ld * e, (cuuint64_t)ld * e * L};
    const cuuint32_t box[4] = {values ? (cuuint32_t)values : f32 ? 32u : 64u, 1, (cuuint32_t)tokens, 1};
    return encode(m, f32, 4, p, dims, strides, box);
}
// Matrices [n][Dk][Dv] of floats in boxes of Dk rows x 32 columns.
inline cudaError_t encode_states(CUtensorMap *m, const void *p, long long n, int Dk, int Dv) {
    const cuuint64_t dims[3] = {(cuuint64_t)Dv, (cuuint64_t)Dk, (cuuint64_t)n};
    const cuuint64_t strides[2] = {(cuuint64_t)Dv * 4, (cuuint64_t)Dk * Dv * 4};
    const cuuint32_t box[3] = {32, (cuuint32_t)Dk, 1};
    return encode(m, true, 3, p, dims, strides, box);
}
template <typename K> inline cudaError_t big_smem(K *kernel, size_t bytes) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

}  // namespace
}  // namespace delta
}  // namespace s5
