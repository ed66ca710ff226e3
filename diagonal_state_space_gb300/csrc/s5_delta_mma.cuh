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
// Pairs of 32-bit values in one 64-bit register (the low half is the first).
// ---------------------------------------------------------------------------
typedef unsigned long long f2;
__device__ __forceinline__ f2 make2(uint32_t lo, uint32_t hi) { return (f2)hi << 32 | lo; }
__device__ __forceinline__ f2 make2(float lo, float hi) { return make2(__float_as_uint(lo), __float_as_uint(hi)); }
__device__ __forceinline__ f2 both(float x) { return make2(x, x); }
__device__ __forceinline__ uint32_t lo32(f2 x) { return (uint32_t)x; }
__device__ __forceinline__ uint32_t hi32(f2 x) { return (uint32_t)(x >> 32); }
__device__ __forceinline__ float lof(f2 x) { return __uint_as_float(lo32(x)); }
__device__ __forceinline__ float hif(f2 x) { return __uint_as_float(hi32(x)); }
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
    f2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
    f2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
    f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
// Two bf16 values as two floats.
__device__ __forceinline__ f2 widen(uint32_t v) { return make2(v << 16, v & 0xffff0000u); }
// Two floats rounded to bf16.
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Parts.  x = h + m + l with bf16 h, m, l: 8 significant bits each, cut off and
// not rounded, so that three parts hold all 24 bits of a normal x and the
// differences are exact.
__device__ __forceinline__ uint32_t tops(f2 x) { return __byte_perm(lo32(x), hi32(x), 0x7632); }
__device__ __forceinline__ f2 minus_tops(f2 x) {   // -(the tops' values), to be added
    return make2((lo32(x) & 0xffff0000u) ^ 0x80000000u, (hi32(x) & 0xffff0000u) ^ 0x80000000u);
}
__device__ __forceinline__ void split3(f2 x, uint32_t &h, uint32_t &m, uint32_t &l) {
    h = tops(x);
    x = add2(x, minus_tops(x));
    m = tops(x);
    x = add2(x, minus_tops(x));
    l = tops(x);
}
// Two parts, the second rounded: 17 bits.
__device__ __forceinline__ void split2(f2 x, uint32_t &h, uint32_t &m) {
    h = tops(x);
    x = add2(x, minus_tops(x));
    m = pack2(lof(x), hif(x));
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
// W values (pairs v) of a row from column c0 on, as three images `stride`
// bytes apart.
template <int W> __device__ __forceinline__ void put3(uint32_t img, uint32_t stride, int row, int c0, const f2 *v) {
#pragma unroll
    for (int j = 0; j < W / 8; ++j) {
        uint32_t h[4], m[4], l[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) split3(v[4 * j + i], h[i], m[i], l[i]);
        const uint32_t to = piece(img, row, c0 / 8 + j);
        sts128(to, h[0], h[1], h[2], h[3]);
        sts128(to + stride, m[0], m[1], m[2], m[3]);
        sts128(to + 2 * stride, l[0], l[1], l[2], l[3]);
    }
}
// 32 floats as the 128-byte row of a staged tile.
__device__ __forceinline__ void put_row(uint32_t tile, int row, const f2 *v) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
        sts128(piece(tile, row, j), lo32(v[2 * j]), hi32(v[2 * j]), lo32(v[2 * j + 1]), hi32(v[2 * j + 1]));
}

// ---------------------------------------------------------------------------
// Accumulators.
// ---------------------------------------------------------------------------
constexpr int NV = 64;                       // value columns of a slice

__device__ __forceinline__ void tmem_ldw(uint32_t addr, uint32_t (&r)[8]) { tmem_ld8(addr, r); }
__device__ __forceinline__ void tmem_ldw(uint32_t addr, uint32_t (&r)[16]) { tmem_ld16(addr, r); }
__device__ __forceinline__ void tmem_ldw(uint32_t addr, uint32_t (&r)[32]) { tmem_ld32(addr, r); }
// W columns as W / 2 pairs: the sum of P column blocks, 64 apart, one for each
// part of a split operand.
template <int P, int W> __device__ __forceinline__ void load_parts(uint32_t addr, f2 *v) {
    uint32_t r[P][W];
#pragma unroll
    for (int p = 0; p < P; ++p) tmem_ldw(addr + p * NV, r[p]);
    tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < W / 2; ++i) {
        v[i] = make2(r[P - 1][2 * i], r[P - 1][2 * i + 1]);
#pragma unroll
        for (int p = P - 2; p >= 0; --p) v[i] = add2(v[i], make2(r[p][2 * i], r[p][2 * i + 1]));
    }
}

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
constexpr uint32_t KQ_BOX = 128 * 128;       // 128 rows (64 keys, 64 queries) of 64 values
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
// tokens x 128 bytes of one head; tokens past L read as zeros and are not
// written.
// ---------------------------------------------------------------------------
inline cudaError_t encode(CUtensorMap *m, bool f32, int rank, const void *p, const cuuint64_t *dims, const cuuint64_t *strides,
                          const cuuint32_t *box) {
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
              strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? cudaSuccess
               : cudaErrorInvalidValue;
}
inline cudaError_t encode_rows(CUtensorMap *m, bool f32, const void *p, long long ld, int B, int L, int H, int D) {
    const cuuint64_t e = f32 ? 4 : 2;
    const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)H, (cuuint64_t)L, (cuuint64_t)B};
    const cuuint64_t strides[3] = {(cuuint64_t)D * e, (cuuint64_t)ld * e, (cuuint64_t)ld * e * L};
    const cuuint32_t box[4] = {f32 ? 32u : 64u, 1, 64, 1};
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
