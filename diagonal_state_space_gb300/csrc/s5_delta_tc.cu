// s5_delta_tc.cu -- the gated delta rule on the 5th-generation tensor cores:
// bf16 queries, keys and values, heads of 64 or 128.
//
// A chunk of 64 tokens that starts from the state S0, with G_i the sum of the
// chunk's log decays up to token i and D_ij = exp(G_i - G_j):
//   E = (I + strict lower(D_ij k_i.k_j beta_j))^-1,   P_ij = scale D_ij q_i.k_j (j <= i)
//   R = V - e^G K S0
//   e = E R,  o = scale e^G Q S0 + (P beta E) R
//   S = e^{G_64} S0 + K^T (e^{G_64 - G} beta e)
// Everything without S0 is done for all chunks at once by delta_prep_kernel:
// it leaves the 128 x 64 matrix [E; P beta E] of each chunk.  The recurrence
// over chunks then is three matrix products in a row, one CTA per sequence,
// head and 64 value columns:
//   D1 = [K; Q] S0      (128 x 64, depth Dk)
//   D2 = [E; P beta E] R  (128 x 64, depth 64)
//   D3 = K^T U          (Dk x 64, depth 64)
// all of M = 128: the rows 64..127 of the first two give the outputs beside
// the rows that the recurrence needs.
//
// Precision.  Keys, queries and values are bf16 and enter the products as they
// are.  S0, R, U and [E; P beta E] are 32-bit values, carried as sums of three
// bf16 values (8 + 8 + 8 significant bits): three products against a bf16
// operand, six against another split one (the three smallest, below 2^-24, are
// left out).  One rounding to bf16 instead would leave 2^-9 in the state.
#include <cuda.h>
#include <cudaTypedefs.h>

#include "s5_delta.cuh"
#include "s5_sm100.cuh"

namespace s5 {
namespace delta {
using namespace sm100;

namespace {

constexpr int C = CHUNK;
constexpr uint32_t M2_BYTES = 128 * 128;              // one split of a 128 x 64 matrix
constexpr uint32_t META_BYTES = 2048;                 // the chunk's factors (Meta)
constexpr uint32_t IMG_BYTES = 3 * M2_BYTES + META_BYTES;
constexpr unsigned long long WAIT_NS = 2000000000ull;

__device__ int g_delta_fault = 0;   // a bounded wait ran out

struct Meta {            // of one chunk and value head
    float up[C];         // e^{G_i}
    float down[C];       // e^{G_64 - G_i}
    float beta[C];
    float hi[C], lo[C];  // G_i as a pair of floats
    float last;          // e^{G_64}
};
static_assert(sizeof(Meta) <= META_BYTES, "meta block");

// ---------------------------------------------------------------------------
// Splits.  x = h + m + l with bf16 h, m, l; two values at a time.
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ void split3(float a, float b, uint32_t &h, uint32_t &m, uint32_t &l) {
    h = pack2(a, b);
    a -= __uint_as_float(h << 16), b -= __uint_as_float(h & 0xffff0000u);
    m = pack2(a, b);
    a -= __uint_as_float(m << 16), b -= __uint_as_float(m & 0xffff0000u);
    l = pack2(a, b);
}

__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

__device__ __forceinline__ void bulk_store(void *dst, const void *src, uint32_t bytes) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(smem_addr(src)), "r"(bytes)
                 : "memory");
}

// Writes 32 values of row `row` (columns c0 .. c0 + 31 of 64) as three images
// `stride` bytes apart, 128 bytes a row in the 128-byte swizzle.
__device__ __forceinline__ void store_split32(uint32_t img, uint32_t stride, int row, int c0, const float (&v)[32]) {
    const uint32_t at = img + (uint32_t)row * 128u;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        uint32_t h[4], m[4], l[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) split3(v[8 * j + 2 * i], v[8 * j + 2 * i + 1], h[i], m[i], l[i]);
        const uint32_t to = at + (uint32_t)(((c0 / 8 + j) ^ (row & 7)) << 4);
        sts128(to, h[0], h[1], h[2], h[3]);
        sts128(to + stride, m[0], m[1], m[2], m[3]);
        sts128(to + 2 * stride, l[0], l[1], l[2], l[3]);
    }
}

// ---------------------------------------------------------------------------
// Preparation: one CTA per chunk and key head; the products k.k and q.k are
// taken once (mma.sync, exact bf16 operands) and stay in registers for the
// key head's value heads.
//
// Decay factors D_ij of two different blocks of 16 tokens are products
// e^{G_i - G_b} e^{G_b - G_j} at the end b of j's block (both at most 1 where
// g <= 0); inside a block each is an exponential of its own.
//
// The inverse goes by blocks, in place and in 32 bits: the four 16 x 16 blocks
// on the diagonal by substitution (one column per lane), then
//   [[A, 0], [B, D]]^-1 = [[A^-1, 0], [-D^-1 B A^-1, D^-1]]
// to 32 and to 64 rows.  P E is a product of two triangular 64 x 64 matrices
// in three bf16 parts each (mma.sync, the 20 of 64 block products that are not
// zero).  The whole image is built in shared memory in the layout that the
// recurrences' products read, and leaves by one bulk copy.
//
// TRANS: (I + strict lower(beta_i D_ij k_i.k_j))^-1 = T and [T; P T] instead,
// which the backward pass uses.
// ---------------------------------------------------------------------------
constexpr int PT = 256;             // threads
constexpr int LD = 68;              // pitch of the fp32 tile: 16-byte rows, no conflicts on 8 rows of 4

template <int DK> struct PrepSmem {
    static constexpr int KP = DK + 8;                    // bf16 pitch of the tiles: conflict-free fragments
    static constexpr uint32_t tiles = 2 * C * KP * 2;    // keys and queries, before the image
    static constexpr uint32_t a = IMG_BYTES;             // [64][LD] fp32, after the image (and the tiles)
    static constexpr uint32_t near = a + C * LD * 4;     // e^{G_b - G_j}
    static constexpr uint32_t total = near + C * 4;
    static_assert(tiles <= IMG_BYTES, "the tiles lie in the image's place");
};

// mma.sync m16n8k16: D += A B.
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
        "%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldmatrix4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldmatrix4t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

template <int DK, bool TRANS> __global__ void __launch_bounds__(PT, 3) delta_prep_kernel(const Args a) {
    using L = PrepSmem<DK>;
    extern __shared__ __align__(128) unsigned char psm[];
    unsigned char *img = psm;
    float(*A)[LD] = reinterpret_cast<float(*)[LD]>(psm + L::a);
    float *near = reinterpret_cast<float *>(psm + L::near);
    Meta *meta = reinterpret_cast<Meta *>(psm + 3 * M2_BYTES);
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int c = blockIdx.x, hk = blockIdx.y, b = blockIdx.z, group = a.Hv / a.Hk;
    const int t0 = c * C, nt = min(C, a.L - t0), N = chunks(a.L);
    const long long row0 = (long long)b * a.L + t0;
    const int rb = warp & 3, g = lane / 4, q2 = lane % 4 * 2;   // block of 16 rows; fragment row and column
    const bool isq = warp >= 4;                                 // warps 0..3: k.k, 4..7: q.k
    float acc[8][4] = {};
    {
        constexpr int KP = L::KP;
        __nv_bfloat16 *sk = reinterpret_cast<__nv_bfloat16 *>(psm), *sq = sk + C * KP;
        for (int i = tid; i < C * (DK / 8); i += PT) {
            const int t = i / (DK / 8), d = i % (DK / 8) * 8;
            uint4 xk = make_uint4(0, 0, 0, 0), xq = xk;
            if (t < nt) {
                xk = *reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(a.k) + (row0 + t) * a.ldk + hk * DK + d);
                xq = *reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(a.q) + (row0 + t) * a.ldq + hk * DK + d);
            }
            *reinterpret_cast<uint4 *>(sk + t * KP + d) = xk;
            *reinterpret_cast<uint4 *>(sq + t * KP + d) = xq;
        }
        __syncthreads();
        const __nv_bfloat16 *rows = isq ? sq : sk;
#pragma unroll 2
        for (int k0 = 0; k0 < DK; k0 += 16) {
            uint32_t f[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                f[i] = *reinterpret_cast<const uint32_t *>(rows + (16 * rb + g + (i & 1) * 8) * KP + k0 + q2 + (i >> 1) * 8);
#pragma unroll
            for (int n = 0; n < 8; ++n) {
                if (n > 2 * rb + 1) continue;
                const int at = (8 * n + g) * KP + k0 + q2;
                mma16816(acc[n], f, *reinterpret_cast<const uint32_t *>(sk + at), *reinterpret_cast<const uint32_t *>(sk + at + 8));
            }
        }
        if (isq)
#pragma unroll
            for (int n = 0; n < 8; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[n][i] *= a.scale;
    }
    // rows 64..127 of the image: three parts of two neighbouring values
    auto put2 = [&](int r, int n, float x, float y) {
        uint32_t h, m, l;
        split3(x, y, h, m, l);
        unsigned char *to = img + (C + r) * 128 + ((n ^ (r & 7)) << 4) + q2 * 2;
        *reinterpret_cast<uint32_t *>(to) = h;
        *reinterpret_cast<uint32_t *>(to + M2_BYTES) = m;
        *reinterpret_cast<uint32_t *>(to + 2 * M2_BYTES) = l;
    };
    const uint32_t simg = smem_addr(img);
    for (int j = 0; j < group; ++j) {
        const int h = hk * group + j;
        if (j > 0 && tid == 0) bulk_wait_read_all();   // the last image has left
        __syncthreads();
        if (warp == 0) {
            // G in float64 (64 terms of up to 128), kept as two floats, so that
            // a small difference of large sums keeps 24 bits
            double x0 = 2 * lane < nt ? (double)clamp_g(a.g[(row0 + 2 * lane) * a.Hv + h]) : 0.0;
            double x1 = 2 * lane + 1 < nt ? (double)clamp_g(a.g[(row0 + 2 * lane + 1) * a.Hv + h]) : 0.0;
            double w = x0 + x1;
#pragma unroll
            for (int m = 1; m < 32; m <<= 1) {
                const double up = __shfl_up_sync(0xffffffffu, w, m);
                if (lane >= m) w += up;
            }
            const double tot = __shfl_sync(0xffffffffu, w, 31), edge = __shfl_sync(0xffffffffu, w, lane | 7);
            const double G[2] = {w - x1, w};
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int t = 2 * lane + i;
                const float hi = (float)G[i];
                meta->hi[t] = hi;
                meta->lo[t] = (float)(G[i] - (double)hi);
                meta->beta[t] = t < nt ? a.beta[(row0 + t) * a.Hv + h] : 0.0f;
                meta->up[t] = expf(hi);
                meta->down[t] = expf((float)(tot - G[i]));
                near[t] = expf((float)(edge - G[i]));
            }
            if (lane == 0) meta->last = expf((float)tot);
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 2; ++i) {      // rows g and g + 8 of the warp's block
            const int r = 16 * rb + g + 8 * i;
            const float gh = meta->hi[r], gl = meta->lo[r], br = meta->beta[r];
#pragma unroll
            for (int nb = 0; nb < 4; ++nb) {
                float w[4] = {0, 0, 0, 0};
                if (nb <= rb) {
                    const float far = nb < rb ? expf((gh - meta->hi[16 * nb + 15]) + (gl - meta->lo[16 * nb + 15])) : 0.0f;
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const int n = 2 * nb + x / 2, col = 8 * n + q2 + x % 2;
                        const float p = acc[n][2 * i + x % 2];
                        const float d = nb < rb ? far * near[col] : expf((gh - meta->hi[col]) + (gl - meta->lo[col]));
                        const bool in = isq ? col <= r : col < r;
                        const float by = isq ? (TRANS ? 1.0f : meta->beta[col]) : (TRANS ? br : meta->beta[col]);
                        w[x] = in ? p * (d * by) : 0.0f;
                    }
                }
                if (isq) {
                    put2(r, 2 * nb, w[0], w[1]);
                    put2(r, 2 * nb + 1, w[2], w[3]);
                } else {
                    *reinterpret_cast<float2 *>(&A[r][16 * nb + q2]) = make_float2(w[0], w[1]);
                    *reinterpret_cast<float2 *>(&A[r][16 * nb + 8 + q2]) = make_float2(w[2], w[3]);
                }
            }
        }
        __syncthreads();
        if (warp < 2) {   // two blocks of the diagonal per warp; lane: a column of the inverse
            const int o = 32 * warp + (lane & 16), col = lane & 15;
            float x[16];
#pragma unroll
            for (int r = 0; r < 16; ++r) x[r] = r == col ? 1.0f : 0.0f;
#pragma unroll
            for (int r = 1; r < 16; ++r)
#pragma unroll
                for (int m = 0; m < r; m += 4) {
                    const float4 f = *reinterpret_cast<const float4 *>(&A[o + r][o + m]);
                    x[r] = fmaf(-f.x, x[m], x[r]);
                    if (m + 1 < r) x[r] = fmaf(-f.y, x[m + 1], x[r]);
                    if (m + 2 < r) x[r] = fmaf(-f.z, x[m + 2], x[r]);
                    if (m + 3 < r) x[r] = fmaf(-f.w, x[m + 3], x[r]);
                }
            __syncwarp();
#pragma unroll
            for (int r = 0; r < 16; ++r) A[o + r][o + col] = x[r];
        }
        __syncthreads();
        {   // 32-row blocks, both pairs at once: B A^-1 into the unused upper part, then -D^-1 of it
            const int o = 32 * (tid / 128), r = tid % 128 / 8, c2 = tid % 8 * 2;
            float v0 = 0.0f, v1 = 0.0f;
#pragma unroll
            for (int m = 0; m < 16; ++m) {
                const float x = A[o + 16 + r][o + m];
                const float2 y = *reinterpret_cast<const float2 *>(&A[o + m][o + c2]);
                v0 = fmaf(x, y.x, v0), v1 = fmaf(x, y.y, v1);
            }
            *reinterpret_cast<float2 *>(&A[o + r][o + 16 + c2]) = make_float2(v0, v1);
            __syncthreads();
            v0 = v1 = 0.0f;
#pragma unroll
            for (int m = 0; m < 16; ++m) {
                const float x = A[o + 16 + r][o + 16 + m];
                const float2 y = *reinterpret_cast<const float2 *>(&A[o + m][o + 16 + c2]);
                v0 = fmaf(-x, y.x, v0), v1 = fmaf(-x, y.y, v1);
            }
            *reinterpret_cast<float2 *>(&A[o + 16 + r][o + c2]) = make_float2(v0, v1);
            __syncthreads();
            *reinterpret_cast<float2 *>(&A[o + r][o + 16 + c2]) = make_float2(0.0f, 0.0f);
        }
        __syncthreads();
        {   // 64 rows
            const int r = tid / 8, c4 = tid % 8 * 4;
            float4 v = make_float4(0, 0, 0, 0);
#pragma unroll 8
            for (int m = 0; m < 32; ++m) {
                const float x = A[32 + r][m];
                const float4 y = *reinterpret_cast<const float4 *>(&A[m][c4]);
                v.x = fmaf(x, y.x, v.x), v.y = fmaf(x, y.y, v.y), v.z = fmaf(x, y.z, v.z), v.w = fmaf(x, y.w, v.w);
            }
            *reinterpret_cast<float4 *>(&A[r][32 + c4]) = v;
            __syncthreads();
            v = make_float4(0, 0, 0, 0);
#pragma unroll 8
            for (int m = 0; m < 32; ++m) {
                const float x = A[32 + r][32 + m];
                const float4 y = *reinterpret_cast<const float4 *>(&A[m][32 + c4]);
                v.x = fmaf(-x, y.x, v.x), v.y = fmaf(-x, y.y, v.y), v.z = fmaf(-x, y.z, v.z), v.w = fmaf(-x, y.w, v.w);
            }
            *reinterpret_cast<float4 *>(&A[32 + r][c4]) = v;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < C * 8 / PT; ++k) {   // E's three parts
            const int i = tid + k * PT, r = i / 8, ch = i % 8;
            float4 x = make_float4(0, 0, 0, 0), y = x;
            if (!(r < 32 && ch >= 4)) {          // that quarter holds the intermediate product
                x = *reinterpret_cast<const float4 *>(&A[r][8 * ch]);
                y = *reinterpret_cast<const float4 *>(&A[r][8 * ch + 4]);
            }
            uint32_t hh[4], mm[4], ll[4];
            split3(x.x, x.y, hh[0], mm[0], ll[0]);
            split3(x.z, x.w, hh[1], mm[1], ll[1]);
            split3(y.x, y.y, hh[2], mm[2], ll[2]);
            split3(y.z, y.w, hh[3], mm[3], ll[3]);
            unsigned char *to = img + r * 128 + ((ch ^ (r & 7)) << 4);
            *reinterpret_cast<uint4 *>(to) = make_uint4(hh[0], hh[1], hh[2], hh[3]);
            *reinterpret_cast<uint4 *>(to + M2_BYTES) = make_uint4(mm[0], mm[1], mm[2], mm[3]);
            *reinterpret_cast<uint4 *>(to + 2 * M2_BYTES) = make_uint4(ll[0], ll[1], ll[2], ll[3]);
        }
        __syncthreads();
        // P E: warp w takes the rows of block w % 4 and the columns 32 (w / 4) on
        float pe[4][4] = {};
#pragma unroll
        for (int jb = 0; jb < 2; ++jb) {
            const int cb = 2 * (warp >> 2) + jb;       // block of 16 columns
            for (int kb = cb; kb <= rb; ++kb) {
                uint32_t fa[3][4], fb[3][4];
                const int r = C + 16 * rb + (lane & 15), m = 16 * kb + (lane & 15);
#pragma unroll
                for (int p = 0; p < 3; ++p) {
                    ldmatrix4(simg + p * M2_BYTES + r * 128 + (((2 * kb + (lane >> 4)) ^ (r & 7)) << 4), fa[p]);
                    ldmatrix4t(simg + p * M2_BYTES + m * 128 + (((2 * cb + (lane >> 4)) ^ (m & 7)) << 4), fb[p]);
                }
#pragma unroll
                for (int sum = 2; sum >= 0; --sum)
#pragma unroll
                    for (int p = 0; p <= sum; ++p) {
                        mma16816(pe[2 * jb], fa[p], fb[sum - p][0], fb[sum - p][1]);
                        mma16816(pe[2 * jb + 1], fa[p], fb[sum - p][2], fb[sum - p][3]);
                    }
            }
        }
        __syncthreads();   // P has been read
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) put2(16 * rb + g + 8 * i, 4 * (warp >> 2) + n, pe[n][2 * i], pe[n][2 * i + 1]);
        fence_proxy_async_smem();
        __syncthreads();
        if (tid == 0) {
            bulk_store(static_cast<unsigned char *>(a.images) + (((long long)b * a.Hv + h) * N + c) * IMG_BYTES, img, IMG_BYTES);
            bulk_commit();
        }
    }
    if (tid == 0) bulk_wait_all();
}

// ---------------------------------------------------------------------------
// Recurrence over chunks.
// ---------------------------------------------------------------------------
constexpr int NV = 64;                       // value columns of a CTA
constexpr int SCAN_THREADS = 320;            // 8 compute warps, MMA issue, copies
constexpr uint32_t KQ_BOX = 128 * 128;       // 128 rows (64 keys, 64 queries) of 64 values
constexpr uint32_t RU_IMG = 64 * 128;        // one split of a 64 x 64 operand

template <int DK> struct ScanSmem {
    static constexpr uint32_t KQ = KQ_BOX * (DK / 64);
    static constexpr uint32_t S_IMG = DK * 128;
    static constexpr uint32_t kq = 0;                      // two stages
    static constexpr uint32_t img = kq + 2 * KQ;           // [E; P beta E] and meta
    static constexpr uint32_t s = img + IMG_BYTES;
    static constexpr uint32_t ru = s + 3 * S_IMG;
    static constexpr uint32_t bars = ru + 3 * RU_IMG;
    static constexpr uint32_t total = bars + 256 + 1024;   // + alignment slack
};

struct ScanBars {
    uint64_t kq_full[2], kq_empty[2], img_full, img_empty, d1, d2, d3, s_ready, r_ready, u_ready, g_ready, drain;
    uint32_t tmem;
    int abort;
};

__device__ __forceinline__ uint64_t desc128(uint32_t addr, uint32_t lbo, uint32_t sbo) {
    uint64_t d = 0;
    d |= (uint64_t)((addr >> 4) & 0x3FFFu);
    d |= (uint64_t)((lbo >> 4) & 0x3FFFu) << 16;
    d |= (uint64_t)((sbo >> 4) & 0x3FFFu) << 32;
    d |= (uint64_t)1u << 46;
    d |= (uint64_t)2u << 61;
    return d;
}
// K-major: 128-byte rows of 64 K values; a step of 16 is 32 bytes on.
// MN-major: 128-byte rows of 64 M or N values, one row per K value; a step of
// 16 is 2048 bytes on, the next 64 values of M or N are `far` on.
__device__ __forceinline__ uint64_t desc_k(uint32_t base) { return desc128(base, 16u, 1024u); }
__device__ __forceinline__ uint64_t desc_mn(uint32_t base, uint32_t far) { return desc128(base, far, 1024u); }
// The same operand `bytes` on (the address field cannot carry: shared memory
// ends below its 256 KB).
__device__ __forceinline__ uint64_t on(uint64_t desc, uint32_t bytes) { return desc + (bytes >> 4); }
constexpr uint32_t K_STEP = 32, MN_STEP = 2048;
constexpr uint32_t A_MN = 1u << 15, B_MN = 1u << 16;

__device__ __forceinline__ bool scan_wait(uint64_t *bar, uint32_t parity, ScanBars *sb) {
    if (mbar_try_wait(bar, parity)) return true;
    const unsigned long long t0 = global_ns();
    for (;;) {
        if (mbar_try_wait_sleep(bar, parity, 100000)) return true;
        if (*reinterpret_cast<volatile int *>(&sb->abort)) return false;
        if (global_ns() - t0 > WAIT_NS) {
            *reinterpret_cast<volatile int *>(&sb->abort) = 1;
            atomicExch(&g_delta_fault, 1);
            return false;
        }
    }
}

__device__ __forceinline__ void tma_load_4d(void *dst, const void *tmap, int c0, int c1, int c2, int c3, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_addr(dst)),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(smem_addr(bar))
        : "memory");
}

// The 32 values of one token row from column c0 on.
__device__ __forceinline__ void load_bf16_32(const __nv_bfloat16 *p, bool on, uint4 (&v)[4]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = on ? *reinterpret_cast<const uint4 *>(p + 8 * j) : make_uint4(0, 0, 0, 0);
}
__device__ __forceinline__ float bf_at(const uint4 (&v)[4], int i) {
    const uint32_t w = i % 8 / 2 == 0 ? v[i / 8].x : i % 8 / 2 == 1 ? v[i / 8].y : i % 8 / 2 == 2 ? v[i / 8].z : v[i / 8].w;
    return __uint_as_float(i % 2 ? (w & 0xffff0000u) : (w << 16));
}
__device__ __forceinline__ void store_f32_32(float *p, const float (&v)[32]) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
        *reinterpret_cast<float4 *>(p + 4 * j) = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
}
__device__ __forceinline__ void store_bf16_32(__nv_bfloat16 *p, const float (&v)[32]) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
        *reinterpret_cast<uint4 *>(p + 8 * j) =
            make_uint4(pack2(v[8 * j], v[8 * j + 1]), pack2(v[8 * j + 2], v[8 * j + 3]), pack2(v[8 * j + 4], v[8 * j + 5]),
                       pack2(v[8 * j + 6], v[8 * j + 7]));
}
__device__ __forceinline__ void load_acc(uint32_t addr, float (&v)[32]) {
    uint32_t r[32];
    tmem_ld32(addr, r);
    tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
// The sum of P column blocks, 64 apart: an accumulator for each part of the
// split operand, so that one product covers all parts.
template <int P> __device__ __forceinline__ void load_parts(uint32_t addr, float (&v)[32]) {
    uint32_t r[P][32];
#pragma unroll
    for (int p = 0; p < P; ++p) tmem_ld32(addr + p * NV, r[p]);
    tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        float t = __uint_as_float(r[P - 1][i]);
#pragma unroll
        for (int p = P - 2; p >= 0; --p) t += __uint_as_float(r[p][i]);
        v[i] = t;
    }
}
// What the compute warps wrote to shared memory and read from TMEM is done
// before the MMA warp goes on.
__device__ __forceinline__ void hand_over(uint64_t *bar, int lane) {
    fence_proxy_async_smem();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
}

// The copy warp of both recurrences: each chunk's keys and queries (two
// stages) and its matrix with the factors (one), in the order of the chunks
// or, REV, from the last one.
template <int DK, bool REV>
__device__ __forceinline__ void copy_chunks(unsigned char *kq, unsigned char *img, const CUtensorMap *tmap_k,
                                            const CUtensorMap *tmap_q, const Args &a, ScanBars *sb, int hk, int b,
                                            long long bh, int N) {
    constexpr uint32_t KQ = KQ_BOX * (DK / 64);
    bool ok = true;
    int it = 0;
    for (; it < N; ++it) {
        const int st = it & 1, c = REV ? N - 1 - it : it;
        if (it >= 2) ok = __all_sync(0xffffffffu, scan_wait(&sb->kq_empty[st], ((it >> 1) - 1) & 1, sb));
        if (!ok) break;
        if (elect_one()) {
            unsigned char *to = kq + st * KQ;
            mbar_arrive_tx(&sb->kq_full[st], KQ);
#pragma unroll
            for (int x = 0; x < DK / 64; ++x) {
                tma_load_4d(to + x * KQ_BOX, tmap_k, 64 * x, hk, c * C, b, &sb->kq_full[st]);
                tma_load_4d(to + x * KQ_BOX + KQ_BOX / 2, tmap_q, 64 * x, hk, c * C, b, &sb->kq_full[st]);
            }
        }
        __syncwarp();
        if (it >= 1) ok = __all_sync(0xffffffffu, scan_wait(&sb->img_empty, (it - 1) & 1, sb));
        if (!ok) {
            ++it;
            break;
        }
        if (elect_one()) {
            mbar_arrive_tx(&sb->img_full, IMG_BYTES);
            bulk_load(img, static_cast<const unsigned char *>(a.images) + (bh * N + c) * IMG_BYTES, IMG_BYTES, &sb->img_full);
        }
        __syncwarp();
    }
    if (!ok) {   // a wait gave up: copies in flight land before the CTA ends
        const unsigned long long t0 = global_ns();
        for (int j = max(0, it - 2); j < it; ++j)
            while (!mbar_try_wait_sleep(&sb->kq_full[j & 1], (j >> 1) & 1, 100000))
                if (global_ns() - t0 > 200000000ull) break;
        while (global_ns() - t0 < 1000000ull) {}
    }
}

// Every MMA issued has completed before TMEM is freed (whole warp).
__device__ __forceinline__ void drain_products(ScanBars *sb) {
    if (elect_one()) mma_commit(&sb->drain);
    __syncwarp();
    const unsigned long long t0 = global_ns();
    while (!mbar_try_wait_sleep(&sb->drain, 0, 100000))
        if (global_ns() - t0 > 200000000ull) break;
}

template <int DK>
__global__ void __launch_bounds__(SCAN_THREADS, 1)
delta_scan_kernel(const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_q, const Args a) {
    using L = ScanSmem<DK>;
    extern __shared__ __align__(1024) unsigned char raw[];
    unsigned char *smem = raw + ((1024u - (smem_addr(raw) & 1023u)) & 1023u);
    ScanBars *sb = reinterpret_cast<ScanBars *>(smem + L::bars);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int n0 = blockIdx.x * NV, h = blockIdx.y, b = blockIdx.z, hk = h / (a.Hv / a.Hk);
    const int N = chunks(a.L);
    const long long bh = (long long)b * a.Hv + h;
    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) mbar_init(&sb->kq_full[i], 1), mbar_init(&sb->kq_empty[i], 1);
        mbar_init(&sb->img_full, 1), mbar_init(&sb->img_empty, 8);
        mbar_init(&sb->d1, 1), mbar_init(&sb->d2, 1), mbar_init(&sb->d3, 1);
        mbar_init(&sb->s_ready, 8), mbar_init(&sb->r_ready, 4), mbar_init(&sb->u_ready, 4);
        mbar_init(&sb->drain, 1);
        sb->abort = 0;
        fence_mbar_init();
    }
    if (warp == 8) {
        tmem_alloc(&sb->tmem, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sb->tmem, D1 = tmem, D2 = tmem + 3 * NV, D3 = tmem + 5 * NV;

    if (warp == 9) {
        copy_chunks<DK, false>(smem + L::kq, smem + L::img, &tmap_k, &tmap_q, a, sb, hk, b, bh, N);
    } else if (warp == 8) {
        // ---------------------------------------------------------- products
        const uint32_t w1 = idesc_bf16_f32(128, NV) | B_MN, w2 = idesc_bf16_f32(128, 2 * NV) | B_MN,
                       w3 = idesc_bf16_f32(128, 3 * NV) | B_MN;
        const uint64_t mat = desc_k(smem_addr(smem + L::img)), S = desc_mn(smem_addr(smem + L::s), L::S_IMG),
                       R = desc_mn(smem_addr(smem + L::ru), RU_IMG);
        bool ok = true;
        for (int c = 0; ok && c < N; ++c) {
            const int st = c & 1;
            const uint32_t kq = smem_addr(smem + L::kq + st * L::KQ);
            const uint64_t rows = desc_k(kq), cols = desc_mn(kq, KQ_BOX);
            ok = scan_wait(&sb->kq_full[st], (c >> 1) & 1, sb) && scan_wait(&sb->s_ready, c & 1, sb);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
                for (int k = 0; k < DK / 16; ++k)
                    mma_bf16(D1, on(rows, k / 4 * KQ_BOX + k % 4 * K_STEP), on(S, k * MN_STEP), w3, k > 0);
                mma_commit(&sb->d1);
            }
            __syncwarp();
            ok = scan_wait(&sb->img_full, c & 1, sb) && scan_wait(&sb->r_ready, c & 1, sb);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
                for (int k = 0; k < C / 16; ++k) {
                    mma_bf16(D2, on(mat, M2_BYTES + k * K_STEP), on(R, k * MN_STEP), w2, k > 0);
                    mma_bf16(D2, on(mat, 2 * M2_BYTES + k * K_STEP), on(R, k * MN_STEP), w1, 1);
                    mma_bf16(D2, on(mat, k * K_STEP), on(R, 2 * RU_IMG + k * MN_STEP), w1, 1);
                    mma_bf16(D2, on(mat, k * K_STEP), on(R, k * MN_STEP), w2, 1);
                }
                mma_commit(&sb->d2);
            }
            __syncwarp();
            ok = __all_sync(0xffffffffu, scan_wait(&sb->u_ready, c & 1, sb));
            if (!ok) break;
            tc_fence_after();
            // M is 128 for heads of 64 too: their lanes 64..127 of D3 come from
            // whatever follows the keys in shared memory, and are not read
            if (elect_one()) {
#pragma unroll
                for (int k = 0; k < C / 16; ++k) mma_bf16(D3, on(cols, k * MN_STEP), on(R, k * MN_STEP), w3 | A_MN, k > 0);
                mma_commit(&sb->d3);
                mma_commit(&sb->kq_empty[st]);
            }
            __syncwarp();
        }
        drain_products(sb);
    } else {
        // ---------------------------------------------------------- compute
        // warp w: TMEM lanes 32 (w % 4) on, columns 32 (w / 4) on.  Lanes 0..63
        // are tokens of R, e and U, lanes 64..127 tokens of o; in D3 and in
        // the state a lane is a key index.
        const int q = warp & 3, c0 = warp / 4 * 32, row = 32 * q + lane;
        __syncwarp();
        const bool keys = q < 2;                 // R, U rows; else o rows
        const int tk = row & 63;                 // token in the chunk
        const uint32_t lane_base = (uint32_t)(32 * q) << 16;
        const uint32_t d1 = D1 + lane_base + c0, d2 = D2 + lane_base + c0, d3 = D3 + lane_base + c0;
        const uint32_t sS = smem_addr(smem + L::s), sR = smem_addr(smem + L::ru);
        const Meta *meta = reinterpret_cast<const Meta *>(smem + L::img + 3 * M2_BYTES);
        const bool state = row < DK;
        const long long mat = (long long)DK * a.Dv;
        float S[32];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float4 t = (a.s0 && state) ? *reinterpret_cast<const float4 *>(a.s0 + bh * mat + (long long)row * a.Dv + n0 + c0 + 4 * j)
                                             : make_float4(0, 0, 0, 0);
            S[4 * j] = t.x, S[4 * j + 1] = t.y, S[4 * j + 2] = t.z, S[4 * j + 3] = t.w;
        }
        if (state) store_split32(sS, L::S_IMG, row, c0, S);
        hand_over(&sb->s_ready, lane);
        bool ok = true;
        for (int c = 0; c < N; ++c) {
            const int t = c * C + tk;
            const bool on = t < a.L;
            const long long tok = (long long)b * a.L + t;
            const long long out = (tok * a.Hv + h) * a.Dv + n0 + c0;
            uint4 v[4];
            if (keys)
                load_bf16_32(static_cast<const __nv_bfloat16 *>(a.v) + tok * a.ldv + (long long)h * a.Dv + n0 + c0, on, v);
            if (a.states && state) store_f32_32(a.states + (bh * (N + 1) + c) * mat + (long long)row * a.Dv + n0 + c0, S);
            float x[32], y[32];
            ok = scan_wait(&sb->img_full, c & 1, sb) && scan_wait(&sb->d1, c & 1, sb);
            if (!__all_sync(0xffffffffu, ok)) break;
            tc_fence_after();
            load_parts<3>(d1, x);
            const float up = meta->up[tk], down = meta->down[tk], be = meta->beta[tk], last = meta->last;
            if (keys) {
#pragma unroll
                for (int i = 0; i < 32; ++i) x[i] = fmaf(-up, x[i], bf_at(v, i));
                store_split32(sR, RU_IMG, tk, c0, x);
                hand_over(&sb->r_ready, lane);
            }
            ok = scan_wait(&sb->d2, c & 1, sb);
            if (!__all_sync(0xffffffffu, ok)) break;
            tc_fence_after();
            if (lane == 0) mbar_arrive(&sb->img_empty);   // D2 is done with the matrix, this warp with its factors
            load_parts<2>(d2, y);
            if (keys) {
                if (a.e && on) store_f32_32(a.e + out, y);
#pragma unroll
                for (int i = 0; i < 32; ++i) y[i] *= be * down;
                store_split32(sR, RU_IMG, tk, c0, y);
                hand_over(&sb->u_ready, lane);
            } else if (on) {
                const float w = a.scale * up;
#pragma unroll
                for (int i = 0; i < 32; ++i) y[i] = fmaf(w, x[i], y[i]);
                store_bf16_32(static_cast<__nv_bfloat16 *>(a.o) + tok * a.ldo + (long long)h * a.Dv + n0 + c0, y);
                if (a.o32) store_f32_32(a.o32 + out, y);
            }
            ok = scan_wait(&sb->d3, c & 1, sb);
            if (!__all_sync(0xffffffffu, ok)) break;
            tc_fence_after();
            if (state) {
                load_parts<3>(d3, x);
#pragma unroll
                for (int i = 0; i < 32; ++i) S[i] = fmaf(last, S[i], x[i]);
                if (c + 1 < N) store_split32(sS, L::S_IMG, row, c0, S);
            }
            if (c + 1 < N) hand_over(&sb->s_ready, lane);
        }
        if (state) {
            if (a.s_last) store_f32_32(a.s_last + bh * mat + (long long)row * a.Dv + n0 + c0, S);
            if (a.states) store_f32_32(a.states + (bh * (N + 1) + N) * mat + (long long)row * a.Dv + n0 + c0, S);
        }
        tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
    if (warp == 8) tmem_dealloc(tmem, 512);
}

// ---------------------------------------------------------------------------
// The adjoint over chunks, last chunk first, with Z = dL/dS at the chunk's end
// and [T; P T] from the preparation (T = (I + strict lower(beta_i D_ij k_i.k_j))^-1):
//   X = T^T (e^{G_64 - G} K Z) + (P T)^T dO          X_t = dL/du_t
//   dv = beta X
//   Z_start = e^{G_64} Z + K^T (-e^G dv) + Q^T (scale e^G dO)
// the forward's three products transposed, on the same tiles: D1 = [K; Q] Z,
// D2 = [T; P T]^T [e^{..} K Z; dO] (depth 128), D3 = [K; Q]^T [..; ..] (depth
// 128).  Each token's parts of X . e, v . dv and o . dO (32 columns a thread)
// and each chunk's <S, Z> go to the workspace for the gates' gradients.
// ---------------------------------------------------------------------------
template <int DK> struct AdjSmem {
    static constexpr uint32_t KQ = KQ_BOX * (DK / 64);
    static constexpr uint32_t S_IMG = DK * 128;
    static constexpr uint32_t kq = 0;                      // two stages
    static constexpr uint32_t img = kq + 2 * KQ;
    static constexpr uint32_t s = img + IMG_BYTES;         // Z, three images
    static constexpr uint32_t ru = s + 3 * S_IMG;          // e^{..} K Z, then -e^G dv: three images
    static constexpr uint32_t yq = ru + 3 * RU_IMG;        // scale e^G dO: three images
    static constexpr uint32_t go = yq + 3 * RU_IMG;        // dO
    static constexpr uint32_t bars = go + RU_IMG;
    static constexpr uint32_t total = bars + 256 + 1024;
};

template <int DK>
__global__ void __launch_bounds__(SCAN_THREADS, 1)
delta_adjoint_kernel(const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_q, const Args a) {
    using L = AdjSmem<DK>;
    extern __shared__ __align__(1024) unsigned char raw[];
    unsigned char *smem = raw + ((1024u - (smem_addr(raw) & 1023u)) & 1023u);
    ScanBars *sb = reinterpret_cast<ScanBars *>(smem + L::bars);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int n0 = blockIdx.x * NV, h = blockIdx.y, b = blockIdx.z, hk = h / (a.Hv / a.Hk);
    const int N = chunks(a.L);
    const long long bh = (long long)b * a.Hv + h;
    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) mbar_init(&sb->kq_full[i], 1), mbar_init(&sb->kq_empty[i], 1);
        mbar_init(&sb->img_full, 1), mbar_init(&sb->img_empty, 8);
        mbar_init(&sb->d1, 1), mbar_init(&sb->d2, 1), mbar_init(&sb->d3, 1);
        mbar_init(&sb->s_ready, 8), mbar_init(&sb->r_ready, 4), mbar_init(&sb->u_ready, 4), mbar_init(&sb->g_ready, 4);
        mbar_init(&sb->drain, 1);
        sb->abort = 0;
        fence_mbar_init();
    }
    if (warp == 8) {
        tmem_alloc(&sb->tmem, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // D3 takes D1's place: the warps that read D1 hand over after it
    const uint32_t tmem = sb->tmem, D1 = tmem, D2 = tmem + 3 * NV, D3 = tmem;

    if (warp == 9) {
        copy_chunks<DK, true>(smem + L::kq, smem + L::img, &tmap_k, &tmap_q, a, sb, hk, b, bh, N);
    } else if (warp == 8) {
        const uint32_t w1 = idesc_bf16_f32(128, NV) | B_MN, w2 = idesc_bf16_f32(128, 2 * NV) | B_MN,
                       w3 = idesc_bf16_f32(128, 3 * NV) | B_MN;
        const uint64_t mat = desc_mn(smem_addr(smem + L::img), M2_BYTES), S = desc_mn(smem_addr(smem + L::s), L::S_IMG),
                       R = desc_mn(smem_addr(smem + L::ru), RU_IMG), Y = desc_mn(smem_addr(smem + L::yq), RU_IMG),
                       G = desc_mn(smem_addr(smem + L::go), RU_IMG);
        bool ok = true;
        for (int it = 0; ok && it < N; ++it) {
            const int st = it & 1;
            const uint32_t kq = smem_addr(smem + L::kq + st * L::KQ);
            const uint64_t rows = desc_k(kq), cols = desc_mn(kq, KQ_BOX);
            ok = scan_wait(&sb->kq_full[st], (it >> 1) & 1, sb) && scan_wait(&sb->s_ready, it & 1, sb);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
                for (int k = 0; k < DK / 16; ++k)
                    mma_bf16(D1, on(rows, k / 4 * KQ_BOX + k % 4 * K_STEP), on(S, k * MN_STEP), w3, k > 0);
                mma_commit(&sb->d1);
            }
            __syncwarp();
            // (P T)^T dO waits for nothing but its operands
            ok = scan_wait(&sb->img_full, it & 1, sb) && scan_wait(&sb->g_ready, it & 1, sb);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tc_fence_after();
            // the matrix transposed has 64 rows: lanes 64..127 of D2 come from
            // what follows it in shared memory, and are not read
            if (elect_one()) {
#pragma unroll
                for (int k = 0; k < C / 16; ++k)
#pragma unroll
                    for (int p = 2; p >= 0; --p)
                        mma_bf16(D2, on(mat, p * M2_BYTES + M2_BYTES / 2 + k * MN_STEP), on(G, k * MN_STEP), w1 | A_MN,
                                 k > 0 || p < 2);
            }
            __syncwarp();
            ok = __all_sync(0xffffffffu, scan_wait(&sb->r_ready, it & 1, sb));
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
                for (int k = 0; k < C / 16; ++k) {
                    mma_bf16(D2 + NV, on(mat, M2_BYTES + k * MN_STEP), on(R, k * MN_STEP), w2 | A_MN, k > 0);
                    mma_bf16(D2, on(mat, 2 * M2_BYTES + k * MN_STEP), on(R, k * MN_STEP), w1 | A_MN, 1);
                    mma_bf16(D2, on(mat, k * MN_STEP), on(R, 2 * RU_IMG + k * MN_STEP), w1 | A_MN, 1);
                    mma_bf16(D2 + NV, on(mat, k * MN_STEP), on(R, k * MN_STEP), w2 | A_MN, 1);
                }
                mma_commit(&sb->d2);
            }
            __syncwarp();
            ok = __all_sync(0xffffffffu, scan_wait(&sb->u_ready, it & 1, sb));
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
                for (int k = 0; k < 2 * C / 16; ++k)
                    mma_bf16(D3, on(cols, k * MN_STEP), on(k < 4 ? R : Y, k % 4 * MN_STEP), w3 | A_MN, k > 0);
                mma_commit(&sb->d3);
                mma_commit(&sb->kq_empty[st]);
            }
            __syncwarp();
        }
        drain_products(sb);
    } else {
        const int q = warp & 3, c0 = warp / 4 * 32, row = 32 * q + lane;
        const bool keys = q < 2;
        const int tk = row & 63;
        const uint32_t lane_base = (uint32_t)(32 * q) << 16;
        const uint32_t d1 = D1 + lane_base + c0, d2 = D2 + lane_base + c0, d3 = D3 + lane_base + c0;
        const uint32_t sS = smem_addr(smem + L::s), sR = smem_addr(smem + L::ru), sY = smem_addr(smem + L::yq),
                       sG = smem_addr(smem + L::go);
        const Meta *meta = reinterpret_cast<const Meta *>(smem + L::img + 3 * M2_BYTES);
        const bool state = row < DK;
        const long long mat = (long long)DK * a.Dv;
        const int parts = a.Dv / 32, part = (n0 + c0) / 32;
        const long long nrows = (long long)a.B * a.L * a.Hv;
        float *pb = a.dots, *pk = a.dots + nrows * parts, *pq = pk + nrows * parts;
        float S[32];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float4 t = (a.ds_last && state)
                                 ? *reinterpret_cast<const float4 *>(a.ds_last + bh * mat + (long long)row * a.Dv + n0 + c0 + 4 * j)
                                 : make_float4(0, 0, 0, 0);
            S[4 * j] = t.x, S[4 * j + 1] = t.y, S[4 * j + 2] = t.z, S[4 * j + 3] = t.w;
        }
        if (state) store_split32(sS, L::S_IMG, row, c0, S);
        hand_over(&sb->s_ready, lane);
        for (int it = 0; it < N; ++it) {
            const int c = N - 1 - it, t = c * C + tk;
            const bool on = t < a.L;
            const long long tok = (long long)b * a.L + t, hv = tok * a.Hv + h;
            const long long out = hv * a.Dv + n0 + c0;
            uint4 v[4];
            load_bf16_32(keys ? static_cast<const __nv_bfloat16 *>(a.v) + tok * a.ldv + (long long)h * a.Dv + n0 + c0
                              : static_cast<const __nv_bfloat16 *>(a.dout) + tok * a.lddo + (long long)h * a.Dv + n0 + c0,
                         on, v);
            float x[32];
            bool ok = scan_wait(&sb->img_full, it & 1, sb);
            if (!__all_sync(0xffffffffu, ok)) break;
            const float up = meta->up[tk], down = meta->down[tk], be = meta->beta[tk], last = meta->last;
            if (!keys) {   // dO as it is for D2, scaled for D3
                const uint32_t at = sG + (uint32_t)tk * 128u;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    sts128(at + (uint32_t)(((c0 / 8 + j) ^ (tk & 7)) << 4), v[j].x, v[j].y, v[j].z, v[j].w);
                const float w = a.scale * up;
#pragma unroll
                for (int i = 0; i < 32; ++i) x[i] = w * bf_at(v, i);
                store_split32(sY, RU_IMG, tk, c0, x);
                hand_over(&sb->g_ready, lane);
            }
            // Z for the chunk's local gradients, <S, Z> at its end
            if (state) {
                store_f32_32(a.z + (bh * N + c) * mat + (long long)row * a.Dv + n0 + c0, S);
                const float *s = a.states + (bh * (N + 1) + c + 1) * mat + (long long)row * a.Dv + n0 + c0;
                float w = 0.0f;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float4 f = *reinterpret_cast<const float4 *>(s + 4 * j);
                    w += f.x * S[4 * j] + f.y * S[4 * j + 1] + f.z * S[4 * j + 2] + f.w * S[4 * j + 3];
                }
                for (int m = 16; m > 0; m >>= 1) w += __shfl_xor_sync(0xffffffffu, w, m);
                if (lane == 0) a.inner[(bh * (N + 1) + c + 1) * a.parts + blockIdx.x * (DK / 16) + q * 2 + warp / 4] = w;
            }
            if (!keys && on) {
                float w = 0.0f;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float4 f = *reinterpret_cast<const float4 *>(a.o32 + out + 4 * j);
                    w += f.x * bf_at(v, 4 * j) + f.y * bf_at(v, 4 * j + 1) + f.z * bf_at(v, 4 * j + 2) + f.w * bf_at(v, 4 * j + 3);
                }
                pq[hv * parts + part] = w;
            }
            ok = scan_wait(&sb->d1, it & 1, sb);
            if (!__all_sync(0xffffffffu, ok)) break;
            tc_fence_after();
            if (keys) {
                load_parts<3>(d1, x);
#pragma unroll
                for (int i = 0; i < 32; ++i) x[i] *= down;
                store_split32(sR, RU_IMG, tk, c0, x);
                hand_over(&sb->r_ready, lane);
            }
            ok = scan_wait(&sb->d2, it & 1, sb);
            if (!__all_sync(0xffffffffu, ok)) break;
            tc_fence_after();
            if (lane == 0) mbar_arrive(&sb->img_empty);
            if (keys) {
                load_parts<3>(d2, x);
                float y[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) y[i] = -up * (be * x[i]);
                store_split32(sR, RU_IMG, tk, c0, y);
                hand_over(&sb->u_ready, lane);
                if (on) {
                    float w = 0.0f, r = 0.0f;
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float4 f = *reinterpret_cast<const float4 *>(a.e + out + 4 * j);
                        w += f.x * x[4 * j] + f.y * x[4 * j + 1] + f.z * x[4 * j + 2] + f.w * x[4 * j + 3];
                    }
                    store_f32_32(a.x + out, x);
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        x[i] *= be;
                        r = fmaf(x[i], bf_at(v, i), r);
                    }
                    store_bf16_32(static_cast<__nv_bfloat16 *>(a.dv) + tok * a.lddv + (long long)h * a.Dv + n0 + c0, x);
                    pb[hv * parts + part] = w, pk[hv * parts + part] = r;
                }
            }
            ok = scan_wait(&sb->d3, it & 1, sb);
            if (!__all_sync(0xffffffffu, ok)) break;
            tc_fence_after();
            if (state) {
                load_parts<3>(d3, x);
#pragma unroll
                for (int i = 0; i < 32; ++i) S[i] = fmaf(last, S[i], x[i]);
                if (c > 0) store_split32(sS, L::S_IMG, row, c0, S);
            }
            if (c > 0) hand_over(&sb->s_ready, lane);
        }
        if (state && a.ds0) store_f32_32(a.ds0 + bh * mat + (long long)row * a.Dv + n0 + c0, S);
        tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
    if (warp == 8) tmem_dealloc(tmem, 512);
}

// ---------------------------------------------------------------------------
// dq and dk, all chunks at once: one CTA per chunk and key head, summing over
// its value heads.  With S0 and Z the state at the chunk's start and the
// adjoint at its end, U = beta e, and N_ij = scale D_ij dO_i.U_j (j <= i),
// W_ij = -D_ij dv_i.U_j (j < i):
//   dq = scale e^G dO S0^T + N K
//   dk = e^{G_64 - G} U Z^T - e^G dv S0^T + W K + W^T K + N^T Q
// as tcgen05 products of M = 128 with the rows of [dv; dO] stacked, so that
// dk lies in TMEM lanes 0..63 and dq in 64..127:
//   D1 = [dv; dO] S0^T,  D3 = [dv; dO] U^T,  D2 = [U; -] Z^T,
//   D4 = [W; N] K,  D5 = [W; N]^T [K; Q].
// dq and dk are rounded to bf16, so that 32-bit operands are carried as two
// bf16 values here (2^-17), three products against another pair, two against
// a bf16 operand.
// Bound: the states and adjoints it reads (128 KB per chunk and head).
// ---------------------------------------------------------------------------
constexpr int LT = 512;

template <int DK, int DV> struct LocalSmem {
    static constexpr uint32_t KQ = KQ_BOX * (DK / 64);
    static constexpr uint32_t A_IMG = 128 * 128 * (DV / 64);   // [dv; dO]
    static constexpr uint32_t U_IMG = 64 * 128 * (DV / 64);
    static constexpr uint32_t S_IMG = DK * 128 * (DV / 64);
    static constexpr uint32_t kq = 0;
    static constexpr uint32_t a = kq + KQ;                     // two images; [W; N], two images, later
    static constexpr uint32_t u = a + (2 * A_IMG > 2 * M2_BYTES ? 2 * A_IMG : 2 * M2_BYTES);
    static constexpr uint32_t s = u + 2 * U_IMG;               // S0, then Z: two images
    static constexpr uint32_t meta = s + 2 * S_IMG;
    static constexpr uint32_t bars = meta + META_BYTES;
    static constexpr uint32_t total = bars + 64 + 1024;
    // M = 128 over 64 rows of U reads 8 KB past the last box
    static_assert(2 * S_IMG >= 8192, "rows past U are in shared memory");
};

struct LocalBars {
    uint64_t first, second;
    uint32_t tmem;
};

__device__ __forceinline__ void split2(float a, float b, uint32_t &h, uint32_t &m) {
    h = pack2(a, b);
    m = pack2(a - __uint_as_float(h << 16), b - __uint_as_float(h & 0xffff0000u));
}
// Eight fp32 values times w as a 16-byte piece of two images.
__device__ __forceinline__ void put_split8(unsigned char *img, uint32_t stride, uint32_t box, int row, int d,
                                           const float4 &x, const float4 &y, float w) {
    uint32_t h[4], m[4];
    split2(x.x * w, x.y * w, h[0], m[0]);
    split2(x.z * w, x.w * w, h[1], m[1]);
    split2(y.x * w, y.y * w, h[2], m[2]);
    split2(y.z * w, y.w * w, h[3], m[3]);
    unsigned char *to = img + d / 64 * box + row * 128 + (((d % 64 / 8) ^ (row & 7)) << 4);
    *reinterpret_cast<uint4 *>(to) = make_uint4(h[0], h[1], h[2], h[3]);
    *reinterpret_cast<uint4 *>(to + stride) = make_uint4(m[0], m[1], m[2], m[3]);
}
__device__ __forceinline__ bool local_wait(uint64_t *bar, uint32_t parity) {
    if (mbar_try_wait(bar, parity)) return true;
    const unsigned long long t0 = global_ns();
    while (!mbar_try_wait_sleep(bar, parity, 100000))
        if (global_ns() - t0 > WAIT_NS) {
            atomicExch(&g_delta_fault, 1);
            return false;
        }
    return true;
}

template <int DK, int DV> __global__ void __launch_bounds__(LT, 1) delta_local_kernel(const Args a) {
    using L = LocalSmem<DK, DV>;
    extern __shared__ __align__(1024) unsigned char raw[];
    unsigned char *smem = raw + ((1024u - (smem_addr(raw) & 1023u)) & 1023u);
    LocalBars *lb = reinterpret_cast<LocalBars *>(smem + L::bars);
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int c = blockIdx.x, hk = blockIdx.y, b = blockIdx.z, group = a.Hv / a.Hk;
    const int t0 = c * C, nt = min(C, a.L - t0), N = chunks(a.L);
    const long long row0 = (long long)b * a.L + t0, mat = (long long)DK * DV;
    if (tid == 0) {
        mbar_init(&lb->first, 1);
        mbar_init(&lb->second, 1);
        fence_mbar_init();
    }
    if (warp == 0) {
        tmem_alloc(&lb->tmem, 512);
        tmem_relinquish();
    }
    const uint4 none = make_uint4(0, 0, 0, 0);
    for (int i = tid; i < 128 * (DK / 8); i += LT) {
        const int r = i / (DK / 8), d = i % (DK / 8) * 8, t = r & 63;
        const __nv_bfloat16 *p = r < C ? static_cast<const __nv_bfloat16 *>(a.k) + (row0 + t) * a.ldk + hk * DK + d
                                       : static_cast<const __nv_bfloat16 *>(a.q) + (row0 + t) * a.ldq + hk * DK + d;
        *reinterpret_cast<uint4 *>(smem + L::kq + d / 64 * KQ_BOX + r * 128 + (((d % 64 / 8) ^ (r & 7)) << 4)) =
            t < nt ? *reinterpret_cast<const uint4 *>(p) : none;
    }
    for (int i = tid; i < C * (DV / 8); i += LT) {   // dO is bf16: the rows of its second image are zero
        const int r = C + i / (DV / 8), d = i % (DV / 8) * 8;
        *reinterpret_cast<uint4 *>(smem + L::a + L::A_IMG + d / 64 * M2_BYTES + r * 128 + (((d % 64 / 8) ^ (r & 7)) << 4)) = none;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = lb->tmem, D1 = tmem, D2 = tmem + 128, D4 = tmem + 256, D3 = tmem + 384, D5 = tmem + 384;
    const uint64_t A0 = desc_k(smem_addr(smem + L::a)), AT = desc_mn(smem_addr(smem + L::a), M2_BYTES),
                   U0 = desc_k(smem_addr(smem + L::u)), S0 = desc_k(smem_addr(smem + L::s)),
                   cols = desc_mn(smem_addr(smem + L::kq), KQ_BOX);
    Meta *meta = reinterpret_cast<Meta *>(smem + L::meta);
    // warp w: TMEM lanes 32 (w % 4) on, columns 32 (w / 4) on
    const int row = 32 * (warp & 3) + lane, c0 = warp / 4 * 32, tk = row & 63;
    const bool keys = row < C;
    const uint32_t lane_base = (uint32_t)(32 * (warp & 3)) << 16;
    float acc[32] = {};
    bool ok = true;
    for (int j = 0; j < group; ++j) {
        const int h = hk * group + j;
        const long long bh = (long long)b * a.Hv + h;
        const unsigned char *img = static_cast<const unsigned char *>(a.images) + (bh * N + c) * IMG_BYTES;
        for (int i = tid; i < (int)(sizeof(Meta) / 4); i += LT)
            reinterpret_cast<float *>(meta)[i] = reinterpret_cast<const float *>(img + 3 * M2_BYTES)[i];
        for (int i = tid; i < C * (DV / 8); i += LT) {
            const int t = i / (DV / 8), d = i % (DV / 8) * 8;
            const long long hv = (row0 + t) * a.Hv + h;
            float4 x0 = make_float4(0, 0, 0, 0), x1 = x0, e0 = x0, e1 = x0;
            uint4 g = none;
            float be = 0.0f;
            if (t < nt) {
                x0 = *reinterpret_cast<const float4 *>(a.x + hv * DV + d), x1 = *reinterpret_cast<const float4 *>(a.x + hv * DV + d + 4);
                e0 = *reinterpret_cast<const float4 *>(a.e + hv * DV + d), e1 = *reinterpret_cast<const float4 *>(a.e + hv * DV + d + 4);
                g = *reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(a.dout) + (row0 + t) * a.lddo +
                                                     (long long)h * DV + d);
                be = a.beta[hv];
            }
            put_split8(smem + L::a, L::A_IMG, M2_BYTES, t, d, x0, x1, be);
            put_split8(smem + L::u, L::U_IMG, RU_IMG, t, d, e0, e1, be);
            const int r = C + t;
            *reinterpret_cast<uint4 *>(smem + L::a + d / 64 * M2_BYTES + r * 128 + (((d % 64 / 8) ^ (r & 7)) << 4)) = g;
        }
        const float *s0 = a.states + (bh * (N + 1) + c) * mat, *z = a.z + (bh * N + c) * mat;
        for (int i = tid; i < DK * (DV / 8); i += LT) {
            const int r = i / (DV / 8), d = i % (DV / 8) * 8;
            put_split8(smem + L::s, L::S_IMG, DK * 128, r, d, *reinterpret_cast<const float4 *>(s0 + r * DV + d),
                       *reinterpret_cast<const float4 *>(s0 + r * DV + d + 4), 1.0f);
        }
        fence_proxy_async_smem();
        __syncthreads();
        if (warp == 0) {
            const uint32_t id = idesc_bf16_f32(128, DK), idU = idesc_bf16_f32(128, 64);
            if (elect_one()) {
#pragma unroll
                for (int sum = 1; sum >= 0; --sum)
#pragma unroll
                    for (int p = 0; p <= sum; ++p)
#pragma unroll
                        for (int k = 0; k < DV / 16; ++k) {
                            const uint64_t da = on(A0, p * L::A_IMG + k / 4 * M2_BYTES + k % 4 * K_STEP);
                            const bool add = !(sum == 1 && p == 0 && k == 0);
                            mma_bf16(D1, da, on(S0, (sum - p) * L::S_IMG + k / 4 * (DK * 128) + k % 4 * K_STEP), id, add);
                            mma_bf16(D3, da, on(U0, (sum - p) * L::U_IMG + k / 4 * RU_IMG + k % 4 * K_STEP), idU, add);
                        }
                mma_commit(&lb->first);
            }
            __syncwarp();
        }
        float4 zr[(DK * DV / 4 + LT - 1) / LT];
#pragma unroll
        for (int n = 0; n < DK * DV / 8 / LT; ++n) {
            const int i = tid + n * LT;
            zr[2 * n] = *reinterpret_cast<const float4 *>(z + i * 8);
            zr[2 * n + 1] = *reinterpret_cast<const float4 *>(z + i * 8 + 4);
        }
        ok = local_wait(&lb->first, j & 1) && ok;
        tc_fence_after();
#pragma unroll
        for (int n = 0; n < DK * DV / 8 / LT; ++n) {
            const int i = tid + n * LT;
            put_split8(smem + L::s, L::S_IMG, DK * 128, i / (DV / 8), i % (DV / 8) * 8, zr[2 * n], zr[2 * n + 1], 1.0f);
        }
        if (c0 < 64) {   // [W; N] into the first images' place
            float x[32];
            load_acc(D3 + lane_base + c0, x);
            const float gh = meta->hi[tk], gl = meta->lo[tk];
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                const int col = c0 + i;
                const bool in = keys ? col < tk : col <= tk;
                const float w = in ? expf((gh - meta->hi[col]) + (gl - meta->lo[col])) : 0.0f;
                x[i] = in ? (keys ? -w : a.scale * w) * x[i] : 0.0f;
            }
#pragma unroll
            for (int n = 0; n < 4; ++n)
                put_split8(smem + L::a, M2_BYTES, 0, row, c0 + 8 * n, make_float4(x[8 * n], x[8 * n + 1], x[8 * n + 2], x[8 * n + 3]),
                           make_float4(x[8 * n + 4], x[8 * n + 5], x[8 * n + 6], x[8 * n + 7]), 1.0f);
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
        if (warp == 0) {
            const uint32_t id = idesc_bf16_f32(128, DK), idB = id | B_MN, idAB = idB | A_MN;
            if (elect_one()) {
#pragma unroll
                for (int sum = 1; sum >= 0; --sum)
#pragma unroll
                    for (int p = 0; p <= sum; ++p)
#pragma unroll
                        for (int k = 0; k < DV / 16; ++k)
                            mma_bf16(D2, on(U0, p * L::U_IMG + k / 4 * RU_IMG + k % 4 * K_STEP),
                                     on(S0, (sum - p) * L::S_IMG + k / 4 * (DK * 128) + k % 4 * K_STEP), id,
                                     !(sum == 1 && p == 0 && k == 0));
#pragma unroll
                for (int p = 1; p >= 0; --p) {
#pragma unroll
                    for (int k = 0; k < C / 16; ++k)
                        mma_bf16(D4, on(A0, p * M2_BYTES + k * K_STEP), on(cols, k * MN_STEP), idB, !(p == 1 && k == 0));
#pragma unroll
                    for (int k = 0; k < 2 * C / 16; ++k)
                        mma_bf16(D5, on(AT, p * M2_BYTES + k * MN_STEP), on(cols, k * MN_STEP), idAB, !(p == 1 && k == 0));
                }
                mma_commit(&lb->second);
            }
            __syncwarp();
        }
        ok = local_wait(&lb->second, j & 1) && ok;
        tc_fence_after();
        if (c0 < DK) {
            float x[32];
            const float up = meta->up[tk], down = meta->down[tk], w = keys ? -up : a.scale * up;
            load_acc(D1 + lane_base + c0, x);
#pragma unroll
            for (int i = 0; i < 32; ++i) acc[i] = fmaf(w, x[i], acc[i]);
            load_acc(D4 + lane_base + c0, x);
#pragma unroll
            for (int i = 0; i < 32; ++i) acc[i] += x[i];
            if (keys) {
                load_acc(D2 + lane_base + c0, x);
#pragma unroll
                for (int i = 0; i < 32; ++i) acc[i] = fmaf(down, x[i], acc[i]);
                load_acc(D5 + lane_base + c0, x);
#pragma unroll
                for (int i = 0; i < 32; ++i) acc[i] += x[i];
            }
        }
        if (j + 1 < group && ok)   // the second images' zero rows were [W; N]'s place only where DV is 64
            if (DV == 64)
                for (int i = tid; i < C * (DV / 8); i += LT) {
                    const int r = C + i / (DV / 8), d = i % (DV / 8) * 8;
                    *reinterpret_cast<uint4 *>(smem + L::a + L::A_IMG + r * 128 + (((d / 8) ^ (r & 7)) << 4)) = none;
                }
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
    }
    if (c0 < DK && tk < nt) {
        __nv_bfloat16 *p = keys ? static_cast<__nv_bfloat16 *>(a.dk) + (row0 + tk) * a.lddk + hk * DK + c0
                                : static_cast<__nv_bfloat16 *>(a.dq) + (row0 + tk) * a.lddq + hk * DK + c0;
        store_bf16_32(p, acc);
    }
    if (warp == 0) tmem_dealloc(tmem, 512);
}

// Rows [B][L][H][D] of bf16 as boxes of 64 tokens x 64 values of one head;
// tokens past L read as zeros.
cudaError_t encode_rows(CUtensorMap *m, const void *p, long long ld, int B, int Ltok, int H, int D) {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    if (!fn) {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            return cudaErrorNotSupported;
        fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
    }
    const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)H, (cuuint64_t)Ltok, (cuuint64_t)B};
    const cuuint64_t strides[3] = {(cuuint64_t)D * 2, (cuuint64_t)ld * 2, (cuuint64_t)ld * 2 * Ltok};
    const cuuint32_t box[4] = {64, 1, 64, 1}, es[4] = {1, 1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(p), dims, strides, box, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? cudaSuccess
               : cudaErrorInvalidValue;
}

template <typename K> cudaError_t big_smem(K *kernel, size_t bytes) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

template <int DK, bool TRANS> cudaError_t launch_prep(const Args &a, cudaStream_t st) {
    const cudaError_t e = big_smem(delta_prep_kernel<DK, TRANS>, PrepSmem<DK>::total);
    if (e != cudaSuccess) return e;
    delta_prep_kernel<DK, TRANS><<<dim3(chunks(a.L), a.Hk, a.B), PT, PrepSmem<DK>::total, st>>>(a);
    return cudaGetLastError();
}

template <int DK> cudaError_t forward(const Args &a, cudaStream_t st) {
    CUtensorMap mk, mq;
    cudaError_t e = encode_rows(&mk, a.k, a.ldk, a.B, a.L, a.Hk, DK);
    if (e == cudaSuccess) e = encode_rows(&mq, a.q, a.ldq, a.B, a.L, a.Hk, DK);
    if (e == cudaSuccess) e = launch_prep<DK, false>(a, st);
    if (e == cudaSuccess) e = big_smem(delta_scan_kernel<DK>, ScanSmem<DK>::total);
    if (e != cudaSuccess) return e;
    delta_scan_kernel<DK><<<dim3(a.Dv / NV, a.Hv, a.B), SCAN_THREADS, ScanSmem<DK>::total, st>>>(mk, mq, a);
    return cudaGetLastError();
}

template <int DK, int DV> cudaError_t launch_local(const Args &a, cudaStream_t st) {
    const cudaError_t e = big_smem(delta_local_kernel<DK, DV>, LocalSmem<DK, DV>::total);
    if (e != cudaSuccess) return e;
    delta_local_kernel<DK, DV><<<dim3(chunks(a.L), a.Hk, a.B), LT, LocalSmem<DK, DV>::total, st>>>(a);
    return cudaGetLastError();
}

template <int DK> cudaError_t backward(const Args &a, cudaStream_t st) {
    CUtensorMap mk, mq;
    cudaError_t e = encode_rows(&mk, a.k, a.ldk, a.B, a.L, a.Hk, DK);
    if (e == cudaSuccess) e = encode_rows(&mq, a.q, a.ldq, a.B, a.L, a.Hk, DK);
    if (e == cudaSuccess) e = launch_prep<DK, true>(a, st);
    if (e == cudaSuccess) e = big_smem(delta_adjoint_kernel<DK>, AdjSmem<DK>::total);
    if (e != cudaSuccess) return e;
    delta_adjoint_kernel<DK><<<dim3(a.Dv / NV, a.Hv, a.B), SCAN_THREADS, AdjSmem<DK>::total, st>>>(mk, mq, a);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return a.Dv == 128 ? launch_local<DK, 128>(a, st) : launch_local<DK, 64>(a, st);
}

}  // namespace

// bf16 with heads of 64 or 128; pitches that the copies can address (multiples
// of 16 bytes).  From how many tokens on, both sides measured: see tc_forward.
bool tc_supported(const Args &a, s5_dtype dtype, bool backward) {
    if (dtype != S5_BF16 || a.L < 1) return false;
    if ((a.Dk != 64 && a.Dk != 128) || (a.Dv != 64 && a.Dv != 128)) return false;
    if (a.ldq % 8 || a.ldk % 8 || a.ldv % 8) return false;
    return backward ? a.lddo % 8 == 0 && a.lddq % 8 == 0 && a.lddk % 8 == 0 && a.lddv % 8 == 0 : a.ldo % 8 == 0;
}

size_t tc_image_bytes(int B, int L, int Hv, int Dk, int Dv) {
    if ((Dk != 64 && Dk != 128) || (Dv != 64 && Dv != 128)) return 0;
    return (size_t)B * Hv * chunks(L) * IMG_BYTES;
}

cudaError_t tc_forward(const Args &a, cudaStream_t st) {
    return a.Dk == 128 ? forward<128>(a, st) : forward<64>(a, st);
}

cudaError_t tc_backward(const Args &a, cudaStream_t st) {
    return a.Dk == 128 ? backward<128>(a, st) : backward<64>(a, st);
}

int tc_inner_parts(int Dk, int Dv) { return Dv / NV * (Dk / 16); }

int fault_take() {
    int v = 0, zero = 0;
    if (cudaMemcpyFromSymbol(&v, g_delta_fault, sizeof(int)) != cudaSuccess) return -1;
    if (v && cudaMemcpyToSymbol(g_delta_fault, &zero, sizeof(int)) != cudaSuccess) return -1;
    return v;
}

}  // namespace delta
}  // namespace s5

extern "C" int s5_delta_fault(void) { return s5::delta::fault_take(); }
