// s5_delta_prep.cu -- what a chunk of the gated delta rule needs besides its
// state, for all chunks at once (s5_delta_scan.cu has the mathematics).
#include "s5_delta_mma.cuh"

namespace s5 {
namespace delta {
namespace {

// ---------------------------------------------------------------------------
// One CTA per chunk and key head; the products k.k and q.k are
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
// zero).  In the image 16 rows of E and 16 of P E take turns.  The whole image is built in shared memory in the layout that the
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
    // row r of the image's lower matrix: three parts of two neighbouring values
    auto put2 = [&](int r, int n, float x, float y) {
        uint32_t h, m, l;
        split3(x, y, h, m, l);
        unsigned char *to = img + (2 * r - (r & 15) + 16) * 128 + ((n ^ (r & 7)) << 4) + q2 * 2;
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
            unsigned char *to = img + (2 * r - (r & 15)) * 128 + ((ch ^ (r & 7)) << 4);
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
                const int r = 32 * rb + 16 + (lane & 15), m = 32 * kb + (lane & 15);
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

template <int DK, bool TRANS> cudaError_t launch(const Args &a, cudaStream_t st) {
    const cudaError_t e = big_smem(delta_prep_kernel<DK, TRANS>, PrepSmem<DK>::total);
    if (e != cudaSuccess) return e;
    delta_prep_kernel<DK, TRANS><<<dim3(chunks(a.L), a.Hk, a.B), PT, PrepSmem<DK>::total, st>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t tc_prepare(const Args &a, bool transposed, cudaStream_t st) {
    if (a.Dk == 128) return transposed ? launch<128, true>(a, st) : launch<128, false>(a, st);
    return transposed ? launch<64, true>(a, st) : launch<64, false>(a, st);
}

}  // namespace delta
}  // namespace s5
