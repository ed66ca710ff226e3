// s5_delta_prep.cu -- what a chunk of the gated delta rule needs besides its
// state, for all chunks at once (s5_delta_scan.cu has the mathematics): one
// CTA per chunk and key head, over the key head's value heads (or, where there
// are few, per value head).
//
// k_i.k_j and q_i.k_j are one tcgen05 product [K; Q] K^T, taken once and kept
// in registers.  Decay factors D_ij of two different blocks of 16 tokens are
// products e^{G_i - G_b} e^{G_b - G_j} at the end b of j's block (both at most
// 1 where g <= 0); inside a block each is an exponential of its own.
//
// The inverse goes by blocks, in place and in 32 bits on the CUDA cores (a
// split product would cost more in conversions): the four 16 x 16 blocks on
// the diagonal by substitution, one column per lane, then
//   [[A, 0], [B, D]]^-1 = [[A^-1, 0], [-D^-1 B A^-1, D^-1]]
// to 32 and to 64 rows.  P E is a tcgen05 product of the image's own parts:
// [E; P] E, of which the rows of P E are kept, in 24 bits: o is the same
// whether the call keeps anything for a backward pass or not.
// In the image 16 rows of E and 16 of P E take turns; it is built in shared
// memory in the layout that the recurrences' products read and leaves by one
// bulk copy.
//
// TRANS: T = (I + strict lower(beta_i D_ij k_i.k_j))^-1 and [T; P T] instead,
// which the backward pass uses.
//
// Bound: the latency of the block steps between barriers, which three CTAs an SM
// cover for one another (issue slots 43 % busy): 8 sequences of 1999 tokens, 32
// heads of 128 on 16 key heads, 181 us, 8192 images of 50 KB at 2.3 TB/s.
#include "s5_delta_mma.cuh"

namespace s5 {
namespace delta {
namespace {

constexpr int PT = 256;   // threads
constexpr int LD = 68;    // pitch of the fp32 tile: 16-byte rows, conflict-free on 8 rows of 4 values
constexpr int TD = 20;    // pitch of a transposed diagonal block

struct PrepMaps {
    CUtensorMap k16, q16, k64;   // boxes of 16 and of 64 tokens
};

template <int DK> struct PrepSmem {
    static constexpr uint32_t KQ = KQ_BOX * (DK / 64), K = 64 * 128 * (DK / 64);
    // the image, and before it the tiles: [K; Q] in turns, then K
    static constexpr uint32_t a = MAT_BYTES;                 // [64][LD]: the system, its inverse in its place
    static constexpr uint32_t td = a + C * LD * 4;           // diagonal blocks, transposed
    static constexpr uint32_t meta = td + 4 * 16 * TD * 4;   // this head's and the next one's factors
    static constexpr uint32_t near = meta + 2 * META_BYTES;  // e^{G_b - G_j}, twice
    static constexpr uint32_t bars = near + 2 * C * 4;
    static constexpr uint32_t total = bars + 64 + 1024;
    static_assert(KQ + K <= MAT_BYTES, "the tiles lie in the image's place");
};

struct PrepBars {
    uint64_t tiles, done;
    uint32_t tmem;
    int abort;
};

// One warp: the factors of a chunk and value head.
__device__ __forceinline__ void chunk_factors(const Args &a, long long row0, int nt, int h, Meta *meta, float *near, int lane) {
    const int t = 2 * lane;
    const float b0 = t < nt ? a.beta[(row0 + t) * a.Hv + h] : 0.0f;
    const float b1 = t + 1 < nt ? a.beta[(row0 + t + 1) * a.Hv + h] : 0.0f;
    float G[2], g[2];
    decay_sums(a, row0, nt, h, lane, G, g);
    const float th = __shfl_sync(0xffffffffu, G[1], 31), tl = __shfl_sync(0xffffffffu, g[1], 31);
    const float eh = __shfl_sync(0xffffffffu, G[1], lane | 7), el = __shfl_sync(0xffffffffu, g[1], lane | 7);
    const float be[2] = {b0, b1};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        meta->hi[t + i] = G[i];
        meta->lo[t + i] = g[i];
        meta->beta[t + i] = be[i];
        meta->up[t + i] = expf(G[i]);
        meta->down[t + i] = expf((th - G[i]) + (tl - g[i]));
        near[t + i] = expf((eh - G[i]) + (el - g[i]));
    }
    if (lane == 0) meta->last = expf(th);
}

template <int DK, bool TRANS>
__global__ void __launch_bounds__(PT, 3) delta_prep_kernel(const __grid_constant__ PrepMaps maps, const Args a) {
    using L = PrepSmem<DK>;
    extern __shared__ __align__(1024) unsigned char raw[];
    unsigned char *smem = raw + ((1024u - (smem_addr(raw) & 1023u)) & 1023u);
    float(*A)[LD] = reinterpret_cast<float(*)[LD]>(smem + L::a);
    float(*T)[16][TD] = reinterpret_cast<float(*)[16][TD]>(smem + L::td);
    PrepBars *pb = reinterpret_cast<PrepBars *>(smem + L::bars);
    const uint32_t img = smem_addr(smem);
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    // this block's value heads: `per` of them from h0 on, all of one key head
    const int per = a.Hv / gridDim.y, h0 = blockIdx.y * per, hk = h0 / (a.Hv / a.Hk);
    const int c = a.from + blockIdx.x, b = blockIdx.z;
    const int t0 = c * C, nt = min(C, a.L - t0), N = chunks(a.L);
    const long long row0 = (long long)b * a.L + t0;
    const int q = warp & 3, c0 = warp / 4 * 32;   // the warp's fragment: tokens 16 q on, columns c0 on
    auto meta_of = [&](int j) { return reinterpret_cast<Meta *>(smem + L::meta + (j & 1) * META_BYTES); };
    auto near_of = [&](int j) { return reinterpret_cast<float *>(smem + L::near) + (j & 1) * C; };
    auto wait = [&](uint64_t *bar, int parity) { return bounded_wait(bar, (uint32_t)parity, &pb->abort); };
    if (!a.beside) griddep_wait();
    if (tid == 0) {
        mbar_init(&pb->tiles, 1);
        mbar_init(&pb->done, 1);
        pb->abort = 0;
        fence_mbar_init();
        mbar_arrive_tx(&pb->tiles, L::KQ + L::K);
#pragma unroll 1
        for (int x = 0; x < DK / 64; ++x) {
#pragma unroll 1
            for (int i = 0; i < C / 16; ++i) {
                tma_load_4d(smem + x * KQ_BOX + 2 * i * KQ_GROUP, &maps.k16, 64 * x, hk, t0 + 16 * i, b, &pb->tiles);
                tma_load_4d(smem + x * KQ_BOX + (2 * i + 1) * KQ_GROUP, &maps.q16, 64 * x, hk, t0 + 16 * i, b, &pb->tiles);
            }
            tma_load_4d(smem + L::KQ + x * 8192, &maps.k64, 64 * x, hk, t0, b, &pb->tiles);
        }
    }
    if (warp == 0) {
        __syncwarp();
        tmem_alloc(&pb->tmem, 128);
        tmem_relinquish();
    }
    if (warp == 7) chunk_factors(a, row0, nt, h0, meta_of(0), near_of(0), lane);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = pb->tmem, frag = tmem + ((uint32_t)(32 * q) << 16) + c0;
    const uint64_t rows = desc_k(img), cols = desc_mn(img, M2_BYTES);
    const uint32_t n1 = idesc_bf16_f32(128, 64), n2 = idesc_bf16_f32(128, 128);
    bool ok = true;
    if (tid == 0) {
        if (wait(&pb->tiles, 0)) {
            const uint64_t K = desc_k(img + L::KQ);
#pragma unroll
            for (int k = 0; k < DK / 16; ++k)
                mma_bf16(tmem, on(rows, k / 4 * KQ_BOX + k % 4 * K_STEP), on(K, k / 4 * 8192 + k % 4 * K_STEP), n1, k > 0);
        }
        mma_commit(&pb->done);
    }
    __syncwarp();
    ok = wait(&pb->done, 0) && ok;
    tc_fence_after();
    float kk[16], qk[16];
    frag_load<1>(frag, kk);
    frag_load<1>(frag + QUERY_LANES, qk);
    frag_scale(qk, a.scale, a.scale);
    for (int j = 0; j < per; ++j) {
        const int h = h0 + j;
        Meta *meta = meta_of(j);
        const float *near = near_of(j);
        unsigned char *out = static_cast<unsigned char *>(a.images) + (((long long)b * a.Hv + h) * N + c) * IMG_BYTES;
        if (j > 0 && tid == 0) bulk_wait_read_all();   // the last image has left
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
        {
            float p[16];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = 16 * q + lane / 4 + 8 * i;
                const float gh = meta->hi[r], gl = meta->lo[r], br = meta->beta[r];
#pragma unroll
                for (int jb = 0; jb < 2; ++jb) {
                    const int nb = c0 / 16 + jb;
                    if (nb > q) {   // above the diagonal
#pragma unroll
                        for (int jj = 2 * jb; jj < 2 * jb + 2; ++jj) {
                            p[4 * jj + 2 * i] = p[4 * jj + 2 * i + 1] = 0.0f;
                            *reinterpret_cast<float2 *>(&A[r][c0 + 8 * jj + 2 * (lane & 3)]) = make_float2(0.0f, 0.0f);
                        }
                        continue;
                    }
                    float far = 1.0f;
                    if (nb < q) far = expf((gh - meta->hi[16 * nb + 15]) + (gl - meta->lo[16 * nb + 15]));
#pragma unroll
                    for (int jj = 2 * jb; jj < 2 * jb + 2; ++jj) {
                        float s[2];
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const int col = c0 + 8 * jj + 2 * (lane & 3) + k, at = 4 * jj + 2 * i + k;
                            const float d = nb < q ? far * near[col] : expf((gh - meta->hi[col]) + (gl - meta->lo[col]));
                            const float bc = meta->beta[col];
                            s[k] = col < r ? kk[at] * (d * (TRANS ? br : bc)) : 0.0f;
                            p[at] = col <= r ? qk[at] * (TRANS ? d : d * bc) : 0.0f;
                            if (nb == q) T[nb][col & 15][r & 15] = s[k];
                        }
                        *reinterpret_cast<float2 *>(&A[r][c0 + 8 * jj + 2 * (lane & 3)]) = make_float2(s[0], s[1]);
                    }
                }
            }
            frag_put3(img, M2_BYTES, 32 * q + 16, c0, lane, p, q);
        }
        __syncthreads();
        if (warp < 2) {   // two blocks of the diagonal per warp; lane: a column of the inverse
            const int blk = 2 * warp + (lane >> 4), o = 16 * blk, col = lane & 15;
            float x[16];
#pragma unroll
            for (int r = 0; r < 16; ++r) x[r] = r == col ? 1.0f : 0.0f;
#pragma unroll
            for (int m = 0; m < 15; ++m)
#pragma unroll
                for (int r4 = (m + 1) / 4 * 4; r4 < 16; r4 += 4) {
                    const float4 f = *reinterpret_cast<const float4 *>(&T[blk][m][r4]);
                    if (r4 > m) x[r4] = fmaf(-f.x, x[m], x[r4]);
                    if (r4 + 1 > m) x[r4 + 1] = fmaf(-f.y, x[m], x[r4 + 1]);
                    if (r4 + 2 > m) x[r4 + 2] = fmaf(-f.z, x[m], x[r4 + 2]);
                    if (r4 + 3 > m) x[r4 + 3] = fmaf(-f.w, x[m], x[r4 + 3]);
                }
#pragma unroll
            for (int r = 0; r < 16; ++r) A[o + r][o + col] = x[r];
        } else if (warp == 7 && j + 1 < per) {
            chunk_factors(a, row0, nt, h + 1, meta_of(j + 1), near_of(j + 1), lane);
        }
        __syncthreads();
        {   // 32-row blocks, both pairs at once: B A^-1 into the unused upper part, then -D^-1 of it
            const int o = 32 * (tid / 128), r = tid % 128 / 8, c2 = tid % 8 * 2;
            float v0 = 0.0f, v1 = 0.0f;
#pragma unroll
            for (int m = 0; m < 16; m += 4) {
                const float4 x = *reinterpret_cast<const float4 *>(&A[o + 16 + r][o + m]);
                const float xs[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float2 y = *reinterpret_cast<const float2 *>(&A[o + m + k][o + c2]);
                    v0 = fmaf(xs[k], y.x, v0), v1 = fmaf(xs[k], y.y, v1);
                }
            }
            *reinterpret_cast<float2 *>(&A[o + r][o + 16 + c2]) = make_float2(v0, v1);
            __syncthreads();
            v0 = v1 = 0.0f;
#pragma unroll
            for (int m = 0; m < 16; m += 4) {
                const float4 x = *reinterpret_cast<const float4 *>(&A[o + 16 + r][o + 16 + m]);
                const float xs[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float2 y = *reinterpret_cast<const float2 *>(&A[o + m + k][o + 16 + c2]);
                    v0 = fmaf(-xs[k], y.x, v0), v1 = fmaf(-xs[k], y.y, v1);
                }
            }
            *reinterpret_cast<float2 *>(&A[o + 16 + r][o + c2]) = make_float2(v0, v1);
            // the products below read the upper part as zeros
            __syncthreads();
            *reinterpret_cast<float2 *>(&A[o + r][o + 16 + c2]) = make_float2(0.0f, 0.0f);
        }
        __syncthreads();
        // 64 rows: two rows x four columns a thread, so that eight products
        // share six reads of 16 bytes over four steps
        auto block64 = [&](int xr, int xc, int yr, int yc, int zr, int zc, float sign) {
            const int r = tid / 8 * 2, c4 = tid % 8 * 4;
            float v[2][4] = {};
#pragma unroll
            for (int m = 0; m < 32; m += 4) {
                const float4 x0 = *reinterpret_cast<const float4 *>(&A[xr + r][xc + m]);
                const float4 x1 = *reinterpret_cast<const float4 *>(&A[xr + r + 1][xc + m]);
                const float xs[2][4] = {{x0.x, x0.y, x0.z, x0.w}, {x1.x, x1.y, x1.z, x1.w}};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float4 y = *reinterpret_cast<const float4 *>(&A[yr + m + k][yc + c4]);
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        v[i][0] = fmaf(xs[i][k], y.x, v[i][0]), v[i][1] = fmaf(xs[i][k], y.y, v[i][1]);
                        v[i][2] = fmaf(xs[i][k], y.z, v[i][2]), v[i][3] = fmaf(xs[i][k], y.w, v[i][3]);
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < 2; ++i)
                *reinterpret_cast<float4 *>(&A[zr + r + i][zc + c4]) =
                    make_float4(sign * v[i][0], sign * v[i][1], sign * v[i][2], sign * v[i][3]);
        };
        if (tid < 128) block64(32, 0, 0, 0, 0, 32, 1.0f);
        __syncthreads();
        if (tid < 128) block64(32, 32, 0, 32, 32, 0, -1.0f);
        __syncthreads();
#pragma unroll
        for (int k = 0; k < C * 8 / PT; ++k) {   // E's three parts
            // a warp's 32 pieces are one 8-wide column of 32 rows: whole blocks of
            // zeros above the diagonal are not split
            const int r = lane + 32 * (warp & 1), ch = warp / 2 + 4 * k;
            uint32_t hh[4] = {}, mm[4] = {}, ll[4] = {};
            if (ch / 2 <= 2 * (warp & 1) + 1) {
                float4 x = make_float4(0, 0, 0, 0), y = x;
                if (ch / 2 <= r / 16) {
                    x = *reinterpret_cast<const float4 *>(&A[r][8 * ch]);
                    y = *reinterpret_cast<const float4 *>(&A[r][8 * ch + 4]);
                }
                split3(x.x, x.y, hh[0], mm[0], ll[0]);
                split3(x.z, x.w, hh[1], mm[1], ll[1]);
                split3(y.x, y.y, hh[2], mm[2], ll[2]);
                split3(y.z, y.w, hh[3], mm[3], ll[3]);
            }
            const uint32_t to = piece(img, 2 * r - (r & 15), ch);
            sts128(to, hh[0], hh[1], hh[2], hh[3]);
            sts128(to + M2_BYTES, mm[0], mm[1], mm[2], mm[3]);
            sts128(to + 2 * M2_BYTES, ll[0], ll[1], ll[2], ll[3]);
        }
        fence_proxy_async_smem();
        __syncthreads();
        if (tid == 0) {   // [E; P] E: the second operand's rows are every second 16
#pragma unroll
            for (int k = 0; k < C / 16; ++k) {
                const uint64_t P = on(rows, k * K_STEP), E = on(cols, 2 * k * KQ_GROUP);
                mma_bf16(tmem, on(P, M2_BYTES), E, n2 | B_MN, k > 0);
                mma_bf16(tmem, P, E, n2 | B_MN, 1);
                mma_bf16(tmem, on(P, 2 * M2_BYTES), E, n1 | B_MN, 1);
                mma_bf16(tmem, P, on(E, 2 * M2_BYTES), n1 | B_MN, 1);
            }
            mma_commit(&pb->done);
        }
        __syncwarp();
        ok = wait(&pb->done, (j + 1) & 1) && ok;
        tc_fence_after();
        {
            float p[16];
            frag_load<2>(frag + QUERY_LANES, p);
            frag_put3(img, M2_BYTES, 32 * q + 16, c0, lane, p, q);
        }
        fence_proxy_async_smem();
        __syncthreads();
        if (tid == 0) {
            bulk_store(out, smem, MAT_BYTES);
            bulk_store(out + MAT_BYTES, meta, META_BYTES);
            bulk_commit();
        }
    }
    if (tid == 0) bulk_wait_all();
    if (!ok) settle_copies();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0) tmem_dealloc(tmem, 128);
    // beside the scan of earlier chunks: this grid ends after that one
    if (a.beside && blockIdx.x == gridDim.x - 1 && blockIdx.y == gridDim.y - 1 && blockIdx.z == gridDim.z - 1) griddep_wait();
}

// Blocks of a key head (chunk by chunk) up to which each is split into blocks of
// one value head, which take its products again but not one after the other.
// Heads of 128, a block a key head / a value head, us of the whole forward call: 16
// value heads on 8 key heads, 8 chunks (64 blocks) 32.8 / 28.0, 24 chunks 69.0 /
// 65.0, 32 chunks (256) 86.1 / 87.3; on 4 key heads, 32 chunks (128) 92.9 / 85.8.
constexpr int SPLIT_BLOCKS = 228;

template <int DK, bool TRANS> cudaError_t launch(const Args &a, cudaStream_t st) {
    PrepMaps m = {};
    cudaError_t e = encode_rows(&m.k16, false, a.k, a.ldk, a.B, a.L, a.Hk, DK, 16);
    if (e == cudaSuccess) e = encode_rows(&m.q16, false, a.q, a.ldq, a.B, a.L, a.Hk, DK, 16);
    if (e == cudaSuccess) e = encode_rows(&m.k64, false, a.k, a.ldk, a.B, a.L, a.Hk, DK);
    if (e == cudaSuccess) e = big_smem(delta_prep_kernel<DK, TRANS>, PrepSmem<DK>::total);
    if (e != cudaSuccess) return e;
    const bool single = (long long)a.count * a.Hk * a.B <= SPLIT_BLOCKS;
    return launch_after(delta_prep_kernel<DK, TRANS>, dim3(a.count, single ? a.Hv : a.Hk, a.B), PT, PrepSmem<DK>::total, st, m, a);
}

}  // namespace

cudaError_t tc_prepare(const Args &a, bool transposed, cudaStream_t st) {
    if (a.Dk == 128) return transposed ? launch<128, true>(a, st) : launch<128, false>(a, st);
    return transposed ? launch<64, true>(a, st) : launch<64, false>(a, st);
}

int prep_fault_take() { return fault_take(); }

}  // namespace delta
}  // namespace s5
