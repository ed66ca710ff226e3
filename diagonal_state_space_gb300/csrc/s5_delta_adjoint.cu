// s5_delta_adjoint.cu -- the gated delta rule's backward pass on the tensor
// cores; notation and precision as in s5_delta_scan.cu.
//
// The adjoint over chunks, last chunk first, with Z = dL/dS at the chunk's end
// and T = (I + strict lower(beta_i D_ij k_i.k_j))^-1:
//   X = T^T (e^{G_64 - G} K Z) + (P T)^T dO          X_t = dL/du_t
//   dv = beta X
//   Z_start = e^{G_64} Z + K^T (-e^G dv) + Q^T (scale e^G dO)
// the forward's three products transposed, on the same tiles: D1 = [K; Q] Z,
// D2 = [T; P T]^T [e^{..} K Z; dO] (depth 128), D3 = [K; Q]^T [..; ..] (depth
// 128).  Z leaves chunk by chunk as the two upper parts of its operand (rounded
// ones), in the layout that the local products below read.  Of the decays' gradients
// (formula in s5_delta.cu) <S, Z> and the b_j are taken in 32 bits on the way.
//
// Bound: as the forward scan, the chain product -> sums, splits -> product three
// times a chunk, 4.2 us with 64 columns a CTA and the tiles of X, Z and the state
// beside it: 4 sequences of 2048 tokens, 16 heads of 128, 134 us (131 without the
// b_j, which are added up while D3 runs).
//
// All else is local to a chunk (delta_local_kernel).
#include "s5_delta_mma.cuh"

namespace s5 {
namespace delta {
namespace {

struct AdjMaps {
    CUtensorMap k, q, g, x, s;   // keys, queries, dO, X, states
};

template <int DK> struct AdjSmem {
    static constexpr uint32_t KQ = KQ_BOX * (DK / 64);
    static constexpr uint32_t S_IMG = DK * 128;
    static constexpr uint32_t kq = 0;                      // two stages
    static constexpr uint32_t mat = kq + 2 * KQ;
    // Z's parts until D1 is done; then e^{..} K Z's, later -e^G dv's, and
    // behind them scale e^G dO's
    static constexpr uint32_t ops = mat + MAT_BYTES;
    static constexpr uint32_t go = ops + 6 * RU_IMG;       // dO
    static constexpr uint32_t xs = go + RU_IMG;            // X, to be stored
    static constexpr uint32_t sin = xs + 2 * RU_IMG;       // the state at the chunk's start
    static constexpr uint32_t meta = sin + DK * 256;
    static constexpr uint32_t bars = meta + META_BYTES;
    static constexpr uint32_t total = bars + 256 + 1024;
    static_assert(total <= 232448, "shared memory of a CTA");
    static_assert(3 * S_IMG <= 6 * RU_IMG, "Z fits");
};

struct AdjBars {
    uint64_t kq_full[2], kq_empty[2], img_full, img_empty, go_full, go_empty, sin_full, sin_empty;
    uint64_t d1, d2, d3, z_ready, r_ready, y_ready, z_left, x_ready, x_left, drain;
    uint32_t tmem;
    int abort;
};
static_assert(sizeof(AdjBars) <= 256, "barriers");

constexpr int ADJ_THREADS = 320;   // 8 compute warps, products, copies

template <int DK> __global__ void __launch_bounds__(ADJ_THREADS, 1) delta_adjoint_kernel(const __grid_constant__ AdjMaps maps, const Args a) {
    using L = AdjSmem<DK>;
    extern __shared__ __align__(1024) unsigned char raw[];
    unsigned char *smem = raw + ((1024u - (smem_addr(raw) & 1023u)) & 1023u);
    AdjBars *sb = reinterpret_cast<AdjBars *>(smem + L::bars);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int n0 = blockIdx.x * NV, h = blockIdx.y, b = blockIdx.z, hk = h / (a.Hv / a.Hk);
    const int N = chunks(a.L);
    const long long bh = (long long)b * a.Hv + h;
    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) mbar_init(&sb->kq_full[i], 1), mbar_init(&sb->kq_empty[i], 1);
        mbar_init(&sb->img_full, 1), mbar_init(&sb->img_empty, 8);
        mbar_init(&sb->go_full, 1), mbar_init(&sb->go_empty, 8);
        mbar_init(&sb->sin_full, 1), mbar_init(&sb->sin_empty, 8);
        mbar_init(&sb->d1, 1), mbar_init(&sb->d2, 1), mbar_init(&sb->d3, 1);
        mbar_init(&sb->z_ready, 8), mbar_init(&sb->r_ready, 8), mbar_init(&sb->y_ready, 8);
        mbar_init(&sb->z_left, 1), mbar_init(&sb->x_ready, 8), mbar_init(&sb->x_left, 1);
        mbar_init(&sb->drain, 1);
        sb->abort = 0;
        fence_mbar_init();
    }
    griddep_wait();
    if (warp == 8) {
        tmem_alloc(&sb->tmem, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // D3 takes D1's place: every warp that reads D1 has done so before it hands
    // the operands of D3 over
    const uint32_t tmem = sb->tmem, D1 = tmem, D2 = tmem + 3 * NV, D3 = tmem;
    auto wait = [&](uint64_t *bar, int parity) { return bounded_wait(bar, (uint32_t)parity, &sb->abort); };

    if (warp == 9) {
        if (lane == 0) {
            // ------------------------------------------------------ copies
            auto load_kq = [&](int it) {
                load_chunk_rows<DK>(smem + L::kq + (it & 1) * L::KQ, &maps.k, &maps.q, hk, (N - 1 - it) * C, b, &sb->kq_full[it & 1]);
            };
            auto load_img = [&](int it) {
                const unsigned char *from = static_cast<const unsigned char *>(a.images) + (bh * N + N - 1 - it) * IMG_BYTES;
                mbar_arrive_tx(&sb->img_full, IMG_BYTES);
                bulk_load(smem + L::mat, from, MAT_BYTES, &sb->img_full);
                bulk_load(smem + L::meta, from + MAT_BYTES, META_BYTES, &sb->img_full);
            };
            auto load_go = [&](int it) {
                mbar_arrive_tx(&sb->go_full, RU_IMG);
                tma_load_4d(smem + L::go, &maps.g, n0, h, (N - 1 - it) * C, b, &sb->go_full);
            };
            auto load_state = [&](int it) {
                mbar_arrive_tx(&sb->sin_full, DK * 256);
                for (int x = 0; x < 2; ++x)
                    tma_load_3d(smem + L::sin + x * DK * 128, &maps.s, n0 + 32 * x, 0, (int)(bh * (N + 1) + N - 1 - it), &sb->sin_full);
            };
            load_kq(0);
            load_state(0);
            load_img(0);
            load_go(0);
            if (N > 1) load_kq(1);
            bool ok = true;
            for (int it = 0; it < N; ++it) {
                const int c = N - 1 - it;
                if (!(ok = wait(&sb->z_ready, it & 1))) break;
                bulk_store(static_cast<unsigned char *>(a.z) + ((bh * N + c) * (a.Dv / NV) + blockIdx.x) * (2 * L::S_IMG),
                           smem + L::ops, 2 * L::S_IMG);
                bulk_commit();
                bulk_wait_read_all();
                mbar_arrive(&sb->z_left);
                if (it + 1 < N) {
                    if (!(ok = wait(&sb->sin_empty, it & 1))) break;
                    load_state(it + 1);
                    if (!(ok = wait(&sb->img_empty, it & 1) && wait(&sb->go_empty, it & 1))) break;
                    load_img(it + 1);
                    load_go(it + 1);
                }
                if (!(ok = wait(&sb->x_ready, it & 1))) break;
                for (int x = 0; x < 2; ++x) tma_store_4d(&maps.x, smem + L::xs + x * RU_IMG, n0 + 32 * x, h, c * C, b);
                bulk_commit();
                bulk_wait_read_all();
                mbar_arrive(&sb->x_left);
                if (it + 2 < N) {
                    if (!(ok = wait(&sb->kq_empty[it & 1], (it >> 1) & 1))) break;
                    load_kq(it + 2);
                }
            }
            bulk_wait_all();
            if (!ok) settle_copies();
        }
        __syncwarp();
    } else if (warp == 8) {
        if (lane == 0) {
            // ------------------------------------------------------ products
            // D2 has 64 rows (the matrix transposed): M = 64 spreads them over
            // 16 of each 32 lanes
            const uint32_t w1 = idesc_bf16_f32(64, NV) | A_MN | B_MN, w2 = idesc_bf16_f32(64, 2 * NV) | A_MN | B_MN,
                           w3 = idesc_bf16_f32(128, 3 * NV) | B_MN;
            const uint64_t mat = desc_mn(smem_addr(smem + L::mat), M2_BYTES), Z = desc_mn(smem_addr(smem + L::ops), L::S_IMG),
                           R = desc_mn(smem_addr(smem + L::ops), RU_IMG), Y = desc_mn(smem_addr(smem + L::ops + 3 * RU_IMG), RU_IMG),
                           G = desc_mn(smem_addr(smem + L::go), RU_IMG);
            bool ok = true;
            for (int it = 0; ok && it < N; ++it) {
                const uint32_t kq = smem_addr(smem + L::kq + (it & 1) * L::KQ);
                const uint64_t rows = desc_k(kq), cols = desc_mn(kq, KQ_BOX);
                if (!(ok = wait(&sb->kq_full[it & 1], (it >> 1) & 1) && wait(&sb->z_ready, it & 1))) break;
                tc_fence_after();
#pragma unroll
                for (int k = 0; k < DK / 16; ++k)
                    mma_bf16(D1, on(rows, k / 4 * KQ_BOX + k % 4 * K_STEP), on(Z, k * MN_STEP), w3, k > 0);
                mma_commit(&sb->d1);
                // (P T)^T dO waits for nothing else
                if (!(ok = wait(&sb->img_full, it & 1) && wait(&sb->go_full, it & 1))) break;
#pragma unroll
                for (int k = 0; k < C / 16; ++k)
#pragma unroll
                    for (int p = 2; p >= 0; --p)
                        mma_bf16(D2, on(mat, p * M2_BYTES + (2 * k + 1) * KQ_GROUP), on(G, k * MN_STEP), w1, k > 0 || p < 2);
                if (!(ok = wait(&sb->r_ready, it & 1))) break;
                tc_fence_after();
#pragma unroll
                for (int k = 0; k < C / 16; ++k) {
                    const uint64_t T = on(mat, 2 * k * KQ_GROUP);
                    mma_bf16(D2 + NV, on(T, M2_BYTES), on(R, k * MN_STEP), w2, k > 0);
                    mma_bf16(D2, on(T, 2 * M2_BYTES), on(R, k * MN_STEP), w1, 1);
                    mma_bf16(D2, T, on(R, 2 * RU_IMG + k * MN_STEP), w1, 1);
                    mma_bf16(D2 + NV, T, on(R, k * MN_STEP), w2, 1);
                }
                mma_commit(&sb->d2);
                if (!(ok = wait(&sb->y_ready, it & 1))) break;
                tc_fence_after();
#pragma unroll
                for (int k = 0; k < 2 * C / 16; ++k)   // keys and queries in turn
                    mma_bf16(D3, on(cols, k * KQ_GROUP), on(k % 2 ? Y : R, k / 2 * MN_STEP), w3 | A_MN, k > 0);
                mma_commit(&sb->d3);
                mma_commit(&sb->kq_empty[it & 1]);
            }
            drain_products(&sb->drain);
        }
        __syncwarp();
    } else {
        // ---------------------------------------------------------- compute
        const int q = warp & 3, c0 = warp / 4 * 32, row = 32 * q + lane;
        const int t16 = 16 * q, ta = t16 + lane / 4, tb = ta + 8;   // tokens of a fragment's rows
        const uint32_t lanes = ((uint32_t)(32 * q) << 16) + c0;
        const uint32_t ops = smem_addr(smem + L::ops), go = smem_addr(smem + L::go), xs = smem_addr(smem + L::xs),
                       sin = smem_addr(smem + L::sin);
        const Meta *meta = reinterpret_cast<const Meta *>(smem + L::meta);
        const bool state = row < DK;
        const long long place = bh * DK * a.Dv + (long long)row * a.Dv + n0 + c0;   // this row in ds_last, ds0
        float Z[32];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float4 t = (a.ds_last && state) ? *reinterpret_cast<const float4 *>(a.ds_last + place + 4 * j) : make_float4(0, 0, 0, 0);
            Z[4 * j] = t.x, Z[4 * j + 1] = t.y, Z[4 * j + 2] = t.z, Z[4 * j + 3] = t.w;
        }
        if (state) put3<32, false, true>(ops, L::S_IMG, row, c0, Z);
        hand_over(&sb->z_ready, lane);
        for (int it = 0; it < N; ++it) {
            const int c = N - 1 - it;
            // <S, Z> of the chunk's start and end
            bool ok = wait(&sb->sin_full, it & 1);
            if (!__all_sync(0xffffffffu, ok)) break;
            if (state) {
                float w = 0.0f, v = 0.0f;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const uint4 t = lds128(piece(sin + c0 / 32 * (DK * 128), row, j));
                    w = fmaf(__uint_as_float(t.x), Z[4 * j], w), v = fmaf(__uint_as_float(t.y), Z[4 * j + 1], v);
                    w = fmaf(__uint_as_float(t.z), Z[4 * j + 2], w), v = fmaf(__uint_as_float(t.w), Z[4 * j + 3], v);
                }
                w += v;
                for (int m = 16; m > 0; m >>= 1) w += __shfl_xor_sync(0xffffffffu, w, m);
                if (lane == 0) a.inner[(bh * N + c) * inner_parts(DK, a.Dv) + blockIdx.x * (DK / 16) + q * 2 + warp / 4] = w;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&sb->sin_empty);
            // e of this warp's fragment is on its way during D1
            float2 e[8];
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int t = c * C + ta + 8 * i;
                    e[4 * i + j] = t < a.L ? *reinterpret_cast<const float2 *>(a.e + (((long long)b * a.L + t) * a.Hv + h) * a.Dv + n0 + c0 +
                                                                               8 * j + 2 * (lane & 3))
                                           : make_float2(0.0f, 0.0f);
                }
            ok = wait(&sb->img_full, it & 1) && wait(&sb->go_full, it & 1) && wait(&sb->z_left, it & 1) && wait(&sb->d1, it & 1);
            if (!__all_sync(0xffffffffu, ok)) break;
            tc_fence_after();
            float f[16];
            frag_load<3>(D1 + lanes, f);
            frag_scale(f, meta->down[ta], meta->down[tb]);
            frag_put3(ops, RU_IMG, t16, c0, lane, f);
            hand_over(&sb->r_ready, lane);
            const float last = meta->last, ua = meta->up[ta], ub = meta->up[tb];
            const float ba = meta->beta[ta], bb = meta->beta[tb], ya = -ua * ba, yb = -ub * bb;
            float kz[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) kz[i] = f[i];
            frag_get(go, t16, c0, lane, f);
            frag_scale(f, a.scale * ua, a.scale * ub);
            frag_put3(ops + 3 * RU_IMG, RU_IMG, t16, c0, lane, f);
            ok = wait(&sb->d2, it & 1);
            if (!__all_sync(0xffffffffu, ok)) break;
            tc_fence_after();
            if (lane == 0) mbar_arrive(&sb->img_empty), mbar_arrive(&sb->go_empty);
            frag_load<3>(D2 + lanes, f);
            float y[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) y[i] = f[i] * ((i & 2) ? yb : ya);
            frag_put3(ops, RU_IMG, t16, c0, lane, y);
            hand_over(&sb->y_ready, lane);
            ok = it == 0 || wait(&sb->x_left, (it - 1) & 1);
            if (!__all_sync(0xffffffffu, ok)) break;
            frag_put_rows(xs + c0 / 32 * RU_IMG, t16, lane, f);
            hand_over(&sb->x_ready, lane);
            {   // this slice's share of b_j = e^{G_64 - G_j} (Z^T k_j).u_j, for the decays,
                // while D3 runs
                float w[2] = {0.0f, 0.0f};
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        w[i] = fmaf(kz[4 * j + 2 * i], e[4 * i + j].x, fmaf(kz[4 * j + 2 * i + 1], e[4 * i + j].y, w[i]));
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    w[i] += __shfl_xor_sync(0xffffffffu, w[i], 1);
                    w[i] += __shfl_xor_sync(0xffffffffu, w[i], 2);
                    if ((lane & 3) == 0)
                        a.writes[((bh * N + c) * C + ta + 8 * i) * write_parts(a.Dv) + blockIdx.x * 2 + warp / 4] = (i ? bb : ba) * w[i];
                }
            }
            ok = wait(&sb->d3, it & 1);
            if (!__all_sync(0xffffffffu, ok)) break;
            tc_fence_after();
            if (state) {
                float x[32];
                load_parts<3, 32>(D3 + lanes, x);
#pragma unroll
                for (int i = 0; i < 32; ++i) Z[i] = fmaf(last, Z[i], x[i]);
                if (c > 0) put3<32, false, true>(ops, L::S_IMG, row, c0, Z);
            }
            if (c > 0) hand_over(&sb->z_ready, lane);
        }
        if (state && a.ds0)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                *reinterpret_cast<float4 *>(a.ds0 + place + 4 * j) = make_float4(Z[4 * j], Z[4 * j + 1], Z[4 * j + 2], Z[4 * j + 3]);
        tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
    if (warp == 8) tmem_dealloc(tmem, 512);
}

// ---------------------------------------------------------------------------
// What is local to a chunk: persistent CTAs over chunks and key heads, each
// over its value heads, the next head's tiles on their way to L2.  Per token
// dv = beta X, dbeta = X . e.  With S0 and Z the state at the chunk's start and the
// adjoint at its end, U = beta e, and
// N_ij = scale D_ij dO_i.U_j (j <= i), W_ij = -D_ij dv_i.U_j (j < i):
//   dq = scale e^G dO S0^T + N K
//   dk = e^{G_64 - G} U Z^T - e^G dv S0^T + W K + W^T K + N^T Q
// as products of M = 128 with the rows of [dv; dO] stacked, so that dk lies in
// TMEM lanes 0..63 and dq in 64..127:
//   D2 = [U; -] Z^T,  D3 = [dv; dO] U^T,
//   D1 = [dv; dO] S0^T,  D4 = [W; N] K,  D5 = [W; N]^T [K; Q].
// dq and dk are rounded to bf16, off by up to 2^-9: 32-bit operands are carried as
// two bf16 values there, off by up to 2^-17, three products against another pair, two
// against a bf16 operand.
//
// The decays' gradients (formula in s5_delta.cu) keep 32 bits.  With KK = [K; Q] K^T
// and E1 = [K; Q] S0,
//   M = W o KK above + N o KK below (row i of either half),
//   a_i = scale e^{G_i} E1_{64+i}.dO_i - e^{G_i} E1_i.dv_i,
// and D3 and E1 take third parts of dv, U and S0 besides.  A thread has a row's 16
// columns of M: their running sums go to the tokens of its own columns' block, their
// total to those of the later blocks.  The sums over rows are butterflies and scans
// over lanes, while D1, D4, D5 and E1 run.
// Bound: what it reads (the state, the adjoint and 64 tokens' X, e, dO: 208 KB per
// chunk and head of 128 x 128), and the phases between its products in a CTA alone on
// its SM: 2048 chunks and heads in 197 us, 2.2 TB/s (161 us without the decays' sums;
// 265 with D3 in products of 64 columns, the sums' registers spilled, and the same
// warp issuing the products, finishing the decays and copying the adjoint).
// ---------------------------------------------------------------------------
constexpr int LT = 512;
// Warps with an errand besides: one issues the products, one adds up the decays'
// gradients and then copies the next adjoint over the sums it read.  Both have
// query rows and a block of [W; N] off the diagonal, the least work otherwise.
constexpr int ISSUE = 3, TAIL = 14;

template <int DK, int DV> struct LocalSmem {
    static constexpr uint32_t KQ = KQ_BOX * (DK / 64);
    static constexpr uint32_t A_IMG = 128 * 128 * (DV / 64);   // [dv; dO]
    static constexpr uint32_t U_IMG = 64 * 128 * (DV / 64);
    static constexpr uint32_t S_IMG = DK * 128 * (DV / 64);
    static constexpr uint32_t kq = 0;                          // 64 keys, then 64 queries
    static constexpr uint32_t a = kq + KQ;                     // two parts
    static constexpr uint32_t u = a + 2 * A_IMG;               // a box's three parts side by side
    static constexpr uint32_t dv3 = u + 3 * U_IMG;             // dv's third part
    // later: the two parts of [W; N] in the place of U, where they fit, and S0's third part behind them
    static constexpr bool APART = U_IMG < M2_BYTES;
    static constexpr uint32_t wn = APART ? dv3 + U_IMG : u;
    static constexpr uint32_t s3 = u + 2 * U_IMG;
    static constexpr uint32_t s = APART ? wn + 2 * M2_BYTES : dv3 + U_IMG;   // Z, then S0: a box's two parts side by side
    static constexpr uint32_t meta = s + 2 * S_IMG;
    static constexpr uint32_t bars = meta + META_BYTES;
    static constexpr uint32_t total = bars + 64 + 1024;
    static_assert(total <= 232448, "shared memory of a CTA");
    static_assert(S_IMG <= 2 * U_IMG, "S0's third part fits");
    // products of M = 128 over 64 rows or columns read on into what follows:
    // 8 KB past U and dv's third part, 16 KB past [W; N]
    static_assert(2 * S_IMG >= M2_BYTES, "what the products read on is the CTA's own memory");
    // sums on their way to the decays' gradients, in the state's place after its products
    static constexpr uint32_t part = s, suffix = part + 16 * 16 * 4, rows = suffix + 16 * 32 * 4;
    static_assert(rows + 128 * 4 * 4 <= s + 2 * S_IMG, "they fit");
};

struct LocalBars {
    uint64_t z_full, first, second, third, fourth;
    uint32_t tmem;
    int abort;
};

__device__ __forceinline__ void prefetch_line(const void *p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// The tiles of a chunk and value head, line by line over the block's threads
// (a bulk prefetch for each row costs the SM 25 cycles a row).
template <int DK, int DV>
__device__ __forceinline__ void prefetch_head(const Args &a, int c, int b, int h, bool rows_too, int N, int tid) {
    const int nt = min(C, a.L - c * C), hk = h / (a.Hv / a.Hk);
    const long long row0 = (long long)b * a.L + c * C, bh = (long long)b * a.Hv + h;
    constexpr int RL = DV / 32, HL = DV / 64, KL = DK / 64;   // lines of a row of floats, of bf16
    for (int i = tid; i < C * 8; i += LT) {      // eight threads a token
        const int t = i / 8, k = i % 8;
        if (t >= nt) continue;
        const long long at = ((row0 + t) * a.Hv + h) * DV;
        if (k < RL) prefetch_line(a.x + at + k * 32), prefetch_line(a.e + at + k * 32);
        if (k < HL) prefetch_line(static_cast<const __nv_bfloat16 *>(a.dout) + (row0 + t) * a.lddo + (long long)h * DV + k * 64);
        if (rows_too && k >= 4 && k < 4 + KL) {
            prefetch_line(static_cast<const __nv_bfloat16 *>(a.k) + (row0 + t) * a.ldk + hk * DK + (k - 4) * 64);
            prefetch_line(static_cast<const __nv_bfloat16 *>(a.q) + (row0 + t) * a.ldq + hk * DK + (k - 4) * 64);
        }
    }
    const char *s = reinterpret_cast<const char *>(a.states + (bh * (N + 1) + c) * DK * DV);
    const char *z = static_cast<const char *>(a.z) + (bh * N + c) * DK * DV * 4;
#pragma unroll
    for (int i = 0; i < DK * DV / 32 / LT + (DK * DV / 32 % LT != 0); ++i)
        if (tid + i * LT < DK * DV / 32) prefetch_line(s + (tid + i * LT) * 128), prefetch_line(z + (tid + i * LT) * 128);
}

// Eight values as a 16-byte piece of two images.
__device__ __forceinline__ void put2(uint32_t img, uint32_t stride, int row, int j, const float (&v)[8]) {
    uint32_t h[4], m[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) split2(v[2 * i], v[2 * i + 1], h[i], m[i]);
    const uint32_t to = piece(img, row, j);
    sts128(to, h[0], h[1], h[2], h[3]);
    sts128(to + stride, m[0], m[1], m[2], m[3]);
}
// As a piece of three images, the third at `low`.
__device__ __forceinline__ void put3(uint32_t img, uint32_t stride, uint32_t low, int row, int j, const float (&v)[8]) {
    uint32_t h[4], m[4], l[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) split3_rounded(v[2 * i], v[2 * i + 1], h[i], m[i], l[i]);
    const uint32_t to = piece(img, row, j);
    sts128(to, h[0], h[1], h[2], h[3]);
    sts128(to + stride, m[0], m[1], m[2], m[3]);
    sts128(piece(low, row, j), l[0], l[1], l[2], l[3]);
}
// Sums over the warp of 16 values a lane; lane l gets that of value l / 2.
__device__ __forceinline__ float sum16(const float (&v)[16], int lane) {
    float a[8], b[4], c[2], d;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const bool up = lane & 16;
        a[i] = (up ? v[i + 8] : v[i]) + __shfl_xor_sync(0xffffffffu, up ? v[i] : v[i + 8], 16);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const bool up = lane & 8;
        b[i] = (up ? a[i + 4] : a[i]) + __shfl_xor_sync(0xffffffffu, up ? a[i] : a[i + 4], 8);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const bool up = lane & 4;
        c[i] = (up ? b[i + 2] : b[i]) + __shfl_xor_sync(0xffffffffu, up ? b[i] : b[i + 2], 4);
    }
    const bool up = lane & 2;
    d = (up ? c[1] : c[0]) + __shfl_xor_sync(0xffffffffu, up ? c[0] : c[1], 2);
    return d + __shfl_xor_sync(0xffffffffu, d, 1);
}
// The sum of this lane's and all later lanes' values.
__device__ __forceinline__ float later_lanes(float v, int lane) {
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const float x = __shfl_down_sync(0xffffffffu, v, m);
        if (lane + m < 32) v += x;
    }
    return v;
}
// The sum of all earlier lanes' values.
__device__ __forceinline__ float earlier_lanes(float v, int lane) {
    float w = v;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const float x = __shfl_up_sync(0xffffffffu, w, m);
        if (lane >= m) w += x;
    }
    const float x = __shfl_up_sync(0xffffffffu, w, 1);
    return lane ? x : 0.0f;
}
__device__ __forceinline__ void load8(const float *p, float (&v)[8]) {
    const float4 x = *reinterpret_cast<const float4 *>(p), y = *reinterpret_cast<const float4 *>(p + 4);
    v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w, v[4] = y.x, v[5] = y.y, v[6] = y.z, v[7] = y.w;
}

template <int DK, int DV> __global__ void __launch_bounds__(LT, 1) delta_local_kernel(const Args a) {
    using L = LocalSmem<DK, DV>;
    constexpr int PR = DV / 8;     // lanes of a token's row, 8 values each
    extern __shared__ __align__(1024) unsigned char raw[];
    unsigned char *smem = raw + ((1024u - (smem_addr(raw) & 1023u)) & 1023u);
    LocalBars *lb = reinterpret_cast<LocalBars *>(smem + L::bars);
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid / 32, 0), lane = tid % 32;
    const int N = chunks(a.L), group = a.Hv / a.Hk;
    const long long mat = (long long)DK * DV;
    const int items = N * a.Hk * a.B;   // below 2^30: a token and value head each at least
    if (tid == 0) {
        mbar_init(&lb->z_full, 1);
        mbar_init(&lb->first, 1);
        mbar_init(&lb->second, 1);
        mbar_init(&lb->third, 1);
        mbar_init(&lb->fourth, 1);
        lb->abort = 0;
        fence_mbar_init();
    }
    griddep_wait();
    if (warp == 0) {
        __syncwarp();
        tmem_alloc(&lb->tmem, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t kq = smem_addr(smem + L::kq), sA = smem_addr(smem + L::a), sU = smem_addr(smem + L::u),
                   sS = smem_addr(smem + L::s), sW = smem_addr(smem + L::wn), dv3 = smem_addr(smem + L::dv3),
                   s3 = smem_addr(smem + L::s3);
    // KK lies where D1 will, E1 where D2 has been, D3 (and dv's third part by U, D3L) where D4 and D5 will
    const uint32_t tmem = lb->tmem, D1 = tmem, D2 = tmem + 128, D4 = tmem + 256, D3 = tmem + 256, D3L = tmem + 448, D5 = tmem + 384,
                   KK = tmem, E1 = tmem + 128;
    const uint64_t A0 = desc_k(sA), W0 = desc_k(sW), WT = desc_mn(sW, M2_BYTES), U0 = desc_k(sU), S0 = desc_k(sS),
                   cols = desc_mn(kq, KQ_BOX), rows = desc_k(kq);
    Meta *meta = reinterpret_cast<Meta *>(smem + L::meta);
    float(*part)[16] = reinterpret_cast<float(*)[16]>(smem + L::part);       // [warp][column]
    float(*suffix)[32] = reinterpret_cast<float(*)[32]>(smem + L::suffix);   // [warp][row]
    float(*reads)[4] = reinterpret_cast<float(*)[4]>(smem + L::rows);        // [row][32 columns]
    auto wait = [&](uint64_t *bar, int parity) { return bounded_wait(bar, (uint32_t)parity, &lb->abort); };
    // warp w: TMEM lanes 32 (w % 4) on, columns 32 (w / 4) on; of D3 and [W; N]
    // columns 16 (w / 4) on
    const int row = 32 * (warp & 3) + lane, c0 = warp / 4 * 32, tk = row & 63;
    const bool keys = row < C;
    const uint32_t quarter = (uint32_t)(32 * (warp & 3)) << 16;
    bool ok = true;
    int phase = 0;
    for (int item = blockIdx.x; item < items; item += gridDim.x) {
        const int c = item % N, hk = item / N % a.Hk, b = item / N / a.Hk;
        const int t0 = c * C, nt = min(C, a.L - t0);
        const long long row0 = (long long)b * a.L + t0;
#pragma unroll
        for (int n = 0; n < 128 * (DK / 8) / LT; ++n) {
            const int i = tid + n * LT, r = i / (DK / 8), d = i % (DK / 8) * 8, t = r & 63;
            uint4 v = make_uint4(0, 0, 0, 0);
            if (t < nt)
                v = r < C ? *reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(a.k) + (row0 + t) * a.ldk + hk * DK + d)
                          : *reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(a.q) + (row0 + t) * a.ldq + hk * DK + d);
            sts128(piece(kq + d / 64 * KQ_BOX, r, d % 64 / 8), v.x, v.y, v.z, v.w);
        }
        float sum[32] = {};
        for (int j = 0; j < group; ++j, phase ^= 1) {
            const int h = hk * group + j;
            const long long bh = (long long)b * a.Hv + h;
            if (warp == TAIL && lane == 0) {
                mbar_arrive_tx(&lb->z_full, 2 * L::S_IMG + META_BYTES);
                const unsigned char *z = static_cast<const unsigned char *>(a.z) + (bh * N + c) * (2 * L::S_IMG);
                for (int x = 0; x < DV / 64; ++x)
                    for (int p = 0; p < 2; ++p)
                        bulk_load(smem + L::s + (2 * x + p) * (DK * 128), z + (2 * x + p) * (DK * 128), DK * 128, &lb->z_full);
                bulk_load(meta, static_cast<const unsigned char *>(a.images) + (bh * N + c) * IMG_BYTES + MAT_BYTES, META_BYTES, &lb->z_full);
            }
#pragma unroll
            for (int n = 0; n < C * PR / LT; ++n) {
                const int i = tid + n * LT, t = i / PR, d = i % PR * 8;
                const long long hv = (row0 + t) * a.Hv + h;
                float x[8] = {}, e[8] = {}, s1 = 0.0f, be = 0.0f;
                uint4 g = make_uint4(0, 0, 0, 0);
                if (t < nt) {
                    load8(a.x + hv * DV + d, x);
                    load8(a.e + hv * DV + d, e);
                    g = *reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(a.dout) + (row0 + t) * a.lddo + (long long)h * DV + d);
                    be = a.beta[hv];
                }
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    s1 = fmaf(x[k], e[k], s1);
                    x[k] *= be, e[k] *= be;
                }
                const int box = d / 64, at = d % 64 / 8;
                put3(sA + box * M2_BYTES, L::A_IMG, dv3 + box * RU_IMG, t, at, x);
                put3(sU + box * 3 * RU_IMG, RU_IMG, sU + (box * 3 + 2) * RU_IMG, t, at, e);
                sts128(piece(sA + box * M2_BYTES, C + t, at), g.x, g.y, g.z, g.w);
                sts128(piece(sA + L::A_IMG + box * M2_BYTES, C + t, at), 0, 0, 0, 0);   // dO is bf16: no second part
#pragma unroll
                for (int m = PR / 2; m > 0; m >>= 1) s1 += __shfl_xor_sync(0xffffffffu, s1, m);
                if (t < nt) {
                    *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.dv) + (row0 + t) * a.lddv + (long long)h * DV + d) =
                        make_uint4(pack2(x[0], x[1]), pack2(x[2], x[3]), pack2(x[4], x[5]), pack2(x[6], x[7]));
                    if (d == 0) a.dbeta[hv] = s1;
                }
            }
            fence_proxy_async_smem();
            __syncthreads();
            const uint32_t id = idesc_bf16_f32(128, DK), idU = idesc_bf16_f32(128, 64);
            if (warp == ISSUE) {
                if (elect_one()) {
                    // U's parts are columns of one product each; D3's blocks are added when they are read
                    const uint32_t id3 = idesc_bf16_f32(128, 192), id2 = idesc_bf16_f32(128, 128);
#pragma unroll
                    for (int k = 0; k < DV / 16; ++k)
                        mma_bf16(D3, on(A0, k / 4 * M2_BYTES + k % 4 * K_STEP), on(U0, k / 4 * 3 * RU_IMG + k % 4 * K_STEP), id3, k > 0);
#pragma unroll
                    for (int k = 0; k < DV / 16; ++k)
                        mma_bf16(D3, on(A0, L::A_IMG + k / 4 * M2_BYTES + k % 4 * K_STEP), on(U0, k / 4 * 3 * RU_IMG + k % 4 * K_STEP), id2, 1);
#pragma unroll
                    for (int k = 0; k < DV / 16; ++k)
                        mma_bf16(D3L, on(desc_k(dv3), k / 4 * RU_IMG + k % 4 * K_STEP), on(U0, k / 4 * 3 * RU_IMG + k % 4 * K_STEP), idU, k > 0);
#pragma unroll
                    for (int k = 0; k < DK / 16; ++k) {
                        const uint64_t K = on(rows, k / 4 * KQ_BOX + k % 4 * K_STEP);
                        mma_bf16(KK, K, K, idU, k > 0);
                    }
                    mma_commit(&lb->first);
                }
                __syncwarp();
                const bool z = wait(&lb->z_full, phase);
                if (elect_one()) {
                    if (z) {
#pragma unroll
                        for (int ps = 1; ps >= 0; --ps)
#pragma unroll
                            for (int p = 0; p <= ps; ++p)
#pragma unroll
                                for (int k = 0; k < DV / 16; ++k)
                                    mma_bf16(D2, on(U0, p * RU_IMG + k / 4 * 3 * RU_IMG + k % 4 * K_STEP),
                                             on(S0, (ps - p) * (DK * 128) + k / 4 * (2 * DK * 128) + k % 4 * K_STEP), id,
                                             !(ps == 1 && p == 0 && k == 0));
                    }
                    mma_commit(&lb->second);
                }
                __syncwarp();
            }
            // the next head's tiles come to L2 while the first products run
            if (j + 1 < group) {
                prefetch_head<DK, DV>(a, c, b, h + 1, false, N, tid);
            } else if (const int next = item + (int)gridDim.x; next < items) {
                prefetch_head<DK, DV>(a, next % N, next / N / a.Hk, next / N % a.Hk * group, true, N, tid);
            }
            // [W; N], and M in mm: a block of 16 columns a warp.  Decay factors of
            // two blocks are products at the end of the columns' block, as in the
            // preparation
            ok = wait(&lb->z_full, phase) && wait(&lb->first, phase) && ok;
            tc_fence_after();
            const int nb = warp >> 2, cb = 16 * nb;
            float w[16], mm[16];
            {
                const int rb = tk >> 4;
                load_parts<3, 16>(D3 + quarter + cb, w);
                if (keys) {
                    load_parts<1, 16>(D3L + quarter + cb, mm);
#pragma unroll
                    for (int i = 0; i < 16; ++i) w[i] += mm[i];
                }
                load_parts<1, 16>(KK + quarter + cb, mm);
                const float gh = meta->hi[tk], gl = meta->lo[tk], eh = meta->hi[cb + 15], el = meta->lo[cb + 15];
                const int mine = cb + (lane & 15);
                const float near = expf((eh - meta->hi[mine]) + (el - meta->lo[mine]));
                const float sign = keys ? -1.0f : a.scale, far = nb < rb ? sign * expf((gh - eh) + (gl - el)) : 0.0f;
                const bool own = nb == rb, any = __any_sync(0xffffffffu, own);
                float e[8] = {};
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int col = cb + i;
                    if (any && i % 8 == 0)   // eight at a time in flight
#pragma unroll
                        for (int k = 0; k < 8; ++k) e[k] = expf((gh - meta->hi[col + k]) + (gl - meta->lo[col + k]));
                    const float f = far * __shfl_sync(0xffffffffu, near, i), d = own ? sign * e[i % 8] : f;
                    // a masked product may be infinite: it is not multiplied by 0
                    w[i] = (keys ? col < tk : col <= tk) ? d * w[i] : 0.0f;
                    mm[i] = col < tk ? w[i] * mm[i] : 0.0f;
                }
            }
            // M's sums: mm[i] becomes the row's sum up to column cb + i - 1, for the
            // token cb + i where it is at or before the row
            float total = 0.0f;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float v = mm[i];
                mm[i] = tk >= cb + i ? total : 0.0f;
                total += v;
            }
            const float crossing = sum16(mm, lane), rest = later_lanes(total, lane);
            // S0 is on its way while the second products run
            const float *s0 = a.states + (bh * (N + 1) + c) * mat;
            constexpr int SN = DK * DV / 8 / LT;
            float4 sr[2 * SN];
#pragma unroll
            for (int n = 0; n < SN; ++n) {
                sr[2 * n] = *reinterpret_cast<const float4 *>(s0 + (tid + n * LT) * 8);
                sr[2 * n + 1] = *reinterpret_cast<const float4 *>(s0 + (tid + n * LT) * 8 + 4);
            }
            ok = wait(&lb->second, phase) && ok;
            tc_fence_after();
#pragma unroll
            for (int n = 0; n < SN; ++n) {
                const int i = tid + n * LT, r = i / PR, d = i % PR * 8;
                const float v[8] = {sr[2 * n].x,     sr[2 * n].y,     sr[2 * n].z,     sr[2 * n].w,
                                    sr[2 * n + 1].x, sr[2 * n + 1].y, sr[2 * n + 1].z, sr[2 * n + 1].w};
                put3(sS + d / 64 * (2 * DK * 128), DK * 128, s3 + d / 64 * (DK * 128), r, d % 64 / 8, v);
            }
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                const float v[8] = {w[8 * n], w[8 * n + 1], w[8 * n + 2], w[8 * n + 3], w[8 * n + 4], w[8 * n + 5], w[8 * n + 6], w[8 * n + 7]};
                put2(sW, M2_BYTES, row, 2 * nb + n, v);
            }
            const float up = meta->up[tk], down = meta->down[tk];
            if (c0 < DK && keys) {   // D2, before E1 takes its place
                float x[32];
                load_parts<1, 32>(D2 + quarter + c0, x);
#pragma unroll
                for (int i = 0; i < 32; ++i) sum[i] = fmaf(down, x[i], sum[i]);
            }
            fence_proxy_async_smem();
            tc_fence_before();
            __syncthreads();
            tc_fence_after();
            if (warp == ISSUE && elect_one()) {
                const uint32_t idB = id | B_MN, idAB = idB | A_MN, idE = idesc_bf16_f32(128, DV) | B_MN;
                const uint64_t SE = desc_mn(sS, 2 * DK * 128), SL = desc_mn(s3, DK * 128);
#pragma unroll
                for (int p = 1; p >= 0; --p) {
#pragma unroll
                    for (int k = 0; k < C / 16; ++k)
                        mma_bf16(D4, on(W0, p * M2_BYTES + k * K_STEP), on(cols, k * MN_STEP), idB, !(p == 1 && k == 0));
#pragma unroll
                    for (int k = 0; k < 2 * C / 16; ++k)
                        mma_bf16(D5, on(WT, p * M2_BYTES + k * MN_STEP), on(cols, k * MN_STEP), idAB, !(p == 1 && k == 0));
                }
#pragma unroll
                for (int ps = 1; ps >= 0; --ps)
#pragma unroll
                    for (int p = 0; p <= ps; ++p)
#pragma unroll
                        for (int k = 0; k < DV / 16; ++k)
                            mma_bf16(D1, on(A0, p * L::A_IMG + k / 4 * M2_BYTES + k % 4 * K_STEP),
                                     on(S0, (ps - p) * (DK * 128) + k / 4 * (2 * DK * 128) + k % 4 * K_STEP), id, !(ps == 1 && p == 0 && k == 0));
                mma_commit(&lb->third);
#pragma unroll
                for (int p = 2; p >= 0; --p)
#pragma unroll
                    for (int k = 0; k < DK / 16; ++k)
                        mma_bf16(E1, on(rows, k / 4 * KQ_BOX + k % 4 * K_STEP), p == 2 ? on(SL, k * MN_STEP) : on(SE, p * (DK * 128) + k * MN_STEP),
                                 idE, !(p == 2 && k == 0));
                mma_commit(&lb->fourth);
            }
            __syncwarp();
            float bj[2] = {}, inner = 0.0f;   // the tail's terms from the adjoint
            if (warp == TAIL) {
                constexpr int WP = write_parts(DV), IP = inner_parts(DK, DV);
                if (lane < IP) inner = a.inner[(bh * N + c) * IP + lane];
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int p = 0; p < WP; ++p) bj[i] += a.writes[((bh * N + c) * C + lane + 32 * i) * WP + p];
            }
            ok = wait(&lb->third, phase) && ok;
            tc_fence_after();
            if (c0 < DK) {
                float x[32];
                const float wd = keys ? -up : a.scale * up;
                load_parts<1, 32>(D1 + quarter + c0, x);
#pragma unroll
                for (int i = 0; i < 32; ++i) sum[i] = fmaf(wd, x[i], sum[i]);
                load_parts<1, 32>(D4 + quarter + c0, x);
#pragma unroll
                for (int i = 0; i < 32; ++i) sum[i] += x[i];
                if (keys) {
                    load_parts<1, 32>(D5 + quarter + c0, x);
#pragma unroll
                    for (int i = 0; i < 32; ++i) sum[i] += x[i];
                }
            }
            ok = wait(&lb->fourth, phase) && ok;
            tc_fence_after();
            float y[2][2] = {};   // E1's rows by dv or dO
            if (c0 < DV)
#pragma unroll
                for (int f = 0; f < 2; ++f) {
                    float x[16];
                    frag_load<1>(E1 + quarter + c0 + (f ? QUERY_LANES : 0u), x);
                    if (keys) {
                        float2 dx[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const int t = (row - lane) + 16 * f + lane / 4 + 8 * (i / 4);
                            dx[i] = t < nt ? *reinterpret_cast<const float2 *>(a.x + ((row0 + t) * a.Hv + h) * DV + c0 + 8 * (i % 4) + 2 * (lane & 3))
                                           : make_float2(0.0f, 0.0f);
                        }
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            y[f][i / 4] = fmaf(x[4 * (i % 4) + 2 * (i / 4)], dx[i].x, fmaf(x[4 * (i % 4) + 2 * (i / 4) + 1], dx[i].y, y[f][i / 4]));
                    } else {
                        float g[16];
                        frag_get(sA + c0 / 64 * M2_BYTES, row - lane + 16 * f, c0 % 64, lane, g);
#pragma unroll
                        for (int i = 0; i < 16; ++i) y[f][(i >> 1) & 1] = fmaf(x[i], g[i], y[f][(i >> 1) & 1]);
                    }
                }
            // the products are done with the state: its place takes the sums
            if ((lane & 1) == 0) part[warp][lane / 2] = crossing;
            suffix[warp][lane] = rest;
            if (c0 < DV)
#pragma unroll
                for (int f = 0; f < 2; ++f)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int r = row - lane + 16 * f + lane / 4 + 8 * i, t = r & 63;
                        float v = y[f][i];
                        v += __shfl_xor_sync(0xffffffffu, v, 1);
                        v += __shfl_xor_sync(0xffffffffu, v, 2);
                        if ((lane & 3) == 0) reads[r][c0 / 32] = meta->up[t] * (keys ? -meta->beta[t] : a.scale) * v;
                    }
            fence_proxy_async_smem();   // the next adjoint is copied over these
            tc_fence_before();
            __syncthreads();
            tc_fence_after();
            if (warp == TAIL) {   // tokens `lane` and `lane` + 32
                float ai[2] = {}, pairs[2] = {};
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int t = lane + 32 * i;
#pragma unroll
                    for (int g = 0; g < DV / 32; ++g) ai[i] += reads[t][g] + reads[C + t][g];
#pragma unroll
                    for (int q = 0; q < 4; ++q) pairs[i] += part[t / 16 * 4 + q][t % 16];
#pragma unroll
                    for (int n = 0; n < 2 * i + 1; ++n)   // whole blocks before the token's
                        if (n < t / 16) {
                            pairs[i] += suffix[4 * n + i][lane] + suffix[4 * n + 2 + i][lane];
                            if (i == 0) pairs[i] += suffix[4 * n + 1][0] + suffix[4 * n + 3][0];
                        }
                }
                const float m = meta->last * warp_sum(inner);
                // a from the token on, b up to it
                const float a1 = later_lanes(ai[1], lane), a0 = later_lanes(ai[0], lane) + __shfl_sync(0xffffffffu, a1, 0);
                const float b0 = earlier_lanes(bj[0], lane), b1 = earlier_lanes(bj[1], lane) + warp_sum(bj[0]);
                if (lane < nt) a.dg[(row0 + lane) * a.Hv + h] = (a0 + b0) + (m + pairs[0]);
                if (lane + 32 < nt) a.dg[(row0 + lane + 32) * a.Hv + h] = (a1 + b1) + (m + pairs[1]);
                __syncwarp();   // then the next adjoint is copied over what was read here
            }
        }
        // out by way of shared memory (A's place), whole rows at a time
        if (c0 < DK)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                sts128(piece(sA + c0 / 64 * M2_BYTES, row, c0 % 64 / 8 + j), pack2(sum[8 * j], sum[8 * j + 1]),
                       pack2(sum[8 * j + 2], sum[8 * j + 3]), pack2(sum[8 * j + 4], sum[8 * j + 5]), pack2(sum[8 * j + 6], sum[8 * j + 7]));
        __syncthreads();
        for (int i = tid; i < 128 * (DK / 8); i += LT) {
            const int r = i / (DK / 8), d = i % (DK / 8) * 8, t = r & 63;
            if (t >= nt) continue;
            __nv_bfloat16 *p = r < C ? static_cast<__nv_bfloat16 *>(a.dk) + (row0 + t) * a.lddk + hk * DK + d
                                     : static_cast<__nv_bfloat16 *>(a.dq) + (row0 + t) * a.lddq + hk * DK + d;
            *reinterpret_cast<uint4 *>(p) = lds128(piece(sA + d / 64 * M2_BYTES, r, d % 64 / 8));
        }
        __syncthreads();
        if (lb->abort) break;   // read behind a barrier: the same for all
    }
    if (!ok) settle_copies();
    __syncthreads();
    if (warp == 0) tmem_dealloc(tmem, 512);
}

template <int DK, int DV> cudaError_t launch_local(const Args &a, cudaStream_t st) {
    const cudaError_t e = big_smem(delta_local_kernel<DK, DV>, LocalSmem<DK, DV>::total);
    if (e != cudaSuccess) return e;
    const long long items = (long long)chunks(a.L) * a.Hk * a.B;
    return launch_after(delta_local_kernel<DK, DV>, (unsigned)(items < 152 ? items : 152), LT, LocalSmem<DK, DV>::total, st, a);
}

template <int DK> cudaError_t backward(const Args &a, cudaStream_t st) {
    AdjMaps m = {};
    cudaError_t e = encode_rows(&m.k, false, a.k, a.ldk, a.B, a.L, a.Hk, DK, 16);
    if (e == cudaSuccess) e = encode_rows(&m.q, false, a.q, a.ldq, a.B, a.L, a.Hk, DK, 16);
    if (e == cudaSuccess) e = encode_rows(&m.g, false, a.dout, a.lddo, a.B, a.L, a.Hv, a.Dv);
    if (e == cudaSuccess) e = encode_rows(&m.x, true, a.x, (long long)a.Hv * a.Dv, a.B, a.L, a.Hv, a.Dv);
    if (e == cudaSuccess) e = encode_states(&m.s, a.states, (long long)a.B * a.Hv * (chunks(a.L) + 1), DK, a.Dv);
    Args all = a;
    all.count = chunks(a.L);
    if (e == cudaSuccess) e = tc_prepare(all, true, st);
    if (e == cudaSuccess) e = big_smem(delta_adjoint_kernel<DK>, AdjSmem<DK>::total);
    if (e != cudaSuccess) return e;
    e = launch_after(delta_adjoint_kernel<DK>, dim3(a.Dv / NV, a.Hv, a.B), ADJ_THREADS, AdjSmem<DK>::total, st, m, a);
    if (e != cudaSuccess) return e;
    return a.Dv == 128 ? launch_local<DK, 128>(a, st) : launch_local<DK, 64>(a, st);
}

}  // namespace

cudaError_t tc_backward(const Args &a, cudaStream_t st) {
    return a.Dk == 128 ? backward<128>(a, st) : backward<64>(a, st);
}

int adjoint_fault_take() { return fault_take(); }

}  // namespace delta
}  // namespace s5
