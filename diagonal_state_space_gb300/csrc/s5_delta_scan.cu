// s5_delta_scan.cu -- the gated delta rule forward on the 5th-generation
// tensor cores: bf16 queries, keys and values, heads of 64 or 128.
//
// A chunk of 64 tokens that starts from the state S0, with G_i the sum of the
// chunk's log decays up to token i and D_ij = exp(G_i - G_j):
//   E = (I + strict lower(D_ij k_i.k_j beta_j))^-1,   P_ij = scale D_ij q_i.k_j (j <= i)
//   R = V - e^G K S0
//   e = E R,  o = scale e^G Q S0 + (P beta E) R
//   S = e^{G_64} S0 + K^T (e^{G_64 - G} beta e)
// Everything without S0 is done for all chunks at once (s5_delta_prep.cu): it
// leaves the 128 x 64 matrix [E; P beta E] of each chunk.  The recurrence over
// chunks then is three matrix products in a row for 64 value columns (a
// slice), whose state stays in registers:
//   D1 = [K; Q] S0        (128 x 64, depth Dk)
//   D2 = [E; P beta E] R  (128 x 64, depth 64)
//   D3 = K^T U            (Dk x 64, depth 64)
// all of M = 128: half the rows of the first two give the outputs beside the
// rows that the recurrence needs, 16 of each in turn, so that every warp's 32
// accumulator lanes hold 16 tokens of either.
//
// Precision.  Keys, queries and values are bf16 and enter the products as they
// are.  S0, R, U and [E; P beta E] are 32-bit values, carried as sums of three
// bf16 values that hold all their 24 bits: three products against a bf16
// operand, six against another split one (the three smallest, below 2^-23, are
// left out).  One rounding to bf16 instead would leave 2^-9 in the state.  The
// parts of an operand lie side by side, so that one MMA of N = 192 or 128
// covers them (an MMA of N = 64 costs 48 cycles here, of N = 192 96), and the
// reading thread adds the column blocks.
//
// A CTA takes one or two slices of a head, of 64 columns, or one of 32.  Bound:
// the chain product -> sums, splits -> product, three times a chunk.  With two
// slices the products of one run while the other converts; that pays once
// there are enough heads to fill the SMs anyway.  With few heads slices of 32
// columns shorten the chain (launch rule below): 2.1 us a chunk with heads of
// 128, 2.8 in slices of 64, whatever the number of heads that fit at once.  In
// two slices a CTA 8 sequences of 1999 tokens with 32 heads take 250 us, 275
// TFLOP/s of the three products, each of which is three to six bf16 products.
#include "s5_delta_mma.cuh"

namespace s5 {
namespace delta {
namespace {

struct ScanMaps {
    CUtensorMap k, q, v, o;
    CUtensorMap e, s;   // KEEP
};

template <int DK, int SL, bool KEEP, int NC> struct ScanSmem {
    static constexpr uint32_t KQ = KQ_BOX * (DK / 64);
    static constexpr uint32_t S_IMG = DK * 128;
    // S0's parts until D1 is done, R's until D2 is done, U's until D3 is done
    static constexpr uint32_t IMAGES = NC == 64 ? 3 : 2, OPS = IMAGES * S_IMG;
    static constexpr uint32_t VO = C * NC * 2;
    static constexpr uint32_t kq = 0;                      // two stages
    static constexpr uint32_t mat = kq + 2 * KQ;
    static constexpr uint32_t ops = mat + MAT_BYTES;
    static constexpr uint32_t vo = ops + SL * OPS;         // V, then o
    static constexpr uint32_t stage = vo + SL * VO;        // KEEP: a state, or e in 32 bits
    static constexpr uint32_t meta = stage + (KEEP ? 32768 : 0);
    static constexpr uint32_t bars = meta + META_BYTES;
    static constexpr uint32_t total = bars + 256 + 1024;   // + alignment slack
    static_assert(total <= 232448, "shared memory of a CTA");
    static_assert(S_IMG >= RU_IMG, "R and U fit S0's place");
};

struct ScanBars {
    uint64_t kq_full[2], kq_empty[2], img_full, img_empty;
    uint64_t d1[2], d2[2], d3[2];                    // products done, per slice
    uint64_t s_ready[2], r_ready[2], u_ready[2];     // operands in place
    uint64_t v_full[2], o_ready[2];
    uint64_t state_staged, rows_staged, stage_free, drain;
    uint32_t tmem;
    int abort;
};
static_assert(sizeof(ScanBars) <= 256, "barriers");

template <int SL> constexpr int SCAN_THREADS = SL == 1 ? 320 : 576;

// NC: value columns of a slice, 64 or 32.
template <int DK, int SL, bool KEEP, int NC>
__global__ void __launch_bounds__(SCAN_THREADS<SL>, 1) delta_scan_kernel(const __grid_constant__ ScanMaps maps, const Args a) {
    using L = ScanSmem<DK, SL, KEEP, NC>;
    static_assert(!(KEEP && SL == 2), "the staged tiles take the second slice's place");
    static_assert(NC == 64 || (SL == 1 && !KEEP), "slices of 32 columns: one a CTA, nothing kept");
    constexpr bool NARROW = NC == 32;
    constexpr uint32_t L_PART = NARROW ? 1 : 2;   // the image of the third parts
    constexpr int P1 = SL == 1 ? 3 : 2;     // column blocks of D1 and D3: TMEM has 256 columns for each of two slices
    constexpr int PW = NC / 2, F = NC / 4;  // a warp's columns, and a thread's values of a fragment
    // narrow slices leave columns to the preparation of later chunks (P1, 2, P1 blocks of 32)
    constexpr int TMEM = NARROW ? 256 : 512;
    constexpr int W = SL == 1 ? PW : 16;    // columns converted at a time: registers for each of 16 warps
    extern __shared__ __align__(1024) unsigned char raw[];
    unsigned char *smem = raw + ((1024u - (smem_addr(raw) & 1023u)) & 1023u);
    ScanBars *sb = reinterpret_cast<ScanBars *>(smem + L::bars);
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0), lane = threadIdx.x % 32;
    const int n0 = blockIdx.x * SL * NC, h = blockIdx.y, b = blockIdx.z, hk = h / (a.Hv / a.Hk);
    // this launch's chunks: N of them, from `from` on
    const int N = a.count, from = a.from, all = chunks(a.L);
    const long long bh = (long long)b * a.Hv + h;
    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sb->kq_full[i], 1), mbar_init(&sb->kq_empty[i], 1);
            mbar_init(&sb->d1[i], 1), mbar_init(&sb->d2[i], 1), mbar_init(&sb->d3[i], 1);
            mbar_init(&sb->s_ready[i], 8), mbar_init(&sb->r_ready[i], 8), mbar_init(&sb->u_ready[i], 8);
            mbar_init(&sb->v_full[i], 1), mbar_init(&sb->o_ready[i], 8);
        }
        mbar_init(&sb->img_full, 1), mbar_init(&sb->img_empty, 8 * SL);
        mbar_init(&sb->state_staged, 8), mbar_init(&sb->rows_staged, 8), mbar_init(&sb->stage_free, 1);
        mbar_init(&sb->drain, 1);
        sb->abort = 0;
        fence_mbar_init();
    }
    constexpr int MMA_WARP = 8 * SL, COPY_WARP = MMA_WARP + 1;
    griddep_wait();
    if (a.first) griddep_launch_dependents();   // the rest's preparation needs nothing from here
    if (warp == MMA_WARP) {
        tmem_alloc(&sb->tmem, TMEM);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sb->tmem;
    // D3 takes D1's place where two slices share the columns: every warp has
    // read D1 before it hands U over
    constexpr uint32_t SLICE = 256, D1 = 0, D2 = P1 * NC, D3 = SL == 1 ? 5 * NC : 0;
    auto wait = [&](uint64_t *bar, int parity) { return bounded_wait(bar, (uint32_t)parity, &sb->abort); };

    if (warp >= 8 * SL) {
        if (warp == COPY_WARP && lane == 0) {
            // ------------------------------------------------------ copies
            auto load_kq = [&](int c) {
                load_chunk_rows<DK>(smem + L::kq + (c & 1) * L::KQ, &maps.k, &maps.q, hk, (from + c) * C, b, &sb->kq_full[c & 1]);
            };
            auto load_img = [&](int c) {
                const unsigned char *image = static_cast<const unsigned char *>(a.images) + (bh * all + from + c) * IMG_BYTES;
                mbar_arrive_tx(&sb->img_full, IMG_BYTES);
                bulk_load(smem + L::mat, image, MAT_BYTES, &sb->img_full);
                bulk_load(smem + L::meta, image + MAT_BYTES, META_BYTES, &sb->img_full);
            };
            auto load_v = [&](int c, int s) {
                mbar_arrive_tx(&sb->v_full[s], L::VO);
                tma_load_4d(smem + L::vo + s * L::VO, &maps.v, n0 + s * NC, h, (from + c) * C, b, &sb->v_full[s]);
            };
            load_kq(0);
            load_img(0);
            for (int s = 0; s < SL; ++s) load_v(0, s);
            if (N > 1) load_kq(1);
            bool ok = true;
            for (int c = 0; c < N; ++c) {
                if constexpr (KEEP) {
                    if (!(ok = wait(&sb->state_staged, c & 1))) break;
                    for (int x = 0; x < 2; ++x)
                        tma_store_3d(&maps.s, smem + L::stage + x * (DK * 128), n0 + 32 * x, 0, (int)(bh * (N + 1) + c));
                    bulk_commit();
                    bulk_wait_read_all();
                    mbar_arrive(&sb->stage_free);
                }
                if (c + 1 < N) {
                    if (!(ok = wait(&sb->img_empty, c & 1))) break;
                    load_img(c + 1);
                }
                for (int s = 0; ok && s < SL; ++s) {
                    if (!(ok = wait(&sb->o_ready[s], c & 1))) break;
                    tma_store_4d(&maps.o, smem + L::vo + s * L::VO, n0 + s * NC, h, (from + c) * C, b);
                    bulk_commit();
                    if (c + 1 < N) {
                        bulk_wait_read_all();
                        load_v(c + 1, s);
                    }
                }
                if (!ok) break;
                if constexpr (KEEP) {
                    if (!(ok = wait(&sb->rows_staged, c & 1))) break;
                    for (int x = 0; x < 2; ++x) tma_store_4d(&maps.e, smem + L::stage + x * RU_IMG, n0 + 32 * x, h, c * C, b);
                    bulk_commit();
                    bulk_wait_read_all();
                    mbar_arrive(&sb->stage_free);
                }
                if (c + 2 < N) {
                    if (!(ok = wait(&sb->kq_empty[c & 1], (c >> 1) & 1))) break;
                    load_kq(c + 2);
                }
            }
            if constexpr (KEEP)
                if (ok && (ok = wait(&sb->state_staged, N & 1))) {
                    for (int x = 0; x < 2; ++x)
                        tma_store_3d(&maps.s, smem + L::stage + x * (DK * 128), n0 + 32 * x, 0, (int)(bh * (N + 1) + N));
                    bulk_commit();
                }
            bulk_wait_all();
            if (!ok) settle_copies();
        } else if (warp == MMA_WARP) {
            // ------------------------------------------------------ products
            const uint32_t w1 = idesc_bf16_f32(128, NC) | B_MN, w2 = idesc_bf16_f32(128, 2 * NC) | B_MN,
                           w3 = idesc_bf16_f32(128, 3 * NC) | B_MN;
            const uint64_t mat = desc_k(smem_addr(smem + L::mat));
            bool ok = true;
            for (int c = 0; ok && c < N; ++c) {
                const uint32_t kq = smem_addr(smem + L::kq + (c & 1) * L::KQ);
                const uint64_t rows = desc_k(kq), cols = desc_mn(kq, KQ_BOX);
                ok = wait(&sb->kq_full[c & 1], (c >> 1) & 1);
#pragma unroll
                for (int s = 0; s < SL; ++s) {
                    const uint32_t d = tmem + s * SLICE + D1;
                    const uint64_t S = desc_mn(smem_addr(smem + L::ops + s * L::OPS), L::S_IMG);
                    ok = __all_sync(0xffffffffu, ok && wait(&sb->s_ready[s], c & 1));
                    if (!ok) break;
                    tc_fence_after();
                    if (elect_one()) {
#pragma unroll
                        for (int k = 0; k < DK / 16; ++k) {
                            const uint64_t A = on(rows, k / 4 * KQ_BOX + k % 4 * K_STEP);
                            if constexpr (P1 == 3) {
                                mma_bf16(d, A, on(S, k * MN_STEP), w3, k > 0);
                            } else {
                                mma_bf16(d, A, on(S, k * MN_STEP), w2, k > 0);
                                mma_bf16(d, A, on(S, 2 * L::S_IMG + k * MN_STEP), w1, 1);
                            }
                        }
                        mma_commit(&sb->d1[s]);
                    }
                    __syncwarp();
                }
                ok = __all_sync(0xffffffffu, ok && wait(&sb->img_full, c & 1));
                if (!ok) break;
#pragma unroll
                for (int s = 0; s < SL; ++s) {
                    const uint32_t d = tmem + s * SLICE + D2;
                    const uint64_t R = desc_mn(smem_addr(smem + L::ops + s * L::OPS), RU_IMG);
                    ok = __all_sync(0xffffffffu, ok && wait(&sb->r_ready[s], c & 1));
                    if (!ok) break;
                    tc_fence_after();
                    if (elect_one()) {
#pragma unroll
                        for (int k = 0; k < C / 16; ++k) {
                            mma_bf16(d, on(mat, M2_BYTES + k * K_STEP), on(R, k * MN_STEP), w2, k > 0);
                            mma_bf16(d, on(mat, 2 * M2_BYTES + k * K_STEP), on(R, k * MN_STEP), w1, 1);
                            mma_bf16(d, on(mat, k * K_STEP), on(R, L_PART * RU_IMG + k * MN_STEP), w1, 1);
                            mma_bf16(d, on(mat, k * K_STEP), on(R, k * MN_STEP), w2, 1);
                        }
                        mma_commit(&sb->d2[s]);
                    }
                    __syncwarp();
                }
                // M is 128 for heads of 64 too: their lanes 64..127 of D3 come
                // from whatever follows the keys in shared memory, and are not read
#pragma unroll
                for (int s = 0; s < SL; ++s) {
                    const uint32_t d = tmem + s * SLICE + D3;
                    const uint64_t U = desc_mn(smem_addr(smem + L::ops + s * L::OPS), RU_IMG);
                    ok = __all_sync(0xffffffffu, ok && wait(&sb->u_ready[s], c & 1));
                    if (!ok) break;
                    tc_fence_after();
                    if (elect_one()) {
#pragma unroll
                        for (int k = 0; k < C / 16; ++k) {
                            const uint64_t A = on(cols, 2 * k * KQ_GROUP);
                            if constexpr (P1 == 3) {
                                mma_bf16(d, A, on(U, k * MN_STEP), w3 | A_MN, k > 0);
                            } else {
                                mma_bf16(d, A, on(U, k * MN_STEP), w2 | A_MN, k > 0);
                                mma_bf16(d, A, on(U, 2 * RU_IMG + k * MN_STEP), w1 | A_MN, 1);
                            }
                        }
                        mma_commit(&sb->d3[s]);
                        if (s == SL - 1) mma_commit(&sb->kq_empty[c & 1]);
                    }
                    __syncwarp();
                }
            }
            if (elect_one()) drain_products(&sb->drain);
        }
        __syncwarp();
    } else {
        // ---------------------------------------------------------- compute
        // Eight warps a slice; warp w: TMEM lanes 32 (w % 4) on, columns
        // PW (w / 4) on.  In D1 and D2 its first 16 lanes are tokens of R and
        // e, the others tokens of o; in D3 and in the state a lane is a key
        // index.
        const int s = warp / 8, q = warp & 3, c0 = warp % 8 / 4 * PW, row = 32 * q + lane;
        const int t16 = 16 * q, ta = t16 + lane / 4, tb = ta + 8;   // tokens of a fragment's rows
        const uint32_t acc = tmem + s * SLICE + ((uint32_t)(32 * q) << 16) + c0;
        const uint32_t ops = smem_addr(smem + L::ops + s * L::OPS), vo = smem_addr(smem + L::vo + s * L::VO);
        const uint32_t stage = smem_addr(smem + L::stage);
        const Meta *meta = reinterpret_cast<const Meta *>(smem + L::meta);
        const bool state = row < DK;
        const long long place = bh * DK * a.Dv + (long long)row * a.Dv + n0 + s * NC + c0;   // this row in s0, s_last
        float S[PW];
#pragma unroll
        for (int j = 0; j < PW / 4; ++j) {
            const float4 t = (a.s0 && state) ? *reinterpret_cast<const float4 *>(a.s0 + place + 4 * j) : make_float4(0, 0, 0, 0);
            S[4 * j] = t.x, S[4 * j + 1] = t.y, S[4 * j + 2] = t.z, S[4 * j + 3] = t.w;
        }
        if (state) put3<PW, NARROW>(ops, L::S_IMG, row, c0, S);
        hand_over(&sb->s_ready[s], lane);
        if constexpr (KEEP) {
            if (state) put_row(stage + c0 / 32 * (DK * 128), row, S);
            hand_over(&sb->state_staged, lane);
        }
        for (int c = 0; c < N; ++c) {
            bool ok = wait(&sb->img_full, c & 1) && wait(&sb->v_full[s], c & 1) && wait(&sb->d1[s], c & 1);
            if (!__all_sync(0xffffffffu, ok)) break;
            tc_fence_after();
            float f[F], o[F];
            const float ua = meta->up[ta], ub = meta->up[tb];
            {   // R
                frag_get(vo, t16, c0, lane, o);
                frag_load<P1>(acc + D1, f);
#pragma unroll
                for (int i = 0; i < F; ++i) f[i] = fmaf(-((i & 2) ? ub : ua), f[i], o[i]);
                frag_put3(ops, RU_IMG, t16, c0, lane, f);
                hand_over(&sb->r_ready[s], lane);
            }
            const float da = meta->beta[ta] * meta->down[ta], db = meta->beta[tb] * meta->down[tb], last = meta->last;
            frag_load<P1>(acc + D1 + QUERY_LANES, o);
            frag_scale(o, a.scale * ua, a.scale * ub);
            ok = wait(&sb->d2[s], c & 1);
            if (!__all_sync(0xffffffffu, ok)) break;
            tc_fence_after();
            if (lane == 0) mbar_arrive(&sb->img_empty);   // D2 is done with the matrix, this warp with its factors
            {   // e, U
                frag_load<2>(acc + D2, f);
                float u[F];
#pragma unroll
                for (int i = 0; i < F; ++i) u[i] = f[i] * ((i & 2) ? db : da);
                frag_put3(ops, RU_IMG, t16, c0, lane, u);
                hand_over(&sb->u_ready[s], lane);
                frag_load<2>(acc + D2 + QUERY_LANES, u);
#pragma unroll
                for (int i = 0; i < F; ++i) o[i] += u[i];
                frag_round(vo, t16, c0, lane, o);
                hand_over(&sb->o_ready[s], lane);
            }
            if constexpr (KEEP) {
                ok = wait(&sb->stage_free, 0);
                if (!__all_sync(0xffffffffu, ok)) break;
                frag_put_rows(stage + c0 / 32 * RU_IMG, t16, lane, f);
                hand_over(&sb->rows_staged, lane);
            }
            ok = wait(&sb->d3[s], c & 1);
            if (!__all_sync(0xffffffffu, ok)) break;
            tc_fence_after();
            if (state) {
#pragma unroll
                for (int w = 0; w < PW; w += W) {
                    float y[W];
                    load_parts<P1, W, NC>(acc + D3 + w, y);
#pragma unroll
                    for (int i = 0; i < W; ++i) S[w + i] = fmaf(last, S[w + i], y[i]);
                    if (c + 1 < N) put3<W, NARROW>(ops, L::S_IMG, row, c0 + w, S + w);
                }
            }
            if (c + 1 < N) hand_over(&sb->s_ready[s], lane);
            if constexpr (KEEP) {
                ok = wait(&sb->stage_free, 1);
                if (!__all_sync(0xffffffffu, ok)) break;
                if (state) put_row(stage + c0 / 32 * (DK * 128), row, S);
                hand_over(&sb->state_staged, lane);
            }
        }
        if (state && a.s_last)
#pragma unroll
            for (int j = 0; j < PW / 4; ++j)
                *reinterpret_cast<float4 *>(a.s_last + place + 4 * j) = make_float4(S[4 * j], S[4 * j + 1], S[4 * j + 2], S[4 * j + 3]);
        tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
    if (warp == MMA_WARP) tmem_dealloc(tmem, TMEM);
}

template <int DK, int SL, bool KEEP, int NC> cudaError_t launch(const ScanMaps &m, const Args &a, cudaStream_t st) {
    using L = ScanSmem<DK, SL, KEEP, NC>;
    const cudaError_t e = big_smem(delta_scan_kernel<DK, SL, KEEP, NC>, L::total);
    if (e != cudaSuccess) return e;
    return launch_after(delta_scan_kernel<DK, SL, KEEP, NC>, dim3(a.Dv / (SL * NC), a.Hv, a.B), SCAN_THREADS<SL>, L::total, st, m, a);
}

// Where the scan leaves half of the SMs free, the first quarter of the chunks is
// prepared and scanned, and the rest prepared beside that scan, from this many
// chunks of all heads on (below, two more launches gain little or nothing).  One
// piece / two, heads of 128, us: 16 heads, 32 chunks 86 / 83, 64 chunks 170 / 155,
// 256 chunks 636 / 591; 8 heads, 256 chunks 586 / 562; 32 heads (128 of 152 SMs
// scan), 64 chunks 199 / 203.  A half or a sixth first: 15 and 3 more at 16 heads, 256
// chunks.
constexpr int SPLIT_CHUNKS = 1024, SPLIT = 4;

template <int DK> cudaError_t forward(const Args &a, cudaStream_t st) {
    ScanMaps m = {};
    // Slices of 32 columns where one CTA each still fits the SMs at once; two
    // slices a CTA where one would not.  10 chunks, heads of 128, one slice of 64
    // / two / one of 32, us of the whole call: 38 heads 45 / 54 / 37, 76 heads 55 /
    // 63 / 72, 80 heads 85 / 64 / 94, 256 heads 195 / 149 / 240.
    const long long heads = (long long)a.B * a.Hv;
    const bool narrow = !a.states && heads * (a.Dv / 32) <= 152;
    cudaError_t e = encode_rows(&m.k, false, a.k, a.ldk, a.B, a.L, a.Hk, DK, 16);
    if (e == cudaSuccess) e = encode_rows(&m.q, false, a.q, a.ldq, a.B, a.L, a.Hk, DK, 16);
    if (e == cudaSuccess) e = encode_rows(&m.v, false, a.v, a.ldv, a.B, a.L, a.Hv, a.Dv, C, narrow ? 32 : 64);
    if (e == cudaSuccess) e = encode_rows(&m.o, false, a.o, a.ldo, a.B, a.L, a.Hv, a.Dv, C, narrow ? 32 : 64);
    if (a.states) {
        const long long ld = (long long)a.Hv * a.Dv;
        if (e == cudaSuccess) e = encode_rows(&m.e, true, a.e, ld, a.B, a.L, a.Hv, a.Dv);
        if (e == cudaSuccess) e = encode_states(&m.s, a.states, (long long)a.B * a.Hv * (chunks(a.L) + 1), DK, a.Dv);
    }
    Args all = a;
    all.count = chunks(a.L);
    if (narrow && heads * (a.Dv / 32) <= 76 && heads * all.count >= SPLIT_CHUNKS) {
        Args first = all, rest = all;
        first.count = rest.from = all.count / SPLIT;
        rest.count -= first.count;
        float *carry = reinterpret_cast<float *>(static_cast<char *>(a.images) + heads * all.count * IMG_BYTES);
        first.s_last = carry, rest.s0 = carry, first.first = rest.beside = true;
        if (e == cudaSuccess) e = tc_prepare(first, false, st);
        if (e == cudaSuccess) e = launch<DK, 1, false, 32>(m, first, st);
        if (e == cudaSuccess) e = tc_prepare(rest, false, st);
        return e == cudaSuccess ? launch<DK, 1, false, 32>(m, rest, st) : e;
    }
    if (e == cudaSuccess) e = tc_prepare(all, false, st);
    if (e != cudaSuccess) return e;
    if (a.states) return launch<DK, 1, true, 64>(m, all, st);
    if (narrow) return launch<DK, 1, false, 32>(m, all, st);
    if (a.Dv == 128 && heads * 2 > 152) return launch<DK, 2, false, 64>(m, all, st);
    return launch<DK, 1, false, 64>(m, all, st);
}

}  // namespace

// bf16 with heads of 64 or 128; pitches that the copies can address (multiples
// of 16 bytes).
bool tc_supported(const Args &a, s5_dtype dtype, bool backward) {
    if (dtype != S5_BF16 || a.L < 1) return false;
    if ((a.Dk != 64 && a.Dk != 128) || (a.Dv != 64 && a.Dv != 128)) return false;
    if (a.ldq % 8 || a.ldk % 8 || a.ldv % 8) return false;
    return backward ? a.lddo % 8 == 0 && a.lddq % 8 == 0 && a.lddk % 8 == 0 && a.lddv % 8 == 0 : a.ldo % 8 == 0;
}

size_t tc_image_bytes(int B, int L, int Hv, int Dk, int Dv) {
    if ((Dk != 64 && Dk != 128) || (Dv != 64 && Dv != 128)) return 0;
    return (size_t)B * Hv * (chunks(L) * (size_t)IMG_BYTES + sizeof(float) * Dk * Dv);   // and a state
}

cudaError_t tc_forward(const Args &a, cudaStream_t st) {
    return a.Dk == 128 ? forward<128>(a, st) : forward<64>(a, st);
}

int scan_fault_take() { return fault_take(); }

}  // namespace delta
}  // namespace s5

extern "C" int s5_delta_fault(void) {
    const int f[3] = {s5::delta::prep_fault_take(), s5::delta::scan_fault_take(), s5::delta::adjoint_fault_take()};
    return f[0] < 0 || f[1] < 0 || f[2] < 0 ? -1 : f[0] | f[1] | f[2];
}
