// s5_delta.cu -- the gated delta rule: a linear recurrence whose state is a
// matrix S [Dk][Dv] per sequence and value head, with a = exp(g):
//   e_t = v_t - a_t S_{t-1}^T k_t,  u_t = beta_t e_t,
//   S_t = a_t S_{t-1} + k_t u_t^T,  o_t = scale S_t^T q_t.
// This file has the entry points, the single-token step and the CUDA-core
// sweeps that serve every type and head size; bf16 heads of 64 or 128 run on
// the tensor cores in chunks of 64 tokens (s5_delta_prep.cu, s5_delta_scan.cu,
// s5_delta_adjoint.cu).
//
// Sweeps.  Every column of S (a value index) is a recurrence of its own given
// the keys, and every row (a key index) is one given the u_t.  So the forward
// sweep and the adjoint sweep of Z_t = dL/dS_t,
//   Z_t = scale q_t do_t^T + a_{t+1} (Z_{t+1} - k_{t+1} dv_{t+1}^T),
//   X_t = Z_t^T k_t,  dv_t = beta_t X_t,  dbeta_t = X_t . e_t,
// run with columns spread over the grid and no exchange between blocks, and
//   dq_t = scale S_t do_t,   dk_t = Z_t u_t - a_t S_{t-1} dv_t
// come from sweeps with rows spread over the grid, all chunks of 64 tokens at
// once from the kept states and adjoints.  All sums are inside 8 or 16 lanes, no
// atomics, one order of addition.
//
// The decay's gradient dg_t = <a_t S_{t-1}, Z_t - k_t dv_t^T> is the sum of all
// that crosses token t, from writes before it (or the state S of the chunk's start)
// to reads at or after it (or the adjoint Z of the chunk's end).  With G_i the sum
// of the chunk's log decays up to i and D_ij = exp(G_i - G_j),
//   dg_t = sum over j < t <= i of M_ij + sum over i >= t of a_i
//          + sum over j < t of b_j + e^{G_64} <S, Z>,
//   M_ij = D_ij (scale (q_i.k_j) (do_i.u_j) - (k_i.k_j) (dv_i.u_j)),
//   a_i = e^{G_i} (scale (S^T q_i).do_i - (S^T k_i).dv_i),
//   b_j = e^{G_64 - G_j} (Z^T k_j).u_j
// (decay_grads_kernel).  Every term carries its own decay and nothing is
// subtracted, so that the gradient of a gate that is all but shut keeps its digits;
// dg_t - dg_{t+1} = o_t.do_t - v_t.dv_t, which costs nothing, would leave 2^-24 of
// o.do in it.
//
// Bound: the chain of a token in the column sweeps (product, sum over 8 lanes,
// update); the state stays in registers, two warps of a block bring the next
// tokens to shared memory while the others run these.
#include "s5_delta.cuh"

namespace s5 {
namespace delta {
namespace {

constexpr int TB = 16;        // tokens staged in shared memory (8 for heads above 128)
constexpr int OWN = 32;       // rows of a block
// Blocks of 8 columns up to which the column sweep uses them, against blocks of
// 32 (one read of the keys for four times the columns, but a fourth of the SMs
// when heads are few).  Forward, 400 tokens, 8 / 32 columns, us: 128 x 128 heads,
// 77 / 119 at 64 blocks, 103 / 120 at 256, 204 / 120 at 512; 64 x 64, 66 / 82 at
// 64, 81 / 83 at 256, 92 / 83 at 512.
constexpr int NARROW_BLOCKS = 256;
constexpr int SWT = 128;      // threads of a sweep
// Heads (B Hv) from which on a step takes a block for each, against a block for
// 32 columns: 3.8 / 4.5 us at 96 heads of 128 x 128, 3.7 / 3.2 at 64, 63 / 77 for
// 96 sequences of 32 heads (6.4 TB/s).
constexpr int HEAD_BLOCKS = 80;

// The sum over the 8 lanes that hold one column (lane bits 2 to 4).
__device__ __forceinline__ float column_sum(float v) {
    v += __shfl_xor_sync(0xffffffffu, v, 4);
    v += __shfl_xor_sync(0xffffffffu, v, 8);
    v += __shfl_xor_sync(0xffffffffu, v, 16);
    return v;
}
// Sums of four values over 16 lanes; lane l gets the sum of value l / 4 % 4.
__device__ __forceinline__ float sum4_16(const float (&v)[4], int lane) {
    const bool up = lane & 8, up2 = lane & 4;
    float a = up ? v[2] : v[0], b = up ? v[3] : v[1];
    a += __shfl_xor_sync(0xffffffffu, up ? v[0] : v[2], 8);
    b += __shfl_xor_sync(0xffffffffu, up ? v[1] : v[3], 8);
    float c = up2 ? b : a;
    c += __shfl_xor_sync(0xffffffffu, up2 ? a : b, 4);
    c += __shfl_xor_sync(0xffffffffu, c, 2);
    c += __shfl_xor_sync(0xffffffffu, c, 1);
    return c;
}

template <typename T> __device__ __forceinline__ float elem(const void *p, long long i) {
    return load_elem<T>(static_cast<const T *>(p) + i);
}

// Columns over the grid.  REV false: the forward recurrence, writing o (and
// what the backward pass needs); REV true: the adjoint, writing X and the
// adjoint at each chunk's end.  A column is held by 8 lanes, rows 32 i + 4 lane +
// 0..3 (one 16-byte read of a key for four rows), a block has C columns; two more
// warps stage the tokens.  Bound by the chain from token to token (smem read,
// products, three shuffles, update): 0.17 us a token forward, 0.11 back at heads of
// 64 x 64, whatever their number while the blocks fit the SMs.
template <typename T, int RPT, int C, bool REV>
__global__ void __launch_bounds__(8 * C + 64) column_sweep_kernel(const Args a) {
    constexpr int COLT = 8 * C;
    constexpr int NT = RPT > 16 ? TB / 2 : TB, D = 8 * RPT;
    __shared__ __align__(16) float sq[2][NT][D], sk[2][NT][D];
    __shared__ float sv[2][NT][C], sa[2][NT], sb[2][NT];
    const int lane = threadIdx.x / 4 % 8, own = threadIdx.x / 32 * 4 + threadIdx.x % 4;   // row lane, column
    const bool loads = threadIdx.x >= COLT;
    const int h = blockIdx.y, b = blockIdx.z, hk = h / (a.Hv / a.Hk);
    const int col = blockIdx.x * C + own;
    const bool on = !loads && col < a.Dv, first = on && lane == 0;
    const int N = chunks(a.L);
    const long long bh = (long long)b * a.Hv + h, mat = (long long)a.Dk * a.Dv;
    griddep_wait();
    const float *init = REV ? a.ds_last : a.s0;
    float S[RPT];
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
        const int r = 32 * (i / 4) + 4 * lane + i % 4;
        S[i] = (init && on && r < a.Dk) ? init[bh * mat + (long long)r * a.Dv + col] : 0.0f;
    }
    auto keep = [&](float *to) {
#pragma unroll
        for (int i = 0; i < RPT; ++i) {
            const int r = 32 * (i / 4) + 4 * lane + i % 4;
            if (on && r < a.Dk) to[(long long)r * a.Dv + col] = S[i];
        }
    };
    const int stages = (a.L + NT - 1) / NT;
    // Staging by 64 threads, a column of values each: `fetch` has all of a
    // stage's loads in flight, `put` writes them a stage later.
    const int tid = threadIdx.x - COLT, own_v = tid % C, first_t = tid / C;
    constexpr int PER = D / 64, TS = 64 / C;   // tokens a pass of values
    float fq[PER][NT], fk[PER][NT], fv[NT / TS], fg = 0.0f, fb = 0.0f;
    auto fetch = [&](int st) {
        const int t0 = (REV ? stages - 1 - st : st) * NT, nt = min(NT, a.L - t0);
        const long long row0 = (long long)b * a.L + t0;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int r = tid + 64 * i;
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const bool in = t < nt && r < a.Dk;
                fq[i][t] = in ? elem<T>(a.q, (row0 + t) * a.ldq + hk * a.Dk + r) : 0.0f;
                fk[i][t] = in ? elem<T>(a.k, (row0 + t) * a.ldk + hk * a.Dk + r) : 0.0f;
            }
        }
        const int v = blockIdx.x * C + own_v;
#pragma unroll
        for (int i = 0; i < NT / TS; ++i) {
            const int t = TS * i + first_t;
            const bool in = t < nt && v < a.Dv;
            fv[i] = !in   ? 0.0f
                    : REV ? elem<T>(a.dout, (row0 + t) * a.lddo + (long long)h * a.Dv + v)
                          : elem<T>(a.v, (row0 + t) * a.ldv + (long long)h * a.Dv + v);
        }
        if (tid < nt) fg = a.g[(row0 + tid) * a.Hv + h], fb = a.beta[(row0 + tid) * a.Hv + h];
    };
    auto put = [&](int buf) {
#pragma unroll
        for (int i = 0; i < PER; ++i)
#pragma unroll
            for (int t = 0; t < NT; ++t) sq[buf][t][tid + 64 * i] = a.scale * fq[i][t], sk[buf][t][tid + 64 * i] = fk[i][t];
#pragma unroll
        for (int i = 0; i < NT / TS; ++i) sv[buf][TS * i + first_t][own_v] = fv[i];
        if (tid < NT) sa[buf][tid] = expf(clamp_g(fg)), sb[buf][tid] = fb;
    };
    if (loads && stages > 0) {
        fetch(0), put(0);
        if (stages > 1) fetch(1);
    }
    __syncthreads();
    for (int st = 0; st < stages; ++st) {
        const int buf = st & 1;
        if (loads) {
            if (st + 1 < stages) put(buf ^ 1);
            if (st + 2 < stages) fetch(st + 2);
            __syncthreads();
            continue;
        }
        const int t0 = (REV ? stages - 1 - st : st) * NT, nt = min(NT, a.L - t0);
        const long long row0 = (long long)b * a.L + t0;
        float *const ke = a.e ? a.e + (row0 * a.Hv + h) * a.Dv + col : nullptr;
        // a stage lies within a chunk
        if (!REV && a.states && t0 % CHUNK == 0) keep(a.states + (bh * (N + 1) + t0 / CHUNK) * mat);
        if (REV && ((t0 + nt) % CHUNK == 0 || t0 + nt == a.L)) keep(static_cast<float *>(a.z) + (bh * N + t0 / CHUNK) * mat);
#pragma unroll 4
        for (int j = 0; j < nt; ++j) {
            const int t = REV ? nt - 1 - j : j;
            const long long out = ((row0 + t) * a.Hv + h) * a.Dv + col;
            const float4 *kt = reinterpret_cast<const float4 *>(sk[buf][t]) + lane, *qt = reinterpret_cast<const float4 *>(sq[buf][t]) + lane;
            const float al = sa[buf][t], be = sb[buf][t], x = sv[buf][t][own];
            float p[4] = {0, 0, 0, 0};   // four sums: a short chain
            if (!REV) {
                float y[4] = {0, 0, 0, 0}, z[4] = {0, 0, 0, 0};
#pragma unroll
                for (int i = 0; i < RPT / 4; ++i) {
                    const float4 k = kt[8 * i], q = qt[8 * i];
                    p[0] = fmaf(S[4 * i], k.x, p[0]), p[1] = fmaf(S[4 * i + 1], k.y, p[1]);
                    p[2] = fmaf(S[4 * i + 2], k.z, p[2]), p[3] = fmaf(S[4 * i + 3], k.w, p[3]);
                    y[0] = fmaf(S[4 * i], q.x, y[0]), y[1] = fmaf(S[4 * i + 1], q.y, y[1]);
                    y[2] = fmaf(S[4 * i + 2], q.z, y[2]), y[3] = fmaf(S[4 * i + 3], q.w, y[3]);
                    z[0] = fmaf(k.x, q.x, z[0]), z[1] = fmaf(k.y, q.y, z[1]);
                    z[2] = fmaf(k.z, q.z, z[2]), z[3] = fmaf(k.w, q.w, z[3]);
                }
                // o = a S^T q + u (k . q) from the state before: its sums run
                // beside e's instead of after them
                float sk = (p[0] + p[1]) + (p[2] + p[3]), sq = (y[0] + y[1]) + (y[2] + y[3]), kq = (z[0] + z[1]) + (z[2] + z[3]);
#pragma unroll
                for (int m = 16; m > 2; m >>= 1) {   // the column's 8 lanes
                    const float x0 = __shfl_xor_sync(0xffffffffu, sk, m), x1 = __shfl_xor_sync(0xffffffffu, sq, m),
                                x2 = __shfl_xor_sync(0xffffffffu, kq, m);
                    sk += x0, sq += x1, kq += x2;
                }
                const float e = fmaf(-al, sk, x), u = be * e, o = fmaf(u, kq, al * sq);
#pragma unroll
                for (int i = 0; i < RPT / 4; ++i) {
                    const float4 k = kt[8 * i];
                    S[4 * i] = fmaf(k.x, u, al * S[4 * i]), S[4 * i + 1] = fmaf(k.y, u, al * S[4 * i + 1]);
                    S[4 * i + 2] = fmaf(k.z, u, al * S[4 * i + 2]), S[4 * i + 3] = fmaf(k.w, u, al * S[4 * i + 3]);
                }
                if (first) {
                    store_elem<T>(static_cast<T *>(a.o) + (row0 + t) * a.ldo + (long long)h * a.Dv + col, o);
                    if (ke) ke[(long long)t * a.Hv * a.Dv] = e;
                }
            } else {
#pragma unroll
                for (int i = 0; i < RPT / 4; ++i) {
                    const float4 k = kt[8 * i], q = qt[8 * i];
                    S[4 * i] = fmaf(q.x, x, S[4 * i]), S[4 * i + 1] = fmaf(q.y, x, S[4 * i + 1]);
                    S[4 * i + 2] = fmaf(q.z, x, S[4 * i + 2]), S[4 * i + 3] = fmaf(q.w, x, S[4 * i + 3]);
                    p[0] = fmaf(S[4 * i], k.x, p[0]), p[1] = fmaf(S[4 * i + 1], k.y, p[1]);
                    p[2] = fmaf(S[4 * i + 2], k.z, p[2]), p[3] = fmaf(S[4 * i + 3], k.w, p[3]);
                }
                const float X = column_sum((p[0] + p[1]) + (p[2] + p[3])), u = be * X;
                if (first) a.x[out] = X;
#pragma unroll
                for (int i = 0; i < RPT / 4; ++i) {
                    const float4 k = kt[8 * i];
                    S[4 * i] = al * fmaf(-k.x, u, S[4 * i]), S[4 * i + 1] = al * fmaf(-k.y, u, S[4 * i + 1]);
                    S[4 * i + 2] = al * fmaf(-k.z, u, S[4 * i + 2]), S[4 * i + 3] = al * fmaf(-k.w, u, S[4 * i + 3]);
                }
            }
        }
        __syncthreads();
    }
    if (loads) return;
    float *last = REV ? a.ds0 : a.s_last;
    if (last) keep(last + bh * mat);
    if (!REV && a.states) keep(a.states + (bh * (N + 1) + N) * mat);
}

// Rows and chunks over the grid, with u_t = beta_t e_t and dv_t = beta_t X_t
// known: half of a block runs forward from the chunk's kept state for dq_t and
// a_t S_{t-1} dv_t, the other half back from its kept adjoint for Z_t u_t; their
// difference is dk_t.  Bound by the chain of a token, 64 of them per half: 2 x 500
// tokens of 4 heads of 64 x 64 in 24 us (38 with one half after the other).  Two
// blocks an SM up to 128 columns: 512 tokens of 16 heads of 128 in 100 us, 135 with one.
template <int RPT> struct RowSmem {
    static constexpr int NT = RPT > 8 ? TB / 2 : TB;
    float e[2][NT][16 * RPT], x[2][NT][16 * RPT], d[2][NT][16 * RPT], q[2][NT][OWN], k[2][NT][OWN], a[2][NT];
    float dk[2][CHUNK][OWN];
};
template <typename T, int RPT>
__global__ void __launch_bounds__(2 * SWT, RPT > 8 ? 1 : 2) row_sweep_kernel(const Args a) {
    constexpr int NT = RowSmem<RPT>::NT;
    extern __shared__ __align__(16) unsigned char raw[];
    RowSmem<RPT> &sm = *reinterpret_cast<RowSmem<RPT> *>(raw);
    const bool back = threadIdx.x >= SWT;
    const int tid = threadIdx.x % SWT;
    auto &se = sm.e[back], &sx = sm.x[back], &sd = sm.d[back];
    auto &sq = sm.q[back], &sk = sm.k[back];
    auto &dk = sm.dk[back];
    auto &sa = sm.a[back];
    auto meet = [&] { asm volatile("bar.sync %0, %1;" ::"r"(1 + (int)back), "n"(SWT) : "memory"); };
    const int lane = tid % 16, grp = tid / 16;
    const int rows = (a.Dk + OWN - 1) / OWN, c = blockIdx.x / rows, r0 = blockIdx.x % rows * OWN;
    const int h = blockIdx.y, b = blockIdx.z, hk = h / (a.Hv / a.Hk);
    const int row = r0 + grp * 4, mine = lane / 4;
    const bool on = row < a.Dk;
    const int N = chunks(a.L), first = c * CHUNK, len = min(CHUNK, a.L - first), stages = (len + NT - 1) / NT;
    const long long bh = (long long)b * a.Hv + h, mat = (long long)a.Dk * a.Dv;
    griddep_wait();
    float S[RPT][4];
    auto load = [&](const float *from) {
#pragma unroll
        for (int i = 0; i < RPT; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                S[i][r] = (on && lane + 16 * i < a.Dv) ? from[(long long)(row + r) * a.Dv + lane + 16 * i] : 0.0f;
    };
    auto stage = [&](int t0, int nt) {
        const long long row0 = (long long)b * a.L + t0;
        meet();
        constexpr int DV = 16 * RPT, PER = NT * DV / SWT;   // a thread's values of each array, all in flight
        {
            float x[PER], y[PER], d[PER], be[PER];
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const int at = tid + i * SWT, t = at / DV, v = at % DV;
                const bool in = t < nt && v < a.Dv;
                const long long hv = (row0 + t) * a.Hv + h;
                be[i] = in ? a.beta[hv] : 0.0f;
                x[i] = in ? a.e[hv * a.Dv + v] : 0.0f;
                y[i] = in ? a.x[hv * a.Dv + v] : 0.0f;
                d[i] = in ? elem<T>(a.dout, (row0 + t) * a.lddo + (long long)h * a.Dv + v) : 0.0f;
            }
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const int at = tid + i * SWT, t = at / DV, v = at % DV;
                se[t][v] = be[i] * x[i], sx[t][v] = be[i] * y[i], sd[t][v] = a.scale * d[i];
            }
        }
#pragma unroll
        for (int i = 0; i < NT * OWN / SWT; ++i) {
            const int at = tid + i * SWT, t = at / OWN, r = r0 + at % OWN;
            const bool in = t < nt && r < a.Dk;
            sq[t][at % OWN] = in ? elem<T>(a.q, (row0 + t) * a.ldq + hk * a.Dk + r) : 0.0f;
            sk[t][at % OWN] = in ? elem<T>(a.k, (row0 + t) * a.ldk + hk * a.Dk + r) : 0.0f;
        }
        if (tid < nt) sa[tid] = expf(clamp_g(a.g[(row0 + tid) * a.Hv + h]));
        meet();
    };
    if (!back) {
        load(a.states + (bh * (N + 1) + c) * mat);
        for (int st = 0; st < stages; ++st) {
            const int t0 = first + st * NT, nt = min(NT, first + len - t0);
            stage(t0, nt);
            for (int t = 0; t < nt; ++t) {
                const float al = sa[t];
                float p[4] = {0, 0, 0, 0}, w[4] = {0, 0, 0, 0};
#pragma unroll
                for (int i = 0; i < RPT; ++i) {
                    const float e = se[t][lane + 16 * i], x = sx[t][lane + 16 * i], d = sd[t][lane + 16 * i];
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        S[i][r] *= al;
                        p[r] = fmaf(S[i][r], x, p[r]);
                        S[i][r] = fmaf(sk[t][grp * 4 + r], e, S[i][r]);
                        w[r] = fmaf(S[i][r], d, w[r]);
                    }
                }
                const float v = sum4_16(p, lane), dq = sum4_16(w, lane);
                if (lane % 4 == 0) {
                    dk[t0 - first + t][grp * 4 + mine] = v;
                    if (on) a.dqh[(((long long)b * a.L + t0 + t) * a.Hv + h) * a.Dk + row + mine] = dq;
                }
            }
        }
    } else {
        load(static_cast<const float *>(a.z) + (bh * N + c) * mat);
        for (int st = stages - 1; st >= 0; --st) {
            const int t0 = first + st * NT, nt = min(NT, first + len - t0);
            stage(t0, nt);
            for (int t = nt - 1; t >= 0; --t) {
                const float al = sa[t];
                float p[4] = {0, 0, 0, 0};
#pragma unroll
                for (int i = 0; i < RPT; ++i) {
                    const float e = se[t][lane + 16 * i], x = sx[t][lane + 16 * i], d = sd[t][lane + 16 * i];
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        S[i][r] = fmaf(sq[t][grp * 4 + r], d, S[i][r]);
                        p[r] = fmaf(S[i][r], e, p[r]);
                        S[i][r] = al * fmaf(-sk[t][grp * 4 + r], x, S[i][r]);
                    }
                }
                const float v = sum4_16(p, lane);
                if (lane % 4 == 0) dk[t0 - first + t][grp * 4 + mine] = v;
            }
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < len * OWN; i += 2 * SWT) {
        const int t = i / OWN, r = i % OWN;
        if (r0 + r < a.Dk)
            a.dkh[(((long long)b * a.L + first + t) * a.Hv + h) * a.Dk + r0 + r] = sm.dk[1][t][r] - sm.dk[0][t][r];
    }
}

// dg of a chunk and value head (the formula is at the top of this file), in
// decay_parts parts that token_grads_kernel adds up: part 0 is M's, the others are
// that of a, b and <S, Z> over 64 columns of the state each.  A part is a block of
// its own: products of 64 x 64 tiles (four rows and columns a thread, slices of 16 of
// the depth staged in shared memory, the next slice on its way).  M's rows are then
// summed along j, its columns along i, both from nothing, so that no term is taken
// away again.  Bound by the products, in 32 bits on the CUDA cores as all of this path:
// 2 x 500 tokens of 4 heads of 64 x 64 in 13 us (22 with one block a chunk and single
// loads), 512 of 16 heads of 128 in 48; with 256 tokens of 4 heads of 256 the whole
// call took 343 us with one block a chunk, 231 now.
constexpr int GT = 256, GS = 16, GP = 68;
int decay_parts(int Dv) { return 1 + (Dv + 63) / 64; }

// Four consecutive values from p on; vec: p is aligned for one load.
template <typename T> __device__ __forceinline__ float4 four(const T *p, bool vec) {
    if constexpr (sizeof(T) == 4) {
        if (vec) return *reinterpret_cast<const float4 *>(p);
    } else if (vec) {
        const uint2 v = *reinterpret_cast<const uint2 *>(p);
        return make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u), __uint_as_float(v.y << 16),
                           __uint_as_float(v.y & 0xffff0000u));
    }
    return make_float4(load_elem<T>(p), load_elem<T>(p + 1), load_elem<T>(p + 2), load_elem<T>(p + 3));
}

template <typename T> __global__ void __launch_bounds__(GT, 2) decay_grads_kernel(const Args a, int parts) {
    __shared__ __align__(16) float st[4][GS][GP];
    __shared__ float hi[CHUNK], lo[CHUNK], av[CHUNK], bv[CHUNK], mv[GT / 32];
    constexpr int MP = CHUNK + 1;
    float *M = &st[0][0][0];   // [64][MP], in the place of the tiles
    static_assert(CHUNK * MP <= 4 * GS * GP, "M fits");
    const int c = blockIdx.x / parts, part = blockIdx.x % parts, h = blockIdx.y, b = blockIdx.z, hk = h / (a.Hv / a.Hk);
    const int tid = threadIdx.x, ti = tid / 16 * 4, tj = tid % 16 * 4;
    const int N = chunks(a.L), t0 = c * CHUNK, nt = min(CHUNK, a.L - t0);
    const long long row0 = (long long)b * a.L + t0, bh = (long long)b * a.Hv + h, mat = (long long)a.Dk * a.Dv;
    griddep_wait();
    if (tid < 32) {
        float G[2], g[2];
        decay_sums(a, row0, nt, h, tid, G, g);
#pragma unroll
        for (int i = 0; i < 2; ++i) hi[2 * tid + i] = G[i], lo[2 * tid + i] = g[i];
    }
    // a slice of 64 tokens x 16 values: this thread's token, and the first of its four values
    const int mt = tid / 4, md = tid % 4 * 4;
    const bool live = mt < nt;
    const float4 zero = make_float4(0, 0, 0, 0);
    const long long row = row0 + (live ? mt : 0), hv = row * a.Hv + h;
    const T *k0 = static_cast<const T *>(a.k) + row * a.ldk + hk * a.Dk + md, *q0 = static_cast<const T *>(a.q) + row * a.ldq + hk * a.Dk + md;
    const T *o0 = static_cast<const T *>(a.dout) + row * a.lddo + (long long)h * a.Dv + md;
    const float *x0 = a.x + hv * a.Dv + md, *e0 = a.e + hv * a.Dv + md;
    const bool vk = a.ldk % 4 == 0, vq = a.ldq % 4 == 0, vo = a.lddo % 4 == 0;
    auto stage = [&](int j, float4 v) { st[j][md][mt] = v.x, st[j][md + 1][mt] = v.y, st[j][md + 2][mt] = v.z, st[j][md + 3][mt] = v.w; };
    auto times = [](float4 v, float f) { return make_float4(v.x * f, v.y * f, v.z * f, v.w * f); };
    auto row4 = [&](int j, int d, int at, float (&r)[4]) {
        const float4 v = *reinterpret_cast<const float4 *>(&st[j][d][at]);
        r[0] = v.x, r[1] = v.y, r[2] = v.z, r[3] = v.w;
    };
    float *out = a.writes + ((long long)part * a.B * a.L + row0) * a.Hv + h;   // [part][B][L][Hv]
    const int ks = (a.Dk + GS - 1) / GS;
    if (part == 0) {
        float kk[4][4] = {}, qk[4][4] = {}, du[4][4] = {}, ou[4][4] = {};
        const float be = live ? a.beta[hv] : 0.0f;
        float4 x[3];
        // first all products along the keys, then all along the values
        const int all = ks + (a.Dv + GS - 1) / GS;
        auto fetch = [&](int s) {
            const int d = (s < ks ? s : s - ks) * GS;
            const bool in = live && d + md < (s < ks ? a.Dk : a.Dv);
            x[0] = x[1] = x[2] = zero;
            if (!in) return;
            if (s < ks)
                x[0] = four<T>(k0 + d, vk), x[1] = four<T>(q0 + d, vq);
            else
                x[0] = four<float>(x0 + d, true), x[1] = four<T>(o0 + d, vo), x[2] = four<float>(e0 + d, true);
        };
        fetch(0);
        for (int s = 0; s < all; ++s) {
            __syncthreads();
            if (s < ks)
                stage(0, x[0]), stage(1, x[1]);
            else
                stage(0, times(x[0], be)), stage(1, x[1]), stage(2, times(x[2], be));
            __syncthreads();
            if (s + 1 < all) fetch(s + 1);
            auto add = [&](float (&p)[4][4], float (&r)[4][4], int w) {
#pragma unroll 4
                for (int d = 0; d < GS; ++d) {
                    float u[4], v[4], y[4];
                    row4(0, d, ti, u), row4(1, d, ti, v), row4(w, d, tj, y);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int j = 0; j < 4; ++j) p[i][j] = fmaf(u[i], y[j], p[i][j]), r[i][j] = fmaf(v[i], y[j], r[i][j]);
                }
            };
            if (s < ks)
                add(kk, qk, 0);
            else
                add(du, ou, 2);
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int r = ti + i, q = tj + j;
                const float d = expf((hi[r] - hi[q]) + (lo[r] - lo[q]));
                M[r * MP + q] = q < r ? d * (a.scale * qk[i][j] * ou[i][j] - kk[i][j] * du[i][j]) : 0.0f;
            }
        __syncthreads();
        // M_it becomes the sum of M_ij over j < t, a row a thread
        if (tid < CHUNK) {
            float w = 0.0f;
#pragma unroll 16
            for (int j = 0; j < CHUNK; ++j) {
                const float v = M[tid * MP + j];
                M[tid * MP + j] = w;
                w += v;
            }
        }
        __syncthreads();
        if (tid < nt) {
            float w = 0.0f;
#pragma unroll 8
            for (int i = 0; i < CHUNK; ++i) w += i >= tid ? M[i * MP + tid] : 0.0f;
            out[(long long)tid * a.Hv] = w;
        }
        return;
    }
    const int v0 = (part - 1) * 64;
    float m = 0.0f, ks4[4][4] = {}, qs4[4][4] = {}, kz4[4][4] = {};
    float4 x[4];
    // a slice of 16 x 64 of the state and its adjoint: this thread's row and first column
    const int sr = tid / 16, sv = v0 + tid % 16 * 4;
    const long long at = (long long)sr * a.Dv + sv;
    const float *S = a.states + (bh * (N + 1) + c) * mat + at, *Z = static_cast<const float *>(a.z) + (bh * N + c) * mat + at;
    auto fetch = [&](int s) {
        const int d = s * GS;
        x[0] = x[1] = x[2] = x[3] = zero;
        if (live && d + md < a.Dk) x[0] = four<T>(k0 + d, vk), x[1] = four<T>(q0 + d, vq);
        if (d + sr < a.Dk && sv < a.Dv) {
            x[2] = four<float>(S + (long long)d * a.Dv, true);
            x[3] = four<float>(Z + (long long)d * a.Dv, true);
        }
    };
    fetch(0);
    for (int s = 0; s < ks; ++s) {
        __syncthreads();
        stage(0, x[0]), stage(1, x[1]);
        *reinterpret_cast<float4 *>(&st[2][sr][tid % 16 * 4]) = x[2];
        *reinterpret_cast<float4 *>(&st[3][sr][tid % 16 * 4]) = x[3];
        m = fmaf(x[2].x, x[3].x, fmaf(x[2].y, x[3].y, fmaf(x[2].z, x[3].z, fmaf(x[2].w, x[3].w, m))));
        __syncthreads();
        if (s + 1 < ks) fetch(s + 1);
#pragma unroll 4
        for (int d = 0; d < GS; ++d) {
            float u[4], v[4], y[4], z[4];
            row4(0, d, ti, u), row4(1, d, ti, v), row4(2, d, tj, y), row4(3, d, tj, z);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    ks4[i][j] = fmaf(u[i], y[j], ks4[i][j]), qs4[i][j] = fmaf(v[i], y[j], qs4[i][j]);
                    kz4[i][j] = fmaf(u[i], z[j], kz4[i][j]);
                }
        }
    }
    // this thread's four tokens and columns
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int t = ti + i, v = v0 + tj;
        float aw = 0.0f, bw = 0.0f;
        if (t < nt && v < a.Dv) {
            const long long r = row0 + t, rh = r * a.Hv + h;
            const float be = a.beta[rh];
            const float4 o = four<T>(static_cast<const T *>(a.dout) + r * a.lddo + (long long)h * a.Dv + v, vo);
            const float4 dv = times(four<float>(a.x + rh * a.Dv + v, true), be), w = times(four<float>(a.e + rh * a.Dv + v, true), be);
            const float o4[4] = {o.x, o.y, o.z, o.w}, d4[4] = {dv.x, dv.y, dv.z, dv.w}, w4[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                aw = fmaf(a.scale * qs4[i][j], o4[j], fmaf(-ks4[i][j], d4[j], aw));
                bw = fmaf(kz4[i][j], w4[j], bw);
            }
        }
#pragma unroll
        for (int w = 1; w < 16; w <<= 1) {
            aw += __shfl_xor_sync(0xffffffffu, aw, w);
            bw += __shfl_xor_sync(0xffffffffu, bw, w);
        }
        if (tid % 16 == 0) {
            av[t] = expf(hi[t]) * aw;
            bv[t] = expf((hi[CHUNK - 1] - hi[t]) + (lo[CHUNK - 1] - lo[t])) * bw;
        }
    }
    m = warp_sum(m);
    if (tid % 32 == 0) mv[tid / 32] = m;
    __syncthreads();
    if (tid < nt) {
        float x = 0.0f, y = 0.0f;
        m = 0.0f;
#pragma unroll
        for (int i = 0; i < GT / 32; ++i) m += mv[i];
#pragma unroll 8
        for (int i = 0; i < CHUNK; ++i) x += i >= tid ? av[i] : 0.0f, y += i < tid ? bv[i] : 0.0f;
        out[(long long)tid * a.Hv] = fmaf(expf(hi[CHUNK - 1]), m, x + y);
    }
}

// One warp per token and value head: dv = beta X, dbeta = X . e, dg from its parts.
template <typename T> __global__ void __launch_bounds__(256) token_grads_kernel(const Args a, int parts) {
    griddep_wait();
    const long long hv = (long long)blockIdx.x * 8 + threadIdx.x / 32, rows = (long long)a.B * a.L * a.Hv;
    const int lane = threadIdx.x % 32;
    if (hv >= rows) return;
    const long long row = hv / a.Hv;
    const int h = (int)(hv % a.Hv);
    const float be = a.beta[hv], dg = warp_sum(lane < parts ? a.writes[lane * rows + hv] : 0.0f);
    float db = 0.0f;
    for (int c = lane; c < a.Dv; c += 32) {
        const float x = a.x[hv * a.Dv + c];
        db = fmaf(x, a.e[hv * a.Dv + c], db);
        store_elem<T>(static_cast<T *>(a.dv) + row * a.lddv + (long long)h * a.Dv + c, be * x);
    }
    db = warp_sum(db);
    if (lane == 0) a.dbeta[hv] = db, a.dg[hv] = dg;
}

// dq and dk of a key head: the sum over its value heads, rounded once.
template <typename T> __global__ void __launch_bounds__(256) group_sum_kernel(const Args a) {
    griddep_wait();
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x, n = (long long)a.B * a.L * a.Hk * a.Dk;
    if (i >= n) return;
    const int d = (int)(i % a.Dk), hk = (int)(i / a.Dk % a.Hk), group = a.Hv / a.Hk;
    const long long row = i / ((long long)a.Dk * a.Hk);
    float q = 0.0f, k = 0.0f;
    for (int j = 0; j < group; ++j) {
        const long long at = (row * a.Hv + hk * group + j) * a.Dk + d;
        q += a.dqh[at], k += a.dkh[at];
    }
    store_elem<T>(static_cast<T *>(a.dq) + row * a.lddq + (long long)hk * a.Dk + d, q);
    store_elem<T>(static_cast<T *>(a.dk) + row * a.lddk + (long long)hk * a.Dk + d, k);
}

// ---------------------------------------------------------------------------
// One token.  The state is read and written once (the bound: its bytes), held
// in registers in between: a block takes 32 columns of one head, 8 lanes of
// four columns by 32 rows at a time.  Both sums over the rows, S^T k and
// S^T q, are taken of the old state, so that one exchange between the warps
// serves them:  o = scale (a S^T q + (q . k) u).
// ---------------------------------------------------------------------------
template <typename T, int RPT>
__global__ void __launch_bounds__(256) delta_step_kernel(const void *q, const void *k, const void *v, const float *g,
                                                         const float *beta, float scale, int Hk, int Hv, int Dk,
                                                         int Dv, float *state, void *o) {
    __shared__ float4 rk[8][8], rq[8][8];
    __shared__ float rd[8];
    const int cv = threadIdx.x % 8, rg = threadIdx.x / 8, warp = threadIdx.x / 32;
    const int col = blockIdx.x * 32 + cv * 4, h = blockIdx.y, b = blockIdx.z, hk = h / (Hv / Hk);
    const long long bh = (long long)b * Hv + h;
    const bool on = col < Dv;
    float *s = state + bh * (long long)Dk * Dv + col;
    const long long kb = ((long long)b * Hk + hk) * Dk;
    griddep_wait();
    griddep_launch_dependents();
    float4 S[RPT];
    float kk[RPT], qk = 0.0f;
    float4 pk = make_float4(0, 0, 0, 0), pq = pk;
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
        const int r = rg + 32 * i;
        S[i] = (on && r < Dk) ? *reinterpret_cast<const float4 *>(s + (long long)r * Dv) : make_float4(0, 0, 0, 0);
    }
    const float al = expf(clamp_g(g[bh])), be = beta[bh];
    float vv[4] = {0, 0, 0, 0};
    if (on)
#pragma unroll
        for (int c = 0; c < 4; ++c) vv[c] = elem<T>(v, bh * Dv + col + c);
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
        const int r = rg + 32 * i;
        kk[i] = r < Dk ? elem<T>(k, kb + r) : 0.0f;
        const float qq = r < Dk ? elem<T>(q, kb + r) : 0.0f;
        qk = fmaf(qq, kk[i], qk);
        pk.x = fmaf(S[i].x, kk[i], pk.x), pk.y = fmaf(S[i].y, kk[i], pk.y);
        pk.z = fmaf(S[i].z, kk[i], pk.z), pk.w = fmaf(S[i].w, kk[i], pk.w);
        pq.x = fmaf(S[i].x, qq, pq.x), pq.y = fmaf(S[i].y, qq, pq.y);
        pq.z = fmaf(S[i].z, qq, pq.z), pq.w = fmaf(S[i].w, qq, pq.w);
    }
#pragma unroll
    for (int m = 8; m < 32; m <<= 1) {
        pk.x += __shfl_xor_sync(0xffffffffu, pk.x, m), pk.y += __shfl_xor_sync(0xffffffffu, pk.y, m);
        pk.z += __shfl_xor_sync(0xffffffffu, pk.z, m), pk.w += __shfl_xor_sync(0xffffffffu, pk.w, m);
        pq.x += __shfl_xor_sync(0xffffffffu, pq.x, m), pq.y += __shfl_xor_sync(0xffffffffu, pq.y, m);
        pq.z += __shfl_xor_sync(0xffffffffu, pq.z, m), pq.w += __shfl_xor_sync(0xffffffffu, pq.w, m);
        qk += __shfl_xor_sync(0xffffffffu, qk, m);
    }
    if (threadIdx.x % 32 < 8) rk[warp][cv] = pk, rq[warp][cv] = pq;
    if (threadIdx.x % 32 == 0) rd[warp] = qk;
    __syncthreads();
    pk = pq = make_float4(0, 0, 0, 0), qk = 0.0f;
#pragma unroll
    for (int w = 0; w < 8; ++w) {
        const float4 x = rk[w][cv], y = rq[w][cv];
        pk.x += x.x, pk.y += x.y, pk.z += x.z, pk.w += x.w;
        pq.x += y.x, pq.y += y.y, pq.z += y.z, pq.w += y.w;
        qk += rd[w];
    }
    const float ux = be * (vv[0] - al * pk.x), uy = be * (vv[1] - al * pk.y), uz = be * (vv[2] - al * pk.z),
                uw = be * (vv[3] - al * pk.w);
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
        const int r = rg + 32 * i;
        if (on && r < Dk)
            *reinterpret_cast<float4 *>(s + (long long)r * Dv) =
                make_float4(fmaf(kk[i], ux, al * S[i].x), fmaf(kk[i], uy, al * S[i].y), fmaf(kk[i], uz, al * S[i].z),
                            fmaf(kk[i], uw, al * S[i].w));
    }
    if (on && rg == 0) {
        T *out = static_cast<T *>(o) + bh * Dv + col;
        store_elem<T>(out, scale * fmaf(al, pq.x, qk * ux));
        store_elem<T>(out + 1, scale * fmaf(al, pq.y, qk * uy));
        store_elem<T>(out + 2, scale * fmaf(al, pq.z, qk * uz));
        store_elem<T>(out + 3, scale * fmaf(al, pq.w, qk * uw));
    }
}

// The same for a whole head a block (heads up to 128 x 128): 256 threads hold
// the 64 KB of its state, LR lanes of four columns by 256 / LR rows at a time,
// read and written with streaming hints; 128 KB an SM in flight.  For few
// heads the blocks above spread the state over more SMs (launch rule).
template <typename T, int LR>
__global__ void __launch_bounds__(256, 2) delta_step_head_kernel(const void *q, const void *k, const void *v, const float *g,
                                                                 const float *beta, float scale, int Hk, int Hv, int Dk,
                                                                 int Dv, float *state, void *o) {
    constexpr int RG = 256 / LR, RPT = 128 / RG;
    __shared__ float4 rk[8][LR], rq[8][LR];
    __shared__ float rd[8];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, cv = lane % LR, rg = threadIdx.x / LR;
    const int col = cv * 4, h = blockIdx.x % Hv, b = blockIdx.x / Hv, hk = h / (Hv / Hk);
    const long long bh = blockIdx.x;
    const bool on = col < Dv;
    float *s = state + bh * (long long)Dk * Dv + col;
    const long long kb = ((long long)b * Hk + hk) * Dk;
    griddep_wait();
    griddep_launch_dependents();
    float4 S[RPT];
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
        const int r = rg + RG * i;
        S[i] = (on && r < Dk) ? __ldcs(reinterpret_cast<const float4 *>(s + (long long)r * Dv)) : make_float4(0, 0, 0, 0);
    }
    const float al = expf(clamp_g(g[bh])), be = beta[bh];
    float vv[4] = {0, 0, 0, 0};
    if (on)
#pragma unroll
        for (int c = 0; c < 4; ++c) vv[c] = elem<T>(v, bh * Dv + col + c);
    // lane c of a row group holds k and q of the group's row c (c < RPT)
    const int mine = rg + RG * cv;
    float kl = 0.0f, ql = 0.0f;
    if (cv < RPT && mine < Dk) kl = elem<T>(k, kb + mine), ql = elem<T>(q, kb + mine);
    float qk = kl * ql;
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) qk += __shfl_xor_sync(0xffffffffu, qk, m);
    float4 pk = make_float4(0, 0, 0, 0), pq = pk;
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
        const float kk = __shfl_sync(0xffffffffu, kl, i, LR), qq = __shfl_sync(0xffffffffu, ql, i, LR);
        pk.x = fmaf(S[i].x, kk, pk.x), pk.y = fmaf(S[i].y, kk, pk.y);
        pk.z = fmaf(S[i].z, kk, pk.z), pk.w = fmaf(S[i].w, kk, pk.w);
        pq.x = fmaf(S[i].x, qq, pq.x), pq.y = fmaf(S[i].y, qq, pq.y);
        pq.z = fmaf(S[i].z, qq, pq.z), pq.w = fmaf(S[i].w, qq, pq.w);
    }
    if (LR == 16) {
        pk.x += __shfl_xor_sync(0xffffffffu, pk.x, 16), pk.y += __shfl_xor_sync(0xffffffffu, pk.y, 16);
        pk.z += __shfl_xor_sync(0xffffffffu, pk.z, 16), pk.w += __shfl_xor_sync(0xffffffffu, pk.w, 16);
        pq.x += __shfl_xor_sync(0xffffffffu, pq.x, 16), pq.y += __shfl_xor_sync(0xffffffffu, pq.y, 16);
        pq.z += __shfl_xor_sync(0xffffffffu, pq.z, 16), pq.w += __shfl_xor_sync(0xffffffffu, pq.w, 16);
    }
    if (lane < LR) rk[warp][cv] = pk, rq[warp][cv] = pq;
    if (lane == 0) rd[warp] = qk;
    __syncthreads();
    pk = make_float4(0, 0, 0, 0);
#pragma unroll
    for (int w = 0; w < 8; ++w) {
        const float4 x = rk[w][cv];
        pk.x += x.x, pk.y += x.y, pk.z += x.z, pk.w += x.w;
    }
    const float ux = be * (vv[0] - al * pk.x), uy = be * (vv[1] - al * pk.y), uz = be * (vv[2] - al * pk.z),
                uw = be * (vv[3] - al * pk.w);
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
        const int r = rg + RG * i;
        const float kk = __shfl_sync(0xffffffffu, kl, i, LR);
        if (on && r < Dk)
            __stcs(reinterpret_cast<float4 *>(s + (long long)r * Dv),
                   make_float4(fmaf(kk, ux, al * S[i].x), fmaf(kk, uy, al * S[i].y), fmaf(kk, uz, al * S[i].z),
                               fmaf(kk, uw, al * S[i].w)));
    }
    if (on && threadIdx.x < LR) {
        pq = make_float4(0, 0, 0, 0), qk = 0.0f;
#pragma unroll
        for (int w = 0; w < 8; ++w) {
            const float4 y = rq[w][cv];
            pq.x += y.x, pq.y += y.y, pq.z += y.z, pq.w += y.w;
            qk += rd[w];
        }
        T *out = static_cast<T *>(o) + bh * Dv + col;
        store_elem<T>(out, scale * fmaf(al, pq.x, qk * ux));
        store_elem<T>(out + 1, scale * fmaf(al, pq.y, qk * uy));
        store_elem<T>(out + 2, scale * fmaf(al, pq.z, qk * uz));
        store_elem<T>(out + 3, scale * fmaf(al, pq.w, qk * uw));
    }
}

template <typename T>
cudaError_t step(const void *q, const void *k, const void *v, const float *g, const float *beta, float scale, int B, int Hk,
                 int Hv, int Dk, int Dv, float *state, void *o, cudaStream_t st) {
    cudaLaunchAttribute attr;
    set_programmatic(attr);
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(256);
    cfg.stream = st;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (Dk <= 128 && Dv <= 128 && (long long)B * Hv >= HEAD_BLOCKS) {
        cfg.gridDim = dim3(B * Hv);
        return Dv > 64 ? cudaLaunchKernelEx(&cfg, delta_step_head_kernel<T, 32>, q, k, v, g, beta, scale, Hk, Hv, Dk, Dv, state, o)
                       : cudaLaunchKernelEx(&cfg, delta_step_head_kernel<T, 16>, q, k, v, g, beta, scale, Hk, Hv, Dk, Dv, state, o);
    }
    cfg.gridDim = dim3((Dv + 31) / 32, Hv, B);
    return Dk > 128 ? cudaLaunchKernelEx(&cfg, delta_step_kernel<T, 8>, q, k, v, g, beta, scale, Hk, Hv, Dk, Dv, state, o)
                    : cudaLaunchKernelEx(&cfg, delta_step_kernel<T, 4>, q, k, v, g, beta, scale, Hk, Hv, Dk, Dv, state, o);
}

// Columns of a block of the column sweep.
int column_width(const Args &a) { return (long long)a.B * a.Hv * ((a.Dv + 7) / 8) <= NARROW_BLOCKS ? 8 : 32; }

template <typename T, int C, bool REV> cudaError_t column_sweep(const Args &a, cudaStream_t st) {
    const dim3 grid((a.Dv + C - 1) / C, a.Hv, a.B);
    auto *kernel = a.Dk <= 64 ? column_sweep_kernel<T, 8, C, REV>
                   : a.Dk <= 128 ? column_sweep_kernel<T, 16, C, REV> : column_sweep_kernel<T, 32, C, REV>;
    return launch_after(kernel, grid, 8 * C + 64, 0, st, a);
}
template <typename T, bool REV> cudaError_t column_sweep(const Args &a, cudaStream_t st) {
    return column_width(a) == 8 ? column_sweep<T, 8, REV>(a, st) : column_sweep<T, 32, REV>(a, st);
}
template <typename T, int RPT> cudaError_t row_sweep(const Args &a, cudaStream_t st) {
    const dim3 grid((a.Dk + OWN - 1) / OWN * chunks(a.L), a.Hv, a.B);
    constexpr int bytes = sizeof(RowSmem<RPT>);
    const cudaError_t e = cudaFuncSetAttribute(row_sweep_kernel<T, RPT>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    return launch_after(row_sweep_kernel<T, RPT>, grid, 2 * SWT, bytes, st, a);
}
template <typename T> cudaError_t row_sweep(const Args &a, cudaStream_t st) {
    return a.Dv <= 64 ? row_sweep<T, 4>(a, st) : a.Dv <= 128 ? row_sweep<T, 8>(a, st) : row_sweep<T, 16>(a, st);
}

template <typename T> cudaError_t backward(const Args &a, cudaStream_t st) {
    cudaError_t e = column_sweep<T, true>(a, st);
    if (e != cudaSuccess || a.L == 0) return e;
    if ((e = row_sweep<T>(a, st)) != cudaSuccess) return e;
    const long long rows = (long long)a.B * a.L * a.Hv, n = (long long)a.B * a.L * a.Hk * a.Dk;
    const int parts = decay_parts(a.Dv);
    if ((e = launch_after(decay_grads_kernel<T>, dim3(chunks(a.L) * parts, a.Hv, a.B), GT, 0, st, a, parts)) != cudaSuccess) return e;
    if ((e = launch_after(token_grads_kernel<T>, (unsigned)((rows + 7) / 8), 256, 0, st, a, parts)) != cudaSuccess) return e;
    return launch_after(group_sum_kernel<T>, (unsigned)((n + 255) / 256), 256, 0, st, a);
}

bool aligned16(const void *p) { return p && (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool floats(const void *p) { return p && (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }   // read one by one
bool aligned16_or_null(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Sizes that every entry point takes; offsets are 64-bit, launches 32-bit.
s5_status check_sizes(long long B, long long L, long long Hk, long long Hv, long long Dk, long long Dv, s5_dtype dtype) {
    if (dtype != S5_F32 && dtype != S5_BF16) return S5_ERR_INVALID_ARGUMENT;
    if (B < 0 || L < 0 || Hk < 1 || Hv < 1 || Dk < 1 || Dv < 1 || Hv % Hk) return S5_ERR_INVALID_ARGUMENT;
    if (Dk % 4 || Dv % 4 || Dk > 256 || Dv > 256 || B > 65535 || Hv > 65535) return S5_ERR_UNSUPPORTED;
    if (B * Hv > (1ll << 24) || L > (1ll << 30) || B * L * Hv > (1ll << 30)) return S5_ERR_UNSUPPORTED;
    return S5_OK;
}

// Regions of the two buffers.  The backward workspace holds what either path
// needs: dq and dk per value head, the chunks' Z (as many bytes in either form,
// one less than the states), parts of the decays' gradients.
struct Sizes {
    size_t e, states, images, heads, inner, writes;
};
Sizes sizes(int B, int L, int Hv, int Dk, int Dv) {
    Sizes s;
    const size_t rows = (size_t)B * L * Hv, N = chunks(L);
    s.e = align256(sizeof(float) * rows * Dv);
    s.states = align256(sizeof(float) * (size_t)B * Hv * (N + 1) * Dk * Dv);
    s.images = align256(tc_image_bytes(B, L, Hv, Dk, Dv));
    s.heads = align256(sizeof(float) * rows * Dk);
    s.inner = s.images ? align256(sizeof(float) * (size_t)B * Hv * N * inner_parts(Dk, Dv)) : 0;
    const size_t tc = s.images ? (size_t)B * Hv * N * CHUNK * write_parts(Dv) : 0, simt = rows * decay_parts(Dv);
    s.writes = align256(sizeof(float) * (tc > simt ? tc : simt));
    return s;
}
}  // namespace
}  // namespace delta
}  // namespace s5

using namespace s5;
using namespace s5::delta;

extern "C" size_t s5_delta_saved_size(int B, int L, int Hv, int Dk, int Dv) {
    if (check_sizes(B, L, Hv, Hv, Dk, Dv, S5_F32) != S5_OK) return 0;
    const Sizes s = sizes(B, L, Hv, Dk, Dv);
    return 2 * s.e + s.states + 256;
}

extern "C" size_t s5_delta_workspace_size(int B, int L, int Hv, int Dk, int Dv, int backward) {
    if (check_sizes(B, L, Hv, Hv, Dk, Dv, S5_F32) != S5_OK) return 0;
    const Sizes s = sizes(B, L, Hv, Dk, Dv);
    size_t n = 256 + s.images;
    if (backward) n += s.e + 2 * s.heads + s.states + s.inner + s.writes;
    return n;
}

extern "C" s5_status s5_delta_forward(const void *q, long long ldq, const void *k, long long ldk, const void *v,
                                      long long ldv, s5_dtype dtype, const float *g, const float *beta,
                                      const float *s0, float scale, int B, int L, int Hk, int Hv, int Dk, int Dv,
                                      void *o, long long ldo, float *s_last, void *saved, size_t saved_bytes,
                                      void *workspace, size_t workspace_bytes, s5_stream_t stream) {
    const s5_status c = check_sizes(B, L, Hk, Hv, Dk, Dv, dtype);
    if (c != S5_OK) return c;
    if (!(scale == scale) || !aligned16_or_null(s0) || !aligned16_or_null(s_last) || !aligned16_or_null(saved))
        return S5_ERR_INVALID_ARGUMENT;
    if (saved && saved_bytes < s5_delta_saved_size(B, L, Hv, Dk, Dv)) return S5_ERR_INVALID_ARGUMENT;
    if (B == 0) return S5_OK;
    if (L > 0) {
        if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !floats(g) || !floats(beta) || !aligned16(o))
            return S5_ERR_INVALID_ARGUMENT;
        if (ldq < (long long)Hk * Dk || ldk < (long long)Hk * Dk || ldv < (long long)Hv * Dv || ldo < (long long)Hv * Dv)
            return S5_ERR_INVALID_ARGUMENT;
        if (!aligned16(workspace) || workspace_bytes < s5_delta_workspace_size(B, L, Hv, Dk, Dv, 0))
            return S5_ERR_INVALID_ARGUMENT;
    }
    Args a = {};
    a.q = q, a.k = k, a.v = v, a.ldq = ldq, a.ldk = ldk, a.ldv = ldv, a.g = g, a.beta = beta, a.s0 = s0;
    a.scale = scale, a.B = B, a.L = L, a.Hk = Hk, a.Hv = Hv, a.Dk = Dk, a.Dv = Dv;
    a.o = o, a.ldo = ldo, a.s_last = s_last;
    const Sizes s = sizes(B, L, Hv, Dk, Dv);
    if (saved) {
        char *p = static_cast<char *>(saved);
        a.e = reinterpret_cast<float *>(p);
        a.states = reinterpret_cast<float *>(p + 2 * s.e);
    }
    a.images = reinterpret_cast<void *>((reinterpret_cast<uintptr_t>(workspace) + 255) & ~uintptr_t(255));
    cudaStream_t st = (cudaStream_t)stream;
    cudaError_t e;
    if (tc_supported(a, dtype, false))
        e = tc_forward(a, st);
    else
        e = dtype == S5_BF16 ? column_sweep<__nv_bfloat16, false>(a, st) : column_sweep<float, false>(a, st);
    return e == cudaSuccess ? S5_OK : cuda_failure(e);
}

extern "C" s5_status s5_delta_backward(const void *q, long long ldq, const void *k, long long ldk, const void *v,
                                       long long ldv, s5_dtype dtype, const float *g, const float *beta,
                                       const float *s0, float scale, int B, int L, int Hk, int Hv, int Dk, int Dv,
                                       const void *dout, long long lddo, const float *ds_last, const void *saved,
                                       size_t saved_bytes, void *dq, long long lddq, void *dk, long long lddk,
                                       void *dv, long long lddv, float *dg, float *dbeta, float *ds0, void *workspace,
                                       size_t workspace_bytes, s5_stream_t stream) {
    const s5_status c = check_sizes(B, L, Hk, Hv, Dk, Dv, dtype);
    if (c != S5_OK) return c;
    if (!(scale == scale) || !aligned16_or_null(s0) || !aligned16_or_null(ds_last) || !aligned16_or_null(ds0))
        return S5_ERR_INVALID_ARGUMENT;
    if (B == 0) return S5_OK;
    if (!aligned16(saved) || saved_bytes < s5_delta_saved_size(B, L, Hv, Dk, Dv) || !aligned16(workspace) ||
        workspace_bytes < s5_delta_workspace_size(B, L, Hv, Dk, Dv, 1))
        return S5_ERR_INVALID_ARGUMENT;
    if (L > 0) {
        const void *all[] = {q, k, v, dout, dq, dk, dv, dg, dbeta};
        for (const void *p : all)
            if (!aligned16(p)) return S5_ERR_INVALID_ARGUMENT;
        if (!floats(g) || !floats(beta)) return S5_ERR_INVALID_ARGUMENT;
        const long long nk = (long long)Hk * Dk, nv = (long long)Hv * Dv;
        if (ldq < nk || ldk < nk || ldv < nv || lddo < nv || lddq < nk || lddk < nk || lddv < nv)
            return S5_ERR_INVALID_ARGUMENT;
    }
    Args a = {};
    a.q = q, a.k = k, a.v = v, a.ldq = ldq, a.ldk = ldk, a.ldv = ldv, a.g = g, a.beta = beta, a.s0 = s0;
    a.scale = scale, a.B = B, a.L = L, a.Hk = Hk, a.Hv = Hv, a.Dk = Dk, a.Dv = Dv;
    const Sizes s = sizes(B, L, Hv, Dk, Dv);
    char *p = static_cast<char *>(const_cast<void *>(saved));   // read only here
    a.e = reinterpret_cast<float *>(p);
    a.states = reinterpret_cast<float *>(p + 2 * s.e);
    a.dout = dout, a.lddo = lddo, a.ds_last = ds_last;
    a.dq = dq, a.dk = dk, a.dv = dv, a.lddq = lddq, a.lddk = lddk, a.lddv = lddv;
    a.dg = dg, a.dbeta = dbeta, a.ds0 = ds0;
    char *w = reinterpret_cast<char *>((reinterpret_cast<uintptr_t>(workspace) + 255) & ~uintptr_t(255));
    a.images = w;
    w += s.images;
    a.x = reinterpret_cast<float *>(w);
    w += s.e;
    a.dqh = reinterpret_cast<float *>(w);
    a.dkh = reinterpret_cast<float *>(w + s.heads);
    w += 2 * s.heads;
    a.z = w;
    w += s.states;
    a.inner = reinterpret_cast<float *>(w);
    w += s.inner;
    a.writes = reinterpret_cast<float *>(w);
    cudaStream_t st = (cudaStream_t)stream;
    cudaError_t e;
    if (tc_supported(a, dtype, true))
        e = tc_backward(a, st);
    else
        e = dtype == S5_BF16 ? backward<__nv_bfloat16>(a, st) : backward<float>(a, st);
    return e == cudaSuccess ? S5_OK : cuda_failure(e);
}

extern "C" s5_status s5_delta_step(const void *q, const void *k, const void *v, s5_dtype dtype, const float *g,
                                   const float *beta, float scale, int B, int Hk, int Hv, int Dk, int Dv,
                                   float *state, void *o, s5_stream_t stream) {
    const s5_status c = check_sizes(B, 1, Hk, Hv, Dk, Dv, dtype);
    if (c != S5_OK) return c;
    if (!(scale == scale)) return S5_ERR_INVALID_ARGUMENT;
    if (B == 0) return S5_OK;
    const uintptr_t four = dtype == S5_BF16 ? 7 : 15;   // a slice of any head size starts at four values
    const void *rows[] = {q, k, v, o};
    for (const void *p : rows)
        if (!p || (reinterpret_cast<uintptr_t>(p) & four)) return S5_ERR_INVALID_ARGUMENT;
    if (!floats(g) || !floats(beta) || !aligned16(state)) return S5_ERR_INVALID_ARGUMENT;
    cudaStream_t st = (cudaStream_t)stream;
    const cudaError_t e = dtype == S5_BF16 ? step<__nv_bfloat16>(q, k, v, g, beta, scale, B, Hk, Hv, Dk, Dv, state, o, st)
                                           : step<float>(q, k, v, g, beta, scale, B, Hk, Hv, Dk, Dv, state, o, st);
    return e == cudaSuccess ? S5_OK : cuda_failure(e);
}
