// s5_rotary.cu -- position rotation of queries and keys, alone or in one pass
// with their norm for each head, and its backward pass.
//
// A row is one head's D values of one token.  With n = rot/2 rotated pairs
// (a_i, b_i) -- (x_i, x_{i+n}) in the half layout, (x_2i, x_2i+1) in the
// interleaved one -- a position p and frequencies f_i:
//   z = x r w,   r = (sum x^2 / count + eps)^-1/2  (count = D, or 1 for unit norm)
//   y_a = A (cos(p f_i) z_a - sin(p f_i) z_b),  y_b = A (sin(p f_i) z_a + cos(p f_i) z_b)
// and the values past rot are z itself.  The rotation is orthogonal up to A,
// so the backward pass turns by the opposite angle first:
//   dz = A R^T dy,  dw = sum over rows of dz x r,
//   dx = r w dz - x r^3 / count * sum(w dz x).
//
// Angles.  p f in 32 bits is off by p 2^-24 radians (0.06 at a million), so a
// frequency is turned once per thread into a 64-bit fraction of a turn,
// f / 2 pi * 2^64, by integer arithmetic (FP64 runs at 1/64 of the FP32 rate
// here); p times it wraps exactly at whole turns, and the top 32 bits give
// sincospif an argument good to 2^-25 half turns at any p.
//
// Bound: memory.  A row is read and written once.  A group of lanes holds one
// row (two vectors of V values per lane: both halves of a pair are in the
// same lane in either layout) and keeps its token's cosines and sines in
// registers over all heads that it takes, so that they cost a few percent of
// the pass; four rows are in flight per group.
#include "s5_internal.cuh"

namespace s5 {
namespace {

constexpr int RT = 128;             // threads per block
constexpr int ROWS = 4;             // rows in flight per group
constexpr int BWD_BLOCKS = 152 * 6; // blocks of the backward pass: one wave, one partial of dw each

struct RotArgs {
    const void *x[2], *dy[2];   // queries, keys (dy: backward only)
    void *y[2];                 // outputs; backward: dx
    const float *w[2];
    long long ldx[2], ldy[2], lddy[2];
    int heads[2];
    const long long *pos;
    const double *freq;
    float *partial;             // [2][blocks][D] of dw (backward)
    long long T;
    int D, rot, count;          // count: divisor of the sum of squares, 0 = no norm
    float eps, amp;             // amp carries the sign of the sines in `turn`
    float turn;                 // +1 forward, -1 transposed
    int per;                    // heads per group
    int segs[2];                // groups per token for queries and keys
    int want_dw[2];
};

template <typename T, int V> struct Vec;
template <int V> struct Vec<float, V> {
    __device__ static void load(const float *p, float (&r)[V]) {
        if constexpr (V >= 4) {
#pragma unroll
            for (int i = 0; i < V; i += 4) {
                const float4 t = *reinterpret_cast<const float4 *>(p + i);
                r[i] = t.x, r[i + 1] = t.y, r[i + 2] = t.z, r[i + 3] = t.w;
            }
        } else if constexpr (V == 2) {
            const float2 t = *reinterpret_cast<const float2 *>(p);
            r[0] = t.x, r[1] = t.y;
        } else
            r[0] = *p;
    }
    __device__ static void store(float *p, const float (&r)[V]) {
        if constexpr (V == 4)
            *reinterpret_cast<float4 *>(p) = make_float4(r[0], r[1], r[2], r[3]);
        else if constexpr (V == 2)
            *reinterpret_cast<float2 *>(p) = make_float2(r[0], r[1]);
        else
            *p = r[0];
    }
};
__device__ __forceinline__ float bf_lo(unsigned v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf_hi(unsigned v) { return __uint_as_float(v & 0xffff0000u); }
__device__ __forceinline__ unsigned bf_pack(float lo, float hi) {
    const __nv_bfloat162 t = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const unsigned *>(&t);
}
template <int V> struct Vec<__nv_bfloat16, V> {
    __device__ static void load(const __nv_bfloat16 *p, float (&r)[V]) {
        if constexpr (V == 8) {
            const uint4 t = *reinterpret_cast<const uint4 *>(p);
            r[0] = bf_lo(t.x), r[1] = bf_hi(t.x), r[2] = bf_lo(t.y), r[3] = bf_hi(t.y);
            r[4] = bf_lo(t.z), r[5] = bf_hi(t.z), r[6] = bf_lo(t.w), r[7] = bf_hi(t.w);
        } else if constexpr (V == 4) {
            const uint2 t = *reinterpret_cast<const uint2 *>(p);
            r[0] = bf_lo(t.x), r[1] = bf_hi(t.x), r[2] = bf_lo(t.y), r[3] = bf_hi(t.y);
        } else if constexpr (V == 2) {
            const unsigned t = *reinterpret_cast<const unsigned *>(p);
            r[0] = bf_lo(t), r[1] = bf_hi(t);
        } else
            r[0] = __bfloat162float(*p);
    }
    __device__ static void store(__nv_bfloat16 *p, const float (&r)[V]) {
        if constexpr (V == 8)
            *reinterpret_cast<uint4 *>(p) =
                make_uint4(bf_pack(r[0], r[1]), bf_pack(r[2], r[3]), bf_pack(r[4], r[5]), bf_pack(r[6], r[7]));
        else if constexpr (V == 4)
            *reinterpret_cast<uint2 *>(p) = make_uint2(bf_pack(r[0], r[1]), bf_pack(r[2], r[3]));
        else if constexpr (V == 2)
            *reinterpret_cast<unsigned *>(p) = bf_pack(r[0], r[1]);
        else
            *p = __float2bfloat16_rn(r[0]);
    }
};

// f / 2 pi as a 64-bit fraction of a turn: the 53-bit significand times
// 2^66 / 2 pi, shifted by the exponent.  Whole turns fall off the top.
__device__ __forceinline__ unsigned long long turns64(double f) {
    const unsigned long long bits = __double_as_longlong(f);
    const int e = (int)((bits >> 52) & 0x7ff);
    if (e == 0) return 0ull;   // zero; a subnormal frequency turns by nothing
    const unsigned long long m = ((bits << 11) | 0x8000000000000000ull);
    unsigned long long t = __umul64hi(m, 0xa2f9836e4e441529ull);   // floor(2^66 / 2 pi)
    const int s = e - 1024;
    t = s >= 64 ? 0ull : s >= 0 ? t << s : s > -64 ? t >> -s : 0ull;
    return (bits >> 63) ? 0ull - t : t;
}

// Lanes of a group, slots of 2 V values in a lane.
template <int V> constexpr int SLOTS = V >= 4 ? 1 : 4 / V;

// Where a slot's two vectors start in the row.
template <int V, bool INTER>
__device__ __forceinline__ void slot_place(int slot, int n, int &lo, int &hi) {
    if (!INTER && slot * V < n) {
        lo = slot * V;
        hi = lo + n;
    } else {
        lo = slot * 2 * V;   // interleaved, or past the rotated part
        hi = lo + V;
    }
}

// cos and sin of the slot's V pairs (identity past the rotated part).
template <int V, bool INTER>
__device__ __forceinline__ void slot_freq(const RotArgs &a, int slot, unsigned long long (&f)[V], bool &rotated) {
    rotated = slot * V < a.rot / 2;
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = rotated ? turns64(a.freq[slot * V + i]) : 0ull;
}
template <int V>
__device__ __forceinline__ void slot_angles(const RotArgs &a, const unsigned long long (&f)[V], bool rotated,
                                            long long pos, float (&c)[V], float (&s)[V]) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
        if (rotated) {
            const int top = (int)(((unsigned long long)pos * f[i]) >> 32);
            sincospif((float)top * 4.656612873077393e-10f, &s[i], &c[i]);   // 2^-31
            c[i] *= a.amp;
            s[i] *= a.amp * a.turn;
        } else {
            c[i] = 1.0f;
            s[i] = 0.0f;
        }
    }
}

// Pair i of the slot: (lo[i], hi[i]) in the half layout; neighbours in the
// interleaved one, where lo and hi are 2 V consecutive values.
template <int V, bool INTER>
__device__ __forceinline__ void rotate(float (&lo)[V], float (&hi)[V], const float (&c)[V], const float (&s)[V]) {
    if constexpr (INTER && V > 1) {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            float a = lo[2 * i], b = lo[2 * i + 1];
            lo[2 * i] = c[i] * a - s[i] * b;
            lo[2 * i + 1] = s[i] * a + c[i] * b;
            a = hi[2 * i], b = hi[2 * i + 1];
            hi[2 * i] = c[V / 2 + i] * a - s[V / 2 + i] * b;
            hi[2 * i + 1] = s[V / 2 + i] * a + c[V / 2 + i] * b;
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float a = lo[i], b = hi[i];
            lo[i] = c[i] * a - s[i] * b;
            hi[i] = s[i] * a + c[i] * b;
        }
    }
}

template <int G> __device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int m = G / 2; m > 0; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
    return v;
}

template <typename T, int V, int G, bool INTER>
__global__ void __launch_bounds__(RT) rotary_fwd_kernel(const RotArgs a) {
    constexpr int S = SLOTS<V>;
    const int lane = threadIdx.x % G;
    const int n = a.rot / 2, nslots = a.D / (2 * V);
    const long long groups = a.T * (a.segs[0] + a.segs[1]);
    const long long gid = (long long)blockIdx.x * (RT / G) + threadIdx.x / G;
    griddep_launch_dependents();
    unsigned long long f[S][V];
    bool rotated[S];
    int lo[S], hi[S];
#pragma unroll
    for (int j = 0; j < S; ++j) {
        const int slot = lane + j * G;
        slot_place<V, INTER>(slot, n, lo[j], hi[j]);
        if (slot >= nslots) lo[j] = -1;
    }
    griddep_wait();
#pragma unroll
    for (int j = 0; j < S; ++j)
        if (lo[j] >= 0)
            slot_freq<V, INTER>(a, lane + j * G, f[j], rotated[j]);
        else
            rotated[j] = false;
    // every lane of a warp makes the same number of passes: the sums over a
    // group use full-warp shuffles
    const bool live = gid < groups;
    const long long token = live ? gid / (a.segs[0] + a.segs[1]) : 0;
    const int seg = live ? (int)(gid % (a.segs[0] + a.segs[1])) : 0;
    const int part = seg >= a.segs[0];
    const int h0 = (part ? seg - a.segs[0] : seg) * a.per;
    const int h1 = live ? min(h0 + a.per, a.heads[part]) : h0;
    const long long pos = (live && n) ? a.pos[token] : 0;
    float c[S][V], s[S][V];
#pragma unroll
    for (int j = 0; j < S; ++j) slot_angles<V>(a, f[j], rotated[j], pos, c[j], s[j]);
    const T *x = static_cast<const T *>(part ? a.x[1] : a.x[0]) + token * (part ? a.ldx[1] : a.ldx[0]);
    T *y = static_cast<T *>(part ? a.y[1] : a.y[0]) + token * (part ? a.ldy[1] : a.ldy[0]);
    const float *w = part ? a.w[1] : a.w[0];
    for (int base = 0; base < a.per; base += ROWS) {
        float u[ROWS][S][V], t[ROWS][S][V];
#pragma unroll
        for (int r = 0; r < ROWS; ++r)
#pragma unroll
            for (int j = 0; j < S; ++j) {
                if (h0 + base + r < h1 && lo[j] >= 0) {
                    const T *row = x + (long long)(h0 + base + r) * a.D;
                    Vec<T, V>::load(row + lo[j], u[r][j]);
                    Vec<T, V>::load(row + hi[j], t[r][j]);
                } else {
#pragma unroll
                    for (int i = 0; i < V; ++i) u[r][j][i] = t[r][j][i] = 0.0f;
                }
            }
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
            if (a.count) {
                float ss = 0.0f;
#pragma unroll
                for (int j = 0; j < S; ++j)
#pragma unroll
                    for (int i = 0; i < V; ++i) ss = fmaf(u[r][j][i], u[r][j][i], fmaf(t[r][j][i], t[r][j][i], ss));
                const float rs = rsqrtf(group_sum<G>(ss) / (float)a.count + a.eps);
#pragma unroll
                for (int j = 0; j < S; ++j)
#pragma unroll
                    for (int i = 0; i < V; ++i) u[r][j][i] *= rs, t[r][j][i] *= rs;
            }
            if (w) {
#pragma unroll
                for (int j = 0; j < S; ++j)
                    if (lo[j] >= 0) {
                        float wl[V], wh[V];
                        Vec<float, V>::load(w + lo[j], wl);
                        Vec<float, V>::load(w + hi[j], wh);
#pragma unroll
                        for (int i = 0; i < V; ++i) u[r][j][i] *= wl[i], t[r][j][i] *= wh[i];
                    }
            }
            if (h0 + base + r < h1) {
                T *row = y + (long long)(h0 + base + r) * a.D;
#pragma unroll
                for (int j = 0; j < S; ++j)
                    if (lo[j] >= 0) {
                        if (rotated[j]) rotate<V, INTER>(u[r][j], t[r][j], c[j], s[j]);
                        Vec<T, V>::store(row + lo[j], u[r][j]);
                        Vec<T, V>::store(row + hi[j], t[r][j]);
                    }
            }
        }
    }
}

// Backward.  Block b takes queries if b < qblocks, else keys; a group keeps
// its slots' part of dw in registers over all rows it takes, the block adds
// its groups in shared memory, in a fixed order, and writes one partial row.
template <typename T, int V, int G, bool INTER>
__global__ void __launch_bounds__(RT) rotary_bwd_kernel(const RotArgs a, int qblocks) {
    constexpr int S = SLOTS<V>, NG = RT / G;
    extern __shared__ float red[];   // [NG][D]
    const int lane = threadIdx.x % G, grp = threadIdx.x / G;
    const int n = a.rot / 2, nslots = a.D / (2 * V);
    const int part = (int)blockIdx.x >= qblocks;
    const int blk = part ? blockIdx.x - qblocks : blockIdx.x;
    const int nblk = part ? gridDim.x - qblocks : qblocks;
    const int heads = part ? a.heads[1] : a.heads[0], segs = part ? a.segs[1] : a.segs[0];
    const float *w = part ? a.w[1] : a.w[0];
    const long long ldx = part ? a.ldx[1] : a.ldx[0], ldy = part ? a.ldy[1] : a.ldy[0],
                    lddy = part ? a.lddy[1] : a.lddy[0];
    const T *xb = static_cast<const T *>(part ? a.x[1] : a.x[0]);
    const T *gb = static_cast<const T *>(part ? a.dy[1] : a.dy[0]);
    T *yb = static_cast<T *>(part ? a.y[1] : a.y[0]);
    unsigned long long f[S][V];
    bool rotated[S];
    int lo[S], hi[S];
    float wl[S][V], wh[S][V], dl[S][V], dh[S][V];
    griddep_wait();
#pragma unroll
    for (int j = 0; j < S; ++j) {
        const int slot = lane + j * G;
        slot_place<V, INTER>(slot, n, lo[j], hi[j]);
        rotated[j] = false;
        if (slot >= nslots)
            lo[j] = -1;
        else
            slot_freq<V, INTER>(a, slot, f[j], rotated[j]);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            wl[j][i] = (w && lo[j] >= 0) ? w[lo[j] + i] : 1.0f;
            wh[j][i] = (w && lo[j] >= 0) ? w[hi[j] + i] : 1.0f;
            dl[j][i] = dh[j][i] = 0.0f;
        }
    }
    const long long items = a.T * segs, stride = (long long)nblk * NG;
    // the trip count is the block's, not the group's: shuffles use full warps
    for (long long it0 = (long long)blk * NG; it0 < items; it0 += stride) {
        const long long it = it0 + grp;
        const bool live = it < items;
        const long long token = live ? it / segs : 0;
        const int h0 = live ? (int)(it % segs) * a.per : 0, h1 = live ? min(h0 + a.per, heads) : 0;
        const long long pos = (live && n) ? a.pos[token] : 0;
        float c[S][V], s[S][V];
#pragma unroll
        for (int j = 0; j < S; ++j) slot_angles<V>(a, f[j], rotated[j], pos, c[j], s[j]);
        for (int base = 0; base < a.per; base += 2) {
            float u[2][S][V], t[2][S][V], p[2][S][V], q[2][S][V];
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int j = 0; j < S; ++j) {
                    if (h0 + base + r < h1 && lo[j] >= 0) {
                        const long long o = (long long)(h0 + base + r) * a.D;
                        Vec<T, V>::load(xb + token * ldx + o + lo[j], u[r][j]);
                        Vec<T, V>::load(xb + token * ldx + o + hi[j], t[r][j]);
                        Vec<T, V>::load(gb + token * lddy + o + lo[j], p[r][j]);
                        Vec<T, V>::load(gb + token * lddy + o + hi[j], q[r][j]);
                    } else {
#pragma unroll
                        for (int i = 0; i < V; ++i) u[r][j][i] = t[r][j][i] = p[r][j][i] = q[r][j][i] = 0.0f;
                    }
                }
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                float ss = 0.0f, sx = 0.0f;
#pragma unroll
                for (int j = 0; j < S; ++j) {
                    if (rotated[j]) rotate<V, INTER>(p[r][j], q[r][j], c[j], s[j]);   // dz
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        ss = fmaf(u[r][j][i], u[r][j][i], fmaf(t[r][j][i], t[r][j][i], ss));
                        sx = fmaf(p[r][j][i] * wl[j][i], u[r][j][i], fmaf(q[r][j][i] * wh[j][i], t[r][j][i], sx));
                    }
                }
                float rs = 1.0f, k = 0.0f;
                if (a.count) {
                    rs = rsqrtf(group_sum<G>(ss) / (float)a.count + a.eps);
                    k = rs * rs * rs * (group_sum<G>(sx) / (float)a.count);
                }
                const bool on = h0 + base + r < h1;
                T *row = yb + token * ldy + (long long)(h0 + base + r) * a.D;
#pragma unroll
                for (int j = 0; j < S; ++j) {
                    float xl[V], xh[V];
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        if (on) {   // a dead row would add 0 * rsqrt(eps): NaN where eps is 0
                            dl[j][i] = fmaf(p[r][j][i], u[r][j][i] * rs, dl[j][i]);
                            dh[j][i] = fmaf(q[r][j][i], t[r][j][i] * rs, dh[j][i]);
                        }
                        xl[i] = rs * wl[j][i] * p[r][j][i] - u[r][j][i] * k;
                        xh[i] = rs * wh[j][i] * q[r][j][i] - t[r][j][i] * k;
                    }
                    if (on && lo[j] >= 0) {
                        Vec<T, V>::store(row + lo[j], xl);
                        Vec<T, V>::store(row + hi[j], xh);
                    }
                }
            }
        }
    }
    if (!(part ? a.want_dw[1] : a.want_dw[0])) return;
#pragma unroll
    for (int j = 0; j < S; ++j)
        if (lo[j] >= 0)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                red[grp * a.D + lo[j] + i] = dl[j][i];
                red[grp * a.D + hi[j] + i] = dh[j][i];
            }
    __syncthreads();
    for (int d = threadIdx.x; d < a.D; d += RT) {
        float v = 0.0f;
        for (int g = 0; g < NG; ++g) v += red[g * a.D + d];
        a.partial[(long long)blockIdx.x * a.D + d] = v;
    }
}

// dw[d] = sum of the blocks' partials: a block takes 8 values, 32 lanes each
// stride over the partials and are added in shared memory in a fixed order.
__global__ void __launch_bounds__(256) rotary_dw_kernel(const float *partial, int qblocks, int blocks, int D, float *dwq,
                                                        float *dwk) {
    __shared__ float red[32][9];
    const int col = threadIdx.x % 8, row = threadIdx.x / 8;
    const int part = blockIdx.y, d = blockIdx.x * 8 + col;
    float *out = part ? dwk : dwq;
    griddep_wait();
    if (!out) return;
    const int b0 = part ? qblocks : 0, b1 = part ? blocks : qblocks;
    float v = 0.0f;
    if (d < D)
        for (int b = b0 + row; b < b1; b += 32) v += partial[(long long)b * D + d];
    red[row][col] = v;
    __syncthreads();
    if (row == 0 && d < D) {
        float s = 0.0f;
        for (int r = 0; r < 32; ++r) s += red[r][col];
        out[d] = s;
    }
}

template <typename... Ks, typename... As>
cudaError_t launch_pdl(void (*k)(Ks...), dim3 grid, int threads, size_t smem, cudaStream_t st, As... args) {
    cudaLaunchAttribute attr;
    set_programmatic(attr);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k, args...);
}

// Values per vector: the widest (16 bytes at most) that divides the pair
// offset, the unrotated rest and every pitch.
int vec_width(int elem, int D, int rot, bool inter, const long long *lds, int nld) {
    for (int V = elem == 2 ? 8 : 4; V > 1; V /= 2) {
        bool ok = D % (2 * V) == 0 && (inter ? rot % (2 * V) == 0 : (rot / 2) % V == 0);
        for (int i = 0; i < nld; ++i) ok = ok && lds[i] % V == 0;
        if (ok) return V;
    }
    return 1;
}

template <typename T, int V, int G, bool INTER>
cudaError_t run_group(RotArgs &a, bool backward, float *dwq, float *dwk, cudaStream_t st) {
    constexpr int NG = RT / G;
    if (!backward) {
        const long long groups = a.T * (a.segs[0] + a.segs[1]);
        return launch_pdl(rotary_fwd_kernel<T, V, G, INTER>, dim3((unsigned)((groups + NG - 1) / NG)), RT, 0, st, a);
    }
    const long long wq = (a.T * a.segs[0] + NG - 1) / NG, wk = (a.T * a.segs[1] + NG - 1) / NG;
    // blocks in the proportion of the work, one wave at most
    long long qb = wq, kb = wk;
    if (wq + wk > BWD_BLOCKS) {
        qb = wq ? BWD_BLOCKS * wq / (wq + wk) : 0;
        if (wq && qb < 1) qb = 1;
        if (wk && qb > BWD_BLOCKS - 1) qb = BWD_BLOCKS - 1;
        kb = wk ? BWD_BLOCKS - qb : 0;
    }
    a.want_dw[0] = dwq != nullptr;
    a.want_dw[1] = dwk != nullptr;
    cudaError_t e = launch_pdl(rotary_bwd_kernel<T, V, G, INTER>, dim3((unsigned)(qb + kb)), RT,
                               sizeof(float) * NG * a.D, st, a, (int)qb);
    if (e == cudaSuccess && (dwq || dwk))
        e = launch_pdl(rotary_dw_kernel, dim3((a.D + 7) / 8, 2), 256, 0, st, (const float *)a.partial, (int)qb,
                       (int)(qb + kb), a.D, dwq, dwk);
    return e;
}

template <typename T, int V, bool INTER>
cudaError_t run_vec(RotArgs &a, bool backward, float *dwq, float *dwk, cudaStream_t st) {
    const int lanes = (a.D / (2 * V) + SLOTS<V> - 1) / SLOTS<V>;
    // odd sizes (V of 1 or 2) take whole warps; else the least power of two
    if constexpr (V == 8)
        if (lanes <= 4) return run_group<T, V, 4, INTER>(a, backward, dwq, dwk, st);
    if constexpr (V >= 4) {
        if (lanes <= 8) return run_group<T, V, 8, INTER>(a, backward, dwq, dwk, st);
        if (lanes <= 16) return run_group<T, V, 16, INTER>(a, backward, dwq, dwk, st);
    }
    if constexpr (V < 8) return run_group<T, V, 32, INTER>(a, backward, dwq, dwk, st);
    return cudaErrorInvalidValue;   // V = 8: at most 16 lanes
}

template <typename T>
cudaError_t run_type(RotArgs &a, int V, bool inter, bool backward, float *dwq, float *dwk, cudaStream_t st) {
    // heads per group: eight, so that a token's angles are paid once for
    // eight rows; fewer where the call is too small to fill the SMs
    // (152 x 2048 lanes), down to one
    const int lanes = a.D / (2 * V) < 32 ? a.D / (2 * V) : 32;
    a.per = 8;
    while (a.per > 1 && a.T * ((a.heads[0] + a.heads[1]) / a.per) * lanes < 152 * 2048) a.per /= 2;
    for (int p = 0; p < 2; ++p) a.segs[p] = (a.heads[p] + a.per - 1) / a.per;
#define S5_ROT(VV) \
    return inter ? run_vec<T, VV, true>(a, backward, dwq, dwk, st) : run_vec<T, VV, false>(a, backward, dwq, dwk, st)
    if constexpr (sizeof(T) == 2)
        if (V == 8) S5_ROT(8);
    if (V == 4) S5_ROT(4);
    if (V == 2) S5_ROT(2);
    S5_ROT(1);
#undef S5_ROT
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Checks what the three entry points share.
s5_status check_common(s5_dtype dtype, const long long *pos, const double *freq, int rot, int layout, float amp,
                       long long T, int H, int D) {
    if (dtype != S5_F32 && dtype != S5_BF16) return S5_ERR_INVALID_ARGUMENT;
    if (layout != S5_ROTARY_HALF && layout != S5_ROTARY_INTERLEAVED) return S5_ERR_INVALID_ARGUMENT;
    if (T < 0 || H < 0 || D < 1 || rot < 0 || rot > D || rot % 2) return S5_ERR_INVALID_ARGUMENT;
    if (!(amp > 0.0f) || amp > 1e30f) return S5_ERR_INVALID_ARGUMENT;
    if (D % 2 || D > 256) return S5_ERR_UNSUPPORTED;
    if (T > (1ll << 31) / (H > 0 ? H : 1)) return S5_ERR_UNSUPPORTED;
    if (T > 0 && rot > 0 && (!pos || !freq || !aligned16(freq) || (reinterpret_cast<uintptr_t>(pos) & 7u)))
        return S5_ERR_INVALID_ARGUMENT;
    return S5_OK;
}
// One of the row arrays: [T][H][D] with a pitch between tokens.
bool rows_ok(const void *p, long long ld, int H, int D, bool used) {
    return !used || (p && aligned16(p) && ld >= (long long)H * D);
}

}  // namespace
}  // namespace s5

using namespace s5;

extern "C" s5_status s5_rotary(const void *x, long long ldx, s5_dtype dtype, const long long *positions,
                               const double *freq, int rot, s5_rotary_layout layout, float amplitude, int inverse,
                               long long T, int H, int D, void *y, long long ldy, s5_stream_t stream) {
    const s5_status c = check_common(dtype, positions, freq, rot, layout, amplitude, T, H, D);
    if (c != S5_OK) return c;
    if (T == 0 || H == 0) return S5_OK;
    if (!rows_ok(x, ldx, H, D, true) || !rows_ok(y, ldy, H, D, true)) return S5_ERR_INVALID_ARGUMENT;
    if (x == y && ldx != ldy) return S5_ERR_INVALID_ARGUMENT;
    RotArgs a = {};
    a.x[0] = x, a.y[0] = y, a.ldx[0] = ldx, a.ldy[0] = ldy, a.heads[0] = H;
    a.pos = positions, a.freq = freq, a.T = T, a.D = D, a.rot = rot;
    a.amp = amplitude, a.turn = inverse ? -1.0f : 1.0f;
    const long long lds[2] = {ldx, ldy};
    const bool inter = layout == S5_ROTARY_INTERLEAVED;
    const int V = vec_width(dtype == S5_BF16 ? 2 : 4, D, rot, inter, lds, 2);
    cudaStream_t st = (cudaStream_t)stream;
    const cudaError_t e = dtype == S5_BF16 ? run_type<__nv_bfloat16>(a, V, inter, false, nullptr, nullptr, st)
                                           : run_type<float>(a, V, inter, false, nullptr, nullptr, st);
    return e == cudaSuccess ? S5_OK : cuda_failure(e);
}

extern "C" s5_status s5_qk_norm_rotary(const void *q, long long ldq, const void *k, long long ldk, s5_dtype dtype,
                                       const float *q_weight, const float *k_weight, s5_norm norm, float eps,
                                       const long long *positions, const double *freq, int rot,
                                       s5_rotary_layout layout, float amplitude, long long T, int Hq, int Hk, int D,
                                       void *q_out, long long ldqo, void *k_out, long long ldko, s5_stream_t stream) {
    if (Hq < 0 || Hk < 0 || Hq > (1 << 20) || Hk > (1 << 20)) return S5_ERR_INVALID_ARGUMENT;
    const s5_status c = check_common(dtype, positions, freq, rot, layout, amplitude, T, Hq + Hk, D);
    if (c != S5_OK) return c;
    if (norm != S5_NORM_NONE && norm != S5_NORM_RMS && norm != S5_NORM_L2) return S5_ERR_INVALID_ARGUMENT;
    if (!(eps >= 0.0f) || eps > 1e30f) return S5_ERR_INVALID_ARGUMENT;
    if ((q_weight && !aligned16(q_weight)) || (k_weight && !aligned16(k_weight))) return S5_ERR_INVALID_ARGUMENT;
    if (T == 0 || Hq + Hk == 0) return S5_OK;
    if (!rows_ok(q, ldq, Hq, D, Hq > 0) || !rows_ok(k, ldk, Hk, D, Hk > 0) || !rows_ok(q_out, ldqo, Hq, D, Hq > 0) ||
        !rows_ok(k_out, ldko, Hk, D, Hk > 0))
        return S5_ERR_INVALID_ARGUMENT;
    if ((Hq && q == q_out && ldq != ldqo) || (Hk && k == k_out && ldk != ldko)) return S5_ERR_INVALID_ARGUMENT;
    RotArgs a = {};
    a.x[0] = q, a.x[1] = k, a.y[0] = q_out, a.y[1] = k_out;
    a.w[0] = q_weight, a.w[1] = k_weight;
    a.ldx[0] = ldq, a.ldx[1] = ldk, a.ldy[0] = ldqo, a.ldy[1] = ldko;
    a.heads[0] = Hq, a.heads[1] = Hk;
    a.pos = positions, a.freq = freq, a.T = T, a.D = D, a.rot = rot;
    a.count = norm == S5_NORM_RMS ? D : norm == S5_NORM_L2 ? 1 : 0;
    a.eps = eps, a.amp = amplitude, a.turn = 1.0f;
    const long long lds[4] = {Hq ? ldq : 0, Hk ? ldk : 0, Hq ? ldqo : 0, Hk ? ldko : 0};
    const bool inter = layout == S5_ROTARY_INTERLEAVED;
    const int V = vec_width(dtype == S5_BF16 ? 2 : 4, D, rot, inter, lds, 4);
    cudaStream_t st = (cudaStream_t)stream;
    const cudaError_t e = dtype == S5_BF16 ? run_type<__nv_bfloat16>(a, V, inter, false, nullptr, nullptr, st)
                                           : run_type<float>(a, V, inter, false, nullptr, nullptr, st);
    return e == cudaSuccess ? S5_OK : cuda_failure(e);
}

extern "C" size_t s5_qk_norm_rotary_workspace_size(int D) {
    return D < 1 || D > 256 ? 0 : sizeof(float) * (size_t)BWD_BLOCKS * D;
}

extern "C" s5_status s5_qk_norm_rotary_backward(
    const void *q, long long ldq, const void *k, long long ldk, s5_dtype dtype, const float *q_weight,
    const float *k_weight, s5_norm norm, float eps, const long long *positions, const double *freq, int rot,
    s5_rotary_layout layout, float amplitude, long long T, int Hq, int Hk, int D, const void *dq_out, long long lddqo,
    const void *dk_out, long long lddko, void *dq, long long lddq, void *dk, long long lddk, float *dq_weight,
    float *dk_weight, void *workspace, size_t workspace_bytes, s5_stream_t stream) {
    if (Hq < 0 || Hk < 0 || Hq > (1 << 20) || Hk > (1 << 20)) return S5_ERR_INVALID_ARGUMENT;
    const s5_status c = check_common(dtype, positions, freq, rot, layout, amplitude, T, Hq + Hk, D);
    if (c != S5_OK) return c;
    if (norm != S5_NORM_NONE && norm != S5_NORM_RMS && norm != S5_NORM_L2) return S5_ERR_INVALID_ARGUMENT;
    if (!(eps >= 0.0f) || eps > 1e30f) return S5_ERR_INVALID_ARGUMENT;
    if ((q_weight && !aligned16(q_weight)) || (k_weight && !aligned16(k_weight))) return S5_ERR_INVALID_ARGUMENT;
    if ((dq_weight && (!aligned16(dq_weight) || !q_weight)) || (dk_weight && (!aligned16(dk_weight) || !k_weight)))
        return S5_ERR_INVALID_ARGUMENT;
    cudaStream_t st = (cudaStream_t)stream;
    if (T == 0 || Hq + Hk == 0) {   // no rows: the weights' gradients are zero
        cudaError_t e = cudaSuccess;
        if (dq_weight) e = cudaMemsetAsync(dq_weight, 0, sizeof(float) * D, st);
        if (dk_weight && e == cudaSuccess) e = cudaMemsetAsync(dk_weight, 0, sizeof(float) * D, st);
        return e == cudaSuccess ? S5_OK : cuda_failure(e);
    }
    if (!rows_ok(q, ldq, Hq, D, Hq > 0) || !rows_ok(k, ldk, Hk, D, Hk > 0) || !rows_ok(dq_out, lddqo, Hq, D, Hq > 0) ||
        !rows_ok(dk_out, lddko, Hk, D, Hk > 0) || !rows_ok(dq, lddq, Hq, D, Hq > 0) || !rows_ok(dk, lddk, Hk, D, Hk > 0))
        return S5_ERR_INVALID_ARGUMENT;
    if ((Hq && ((dq == q && lddq != ldq) || (dq == dq_out && lddq != lddqo))) ||
        (Hk && ((dk == k && lddk != ldk) || (dk == dk_out && lddk != lddko))))
        return S5_ERR_INVALID_ARGUMENT;
    if ((dq_weight || dk_weight) &&
        (!workspace || !aligned16(workspace) || workspace_bytes < s5_qk_norm_rotary_workspace_size(D)))
        return S5_ERR_INVALID_ARGUMENT;
    RotArgs a = {};
    a.x[0] = q, a.x[1] = k, a.y[0] = dq, a.y[1] = dk, a.dy[0] = dq_out, a.dy[1] = dk_out;
    a.w[0] = q_weight, a.w[1] = k_weight;
    a.ldx[0] = ldq, a.ldx[1] = ldk, a.ldy[0] = lddq, a.ldy[1] = lddk, a.lddy[0] = lddqo, a.lddy[1] = lddko;
    a.heads[0] = Hq, a.heads[1] = Hk;
    a.pos = positions, a.freq = freq, a.T = T, a.D = D, a.rot = rot;
    a.count = norm == S5_NORM_RMS ? D : norm == S5_NORM_L2 ? 1 : 0;
    a.eps = eps, a.amp = amplitude, a.turn = -1.0f;
    a.partial = static_cast<float *>(workspace);
    const long long lds[6] = {Hq ? ldq : 0,  Hk ? ldk : 0,  Hq ? lddqo : 0,
                              Hk ? lddko : 0, Hq ? lddq : 0, Hk ? lddk : 0};
    const bool inter = layout == S5_ROTARY_INTERLEAVED;
    const int V = vec_width(dtype == S5_BF16 ? 2 : 4, D, rot, inter, lds, 6);
    const cudaError_t e = dtype == S5_BF16 ? run_type<__nv_bfloat16>(a, V, inter, true, dq_weight, dk_weight, st)
                                           : run_type<float>(a, V, inter, true, dq_weight, dk_weight, st);
    return e == cudaSuccess ? S5_OK : cuda_failure(e);
}
