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
// sincospif an argument good to 2^-25 half turns.  The fraction itself is off by up
// to max(1, f) 2^-63 turns, p times that at position p.
//
// Bound: memory.  A row is read and written once.  Two forms:
//  - Streaming, for rows that 16-byte copies can address: every warp runs a
//    ring of its own, three items of up to 4 KB (some heads of one token) that
//    bulk copies bring into shared memory, that it turns in place and that
//    bulk copies take away; no warp waits for another.  192 KB an SM in
//    flight.  A lane keeps one slot (four pairs) of its token's cosines and
//    sines over the item's rows.
//  - Direct, for small calls and odd pitches: a group of lanes loads four rows
//    of one token at once; their angles are worked out while they are on
//    their way.
// In both a lane holds both halves of its pairs, in either layout.  Norm and
// rotation of 336 MB of bf16 (40 heads of 128): 60 us, 5.6 TB/s; with the backward
// pass 537 MB in 131 us, 4.1 TB/s; rotation alone of 537 MB in 87 us, 6.2 TB/s.  (59,
// 127 and 86 where a wait that ran out did not end the warp's work and frequencies
// that are not finite were not looked for.)
#include <atomic>

#include "s5_internal.cuh"
#include "s5_sm100.cuh"

namespace s5 {
namespace {
using namespace sm100;

constexpr int RT = 128;             // threads per block
constexpr int SWARPS = 8;           // warps of a streaming block, two blocks an SM
// Bytes of rows from which on the streaming form runs: with a norm, the rotation
// alone, backward.  Heads of 128 in bf16, streaming / direct, us: with a norm 11.5
// / 11.2 at 21 MB, 14.5 / 15.5 at 31 MB, 35.8 / 40.2 at 84 MB; the rotation alone
// 4.3 / 4.0 at 1 MB, 4.5 / 4.8 at 2.1 MB, 5.3 / 7.0 at 8.4 MB, 26.5 / 28.8 at 67 MB;
// backward 5.8 / 5.5 at 0.7 MB, 6.0 / 8.4 at 1.3 MB, 55 / 101 at 84 MB.
constexpr long long STREAM_FWD = 24 << 20, STREAM_TURN = 2 << 20, STREAM_BWD = 1 << 20;
constexpr int STAGES = 3;           // items of a warp in shared memory
constexpr int FWD_ITEM = 4096;      // bytes of rows an item holds at most
constexpr int BWD_ITEM = 2048;      // of x, and as many of dy
constexpr int ROWS = 4;             // rows of a group, all in flight
constexpr int BWD_BLOCKS = 152 * 4; // blocks of the backward pass: one wave, one partial of dw each

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
    int D, rot;
    float inv;                  // factor on the sum of squares (1 / D, 1), 0 = no norm
    float eps, amp;             // amp carries the sign of the sines in `turn`
    float turn;                 // +1 forward, -1 transposed
    int per;                    // heads per group
    int segs[2];                // groups per token for queries and keys
    int want_dw[2];
    bool stream;                // which form runs
    unsigned long long limit;   // of a wait for a copy, ns (streaming)
};

// V values as they lie in memory, and as floats.
template <int BYTES> struct Raw;
template <> struct Raw<16> { using type = uint4; };
template <> struct Raw<8> { using type = uint2; };
template <> struct Raw<4> { using type = unsigned; };
template <> struct Raw<2> { using type = unsigned short; };

template <typename T, int V> struct Vec {
    using raw = typename Raw<sizeof(T) * V>::type;
    __device__ static raw load(const T *p) { return *reinterpret_cast<const raw *>(p); }
    __device__ static void widen(const raw &t, float (&r)[V]) {
        const T *e = reinterpret_cast<const T *>(&t);
#pragma unroll
        for (int i = 0; i < V; ++i) r[i] = (float)e[i];
    }
    __device__ static void store(T *p, const float (&r)[V]) {
        raw t;
        T *e = reinterpret_cast<T *>(&t);
        if constexpr (sizeof(T) == 2 && V > 1) {
#pragma unroll
            for (int i = 0; i < V; i += 2) *reinterpret_cast<__nv_bfloat162 *>(e + i) = __floats2bfloat162_rn(r[i], r[i + 1]);
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) e[i] = (T)r[i];
        }
        *reinterpret_cast<raw *>(p) = t;
    }
};
// V floats of a weight.
template <int V> __device__ __forceinline__ void load_weight(const float *p, float (&r)[V]) {
    Vec<float, V>::widen(Vec<float, V>::load(p), r);
}

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

// The slot's frequencies.  rotated: 0 past the rotated part, else bit 0, and
// bit 1 + i where pair i's frequency is not finite, whose values are NaN then.
template <int V, bool INTER>
__device__ __forceinline__ void slot_freq(const RotArgs &a, int slot, unsigned long long (&f)[V], unsigned &rotated) {
    rotated = slot * V < a.rot / 2;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const double x = rotated ? a.freq[slot * V + i] : 0.0;
        f[i] = turns64(x);
        if (!isfinite(x)) rotated |= 2u << i;
    }
}
// cos and sin of the slot's V pairs (identity past the rotated part).
template <int V>
__device__ __forceinline__ void slot_angles(const RotArgs &a, const unsigned long long (&f)[V], unsigned rotated,
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
    if (rotated > 1u)
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (rotated >> (i + 1) & 1u) c[i] = s[i] = __int_as_float(0x7fffffff);
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
    using X = Vec<T, V>;
    const int lane = threadIdx.x % G;
    const int n = a.rot / 2, nslots = a.D / (2 * V);
    const int segs = a.segs[0] + a.segs[1];
    const long long groups = a.T * segs;
    const long long gid = (long long)blockIdx.x * (RT / G) + threadIdx.x / G;
    griddep_launch_dependents();
    int lo[S], hi[S];
#pragma unroll
    for (int j = 0; j < S; ++j) {
        const int slot = lane + j * G;
        slot_place<V, INTER>(slot, n, lo[j], hi[j]);
        if (slot >= nslots) lo[j] = -1;
    }
    // every lane of a warp makes the same passes: the sums over a group use
    // full-warp shuffles
    const bool live = gid < groups;
    const long long token = live ? gid / segs : 0;
    const int seg = live ? (int)(gid - token * segs) : 0;
    const int part = seg >= a.segs[0];
    const int h0 = (part ? seg - a.segs[0] : seg) * a.per;
    const int rows = live ? min(a.per, (part ? a.heads[1] : a.heads[0]) - h0) : 0;
    const T *x = static_cast<const T *>(part ? a.x[1] : a.x[0]) + token * (part ? a.ldx[1] : a.ldx[0]) + (long long)h0 * a.D;
    T *y = static_cast<T *>(part ? a.y[1] : a.y[0]) + token * (part ? a.ldy[1] : a.ldy[0]) + (long long)h0 * a.D;
    const float *w = part ? a.w[1] : a.w[0];
    griddep_wait();
    // all rows are on their way before the angles are worked out
    typename X::raw u[ROWS][S], t[ROWS][S];
#pragma unroll
    for (int r = 0; r < ROWS; ++r)
#pragma unroll
        for (int j = 0; j < S; ++j)
            if (r < rows && lo[j] >= 0) {
                u[r][j] = X::load(x + r * a.D + lo[j]);
                t[r][j] = X::load(x + r * a.D + hi[j]);
            } else
                u[r][j] = t[r][j] = typename X::raw{};
    const long long pos = (live && n) ? a.pos[token] : 0;
    float c[S][V], s[S][V];
    unsigned rotated[S];
#pragma unroll
    for (int j = 0; j < S; ++j) {
        unsigned long long f[V];
        rotated[j] = 0;
        if (lo[j] >= 0) slot_freq<V, INTER>(a, lane + j * G, f, rotated[j]);
        slot_angles<V>(a, f, rotated[j], pos, c[j], s[j]);
    }
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        if (r >= a.per) break;
        float p[S][V], q[S][V];
#pragma unroll
        for (int j = 0; j < S; ++j) X::widen(u[r][j], p[j]), X::widen(t[r][j], q[j]);
        if (a.inv != 0.0f) {
            float ss = 0.0f;
#pragma unroll
            for (int j = 0; j < S; ++j)
#pragma unroll
                for (int i = 0; i < V; ++i) ss = fmaf(p[j][i], p[j][i], fmaf(q[j][i], q[j][i], ss));
            const float rs = rsqrtf(group_sum<G>(ss) * a.inv + a.eps);
#pragma unroll
            for (int j = 0; j < S; ++j)
#pragma unroll
                for (int i = 0; i < V; ++i) p[j][i] *= rs, q[j][i] *= rs;
        }
#pragma unroll
        for (int j = 0; j < S; ++j)
            if (r < rows && lo[j] >= 0) {
                if (w) {
                    float wl[V], wh[V];
                    load_weight<V>(w + lo[j], wl);
                    load_weight<V>(w + hi[j], wh);
#pragma unroll
                    for (int i = 0; i < V; ++i) p[j][i] *= wl[i], q[j][i] *= wh[i];
                }
                if (rotated[j]) rotate<V, INTER>(p[j], q[j], c[j], s[j]);
                X::store(y + r * a.D + lo[j], p[j]);
                X::store(y + r * a.D + hi[j], q[j]);
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
    using X = Vec<T, V>;
    unsigned long long f[S][V];
    unsigned rotated[S];
    int lo[S], hi[S];
    float wl[S][V], wh[S][V], dl[S][V], dh[S][V];
    griddep_wait();
#pragma unroll
    for (int j = 0; j < S; ++j) {
        const int slot = lane + j * G;
        slot_place<V, INTER>(slot, n, lo[j], hi[j]);
        rotated[j] = 0;
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
    // Two rows at a time, the next two on their way.  The trip count is the
    // block's, not the group's: shuffles use full warps.
    const long long items = a.T * segs, stride = (long long)nblk * NG, it0 = (long long)blk * NG;
    const int steps = (a.per + 1) / 2;
    const long long trips = items > it0 ? (items - it0 + stride - 1) / stride * steps : 0;
    typename X::raw nu[2][S], nt[2][S], np[2][S], nq[2][S];
    long long token = 0;
    int h0 = 0;
    auto fetch = [&](long long trip, long long &tk, int &head) {
        const long long it = it0 + trip / steps * stride + grp;
        const bool live = trip < trips && it < items;
        tk = live ? it / segs : 0;
        const int first = live ? (int)(it - tk * segs) * a.per : heads;
        head = first + (int)(trip % steps) * 2;
        const int end = min(first + a.per, heads);
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int j = 0; j < S; ++j)
                if (head + r < end && lo[j] >= 0) {
                    const long long o = (long long)(head + r) * a.D;
                    nu[r][j] = X::load(xb + tk * ldx + o + lo[j]);
                    nt[r][j] = X::load(xb + tk * ldx + o + hi[j]);
                    np[r][j] = X::load(gb + tk * lddy + o + lo[j]);
                    nq[r][j] = X::load(gb + tk * lddy + o + hi[j]);
                } else
                    nu[r][j] = nt[r][j] = np[r][j] = nq[r][j] = typename X::raw{};
        return end;
    };
    float c[S][V], s[S][V];
    int end = fetch(0, token, h0);
    for (long long trip = 0; trip < trips; ++trip) {
        typename X::raw cu[2][S], ct[2][S], cp[2][S], cq[2][S];
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int j = 0; j < S; ++j) cu[r][j] = nu[r][j], ct[r][j] = nt[r][j], cp[r][j] = np[r][j], cq[r][j] = nq[r][j];
        const long long tok = token;
        const int head = h0, last = end;
        if (trip % steps == 0) {
            const long long pos = n ? a.pos[tok] : 0;
#pragma unroll
            for (int j = 0; j < S; ++j) slot_angles<V>(a, f[j], rotated[j], pos, c[j], s[j]);
        }
        end = fetch(trip + 1, token, h0);
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            float u[S][V], t[S][V], p[S][V], q[S][V], ss = 0.0f, sx = 0.0f;
#pragma unroll
            for (int j = 0; j < S; ++j) {
                X::widen(cu[r][j], u[j]), X::widen(ct[r][j], t[j]), X::widen(cp[r][j], p[j]), X::widen(cq[r][j], q[j]);
                if (rotated[j]) rotate<V, INTER>(p[j], q[j], c[j], s[j]);   // dz
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    ss = fmaf(u[j][i], u[j][i], fmaf(t[j][i], t[j][i], ss));
                    sx = fmaf(p[j][i] * wl[j][i], u[j][i], fmaf(q[j][i] * wh[j][i], t[j][i], sx));
                }
            }
            float rs = 1.0f, k = 0.0f;
            if (a.inv != 0.0f) {
                rs = rsqrtf(group_sum<G>(ss) * a.inv + a.eps);
                k = rs * rs * rs * (group_sum<G>(sx) * a.inv);
            }
            if (head + r >= last) continue;   // a dead row would add 0 * rsqrt(eps): NaN where eps is 0
            T *row = yb + tok * ldy + (long long)(head + r) * a.D;
#pragma unroll
            for (int j = 0; j < S; ++j) {
                float xl[V], xh[V];
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    dl[j][i] = fmaf(p[j][i], u[j][i] * rs, dl[j][i]);
                    dh[j][i] = fmaf(q[j][i], t[j][i] * rs, dh[j][i]);
                    xl[i] = rs * wl[j][i] * p[j][i] - u[j][i] * k;
                    xh[i] = rs * wh[j][i] * q[j][i] - t[j][i] * k;
                }
                if (lo[j] >= 0) {
                    X::store(row + lo[j], xl);
                    X::store(row + hi[j], xh);
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


// ---------------------------------------------------------------------------
// Streaming form: V = 4, one slot a lane.  Items are (token, segment of heads),
// item i of a warp being i strides on; segments of queries come first.
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint64_t l2_policy(bool first) {
    uint64_t p;
    if (first)
        asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
    else
        asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
    return p;
}
__device__ __forceinline__ void bulk_in(void *dst, const void *src, uint32_t bytes, uint64_t *bar, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;" ::"r"(
            smem_addr(dst)),
        "l"(src), "r"(bytes), "r"(smem_addr(bar)), "l"(policy)
        : "memory");
}
__device__ __forceinline__ void bulk_out(void *dst, const void *src, uint32_t bytes, uint64_t policy) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group.L2::cache_hint [%0], [%1], %2, %3;" ::"l"(dst),
                 "r"(smem_addr(src)), "r"(bytes), "l"(policy)
                 : "memory");
}
__device__ __forceinline__ void bulk_wait_read_but_1() { asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory"); }
__device__ int g_rotary_fault = 0;
// The whole warp: whether the copy has come.  One that has not by the call's
// limit ends the warp's work: it turns, stores and fetches nothing more
// (copies_settle), and the host is told.
__device__ __forceinline__ bool copy_wait(uint64_t *bar, uint32_t parity, unsigned long long limit) {
    bool came = limit && mbar_try_wait(bar, parity);   // a limit of 0 gives everything up
    if (!came && limit) {
        const unsigned long long t0 = global_ns();
        while (!(came = mbar_try_wait_sleep(bar, parity, 100000)) && global_ns() - t0 < limit) {
        }
    }
    came = __all_sync(0xffffffffu, came);
    if (!came) atomicExch(&g_rotary_fault, 1);
    return came;
}
// After a wait that ran out: what the warp has armed, `count` stages from `st`
// on, lands (or 0.2 s pass) before the block gives its memory back.
__device__ __noinline__ void copies_settle(uint64_t *full, int st, uint32_t parity, int count) {
    const unsigned long long t0 = global_ns();
    for (; count > 0; --count) {
        while (!mbar_try_wait_sleep(full + st, parity, 100000) && global_ns() - t0 < 200000000ull) {
        }
        if (++st == STAGES) st = 0, parity ^= 1;
    }
}

// The items of warp w of W, one after the other.  With a norm and enough tokens a
// warp takes consecutive tokens, all segments of each, and works a token's
// angles and weights out once; the copies go first out of L2.  The rotation
// alone waits for memory more than for its angles: there the segments are dealt
// out one by one, so that all warps are at work on one stretch of memory.
// Dealt / by token, us: norm and rotation of 336 MB 65 / 60, with its backward
// pass 537 MB 134 / 128; rotation alone of 537 MB 86 / 97.
struct Item {
    long long token, place;   // place: of its first head in the token's row
    int part, rows;
};
struct Deal {
    int seg0, segs, seg = 0;
    long long token, count;          // the next item, and how many there are
    long long tokens_on;             // from one item to the next
    int segs_on;
    __device__ Deal(const RotArgs &a, int s0, int n, int w, long long W) : seg0(s0), segs(n) {
        if (a.inv != 0.0f && a.T >= 2 * W) {
            const long long per = (a.T + W - 1) / W;
            token = w * per, tokens_on = 0, segs_on = 1;
            count = a.T > token ? min(per, a.T - token) * n : 0;
        } else {
            const long long units = a.T * n;
            count = units > w ? (units - w + W - 1) / W : 0;
            token = w / n, seg = w % n;
            tokens_on = W / n, segs_on = (int)(W % n);
        }
    }
    __device__ Item next(const RotArgs &a) {
        Item m;
        int at = seg + seg0;
        m.token = token;
        m.part = at >= a.segs[0];
        if (m.part) at -= a.segs[0];
        const int h0 = at * a.per;
        m.place = (long long)h0 * a.D;   // a single token may have more values than 32 bits count
        m.rows = min(a.per, (m.part ? a.heads[1] : a.heads[0]) - h0);
        token += tokens_on, seg += segs_on;
        if (seg >= segs) seg -= segs, ++token;
        return m;
    }
};

// A pair's two values in a slot.
template <int V, bool INTER> __device__ __forceinline__ float &pair_a(float (&lo)[V], float (&hi)[V], int i) {
    return INTER ? (i < V / 2 ? lo[2 * i] : hi[2 * i - V]) : lo[i];
}
template <int V, bool INTER> __device__ __forceinline__ float &pair_b(float (&lo)[V], float (&hi)[V], int i) {
    return INTER ? (i < V / 2 ? lo[2 * i + 1] : hi[2 * i + 1 - V]) : hi[i];
}

template <typename T, int G, bool INTER>
__global__ void __launch_bounds__(SWARPS * 32, 2) rotary_stream_fwd_kernel(const RotArgs a) {
    constexpr int V = 4, RP = 32 / G;
    using X = Vec<T, V>;
    extern __shared__ __align__(128) unsigned char ring[];
    __shared__ uint64_t full[SWARPS][STAGES];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, slot = lane % G;
    T *buf = reinterpret_cast<T *>(ring + warp * STAGES * FWD_ITEM);
    constexpr int STRIDE = FWD_ITEM / sizeof(T);
    if (lane == 0) {
        for (int i = 0; i < STAGES; ++i) mbar_init(&full[warp][i], 1);
        fence_mbar_init();
    }
    __syncwarp();
    const int n = a.rot / 2, segs = a.segs[0] + a.segs[1];
    int lo, hi;
    slot_place<V, INTER>(slot, n, lo, hi);
    const bool in = slot < a.D / (2 * V);
    griddep_launch_dependents();
    griddep_wait();
    unsigned long long f[V];
    unsigned rotated = 0;
    if (in) slot_freq<V, INTER>(a, slot, f, rotated);
    const uint64_t policy = l2_policy(a.inv != 0.0f);
    Deal deal(a, 0, segs, blockIdx.x * SWARPS + warp, (long long)gridDim.x * SWARPS), ahead = deal;
    long long mypos = 0;   // lane i: the position of the item in stage i
    auto fetch = [&](long long i, int st) {
        if (i >= deal.count) return;
        const Item m = ahead.next(a);
        if (n && lane == st) mypos = a.pos[m.token];
        if (lane == 0) {
            const T *x = static_cast<const T *>(m.part ? a.x[1] : a.x[0]) + m.token * (m.part ? a.ldx[1] : a.ldx[0]) + m.place;
            const uint32_t bytes = (uint32_t)(m.rows * a.D * sizeof(T));
            mbar_arrive_tx(&full[warp][st], bytes);
            bulk_in(buf + st * STRIDE, x, bytes, &full[warp][st], policy);
        }
    };
#pragma unroll
    for (int i = 0; i < STAGES; ++i) fetch(i, i);
    int st = 0, phase = 0;
    long long token = -1;
    int part = -1;
    float c[V], s[V], ca[V], sa[V], cb[V], sb[V];   // a pair's cosine and sine, times its values' weights
    for (long long it = 0; it < deal.count; ++it) {
        const Item m = deal.next(a);
        const long long pos = __shfl_sync(0xffffffffu, mypos, st);
        if (m.token != token || m.part != part) {
            if (m.token != token) slot_angles<V>(a, f, rotated, pos, c, s);
            const float *w = m.part ? a.w[1] : a.w[0];
            float wl[V], wh[V];
#pragma unroll
            for (int i = 0; i < V; ++i) wl[i] = wh[i] = 1.0f;
            if (w && in) load_weight<V>(w + lo, wl), load_weight<V>(w + hi, wh);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float wa = pair_a<V, INTER>(wl, wh, i), wb = pair_b<V, INTER>(wl, wh, i);
                ca[i] = c[i] * wa, sa[i] = s[i] * wa, cb[i] = c[i] * wb, sb[i] = s[i] * wb;
            }
            token = m.token, part = m.part;
        }
        if (!copy_wait(&full[warp][st], phase, a.limit)) {
            copies_settle(full[warp], st, phase, (int)min(deal.count - it, it > 0 ? STAGES - 1ll : STAGES));
            break;
        }
        T *x = buf + st * STRIDE;
#pragma unroll 4
        for (int r0 = 0; r0 < m.rows; r0 += RP) {
            const int r = r0 + lane / G;
            const bool on = in && r < m.rows;
            float p[V] = {}, q[V] = {}, rs = 1.0f;
            if (on) X::widen(X::load(x + r * a.D + lo), p), X::widen(X::load(x + r * a.D + hi), q);
            if (a.inv != 0.0f) {
                float ss = 0.0f;
#pragma unroll
                for (int i = 0; i < V; ++i) ss = fmaf(p[i], p[i], fmaf(q[i], q[i], ss));
                rs = rsqrtf(group_sum<G>(ss) * a.inv + a.eps);
            }
            if (on) {
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    float &va = pair_a<V, INTER>(p, q, i), &vb = pair_b<V, INTER>(p, q, i);
                    const float xa = va * rs, xb = vb * rs;
                    va = ca[i] * xa, vb = cb[i] * xb;
                    if (rotated) va = fmaf(-sb[i], xb, va), vb = fmaf(sa[i], xa, vb);
                }
                X::store(x + r * a.D + lo, p);
                X::store(x + r * a.D + hi, q);
            }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
            T *y = static_cast<T *>(m.part ? a.y[1] : a.y[0]) + m.token * (m.part ? a.ldy[1] : a.ldy[0]) + m.place;
            bulk_out(y, x, (uint32_t)(m.rows * a.D * sizeof(T)), policy);
            bulk_commit();
            if (it > 0) bulk_wait_read_but_1();   // the item before has left its stage
        }
        __syncwarp();
        if (it > 0) fetch(it + STAGES - 1, st == 0 ? STAGES - 1 : st - 1);
        if (++st == STAGES) st = 0, phase ^= 1;
    }
    if (lane == 0) bulk_wait_all();
}

template <typename T, int G, bool INTER>
__global__ void __launch_bounds__(SWARPS * 32, 2) rotary_stream_bwd_kernel(const RotArgs a, int qblocks) {
    constexpr int V = 4, RP = 32 / G;
    using X = Vec<T, V>;
    extern __shared__ __align__(128) unsigned char ring[];
    __shared__ uint64_t full[SWARPS][STAGES];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, slot = lane % G;
    T *buf = reinterpret_cast<T *>(ring + warp * STAGES * 2 * BWD_ITEM);
    constexpr int STRIDE = 2 * BWD_ITEM / sizeof(T), DY = BWD_ITEM / sizeof(T);
    if (lane == 0) {
        for (int i = 0; i < STAGES; ++i) mbar_init(&full[warp][i], 1);
        fence_mbar_init();
    }
    __syncwarp();
    const int part = (int)blockIdx.x >= qblocks;
    const int blk = part ? blockIdx.x - qblocks : blockIdx.x, nblk = part ? gridDim.x - qblocks : qblocks;
    const int n = a.rot / 2, segs = part ? a.segs[1] : a.segs[0], seg0 = part ? a.segs[0] : 0;
    const long long ldx = part ? a.ldx[1] : a.ldx[0], ldy = part ? a.ldy[1] : a.ldy[0], lddy = part ? a.lddy[1] : a.lddy[0];
    const T *xb = static_cast<const T *>(part ? a.x[1] : a.x[0]);
    const T *gb = static_cast<const T *>(part ? a.dy[1] : a.dy[0]);
    T *yb = static_cast<T *>(part ? a.y[1] : a.y[0]);
    const float *w = part ? a.w[1] : a.w[0];
    int lo, hi;
    slot_place<V, INTER>(slot, n, lo, hi);
    const bool in = slot < a.D / (2 * V);
    griddep_wait();
    unsigned long long f[V];
    unsigned rotated = 0;
    if (in) slot_freq<V, INTER>(a, slot, f, rotated);
    float wl[V], wh[V], dl[V] = {}, dh[V] = {};
#pragma unroll
    for (int i = 0; i < V; ++i) wl[i] = wh[i] = 1.0f;
    if (w && in) load_weight<V>(w + lo, wl), load_weight<V>(w + hi, wh);
    const uint64_t policy = l2_policy(a.inv != 0.0f);
    Deal deal(a, seg0, segs, blk * SWARPS + warp, (long long)nblk * SWARPS), ahead = deal;
    long long mypos = 0;
    auto fetch = [&](long long i, int st) {
        if (i >= deal.count) return;
        const Item m = ahead.next(a);
        if (n && lane == st) mypos = a.pos[m.token];
        if (lane == 0) {
            const uint32_t bytes = (uint32_t)(m.rows * a.D * sizeof(T));
            mbar_arrive_tx(&full[warp][st], 2 * bytes);
            bulk_in(buf + st * STRIDE, xb + m.token * ldx + m.place, bytes, &full[warp][st], policy);
            bulk_in(buf + st * STRIDE + DY, gb + m.token * lddy + m.place, bytes, &full[warp][st], policy);
        }
    };
#pragma unroll
    for (int i = 0; i < STAGES; ++i) fetch(i, i);
    int st = 0, phase = 0;
    long long token = -1;
    float c[V], s[V];
    for (long long it = 0; it < deal.count; ++it) {
        const Item m = deal.next(a);
        const long long pos = __shfl_sync(0xffffffffu, mypos, st);
        if (m.token != token) slot_angles<V>(a, f, rotated, pos, c, s);
        token = m.token;
        if (!copy_wait(&full[warp][st], phase, a.limit)) {
            copies_settle(full[warp], st, phase, (int)min(deal.count - it, it > 0 ? STAGES - 1ll : STAGES));
            break;
        }
        T *x = buf + st * STRIDE, *g = x + DY;
#pragma unroll 2
        for (int r0 = 0; r0 < m.rows; r0 += RP) {
            const int r = r0 + lane / G;
            const bool on = in && r < m.rows;
            float u[V] = {}, t[V] = {}, p[V] = {}, q[V] = {}, ss = 0.0f, sx = 0.0f;
            if (on) {
                X::widen(X::load(x + r * a.D + lo), u), X::widen(X::load(x + r * a.D + hi), t);
                X::widen(X::load(g + r * a.D + lo), p), X::widen(X::load(g + r * a.D + hi), q);
            }
            if (rotated) rotate<V, INTER>(p, q, c, s);   // dz
            float rs = 1.0f, k = 0.0f, pw[V], qw[V];
#pragma unroll
            for (int i = 0; i < V; ++i) pw[i] = p[i] * wl[i], qw[i] = q[i] * wh[i];
            if (a.inv != 0.0f) {
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    ss = fmaf(u[i], u[i], fmaf(t[i], t[i], ss));
                    sx = fmaf(pw[i], u[i], fmaf(qw[i], t[i], sx));
                }
                rs = rsqrtf(group_sum<G>(ss) * a.inv + a.eps);
                k = rs * rs * (group_sum<G>(sx) * a.inv);
            }
            if (on) {
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float xa = u[i] * rs, xb = t[i] * rs;
                    dl[i] = fmaf(p[i], xa, dl[i]);
                    dh[i] = fmaf(q[i], xb, dh[i]);
                    u[i] = fmaf(-k, xa, rs * pw[i]);
                    t[i] = fmaf(-k, xb, rs * qw[i]);
                }
                X::store(x + r * a.D + lo, u);
                X::store(x + r * a.D + hi, t);
            }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
            bulk_out(yb + m.token * ldy + m.place, x, (uint32_t)(m.rows * a.D * sizeof(T)), policy);
            bulk_commit();
            if (it > 0) bulk_wait_read_but_1();
        }
        __syncwarp();
        if (it > 0) fetch(it + STAGES - 1, st == 0 ? STAGES - 1 : st - 1);
        if (++st == STAGES) st = 0, phase ^= 1;
    }
    if (lane == 0) bulk_wait_all();
    if (!(part ? a.want_dw[1] : a.want_dw[0])) return;
    __syncthreads();                                   // every warp's ring is at rest
    float *red = reinterpret_cast<float *>(ring);      // [SWARPS * RP][D]
    if (in)
#pragma unroll
        for (int i = 0; i < V; ++i) {
            red[(warp * RP + lane / G) * a.D + lo + i] = dl[i];
            red[(warp * RP + lane / G) * a.D + hi + i] = dh[i];
        }
    __syncthreads();
    for (int d = threadIdx.x; d < a.D; d += SWARPS * 32) {
        float v = 0.0f;
        for (int g = 0; g < SWARPS * RP; ++g) v += red[g * a.D + d];
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
int vec_width(int D, int rot, bool inter, const long long *lds, int nld) {
    for (int V = 4; V > 1; V /= 2) {
        bool ok = D % (2 * V) == 0 && (inter ? rot % (2 * V) == 0 : (rot / 2) % V == 0);
        for (int i = 0; i < nld; ++i) ok = ok && lds[i] % V == 0;
        if (ok) return V;
    }
    return 1;
}

// Heads of an item: as many as fill it, their bytes a multiple of 16.
int item_heads(int limit, int row_bytes) {
    int unit = 1;
    while (unit * row_bytes % 16) unit *= 2;
    return limit / row_bytes / unit * unit;
}

// Blocks of queries and of keys in the proportion of their work.
void share_blocks(long long wq, long long wk, long long most, long long &qb, long long &kb) {
    qb = wq, kb = wk;
    if (wq + wk <= most) return;
    qb = wq ? most * wq / (wq + wk) : 0;
    if (wq && qb < 1) qb = 1;
    if (wk && qb > most - 1) qb = most - 1;
    kb = wk ? most - qb : 0;
}

cudaError_t launch_dw(const RotArgs &a, long long qb, long long kb, float *dwq, float *dwk, cudaStream_t st) {
    return launch_pdl(rotary_dw_kernel, dim3((a.D + 7) / 8, 2), 256, 0, st, (const float *)a.partial, (int)qb, (int)(qb + kb), a.D,
                      dwq, dwk);
}

template <typename T, int G, bool INTER>
cudaError_t run_stream(RotArgs &a, bool backward, float *dwq, float *dwk, cudaStream_t st) {
    for (int p = 0; p < 2; ++p) a.segs[p] = (a.heads[p] + a.per - 1) / a.per;
    const size_t smem = (size_t)SWARPS * STAGES * (backward ? 2 * BWD_ITEM : FWD_ITEM);
    cudaError_t e;
    if (!backward) {
        e = cudaFuncSetAttribute(rotary_stream_fwd_kernel<T, G, INTER>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
        const long long blocks = (a.T * (a.segs[0] + a.segs[1]) + SWARPS - 1) / SWARPS;
        return launch_pdl(rotary_stream_fwd_kernel<T, G, INTER>, dim3((unsigned)(blocks < 304 ? blocks : 304)), SWARPS * 32, smem,
                          st, a);
    }
    e = cudaFuncSetAttribute(rotary_stream_bwd_kernel<T, G, INTER>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    long long qb, kb;
    share_blocks((a.T * a.segs[0] + SWARPS - 1) / SWARPS, (a.T * a.segs[1] + SWARPS - 1) / SWARPS, 304, qb, kb);
    e = launch_pdl(rotary_stream_bwd_kernel<T, G, INTER>, dim3((unsigned)(qb + kb)), SWARPS * 32, smem, st, a, (int)qb);
    return e == cudaSuccess && (dwq || dwk) ? launch_dw(a, qb, kb, dwq, dwk, st) : e;
}

template <typename T, int V, int G, bool INTER>
cudaError_t run_group(RotArgs &a, bool backward, float *dwq, float *dwk, cudaStream_t st) {
    constexpr int NG = RT / G;
    if constexpr (V == 4)
        if (a.stream) return run_stream<T, G, INTER>(a, backward, dwq, dwk, st);
    // heads per group: four, all in flight; fewer where the call is too small
    // to fill the SMs (152 x 1024 lanes), down to one
    a.per = ROWS;
    while (a.per > 1 && a.T * ((a.heads[0] + a.heads[1]) / a.per) * G < 152 * 1024) a.per /= 2;
    for (int p = 0; p < 2; ++p) a.segs[p] = (a.heads[p] + a.per - 1) / a.per;
    if (!backward) {
        const long long groups = a.T * (a.segs[0] + a.segs[1]);
        return launch_pdl(rotary_fwd_kernel<T, V, G, INTER>, dim3((unsigned)((groups + NG - 1) / NG)), RT, 0, st, a);
    }
    long long qb, kb;
    share_blocks((a.T * a.segs[0] + NG - 1) / NG, (a.T * a.segs[1] + NG - 1) / NG, BWD_BLOCKS, qb, kb);
    const cudaError_t e =
        launch_pdl(rotary_bwd_kernel<T, V, G, INTER>, dim3((unsigned)(qb + kb)), RT, sizeof(float) * NG * a.D, st, a, (int)qb);
    return e == cudaSuccess && (dwq || dwk) ? launch_dw(a, qb, kb, dwq, dwk, st) : e;
}

template <typename T, int V, bool INTER>
cudaError_t run_vec(RotArgs &a, bool backward, float *dwq, float *dwk, cudaStream_t st) {
    const int lanes = (a.D / (2 * V) + SLOTS<V> - 1) / SLOTS<V>;
    // odd sizes (V of 1 or 2) take whole warps; else the least power of two
    if constexpr (V == 4) {
        if (lanes <= 8) return run_group<T, V, 8, INTER>(a, backward, dwq, dwk, st);
        if (lanes <= 16) return run_group<T, V, 16, INTER>(a, backward, dwq, dwk, st);
    }
    return run_group<T, V, 32, INTER>(a, backward, dwq, dwk, st);
}

template <typename T>
cudaError_t run_type(RotArgs &a, bool inter, const long long *lds, int nld, bool backward, float *dwq, float *dwk, cudaStream_t st) {
    const int V = vec_width(a.D, a.rot, inter, lds, nld);
    // Streaming needs 16-byte pitches and head groups, and enough rows to run
    // the rings
    a.want_dw[0] = dwq != nullptr;
    a.want_dw[1] = dwk != nullptr;
    const int row = a.D * (int)sizeof(T);
    bool ok = V == 4 && a.T * (a.heads[0] + a.heads[1]) * row >= (backward ? STREAM_BWD : a.inv != 0.0f ? STREAM_FWD : STREAM_TURN);
    for (int i = 0; i < nld; ++i) ok = ok && lds[i] * (long long)sizeof(T) % 16 == 0;
    for (int p = 0; p < 2; ++p) ok = ok && (long long)a.heads[p] * row % 16 == 0;
    a.stream = ok;
    if (ok) a.per = item_heads(backward ? BWD_ITEM : FWD_ITEM, row);
#define S5_ROT(VV) \
    return inter ? run_vec<T, VV, true>(a, backward, dwq, dwk, st) : run_vec<T, VV, false>(a, backward, dwq, dwk, st)
    if (V == 4) S5_ROT(4);
    if (V == 2) S5_ROT(2);
    S5_ROT(1);
#undef S5_ROT
}

std::atomic<unsigned long long> wait_limit{2000000000ull};

cudaError_t run(RotArgs &a, s5_dtype dtype, bool inter, const long long *lds, int nld, bool backward, float *dwq, float *dwk,
                cudaStream_t st) {
    a.limit = wait_limit.load(std::memory_order_relaxed);
    return dtype == S5_BF16 ? run_type<__nv_bfloat16>(a, inter, lds, nld, backward, dwq, dwk, st)
                            : run_type<float>(a, inter, lds, nld, backward, dwq, dwk, st);
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
    if (H > 1 << 30 || T > (1ll << 31) / (H > 0 ? H : 1)) return S5_ERR_UNSUPPORTED;
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
    const int nld = 2;
    cudaStream_t st = (cudaStream_t)stream;
    const cudaError_t e = run(a, dtype, inter, lds, nld, false, nullptr, nullptr, st);
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
    a.inv = norm == S5_NORM_RMS ? 1.0f / D : norm == S5_NORM_L2 ? 1.0f : 0.0f;
    a.eps = eps, a.amp = amplitude, a.turn = 1.0f;
    const long long lds[4] = {Hq ? ldq : 0, Hk ? ldk : 0, Hq ? ldqo : 0, Hk ? ldko : 0};
    const bool inter = layout == S5_ROTARY_INTERLEAVED;
    const int nld = 4;
    cudaStream_t st = (cudaStream_t)stream;
    const cudaError_t e = run(a, dtype, inter, lds, nld, false, nullptr, nullptr, st);
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
    a.inv = norm == S5_NORM_RMS ? 1.0f / D : norm == S5_NORM_L2 ? 1.0f : 0.0f;
    a.eps = eps, a.amp = amplitude, a.turn = -1.0f;
    a.partial = static_cast<float *>(workspace);
    const long long lds[6] = {Hq ? ldq : 0,  Hk ? ldk : 0,  Hq ? lddqo : 0,
                              Hk ? lddko : 0, Hq ? lddq : 0, Hk ? lddk : 0};
    const bool inter = layout == S5_ROTARY_INTERLEAVED;
    const int nld = 6;
    const cudaError_t e = run(a, dtype, inter, lds, nld, true, dq_weight, dk_weight, st);
    return e == cudaSuccess ? S5_OK : cuda_failure(e);
}

extern "C" unsigned long long s5_rotary_wait_limit(unsigned long long ns) { return wait_limit.exchange(ns); }

extern "C" int s5_rotary_fault(void) {
    int v = 0, zero = 0;
    if (cudaDeviceSynchronize() != cudaSuccess) return -1;       // a copy alone waits for no stream that does not block
    if (cudaMemcpyFromSymbol(&v, g_rotary_fault, sizeof(int)) != cudaSuccess) return -1;
    if (v && cudaMemcpyToSymbol(g_rotary_fault, &zero, sizeof(int)) != cudaSuccess) return -1;
    return v;
}
