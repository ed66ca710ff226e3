// s5_gated_scan.cu -- the gated linear recurrence of each channel: whole
// sequences, their backward pass, one token.
//
//   r = sigmoid(gate_a),  la = -rate r,  a = exp(la)   (0 at a reset)
//   n = sqrt(1 - a^2)  (or 1),  u = sigmoid(gate_x) x  (or x)
//   h_t = a_t h_{t-1} + n_t u_t
// and, with G_t = dh_t + a_{t+1} G_{t+1}:
//   dla = G (a h_{t-1} - a^2/n u),  drate = -sum dla r,  dgate_a = -rate dla r (1 - r)
//   dx = G n s,  dgate_x = G n x s (1 - s)  (s = sigmoid(gate_x)).
//
// A run of tokens maps a state h to A h + E, and two runs join as (A2 A1,
// A2 E1 + E2).  A block takes a tile of tokens of some channels; its lanes hold
// V channels of S consecutive tokens each, fold them to one pair per lane, and
// the tile's 8 or 16 pairs of a channel are folded by one thread.  A cluster of
// blocks takes consecutive tiles of the same channels at once: each sends its
// tile's pair to all the others' shared memory, and after one cluster barrier
// each folds the pairs before it.  So a sequence is read once and written once,
// no block waits for one that may not run, nothing is kept in global memory
// between tiles, and the order of every sum is fixed.  The next tile is on its
// way into shared memory meanwhile.
//
// The backward pass walks the tiles from the last to the first with the same
// pairs (A, Z) for G, and works the states out again inside a tile from one that
// the forward pass kept every 64 tokens in 32 bits: reading h would cost twice
// the bytes of a 16-bit state and its rounding.
//
// 1 - a and 1 - a^2 come from m = exp(la) - 1, a short series where a is near
// one: a channel that forgets over thousands of tokens keeps the digits of both.
#include "s5_rows.cuh"
#include "s5_sm100.cuh"

namespace s5 {
namespace {
using namespace rows;
using sm100::smem_addr;

constexpr int THREADS = 256;
constexpr int KEEP = 64;        // tokens between two kept states
constexpr int MAX_CLUSTER = 8;

struct ScanArgs {
    const void *x, *ga, *gx;            // gx null: u = x
    long long ldx, ldga, ldgx;
    const float *rate;                  // [C]
    const float *h0;                    // [B][C] or null
    const unsigned char *reset;         // [B][L] or null
    const int *lengths;                 // [B] or null
    int B, L, C;
    bool normalize;
    void *h;
    long long ldh;
    float *h_last;                      // [B][C] or null
    float *states;                      // [B][N][C] or null: the state before token 64 i
    // backward
    const void *dh;
    long long lddh;
    const float *dh_last;               // or null
    void *dx, *dga, *dgx;
    long long lddx, lddga, lddgx;
    float *drate;                       // [parts][C]
    float *dh0;                         // or null
    int cluster, rounds;                // tiles at once, and how often
};

// A run that holds a reset has A = 0 and takes nothing over, not even NaN: zeros stay zeros whatever they are joined
// with, and a pair applied to a state.
__device__ __forceinline__ float join(float A, float a) { return A == 0.0f || a == 0.0f ? 0.0f : A * a; }
__device__ __forceinline__ float apply(float A, float h, float E) { return A == 0.0f ? E : fmaf(A, h, E); }

// a = exp(z) and 1 - a^2 for z <= 0.  Above -1/4 the series of exp(z) - 1 up to z^6 (the rest is below 2^-23 of it).
__device__ __forceinline__ void decay(float z, float &a, float &n2) {
    float q = fmaf(z, 1.0f / 720, 1.0f / 120);
    q = fmaf(z, q, 1.0f / 24);
    q = fmaf(z, q, 1.0f / 6);
    q = fmaf(z, q, 0.5f);
    const float near = fmaf(z * z, q, z), far = ex2(LOG2E * z);
    const bool close = z > -0.25f;
    const float m = close ? near : far - 1.0f;
    a = close ? 1.0f + near : far;
    n2 = -m * (2.0f + m);
}
// sqrt(n2) and 1 / sqrt(n2), both 0 at 0.
__device__ __forceinline__ void root(float n2, float &n, float &inv) {
    const float s = rsqrt_(fmaxf(n2, 1e-37f));
    n = n2 * s;
    inv = n2 > 0.0f ? s : 0.0f;
}

__device__ __forceinline__ void cp_async16(void *dst, const void *src, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(dst)), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group 0;" ::: "memory"); }

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// A pair into block `rank`'s copy of this block's shared variable.
__device__ __forceinline__ void send(float2 *p, unsigned rank, float2 v) {
    unsigned at;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_addr(p)), "r"(rank));
    asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(at), "f"(v.x), "f"(v.y) : "memory");
}

// How a block's threads share a tile: LANES threads side by side hold V
// channels each, and GROUPS such rows S consecutive tokens each.
template <typename T_, int V_, int LANES_, int S_, int ARRAYS_, bool ASYNC_> struct Shape {
    using T = T_;
    static constexpr int V = V_, LANES = LANES_, S = S_, ARRAYS = ARRAYS_;
    static constexpr bool ASYNC = ASYNC_;                     // tiles come by 16-byte copies, one ahead
    static constexpr int GROUPS = THREADS / LANES, WIDE = LANES * V, TILE = GROUPS * S;
    static constexpr int STAGE = ASYNC ? ARRAYS * TILE * WIDE * (int)sizeof(T) : 0;
    static constexpr int PAIRS = MAX_CLUSTER * WIDE;          // of a round
    static constexpr int SMEM = 2 * STAGE + 2 * PAIRS * (int)sizeof(float2) + (ARRAYS == 4 ? 3 : 2) * GROUPS * WIDE * (int)sizeof(float);
    static_assert(TILE % KEEP == 0 && KEEP % S == 0, "kept states lie at a group's start");
};

// A block's place: its sequence, channels and rank, and the arrays in its shared memory.
template <typename Sh> struct Block {
    using T = typename Sh::T;
    T *stage[2];
    float2 *pairs;      // [2][MAX_CLUSTER][WIDE]
    float *A, *E, *Z;   // [GROUPS][WIDE] (Z: backward)
    int b, c0, rank, lane, group, c;
    int len;            // tokens of this sequence
    __device__ Block(const ScanArgs &p, unsigned char *smem) {
        stage[0] = reinterpret_cast<T *>(smem);
        stage[1] = reinterpret_cast<T *>(smem + Sh::STAGE);
        pairs = reinterpret_cast<float2 *>(smem + 2 * Sh::STAGE);
        A = reinterpret_cast<float *>(pairs + 2 * Sh::PAIRS);
        E = A + Sh::GROUPS * Sh::WIDE;
        Z = E + Sh::GROUPS * Sh::WIDE;
        const int K = p.cluster, across = (p.C + Sh::WIDE - 1) / Sh::WIDE;
        rank = blockIdx.x % K;
        const int chain = blockIdx.x / K;
        b = chain / across;
        c0 = chain % across * Sh::WIDE;
        lane = threadIdx.x % Sh::LANES;
        group = threadIdx.x / Sh::LANES;
        c = c0 + lane * Sh::V;
    }
    __device__ void read_length(const ScanArgs &p) { len = p.lengths ? min(max(p.lengths[b], 0), p.L) : p.L; }
    // Copies of tile t0 of the given arrays into a stage: rows of WIDE values one after the other, zeros where there is nothing to read.
    __device__ void fetch(const ScanArgs &p, int which, int t0, const void *const *from, const long long *ld) {
        constexpr int PER = 16 / sizeof(T), CHUNKS = Sh::WIDE / PER, ROWS = THREADS / CHUNKS;
        const int chunk = threadIdx.x % CHUNKS, row = threadIdx.x / CHUNKS, at = c0 + chunk * PER;
#pragma unroll
        for (int k = 0; k < Sh::ARRAYS; ++k) {
            if (!from[k]) continue;
            const T *src = static_cast<const T *>(from[k]) + ((long long)b * p.L + t0 + row) * ld[k] + at;
            T *dst = stage[which] + (k * Sh::TILE + row) * Sh::WIDE + chunk * PER;
#pragma unroll
            for (int i = 0; i < Sh::TILE / ROWS; ++i) {
                const bool there = t0 + row + i * ROWS < len && at < p.C;
                cp_async16(dst + i * ROWS * Sh::WIDE, there ? src + (long long)i * ROWS * ld[k] : from[k], there);
            }
        }
    }
    // V values of array k at this thread's token s of the tile.
    __device__ void load(const ScanArgs &p, int which, int t0, int s, int k, const void *const *from, const long long *ld,
                         float (&r)[Sh::V]) const {
        if constexpr (Sh::ASYNC) {
            Vec<T, Sh::V>::load(stage[which] + (k * Sh::TILE + group * Sh::S + s) * Sh::WIDE + lane * Sh::V, r);
        } else {
            const int t = t0 + group * Sh::S + s;
            if (t < len && c < p.C) {
                Vec<T, Sh::V>::load(static_cast<const T *>(from[k]) + ((long long)b * p.L + t) * ld[k] + c, r);
            } else {
#pragma unroll
                for (int v = 0; v < Sh::V; ++v) r[v] = 0.0f;
            }
        }
    }
    // Which of this thread's tokens of the tile are resets, a bit each.
    __device__ unsigned marks(const ScanArgs &p, int t0) const {
        unsigned m = 0;
        const int t = t0 + group * Sh::S;
        const unsigned char *at = p.reset + (long long)b * p.L + t;
#pragma unroll
        for (int s = 0; s < Sh::S; ++s)
            if (t + s < len && at[s]) m |= 1u << s;
        return m;
    }
    __device__ void rates(const ScanArgs &p, float (&rate)[Sh::V]) const {
#pragma unroll
        for (int v = 0; v < Sh::V; ++v) rate[v] = c + v < p.C ? p.rate[c + v] : 0.0f;
    }
};

template <int V> __device__ __forceinline__ void put_smem(float *p, const float (&r)[V]) { Vec<float, V>::store(p, r); }

template <typename Sh, bool GATED, bool MARKS>
__global__ void __launch_bounds__(THREADS, 2) gated_scan_fwd_kernel(const ScanArgs p) {
    using T = typename Sh::T;
    constexpr int V = Sh::V, S = Sh::S, W = Sh::WIDE;
    extern __shared__ __align__(128) unsigned char smem[];
    Block<Sh> k(p, smem);
    const int K = p.cluster;
    griddep_wait();
    k.read_length(p);
    const void *const from[3] = {p.x, p.ga, GATED ? p.gx : nullptr};
    const long long ld[3] = {p.ldx, p.ldga, p.ldgx};
    int t0 = k.rank * Sh::TILE;
    unsigned marks = 0;
    if (Sh::ASYNC) k.fetch(p, 0, t0, from, ld);
    if (Sh::ASYNC) cp_async_commit();
    if (K > 1) cluster_arrive();
    float rate[V];
    k.rates(p, rate);
    if (MARKS) marks = k.marks(p, t0);
    // the thread that folds channel c0 + threadIdx.x over the tile's groups
    const bool folds = threadIdx.x < W && k.c0 + (int)threadIdx.x < p.C;
    const int ch = k.c0 + threadIdx.x;
    float carry = folds && p.h0 ? p.h0[(long long)k.b * p.C + ch] : 0.0f;   // the state before this round's first tile
    if (K > 1) cluster_wait();   // all blocks run: their shared memory may be written

    for (int round = 0; round < p.rounds; ++round, t0 += K * Sh::TILE) {
        const int now = round & 1;
        unsigned ahead = 0;
        if (Sh::ASYNC) {
            cp_async_wait();
            __syncthreads();
            if (round + 1 < p.rounds) k.fetch(p, 1 - now, t0 + K * Sh::TILE, from, ld);
            cp_async_commit();
        }
        if (MARKS && round + 1 < p.rounds) ahead = k.marks(p, t0 + K * Sh::TILE);
        const int mine = t0 + k.group * S;   // this thread's first token
        float a[S][V], e[S][V], A[V], E[V];
#pragma unroll
        for (int v = 0; v < V; ++v) A[v] = 1.0f, E[v] = 0.0f;
#pragma unroll
        for (int s = 0; s < S; ++s) {
            float x[V], ga[V], gx[V];
            k.load(p, now, t0, s, 0, from, ld, x);
            k.load(p, now, t0, s, 1, from, ld, ga);
            if (GATED) k.load(p, now, t0, s, 2, from, ld, gx);
            const bool fresh = MARKS && (marks >> s & 1);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float n2, n, inv;
                decay(-rate[v] * sigmoid(ga[v]), a[s][v], n2);
                root(n2, n, inv);
                if (!p.normalize) n = 1.0f;
                if (fresh) a[s][v] = 0.0f, n = 1.0f;
                e[s][v] = n * (GATED ? sigmoid(gx[v]) * x[v] : x[v]);
            }
        }
        if (t0 + Sh::TILE > k.len) {         // tokens past the end leave the state as it is
#pragma unroll
            for (int s = 0; s < S; ++s)
                if (mine + s >= k.len) {
#pragma unroll
                    for (int v = 0; v < V; ++v) a[s][v] = 1.0f, e[s][v] = 0.0f;
                }
        }
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const bool fresh = MARKS && (marks >> s & 1);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                A[v] = MARKS ? join(A[v], a[s][v]) : A[v] * a[s][v];
                E[v] = fresh ? e[s][v] : fmaf(a[s][v], E[v], e[s][v]);
            }
        }
        put_smem(k.A + k.group * W + k.lane * V, A);
        put_smem(k.E + k.group * W + k.lane * V, E);
        __syncthreads();
        float before = carry;
        if (K > 1) {
            float2 *slot = k.pairs + (now * MAX_CLUSTER + k.rank) * W + threadIdx.x;
            if (threadIdx.x < W) {
                float2 all = make_float2(1.0f, 0.0f);
#pragma unroll
                for (int g = 0; g < Sh::GROUPS; ++g) {
                    const float Ag = k.A[g * W + threadIdx.x];
                    all = make_float2(join(Ag, all.x), apply(Ag, all.y, k.E[g * W + threadIdx.x]));
                }
                for (int j = 0; j < K; ++j) send(slot, j, all);
            }
            cluster_arrive();
            cluster_wait();
            if (threadIdx.x < W)
                for (int j = 0; j < K; ++j) {
                    const float2 q = k.pairs[(now * MAX_CLUSTER + j) * W + threadIdx.x];
                    if (j == k.rank) before = carry;
                    carry = apply(q.x, carry, q.y);
                }
        }
        if (threadIdx.x < W) {               // the state before each group, in E's place
#pragma unroll
            for (int g = 0; g < Sh::GROUPS; ++g) {
                const float Ag = k.A[g * W + threadIdx.x], Eg = k.E[g * W + threadIdx.x];
                k.E[g * W + threadIdx.x] = before;
                if (g * S % KEEP == 0 && p.states && folds && t0 + g * S < p.L)
                    p.states[((long long)k.b * ((p.L + KEEP - 1) / KEEP) + (t0 + g * S) / KEEP) * p.C + ch] = before;
                before = apply(Ag, before, Eg);
            }
            if (K == 1) carry = before;
        }
        __syncthreads();
        float h[V];
        Vec<float, V>::load(k.E + k.group * W + k.lane * V, h);
        T *out = static_cast<T *>(p.h) + ((long long)k.b * p.L + mine) * p.ldh + k.c;
        const bool ragged = t0 + Sh::TILE > k.len;
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const bool fresh = MARKS && (marks >> s & 1);
#pragma unroll
            for (int v = 0; v < V; ++v) h[v] = fresh ? e[s][v] : fmaf(a[s][v], h[v], e[s][v]);
            if (mine + s < p.L && k.c < p.C) {
                if (ragged && mine + s >= k.len) {
                    const float zero[V] = {};
                    Vec<T, V>::store(out + s * p.ldh, zero);
                } else {
                    Vec<T, V>::store(out + s * p.ldh, h);
                }
            }
        }
        marks = ahead;
    }
    if (k.rank == 0 && folds && p.h_last) p.h_last[(long long)k.b * p.C + ch] = carry;
}

template <typename Sh, bool GATED, bool MARKS>
__global__ void __launch_bounds__(THREADS, 2) gated_scan_bwd_kernel(const ScanArgs p) {
    using T = typename Sh::T;
    constexpr int V = Sh::V, S = Sh::S, W = Sh::WIDE;
    extern __shared__ __align__(128) unsigned char smem[];
    Block<Sh> k(p, smem);
    const int K = p.cluster, N = (p.L + KEEP - 1) / KEEP;
    griddep_wait();
    k.read_length(p);
    const void *const from[4] = {p.x, p.ga, p.dh, GATED ? p.gx : nullptr};
    const long long ld[4] = {p.ldx, p.ldga, p.lddh, p.ldgx};
    int t0 = ((p.rounds - 1) * K + k.rank) * Sh::TILE;   // from the last tiles to the first
    unsigned marks = 0;
    if (Sh::ASYNC) k.fetch(p, 0, t0, from, ld);
    if (Sh::ASYNC) cp_async_commit();
    if (K > 1) cluster_arrive();
    float rate[V], drate[V];
    k.rates(p, rate);
#pragma unroll
    for (int v = 0; v < V; ++v) drate[v] = 0.0f;
    if (MARKS) marks = k.marks(p, t0);
    // threads 0 .. W - 1 fold the adjoints of a channel, the next W its states
    const int col = threadIdx.x % W, ch = k.c0 + col;
    const bool folds = threadIdx.x < W, forward = threadIdx.x / W == 1;
    float carry = folds && ch < p.C && p.dh_last ? p.dh_last[(long long)k.b * p.C + ch] : 0.0f;   // a G of what follows
    if (K > 1) cluster_wait();

    for (int round = 0; round < p.rounds; ++round, t0 -= K * Sh::TILE) {
        const int now = round & 1;
        unsigned ahead = 0;
        if (Sh::ASYNC) {
            cp_async_wait();
            __syncthreads();
            if (round + 1 < p.rounds) k.fetch(p, 1 - now, t0 - K * Sh::TILE, from, ld);
            cp_async_commit();
        }
        if (MARKS && round + 1 < p.rounds) ahead = k.marks(p, t0 - K * Sh::TILE);
        float state = 0.0f;                  // before the tile
        if (forward && ch < p.C && t0 < p.L) state = p.states[((long long)k.b * N + t0 / KEEP) * p.C + ch];
        const int mine = t0 + k.group * S;
        const bool ragged = t0 + Sh::TILE > k.len;
        // per value: a, r, the sigmoid s, n s, and a h - a^2/n u once h is there
        float a[S][V], r[S][V], g[S][V], ns[S][V], D[S][V], A[V], E[V], Z[V];
#pragma unroll
        for (int v = 0; v < V; ++v) A[v] = 1.0f, E[v] = 0.0f, Z[v] = 0.0f;
#pragma unroll
        for (int s = 0; s < S; ++s) {
            float x[V], ga[V], gx[V];
            k.load(p, now, t0, s, 0, from, ld, x);
            k.load(p, now, t0, s, 1, from, ld, ga);
            if (GATED) k.load(p, now, t0, s, 3, from, ld, gx);
            const bool fresh = MARKS && (marks >> s & 1), none = ragged && mine + s >= k.len;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float n2, n, inv;
                r[s][v] = sigmoid(ga[v]);
                decay(-rate[v] * r[s][v], a[s][v], n2);
                root(n2, n, inv);
                if (!p.normalize) n = 1.0f, inv = 0.0f;
                if (fresh) a[s][v] = 0.0f, n = 1.0f;
                if (none) a[s][v] = 1.0f, n = 0.0f, inv = 0.0f;
                g[s][v] = GATED ? sigmoid(gx[v]) : 1.0f;
                ns[s][v] = n * g[s][v];
                D[s][v] = a[s][v] * a[s][v] * inv * (g[s][v] * x[v]);
                A[v] = MARKS ? join(A[v], a[s][v]) : A[v] * a[s][v];
                const float e = ns[s][v] * x[v];
                E[v] = fresh ? e : fmaf(a[s][v], E[v], e);
            }
        }
#pragma unroll
        for (int s = S - 1; s >= 0; --s) {
            float dh[V];
            k.load(p, now, t0, s, 2, from, ld, dh);
            const bool fresh = MARKS && (marks >> s & 1);
#pragma unroll
            for (int v = 0; v < V; ++v) Z[v] = fresh ? 0.0f : a[s][v] * (dh[v] + Z[v]);
        }
        put_smem(k.A + k.group * W + k.lane * V, A);
        put_smem(k.E + k.group * W + k.lane * V, E);
        put_smem(k.Z + k.group * W + k.lane * V, Z);
        __syncthreads();
        float after = carry;
        if (K > 1) {
            if (folds) {
                float2 all = make_float2(1.0f, 0.0f);
#pragma unroll
                for (int j = Sh::GROUPS - 1; j >= 0; --j) {
                    const float Aj = k.A[j * W + col];
                    all = make_float2(join(Aj, all.x), apply(Aj, all.y, k.Z[j * W + col]));
                }
                float2 *slot = k.pairs + (now * MAX_CLUSTER + k.rank) * W + col;
                for (int j = 0; j < K; ++j) send(slot, j, all);
            }
            cluster_arrive();
        }
        if (forward) {                       // the state before each group, in E's place
#pragma unroll
            for (int j = 0; j < Sh::GROUPS; ++j) {
                const float Ej = k.E[j * W + col];
                k.E[j * W + col] = state;
                state = apply(k.A[j * W + col], state, Ej);
            }
        }
        if (K > 1) {
            cluster_wait();
            if (folds)
                for (int j = K - 1; j >= 0; --j) {
                    const float2 q = k.pairs[(now * MAX_CLUSTER + j) * W + col];
                    if (j == k.rank) after = carry;
                    carry = apply(q.x, carry, q.y);
                }
        }
        if (folds) {                         // what arrives from after each group, in Z's place
#pragma unroll
            for (int j = Sh::GROUPS - 1; j >= 0; --j) {
                const float Zj = k.Z[j * W + col];
                k.Z[j * W + col] = after;
                after = apply(k.A[j * W + col], after, Zj);
            }
            if (K == 1) carry = after;
        }
        __syncthreads();
        float h[V], z[V];
        Vec<float, V>::load(k.E + k.group * W + k.lane * V, h);
        Vec<float, V>::load(k.Z + k.group * W + k.lane * V, z);
#pragma unroll
        for (int s = 0; s < S; ++s) {
            float x[V];
            k.load(p, now, t0, s, 0, from, ld, x);
            const bool fresh = MARKS && (marks >> s & 1), none = ragged && mine + s >= k.len;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float e = ns[s][v] * x[v];
                D[s][v] = fresh || none ? 0.0f : fmaf(a[s][v], h[v], -D[s][v]);
                h[v] = fresh ? e : fmaf(a[s][v], h[v], e);
            }
        }
        const long long row = (long long)k.b * p.L + mine;
        T *dx = static_cast<T *>(p.dx) + row * p.lddx + k.c, *dga = static_cast<T *>(p.dga) + row * p.lddga + k.c;
        T *dgx = GATED ? static_cast<T *>(p.dgx) + row * p.lddgx + k.c : nullptr;
#pragma unroll
        for (int s = S - 1; s >= 0; --s) {
            float x[V], dh[V], o1[V], o2[V], o3[V];
            k.load(p, now, t0, s, 2, from, ld, dh);
            if (GATED) k.load(p, now, t0, s, 0, from, ld, x);
            const bool fresh = MARKS && (marks >> s & 1);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float G = dh[v] + z[v];
                const float t = G * D[s][v] * r[s][v];       // dla r
                drate[v] -= t;
                o1[v] = G * ns[s][v];
                o2[v] = rate[v] * t * (r[s][v] - 1.0f);
                if (GATED) o3[v] = o1[v] * x[v] * (1.0f - g[s][v]);
                z[v] = fresh ? 0.0f : a[s][v] * G;
            }
            if (mine + s < p.L && k.c < p.C) {
                Vec<T, V>::store(dx + s * p.lddx, o1);
                Vec<T, V>::store(dga + s * p.lddga, o2);
                if (GATED) Vec<T, V>::store(dgx + s * p.lddgx, o3);
            }
        }
        marks = ahead;
    }
    if (k.rank == 0 && folds && ch < p.C && p.dh0) p.dh0[(long long)k.b * p.C + ch] = carry;
    // the rate's gradient over this block's tokens
    __syncthreads();
    put_smem(k.A + k.group * W + k.lane * V, drate);
    __syncthreads();
    if (folds && ch < p.C) {
        float sum = 0.0f;
#pragma unroll
        for (int j = 0; j < Sh::GROUPS; ++j) sum += k.A[j * W + col];
        p.drate[((long long)k.b * K + k.rank) * p.C + ch] = sum;
    }
}

// drate: the blocks' parts in their order, 8 sums side by side and then joined.
__global__ void __launch_bounds__(256) gated_scan_rate_kernel(const float *part, int parts, int C, float *drate) {
    __shared__ float sums[8][32];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    griddep_wait();
    float s = 0.0f;
    if (c < C)
        for (int i = w; i < parts; i += 8) s += part[(long long)i * C + c];
    sums[w][lane] = s;
    __syncthreads();
    if (w == 0 && c < C) {
#pragma unroll
        for (int i = 1; i < 8; ++i) s += sums[i][lane];
        drate[c] = s;
    }
}

// One token: a thread per V channels of a sequence.
template <typename T, int V>
__global__ void __launch_bounds__(128)
gated_scan_step_kernel(const T *x, const T *ga, const T *gx, const float *rate, bool normalize, long long total, int C, float *state,
                       T *h) {
    const long long i = ((long long)blockIdx.x * 128 + threadIdx.x) * V;
    griddep_wait();
    griddep_launch_dependents();
    if (i >= total) return;
    const int c = (int)(i % C);
    float xv[V], av[V], gv[V], rv[V], s[V];
    Vec<T, V>::load(x + i, xv);
    Vec<T, V>::load(ga + i, av);
    if (gx) Vec<T, V>::load(gx + i, gv);
    Vec<float, V>::load(rate + c, rv);
    Vec<float, V>::load(state + i, s);
#pragma unroll
    for (int v = 0; v < V; ++v) {
        float a, n2, n, inv;
        decay(-rv[v] * sigmoid(av[v]), a, n2);
        root(n2, n, inv);
        if (!normalize) n = 1.0f;
        s[v] = fmaf(a, s[v], n * (gx ? sigmoid(gv[v]) * xv[v] : xv[v]));
    }
    Vec<float, V>::store(state + i, s);
    Vec<T, V>::store(h + i, s);
}

// ------------------------------------------------------------------ launches
// Tiles at once: the cluster that ends first when `slots` blocks run side by
// side and every block of a wave works through its share of the tiles.
int choose_cluster(long long chains, int tiles, int slots) {
    int best = 1;
    long long cost = -1;
    for (int K = 1; K <= MAX_CLUSTER && K <= (tiles > 1 ? tiles : 1); K *= 2) {
        const long long t = (chains * K + slots - 1) / slots * ((tiles + K - 1) / K);
        if (cost < 0 || t < cost) best = K, cost = t;
    }
    return best;
}

template <typename Sh> cudaError_t place(ScanArgs &p, long long &blocks) {
    const int tiles = (p.L + Sh::TILE - 1) / Sh::TILE;
    const long long chains = (long long)p.B * ((p.C + Sh::WIDE - 1) / Sh::WIDE);
    p.cluster = choose_cluster(chains, tiles, 2 * SMS);
    p.rounds = (tiles + p.cluster - 1) / p.cluster;
    blocks = chains * p.cluster;
    return blocks > 0x7fffffffll ? cudaErrorInvalidValue : cudaSuccess;
}

template <typename Sh> cudaError_t run_fwd(ScanArgs &p, cudaStream_t st) {
    long long blocks;
    const cudaError_t e = place<Sh>(p, blocks);
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)blocks);
#define S5_RUN(GATED, MARKS) launch_big(gated_scan_fwd_kernel<Sh, GATED, MARKS>, grid, THREADS, Sh::SMEM, p.cluster, st, p)
    if (p.gx) return p.reset ? S5_RUN(true, true) : S5_RUN(true, false);
    return p.reset ? S5_RUN(false, true) : S5_RUN(false, false);
#undef S5_RUN
}

template <typename Sh> cudaError_t run_bwd(ScanArgs &p, float *drate, cudaStream_t st) {
    long long blocks;
    cudaError_t e = place<Sh>(p, blocks);
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)blocks);
    const int parts = p.B * p.cluster;
    if (parts == 1) p.drate = drate;
#define S5_RUN(GATED, MARKS) launch_big(gated_scan_bwd_kernel<Sh, GATED, MARKS>, grid, THREADS, Sh::SMEM, p.cluster, st, p)
    if (p.gx) e = p.reset ? S5_RUN(true, true) : S5_RUN(true, false);
    else e = p.reset ? S5_RUN(false, true) : S5_RUN(false, false);
#undef S5_RUN
    if (e != cudaSuccess || parts == 1) return e;
    return launch(gated_scan_rate_kernel, dim3((p.C + 31) / 32), 256, 0, 1, st, (const float *)p.drate, parts, p.C, drate);
}

// 16-byte copies where all rows allow them, else pairs of channels, else single ones.
int width(s5_dtype dtype, int C, std::initializer_list<long long> lds) {
    const int per = dtype == S5_BF16 ? 8 : 4;
    int w = C % per == 0 ? per : C % 2 == 0 ? 2 : 1;
    for (long long ld : lds) w = ld % per == 0 ? w : ld % 2 == 0 && w > 1 ? 2 : 1;
    return w;
}

s5_status check_scan(const ScanArgs &p, s5_dtype dtype) {
    if (!type_ok(dtype) || p.B < 0 || p.L < 0 || p.C < 1) return S5_ERR_INVALID_ARGUMENT;
    // the narrowest blocks, in the largest cluster, within a grid; parts within an int
    if ((long long)p.B * ((p.C + 15) / 16) > (1ll << 27)) return S5_ERR_UNSUPPORTED;
    if (p.L > (1 << 30)) return S5_ERR_UNSUPPORTED;
    return S5_OK;
}
s5_status check_scan_inputs(const ScanArgs &p) {
    if (!rows_ok(p.x, p.ldx, p.C) || !rows_ok(p.ga, p.ldga, p.C) || (p.gx && !rows_ok(p.gx, p.ldgx, p.C))) return S5_ERR_INVALID_ARGUMENT;
    if (!p.rate || !aligned(p.rate, 16) || !aligned(p.lengths, 4)) return S5_ERR_INVALID_ARGUMENT;
    return S5_OK;
}

}  // namespace
}  // namespace s5

using namespace s5;

extern "C" size_t s5_gated_scan_saved_size(int B, int L, int C) {
    ScanArgs p = {};
    p.B = B, p.L = L, p.C = C;
    if (check_scan(p, S5_F32) != S5_OK) return 0;
    return 256 + sizeof(float) * (size_t)B * ((L + KEEP - 1) / KEEP) * C;
}

extern "C" size_t s5_gated_scan_workspace_size(int B, int L, int C) {
    ScanArgs p = {};
    p.B = B, p.L = L, p.C = C;
    if (check_scan(p, S5_F32) != S5_OK) return 0;
    return 256 + sizeof(float) * (size_t)B * MAX_CLUSTER * C;
}

extern "C" s5_status s5_gated_scan_forward(const void *x, long long ldx, const void *gate_a, long long ldga, const void *gate_x,
                                           long long ldgx, s5_dtype dtype, const float *rate, const float *h0,
                                           const unsigned char *reset, const int *lengths, int normalize, int B, int L, int C,
                                           void *h, long long ldh, float *h_last, void *saved, size_t saved_bytes,
                                           s5_stream_t stream) {
    ScanArgs p = {};
    p.x = x, p.ga = gate_a, p.gx = gate_x, p.ldx = ldx, p.ldga = ldga, p.ldgx = gate_x ? ldgx : 0;
    p.rate = rate, p.h0 = h0, p.reset = reset, p.lengths = lengths, p.normalize = normalize != 0;
    p.B = B, p.L = L, p.C = C, p.h = h, p.ldh = ldh, p.h_last = h_last;
    s5_status c = check_scan(p, dtype);
    if (c != S5_OK) return c;
    if (!aligned(h0, 16) || !aligned(h_last, 16)) return S5_ERR_INVALID_ARGUMENT;
    if (saved && (!aligned(saved, 16) || saved_bytes < s5_gated_scan_saved_size(B, L, C))) return S5_ERR_INVALID_ARGUMENT;
    if (B == 0) return S5_OK;
    cudaStream_t st = (cudaStream_t)stream;
    if (L == 0) {   // the state stays as it is
        const size_t n = sizeof(float) * (size_t)B * C;
        cudaError_t e = cudaSuccess;
        if (h_last && h0 && h_last != h0) e = cudaMemcpyAsync(h_last, h0, n, cudaMemcpyDeviceToDevice, st);
        if (h_last && !h0) e = cudaMemsetAsync(h_last, 0, n, st);
        return e == cudaSuccess ? S5_OK : cuda_failure(e);
    }
    c = check_scan_inputs(p);
    if (c != S5_OK) return c;
    if (!rows_ok(h, ldh, C)) return S5_ERR_INVALID_ARGUMENT;
    p.states = static_cast<float *>(saved);
    const int w = width(dtype, C, {ldx, ldga, p.ldgx, ldh});
    cudaError_t e;
    if (dtype == S5_BF16)
        e = w == 8   ? run_fwd<Shape<__nv_bfloat16, 4, 16, 8, 3, true>>(p, st)
            : w == 2 ? run_fwd<Shape<__nv_bfloat16, 2, 16, 8, 3, false>>(p, st)
                     : run_fwd<Shape<__nv_bfloat16, 1, 32, 8, 3, false>>(p, st);
    else
        e = w == 4   ? run_fwd<Shape<float, 2, 16, 8, 3, true>>(p, st)
            : w == 2 ? run_fwd<Shape<float, 2, 16, 8, 3, false>>(p, st)
                     : run_fwd<Shape<float, 1, 32, 8, 3, false>>(p, st);
    return e == cudaSuccess ? S5_OK : cuda_failure(e);
}

extern "C" s5_status s5_gated_scan_backward(const void *x, long long ldx, const void *gate_a, long long ldga, const void *gate_x,
                                            long long ldgx, s5_dtype dtype, const float *rate, const unsigned char *reset,
                                            const int *lengths, int normalize, int B, int L, int C, const void *dh, long long lddh,
                                            const float *dh_last, const void *saved, size_t saved_bytes, void *dx, long long lddx,
                                            void *dgate_a, long long lddga, void *dgate_x, long long lddgx, float *drate,
                                            float *dh0, void *workspace, size_t workspace_bytes, s5_stream_t stream) {
    ScanArgs p = {};
    p.x = x, p.ga = gate_a, p.gx = gate_x, p.ldx = ldx, p.ldga = ldga, p.ldgx = gate_x ? ldgx : 0;
    p.rate = rate, p.reset = reset, p.lengths = lengths, p.normalize = normalize != 0;
    p.B = B, p.L = L, p.C = C;
    p.dh = dh, p.lddh = lddh, p.dh_last = dh_last, p.dx = dx, p.lddx = lddx, p.dga = dgate_a, p.lddga = lddga;
    p.dgx = dgate_x, p.lddgx = gate_x ? lddgx : 0, p.dh0 = dh0;
    s5_status c = check_scan(p, dtype);
    if (c != S5_OK) return c;
    if (!drate || !aligned(drate, 16) || !aligned(dh_last, 16) || !aligned(dh0, 16)) return S5_ERR_INVALID_ARGUMENT;
    cudaStream_t st = (cudaStream_t)stream;
    if (B == 0 || L == 0) {
        cudaError_t e = cudaMemsetAsync(drate, 0, sizeof(float) * C, st);
        const size_t n = sizeof(float) * (size_t)B * C;
        if (e == cudaSuccess && n && dh0 && dh_last && dh0 != dh_last) e = cudaMemcpyAsync(dh0, dh_last, n, cudaMemcpyDeviceToDevice, st);
        if (e == cudaSuccess && n && dh0 && !dh_last) e = cudaMemsetAsync(dh0, 0, n, st);
        return e == cudaSuccess ? S5_OK : cuda_failure(e);
    }
    c = check_scan_inputs(p);
    if (c != S5_OK) return c;
    if (!rows_ok(dh, lddh, C) || !rows_ok(dx, lddx, C) || !rows_ok(dgate_a, lddga, C) || (gate_x && !rows_ok(dgate_x, lddgx, C)))
        return S5_ERR_INVALID_ARGUMENT;
    if (!saved || !aligned(saved, 16) || saved_bytes < s5_gated_scan_saved_size(B, L, C)) return S5_ERR_INVALID_ARGUMENT;
    if (!workspace || !aligned(workspace, 16) || workspace_bytes < s5_gated_scan_workspace_size(B, L, C)) return S5_ERR_INVALID_ARGUMENT;
    p.states = static_cast<float *>(const_cast<void *>(saved));
    p.drate = static_cast<float *>(workspace);
    const int w = width(dtype, C, {ldx, ldga, p.ldgx, lddh, lddx, lddga, p.lddgx});
    cudaError_t e;
    if (dtype == S5_BF16)
        e = w == 8   ? run_bwd<Shape<__nv_bfloat16, 4, 16, 4, 4, true>>(p, drate, st)
            : w == 2 ? run_bwd<Shape<__nv_bfloat16, 2, 16, 4, 4, false>>(p, drate, st)
                     : run_bwd<Shape<__nv_bfloat16, 1, 32, 8, 4, false>>(p, drate, st);
    else
        e = w == 4   ? run_bwd<Shape<float, 2, 16, 4, 4, true>>(p, drate, st)
            : w == 2 ? run_bwd<Shape<float, 2, 16, 4, 4, false>>(p, drate, st)
                     : run_bwd<Shape<float, 1, 32, 8, 4, false>>(p, drate, st);
    return e == cudaSuccess ? S5_OK : cuda_failure(e);
}

namespace {
template <typename T>
cudaError_t run_step(const void *x, const void *ga, const void *gx, const float *rate, bool normalize, int B, int C, float *state,
                     void *h, cudaStream_t st) {
    const long long total = (long long)B * C;
    // four channels a thread, two or one where they do not divide or would leave SMs idle
    const int V = C % 4 == 0 && total >= 4 * 128 * SMS ? 4 : C % 2 == 0 ? 2 : 1;
    const dim3 grid((unsigned)((total / V + 127) / 128));
    const T *xs = static_cast<const T *>(x), *as = static_cast<const T *>(ga), *gs = static_cast<const T *>(gx);
    T *hs = static_cast<T *>(h);
    if (V == 4) return launch(gated_scan_step_kernel<T, 4>, grid, 128, 0, 1, st, xs, as, gs, rate, normalize, total, C, state, hs);
    if (V == 2) return launch(gated_scan_step_kernel<T, 2>, grid, 128, 0, 1, st, xs, as, gs, rate, normalize, total, C, state, hs);
    return launch(gated_scan_step_kernel<T, 1>, grid, 128, 0, 1, st, xs, as, gs, rate, normalize, total, C, state, hs);
}
}  // namespace

extern "C" s5_status s5_gated_scan_step(const void *x, const void *gate_a, const void *gate_x, s5_dtype dtype, const float *rate,
                                        int normalize, int B, int C, float *state, void *h, s5_stream_t stream) {
    if (!type_ok(dtype) || B < 0 || C < 1) return S5_ERR_INVALID_ARGUMENT;
    if ((long long)B * C > (1ll << 36)) return S5_ERR_UNSUPPORTED;
    if (B == 0) return S5_OK;
    for (const void *q : {x, gate_a, (const void *)rate, (const void *)state, (const void *)h})
        if (!q || !aligned(q, 16)) return S5_ERR_INVALID_ARGUMENT;
    if (!aligned(gate_x, 16)) return S5_ERR_INVALID_ARGUMENT;
    const cudaError_t e =
        dtype == S5_BF16
            ? run_step<__nv_bfloat16>(x, gate_a, gate_x, rate, normalize != 0, B, C, state, h, (cudaStream_t)stream)
            : run_step<float>(x, gate_a, gate_x, rate, normalize != 0, B, C, state, h, (cudaStream_t)stream);
    return e == cudaSuccess ? S5_OK : cuda_failure(e);
}
