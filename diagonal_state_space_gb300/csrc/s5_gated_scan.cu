// s5_gated_scan.cu -- the gated linear recurrence of each channel: whole
// sequences, their backward pass, one token.
//
//   r = sigmoid(gate_a),  la = -rate r,  a = exp(la)   (0 and a cut at a reset)
//   n = sqrt(1 - a^2)  (or 1),  u = sigmoid(gate_x) x  (or x)
//   h_t = a_t h_{t-1} + n_t u_t
// and, with G_t = dh_t + a_{t+1} G_{t+1}:
//   dla = G (a h_{t-1} - a^2/n u),  drate = -sum dla r,  dgate_a = -rate dla r (1 - r)
//   dx = G n s,  dgate_x = G n x s (1 - s)  (s = sigmoid(gate_x)).
//
// A run of tokens maps a state h to A h + E, and two runs join as (A2 A1,
// A2 E1 + E2).  A block takes a tile of tokens of some channels; its lanes hold
// V channels of S consecutive tokens each, fold them to one pair per lane, and
// shuffles join a warp's, and one thread a channel folds the four warps' pairs.  A
// cluster of blocks takes consecutive tiles of the same channels at once: each sends its
// tile's pair to all the others' shared memory, and folds the pairs before it
// once all have come.  So a sequence is read once and written once, no block
// waits for one that may not run, nothing is kept in global memory between
// tiles, and the order of every sum is fixed.  TMA brings the next tile into shared
// memory meanwhile; odd channels or pitches are read by plain loads instead.
//
// The backward pass walks the tiles from the last to the first with the same
// pairs (A, Z) for G, and works the states out again inside a tile from one that
// the forward pass kept every 32 tokens in 32 bits: reading h would cost twice
// the bytes of a 16-bit state and its rounding.
//
// 1 - a and 1 - a^2 come from m = exp(la) - 1, a short series where a is near
// one: a channel that forgets over thousands of tokens keeps the digits of both.
//
// Bound: nothing is full.  DRAM is busy 34 to 44 %, issue slots 54 to 59 %, the
// pipe of special functions (six a value with both gates and the root) 46 to
// 52 % forward and 24 % backward; a round is a chain of load, tile and exchange, four
// blocks an SM beside each other.  bf16: 16384 tokens of 2048 channels 67 us (4.0 TB/s), 4 x 2048 of
// 2560 with resets 50 us forward (3.4 TB/s) and 96 backward (3.1).  Three blocks
// an SM 74 us for the first, five 92, blocks of 256 threads 111 for 74 (before
// TMA); tiles by 16-byte copies 71.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <atomic>
#include <cfloat>

#include "s5_rows.cuh"
#include "s5_sm100.cuh"

namespace s5 {
namespace {
using namespace rows;
using sm100::smem_addr;

constexpr int KEEP = 32;        // tokens between two kept states, and of a tile backward (twice that forward)
constexpr int MAX_CLUSTER = 16; // beyond 8 a non-portable size

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
    float *states;                      // [B][N][C] or null: the state before token KEEP i
    // backward
    const void *dh;
    long long lddh;
    const float *dh_last;               // or null
    void *dx, *dga, *dgx;
    long long lddx, lddga, lddgx;
    float *drate;                       // [parts][C]
    float *dh0;                         // or null
    int cluster, rounds;                // tiles at once, and how often
    long long row[3], out_step;         // bytes between two rows of the outputs, and (forward) a round's tiles
};

// A run that holds a reset takes nothing over, not even NaN: its A is negative, which no product of decays is (one that
// vanishes is zero, and NaN stays NaN behind it), and stays so whatever it is joined with.
constexpr float CUT = -1.0f;
__device__ __forceinline__ float join(float A, float a) { return A < 0.0f || a < 0.0f ? CUT : A * a; }
__device__ __forceinline__ float apply(float A, float h, float E) { return A < 0.0f ? E : fmaf(A, h, E); }

// a = exp(z) and 1 - a^2 for z <= 0.  Above -1/4 the series of exp(z) - 1 up to z^6 (the rest is below 2^-23 of it).
template <int V> __device__ __forceinline__ void decay(const Many<V> &z, Many<V> &a, Many<V> &n2) {
    using M = Many<V>;
    M q, m, t;
#pragma unroll
    for (int i = 0; i < V; ++i)
        q[i] = fmaf(z[i], fmaf(z[i], fmaf(z[i], fmaf(z[i], 1.0f / 720, 1.0f / 120), 1.0f / 24), 1.0f / 6), 0.5f);
    const M near = fma(z * z, q, z);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const float far = ex2(LOG2E * z[i]);
        const bool close = z[i] > -0.25f;
        m[i] = close ? near[i] : far - 1.0f;
        a[i] = close ? 1.0f + near[i] : far;
        t[i] = -2.0f - m[i];
    }
    n2 = m * t;
}

__device__ __forceinline__ void cluster_arrive() { __syncwarp(); asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { __syncwarp(); asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// This block's shared address as block `rank` of the cluster has it; a pair stored there, counted by a barrier there.
__device__ __forceinline__ unsigned there(unsigned at, unsigned rank) {
    unsigned r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(at), "r"(rank));
    return r;
}
__device__ __forceinline__ void send(unsigned at, unsigned bar, float2 v) {
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1, %2}, [%3];" ::"r"(at), "f"(v.x),
                 "f"(v.y), "r"(bar)
                 : "memory");
}
__device__ int g_scan_fault = 0;     // a wait ran out
constexpr unsigned long long WAIT_NS = 2000000000ull, WAIT_AFTER_NS = 1000000ull;
// For a tile's copies or the cluster's pairs.  The other blocks run beside this one, so the wait ends; were it not to,
// the results would be wrong and said to be, and no later wait would take as long.
__device__ __noinline__ void wait_long(uint64_t *bar, unsigned parity) {
    const unsigned long long t0 = global_ns();
    const unsigned long long limit = *static_cast<volatile int *>(&g_scan_fault) ? WAIT_AFTER_NS : WAIT_NS;
    while (!sm100::mbar_try_wait_sleep(bar, parity, 100000))
        if (global_ns() - t0 > limit) {
            atomicExch(&g_scan_fault, 1);
            return;
        }
}

// The inputs as [B][L][C] in boxes of a tile: x, gate_a, then gate_x (forward) or dh and gate_x.
struct ScanMaps {
    CUtensorMap map[4];
};

// How a block's threads share a tile: LANES threads side by side hold V
// channels each, and GROUPS such rows S consecutive tokens each.
template <typename T_, int V_, int LANES_, int S_, int ARRAYS_, bool ASYNC_> struct Shape {
    static constexpr int THREADS = 128, BLOCKS = 4;          // of an SM
    // The thread that starts the copies: of the last warp, which folds nothing but, backward where a row is 64 channels, states.
    static constexpr int FETCHER = THREADS - 32;
    using T = T_;
    static constexpr int V = V_, LANES = LANES_, S = S_, ARRAYS = ARRAYS_;
    static constexpr bool ASYNC = ASYNC_;                     // tiles come by TMA
    static constexpr int GROUPS = THREADS / LANES, WARPS = THREADS / 32, WIDE = LANES * V, TILE = GROUPS * S;
    static constexpr int STAGE = ASYNC ? ARRAYS * TILE * WIDE * (int)sizeof(T) : 0;
    static constexpr int PAIRS = MAX_CLUSTER * WIDE;          // of a round
    static constexpr int STAGES = ARRAYS == 4 ? 2 : 1;        // backward a tile is read twice
    static constexpr int SMEM = STAGES * STAGE + 2 * PAIRS * (int)sizeof(float2) + 32 + (ARRAYS == 4 ? 4 : 3) * WARPS * WIDE * (int)sizeof(float);
    static_assert(TILE == KEEP || TILE == 2 * KEEP, "kept states lie at a group's start");
    static_assert(LANES * 2 == 32 || LANES == 32, "a warp holds one or two groups");
};

// A block's place: its sequence, channels and rank, and the arrays in its shared memory.
template <typename Sh> struct Block {
    using T = typename Sh::T;
    using M = Many<Sh::V>;
    static constexpr int V = Sh::V, S = Sh::S, W = Sh::WIDE;
    T *stage;           // [STAGES][ARRAYS][TILE][WIDE]
    float2 *pairs;      // [2][MAX_CLUSTER][WIDE]
    float *A, *E, *H, *Z;   // [WARPS][WIDE]: a warp's pairs, what enters it, and backward its adjoints' pairs
    uint64_t *bar;      // [2], one for each half of the pairs
    uint64_t *full;     // [STAGES]
    int b, c0, rank, lane, group, c;
    bool upper;         // the later of a warp's two groups
    int len;            // tokens of this sequence
    __device__ Block(const ScanArgs &p, unsigned char *smem) {
        stage = reinterpret_cast<T *>(smem);
        pairs = reinterpret_cast<float2 *>(smem + Sh::STAGES * Sh::STAGE);
        A = reinterpret_cast<float *>(pairs + 2 * Sh::PAIRS);
        E = A + Sh::WARPS * W;
        H = E + Sh::WARPS * W;
        Z = H + Sh::WARPS * W;
        bar = reinterpret_cast<uint64_t *>(smem + Sh::SMEM - 32);
        full = bar + 2;
        const int K = p.cluster, across = (p.C + W - 1) / W;
        rank = blockIdx.x % K;
        const int chain = blockIdx.x / K;
        b = chain / across;
        c0 = chain % across * W;
        lane = threadIdx.x % Sh::LANES;
        group = threadIdx.x / Sh::LANES;
        c = c0 + lane * V;
        upper = Sh::LANES == 32 || (threadIdx.x & 16);
    }
    __device__ void read_length(const ScanArgs &p) { len = p.lengths ? min(max(p.lengths[b], 0), p.L) : p.L; }
    static constexpr int MINE = Sh::TILE / Sh::WARPS;      // tokens of a warp
    // One thread: the tile at t0 of N arrays into a stage; what lies past the channels or the row's L tokens is zeros.
    template <int N> __device__ void fetch(const ScanMaps &maps, int which, int t0) const {
        sm100::mbar_arrive_tx(full + which, N * Sh::TILE * W * (unsigned)sizeof(T));
#pragma unroll
        for (int k = 0; k < N; ++k) sm100::tma_load_3d(stage + (which * Sh::ARRAYS + k) * Sh::TILE * W, &maps.map[k], c0, t0, b, full + which);
    }
    __device__ void arrived(int which, unsigned phase) const {
        if (!sm100::mbar_try_wait(full + which, phase)) wait_long(full + which, phase);
    }
    __device__ void open_copies() const {
        if (threadIdx.x == 0) {
            for (int i = 0; i < Sh::STAGES; ++i) sm100::mbar_init(full + i, 1);
            sm100::fence_mbar_init();
        }
        __syncthreads();
    }
    // V values of array k at this thread's token s of the tile.
    __device__ M load(const ScanArgs &p, int which, int t0, int s, int k, const void *const *from, const long long *ld) const {
        M r = M::all(0.0f);
        if constexpr (Sh::ASYNC) {
            Vec<T, V>::load(stage + ((which * Sh::ARRAYS + k) * Sh::TILE + group * S + s) * W + lane * V, r.v);
        } else {
            const int t = t0 + group * S + s;
            if (t < len && c < p.C) Vec<T, V>::load(static_cast<const T *>(from[k]) + ((long long)b * p.L + t) * ld[k] + c, r.v);
        }
        return r;
    }
    // Which of this thread's tokens of the tile are resets, a bit each, in two steps: the load is not waited for, and
    // all lanes of the warp take part in both.
    __device__ unsigned char reset_of(const ScanArgs &p, int t0) const {
        const int l = threadIdx.x & 31, t = t0 + threadIdx.x / 32 * MINE + l;
        return l < MINE && t < len ? p.reset[(long long)b * p.L + t] : 0;
    }
    __device__ static unsigned marks(unsigned char reset) {
        const unsigned m = __ballot_sync(0xffffffffu, reset);
        return Sh::LANES == 32 ? m : (threadIdx.x & 31) < 16 ? m & ((1u << S) - 1) : m >> S;
    }
    __device__ M rates(const ScanArgs &p) const {
        M r = M::all(0.0f);
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (c + v < p.C) r[v] = p.rate[c + v];
        return r;
    }
    // A warp's row of A, E or Z.
    __device__ void put(float *at, const M &r) const { Vec<float, V>::store(at + threadIdx.x / 32 * W + lane * V, r.v); }
    __device__ M get(const float *at) const {
        M r;
        Vec<float, V>::load(at + threadIdx.x / 32 * W + lane * V, r.v);
        return r;
    }
    // The values that the lane of the warp's other group holds for the same channels.
    __device__ static M other(const M &x) {
        M r;
#pragma unroll
        for (int v = 0; v < V; ++v) r[v] = __shfl_xor_sync(0xffffffffu, x[v], 16);
        return r;
    }
    // Two pairs joined and one applied, in full where resets may have left cuts.
    __device__ static M joined(bool resets, const M &a, const M &b) { return resets ? joined(a, b) : a * b; }
    __device__ static M applied(bool resets, const M &a, const M &h, const M &e) { return resets ? applied(a, h, e) : fma(a, h, e); }
    __device__ static M joined(const M &a, const M &b) {
        M r;
#pragma unroll
        for (int v = 0; v < V; ++v) r[v] = join(a[v], b[v]);
        return r;
    }
    __device__ static M applied(const M &a, const M &h, const M &e) {
        M r;
#pragma unroll
        for (int v = 0; v < V; ++v) r[v] = apply(a[v], h[v], e[v]);
        return r;
    }
    // The cluster's barriers; afterwards all blocks run, and their shared memory may be written.
    __device__ void open_cluster(const ScanArgs &p) {
        if (threadIdx.x == 0) {
            for (int i = 0; i < 2; ++i) sm100::mbar_init(bar + i, 1);
            sm100::fence_mbar_init();
            for (int i = 0; i < 2 && i < p.rounds; ++i) sm100::mbar_arrive_tx(bar + i, p.cluster * W * sizeof(float2));
        }
        cluster_arrive();
    }
    // All blocks' pairs of this round to all blocks.  carry, what enters the round, becomes what leaves it; returned is
    // what enters this block's tile.  From the tile's rows of A and `e`, folded downwards backward.  Threads below W;
    // the others only help to send.  A block sends its pairs of round r + 2 after it has read those of round r + 1, for
    // which this one has sent its own, after reading round r: no half is overwritten before it is read.
    template <bool DOWN> __device__ float exchange(const ScanArgs &p, int round, const float *e, float &carry) {
        const int K = p.cluster, col = threadIdx.x % W, now = round & 1;
        const bool resets = p.reset;
        float2 all = make_float2(1.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < Sh::WARPS; ++i) {
            const int j = DOWN ? Sh::WARPS - 1 - i : i;
            const float Aj = A[j * W + col], Ej = e[j * W + col];
            all = resets ? make_float2(join(Aj, all.x), apply(Aj, all.y, Ej)) : make_float2(Aj * all.x, fmaf(Aj, all.y, Ej));
        }
        const float2 *slots = pairs + now * MAX_CLUSTER * W + col;
        const unsigned base = smem_addr(pairs), at = smem_addr(slots + rank * W) - base, count = smem_addr(bar + now) - base;
#pragma unroll 4
        for (int j = threadIdx.x / W; j < K; j += Sh::THREADS / W) {
            const unsigned far = there(base, j);
            send(far + at, far + count, all);
        }
        if (threadIdx.x >= W) return 0.0f;
        if (!sm100::mbar_try_wait(bar + now, round >> 1 & 1)) wait_long(bar + now, round >> 1 & 1);
        if (threadIdx.x == 0 && round + 2 < p.rounds) sm100::mbar_arrive_tx(bar + now, K * W * sizeof(float2));
        const int mine = DOWN ? K - 1 - rank : rank;
        auto run = [&](int from, int to) {
            if (resets) {
                for (int i = from; i < to; ++i) {
                    const float2 q = slots[(DOWN ? K - 1 - i : i) * W];
                    carry = apply(q.x, carry, q.y);
                }
            } else {
#pragma unroll 4
                for (int i = from; i < to; ++i) {
                    const float2 q = slots[(DOWN ? K - 1 - i : i) * W];
                    carry = fmaf(q.x, carry, q.y);
                }
            }
        };
        run(0, mine);
        const float before = carry;
        run(mine, K);
        return before;
    }
};

template <typename Sh, bool GATED, bool NORM>
__global__ void __launch_bounds__(Sh::THREADS, Sh::BLOCKS) gated_scan_fwd_kernel(const ScanArgs p, const __grid_constant__ ScanMaps maps) {
    using T = typename Sh::T;
    using M = Many<Sh::V>;
    constexpr int V = Sh::V, S = Sh::S, W = Sh::WIDE;
    extern __shared__ __align__(128) unsigned char smem[];
    Block<Sh> k(p, smem);
    const int K = p.cluster;
    if (Sh::ASYNC) k.open_copies();
    griddep_wait();
    k.read_length(p);
    const void *const from[3] = {p.x, p.ga, GATED ? p.gx : nullptr};
    const long long ld[3] = {p.ldx, p.ldga, p.ldgx};
    int t0 = k.rank * Sh::TILE;
    unsigned marks = 0;
    if (Sh::ASYNC && threadIdx.x == Sh::FETCHER) k.template fetch<GATED ? 3 : 2>(maps, 0, t0);
    if (K > 1) k.open_cluster(p);
    const M rate = M::all(-1.0f) * k.rates(p), none = M::all(0.0f), one = M::all(1.0f);
    if (p.reset) marks = k.marks(k.reset_of(p, t0));
    // the thread that folds channel c0 + threadIdx.x over the tile's warps
    const bool folds = threadIdx.x < W && k.c0 + (int)threadIdx.x < p.C;
    const int ch = k.c0 + threadIdx.x;
    float carry = folds && p.h0 ? p.h0[(long long)k.b * p.C + ch] : 0.0f;   // the state before this round's first tile
    char *out = reinterpret_cast<char *>(static_cast<T *>(p.h) + ((long long)k.b * p.L + t0 + k.group * S) * p.ldh + k.c);
    const int apart = KEEP / (Sh::TILE / Sh::WARPS);      // warps between two kept states
    float *kept = p.states + ((long long)k.b * ((p.L + KEEP - 1) / KEEP) + t0 / KEEP) * p.C + ch;
    const bool resets = p.reset;
    if (K > 1) cluster_wait();

    for (int round = 0; round < p.rounds; ++round, t0 += K * Sh::TILE) {
        unsigned char ahead = 0;
        if (Sh::ASYNC) k.arrived(0, round & 1);
        if (p.reset && round + 1 < p.rounds) ahead = k.reset_of(p, t0 + K * Sh::TILE);
        const int mine = t0 + k.group * S;   // this thread's first token
        const bool ragged = t0 + Sh::TILE > k.len;
        const bool slow = ragged || marks;
        M a[S], e[S], A = one, E = none;
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const M x = k.load(p, 0, t0, s, 0, from, ld);
            M n;
            decay(rate * sigmoid(k.load(p, 0, t0, s, 1, from, ld)), a[s], n);
            e[s] = GATED ? sigmoid(k.load(p, 0, t0, s, 2, from, ld)) * x : x;
            if (NORM) {
#pragma unroll
                for (int v = 0; v < V; ++v) n[v] = sqrt_(n[v]);
                e[s] = n * e[s];
            }
            A = A * a[s];
            E = fma(a[s], E, e[s]);
        }
        if (slow) {
            A = one, E = none;
#pragma unroll
            for (int s = 0; s < S; ++s) {
                if (marks >> s & 1) {
                    a[s] = M::all(CUT), e[s] = k.load(p, 0, t0, s, 0, from, ld);
                    if (GATED) e[s] = sigmoid(k.load(p, 0, t0, s, 2, from, ld)) * e[s];
                }
                if (mine + s >= k.len) a[s] = one, e[s] = none;      // leaves the state as it is
                E = k.applied(a[s], E, e[s]);
                A = k.joined(A, a[s]);
            }
        }
        M pA = one, pE = none;               // of the warp's earlier group, for the later one
        if (Sh::LANES == 16) {
            pA = k.other(A), pE = k.other(E);
            E = k.applied(resets, A, pE, E);
            A = k.joined(resets, A, pA);
        }
        if (k.upper) {
            k.put(k.A, A);
            k.put(k.E, E);
        }
        __syncthreads();
        // the stage is read: the next tile is on its way while the pairs meet
        if (Sh::ASYNC && threadIdx.x == Sh::FETCHER && round + 1 < p.rounds) k.template fetch<GATED ? 3 : 2>(maps, 0, t0 + K * Sh::TILE);
        float before = K > 1 ? k.template exchange<false>(p, round, k.E, carry) : carry;
        if (K > 1 && round + 1 == p.rounds) cluster_arrive();
        if (threadIdx.x < W) {               // the state before each warp's tokens
#pragma unroll
            for (int j = 0; j < Sh::WARPS; ++j) {
                k.H[j * W + threadIdx.x] = before;
                if (j % apart == 0 && p.states && folds && t0 + j * (Sh::TILE / Sh::WARPS) < p.L) kept[j / apart * p.C] = before;
                const float Aj = k.A[j * W + threadIdx.x], Ej = k.E[j * W + threadIdx.x];
                before = resets ? apply(Aj, before, Ej) : fmaf(Aj, before, Ej);
            }
            if (K == 1) carry = before;
            kept += (long long)K * (Sh::TILE / KEEP) * p.C;
        }
        __syncthreads();
        M h = k.get(k.H);
        if (Sh::LANES == 16 && k.upper) h = k.applied(resets, pA, h, pE);
        char *to = out;
        out += p.out_step;
        if (!slow) {
#pragma unroll
            for (int s = 0; s < S; ++s, to += p.row[0]) {
                h = fma(a[s], h, e[s]);
                if (k.c < p.C) Vec<T, V>::store(reinterpret_cast<T *>(to), h.v);
            }
        } else {
#pragma unroll
            for (int s = 0; s < S; ++s, to += p.row[0]) {
                h = k.applied(a[s], h, e[s]);
                const M o = mine + s < k.len ? h : none;
                if (mine + s < p.L && k.c < p.C) Vec<T, V>::store(reinterpret_cast<T *>(to), o.v);
            }
        }
        if (p.reset) marks = k.marks(ahead);
    }
    if (K > 1) cluster_wait();               // no block ends while another may still write to it
    if (k.rank == 0 && folds && p.h_last) p.h_last[(long long)k.b * p.C + ch] = carry;
}

template <typename Sh, bool GATED, bool NORM>
__global__ void __launch_bounds__(Sh::THREADS, Sh::BLOCKS) gated_scan_bwd_kernel(const ScanArgs p, const __grid_constant__ ScanMaps maps) {
    using T = typename Sh::T;
    using M = Many<Sh::V>;
    constexpr int V = Sh::V, S = Sh::S, W = Sh::WIDE;
    extern __shared__ __align__(128) unsigned char smem[];
    Block<Sh> k(p, smem);
    const int K = p.cluster, N = (p.L + KEEP - 1) / KEEP;
    if (Sh::ASYNC) k.open_copies();
    griddep_wait();
    k.read_length(p);
    const void *const from[4] = {p.x, p.ga, p.dh, GATED ? p.gx : nullptr};
    const long long ld[4] = {p.ldx, p.ldga, p.lddh, p.ldgx};
    int t0 = ((p.rounds - 1) * K + k.rank) * Sh::TILE;   // from the last tiles to the first
    unsigned marks = 0;
    if (Sh::ASYNC && threadIdx.x == Sh::FETCHER) k.template fetch<GATED ? 4 : 3>(maps, 0, t0);
    if (K > 1) k.open_cluster(p);
    const M rate = M::all(-1.0f) * k.rates(p), none = M::all(0.0f), one = M::all(1.0f);
    M drate = none;
    if (p.reset) marks = k.marks(k.reset_of(p, t0));
    // threads 0 .. W - 1 fold the adjoints of a channel, the next W its states
    const int col = threadIdx.x % W, ch = k.c0 + col;
    const bool folds = threadIdx.x < W, forward = threadIdx.x / W == 1;
    float carry = folds && ch < p.C && p.dh_last ? p.dh_last[(long long)k.b * p.C + ch] : 0.0f;   // a G of what follows
    const bool resets = p.reset;
    if (K > 1) cluster_wait();

    for (int round = 0; round < p.rounds; ++round, t0 -= K * Sh::TILE) {
        const int now = round & 1;
        unsigned char ahead = 0;
        if (Sh::ASYNC) k.arrived(now, round >> 1 & 1);
        if (p.reset && round + 1 < p.rounds) ahead = k.reset_of(p, t0 - K * Sh::TILE);
        float state = 0.0f;                  // before the tile
        if (forward && ch < p.C && t0 < p.L) state = p.states[((long long)k.b * N + t0 / KEEP) * p.C + ch];
        const int mine = t0 + k.group * S;
        const bool ragged = t0 + Sh::TILE > k.len;
        const bool slow = ragged || marks;
        // per value: a, r, the sigmoid s, n s, and a^2/n u, then a h - a^2/n u
        M a[S], r[S], g[S], ns[S], D[S], A = one, E = none, Z = none;
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const M x = k.load(p, now, t0, s, 0, from, ld);
            r[s] = sigmoid(k.load(p, now, t0, s, 1, from, ld));
            if (GATED) g[s] = sigmoid(k.load(p, now, t0, s, 3, from, ld));
            M n2, n = one, inv = none;
            decay(rate * r[s], a[s], n2);
            if (NORM) {
#pragma unroll
                for (int v = 0; v < V; ++v) inv[v] = n2[v] >= FLT_MIN ? rsqrt_(n2[v]) : 0.0f;   // below the forward root is 0: no slope
                n = inv * n2;
            }
            ns[s] = GATED ? n * g[s] : n;
            D[s] = a[s] * a[s] * (inv * (GATED ? g[s] * x : x));
            A = A * a[s];
            E = fma(a[s], E, ns[s] * x);
        }
        if (!slow) {
#pragma unroll
            for (int s = S - 1; s >= 0; --s) Z = a[s] * (k.load(p, now, t0, s, 2, from, ld) + Z);
        } else {
            A = one, E = none;
#pragma unroll
            for (int s = 0; s < S; ++s) {
                if (marks >> s & 1) a[s] = M::all(CUT), ns[s] = GATED ? g[s] : one, r[s] = none;
                const bool behind = mine + s >= k.len;
                if (behind) a[s] = one, ns[s] = none;
                E = k.applied(a[s], E, behind ? none : ns[s] * k.load(p, now, t0, s, 0, from, ld));
                A = k.joined(A, a[s]);
            }
#pragma unroll
            for (int s = S - 1; s >= 0; --s) {
                if (mine + s < k.len) Z = a[s] * (k.load(p, now, t0, s, 2, from, ld) + Z);
                if (marks >> s & 1) Z = none;
            }
        }
        M pA = one, pE = none, pZ = none;    // of the warp's other group
        if (Sh::LANES == 16) {
            pA = k.other(A), pE = k.other(E), pZ = k.other(Z);
            E = k.applied(resets, A, pE, E);
            Z = k.applied(resets, A, pZ, Z);
            A = k.joined(resets, A, pA);
        }
        if (k.upper) {
            k.put(k.A, A);
            k.put(k.E, E);
        }
        if (Sh::LANES == 32 || !k.upper) k.put(k.Z, Z);
        __syncthreads();
        // the other stage is read
        if (Sh::ASYNC && threadIdx.x == Sh::FETCHER && round + 1 < p.rounds) k.template fetch<GATED ? 4 : 3>(maps, 1 - now, t0 - K * Sh::TILE);
        float after = carry;
        if (K > 1) after = k.template exchange<true>(p, round, k.Z, carry);
        if (K > 1 && round + 1 == p.rounds) cluster_arrive();
        if (forward) {                       // the state before each warp's tokens, in E's place (the others read no E)
#pragma unroll
            for (int j = 0; j < Sh::WARPS; ++j) {
                const float Ej = k.E[j * W + col];
                k.E[j * W + col] = state;
                const float Aj = k.A[j * W + col];
                state = resets ? apply(Aj, state, Ej) : fmaf(Aj, state, Ej);
            }
        }
        if (folds) {                         // what arrives from after each warp's tokens
#pragma unroll
            for (int j = Sh::WARPS - 1; j >= 0; --j) {
                k.H[j * W + col] = after;
                const float Aj = k.A[j * W + col], Zj = k.Z[j * W + col];
                after = resets ? apply(Aj, after, Zj) : fmaf(Aj, after, Zj);
            }
            if (K == 1) carry = after;
        }
        __syncthreads();
        M h = k.get(k.E), z = k.get(k.H);
        if (Sh::LANES == 16) {
            if (k.upper) h = k.applied(resets, pA, h, pE);
            else z = k.applied(resets, pA, z, pZ);
        }
        if (!slow) {
#pragma unroll
            for (int s = 0; s < S; ++s) {
                const M kept = a[s] * h;
#pragma unroll
                for (int v = 0; v < V; ++v) D[s][v] = kept[v] - D[s][v];
                h = fma(ns[s], k.load(p, now, t0, s, 0, from, ld), kept);
            }
        } else {
#pragma unroll
            for (int s = 0; s < S; ++s) {
                const M e = mine + s < k.len ? ns[s] * k.load(p, now, t0, s, 0, from, ld) : none;
                const bool dead = (marks >> s & 1) || mine + s >= k.len;
#pragma unroll
                for (int v = 0; v < V; ++v) D[s][v] = dead ? 0.0f : fmaf(a[s][v], h[v], -D[s][v]);
                h = k.applied(a[s], h, e);
            }
        }
        const long long last = (long long)k.b * p.L + mine + S - 1;
        char *to1 = reinterpret_cast<char *>(static_cast<T *>(p.dx) + last * p.lddx + k.c);
        char *to2 = reinterpret_cast<char *>(static_cast<T *>(p.dga) + last * p.lddga + k.c);
        char *to3 = GATED ? reinterpret_cast<char *>(static_cast<T *>(p.dgx) + last * p.lddgx + k.c) : nullptr;
#pragma unroll
        for (int s = S - 1; s >= 0; --s) {
            if (slow && mine + s >= k.len) {             // zeros; the gates there, which may be NaN, meet nothing
                if (k.c < p.C && mine + s < p.L) {
                    Vec<T, V>::store(reinterpret_cast<T *>(to1), none.v);
                    Vec<T, V>::store(reinterpret_cast<T *>(to2), none.v);
                    if (GATED) Vec<T, V>::store(reinterpret_cast<T *>(to3), none.v);
                }
            } else {
                const M G = k.load(p, now, t0, s, 2, from, ld) + z;
                const M Gz = slow && (marks >> s & 1) ? none : G;        // a reset's decay has no gradient, nor what is before
                const M t = Gz * D[s] * r[s], o1 = G * ns[s], w = rate * t;   // t: dla r
                M o2, o3;
#pragma unroll
                for (int v = 0; v < V; ++v) drate[v] -= t[v], o2[v] = fmaf(w[v], -r[s][v], w[v]);
                z = a[s] * Gz;
                if (GATED) {
                    const M q = o1 * k.load(p, now, t0, s, 0, from, ld);
#pragma unroll
                    for (int v = 0; v < V; ++v) o3[v] = fmaf(q[v], -g[s][v], q[v]);
                }
                if (k.c < p.C) {
                    Vec<T, V>::store(reinterpret_cast<T *>(to1), o1.v);
                    Vec<T, V>::store(reinterpret_cast<T *>(to2), o2.v);
                    if (GATED) Vec<T, V>::store(reinterpret_cast<T *>(to3), o3.v);
                }
            }
            to1 -= p.row[0], to2 -= p.row[1];
            if (GATED) to3 -= p.row[2];
        }
        if (p.reset) marks = k.marks(ahead);
    }
    if (K > 1) cluster_wait();               // no block ends while another may still write to it
    if (k.rank == 0 && folds && ch < p.C && p.dh0) p.dh0[(long long)k.b * p.C + ch] = carry;
    // the rate's gradient over this block's tokens
    if (Sh::LANES == 16) drate = drate + k.other(drate);
    __syncthreads();
    if (k.upper) k.put(k.A, drate);
    __syncthreads();
    if (folds && ch < p.C) {
        float sum = 0.0f;
#pragma unroll
        for (int j = 0; j < Sh::WARPS; ++j) sum += k.A[j * W + col];
        p.drate[((long long)k.b * K + k.rank) * p.C + ch] = sum;
    }
}

// drate from the blocks' parts.
__global__ void __launch_bounds__(SUM_THREADS) gated_scan_rate_kernel(const float *part, int parts, int C, float *drate) {
    sum_parts(part, parts, C, [=](long long c, float s) { drate[c] = s; });
}

// One token: a thread per V channels of a sequence.  Bound: the launch (8 x 2048 in bf16 1.5 us, its bytes 0.04).
template <typename T, int V>
__global__ void __launch_bounds__(128)
gated_scan_step_kernel(const T *x, const T *ga, const T *gx, const float *rate, bool normalize, long long total, int C, float *state,
                       T *h) {
    const long long i = ((long long)blockIdx.x * 128 + threadIdx.x) * V;
    griddep_wait();
    griddep_launch_dependents();
    if (i >= total) return;
    const int c = (int)(i % C);
    Many<V> xv, av, gv, rv, s, a, n;
    Vec<T, V>::load(x + i, xv.v);
    Vec<T, V>::load(ga + i, av.v);
    if (gx) Vec<T, V>::load(gx + i, gv.v);
    Vec<float, V>::load(rate + c, rv.v);
    Vec<float, V>::load(state + i, s.v);
    decay(Many<V>::all(-1.0f) * rv * sigmoid(av), a, n);
#pragma unroll
    for (int v = 0; v < V; ++v) n[v] = normalize ? sqrt_(n[v]) : 1.0f;
    s = fma(a, s, n * (gx ? sigmoid(gv) * xv : xv));
    Vec<float, V>::store(state + i, s.v);
    Vec<T, V>::store(h + i, s.v);
}

// ------------------------------------------------------------------ launches
// Tiles at once: the cluster that ends first when as many of them run side by
// side as the card has room for, a wave costs two tiles to begin, and each block
// of it works through its share of the tiles.  Room: what the driver says of this
// kernel, asked once for each size and device.
template <auto kernel> cudaError_t room(int device, int threads, int smem, int cluster, int &clusters) {
    static std::atomic<int> known[DEVICES][MAX_CLUSTER + 1];     // 0: not asked, else one more than the clusters
    cudaError_t e;
    std::atomic<int> *here = device < DEVICES ? &known[device][cluster] : nullptr;
    if (here && (clusters = here->load(std::memory_order_relaxed) - 1) >= 0) return cudaSuccess;
    if (cluster == 1) {
        int blocks = 0;
        e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&blocks, kernel, threads, smem);
        clusters = blocks * SMS;
    } else {
        cudaLaunchAttribute attr;
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = cluster, attr.val.clusterDim.y = 1, attr.val.clusterDim.z = 1;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(cluster), cfg.blockDim = dim3(threads), cfg.dynamicSmemBytes = smem, cfg.attrs = &attr, cfg.numAttrs = 1;
        e = cudaOccupancyMaxActiveClusters(&clusters, kernel, &cfg);
    }
    if (e != cudaSuccess) return e;
    if (here) here->store(clusters + 1, std::memory_order_relaxed);
    return cudaSuccess;
}
template <auto kernel> cudaError_t choose_cluster(int threads, int smem, long long chains, int tiles, int &best) {
    long long cost = -1;
    int device = 0;
    cudaError_t e = allow<kernel, true>(smem, device);
    if (e != cudaSuccess) return e;
    best = 1;
    for (int n = 1; n <= MAX_CLUSTER && n <= tiles; ++n) {
        int clusters = 0;
        e = room<kernel>(device, threads, smem, n, clusters);
        if (e != cudaSuccess) return e;
        if (clusters < 1) continue;
        const long long t = (chains + clusters - 1) / clusters * ((tiles + n - 1) / n + 2);
        if (cost < 0 || t < cost) best = n, cost = t;
    }
    return cudaSuccess;
}

template <typename Sh, auto kernel> cudaError_t place(ScanArgs &p, long long &blocks) {
    const int tiles = (p.L + Sh::TILE - 1) / Sh::TILE;
    const long long chains = (long long)p.B * ((p.C + Sh::WIDE - 1) / Sh::WIDE);
    const cudaError_t e = choose_cluster<kernel>(Sh::THREADS, Sh::SMEM, chains, tiles, p.cluster);
    if (e != cudaSuccess) return e;
    p.rounds = (tiles + p.cluster - 1) / p.cluster;
    blocks = chains * p.cluster;
    const long long bytes = sizeof(typename Sh::T);
    const long long out[3] = {Sh::ARRAYS == 4 ? p.lddx : p.ldh, p.lddga, p.lddgx};
    for (int i = 0; i < 3; ++i) p.row[i] = bytes * out[i];
    p.out_step = bytes * p.cluster * Sh::TILE * out[0];
    return blocks > 0x7fffffffll ? cudaErrorInvalidValue : cudaSuccess;
}

// Rows [B][L][C] of one array in boxes of `tokens` tokens of 128 bytes.
cudaError_t encode(CUtensorMap *m, bool f32, const void *base, long long ld, const ScanArgs &p, int tokens) {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    if (!fn) {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            return cudaErrorNotSupported;
        fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
    }
    const cuuint64_t e = f32 ? 4 : 2, dims[3] = {(cuuint64_t)p.C, (cuuint64_t)p.L, (cuuint64_t)p.B};
    const cuuint64_t strides[2] = {(cuuint64_t)ld * e, (cuuint64_t)ld * e * p.L};
    const cuuint32_t box[3] = {(cuuint32_t)(128 / e), (cuuint32_t)tokens, 1}, es[3] = {1, 1, 1};
    return fn(m, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? cudaSuccess
               : cudaErrorInvalidValue;
}

template <typename Sh, auto kernel> cudaError_t launch_scan(ScanArgs &p, float *drate, cudaStream_t st) {
    long long blocks;
    cudaError_t e = place<Sh, kernel>(p, blocks);
    ScanMaps maps = {};
    if constexpr (Sh::ASYNC) {
        const bool f32 = sizeof(typename Sh::T) == 4;
        if (e == cudaSuccess) e = encode(&maps.map[0], f32, p.x, p.ldx, p, Sh::TILE);
        if (e == cudaSuccess) e = encode(&maps.map[1], f32, p.ga, p.ldga, p, Sh::TILE);
        if (Sh::ARRAYS == 4 && e == cudaSuccess) e = encode(&maps.map[2], f32, p.dh, p.lddh, p, Sh::TILE);
        if (p.gx && e == cudaSuccess) e = encode(&maps.map[Sh::ARRAYS - 1], f32, p.gx, p.ldgx, p, Sh::TILE);
    }
    if (e != cudaSuccess) return e;
    const int parts = p.B * p.cluster;
    if (parts == 1) p.drate = drate;     // backward: nothing to sum
    e = launch_big<kernel, true>(dim3((unsigned)blocks), Sh::THREADS, Sh::SMEM, Sh::SMEM, p.cluster, st, p, maps);
    if (e != cudaSuccess || !drate || parts == 1) return e;
    return launch(gated_scan_rate_kernel, dim3((p.C + 31) / 32), sum_threads(parts), 0, 1, st, (const float *)p.drate, parts, p.C, drate);
}

template <typename Sh> cudaError_t run_fwd(ScanArgs &p, cudaStream_t st) {
    if (p.gx && p.normalize) return launch_scan<Sh, gated_scan_fwd_kernel<Sh, true, true>>(p, nullptr, st);
    if (p.gx) return launch_scan<Sh, gated_scan_fwd_kernel<Sh, true, false>>(p, nullptr, st);
    if (p.normalize) return launch_scan<Sh, gated_scan_fwd_kernel<Sh, false, true>>(p, nullptr, st);
    return launch_scan<Sh, gated_scan_fwd_kernel<Sh, false, false>>(p, nullptr, st);
}
template <typename Sh> cudaError_t run_bwd(ScanArgs &p, float *drate, cudaStream_t st) {
    static_assert(Sh::TILE >= KEEP, "the workspace has a part for each tile of KEEP tokens, up to a cluster's");
    if (p.gx && p.normalize) return launch_scan<Sh, gated_scan_bwd_kernel<Sh, true, true>>(p, drate, st);
    if (p.gx) return launch_scan<Sh, gated_scan_bwd_kernel<Sh, true, false>>(p, drate, st);
    if (p.normalize) return launch_scan<Sh, gated_scan_bwd_kernel<Sh, false, true>>(p, drate, st);
    return launch_scan<Sh, gated_scan_bwd_kernel<Sh, false, false>>(p, drate, st);
}

// TMA where all rows allow it (starts and pitches of 16 bytes, a batch below 2^40 bytes), else pairs of channels, else
// single ones.
int width(s5_dtype dtype, int L, int C, std::initializer_list<long long> lds) {
    const int per = dtype == S5_BF16 ? 8 : 4;
    int w = C % per == 0 ? per : C % 2 == 0 ? 2 : 1;
    for (long long ld : lds) w = ld % per == 0 && ld < (1ll << 37) / L ? w : ld % 2 == 0 && w > 1 ? 2 : 1;
    return w;
}

s5_status check_scan(const ScanArgs &p, s5_dtype dtype) {
    if (!type_ok(dtype) || p.B < 0 || p.L < 0 || p.C < 1) return S5_ERR_INVALID_ARGUMENT;
    // the narrowest blocks, in the largest cluster, within a grid; parts within an int
    if (p.C > MAX_C) return S5_ERR_UNSUPPORTED;
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
    const int tiles = L <= KEEP ? 1 : (L + KEEP - 1) / KEEP;     // a cluster has no more blocks than a row has tiles
    return 256 + sizeof(float) * (size_t)B * (tiles < MAX_CLUSTER ? tiles : MAX_CLUSTER) * C;
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
    const int w = width(dtype, L, C, {ldx, ldga, p.ldgx, ldh});
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
    const int w = width(dtype, L, C, {ldx, ldga, p.ldgx, lddh, lddx, lddga, p.lddgx});
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

extern "C" int s5_gated_scan_fault(void) {
    int v = 0, zero = 0;
    if (cudaDeviceSynchronize() != cudaSuccess) return -1;       // a copy alone waits for no stream that does not block
    if (cudaMemcpyFromSymbol(&v, g_scan_fault, sizeof(int)) != cudaSuccess) return -1;
    if (v && cudaMemcpyToSymbol(g_scan_fault, &zero, sizeof(int)) != cudaSuccess) return -1;
    return v;
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
