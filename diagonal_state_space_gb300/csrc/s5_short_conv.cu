// s5_short_conv.cu -- the short causal convolution of each channel along the
// tokens: whole sequences, their backward pass, one token.
//
//   p_t = bias + sum_{j < K} w_j x_{t-K+1+j},   y = p  or  p sigmoid(p)
// where a token before the sequence is `past` (or 0) and one before a reset 0;
//   dp = dy act'(p),  dx_t = sum_j w_j dp_{t+K-1-j},  dw_j = sum dp_t x_{t-K+1+j}.
//
// Bound: memory forward, with little to spare; backward no single one.  With K = 4,
// silu and resets a value takes about 13 instructions forward and 26 backward.
// bf16, 4 x 2048 tokens of 4096 channels with resets: 25.5 us forward (5.3 TB/s) and
// 51 backward (3.9); 8 x 1999 of 2048 without 23.5 forward (5.6).  A lane walks a segment of tokens of V
// channels with the last K - 1 inputs (and, backward, the K sums of dx that are
// not whole yet) in registers, so that an input is read once and the K - 1
// around a segment twice, out of L2.  Each warp has a ring of its own in shared
// memory, that 16-byte copies fill some tokens ahead, and waits for no other.  A
// warp's lanes are at one token, so what a reset clears is the same for all of
// them: the window itself, and nothing behind it is multiplied, not even by
// zero.  Tokens in the middle of a segment without resets take a path without
// any test.
#include "s5_rows.cuh"
#include "s5_sm100.cuh"

namespace s5 {
namespace {
using namespace rows;
using sm100::smem_addr;

constexpr int WARPS = 4;                 // of a block
constexpr int U = 8;                     // tokens of a ring's stage, and of one pass of the loop
constexpr int MAX_TAPS = 8;
// Blocks that the segments are cut for; backward as many as run at once, a part of the weights' gradient each.
// Forward six could fit an SM, but longer segments for four are no slower and better where resets send some chunks the
// longer way (4 x 2048 tokens of 4096 channels with resets 25.3 us for four, 27.2 for six; 8 x 1999 of 2048 without
// 23.4 and 22.6).
constexpr int BLOCKS = 4 * SMS;

struct ConvArgs {
    const void *x;
    long long ldx;
    const float *w, *bias;               // [C][K], [C] or null
    int act;
    const void *past;                    // [B][K-1][C] or null
    const unsigned char *reset;          // [B][L] or null
    const int *lengths;                  // [B] or null
    int B, L, C, across, segs, R;        // blocks of channels; segments of R tokens of a sequence
    void *y;
    long long ldy;
    void *past_out;                      // [B][K-1][C] or null, may be past
    // backward
    const void *dy;
    long long lddy;
    const void *dpast_out;               // or null
    void *dx;
    long long lddx;
    void *dpast;                         // or null
    float *part;                         // [blocks along the tokens][K + 1][C]
    int along;                           // blocks along the tokens
};

template <int V, int K> __device__ __forceinline__ void load_taps(const ConvArgs &p, int c, bool in, Many<V> (&w)[K], Many<V> &bias) {
    float flat[V * K] = {};
    if (in) {
#pragma unroll
        for (int j = 0; j < K; ++j) Vec<float, V>::load(p.w + (long long)c * K + j * V, *reinterpret_cast<float(*)[V]>(flat + j * V));
    }
#pragma unroll
    for (int j = 0; j < K; ++j)
#pragma unroll
        for (int v = 0; v < V; ++v) w[j][v] = flat[v * K + j];
    bias = Many<V>::all(0.0f);
    if (in && p.bias) Vec<float, V>::load(p.bias + c, bias.v);
}

// Bit i: token t + i of the sequence is a reset.  All lanes of the warp call it.
template <int N> __device__ __forceinline__ unsigned resets(const ConvArgs &p, int b, int t, int len) {
    const int lane = threadIdx.x & 31, at = t + lane;
    return __ballot_sync(0xffffffffu, lane < N && at >= 0 && at < len && p.reset[(long long)b * p.L + at]);
}

// The same for the U tokens of a stage in two steps, so that the load is not waited for.
__device__ __forceinline__ unsigned char reset_of(const ConvArgs &p, int b, int t, int len) {
    const int at = t + (threadIdx.x & 31);
    return (threadIdx.x & 31) < U && at < len ? p.reset[(long long)b * p.L + at] : 0;
}

// What one segment's walk shares in both directions.
template <typename T, int V, int K, int ARRAYS, bool ASYNC> struct Walk {
    using M = Many<V>;
    static constexpr int ROW = 32 * V * (int)sizeof(T);          // bytes of a warp's row
    static constexpr int CHUNKS = ROW / 16, ROWS = ASYNC ? 32 / CHUNKS : 1;
    static constexpr int STAGES = ARRAYS == 1 ? 4 : 3;
    static constexpr int RING = ASYNC ? STAGES * ARRAYS * U * ROW : 0;   // bytes of a warp
    int b, t0, len, c;
    bool in;                             // this lane has channels
    M win[K - 1];                        // the inputs before the token
    int age;                             // tokens since the last reset, K where it is too long ago to matter
    unsigned char *ring;                 // [STAGES][ARRAYS][U][ROW]

    __device__ Walk(const ConvArgs &p, unsigned char *smem) {
        c = (blockIdx.x % p.across * 32 + (threadIdx.x & 31)) * V;
        in = c < p.C;
        ring = smem + threadIdx.x / 32 * RING;
    }
    __device__ const T *row(const ConvArgs &p, const void *a, long long ld, int t) const {
        return static_cast<const T *>(a) + ((long long)b * p.L + t) * ld + c;
    }
    __device__ void place(const ConvArgs &p, int segment) {
        b = segment / p.segs;
        t0 = segment % p.segs * p.R;
        len = p.lengths ? min(max(p.lengths[b], 0), p.L) : p.L;
    }
    // Tokens t .. t + U - 1, as far as they are before `stop`, on their way into a stage.
    __device__ void fetch(const ConvArgs &p, int stage, int t, int stop, const void *const *from, const long long *ld) {
        if constexpr (ASYNC) {
            const int l = threadIdx.x & 31, at = blockIdx.x % p.across * 32 * V + l % CHUNKS * (16 / (int)sizeof(T));
            const bool wide = (blockIdx.x % p.across + 1) * 32 * V <= p.C;
#pragma unroll
            for (int k = 0; k < ARRAYS; ++k) {
                const char *src = reinterpret_cast<const char *>(static_cast<const T *>(from[k]) + ((long long)b * p.L + t + l / CHUNKS) * ld[k] + at);
                const unsigned dst = smem_addr(ring + ((stage * ARRAYS + k) * U + l / CHUNKS) * ROW + l % CHUNKS * 16);
                const long long hop = ROWS * ld[k] * (long long)sizeof(T);
                if (t + U <= stop && wide) {
#pragma unroll
                    for (int i = 0; i < U / ROWS; ++i, src += hop) cp_async16(dst + i * ROWS * ROW, src);
                } else {
#pragma unroll
                    for (int i = 0; i < U / ROWS; ++i, src += hop)
                        if (at < p.C && t + l / CHUNKS + i * ROWS < stop) cp_async16(dst + i * ROWS * ROW, src);
                }
            }
        }
        cp_async_commit();
    }
    // This lane's values of array k at token t, the i-th of the stage; whatever where there is none.
    __device__ M load(const ConvArgs &p, int stage, int t, int i, int k, int stop, const void *const *from, const long long *ld) const {
        M r = M::all(0.0f);
        if constexpr (ASYNC) {
            Vec<T, V>::load(reinterpret_cast<const T *>(ring + ((stage * ARRAYS + k) * U + i) * ROW) + (threadIdx.x & 31) * V, r.v);
        } else {
            if (in && t + i < stop) Vec<T, V>::load(row(p, from[k], ld[k], t + i), r.v);
        }
        return r;
    }
    // N tokens' values as they lie there, all loaded before any output is stored, behind which no load may move.
    template <int N> __device__ void load_raw(const ConvArgs &p, int stage, int t, int i, int k, int stop, const void *const *from,
                                              const long long *ld, typename Vec<T, V>::raw (&r)[N]) const {
#pragma unroll
        for (int n = 0; n < N; ++n) {
            if constexpr (ASYNC) {
                r[n] = Vec<T, V>::get(reinterpret_cast<const T *>(ring + ((stage * ARRAYS + k) * U + i + n) * ROW) + (threadIdx.x & 31) * V);
            } else {
                r[n] = {};
                if (in && t + i + n < stop) r[n] = Vec<T, V>::get(row(p, from[k], ld[k], t + i + n));
            }
        }
    }
    __device__ void fresh() {
        age = 0;
#pragma unroll
        for (int i = 0; i < K - 1; ++i) win[i] = M::all(0.0f);
    }
    __device__ void push(const M &x) {
#pragma unroll
        for (int i = 0; i < K - 2; ++i) win[i] = win[i + 1];
        win[K - 2] = x;
    }
    // The K - 1 inputs before the segment.
    __device__ void open(const ConvArgs &p) {
        typename Vec<T, V>::raw raw[K - 1] = {};
#pragma unroll
        for (int i = 0; i < K - 1; ++i) {
            const int t = t0 - (K - 1) + i;
            if (in && t >= 0 && t < len) raw[i] = Vec<T, V>::get(row(p, p.x, p.ldx, t));
            if (in && t < 0 && p.past) raw[i] = Vec<T, V>::get(static_cast<const T *>(p.past) + ((long long)b * (K - 1) + i) * p.C + c);
        }
        const unsigned marks = p.reset ? resets<K - 1>(p, b, t0 - (K - 1), len) : 0;
        fresh();
        age = K;
#pragma unroll
        for (int i = 0; i < K - 1; ++i) {
            M x;
            Vec<T, V>::widen(raw[i], x.v);
            if (marks >> i & 1) fresh();
            push(x);
            age = min(age + 1, K);
        }
    }
    __device__ M taps(const M (&w)[K], const M &bias, const M &x) const {
        M s = fma(w[K - 1], x, bias);
#pragma unroll
        for (int j = 0; j < K - 1; ++j) s = fma(w[j], win[j], s);
        return s;
    }
    // The last reset of the sequence's last K - 1 tokens, or -K.
    __device__ int last_reset(const ConvArgs &p) const {
        const unsigned m = p.reset ? resets<K - 1>(p, b, len - (K - 1), len) : 0;
        return m ? len - (K - 1) + 31 - __clz(m) : -K;
    }
};

template <typename T, int V, int K, bool ASYNC>
__global__ void __launch_bounds__(WARPS * 32, 4) short_conv_fwd_kernel(const ConvArgs p) {
    using M = Many<V>;
    extern __shared__ __align__(128) unsigned char smem[];
    constexpr int STAGES = Walk<T, V, K, 1, ASYNC>::STAGES;
    Walk<T, V, K, 1, ASYNC> k(p, smem);
    const long long segment = (long long)(blockIdx.x / p.across) * WARPS + threadIdx.x / 32;
    if (segment >= (long long)p.B * p.segs) return;
    griddep_wait();
    k.place(p, (int)segment);
    const int end = min(k.t0 + p.R, p.L), stop = min(end, k.len);
    const void *const from[1] = {p.x};
    const long long ld[1] = {p.ldx};
#pragma unroll
    for (int i = 0; i < STAGES - 1; ++i) k.fetch(p, i, k.t0 + i * U, stop, from, ld);
    M w[K], bias;
    load_taps<V, K>(p, k.c, k.in, w, bias);
    k.open(p);
    if (k.t0 == 0 && p.past_out) {       // all of `past` that any warp reads is read by this one, above or here
        const int last = k.last_reset(p);
        typename Vec<T, V>::raw keep[K - 1] = {};
#pragma unroll
        for (int i = 0; i < K - 1; ++i) {
            const int t = k.len - (K - 1) + i;
            if (!k.in || last > t) continue;
            if (t >= 0) keep[i] = Vec<T, V>::get(k.row(p, p.x, p.ldx, t));
            else if (p.past) keep[i] = Vec<T, V>::get(static_cast<const T *>(p.past) + ((long long)k.b * (K - 1) + K - 1 + t) * p.C + k.c);
        }
#pragma unroll
        for (int i = 0; i < K - 1; ++i)
            if (k.in) Vec<T, V>::put(static_cast<T *>(p.past_out) + ((long long)k.b * (K - 1) + i) * p.C + k.c, keep[i]);
    }
    char *out = reinterpret_cast<char *>(static_cast<T *>(p.y) + ((long long)k.b * p.L + k.t0) * p.ldy + k.c);
    const long long hop = p.ldy * (long long)sizeof(T);
    int stage = 0;
    unsigned char ahead = p.reset ? reset_of(p, k.b, k.t0, k.len) : 0;
    for (int t = k.t0; t < end; t += U, stage = (stage + 1) % STAGES) {
        const unsigned marks = p.reset ? __ballot_sync(0xffffffffu, ahead) : 0;
        if (p.reset) ahead = reset_of(p, k.b, t + U, k.len);
        if (ASYNC) {
            cp_async_wait<STAGES - 2>();
            __syncwarp();                // the stage is here, and all lanes are done with the one before it
            k.fetch(p, (stage + STAGES - 1) % STAGES, t + (STAGES - 1) * U, stop, from, ld);
        }
        if (!marks && t + U <= stop) {
            typename Vec<T, V>::raw raw[U];
            k.load_raw(p, stage, t, 0, 0, stop, from, ld, raw);
#pragma unroll
            for (int i = 0; i < U; ++i, out += hop) {
                M x;
                Vec<T, V>::widen(raw[i], x.v);
                M y = k.taps(w, bias, x);
                if (p.act) y = y * sigmoid(y);
                if (k.in) Vec<T, V>::store(reinterpret_cast<T *>(out), y.v);
                k.push(x);
            }
            k.age = K;
        } else {
#pragma unroll 1
            for (int i = 0; i < U; ++i, out += hop) {
                const M x = t + i < stop ? k.load(p, stage, t, i, 0, stop, from, ld) : M::all(0.0f);
                if (marks >> i & 1) k.fresh();
                M y = k.taps(w, bias, x);
                if (p.act) y = y * sigmoid(y);
                if (t + i >= k.len) y = M::all(0.0f);
                if (k.in && t + i < end) Vec<T, V>::store(reinterpret_cast<T *>(out), y.v);
                k.push(x);
            }
        }
    }
}

template <typename T, int V, int K, bool ASYNC>
__global__ void __launch_bounds__(WARPS * 32, 4) short_conv_bwd_kernel(const ConvArgs p) {
    using M = Many<V>;
    extern __shared__ __align__(128) unsigned char smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, block = blockIdx.x / p.across;
    constexpr int STAGES = Walk<T, V, K, 2, ASYNC>::STAGES;
    Walk<T, V, K, 2, ASYNC> k(p, smem);
    griddep_wait();
    const void *const from[2] = {p.x, p.dy};
    const long long ld[2] = {p.ldx, p.lddy};
    const M none = M::all(0.0f);
    M w[K], bias, dw[K], db = none;
    load_taps<V, K>(p, k.c, k.in, w, bias);
#pragma unroll
    for (int j = 0; j < K; ++j) dw[j] = none;
    const long long segments = (long long)p.B * p.segs, hop = p.lddx * (long long)sizeof(T);
    for (long long segment = (long long)block * WARPS + warp; segment < segments; segment += (long long)p.along * WARPS) {
        k.place(p, (int)segment);
        const int end = min(k.t0 + p.R, p.L);            // of the gradients that this walk writes
        const int stop = min(end + K - 1, k.len);        // of the tokens that it reads
        __syncwarp();
#pragma unroll
        for (int i = 0; i < STAGES - 1; ++i) k.fetch(p, i, k.t0 + i * U, stop, from, ld);
        k.open(p);
        const int last = p.dpast_out ? k.last_reset(p) : 0;
        M acc[K];                                        // acc[j]: dx of the token j before the next one, as far as it is; [0] unused
#pragma unroll
        for (int j = 0; j < K; ++j) acc[j] = none;
        char *out = reinterpret_cast<char *>(const_cast<T *>(k.row(p, p.dx, p.lddx, k.t0 - (K - 1))));   // stored to from t0 on
        int stage = 0;
        unsigned char ahead = p.reset ? reset_of(p, k.b, k.t0, k.len) : 0;
        for (int t = k.t0; t < end + K - 1; t += U, stage = (stage + 1) % STAGES) {
            const unsigned marks = p.reset ? __ballot_sync(0xffffffffu, ahead) : 0;
            if (p.reset) ahead = reset_of(p, k.b, t + U, k.len);
            if (ASYNC) {
                cp_async_wait<STAGES - 2>();
                __syncwarp();
                k.fetch(p, (stage + STAGES - 1) % STAGES, t + (STAGES - 1) * U, stop, from, ld);
            }
            if (!marks && k.age >= K && t + U <= end && t + U <= k.len && (t > k.t0 || !p.dpast)) {
                constexpr int N = 4;         // tokens at a time
                typename Vec<T, V>::raw raw[N], rawd[N];
#pragma unroll
                for (int i = 0; i < U; ++i, out += hop) {
                    if (i % N == 0) {
                        k.load_raw(p, stage, t, i, 0, stop, from, ld, raw);
                        k.load_raw(p, stage, t, i, 1, stop, from, ld, rawd);
                    }
                    M x, dp;
                    Vec<T, V>::widen(raw[i % N], x.v);
                    Vec<T, V>::widen(rawd[i % N], dp.v);
                    if (p.act) {
                        const M s = k.taps(w, bias, x), g = sigmoid(s), sg = s * g;
                        M r;
#pragma unroll
                        for (int v = 0; v < V; ++v) r[v] = 1.0f - g[v];
                        dp = dp * fma(sg, r, g);
                    }
                    db = db + dp;
                    dw[K - 1] = fma(dp, x, dw[K - 1]);
#pragma unroll
                    for (int j = 0; j < K - 1; ++j) dw[j] = fma(dp, k.win[j], dw[j]);
                    const M whole = fma(w[0], dp, acc[K - 1]);
                    if (k.in && (i >= K - 1 || t > k.t0)) Vec<T, V>::store(reinterpret_cast<T *>(out), whole.v);
#pragma unroll
                    for (int j = K - 1; j > 1; --j) acc[j] = fma(w[K - j], dp, acc[j - 1]);
                    acc[1] = w[K - 1] * dp;
                    k.push(x);
                }
                continue;
            }
#pragma unroll 1
            for (int i = 0; i < U && t + i < end + K - 1; ++i, out += hop) {
                const bool here = t + i < stop;
                const M x = here ? k.load(p, stage, t, i, 0, stop, from, ld) : none;
                M dp = here ? k.load(p, stage, t, i, 1, stop, from, ld) : none;
                if (marks >> i & 1) k.fresh();
                if (here) {
                    if (p.act) {
                        const M s = k.taps(w, bias, x), g = sigmoid(s), sg = s * g;
                        M r;
#pragma unroll
                        for (int v = 0; v < V; ++v) r[v] = 1.0f - g[v];
                        dp = dp * fma(sg, r, g);
                    }
                    if (t + i < end) {
                        db = db + dp;
                        dw[K - 1] = fma(dp, x, dw[K - 1]);
#pragma unroll
                        for (int j = 0; j < K - 1; ++j) dw[j] = fma(dp, k.win[j], dw[j]);
                    }
                    acc[0] = w[K - 1] * dp;
#pragma unroll
                    for (int j = 1; j < K; ++j)
                        if (k.age >= j) acc[j] = fma(w[K - 1 - j], dp, acc[j]);
                } else {
                    acc[0] = none;
                }
                // the token K - 1 before is whole
                const int o = t + i - (K - 1), late = o - (k.len - (K - 1));
                if (k.in && p.dpast_out && late >= 0 && late < K - 1 && last <= o && (o >= k.t0 || k.t0 == 0)) {
                    M d;
                    Vec<T, V>::load(static_cast<const T *>(p.dpast_out) + ((long long)k.b * (K - 1) + late) * p.C + k.c, d.v);
                    acc[K - 1] = acc[K - 1] + d;
                }
                if (k.in && o >= k.t0 && o < end) Vec<T, V>::store(reinterpret_cast<T *>(out), acc[K - 1].v);
                if (k.in && o < 0 && p.dpast)
                    Vec<T, V>::store(static_cast<T *>(p.dpast) + ((long long)k.b * (K - 1) + K - 1 + o) * p.C + k.c, acc[K - 1].v);
#pragma unroll
                for (int j = K - 1; j > 0; --j) acc[j] = acc[j - 1];
                k.push(x);
                k.age = min(k.age + 1, K);
            }
        }
    }
    // the block's sums, in the rings' place
    float *sums = reinterpret_cast<float *>(smem);       // [WARPS - 1][K + 1][V][32]
    cp_async_wait<0>();
    __syncthreads();
    if (warp > 0) {
#pragma unroll
        for (int j = 0; j <= K; ++j)
#pragma unroll
            for (int v = 0; v < V; ++v) sums[(((warp - 1) * (K + 1) + j) * V + v) * 32 + lane] = j < K ? dw[j < K ? j : 0][v] : db[v];
    }
    __syncthreads();
    if (warp == 0 && k.in) {
        float *part = p.part + (long long)block * (K + 1) * p.C + k.c;
#pragma unroll
        for (int j = 0; j <= K; ++j) {
            M s = j < K ? dw[j < K ? j : 0] : db;
#pragma unroll
            for (int q = 0; q < WARPS - 1; ++q)
#pragma unroll
                for (int v = 0; v < V; ++v) s[v] += sums[((q * (K + 1) + j) * V + v) * 32 + lane];
            Vec<float, V>::store(part + (long long)j * p.C, s.v);
        }
    }
}

// The weights' gradients from the blocks' parts [parts][K + 1][C]: the taps, then the bias.
__global__ void __launch_bounds__(SUM_THREADS) short_conv_weight_kernel(const float *part, int parts, int K, int C, float *dw, float *db) {
    sum_parts(part, parts, (long long)(K + 1) * C, [=](long long q, float s) {
        const int j = (int)(q / C), c = (int)(q % C);
        if (j < K) dw[(long long)c * K + j] = s;
        else if (db) db[c] = s;
    });
}

// One token: a thread per V channels of a sequence.  Bound: the launch (96 x 4096 in bf16, 4 taps, 2.6 us, its bytes 0.9).
template <typename T, int V, int K>
__global__ void __launch_bounds__(128)
short_conv_step_kernel(const T *x, const float *w, const float *bias, int act, long long total, int C, T *state, T *y) {
    const long long i = ((long long)blockIdx.x * 128 + threadIdx.x) * V;
    griddep_wait();
    griddep_launch_dependents();
    if (i >= total) return;
    const int c = (int)(i % C);
    T *s = state + i / C * (K - 1) * C + c;
    typename Vec<T, V>::raw now = Vec<T, V>::get(x + i), old[K - 1];
#pragma unroll
    for (int j = 0; j < K - 1; ++j) old[j] = Vec<T, V>::get(s + (long long)j * C);
    ConvArgs p = {};
    p.w = w, p.bias = bias;
    Many<V> taps[K], out, r;
    load_taps<V, K>(p, c, true, taps, out);
#pragma unroll
    for (int j = 0; j < K; ++j) {
        Vec<T, V>::widen(j < K - 1 ? old[j < K - 1 ? j : 0] : now, r.v);
        out = fma(taps[j], r, out);
    }
    if (act) out = out * sigmoid(out);
    Vec<T, V>::store(y + i, out.v);
#pragma unroll
    for (int j = 0; j < K - 1; ++j) Vec<T, V>::put(s + (long long)j * C, j < K - 2 ? old[j < K - 2 ? j + 1 : 0] : now);
}

// ------------------------------------------------------------------ launches
// Channels of a lane: `most` (four; backward two where two rings of 32-bit rows would fill the shared memory), two where more
// taps would fill the registers or the sizes ask for it, or one.
template <typename T> constexpr int BWD_MOST = sizeof(T) == 2 ? 4 : 2;
int vector(int C, int K, int most, std::initializer_list<long long> lds) {
    int V = K > 4 ? 2 : most;
    while (C % V) V /= 2;
    for (long long ld : lds)
        while (ld % V) V /= 2;
    return V;
}
// Whether 16-byte copies can fetch the rows.
template <typename T> bool copies(int V, int C, std::initializer_list<long long> lds) {
    bool ok = V * sizeof(T) >= 4 && C * sizeof(T) % 16 == 0;
    for (long long ld : lds) ok = ok && ld * sizeof(T) % 16 == 0;
    return ok;
}

// Segments as short as it takes to give every one of the warps that run at once one, from 16 tokens to 256.
void cut(ConvArgs &p, int V) {
    p.across = (p.C + 32 * V - 1) / (32 * V);
    const long long each = ((long long)p.B * p.L * p.across + BLOCKS * WARPS - 1) / (BLOCKS * WARPS);
    p.R = each < 16 ? 16 : each > 256 ? 256 : (int)((each + U - 1) / U * U);
    p.segs = (p.L + p.R - 1) / p.R;
}

template <typename T, int V, int K, bool ASYNC> cudaError_t start_fwd(const ConvArgs &p, int blocks, cudaStream_t st) {
    constexpr int SMEM = WARPS * Walk<T, V, K, 1, ASYNC>::RING;
    return launch_big<short_conv_fwd_kernel<T, V, K, ASYNC>>(dim3(blocks), WARPS * 32, SMEM, SMEM, 1, st, p);
}
template <typename T, int V, int K> cudaError_t run_fwd(ConvArgs &p, cudaStream_t st) {
    cut(p, V);
    const long long blocks = ((long long)p.B * p.segs + WARPS - 1) / WARPS * p.across;
    if (blocks > 0x7fffffffll) return cudaErrorInvalidValue;
    if constexpr (V * sizeof(T) >= 4)
        if (copies<T>(V, p.C, {p.ldx, p.ldy})) return start_fwd<T, V, K, true>(p, (int)blocks, st);
    if constexpr (V * sizeof(T) < 16) return start_fwd<T, V, K, false>(p, (int)blocks, st);
    return cudaErrorInvalidValue;        // rows of whole 16 bytes a lane can be copied
}

int along_blocks(long long segments, int across) {
    const long long all = (segments + WARPS - 1) / WARPS, want = (BLOCKS + across - 1) / across;
    return (int)(all < want ? all : want);
}

template <typename T, int V, int K, bool ASYNC> cudaError_t start_bwd(const ConvArgs &p, cudaStream_t st) {
    constexpr int RING = WARPS * Walk<T, V, K, 2, ASYNC>::RING, SUMS = (int)sizeof(float) * (WARPS - 1) * (K + 1) * V * 32;
    constexpr int SMEM = RING > SUMS ? RING : SUMS;
    return launch_big<short_conv_bwd_kernel<T, V, K, ASYNC>>(dim3(p.along * p.across), WARPS * 32, SMEM, SMEM, 1, st, p);
}
template <typename T, int V, int K> cudaError_t run_bwd(ConvArgs &p, float *dw, float *db, cudaStream_t st) {
    cut(p, V);
    p.along = along_blocks((long long)p.B * p.segs, p.across);
    cudaError_t e = cudaSuccess;
    bool done = false;
    if constexpr (V * sizeof(T) >= 4)
        if (copies<T>(V, p.C, {p.ldx, p.lddy, p.lddx})) e = start_bwd<T, V, K, true>(p, st), done = true;
    if (!done) e = start_bwd<T, V, K, false>(p, st);
    if (e != cudaSuccess) return e;
    return launch(short_conv_weight_kernel, dim3((unsigned)(((long long)(K + 1) * p.C + 31) / 32)), sum_threads(p.along), 0, 1, st, (const float *)p.part, p.along, K, p.C, dw, db);
}

struct StepArgs {
    const void *x;
    const float *w, *bias;
    int act, B, C;
    void *state, *y;
};
template <typename T, int V, int K> cudaError_t run_step(const StepArgs &a, cudaStream_t st) {
    const long long total = (long long)a.B * a.C;
    return launch(short_conv_step_kernel<T, V, K>, dim3((unsigned)((total / V + 127) / 128)), 128, 0, 1, st, static_cast<const T *>(a.x),
                  a.w, a.bias, a.act, total, a.C, static_cast<T *>(a.state), static_cast<T *>(a.y));
}

// f<T, V, K>() for the run-time vector, of `most` channels, and tap counts.
#define S5_TAPS(f, T, V, K, ...) \
    case K: return f<T, V, K>(__VA_ARGS__);
#define S5_FEW(f, T, V, ...) S5_TAPS(f, T, V, 2, __VA_ARGS__) S5_TAPS(f, T, V, 3, __VA_ARGS__) S5_TAPS(f, T, V, 4, __VA_ARGS__)
#define S5_MORE(f, T, V, ...) \
    S5_TAPS(f, T, V, 5, __VA_ARGS__) S5_TAPS(f, T, V, 6, __VA_ARGS__) S5_TAPS(f, T, V, 7, __VA_ARGS__) S5_TAPS(f, T, V, 8, __VA_ARGS__)
#define S5_BY_SIZE(f, T, most, V, taps, ...)                                                                  \
    do {                                                                                                      \
        if constexpr (most >= 4)                                                                              \
            if (V == 4) switch (taps) { S5_FEW(f, T, 4, __VA_ARGS__) }                                        \
        if (V == 2) switch (taps) { S5_FEW(f, T, 2, __VA_ARGS__) S5_MORE(f, T, 2, __VA_ARGS__) }              \
        switch (taps) { S5_FEW(f, T, 1, __VA_ARGS__) S5_MORE(f, T, 1, __VA_ARGS__) }                          \
        return cudaErrorInvalidValue;                                                                         \
    } while (0)

template <typename T> cudaError_t fwd(ConvArgs &p, int V, int K, cudaStream_t st) { S5_BY_SIZE(run_fwd, T, 4, V, K, p, st); }
template <typename T> cudaError_t bwd(ConvArgs &p, int V, int K, float *dw, float *db, cudaStream_t st) {
    S5_BY_SIZE(run_bwd, T, BWD_MOST<T>, V, K, p, dw, db, st);
}
template <typename T> cudaError_t step(const StepArgs &a, int V, int K, cudaStream_t st) { S5_BY_SIZE(run_step, T, 4, V, K, a, st); }

s5_status check_conv(s5_dtype dtype, const float *w, const float *bias, int act, int B, int L, int C, int K) {
    if (!type_ok(dtype) || B < 0 || L < 0 || C < 1 || K < 1) return S5_ERR_INVALID_ARGUMENT;
    if (act != S5_ACT_NONE && act != S5_ACT_SILU) return S5_ERR_INVALID_ARGUMENT;
    if (K < 2 || K > MAX_TAPS || C > MAX_C) return S5_ERR_UNSUPPORTED;
    // segments of 16 tokens or more, and blocks of 32 channels times those of four segments, within an int
    if (L > (1 << 30) || (long long)B * ((L + 7) / 8) > (1ll << 30)) return S5_ERR_UNSUPPORTED;
    if (((long long)B * ((L + 7) / 8) / 4 + 1) * ((C + 31) / 32) > (1ll << 30) || (long long)B * C > (1ll << 36)) return S5_ERR_UNSUPPORTED;
    if (B > 0 && (!w || !aligned(w, 16))) return S5_ERR_INVALID_ARGUMENT;
    if (!aligned(bias, 16)) return S5_ERR_INVALID_ARGUMENT;
    return S5_OK;
}

}  // namespace
}  // namespace s5

using namespace s5;

extern "C" s5_status s5_short_conv_forward(const void *x, long long ldx, s5_dtype dtype, const float *weight, const float *bias,
                                           s5_activation activation, const void *past, const unsigned char *reset,
                                           const int *lengths, int B, int L, int C, int K, void *y, long long ldy, void *past_out,
                                           s5_stream_t stream) {
    s5_status c = check_conv(dtype, weight, bias, activation, B, L, C, K);
    if (c != S5_OK) return c;
    if (!aligned(past, 16) || !aligned(past_out, 16) || !aligned(lengths, 4)) return S5_ERR_INVALID_ARGUMENT;
    if (B == 0) return S5_OK;
    cudaStream_t st = (cudaStream_t)stream;
    if (L == 0) {   // the past stays as it is
        const size_t n = (dtype == S5_BF16 ? 2 : 4) * (size_t)B * (K - 1) * C;
        cudaError_t e = cudaSuccess;
        if (past_out && past && past_out != past) e = cudaMemcpyAsync(past_out, past, n, cudaMemcpyDeviceToDevice, st);
        if (past_out && !past) e = cudaMemsetAsync(past_out, 0, n, st);
        return e == cudaSuccess ? S5_OK : cuda_failure(e);
    }
    if (!rows_ok(x, ldx, C) || !rows_ok(y, ldy, C) || x == y) return S5_ERR_INVALID_ARGUMENT;
    ConvArgs p = {};
    p.x = x, p.ldx = ldx, p.w = weight, p.bias = bias, p.act = activation, p.past = past, p.reset = reset, p.lengths = lengths;
    p.B = B, p.L = L, p.C = C, p.y = y, p.ldy = ldy, p.past_out = past_out;
    const int V = vector(C, K, 4, {ldx, ldy});
    const cudaError_t e = dtype == S5_BF16 ? fwd<__nv_bfloat16>(p, V, K, st) : fwd<float>(p, V, K, st);
    return e == cudaSuccess ? S5_OK : cuda_failure(e);
}

extern "C" size_t s5_short_conv_workspace_size(int C, int K) {
    if (C < 1 || C > MAX_C || K < 2 || K > MAX_TAPS) return 0;
    // along_blocks() times C is the most with the widest blocks of channels
    return 256 + sizeof(float) * (size_t)(K + 1) * C * ((BLOCKS + (C + 127) / 128 - 1) / ((C + 127) / 128));
}

extern "C" s5_status s5_short_conv_backward(const void *x, long long ldx, s5_dtype dtype, const float *weight, const float *bias,
                                            s5_activation activation, const void *past, const unsigned char *reset,
                                            const int *lengths, int B, int L, int C, int K, const void *dy, long long lddy,
                                            const void *dpast_out, void *dx, long long lddx, float *dweight, float *dbias,
                                            void *dpast, void *workspace, size_t workspace_bytes, s5_stream_t stream) {
    s5_status c = check_conv(dtype, weight, bias, activation, B, L, C, K);
    if (c != S5_OK) return c;
    if (!aligned(past, 16) || !aligned(dpast_out, 16) || !aligned(dpast, 16) || !aligned(lengths, 4)) return S5_ERR_INVALID_ARGUMENT;
    if (!dweight || !aligned(dweight, 16) || !aligned(dbias, 16)) return S5_ERR_INVALID_ARGUMENT;
    cudaStream_t st = (cudaStream_t)stream;
    if (B == 0 || L == 0) {
        cudaError_t e = cudaMemsetAsync(dweight, 0, sizeof(float) * (size_t)C * K, st);
        if (e == cudaSuccess && dbias) e = cudaMemsetAsync(dbias, 0, sizeof(float) * C, st);
        const size_t n = (dtype == S5_BF16 ? 2 : 4) * (size_t)B * (K - 1) * C;
        if (e == cudaSuccess && n && dpast && dpast_out && dpast != dpast_out) e = cudaMemcpyAsync(dpast, dpast_out, n, cudaMemcpyDeviceToDevice, st);
        if (e == cudaSuccess && n && dpast && !dpast_out) e = cudaMemsetAsync(dpast, 0, n, st);
        return e == cudaSuccess ? S5_OK : cuda_failure(e);
    }
    if (!rows_ok(x, ldx, C) || !rows_ok(dy, lddy, C) || !rows_ok(dx, lddx, C) || dx == x || dx == dy) return S5_ERR_INVALID_ARGUMENT;
    if (!workspace || !aligned(workspace, 16) || workspace_bytes < s5_short_conv_workspace_size(C, K)) return S5_ERR_INVALID_ARGUMENT;
    ConvArgs p = {};
    p.x = x, p.ldx = ldx, p.w = weight, p.bias = bias, p.act = activation, p.past = past, p.reset = reset, p.lengths = lengths;
    p.B = B, p.L = L, p.C = C, p.dy = dy, p.lddy = lddy, p.dpast_out = dpast_out, p.dx = dx, p.lddx = lddx, p.dpast = dpast;
    p.part = static_cast<float *>(workspace);
    const int V = vector(C, K, dtype == S5_BF16 ? BWD_MOST<__nv_bfloat16> : BWD_MOST<float>, {ldx, lddy, lddx});
    const cudaError_t e = dtype == S5_BF16 ? bwd<__nv_bfloat16>(p, V, K, dweight, dbias, st) : bwd<float>(p, V, K, dweight, dbias, st);
    return e == cudaSuccess ? S5_OK : cuda_failure(e);
}

extern "C" s5_status s5_short_conv_step(const void *x, s5_dtype dtype, const float *weight, const float *bias,
                                        s5_activation activation, int B, int C, int K, void *state, void *y, s5_stream_t stream) {
    const s5_status c = check_conv(dtype, weight, bias, activation, B, 1, C, K);
    if (c != S5_OK) return c;
    if (B == 0) return S5_OK;
    for (const void *q : {x, (const void *)state, (const void *)y})
        if (!q || !aligned(q, 16)) return S5_ERR_INVALID_ARGUMENT;
    const StepArgs a = {x, weight, bias, activation, B, C, state, y};
    // four channels a thread, two where that would leave SMs idle
    const int V = vector(C, K, (long long)B * C < 4 * 128 * SMS ? 2 : 4, {});
    const cudaError_t e = dtype == S5_BF16 ? step<__nv_bfloat16>(a, V, K, (cudaStream_t)stream) : step<float>(a, V, K, (cudaStream_t)stream);
    return e == cudaSuccess ? S5_OK : cuda_failure(e);
}
