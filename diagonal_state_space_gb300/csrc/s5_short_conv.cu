// s5_short_conv.cu -- the short causal convolution of each channel along the
// tokens: whole sequences, their backward pass, one token.
//
//   p_t = bias + sum_{j < K} w_j x_{t-K+1+j},   y = p  or  p sigmoid(p)
// where a token before the sequence is `past` (or 0) and one before a reset 0;
//   dp = dy act'(p),  dx_t = sum_j w_j dp_{t+K-1-j},  dw_j = sum dp_t x_{t-K+1+j}.
//
// Bound: memory, with little to spare: a value is 2 K + 12 instructions
// forward and 6 K + 20 backward.  A lane walks a segment of tokens of V
// channels with the last K - 1 inputs (and, backward, the K sums of dx that are
// not whole yet) in registers, so that an input is read once and the K - 1
// around a segment twice, out of L2.  A warp's lanes are at one token, so what
// a reset clears is the same for all of them: the window itself, and nothing
// behind it is multiplied, not even by zero.
#include "s5_rows.cuh"

namespace s5 {
namespace {
using namespace rows;

constexpr int WARPS = 4;                 // of a block
constexpr int UF = 8, UB = 4;            // tokens that are loaded at once, forward and backward
constexpr int MAX_TAPS = 8;
constexpr int BWD_BLOCKS = 4 * SMS;      // of the backward pass, about: a part of the weights' gradient each

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

template <int V, int K> __device__ __forceinline__ void load_taps(const ConvArgs &p, int c, bool in, float (&w)[V * K], float (&bias)[V]) {
#pragma unroll
    for (int j = 0; j < K; ++j) {
        float t[V] = {};
        if (in) Vec<float, V>::load(p.w + (long long)c * K + j * V, t);
#pragma unroll
        for (int v = 0; v < V; ++v) w[j * V + v] = t[v];
    }
#pragma unroll
    for (int v = 0; v < V; ++v) bias[v] = 0.0f;
    if (in && p.bias) Vec<float, V>::load(p.bias + c, bias);
}

// Bit i: token t + i of the sequence is a reset.  All lanes of the warp call it.
template <int U> __device__ __forceinline__ unsigned resets(const ConvArgs &p, int b, int t, int len) {
    const int lane = threadIdx.x & 31, at = t + lane;
    return __ballot_sync(0xffffffffu, lane < U && at >= 0 && at < len && p.reset[(long long)b * p.L + at]);
}

// What one segment's walk shares in both directions.
template <typename T, int V, int K> struct Walk {
    int b, t0, len, c;
    bool in;                             // this lane has channels
    float win[K - 1][V];                 // the inputs before the token
    int age;                             // tokens since the last reset, K where it is too long ago to matter

    __device__ const T *row(const ConvArgs &p, const void *a, long long ld, int t) const {
        return static_cast<const T *>(a) + ((long long)b * p.L + t) * ld + c;
    }
    __device__ void place(const ConvArgs &p, int segment) {
        b = segment / p.segs;
        t0 = segment % p.segs * p.R;
        len = p.lengths ? min(max(p.lengths[b], 0), p.L) : p.L;
    }
    __device__ void fresh() {
        age = 0;
#pragma unroll
        for (int i = 0; i < K - 1; ++i)
#pragma unroll
            for (int v = 0; v < V; ++v) win[i][v] = 0.0f;
    }
    __device__ void push(const float (&x)[V]) {
#pragma unroll
        for (int i = 0; i < K - 2; ++i)
#pragma unroll
            for (int v = 0; v < V; ++v) win[i][v] = win[i + 1][v];
#pragma unroll
        for (int v = 0; v < V; ++v) win[K - 2][v] = x[v];
        if (age < K) ++age;
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
            float x[V];
            Vec<T, V>::widen(raw[i], x);
            if (marks >> i & 1) fresh();
            push(x);
        }
    }
    __device__ float tap(const float (&w)[V * K], const float (&bias)[V], const float (&x)[V], int v) const {
        float s = fmaf(w[v * K + K - 1], x[v], bias[v]);
#pragma unroll
        for (int j = 0; j < K - 1; ++j) s = fmaf(w[v * K + j], win[j][v], s);
        return s;
    }
    // The last reset of the sequence's last K - 1 tokens, or -K.
    __device__ int last_reset(const ConvArgs &p) const {
        const unsigned m = p.reset ? resets<K - 1>(p, b, len - (K - 1), len) : 0;
        return m ? len - (K - 1) + 31 - __clz(m) : -K;
    }
};

template <typename T, int V, int K>
__global__ void __launch_bounds__(WARPS * 32) short_conv_fwd_kernel(const ConvArgs p) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    Walk<T, V, K> k;
    k.c = (blockIdx.x % p.across * 32 + lane) * V;
    k.in = k.c < p.C;
    const long long segment = (long long)(blockIdx.x / p.across) * WARPS + warp;
    if (segment >= (long long)p.B * p.segs) return;
    griddep_wait();
    k.place(p, (int)segment);
    const int end = min(k.t0 + p.R, p.L);
    typename Vec<T, V>::raw next[UF] = {}, raw[UF];
    auto fetch = [&](int t) {
#pragma unroll
        for (int i = 0; i < UF; ++i)
            if (k.in && t + i < k.len && t + i < end) next[i] = Vec<T, V>::get(k.row(p, p.x, p.ldx, t + i));
    };
    fetch(k.t0);
    float w[V * K], bias[V];
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
    T *out = static_cast<T *>(p.y) + ((long long)k.b * p.L + k.t0) * p.ldy + k.c;
    for (int t = k.t0; t < end; t += UF, out += UF * p.ldy) {
#pragma unroll
        for (int i = 0; i < UF; ++i) raw[i] = next[i];
        fetch(t + UF);
        const unsigned marks = p.reset ? resets<UF>(p, k.b, t, k.len) : 0;
#pragma unroll
        for (int i = 0; i < UF; ++i) {
            float x[V], y[V];
            Vec<T, V>::widen(raw[i], x);
            if (marks >> i & 1) k.fresh();
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float s = k.tap(w, bias, x, v);
                y[v] = p.act ? s * sigmoid(s) : s;
                if (t + i >= k.len) y[v] = 0.0f;
            }
            if (k.in && t + i < end) Vec<T, V>::store(out + i * p.ldy, y);
            k.push(x);
        }
    }
}

template <typename T, int V, int K>
__global__ void __launch_bounds__(WARPS * 32) short_conv_bwd_kernel(const ConvArgs p) {
    __shared__ float sums[WARPS - 1][(K + 1) * V][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    Walk<T, V, K> k;
    k.c = (blockIdx.x % p.across * 32 + lane) * V;
    k.in = k.c < p.C;
    const int block = blockIdx.x / p.across;
    griddep_wait();
    float w[V * K], bias[V], dw[V * K], db[V];
    load_taps<V, K>(p, k.c, k.in, w, bias);
#pragma unroll
    for (int i = 0; i < V * K; ++i) dw[i] = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) db[v] = 0.0f;
    const long long segments = (long long)p.B * p.segs;
    for (long long segment = (long long)block * WARPS + warp; segment < segments; segment += (long long)p.along * WARPS) {
        k.place(p, (int)segment);
        const int end = min(k.t0 + p.R, p.L);            // of the gradients that this walk writes
        const int stop = min(end + K - 1, k.len);        // of the tokens that it reads
        typename Vec<T, V>::raw nx[UB] = {}, nd[UB] = {}, rx[UB], rd[UB];
        auto fetch = [&](int t) {
#pragma unroll
            for (int i = 0; i < UB; ++i)
                if (k.in && t + i < stop) {
                    nx[i] = Vec<T, V>::get(k.row(p, p.x, p.ldx, t + i));
                    nd[i] = Vec<T, V>::get(k.row(p, p.dy, p.lddy, t + i));
                }
        };
        fetch(k.t0);
        k.open(p);
        const int last = p.dpast_out ? k.last_reset(p) : 0;
        float acc[K][V];                                 // acc[i]: dx of the token i before
#pragma unroll
        for (int i = 0; i < K; ++i)
#pragma unroll
            for (int v = 0; v < V; ++v) acc[i][v] = 0.0f;
        for (int t = k.t0; t < end + K - 1; t += UB) {
#pragma unroll
            for (int i = 0; i < UB; ++i) rx[i] = nx[i], rd[i] = nd[i];
            fetch(t + UB);
            const unsigned marks = p.reset ? resets<UB>(p, k.b, t, k.len) : 0;
#pragma unroll
            for (int i = 0; i < UB; ++i) {
                float x[V], dp[V];
                Vec<T, V>::widen(rx[i], x);
                Vec<T, V>::widen(rd[i], dp);
                if (marks >> i & 1) k.fresh();
                if (p.act) {
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        const float s = k.tap(w, bias, x, v), g = sigmoid(s);
                        dp[v] *= fmaf(s * g, 1.0f - g, g);
                    }
                }
                if (t + i < stop) {
                    if (t + i < end) {
#pragma unroll
                        for (int v = 0; v < V; ++v) {
                            db[v] += dp[v];
                            dw[v * K + K - 1] = fmaf(dp[v], x[v], dw[v * K + K - 1]);
#pragma unroll
                            for (int j = 0; j < K - 1; ++j) dw[v * K + j] = fmaf(dp[v], k.win[j][v], dw[v * K + j]);
                        }
                    }
#pragma unroll
                    for (int j = 0; j < K; ++j)
                        if (k.age >= j) {
#pragma unroll
                            for (int v = 0; v < V; ++v) acc[j][v] = fmaf(w[v * K + K - 1 - j], dp[v], acc[j][v]);
                        }
                }
                // the token K - 1 before is whole
                const int o = t + i - (K - 1), from = o - (k.len - (K - 1));
                if (k.in && p.dpast_out && from >= 0 && from < K - 1 && last <= o && (o >= k.t0 || k.t0 == 0)) {
                    float d[V];
                    Vec<T, V>::load(static_cast<const T *>(p.dpast_out) + ((long long)k.b * (K - 1) + from) * p.C + k.c, d);
#pragma unroll
                    for (int v = 0; v < V; ++v) acc[K - 1][v] += d[v];
                }
                if (k.in && o >= k.t0 && o < end) Vec<T, V>::store(const_cast<T *>(k.row(p, p.dx, p.lddx, o)), acc[K - 1]);
                if (k.in && o < 0 && o > -K && p.dpast)
                    Vec<T, V>::store(static_cast<T *>(p.dpast) + ((long long)k.b * (K - 1) + K - 1 + o) * p.C + k.c, acc[K - 1]);
#pragma unroll
                for (int j = K - 1; j > 0; --j)
#pragma unroll
                    for (int v = 0; v < V; ++v) acc[j][v] = acc[j - 1][v];
#pragma unroll
                for (int v = 0; v < V; ++v) acc[0][v] = 0.0f;
                k.push(x);
            }
        }
    }
    if (warp > 0) {
#pragma unroll
        for (int i = 0; i < V * K; ++i) sums[warp - 1][i][lane] = dw[i];
#pragma unroll
        for (int v = 0; v < V; ++v) sums[warp - 1][V * K + v][lane] = db[v];
    }
    __syncthreads();
    if (warp == 0 && k.in) {
        float *part = p.part + (long long)block * (K + 1) * p.C + k.c;
#pragma unroll
        for (int j = 0; j <= K; ++j) {
            float s[V];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int at = j < K ? v * K + j : V * K + v;
                s[v] = j < K ? dw[v * K + (j < K ? j : 0)] : db[v];
#pragma unroll
                for (int q = 0; q < WARPS - 1; ++q) s[v] += sums[q][at][lane];
            }
            Vec<float, V>::store(part + (long long)j * p.C, s);
        }
    }
}

// The parts in their order, 8 sums side by side and then joined.  blockIdx.y: the tap, or K for the bias.
__global__ void __launch_bounds__(256) short_conv_weight_kernel(const float *part, int parts, int K, int C, float *dw, float *db) {
    __shared__ float sums[8][32];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, c = blockIdx.x * 32 + lane, j = blockIdx.y;
    griddep_wait();
    float s = 0.0f;
    if (c < C)
        for (int i = w; i < parts; i += 8) s += part[((long long)i * (K + 1) + j) * C + c];
    sums[w][lane] = s;
    __syncthreads();
    if (w == 0 && c < C) {
#pragma unroll
        for (int i = 1; i < 8; ++i) s += sums[i][lane];
        if (j < K) dw[(long long)c * K + j] = s;
        else if (db) db[c] = s;
    }
}

// One token: a thread per V channels of a sequence.
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
    float taps[V * K], out[V], r[V];
    load_taps<V, K>(p, c, true, taps, out);
#pragma unroll
    for (int j = 0; j < K; ++j) {
        Vec<T, V>::widen(j < K - 1 ? old[j < K - 1 ? j : 0] : now, r);
#pragma unroll
        for (int v = 0; v < V; ++v) out[v] = fmaf(taps[v * K + j], r[v], out[v]);
    }
    if (act) {
#pragma unroll
        for (int v = 0; v < V; ++v) out[v] *= sigmoid(out[v]);
    }
    Vec<T, V>::store(y + i, out);
#pragma unroll
    for (int j = 0; j < K - 1; ++j) Vec<T, V>::put(s + (long long)j * C, j < K - 2 ? old[j < K - 2 ? j + 1 : 0] : now);
}

// ------------------------------------------------------------------ launches
int vector(int C, std::initializer_list<long long> lds) {
    int V = C % 4 == 0 ? 4 : C % 2 == 0 ? 2 : 1;
    for (long long ld : lds)
        while (ld % V) V /= 2;
    return V;
}

// Segments as long as there are enough of them for 16 warps an SM.
void cut(ConvArgs &p, int V) {
    p.across = (p.C + 32 * V - 1) / (32 * V);
    for (p.R = 64; p.R > 8; p.R /= 2)
        if ((long long)p.across * p.B * ((p.L + p.R - 1) / p.R) >= 16 * SMS) break;
    p.segs = (p.L + p.R - 1) / p.R;
}

template <typename T, int V, int K> cudaError_t run_fwd(ConvArgs &p, cudaStream_t st) {
    cut(p, V);
    const long long blocks = ((long long)p.B * p.segs + WARPS - 1) / WARPS * p.across;
    if (blocks > 0x7fffffffll) return cudaErrorInvalidValue;
    return launch(short_conv_fwd_kernel<T, V, K>, dim3((unsigned)blocks), WARPS * 32, 0, 1, st, p);
}

int along_blocks(long long segments, int across) {
    const long long all = (segments + WARPS - 1) / WARPS, want = (BWD_BLOCKS + across - 1) / across;
    return (int)(all < want ? all : want);
}

template <typename T, int V, int K> cudaError_t run_bwd(ConvArgs &p, float *dw, float *db, cudaStream_t st) {
    cut(p, V);
    p.along = along_blocks((long long)p.B * p.segs, p.across);
    cudaError_t e = launch(short_conv_bwd_kernel<T, V, K>, dim3((unsigned)(p.along * p.across)), WARPS * 32, 0, 1, st, p);
    if (e != cudaSuccess) return e;
    return launch(short_conv_weight_kernel, dim3((p.C + 31) / 32, K + 1), 256, 0, 1, st, (const float *)p.part, p.along, K, p.C, dw, db);
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

// f<V, K>() for the run-time vector and tap counts.
#define S5_BY_TAPS(f, T, V, taps, ...)                    \
    switch (taps) {                                       \
        case 2: return f<T, V, 2>(__VA_ARGS__);           \
        case 3: return f<T, V, 3>(__VA_ARGS__);           \
        case 4: return f<T, V, 4>(__VA_ARGS__);           \
        case 5: return f<T, V, 5>(__VA_ARGS__);           \
        case 6: return f<T, V, 6>(__VA_ARGS__);           \
        case 7: return f<T, V, 7>(__VA_ARGS__);           \
        default: return f<T, V, 8>(__VA_ARGS__);          \
    }
#define S5_BY_SIZE(f, T, V, taps, ...)                    \
    do {                                                  \
        if (V == 4) { S5_BY_TAPS(f, T, 4, taps, __VA_ARGS__) } \
        if (V == 2) { S5_BY_TAPS(f, T, 2, taps, __VA_ARGS__) } \
        S5_BY_TAPS(f, T, 1, taps, __VA_ARGS__)            \
    } while (0)

template <typename T> cudaError_t fwd(ConvArgs &p, int V, int K, cudaStream_t st) { S5_BY_SIZE(run_fwd, T, V, K, p, st); }
template <typename T> cudaError_t bwd(ConvArgs &p, int V, int K, float *dw, float *db, cudaStream_t st) {
    S5_BY_SIZE(run_bwd, T, V, K, p, dw, db, st);
}
template <typename T> cudaError_t step(const StepArgs &a, int V, int K, cudaStream_t st) { S5_BY_SIZE(run_step, T, V, K, a, st); }

s5_status check_conv(s5_dtype dtype, const float *w, const float *bias, int act, int B, int L, int C, int K) {
    if (!type_ok(dtype) || B < 0 || L < 0 || C < 1 || K < 1) return S5_ERR_INVALID_ARGUMENT;
    if (act != S5_ACT_NONE && act != S5_ACT_SILU) return S5_ERR_INVALID_ARGUMENT;
    if (K < 2 || K > MAX_TAPS) return S5_ERR_UNSUPPORTED;
    // segments of 8 tokens, and blocks of 32 channels times those of four segments, within an int
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
    const int V = vector(C, {ldx, ldy});
    const cudaError_t e = dtype == S5_BF16 ? fwd<__nv_bfloat16>(p, V, K, st) : fwd<float>(p, V, K, st);
    return e == cudaSuccess ? S5_OK : cuda_failure(e);
}

extern "C" size_t s5_short_conv_workspace_size(int C, int K) {
    if (C < 1 || K < 2 || K > MAX_TAPS) return 0;
    // along_blocks() times C is the most with the widest blocks of channels
    return 256 + sizeof(float) * (size_t)(K + 1) * C * ((BWD_BLOCKS + (C + 127) / 128 - 1) / ((C + 127) / 128));
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
    const int V = vector(C, {ldx, lddy, lddx});
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
    const int V = vector(C, {}) == 4 && (long long)B * C < 4 * 128 * SMS ? 2 : vector(C, {});
    const cudaError_t e = dtype == S5_BF16 ? step<__nv_bfloat16>(a, V, K, (cudaStream_t)stream) : step<float>(a, V, K, (cudaStream_t)stream);
    return e == cudaSuccess ? S5_OK : cuda_failure(e);
}
