// s5_add_layernorm.cu -- layer norm of a row, or of the sum of two, and its
// backward pass with the weights' gradients.
//
//   s = x + residual,  mean = sum s / H,  inv = (sum (s - mean)^2 / H + eps)^-1/2
//   y = n w + b,  n = (s - mean) inv
//   g = dy w,  dx = inv (g - sum g / H - n sum(g n) / H) + dtotal
//   dw = sum over rows of dy n,  db = sum over rows of dy.
//
// Bound: memory.  Forward, a row lies in the registers of one warp, or of as
// many as it takes, between its loads and its stores: the mean first and then
// the squares about it, so that a row far from zero keeps its digits.
// Backward, a row is spread over more lanes, 8 columns each, because a lane
// also keeps the weights' gradients of its columns over all the rows that it
// sees; one block an SM adds its warps' sums up, and a second launch the
// blocks'.  No atomics.  bf16: 16384 rows of 2048 with the residual 43 us forward
// (6.2 TB/s) and 63.6 backward (5.3), 4099 of 8192 47.0 forward (5.7).  Odd widths
// move single values (3000 of 7001 backward 164 us, 1.3 TB/s), and backward rows of
// more than 6144 columns are read without the next one on its way (2000 of 12288
// 104 us, 2.4 TB/s; 12289, single values again, 312).
#include "s5_rows.cuh"
#include "s5_sm100.cuh"

namespace s5 {
namespace {
using namespace rows;

constexpr int MAX_H = 16384;
// A backward block: its warps and a lane's columns.  Eight columns leave registers for the next row: 24 warps where a
// lane has one vector of eight, else 16 (narrower vectors spill with 24: 8000 rows of 1799 in bf16 137 us, 66 with 16).
// Rows of 13 to 16 warps leave no room for a second one, and go better with 16 warps' registers (8192 of 4096 74 us, 82
// with 24).  Still wider rows take 24 warps again, only full vectors with the next row.  Above 6144 columns the sums of
// the weights' gradients lie in shared memory, 32 warps with 8 columns a lane and above 8192 with 16 (3000 of 7001 in
// bf16 164 us, 226 with the sums in registers; of 8192 in 32 bits 109, 124; 2000 of 12288 in bf16 104, 259), but for two
// kinds: bf16 in vectors up to 8192, 16 columns a lane in 16 warps (3000 of 8192 71, 87), and single values above it
// (2000 of 12289 312, 335).  What a thread spills, in bytes stored: single values above 8192 columns 1328 to 1380, the
// vectors there 24 to 156; below, up to 6144 with 24 warps and no next row 0 to 88, the others 20 at most.
constexpr int BWD_SMEM = 96 << 10;   // most of it: sums of two times 24 x 256 columns, or a weight of 16384
constexpr int SHARED_SMEM = 3 * MAX_H * (int)sizeof(float);

struct NormArgs {
    const void *x, *residual, *dy, *dtotal;
    long long ldx, ldr, lddy, lddt;
    const float *w, *bias;
    float eps;
    long long N;
    int H, warps;                    // warps of a row
    void *y, *total, *dx;
    long long ldy, ldt, lddx;
    float2 *saved;                   // [N] mean, inv
    float *part;                     // [blocks][2][H]
};

// The sum over a row's warps, to all of them.  Every warp of the block calls it.
__device__ __forceinline__ float row_sum(float v, int warps, float *smem) {
#pragma unroll
    for (int o = 16; o; o /= 2) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (warps == 1) return v;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (lane == 0) smem[warp] = v;
    __syncthreads();
    v = lane < warps ? smem[lane] : 0.0f;
#pragma unroll
    for (int o = 16; o; o /= 2) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// NV vectors of V values a lane.  One warp a row: four rows a block; else a row a block.
template <typename T, int V, int NV>
__global__ void __launch_bounds__(V * NV >= 32 ? 512 : 1024) add_layernorm_fwd_kernel(const NormArgs p) {
    __shared__ float sums[2][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long row = p.warps == 1 ? (long long)blockIdx.x * (blockDim.x >> 5) + warp : blockIdx.x;
    if (row >= p.N) return;
    const int at = ((p.warps == 1 ? 0 : warp * 32) + lane) * V, step = p.warps * 32 * V;
    griddep_wait();
    float s[NV][V];
    {
        typename Vec<T, V>::raw rx[NV], rr[NV];
        const T *x = static_cast<const T *>(p.x) + row * p.ldx, *r = static_cast<const T *>(p.residual) + row * p.ldr;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (at + i * step < p.H) rx[i] = Vec<T, V>::get(x + at + i * step);
        if (p.residual) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (at + i * step < p.H) rr[i] = Vec<T, V>::get(r + at + i * step);
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float t[V] = {};
            if (at + i * step < p.H) {
                Vec<T, V>::widen(rx[i], t);
                if (p.residual) {
                    float u[V];
                    Vec<T, V>::widen(rr[i], u);
#pragma unroll
                    for (int v = 0; v < V; ++v) t[v] += u[v];
                }
            }
#pragma unroll
            for (int v = 0; v < V; ++v) s[i][v] = t[v];
        }
    }
    if (p.total) {
        T *t = static_cast<T *>(p.total) + row * p.ldt;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (at + i * step < p.H) Vec<T, V>::store(t + at + i * step, s[i]);
    }
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int v = 0; v < V; ++v) sum += s[i][v];
    const float mean = row_sum(sum, p.warps, sums[0]) / p.H;
    sum = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if (at + i * step < p.H) {
#pragma unroll
            for (int v = 0; v < V; ++v) s[i][v] -= mean, sum = fmaf(s[i][v], s[i][v], sum);
        }
    const float inv = 1.0f / sqrtf(row_sum(sum, p.warps, sums[1]) / p.H + p.eps);
    if (p.saved && lane == 0 && (p.warps == 1 || warp == 0)) p.saved[row] = make_float2(mean, inv);
    T *y = static_cast<T *>(p.y) + row * p.ldy;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = at + i * step;
        if (c >= p.H) continue;
        float w[V], b[V], o[V];
        if (p.w) load_floats<V>(p.w + c, w);
        if (p.bias) load_floats<V>(p.bias + c, b);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            o[v] = s[i][v] * inv;
            if (p.w) o[v] *= w[v];
            if (p.bias) o[v] += b[v];
        }
        Vec<T, V>::store(y + c, o);
    }
}

// A block's warps in slots of `warps`, a row each at a time; the next row is on its way while a row's warps meet.
// SHARED: one slot, the sums of the weights' gradients in shared memory, where each lane has its own columns, dy widened
// again and dtotal read when they are needed, so that 16 columns a lane spill few of their 64 registers' values.
template <typename T, int V, int NV, int MOST, bool AHEAD, bool SHARED>
__global__ void __launch_bounds__(MOST * 32) add_layernorm_bwd_kernel(const NormArgs p) {
    __shared__ float2 sums[2][MOST];
    extern __shared__ __align__(16) float smem[];    // [H] the weight; at the end [slots - 1][2][H] sums; SHARED [3][H]
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int slots = (int)(blockDim.x >> 5) / p.warps, slot = warp / p.warps, first = slot * p.warps;
    const int at = ((warp - first) * 32 + lane) * V, step = p.warps * 32 * V;
    griddep_wait();
    for (int c = threadIdx.x; c < p.H; c += blockDim.x) smem[c] = p.w ? p.w[c] : 1.0f;
    constexpr int KEPT = SHARED ? 1 : NV;
    float dw[KEPT][V], db[KEPT][V];
#pragma unroll
    for (int i = 0; i < KEPT; ++i)
#pragma unroll
        for (int v = 0; v < V; ++v) dw[i][v] = 0.0f, db[i][v] = 0.0f;
    if constexpr (SHARED)
        for (int c = threadIdx.x; c < 2 * p.H; c += blockDim.x) smem[p.H + c] = 0.0f;
    const long long stride = (long long)gridDim.x * slots;
    const float per = 1.0f / p.H;
    using raw = typename Vec<T, V>::raw;
    raw rs[NV], rr[NV], rd[NV], rt[NV];
    float2 stat;
    long long row = (long long)blockIdx.x * slots + slot;
    auto fetch = [&](long long row) {
        if (row >= p.N) return;
        const T *s = static_cast<const T *>(p.x) + row * p.ldx + at, *d = static_cast<const T *>(p.dy) + row * p.lddy + at;
        const T *t = static_cast<const T *>(p.dtotal) + row * p.lddt + at, *r = static_cast<const T *>(p.residual) + row * p.ldr + at;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (at + i * step >= p.H) continue;
            rs[i] = Vec<T, V>::get(s + i * step);
            rd[i] = Vec<T, V>::get(d + i * step);
            if (p.residual) rr[i] = Vec<T, V>::get(r + i * step);
            if (!SHARED && p.dtotal) rt[i] = Vec<T, V>::get(t + i * step);
        }
        stat = p.saved[row];
    };
    if (AHEAD) fetch(row);
    __syncthreads();
    for (int turn = 0; row < p.N; row += stride, turn ^= 1) {
        if (!AHEAD) fetch(row);
        float n[NV][V], g[KEPT][V];
        float2 sum = make_float2(0.0f, 0.0f);
        const float inv = stat.y;
        raw late[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float s[V] = {}, d[V] = {}, w[V] = {};
            const bool in = at + i * step < p.H;
            if (in) {
                Vec<T, V>::widen(rs[i], s), Vec<T, V>::widen(rd[i], d), load_floats<V>(smem + at + i * step, w);
                if (p.residual) {
                    float u[V];
                    Vec<T, V>::widen(rr[i], u);
#pragma unroll
                    for (int v = 0; v < V; ++v) s[v] += u[v];
                }
            }
            if constexpr (!SHARED) late[i] = rt[i];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                n[i][v] = in ? (s[v] - stat.x) * inv : 0.0f;
                const float e = d[v] * w[v];
                if constexpr (!SHARED) g[i][v] = e;
                if constexpr (!SHARED) dw[i][v] = fmaf(d[v], n[i][v], dw[i][v]), db[i][v] += d[v];
                sum.x += e;
                sum.y = fmaf(e, n[i][v], sum.y);
            }
            if (SHARED && in && p.part) {
                float *own = smem + p.H + at + i * step, a[V], b[V];
                load_floats<V>(own, a), load_floats<V>(own + p.H, b);
#pragma unroll
                for (int v = 0; v < V; ++v) a[v] = fmaf(d[v], n[i][v], a[v]), b[v] += d[v];
                store_floats<V>(own, a), store_floats<V>(own + p.H, b);
            }
        }
        if (AHEAD) fetch(row + stride);
#pragma unroll
        for (int o = 16; o; o /= 2) {
            sum.x += __shfl_xor_sync(0xffffffffu, sum.x, o);
            sum.y += __shfl_xor_sync(0xffffffffu, sum.y, o);
        }
        if (p.warps > 1) {
            if (lane == 0) sums[turn][warp] = sum;
            sm100::named_bar_sync(1 + slot, p.warps * 32);
            sum = make_float2(0.0f, 0.0f);
            for (int j = 0; j < p.warps; ++j) sum.x += sums[turn][first + j].x, sum.y += sums[turn][first + j].y;
        }
        sum.x *= per, sum.y *= per;
        T *dx = static_cast<T *>(p.dx) + row * p.lddx + at;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (at + i * step >= p.H) continue;
            float o[V], t[V], e[V];
            if constexpr (SHARED) {
                Vec<T, V>::widen(rd[i], e), load_floats<V>(smem + at + i * step, t);
#pragma unroll
                for (int v = 0; v < V; ++v) e[v] *= t[v];
                if (p.dtotal) Vec<T, V>::load(static_cast<const T *>(p.dtotal) + row * p.lddt + at + i * step, t);
            } else {
#pragma unroll
                for (int v = 0; v < V; ++v) e[v] = g[i][v];
                if (p.dtotal) Vec<T, V>::widen(late[i], t);
            }
#pragma unroll
            for (int v = 0; v < V; ++v) {
                o[v] = inv * (e[v] - sum.x - n[i][v] * sum.y);
                if (p.dtotal) o[v] += t[v];
            }
            Vec<T, V>::store(dx + i * step, o);
        }
    }
    if (!p.part) return;
    if constexpr (SHARED) {
        float *part = p.part + (long long)blockIdx.x * 2 * p.H;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = at + i * step;
            if (c >= p.H) continue;
            load_floats<V>(smem + p.H + c, dw[0]), load_floats<V>(smem + 2 * p.H + c, db[0]);
            store_floats<V>(part + c, dw[0]), store_floats<V>(part + p.H + c, db[0]);
        }
    } else {
        __syncthreads();                     // the weight is read no more
        if (slot > 0) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (at + i * step < p.H) {
                    store_floats<V>(smem + (long long)(slot - 1) * 2 * p.H + at + i * step, dw[i]);
                    store_floats<V>(smem + (long long)(slot - 1) * 2 * p.H + p.H + at + i * step, db[i]);
                }
        }
        __syncthreads();
        if (slot > 0) return;
        float *part = p.part + (long long)blockIdx.x * 2 * p.H;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = at + i * step;
            if (c >= p.H) continue;
            for (int q = 1; q < slots; ++q) {
                float a[V], b[V];
                load_floats<V>(smem + (long long)(q - 1) * 2 * p.H + c, a);
                load_floats<V>(smem + (long long)(q - 1) * 2 * p.H + p.H + c, b);
#pragma unroll
                for (int v = 0; v < V; ++v) dw[i][v] += a[v], db[i][v] += b[v];
            }
            store_floats<V>(part + c, dw[i]);
            store_floats<V>(part + p.H + c, db[i]);
        }
    }
}

// The weights' gradients from the blocks' parts [parts][2][H].
__global__ void __launch_bounds__(SUM_THREADS) add_layernorm_weight_kernel(const float *part, int parts, int H, float *dw, float *db) {
    sum_parts(part, parts, 2ll * H, [=](long long q, float s) {
        if (q < H && dw) dw[q] = s;
        if (q >= H && db) db[q - H] = s;
    });
}

// ------------------------------------------------------------------ launches
template <typename T, int V, int NV> cudaError_t fwd_as(NormArgs &p, cudaStream_t st) {
    const int per = 32 * V * NV;
    p.warps = (p.H + per - 1) / per;
    const int rows = p.warps == 1 ? 4 : 1;
    return launch(add_layernorm_fwd_kernel<T, V, NV>, dim3((unsigned)((p.N + rows - 1) / rows)), 32 * p.warps * rows, 0, 1, st, p);
}
// A row in as few warps as a lane's columns allow (32 of 16 bits, 16 of 32) where the rows fill the SMs, else spread over more.
// Twice the columns a lane leave too few warps an SM: 16384 rows of 2048 46.4 us for 42.9, 4099 of 8192 53.6 for 48.2.
template <typename T, int V> cudaError_t fwd_by(NormArgs &p, cudaStream_t st) {
    constexpr int MOST = V * sizeof(T) == 16 && sizeof(T) == 2 ? 32 : 16;
    auto warps = [&](int cols) { return (p.H + 32 * cols - 1) / (32 * cols); };
    // single 32-bit values spill with 16 (8000 rows of 1799 80 us, 47 with 8)
    int cols = sizeof(T) == 4 && V == 1 && warps(8) <= 16 ? 8 : MOST;
    while (cols > V && warps(cols / 2) <= 32 && (warps(cols / 2) == 1 || p.N * warps(cols) < 8 * SMS)) cols /= 2;
    if (cols == V) return fwd_as<T, V, 1>(p, st);
    if (cols == 2 * V) return fwd_as<T, V, 2>(p, st);
    if (cols == 4 * V) return fwd_as<T, V, 4>(p, st);
    if constexpr (MOST >= 8 * V)
        if (cols == 8 * V) return fwd_as<T, V, 8>(p, st);
    if constexpr (MOST >= 16 * V)
        if (cols == 16 * V) return fwd_as<T, V, 16>(p, st);
    return cudaErrorInvalidValue;
}

template <typename T, int V, int NV, int MOST, bool AHEAD, bool SHARED = false>
cudaError_t bwd_as(NormArgs &p, float *dw, float *db, cudaStream_t st) {
    p.warps = (p.H + 32 * V * NV - 1) / (32 * V * NV);
    const int slots = MOST / p.warps;
    const long long need = (p.N + slots - 1) / slots;
    const int blocks = (int)(need < SMS ? need : SMS);
    const size_t smem = sizeof(float) * (size_t)p.H * (SHARED ? 3 : slots > 1 ? (slots - 1) * 2 : 1);
    const cudaError_t e = launch_big<add_layernorm_bwd_kernel<T, V, NV, MOST, AHEAD, SHARED>>(dim3(blocks), 32 * p.warps * slots, smem,
                                                                                              SHARED ? SHARED_SMEM : BWD_SMEM, 1, st, p);
    if (e != cudaSuccess || !p.part) return e;
    return launch(add_layernorm_weight_kernel, dim3((2 * p.H + 31) / 32), sum_threads(blocks), 0, 1, st, (const float *)p.part, blocks, p.H,
                  dw, db);
}
template <typename T, int V> cudaError_t bwd_by(NormArgs &p, float *dw, float *db, cudaStream_t st) {
    constexpr int MOST = V == 8 ? 24 : 16;
    if (p.H <= 32 * 8 * MOST / 2) return bwd_as<T, V, 8 / V, MOST, true>(p, dw, db, st);
    if (p.H <= 32 * 8 * 16) return bwd_as<T, V, 8 / V, 16, true>(p, dw, db, st);
    if (p.H <= 32 * 8 * 24) return bwd_as<T, V, 8 / V, 24, V == 8>(p, dw, db, st);
    if (p.H <= 32 * 8 * 32) {
        if constexpr (V == 1 || sizeof(T) == 4) return bwd_as<T, V, 8 / V, 32, false, true>(p, dw, db, st);
        else return bwd_as<T, V, 16 / V, 16, false>(p, dw, db, st);
    }
    return bwd_as<T, V, 16 / V, 32, false, (V > 1)>(p, dw, db, st);
}

int width(s5_dtype dtype, int H, std::initializer_list<long long> lds) {
    const int per = dtype == S5_BF16 ? 8 : 4;
    int w = H % per == 0 ? per : H % 2 == 0 ? 2 : 1;
    for (long long ld : lds) w = ld % per == 0 ? w : ld % 2 == 0 && w > 1 ? 2 : 1;
    return w;
}

s5_status check_norm(s5_dtype dtype, long long N, int H, const float *w, const float *bias) {
    if (!type_ok(dtype) || N < 0 || H < 1) return S5_ERR_INVALID_ARGUMENT;
    if (H > MAX_H || N > (1ll << 31) - 4) return S5_ERR_UNSUPPORTED;
    if (!aligned(w, 16) || !aligned(bias, 16)) return S5_ERR_INVALID_ARGUMENT;
    return S5_OK;
}

}  // namespace
}  // namespace s5

using namespace s5;

extern "C" s5_status s5_add_layernorm(const void *x, long long ldx, const void *residual, long long ldr, s5_dtype dtype,
                                      const float *weight, const float *bias, float eps, long long N, int H, void *y,
                                      long long ldy, void *total, long long ldt, float *saved, s5_stream_t stream) {
    const s5_status c = check_norm(dtype, N, H, weight, bias);
    if (c != S5_OK) return c;
    if (!(eps >= 0.0f) || eps > 1e30f) return S5_ERR_INVALID_ARGUMENT;
    if (N == 0) return S5_OK;
    if (!rows_ok(x, ldx, H) || !rows_ok(y, ldy, H) || (residual && !rows_ok(residual, ldr, H)) || (total && !rows_ok(total, ldt, H)))
        return S5_ERR_INVALID_ARGUMENT;
    if (!aligned(saved, 16) || y == total) return S5_ERR_INVALID_ARGUMENT;
    for (const void *in : {x, residual})
        if (in && ((y == in && ldy != (in == x ? ldx : ldr)) || (total == in && ldt != (in == x ? ldx : ldr)))) return S5_ERR_INVALID_ARGUMENT;
    NormArgs p = {};
    p.x = x, p.ldx = ldx, p.residual = residual, p.ldr = residual ? ldr : 0, p.w = weight, p.bias = bias, p.eps = eps, p.N = N, p.H = H;
    p.y = y, p.ldy = ldy, p.total = total, p.ldt = total ? ldt : 0, p.saved = reinterpret_cast<float2 *>(saved);
    const int w = width(dtype, H, {ldx, p.ldr, ldy, p.ldt});
    cudaStream_t st = (cudaStream_t)stream;
    cudaError_t e;
    if (dtype == S5_BF16) e = w == 8 ? fwd_by<__nv_bfloat16, 8>(p, st) : w == 2 ? fwd_by<__nv_bfloat16, 2>(p, st) : fwd_by<__nv_bfloat16, 1>(p, st);
    else e = w == 4 ? fwd_by<float, 4>(p, st) : w == 2 ? fwd_by<float, 2>(p, st) : fwd_by<float, 1>(p, st);
    return e == cudaSuccess ? S5_OK : cuda_failure(e);
}

extern "C" size_t s5_add_layernorm_workspace_size(int H) {
    return H < 1 || H > MAX_H ? 0 : 256 + sizeof(float) * 2 * (size_t)SMS * H;
}

extern "C" s5_status s5_add_layernorm_backward(const void *x, long long ldx, const void *residual, long long ldr, const void *dy,
                                               long long lddy, const void *dtotal, long long lddt, s5_dtype dtype, const float *weight, const float *saved, long long N,
                                               int H, void *dx, long long lddx, float *dweight, float *dbias, void *workspace,
                                               size_t workspace_bytes, s5_stream_t stream) {
    const s5_status c = check_norm(dtype, N, H, weight, dweight);
    if (c != S5_OK) return c;
    if (!aligned(dbias, 16)) return S5_ERR_INVALID_ARGUMENT;
    cudaStream_t st = (cudaStream_t)stream;
    if (N == 0) {
        cudaError_t e = cudaSuccess;
        if (dweight) e = cudaMemsetAsync(dweight, 0, sizeof(float) * H, st);
        if (dbias && e == cudaSuccess) e = cudaMemsetAsync(dbias, 0, sizeof(float) * H, st);
        return e == cudaSuccess ? S5_OK : cuda_failure(e);
    }
    if (!rows_ok(x, ldx, H) || !rows_ok(dy, lddy, H) || !rows_ok(dx, lddx, H) || (dtotal && !rows_ok(dtotal, lddt, H)) ||
        (residual && !rows_ok(residual, ldr, H)))
        return S5_ERR_INVALID_ARGUMENT;
    if ((dx == x && lddx != ldx) || (dx == residual && lddx != ldr) || (dx == dy && lddx != lddy) || (dx == dtotal && lddx != lddt))
        return S5_ERR_INVALID_ARGUMENT;
    if (!saved || !aligned(saved, 16)) return S5_ERR_INVALID_ARGUMENT;
    const bool weights = dweight || dbias;
    if (weights && (!workspace || !aligned(workspace, 16) || workspace_bytes < s5_add_layernorm_workspace_size(H)))
        return S5_ERR_INVALID_ARGUMENT;
    NormArgs p = {};
    p.x = x, p.ldx = ldx, p.residual = residual, p.ldr = residual ? ldr : 0, p.dy = dy, p.lddy = lddy, p.dtotal = dtotal, p.lddt = dtotal ? lddt : 0, p.w = weight;
    p.saved = reinterpret_cast<float2 *>(const_cast<float *>(saved)), p.N = N, p.H = H, p.dx = dx, p.lddx = lddx;
    p.part = weights ? static_cast<float *>(workspace) : nullptr;
    const int w = width(dtype, H, {ldx, p.ldr, lddy, lddx, p.lddt});
    cudaError_t e;
    if (dtype == S5_BF16)
        e = w == 8   ? bwd_by<__nv_bfloat16, 8>(p, dweight, dbias, st)
            : w == 2 ? bwd_by<__nv_bfloat16, 2>(p, dweight, dbias, st)
                     : bwd_by<__nv_bfloat16, 1>(p, dweight, dbias, st);
    else
        e = w == 4   ? bwd_by<float, 4>(p, dweight, dbias, st)
            : w == 2 ? bwd_by<float, 2>(p, dweight, dbias, st)
                     : bwd_by<float, 1>(p, dweight, dbias, st);
    return e == cudaSuccess ? S5_OK : cuda_failure(e);
}
