// s5_rows.cuh -- what the kernels on rows of channels share (s5_gated_scan.cu,
// s5_short_conv.cu, s5_add_layernorm.cu): values in vectors, launches.
#pragma once
#include <atomic>

#include "s5_internal.cuh"

namespace s5 {
namespace rows {

template <int BYTES> struct Raw;
template <> struct Raw<16> { using type = uint4; };
template <> struct Raw<8> { using type = uint2; };
template <> struct Raw<4> { using type = unsigned; };
template <> struct Raw<2> { using type = unsigned short; };

// V values as they lie in memory, and as floats.
template <typename T, int V> struct Vec {
    using raw = typename Raw<sizeof(T) * V>::type;
    __device__ static raw get(const T *p) { return *reinterpret_cast<const raw *>(p); }
    __device__ static void put(T *p, const raw &t) { *reinterpret_cast<raw *>(p) = t; }
    __device__ static void widen(const raw &t, float (&r)[V]) {
        if constexpr (sizeof(T) == 2 && V > 1) {     // bf16 is the upper half of its float
            const unsigned *w = reinterpret_cast<const unsigned *>(&t);
#pragma unroll
            for (int i = 0; i < V; i += 2) {
                r[i] = __uint_as_float(w[i / 2] << 16);
                r[i + 1] = __uint_as_float(w[i / 2] & 0xffff0000u);
            }
        } else {
            const T *e = reinterpret_cast<const T *>(&t);
#pragma unroll
            for (int i = 0; i < V; ++i) r[i] = (float)e[i];
        }
    }
    __device__ static raw round(const float (&r)[V]) {
        raw t;
        T *e = reinterpret_cast<T *>(&t);
        if constexpr (sizeof(T) == 2 && V > 1) {
#pragma unroll
            for (int i = 0; i < V; i += 2) *reinterpret_cast<__nv_bfloat162 *>(e + i) = __floats2bfloat162_rn(r[i], r[i + 1]);
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) e[i] = (T)r[i];
        }
        return t;
    }
    __device__ static void load(const T *p, float (&r)[V]) { widen(get(p), r); }
    __device__ static void store(T *p, const float (&r)[V]) { put(p, round(r)); }
};

// V floats of a parameter or a sum, by 16 bytes at most.
template <int V> __device__ __forceinline__ void load_floats(const float *p, float (&r)[V]) {
    constexpr int N = V < 4 ? V : 4;
#pragma unroll
    for (int i = 0; i < V; i += N) Vec<float, N>::load(p + i, *reinterpret_cast<float(*)[N]>(r + i));
}
template <int V> __device__ __forceinline__ void store_floats(float *p, const float (&r)[V]) {
    constexpr int N = V < 4 ? V : 4;
#pragma unroll
    for (int i = 0; i < V; i += N) Vec<float, N>::store(p + i, *reinterpret_cast<const float(*)[N]>(r + i));
}

// 2^x, 1/x, 1/sqrt(x): the machine's own, off by 2^-22, 2^-23, 2^-22.4 relative.
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rsqrt_(float x) {
    float y;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float sqrt_(float x) {
    float y;
    asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
constexpr float LOG2E = 1.4426950408889634f;
__device__ __forceinline__ float sigmoid(float g) { return rcp(1.0f + ex2(-LOG2E * g)); }

// V floats of a lane whose sums and products go two to an instruction: these
// kernels are as short of issue slots as of bandwidth.  A constant takes a pair of
// registers there, and one by one none, so what has one goes one by one.
template <int V> struct Many {
    float v[V];
    __device__ __forceinline__ float &operator[](int i) { return v[i]; }
    __device__ __forceinline__ float operator[](int i) const { return v[i]; }
    __device__ static __forceinline__ Many all(float x) {
        Many r;
#pragma unroll
        for (int i = 0; i < V; ++i) r.v[i] = x;
        return r;
    }
};
#define S5_TWO(op, ...)                                                                                                     \
    asm(op : "=f"(r.v[i]), "=f"(r.v[i + 1]) : __VA_ARGS__)
template <int V> __device__ __forceinline__ Many<V> fma(const Many<V> &a, const Many<V> &b, const Many<V> &c) {
    Many<V> r;
    if constexpr (V % 2 == 0) {
#pragma unroll
        for (int i = 0; i < V; i += 2)
            S5_TWO("{\n\t.reg .b64 a, b, c;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
                   "fma.rn.f32x2 a, a, b, c;\n\tmov.b64 {%0, %1}, a;\n\t}",
                   "f"(a.v[i]), "f"(a.v[i + 1]), "f"(b.v[i]), "f"(b.v[i + 1]), "f"(c.v[i]), "f"(c.v[i + 1]));
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) r.v[i] = fmaf(a.v[i], b.v[i], c.v[i]);
    }
    return r;
}
template <int V> __device__ __forceinline__ Many<V> operator*(const Many<V> &a, const Many<V> &b) {
    Many<V> r;
    if constexpr (V % 2 == 0) {
#pragma unroll
        for (int i = 0; i < V; i += 2)
            S5_TWO("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmul.rn.f32x2 a, a, b;\n\t"
                   "mov.b64 {%0, %1}, a;\n\t}",
                   "f"(a.v[i]), "f"(a.v[i + 1]), "f"(b.v[i]), "f"(b.v[i + 1]));
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) r.v[i] = a.v[i] * b.v[i];
    }
    return r;
}
template <int V> __device__ __forceinline__ Many<V> operator+(const Many<V> &a, const Many<V> &b) {
    Many<V> r;
    if constexpr (V % 2 == 0) {
#pragma unroll
        for (int i = 0; i < V; i += 2)
            S5_TWO("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tadd.rn.f32x2 a, a, b;\n\t"
                   "mov.b64 {%0, %1}, a;\n\t}",
                   "f"(a.v[i]), "f"(a.v[i + 1]), "f"(b.v[i]), "f"(b.v[i + 1]));
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) r.v[i] = a.v[i] + b.v[i];
    }
    return r;
}
#undef S5_TWO
template <int V> __device__ __forceinline__ Many<V> sigmoid(const Many<V> &g) {
    Many<V> e;
#pragma unroll
    for (int i = 0; i < V; ++i) e[i] = sigmoid(g[i]);
    return e;
}

__device__ __forceinline__ void cp_async16(unsigned dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

inline bool aligned(const void *p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }
inline bool type_ok(int dtype) { return dtype == S5_F32 || dtype == S5_BF16; }
// An array that has to be there, 16-byte aligned, of rows with a pitch.
inline bool rows_ok(const void *p, long long ld, long long width) { return p && aligned(p, 16) && ld >= width; }

// A launch that may be scheduled while the kernel before it on the stream
// ends (the kernel waits for that one itself), in clusters of `cluster` blocks.
template <typename... Ks, typename... As>
cudaError_t launch(void (*k)(Ks...), dim3 grid, int threads, size_t smem, int cluster, cudaStream_t st, As... args) {
    cudaLaunchAttribute attr[2];
    set_programmatic(attr[0]);
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster, attr[1].val.clusterDim.y = 1, attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, k, args...);
}
// What a kernel may ask for at a launch, set once for each device: dynamic shared memory up to `most` bytes, and where
// LARGE says so clusters of more than eight blocks, whatever the first launch on a device takes.
constexpr int DEVICES = 64;              // of which something is remembered
template <auto kernel, bool LARGE> cudaError_t allow(int most, int &device) {
    static std::atomic<unsigned long long> done{0};
    cudaError_t e = cudaGetDevice(&device);
    if (e != cudaSuccess || (device < DEVICES && done.load(std::memory_order_relaxed) >> device & 1)) return e;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    if (LARGE && e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e == cudaSuccess && device < DEVICES) done.fetch_or(1ull << device, std::memory_order_relaxed);
    return e;
}
// The launch of such a kernel.
template <auto kernel, bool LARGE = false, typename... As>
cudaError_t launch_big(dim3 grid, int threads, size_t smem, int most, int cluster, cudaStream_t st, As... args) {
    int device = 0;
    const cudaError_t e = allow<kernel, LARGE>(most, device);
    return e != cudaSuccess ? e : launch(kernel, grid, threads, smem, cluster, st, args...);
}

constexpr int SMS = 152;
constexpr int MAX_C = 0x7fffff00;        // channels: the last block of them ends up to 127 behind, still within an int

// Sums of `parts` rows of n columns, in a fixed order: a warp's lanes have 32
// columns, the block's warps (as many as sum_threads says) take turns at the
// rows, eight loads in flight each.  store(column, sum) takes the result.
constexpr int SUM_THREADS = 512;
inline int sum_threads(int parts) { return parts >= 128 ? SUM_THREADS : 32 * ((parts + 7) / 8); }
template <typename Store> __device__ __forceinline__ void sum_parts(const float *part, int parts, long long n, Store store) {
    __shared__ float sums[SUM_THREADS / 32][32];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const long long c = (long long)blockIdx.x * 32 + lane;
    griddep_wait();
    float s = 0.0f;
    for (int i = w; i < parts; i += 8 * warps) {
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int row = i + j * warps;
            v[j] = c < n && row < parts ? part[row * n + c] : 0.0f;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) s += v[j];
    }
    sums[w][lane] = s;
    __syncthreads();
    if (w == 0 && c < n) {
        for (int i = 1; i < warps; ++i) s += sums[i][lane];
        store(c, s);
    }
}

}  // namespace rows
}  // namespace s5
