// s5_delta.cuh -- what the kernels of the gated delta rule share
// (s5_delta.cu: entry points, streaming step, CUDA-core sweeps;
// s5_delta_prep.cu, s5_delta_scan.cu, s5_delta_adjoint.cu: tensor-core chunks).
#pragma once
#include "s5_internal.cuh"

namespace s5 {
namespace delta {

constexpr int CHUNK = 64;   // tokens between two kept states

// Arrays as in include/s5.h.  Row of token t of sequence b: b * L + t.
struct Args {
    const void *q, *k, *v;
    long long ldq, ldk, ldv;          // elements between two tokens
    const float *g, *beta;            // [B][L][Hv]
    const float *s0;                  // [B][Hv][Dk][Dv] or null
    float scale;
    int B, L, Hk, Hv, Dk, Dv;
    void *o;
    long long ldo;
    float *s_last;                    // or null
    // kept for the backward pass (null: nothing is kept)
    float *e;                         // [B][L][Hv][Dv]   v_t - a_t S_{t-1}^T k_t
    float *states;                    // [B][Hv][N + 1][Dk][Dv]   S entering chunk c; [N] is the last state
    // backward
    const void *dout;                 // dL/do
    long long lddo;
    const float *ds_last;             // or null
    void *dq, *dk, *dv;
    long long lddq, lddk, lddv;
    float *dg, *dbeta, *ds0;          // ds0 may be null
    // backward workspace
    float *x;                         // [B][L][Hv][Dv]   dL/du_t
    float *dqh, *dkh;                 // [B][L][Hv][Dk]   per value head
    // of the decays' gradients: on the tensor cores parts of <S, Z> and of b_j, else parts of dg
    float *inner;                     // [B][Hv][N][inner_parts]
    float *writes;                    // [B][Hv][N][CHUNK][write_parts], or [parts][B][L][Hv]
    void *z;                          // dL/dS at the end of chunk c: [B][Hv][N][Dk][Dv] float32, or, for the tensor
                                      // cores, [B][Hv][N][Dv / 64][2][Dk][64] bf16 (two parts)
    void *images;                     // operand images of the tensor-core path; then a state between launches
    int from, count;                  // tensor cores: the chunks of this launch
    bool first;                       // more chunks follow, whose preparation may start
    bool beside;                      // the preparation runs while the kernel before it on the stream does, on which
                                      // it must not depend, and ends after that one
};

__host__ __device__ inline int chunks(int L) { return (L + CHUNK - 1) / CHUNK; }

// Parts of a chunk's <S, Z> and of a token's b_j: a warp of the adjoint each.
__host__ __device__ constexpr int inner_parts(int Dk, int Dv) { return Dv / 64 * (Dk / 16); }
__host__ __device__ constexpr int write_parts(int Dv) { return Dv / 64 * 2; }

// A decay factor: exp(g) is zero in 32 bits below -104, so that g = -inf and
// the type's lowest value (a reset of the state) act as -128, which sums of
// 64 can hold; NaN stays NaN.
__device__ __forceinline__ float clamp_g(float g) { return g < -128.0f ? -128.0f : g; }

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
    return v;
}
// (hi, lo) += (bh, bl): sums of floats with 46 bits.
__device__ __forceinline__ void add_pair(float &hi, float &lo, float bh, float bl) {
    const float s = hi + bh, t = s - hi, e = (hi - (s - t)) + (bh - t);
    const float l = lo + bl + e;
    hi = s + l;
    lo = l - (hi - s);
}
// One warp: G_i, the sums of a chunk's log decays, of tokens 2 lane and
// 2 lane + 1, in pairs of floats, so that a small difference of large sums keeps
// 24 bits.  Tokens past the end do not decay.
__device__ __forceinline__ void decay_sums(const Args &a, long long row0, int nt, int h, int lane, float (&hi)[2], float (&lo)[2]) {
    const int t = 2 * lane;
    const float x0 = t < nt ? clamp_g(a.g[(row0 + t) * a.Hv + h]) : 0.0f;
    const float x1 = t + 1 < nt ? clamp_g(a.g[(row0 + t + 1) * a.Hv + h]) : 0.0f;
    hi[1] = x0, lo[1] = 0.0f;
    add_pair(hi[1], lo[1], x1, 0.0f);
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const float uh = __shfl_up_sync(0xffffffffu, hi[1], m), ul = __shfl_up_sync(0xffffffffu, lo[1], m);
        if (lane >= m) add_pair(hi[1], lo[1], uh, ul);
    }
    hi[0] = hi[1], lo[0] = lo[1];
    add_pair(hi[0], lo[0], -x1, 0.0f);
}

// A launch whose blocks may be scheduled while the kernel before it drains: every
// kernel of the delta rule waits for that one (griddep_wait in all threads)
// before it touches global memory or TMEM, so that it also comes after all
// earlier ones.  None lets the next one in early: blocks that wait crowd some SMs
// (2 x 500 tokens of 4 heads of 64 x 64, forward and backward, 235 against 187 us).
template <typename... P, typename... A>
inline cudaError_t launch_after(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t st, const A &...args) {
    cudaLaunchAttribute attr;
    set_programmatic(attr);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}
// Whether the tensor-core path takes these arguments.
bool tc_supported(const Args &a, s5_dtype dtype, bool backward);
// Workspace of the tensor-core path; 0 for head sizes that it does not take.
size_t tc_image_bytes(int B, int L, int Hv, int Dk, int Dv);
cudaError_t tc_forward(const Args &a, cudaStream_t st);
cudaError_t tc_backward(const Args &a, cudaStream_t st);

}  // namespace delta
}  // namespace s5
