// Launches of the gated recurrence on several devices, with stand-ins for the CUDA calls that choose and make them: a
// device takes clusters of more than eight blocks of a kernel only once that kernel's attribute is set there.  Arguments:
// a device and a length for each call; printed: each call's status and the cluster that was launched.
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <cstdio>
#include <cstdlib>
#include <map>
#include <set>
#include <utility>

namespace fake {
int device = 0, launched = 0;
std::set<std::pair<int, const void *>> large;          // (device, kernel): clusters of more than eight are allowed
std::map<std::pair<int, const void *>, int> memory;    // and the dynamic shared memory
constexpr int SMALL = 2;                               // a device without room for more than eight blocks at once

cudaError_t get_device(int *d) { return *d = device, cudaSuccess; }
template <typename K> cudaError_t set_attribute(K *k, cudaFuncAttribute what, int value) {
    const std::pair<int, const void *> at(device, (const void *)k);
    if (what == cudaFuncAttributeNonPortableClusterSizeAllowed && value) large.insert(at);
    if (what == cudaFuncAttributeMaxDynamicSharedMemorySize) memory[at] = value;
    return cudaSuccess;
}
template <typename K> cudaError_t may(K *k, int cluster, size_t smem) {
    const std::pair<int, const void *> at(device, (const void *)k);
    if (cluster > 8 && !large.count(at)) return cudaErrorInvalidClusterSize;
    return smem > 48 << 10 && (size_t)memory[at] < smem ? cudaErrorInvalidValue : cudaSuccess;
}
template <typename K> cudaError_t blocks(int *n, K *, int, size_t) { return *n = 4, cudaSuccess; }
template <typename K> cudaError_t clusters(int *n, K *k, const cudaLaunchConfig_t *c) {
    const int size = c->attrs[0].val.clusterDim.x;
    *n = device == SMALL && size > 8 ? 0 : 600 / size;
    return may(k, size, c->dynamicSmemBytes);
}
template <typename... Ks, typename... As> cudaError_t launch(const cudaLaunchConfig_t *c, void (*k)(Ks...), As &&...) {
    int cluster = 1;
    for (unsigned i = 0; i < c->numAttrs; ++i)
        if (c->attrs[i].id == cudaLaunchAttributeClusterDimension) cluster = c->attrs[i].val.clusterDim.x;
    launched = cluster;
    return may(k, cluster, c->dynamicSmemBytes);
}
CUresult encode(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill) {
    return CUDA_SUCCESS;
}
cudaError_t entry(const char *, void **f, unsigned, unsigned long long, cudaDriverEntryPointQueryResult *q) {
    *f = (void *)encode, *q = cudaDriverEntryPointSuccess;
    return cudaSuccess;
}
}  // namespace fake

#define cudaGetDevice fake::get_device
#define cudaFuncSetAttribute fake::set_attribute
#define cudaOccupancyMaxActiveBlocksPerMultiprocessor fake::blocks
#define cudaOccupancyMaxActiveClusters fake::clusters
#define cudaLaunchKernelEx fake::launch
#define cudaGetDriverEntryPointByVersion fake::entry
#include "s5_gated_scan.cu"

namespace s5 {
s5_status cuda_failure(cudaError_t) { return S5_ERR_CUDA; }
}  // namespace s5

int main(int argc, char **argv) {
    char *p = (char *)(1 << 20);         // never read: nothing is launched
    for (int i = 1; i + 1 < argc; i += 2) {
        fake::device = atoi(argv[i]), fake::launched = 0;
        const int L = atoi(argv[i + 1]), C = 8;
        const s5_status f = s5_gated_scan_forward(p, C, p, C, p, C, S5_BF16, (float *)p, nullptr, nullptr, nullptr, 1, 1, L, C, p, C, nullptr,
                                                  p, ~0ull, nullptr);
        printf("%d %d ", (int)f, fake::launched);
        const s5_status b = s5_gated_scan_backward(p, C, p, C, p, C, S5_BF16, (float *)p, nullptr, nullptr, 1, 1, L, C, p, C, nullptr, p, ~0ull,
                                                   p, C, p, C, p, C, (float *)p, nullptr, p, ~0ull, nullptr);
        printf("%d\n", (int)b);
    }
}
