// A caller's kernel that writes a batch's metadata on the stream, just before a call that reads it: it
// lets the launch behind it start at once (griddepcontrol.launch_dependents) and writes some `naps`
// microseconds later.
#include <cuda_runtime.h>

__global__ void late_writer(int* dst, const int* src, int n, int naps) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    for (int i = 0; i < naps; ++i) __nanosleep(1000);
    for (int i = threadIdx.x; i < n; i += blockDim.x) dst[i] = src[i];
}

extern "C" __attribute__((visibility("default"))) int late_write(int* dst, const int* src, int n, int naps, cudaStream_t stream) {
    if (n < 0 || naps < 0 || naps > 1000) return -1;
    late_writer<<<1, 128, 0, stream>>>(dst, src, n, naps);
    return (int)cudaGetLastError();
}
