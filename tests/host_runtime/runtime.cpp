// A HIP runtime on the host, for tests of the library's C-ABI files without a
// GPU: device memory is host memory, a chosen call fails and leaves its error
// on the thread as the runtime does, and launches run nothing.
#include <cstdlib>
#include <cstring>

#include <hip/hip_runtime.h>

#include "../../gradient_compression_allreduce_amd/csrc/gq_tensors.h"

namespace {

thread_local hipError_t last = hipSuccess;
int fail_in = 0;        // the fail_in-th call from now on fails (0: none)
int live = 0, calls = 0, launches = 0;

hipError_t call() {
    ++calls;
    if (fail_in > 0 && --fail_in == 0) return last = hipErrorOutOfMemory;
    return hipSuccess;
}

hipError_t launch() {
    ++launches;
    return hipGetLastError();
}

}  // namespace

extern "C" {

void host_fail_in(int n) { fail_in = n; }
int host_calls() { return calls; }
int host_live() { return live; }
int host_launches() { return launches; }

hipError_t hipGetLastError() {
    const hipError_t e = last;
    last = hipSuccess;
    return e;
}
hipError_t hipPeekAtLastError() { return last; }
const char *hipGetErrorString(hipError_t e) { return e == hipSuccess ? "none" : "out of memory"; }

hipError_t hipGetDevice(int *d) {
    const hipError_t e = call();
    if (e == hipSuccess) *d = 0;
    return e;
}
hipError_t hipMalloc(void **p, size_t n) {
    const hipError_t e = call();
    if (e != hipSuccess) return e;
    *p = std::malloc(n ? n : 1);
    ++live;
    return hipSuccess;
}
hipError_t hipFree(void *p) {
    if (p) --live;
    std::free(p);
    return hipSuccess;
}
hipError_t hipMemcpy(void *to, const void *from, size_t n, hipMemcpyKind) {
    const hipError_t e = call();
    if (e == hipSuccess) std::memcpy(to, from, n);
    return e;
}
hipError_t hipMemset(void *p, int v, size_t n) {
    const hipError_t e = call();
    if (e == hipSuccess) std::memset(p, v, n);
    return e;
}
hipError_t hipDeviceSynchronize() { return call(); }
hipError_t hipStreamCreateWithFlags(hipStream_t *s, unsigned) {
    return hipMalloc(reinterpret_cast<void **>(s), 1);
}
hipError_t hipStreamDestroy(hipStream_t s) { return hipFree(s); }
hipError_t hipEventCreateWithFlags(hipEvent_t *e, unsigned) {
    return hipMalloc(reinterpret_cast<void **>(e), 1);
}
hipError_t hipEventDestroy(hipEvent_t e) { return hipFree(e); }

}  // extern "C"

namespace gq {

hipError_t launch_tensors_norm(const TnNormArgs &, hipStream_t) { return launch(); }
hipError_t launch_tensors_each(const TnEachArgs &, hipStream_t) { return launch(); }
hipError_t launch_tensors_clip(const TnClipArgs &, hipStream_t) { return launch(); }

}  // namespace gq
