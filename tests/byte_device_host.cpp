// The host side of the 8-bit cache's calls beside a CUDA runtime of two devices
// that only counts: which device is current, and which one is waited for.
#include <cuda_runtime.h>

#include <cstdio>
#include <cstdlib>
#include <cstring>

#include "ott.h"

static int current = 0, waits[2] = {0, 0}, freed = 0, copies = 0, set_calls = 0;

extern "C" {
cudaError_t cudaGetDevice(int *d) { *d = current; return cudaSuccess; }
cudaError_t cudaSetDevice(int d) { current = d; ++set_calls; return cudaSuccess; }
cudaError_t cudaDeviceGetAttribute(int *v, cudaDeviceAttr, int) { *v = 128; return cudaSuccess; }
cudaError_t cudaDeviceSynchronize(void) { ++waits[current]; return cudaSuccess; }
cudaError_t cudaGetLastError(void) { return cudaSuccess; }
cudaError_t cudaMalloc(void **p, size_t n) { *p = std::malloc(n); return *p ? cudaSuccess : cudaErrorMemoryAllocation; }
cudaError_t cudaFree(void *p) { std::free(p); ++freed; return cudaSuccess; }
cudaError_t cudaMemset(void *p, int v, size_t n) { std::memset(p, v, n); return cudaSuccess; }
cudaError_t cudaMemcpy(void *d, const void *s, size_t n, cudaMemcpyKind) { std::memcpy(d, s, n); ++copies; return cudaSuccess; }
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t *, const void *, void **) { return cudaSuccess; }
// what nvcc's launch and registration code calls
void **__cudaRegisterFatBinary(void *) { static void *h; return &h; }
void __cudaRegisterFatBinaryEnd(void **) {}
void __cudaUnregisterFatBinary(void **) {}
void __cudaRegisterFunction(void **, const char *, char *, const char *, int, uint3 *, uint3 *, dim3 *, dim3 *, int *) {}
unsigned __cudaPushCallConfiguration(dim3, dim3, size_t, void *) { return 0; }
cudaError_t __cudaPopCallConfiguration(dim3 *, dim3 *, size_t *, void *) { return cudaSuccess; }
cudaError_t __cudaGetKernel(cudaKernel_t *, const void *) { return cudaSuccess; }
cudaError_t __cudaLaunchKernel(cudaKernel_t, dim3, dim3, void **, size_t, cudaStream_t) { return cudaSuccess; }
}

struct ott_byte_cache;
namespace ott {
struct ByteCall;
int run_byte_attn(const ott_byte_cache *, const ByteCall &, cudaStream_t, cudaError_t &) { return OTT_OK; }
cudaError_t set_byte_attributes(ott_byte_cache *) { return cudaSuccess; }
}  // namespace ott

#define CHECK(x)                                                \
    if (!(x)) {                                                 \
        std::printf("line %d: %s\n", __LINE__, #x);             \
        return 1;                                               \
    }

int main() {
    ott_byte_cache *c = nullptr;
    CHECK(ott_byte_create(2, 4, 2, 64, 32, OTT_BYTE_INT, 100, 0, &c) == OTT_OK && c);
    alignas(16) static char buf[2 * 4 * 64 * 2 * 4];
    CHECK(ott_byte_append(c, buf, buf, 1, nullptr, nullptr) == OTT_OK);
    CHECK(ott_byte_check(c) == OTT_OK && waits[0] == 2 && copies == 1);   // (one wait by create)

    // another device is current: every call that needs the cache's own is refused, and touches nothing
    current = 1;
    long long T = 0;
    CHECK(ott_byte_check(c) == OTT_ERR_STATE && waits[0] == 2 && waits[1] == 0 && copies == 1);
    CHECK(ott_byte_append(c, buf, buf, 1, nullptr, nullptr) == OTT_ERR_STATE);
    CHECK(ott_byte_append_seq(c, 0, buf, buf, 1, nullptr) == OTT_ERR_STATE);
    CHECK(ott_byte_read(c, buf, buf + 4096, 0, 1, nullptr) == OTT_ERR_STATE);
    CHECK(ott_byte_decode(c, buf, buf + 4096, 0, nullptr, nullptr) == OTT_ERR_STATE);
    CHECK(ott_byte_attn(c, buf, buf, buf, buf + 4096, 1, nullptr, 0, nullptr, nullptr) == OTT_ERR_STATE);
    CHECK(ott_byte_release(c, 0, nullptr) == OTT_ERR_STATE && ott_byte_reset(c, nullptr) == OTT_ERR_STATE);
    CHECK(ott_byte_counts(c, 0, &T, nullptr) == OTT_OK && T == 1);   // the host's own
    CHECK(current == 1 && set_calls == 0);

    // destroying waits for the cache's device, and leaves the current one as it was
    CHECK(ott_byte_destroy(c) == OTT_OK && waits[0] == 3 && waits[1] == 0 && freed == 1 && current == 1);

    current = 0;
    set_calls = 0;
    CHECK(ott_byte_create(1, 1, 1, 64, 32, OTT_BYTE_INT, 100, 4, &c) == OTT_OK);
    CHECK(ott_byte_destroy(c) == OTT_OK && waits[0] == 5 && freed == 2 && set_calls == 0);
    return 0;
}
