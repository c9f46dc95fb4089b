// Host program: the product of rows in 8 bits on a machine without a GPU.  The
// HIP calls that the library makes are defined here, so that none reaches a
// device: kernels are written down instead of launched, and device memory is a
// count of bytes with an end.  Commands come a line each:
//
//   gemm T M N K A LDA W LDW  a product (A, W: addresses); answers with its return
//                            code, the device memory held, the launched kernels
//                            with their workgroups and threads
//   room BYTES               device memory that is left to allocate
//   capture 0|1              whether the stream is being captured
//   workspace BYTES          install a workspace (0: none) for the stream
//   state                    what went wrong so far: calls that a capture does not
//                            allow, allocations refused, and the last error
//   release                  xsymv_release
#include <dlfcn.h>
#include <hip/hip_ext.h>
#include <hip/hip_runtime.h>

#include <cstdio>
#include <cstring>
#include <map>
#include <string>

#include "../../include/xsymv.h"

static std::map<void*, size_t> held;
static size_t room = (size_t)1 << 40, used = 0, next_address = 0x100000000000ull;
static bool capturing = false;
static int forbidden = 0, refused = 0;
static hipError_t last = hipSuccess;
static std::string launched;

static hipError_t result(hipError_t e)
{
    if (e != hipSuccess) last = e;
    return e;
}

static hipError_t while_captured()
{
    if (!capturing) return hipSuccess;
    ++forbidden;
    return result(hipErrorStreamCaptureUnsupported);
}

static void note(const void* f, dim3 grid, dim3 block)
{
    Dl_info i{};
    // (a kernel of one unit alone, the copy of rows, has no name here)
    const char* name = dladdr(f, &i) && i.dli_saddr == f ? i.dli_sname : "?";
    char text[512];
    std::snprintf(text, sizeof text, " %s:%u:%u", name, grid.x * grid.y * grid.z,
                  block.x * block.y * block.z);
    launched += text;
}

extern "C" {
hipError_t hipGetDevice(int* d)
{
    *d = 0;
    return hipSuccess;
}
hipError_t hipMalloc(void** p, size_t bytes)
{
    if (hipError_t e = while_captured()) return e;
    if (bytes > room - used) {
        ++refused;
        return result(hipErrorOutOfMemory);
    }
    *p = (void*)next_address;
    next_address += (bytes + 4095) / 4096 * 4096;
    held[*p] = bytes;
    used += bytes;
    return hipSuccess;
}
hipError_t hipFree(void* p)
{
    if (p == nullptr) return hipSuccess;
    if (hipError_t e = while_captured()) return e;
    auto it = held.find(p);
    if (it == held.end()) return result(hipErrorInvalidValue);
    used -= it->second;
    held.erase(it);
    return hipSuccess;
}
hipError_t hipStreamSynchronize(hipStream_t) { return while_captured(); }
hipError_t hipDeviceSynchronize(void) { return while_captured(); }
hipError_t hipStreamIsCapturing(hipStream_t, hipStreamCaptureStatus* s)
{
    *s = capturing ? hipStreamCaptureStatusActive : hipStreamCaptureStatusNone;
    return hipSuccess;
}
hipError_t hipGetLastError(void)
{
    const hipError_t e = last;
    last = hipSuccess;
    return e;
}
static struct {
    dim3 grid, block;
} configured;
hipError_t __hipPushCallConfiguration(dim3 grid, dim3 block, size_t, hipStream_t)
{
    configured = {grid, block};
    return hipSuccess;
}
hipError_t __hipPopCallConfiguration(dim3* grid, dim3* block, size_t* shared, hipStream_t* stream)
{
    *grid = configured.grid;
    *block = configured.block;
    *shared = 0;
    *stream = nullptr;
    return hipSuccess;
}
hipError_t hipLaunchKernel(const void* f, dim3 grid, dim3 block, void**, size_t, hipStream_t)
{
    note(f, grid, block);
    return hipSuccess;
}
hipError_t hipExtLaunchKernel(const void* f, dim3 grid, dim3 block, void**, size_t, hipStream_t,
                              hipEvent_t, hipEvent_t, int)
{
    note(f, grid, block);
    return hipSuccess;
}
}

int main()
{
    void* const stream = (void*)0x5000;
    float* const f = (float*)0x7000;
    std::setvbuf(stdout, nullptr, _IOLBF, 1 << 16);
    char line[256];
    while (std::fgets(line, sizeof line, stdin)) {
        char word[32] = "", t = 0;
        int m, n, k, lda, ldw, at = 0;
        unsigned long long a, w;
        if (std::sscanf(line, "gemm %c %d %d %d %llu %d %llu %d", &t, &m, &n, &k, &a, &lda, &w,
                        &ldw) == 8) {
            launched.clear();
            const signed char *pa = (const signed char*)a, *pw = (const signed char*)w;
            const int rc = t == 's' ? xsymv_q8gemm_s(m, n, k, pa, lda, f, pw, ldw, f, nullptr, f, n, stream)
                           : t == 'h'
                               ? xsymv_q8gemm_h(m, n, k, pa, lda, f, pw, ldw, f, nullptr, (xhalf*)f, n, stream)
                               : xsymv_q8gemm_b(m, n, k, pa, lda, f, pw, ldw, f, nullptr, (xbfloat16*)f, n,
                                                stream);
            std::printf("%d %zu%s\n", rc, used, launched.c_str());
            continue;
        }
        std::sscanf(line, "%31s %n", word, &at);
        const unsigned long long v = std::strtoull(line + at, nullptr, 10);
        if (!std::strcmp(word, "room")) {
            room = used + v;
            std::printf("%zu\n", room);
        } else if (!std::strcmp(word, "capture")) {
            capturing = v != 0;
            std::printf("%d\n", (int)capturing);
        } else if (!std::strcmp(word, "workspace")) {
            std::printf("%d\n", xsymv_set_workspace(v ? (void*)0x6000 : nullptr, v, stream));
        } else if (!std::strcmp(word, "state")) {
            std::printf("%d %d %d\n", forbidden, refused, (int)last);
        } else if (!std::strcmp(word, "release")) {
            std::printf("%d\n", xsymv_release());
        } else {
            std::printf("? %s", line);
        }
    }
    return 0;
}
