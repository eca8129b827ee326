// api_common.h -- what the files that implement the C ABI (api.cu, api_transformer.cu) share:
// the thread's error text, the device check, pointer checks, workspace alignment and the
// launch profiling scope.  Defined in api.cu.
#pragma once

#include <cstddef>
#include <cstdint>

#include <cuda_runtime.h>

#include "ck_int8.h"
#include "ck_internal.h"

namespace ck {

// Set the calling thread's error text and return `status`.
int fail(int status, const char* fmt, ...);
int cuda_fail(cudaError_t e, const char* where);

// CK_OK on a GB300 (compute capability 10.3), else a status with the text set.
int check_device(DeviceInfo* dev);

inline bool aligned16(const void* p)
{
    return (reinterpret_cast<uintptr_t>(p) & 15u) == 0;
}

#define CK_REQUIRE_PTR(p)                                                                       \
    do {                                                                                        \
        if ((p) == nullptr)                                                                     \
            return fail(CK_ERR_INVALID_ARG, "%s must not be NULL", #p);                         \
        if (!aligned16(p))                                                                      \
            return fail(CK_ERR_INVALID_ARG, "%s must be 16-byte aligned", #p);                  \
    } while (0)

constexpr size_t kAlign = 256;
inline size_t align_up(size_t v)
{
    return (v + kAlign - 1) & ~(kAlign - 1);
}

// Kernel kinds counted between ck_profile_begin() and ck_profile_end().
enum ProfKind {
    kProfQuantize = 0,
    kProfWiden = 1,
    kProfGemm = 2,
    kProfNormRope = 3,
    kProfAttention = 4,
    kProfInt4 = 5,
    kProfAdapter = 6,
    kProfLogprobs = 7,
    kProfCacheRead = 8,
    kProfKinds = 9
};

// Counts the launches made in its lifetime and, when event profiling is on, brackets them
// with two events on `s`.
struct ProfScope {
    ProfScope(int kind, int launches, cudaStream_t s);
    ~ProfScope();
    ProfScope(const ProfScope&) = delete;
    ProfScope& operator=(const ProfScope&) = delete;

private:
    int kind;
    cudaStream_t s;
    bool active = false;
    cudaEvent_t a = nullptr, b = nullptr;
};

}  // namespace ck
