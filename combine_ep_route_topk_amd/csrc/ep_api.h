// ep_api.h -- what the extern "C" entry points share: the calling thread's
// error text, argument checks, and the scope of the one-shot timing hook.
#pragma once

#include <cstdarg>
#include <cstdio>

#include "ep_internal.h"

namespace ep {

// The calling thread's text of ep_last_error (kErrorText bytes, api.hip).
constexpr size_t kErrorText = 512;
char* error_text();

// Clears the one-shot timing hook when a compute entry point returns.
struct TimingScope {
    ~TimingScope() { launch_timing() = LaunchTiming{}; }
};

inline ep_status fail(ep_status st, const char* fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(error_text(), kErrorText, fmt, ap);
    va_end(ap);
    return st;
}

inline ep_status ok() {
    error_text()[0] = '\0';
    return EP_OK;
}

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline ep_status launched(hipError_t e, const char* what) {
    if (e != hipSuccess)
        return fail(EP_ERR_LAUNCH, "%s: launch failed: %s", what, hipGetErrorString(e));
    return ok();
}

#define EP_REQUIRE_PTR(fn, p, a)                                                             \
    do {                                                                                     \
        if (!(p)) return ::ep::fail(EP_ERR_INVALID_ARG, "%s: %s is NULL", fn, #p);           \
        if (!::ep::aligned((p), (a)))                                                        \
            return ::ep::fail(EP_ERR_INVALID_ARG, "%s: %s is not %d-byte aligned", fn, #p,   \
                              int(a));                                                       \
    } while (0)

#define EP_TRY(expr)                  \
    do {                              \
        ep_status st_ = (expr);       \
        if (st_ != EP_OK) return st_; \
    } while (0)

}  // namespace ep
