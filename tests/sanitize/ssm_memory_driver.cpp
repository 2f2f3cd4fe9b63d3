// Entry points of csrc/ssm.cpp when a host allocation fails: each of their
// allocations in turn throws, and the call has to end with an error code, a
// reason and no plan. Launchers are stubs. Prints the number of failed calls.
#include <cstdio>
#include <cstdlib>
#include <new>
#include <string>

#include <hip/hip_runtime_api.h>

#include "../../grouped_convolution_backward_amd/csrc/abi_internal.hpp"
#include "../../grouped_convolution_backward_amd/csrc/ssm_internal.hpp"

namespace {
long g_until = -1;      // allocations until the one that fails; below 0: none does
bool g_failed = false;
std::string g_error;
}  // namespace

void* operator new(std::size_t n) {
    if (g_until >= 0 && g_until-- == 0) {
        g_failed = true;
        throw std::bad_alloc();
    }
    if (void* p = std::malloc(n)) return p;
    throw std::bad_alloc();
}
void operator delete(void* p) noexcept { std::free(p); }
void operator delete(void* p, std::size_t) noexcept { std::free(p); }

namespace wgrad {
void clear_error() { g_error.clear(); }
int set_error(int code, const std::string& msg) {
    g_error = msg;
    return code;
}
int device_model(int, DeviceModel&) { return WGRAD_OK; }
namespace ssm {
int launch_cconv(int, const CconvArgs&, void*) { return 1; }
int launch_cconv_bwd(int, const CconvArgs&, void*) { return 1; }
int launch_cconv_reduce(const CconvReduceArgs&, void*) { return 1; }
int launch_cconv_step(int, const CconvStepArgs&, void*) { return 1; }
int launch_scan_fwd(int, int, const ScanArgs&, void*) { return 1; }
int launch_scan_bwd(int, int, const ScanArgs&, void*) { return 1; }
int launch_scan_reduce(int, const ScanReduceArgs&, void*) { return 1; }
int launch_scan_step(int, int, const ScanStepArgs&, void*) { return 1; }
}  // namespace ssm
}  // namespace wgrad

extern "C" const char* hipGetErrorString(hipError_t) { return "a launch error of some length, as a stub reports it"; }

// Calls f with its first, second, .. allocation failing until none does.
template <class F>
int fail_each(const char* what, F f) {
    for (int n = 0;; ++n) {
        g_failed = false;
        g_until = n;
        const int rc = f();
        g_until = -1;
        if (!g_failed) return n;
        if (rc != WGRAD_ERR_INVALID_ARG || g_error.empty()) {
            std::printf("%s: allocation %d: status %d, reason \"%s\"\n", what, n, rc, g_error.c_str());
            std::exit(1);
        }
    }
}

int main() {
    int failed = 0;
    char* const at = reinterpret_cast<char*>(1 << 20);
    const wgrad_cconv_problem cp{WGRAD_BF16, WGRAD_ACT_SILU, 4, 0, 2, 10, 0, 8};
    const wgrad_scan_problem sp{WGRAD_BF16, 1, 0, 0, 2, 10, 0, 8, 1, 16};
    wgrad_cconv_plan_t* c = nullptr;
    wgrad_scan_plan_t* s = nullptr;
    failed += fail_each("convolution plan", [&] { return c ? WGRAD_OK : wgrad_cconv_plan(&cp, -1, &c); });
    failed += fail_each("scan plan", [&] { return s ? WGRAD_OK : wgrad_scan_plan(&sp, nullptr, -1, &s); });
    wgrad_cconv_problem bad = cp;
    bad.W = 100;                                            // refused, with a reason that takes memory
    wgrad_cconv_plan_t* none = nullptr;
    failed += fail_each("refused plan", [&] { return wgrad_cconv_plan(&bad, -1, &none); });
    wgrad_cconv_args a{};
    a.x = a.y = {at, 8};
    a.w = at;
    failed += fail_each("launch that fails", [&] { return wgrad_cconv_run(c, &a, nullptr); });
    wgrad_scan_args v{};
    failed += fail_each("run without operands", [&] { return wgrad_scan_run(s, &v, nullptr); });
    wgrad_cconv_plan_destroy(c);
    wgrad_scan_plan_destroy(s);
    std::printf("%d\n", none ? -1 : failed);
    return 0;
}
