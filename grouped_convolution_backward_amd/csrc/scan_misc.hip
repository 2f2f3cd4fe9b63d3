// Selective scan: the join of the backward kernel's partial sums, and the
// form for one token per sequence (gfx950).
#include <hip/hip_runtime.h>

#include "scan_kernels.hpp"

namespace wgrad {
namespace ssm {
namespace {

using scan::f32x4;

// Three jobs side by side in one launch, each summing partials in one order:
// dB and dC over the channel blocks of a group, dA over the pieces, dD and
// ddelta_bias over the pieces. Consecutive lanes read consecutive words, 16
// loads at a time, which do not wait for the sum (8192 rows, 16 states, 64
// channel blocks: 14.2 us for 70 MB, which the caches hold).
template <class T>
__global__ __launch_bounds__(256) void scan_reduce_kernel(const ScanReduceArgs a, int64_t n_bc, int64_t n_a) {
    int64_t i = (int64_t)(a.first + blockIdx.x) * 256 + threadIdx.x;
    const int W = 2 * a.SP;
    if (i < n_bc) {
        const int s2 = (int)(i % W);
        const int64_t r = i / W;
        const int g = (int)(r % a.G);
        const int64_t row = r / a.G;
        const int s = s2 < a.SP ? s2 : s2 - a.SP;
        if (s >= a.S) return;
        const float* p = a.part_bc + ((int64_t)g * a.cblks_g * a.rows + row) * W + s2;
        const int64_t step = (int64_t)a.rows * W;
        Pack<T, 1> out;
        out.set(0, sum_of(a.cblks_g, [&](int k) { return p[k * step]; }));
        T* d = s2 < a.SP ? static_cast<T*>(a.dB) + row * a.sdB : static_cast<T*>(a.dC) + row * a.sdC;
        out.store(d + (int64_t)g * a.S + s, true, 1);
        return;
    }
    i -= n_bc;
    if (i < n_a) {
        const int s = (int)(i % a.SP);
        const int64_t c = i / a.SP;
        if (s >= a.S) return;
        a.dA[c * a.S + s] = sum_of(a.pieces, [&](int p) { return a.part_a[((int64_t)p * a.channels + c) * a.SP + s]; });
        return;
    }
    i -= n_a;
    if (i >= 2 * (int64_t)a.channels) return;
    const int which = i >= a.channels;
    const int64_t c = i - (which ? a.channels : 0);
    float* out = which ? a.ddelta_bias : a.dD;
    if (!out) return;
    out[c] = sum_of(a.pieces, [&](int p) { return a.part_d[((int64_t)p * 2 + which) * a.channels + c]; });
}

template <class T>
int reduce(const ScanReduceArgs& a, void* stream) {
    const int64_t n_bc = (int64_t)a.rows * a.G * 2 * a.SP, n_a = (int64_t)a.channels * a.SP;
    const int64_t blocks = (n_bc + n_a + 2 * (int64_t)a.channels + 255) / 256;
    ScanReduceArgs v = a;
    for_launches(blocks, [&](uint32_t first, uint32_t grid) {
        v.first = first;
        scan_reduce_kernel<T><<<grid, 256, 0, static_cast<hipStream_t>(stream)>>>(v, n_bc, n_a);
    });
    return (int)hipGetLastError();
}

// One token per row. A lane takes NS states of a channel through one step;
// LPC adjacent lanes share the channel and its sum. Bound by reading and
// writing the states, 8 bytes each: 16-byte accesses, adjacent over the wave
// (256 rows of 4096 channels, 16 states: 28.8 us for 143 MB, 5.0 TB/s, a large
// copy's rate; one row: 3.4 us, the launch and two trips to memory).
template <class T, int NS, int LPC>
__global__ __launch_bounds__(256) void scan_step_kernel(const ScanStepArgs a) {
    constexpr int CT = 256 / LPC;
    const int cblks = (a.channels + CT - 1) / CT;
    const uint32_t wg = a.first + blockIdx.x;
    const int64_t row = wg / cblks;
    const int cb = (int)(wg - row * cblks);
    const int q = threadIdx.x % LPC, s0 = q * NS;
    const int c = cb * CT + (int)threadIdx.x / LPC;
    const bool ok = c < a.channels;
    const int64_t at = a.slots ? a.slots[row] : row;
    const bool live = at >= 0 && at < a.num_slots;
    const int cc = ok ? c : 0, g = cc / a.Cg;
    const bool vec = a.vec != 0;

    float h[NS], A2[NS];
    float* st = a.state + ((live ? at : 0) * a.channels + cc) * a.S + s0;
    const float* Ap = a.A + (int64_t)cc * a.S + s0;
    Pack<T, NS> B, C;
    B.load(static_cast<const T*>(a.B) + row * a.sB + (int64_t)g * a.S + s0, vec, min(a.S - s0, NS));
    C.load(static_cast<const T*>(a.C) + row * a.sC + (int64_t)g * a.S + s0, vec, min(a.S - s0, NS));
#pragma unroll
    for (int i = 0; i < NS; i += 4) {
        Pack<Fp32, 4> hv, av;
        hv.load(reinterpret_cast<const Fp32*>(st + i), vec, live ? min(a.S - s0 - i, 4) : 0);
        av.load(reinterpret_cast<const Fp32*>(Ap + i), vec, min(a.S - s0 - i, 4));
#pragma unroll
        for (int j = 0; j < 4; ++j) h[i + j] = hv.get(j), A2[i + j] = decay_rate(av.get(j));
    }
    Pack<T, 1> xv, dv, zv;
    xv.load(static_cast<const T*>(a.x) + row * a.sx + cc, true, 1);
    dv.load(static_cast<const T*>(a.delta) + row * a.sdelta + cc, true, 1);
    const float x = xv.get(0);
    float sig, d = dv.get(0) + (a.delta_bias ? a.delta_bias[cc] : 0.f);
    if (a.softplus) d = softplus<__is_same(T, Fp32)>(d, sig);
    const float u = d * x;
    float y = 0.f;
#pragma unroll
    for (int i = 0; i < NS; ++i) {
        h[i] = __builtin_fmaf(__builtin_amdgcn_exp2f(d * A2[i]), h[i], u * B.get(i));
        y = __builtin_fmaf(C.get(i), h[i], y);
    }
    y = lanes_sum<LPC>(y);
#pragma unroll
    for (int i = 0; i < NS; i += 4) {
        Pack<Fp32, 4> hv;
#pragma unroll
        for (int j = 0; j < 4; ++j) hv.set(j, h[i + j]);
        hv.store(reinterpret_cast<Fp32*>(st + i), vec, live && ok ? min(a.S - s0 - i, 4) : 0);
    }
    if (q == 0 && ok) {
        if (a.D) y = __builtin_fmaf(a.D[cc], x, y);
        if (a.z) {
            zv.load(static_cast<const T*>(a.z) + row * a.sz + cc, true, 1);
            const float z = zv.get(0);
            y *= z * gate_sigmoid(z);
        }
        Pack<T, 1> out;
        out.set(0, live ? y : 0.f);
        out.store(static_cast<T*>(a.y) + row * a.sy + cc, true, 1);
    }
}

template <class T, int NS, int LPC>
int step(const ScanStepArgs& a, hipStream_t s) {
    constexpr int CT = 256 / LPC;
    const int64_t blocks = a.rows * ((a.channels + CT - 1) / CT);
    ScanStepArgs v = a;
    for_launches(blocks, [&](uint32_t first, uint32_t grid) {
        v.first = first;
        scan_step_kernel<T, NS, LPC><<<grid, 256, 0, s>>>(v);
    });
    return (int)hipGetLastError();
}
template <class T>
int step_form(int form, const ScanStepArgs& a, void* stream) {
    const hipStream_t s = static_cast<hipStream_t>(stream);
    switch (form) {
        case 0: return step<T, 4, 2>(a, s);
        case 1: return step<T, 4, 4>(a, s);
        case 2: return step<T, 4, 8>(a, s);
        case 3: return step<T, 8, 8>(a, s);
        default: return step<T, 8, 16>(a, s);
    }
}

}  // namespace

int launch_scan_fwd(int dtype, int form, const ScanArgs& a, void* stream) {
    return dtype == WGRAD_BF16 ? scan_fwd_bf16(form, a, stream)
         : dtype == WGRAD_FP16 ? scan_fwd_fp16(form, a, stream) : scan_fwd_fp32(form, a, stream);
}
int launch_scan_bwd(int dtype, int form, const ScanArgs& a, void* stream) {
    return dtype == WGRAD_BF16 ? scan_bwd_bf16(form, a, stream)
         : dtype == WGRAD_FP16 ? scan_bwd_fp16(form, a, stream) : scan_bwd_fp32(form, a, stream);
}
int launch_scan_reduce(int dtype, const ScanReduceArgs& a, void* stream) {
    return dtype == WGRAD_BF16 ? reduce<Bf16>(a, stream) : dtype == WGRAD_FP16 ? reduce<Fp16>(a, stream) : reduce<Fp32>(a, stream);
}
int launch_scan_step(int dtype, int form, const ScanStepArgs& a, void* stream) {
    return dtype == WGRAD_BF16 ? step_form<Bf16>(form, a, stream)
         : dtype == WGRAD_FP16 ? step_form<Fp16>(form, a, stream) : step_form<Fp32>(form, a, stream);
}

}  // namespace ssm
}  // namespace wgrad
