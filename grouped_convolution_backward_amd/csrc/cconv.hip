// Causal depthwise convolution with bias and SiLU: forward, backward and the
// form for one token per sequence (gfx950).
//
//   p[r] = bias + sum_k w[k] x[r - (W-1) + k],   y = p or p sigmoid(p)
//   g = dy (act'(p)),  dx[r] = sum_k w[k] g[r + (W-1) - k],
//   dw[k] = sum_r g[r] x[r - (W-1) + k],  dbias = sum_r g[r]
//
// Every value is read for W - 1 multiply-adds only, so the kernels are bound
// by streaming the rows: lanes own E adjacent channels (16 bytes forward, 8
// backward at 16-bit types), walk down a run of rows with the last W - 1
// inputs in registers, and have a batch of rows in flight ahead of the one
// they work on. A run re-reads the W - 1 rows before it (and the backward
// kernel the W - 1 after it), which the run beside it in the same workgroup
// has just brought into the cache.
//
// Arithmetic is fp32; only the stored outputs are rounded.
#include <hip/hip_runtime.h>

#include "ssm_device.hpp"

namespace wgrad {
namespace ssm {
namespace {

constexpr int kBatch = 4;   // rows loaded ahead

// The rows of a piece and what stands before them, for one lane's channels:
// byte offsets count from `base`, the piece's first row or the window before
// it (uniform over the workgroup), and stay below 2 GiB by the plan's limits on
// strides and rows of a piece. Rows and channels that are not there have
// offsets out of the descriptors' range, so that no access is a branch.
template <class T, int E, int W, bool VEC>
struct Rows {
    __amdgpu_buffer_rsrc_t x, init;
    int base, len, sx, c, C, nv;
    bool have_init;

    __device__ __forceinline__ Rows(const CconvArgs& a, const Piece& pc, int c_, int nv_) {
        base = max(pc.t0 - (W - 1), 0);
        len = pc.len;
        x = tile_rsrc<T>(a.x, (int64_t)pc.row0 + base, a.sx);
        init = tile_rsrc<T>(a.init, (int64_t)pc.n * (W - 1), a.C);
        sx = (int)a.sx * (int)sizeof(T);
        c = c_ * (int)sizeof(T);
        C = a.C * (int)sizeof(T);
        nv = nv_;
        have_init = a.init;
    }
    __device__ __forceinline__ uint32_t at(int t, int stride) const { return row_offset(t, base, stride, c); }
    __device__ __forceinline__ void row(Pack<T, E>& v, int t) const { v.load(x, at(t, sx), VEC, t < len ? nv : 0); }
    // row t of a window: the sequence's for t >= 0, its initial state's for -(W-1) <= t < 0
    __device__ __forceinline__ void window(Pack<T, E>& v, int t) const {
        Pack<T, E> s;
        v.load(x, at(t, sx), VEC, t >= 0 && t < len ? nv : 0);
        s.load(init, row_offset(t, 1 - W, C, c), VEC, have_init && t < 0 ? nv : 0);
#pragma unroll
        for (int i = 0; i < Pack<T, E>::kWords; ++i) v.w[i] |= s.w[i];     // one of them is zeros
    }
};

// A lane's channels. VEC (C >= E): the last lane's are moved back until they
// end with the row, so that every lane has E of them; the ones it shares with
// the lane before it are computed, and written, the same twice. Vector accesses
// need no more than the element's alignment here: they go through buffer
// descriptors, in the unaligned access mode that this platform runs in (through
// pointers the compiler may assume a vector's alignment), and an odd row stride
// costs a few percent, not the vector. Only rows shorter than a vector are accessed by single elements.
template <int E, bool VEC>
struct Lane {
    int c, nv;
    __device__ __forceinline__ Lane(const CconvArgs& a, int at) {
        c = VEC && at < a.C ? min(at, a.C - E) : at;
        nv = min(a.C - c, E);
    }
};

template <class T, int E, int W, bool VEC>
__device__ __forceinline__ void load_params(const CconvArgs& a, int c, int nv, float (&w)[W][E], float (&b)[E]) {
    Pack<T, E * W> taps;
    taps.load(dev::buf_rsrc(a.w, 0x7fffffffu), (uint32_t)(c * W * (int)sizeof(T)), VEC, nv * W);
    Pack<T, E> bias;
    bias.load(dev::buf_rsrc(a.bias, 0x7fffffffu), (uint32_t)(c * (int)sizeof(T)), VEC, a.bias ? nv : 0);
#pragma unroll
    for (int i = 0; i < E; ++i) {
        b[i] = bias.get(i);
#pragma unroll
        for (int k = 0; k < W; ++k) w[k][i] = taps.get(i * W + k);
    }
}

// Forward. bf16, W = 4, SiLU, 8 x 4096 rows of 4096 channels: 104 us, 5.2 TB/s,
// a large copy's rate.
template <class T, int E, int W, bool VEC, bool SILU>
__global__ __launch_bounds__(256) void cconv_kernel(const CconvArgs a) {
    const uint32_t wg = a.first + blockIdx.x;
    const int id = wg / a.cblks, cb = wg - id * a.cblks;
    const Piece pc = find_piece(a.pc, id);
    if (pc.rows <= 0 && !pc.last) return;
    const int cl = a.cl, lane = threadIdx.x & (cl - 1), slot = threadIdx.x / cl;
    const Lane<E, VEC> ln(a, (cb * cl + lane) * E);
    const int c = ln.c, nv = ln.nv;
    if (nv <= 0) return;
    const int first = pc.t0 + slot * a.run;
    const int end = min(first + a.run, pc.len);
    const Rows<T, E, W, VEC> rows(a, pc, c, nv);

    if (first < end) {
        Pack<T, E> next[kBatch], old[W];
#pragma unroll
        for (int k = 1; k < W; ++k) rows.window(old[k], first - W + k);
#pragma unroll
        for (int u = 0; u < kBatch; ++u) rows.row(next[u], first + u);
        float w[W][E], bias[E];
        load_params<T, E, W, VEC>(a, c, nv, w, bias);
        float xw[W][E];               // the last W inputs, oldest first
#pragma unroll
        for (int k = 1; k < W; ++k)
#pragma unroll
            for (int i = 0; i < E; ++i) xw[k][i] = old[k].get(i);
        const auto ry = tile_rsrc<T>(a.y, (int64_t)pc.row0 + rows.base, a.sy);
        const int sy = (int)a.sy * (int)sizeof(T);
        for (int t = first; t < end; t += kBatch) {
            Pack<T, E> cur[kBatch];
#pragma unroll
            for (int u = 0; u < kBatch; ++u) cur[u] = next[u];
#pragma unroll
            for (int u = 0; u < kBatch; ++u) rows.row(next[u], t + kBatch + u < end ? t + kBatch + u : pc.len);
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                Pack<T, E> out;
#pragma unroll
                for (int i = 0; i < E; ++i) {
#pragma unroll
                    for (int k = 0; k < W - 1; ++k) xw[k][i] = xw[k + 1][i];
                    xw[W - 1][i] = cur[u].get(i);
                    float p = bias[i];
#pragma unroll
                    for (int k = 0; k < W; ++k) p = __builtin_fmaf(w[k][i], xw[k][i], p);
                    if constexpr (SILU) p *= __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-p * kLog2e));
                    out.set(i, p);
                }
                out.store(ry, rows.at(t + u, sy), VEC, t + u < end ? nv : 0);
            }
        }
    }
    // the run that ends the sequence leaves its last W - 1 inputs
    if (a.final_state && pc.last && (end == pc.len) && (first < end || (pc.len == 0 && slot == 0))) {
        const auto rf = tile_rsrc<T>(a.final_state, (int64_t)pc.n * (W - 1), a.C);
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
            Pack<T, E> v;
            rows.window(v, pc.len - (W - 1) + j);
            v.store(rf, row_offset(j, 0, rows.C, rows.c), VEC, nv);
        }
    }
}

// A run of rows first .. end-1: walks s = first .. end+W-2, forming g[s] from
// the window of x and dy[s], and after each g[s] finishes dx[s - (W-1)]. The
// run's own rows enter dw and dbias; the W - 1 after them only dx. The first
// run of a sequence also finishes the gradients of the W - 1 rows before it
// (dinit). bf16, W = 4, SiLU, 8 x 2048 rows of 4096 channels: 97 us with its join, 4.2 TB/s of
// x, dy and dx: near the bytes, with 2 x W multiply-adds and an exponential per
// element under them.
template <class T, int E, int W, bool VEC, bool SILU>
__global__ __launch_bounds__(256) void cconv_bwd_kernel(const CconvArgs a) {
    const uint32_t wg = a.first + blockIdx.x;
    const int id = wg / a.cblks, cb = wg - id * a.cblks;
    const Piece pc = find_piece(a.pc, id);
    const int cl = a.cl, lane = threadIdx.x & (cl - 1), slot = threadIdx.x / cl;
    const Lane<E, VEC> ln(a, (cb * cl + lane) * E);
    const int c = ln.c, nv = ln.nv;
    const int first = pc.t0 + slot * a.run;
    const int end = min(first + a.run, pc.len);
    const bool starts = pc.j == 0 && slot == 0;            // the sequence's first run, even of no rows

    float dw[W][E], db[E];
#pragma unroll
    for (int i = 0; i < E; ++i) {
        db[i] = 0.f;
#pragma unroll
        for (int k = 0; k < W; ++k) dw[k][i] = 0.f;
    }
    if (nv > 0 && (first < end || starts)) {
        const Rows<T, E, W, VEC> rows(a, pc, c, nv);
        const auto rdy = tile_rsrc<T>(a.dy, (int64_t)pc.row0 + rows.base, a.sdy),
                   rdx = tile_rsrc<T>(a.dx, (int64_t)pc.row0 + rows.base, a.sdx);
        const int sdy = (int)a.sdy * (int)sizeof(T), sdx = (int)a.sdx * (int)sizeof(T);
        auto read = [&](Pack<T, E>& vx, Pack<T, E>& vd, int t) {
            rows.row(vx, t);
            vd.load(rdy, rows.at(t, sdy), VEC, t < pc.len ? nv : 0);
        };
        Pack<T, E> nx[kBatch], nd[kBatch], old[W];
#pragma unroll
        for (int k = 1; k < W; ++k) rows.window(old[k], first - W + k);
#pragma unroll
        for (int u = 0; u < kBatch; ++u) read(nx[u], nd[u], first + u);
        float w[W][E], bias[E];
        load_params<T, E, W, VEC>(a, c, nv, w, bias);
        float xw[W][E], gw[W][E];      // the last W inputs and gradients, oldest first
#pragma unroll
        for (int k = 1; k < W; ++k)
#pragma unroll
            for (int i = 0; i < E; ++i) xw[k][i] = old[k].get(i), gw[k][i] = 0.f;
        // moves both windows on by row s and returns dx of row s - (W - 1)
        auto advance = [&](const Pack<T, E>& vx, const Pack<T, E>& vd, float (&dx)[E]) {
#pragma unroll
            for (int i = 0; i < E; ++i) {
#pragma unroll
                for (int k = 0; k < W - 1; ++k) xw[k][i] = xw[k + 1][i], gw[k][i] = gw[k + 1][i];
                xw[W - 1][i] = vx.get(i);
                float g = vd.get(i);
                if constexpr (SILU) {
                    float p = bias[i];
#pragma unroll
                    for (int k = 0; k < W; ++k) p = __builtin_fmaf(w[k][i], xw[k][i], p);
                    const float sg = __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-p * kLog2e));
                    g *= sg * __builtin_fmaf(p, 1.f - sg, 1.f);
                }
                gw[W - 1][i] = g;
                dx[i] = 0.f;
#pragma unroll
                for (int k = 0; k < W; ++k) dx[i] = __builtin_fmaf(w[k][i], gw[W - 1 - k][i], dx[i]);
            }
        };
        // dx of row s - (W - 1) again at a sequence's ends, from its own rows only: a weight times the 0 that stands for the
        // gradient of another row is not 0 if the weight is infinite
        auto inner = [&](int s, float (&dx)[E]) {
#pragma unroll
            for (int i = 0; i < E; ++i) {
                dx[i] = 0.f;
#pragma unroll
                for (int k = 0; k < W; ++k)
                    if (s - k >= 0 && s - k < pc.len) dx[i] = __builtin_fmaf(w[k][i], gw[W - 1 - k][i], dx[i]);
            }
        };
        const int fin = a.dfinal ? pc.len - (W - 1) : 1 << 30;   // rows from here on are in the final state too
        auto finish = [&](int r, float (&dx)[E]) {         // r: the row whose dx is complete
            if (r < 0 && starts) inner(r + W - 1, dx);
            if (r >= fin) {
                Pack<T, E> v;
                v.load(tile_rsrc<T>(a.dfinal, (int64_t)pc.n * (W - 1), a.C), row_offset(r, fin, rows.C, rows.c), VEC, nv);
#pragma unroll
                for (int i = 0; i < E; ++i) dx[i] += v.get(i);
            }
            Pack<T, E> out;
#pragma unroll
            for (int i = 0; i < E; ++i) out.set(i, dx[i]);
            out.store(rdx, rows.at(r, sdx), VEC, r >= first && r < end ? nv : 0);
            if (r < 0 && starts && a.dinit)
                out.store(tile_rsrc<T>(a.dinit, (int64_t)pc.n * (W - 1), a.C), row_offset(r, 1 - W, rows.C, rows.c), VEC, nv);
        };
        // whole batches of the run's own rows
        int t = first;
        for (; t + kBatch <= end; t += kBatch) {
            Pack<T, E> cx[kBatch], cd[kBatch];
#pragma unroll
            for (int u = 0; u < kBatch; ++u) cx[u] = nx[u], cd[u] = nd[u];
#pragma unroll
            for (int u = 0; u < kBatch; ++u) read(nx[u], nd[u], t + kBatch + u);
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                float dx[E];
                advance(cx[u], cd[u], dx);
#pragma unroll
                for (int i = 0; i < E; ++i) {
                    const float g = gw[W - 1][i];
                    db[i] += g;
#pragma unroll
                    for (int k = 0; k < W; ++k) dw[k][i] = __builtin_fmaf(g, xw[k][i], dw[k][i]);
                }
                finish(t + u - (W - 1), dx);
            }
        }
        // the rest of them, and the W - 1 rows after
        for (; t < end + W - 1; t += kBatch) {
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                const int r = t + u;
                if (r >= end + W - 1) break;
                float dx[E];
                advance(nx[u], nd[u], dx);
                if (r >= pc.len) {                         // past the sequence: no gradient, whatever a state's NaN made of it
#pragma unroll
                    for (int i = 0; i < E; ++i) gw[W - 1][i] = 0.f;
                    inner(r, dx);
                }
                if (r < end) {
#pragma unroll
                    for (int i = 0; i < E; ++i) {
                        const float g = gw[W - 1][i];
                        db[i] += g;
#pragma unroll
                        for (int k = 0; k < W; ++k) dw[k][i] = __builtin_fmaf(g, xw[k][i], dw[k][i]);
                    }
                }
                finish(r - (W - 1), dx);
            }
            if (t + kBatch < end + W - 1) {
#pragma unroll
                for (int u = 0; u < kBatch; ++u) read(nx[u], nd[u], t + kBatch + u);
            }
        }
    }

    // sum the runs of the workgroup in one order and leave one partial per piece
    __shared__ float part[256][E];
    for (int k = 0; k <= W; ++k) {
#pragma unroll
        for (int i = 0; i < E; ++i) {
            float v = db[i];
#pragma unroll
            for (int q = 0; q < W; ++q) v = k == q ? dw[q][i] : v;
            part[threadIdx.x][i] = v;
        }
        __syncthreads();
        if (slot == 0 && nv > 0) {
#pragma unroll
            for (int i = 0; i < E; ++i) {
                const float v = sum_of(256 / cl, [&](int s) { return part[s * cl + lane][i]; });
                if (i < nv) a.part[((int64_t)id * (W + 1) + k) * a.C + c + i] = v;
            }
        }
        __syncthreads();
    }
}

// dw and dbias from the pieces' partials: 32 channels of one tap per
// workgroup, the pieces dealt to 8 lanes each and joined in one order, in
// levels (65536 sequences of 8 rows, fp32: dw 1.5e-6 off as a running sum).
__global__ __launch_bounds__(256) void cconv_reduce_kernel(const CconvReduceArgs a) {
    const int k = blockIdx.y, c = blockIdx.x * 32 + (threadIdx.x & 31), sl = threadIdx.x >> 5;
    float v = 0.f;
    if (c < a.C)
        v = sum_of((a.pieces - sl + 7) / 8, [&](int p) { return a.part[((int64_t)(8 * p + sl) * (a.W + 1) + k) * a.C + c]; });
    __shared__ float part[256];
    part[threadIdx.x] = v;
    __syncthreads();
    if (sl || c >= a.C) return;
    for (int s = 1; s < 8; ++s) v += part[s * 32 + threadIdx.x];
    if (k < a.W)
        a.dw[(int64_t)c * a.W + k] = v;
    else if (a.dbias)
        a.dbias[c] = v;
}

// One token per row: a lane takes E channels of one row through its state.
// Bound by its bytes: 256 rows of 4096 channels, fp16, W = 4, 5.0 us for 17 MB
// with 2.8 us of it the launch and one trip to memory (which is what a single
// row of 2048 channels takes).
template <class T, int E, int W>
__global__ __launch_bounds__(256) void cconv_step_kernel(const CconvStepArgs a) {
    const int cv = (a.C + E - 1) / E;
    const int64_t idx = (int64_t)(a.first + blockIdx.x) * 256 + threadIdx.x;
    const int64_t row = idx / cv;
    if (row >= a.rows) return;
    const int c = (int)(idx - row * cv) * E;
    const int nv = min(a.C - c, E);
    const bool vec = a.vec != 0;
    const int64_t at = a.slots ? a.slots[row] : row;
    const bool live = at >= 0 && at < a.num_slots;
    T* st = static_cast<T*>(a.state) + (live ? at : 0) * (W - 1) * a.C + c;
    Pack<T, E> x[W], bias;
#pragma unroll
    for (int k = 0; k < W - 1; ++k) x[k].load(st + (int64_t)k * a.C, vec, live ? nv : 0);
    x[W - 1].load(static_cast<const T*>(a.x) + row * a.sx + c, vec, nv);
    bias.load(static_cast<const T*>(a.bias) + c, vec, a.bias ? nv : 0);
    Pack<T, E * W> taps;
    taps.load(static_cast<const T*>(a.w) + (int64_t)c * W, vec, nv * W);
    Pack<T, E> out;
#pragma unroll
    for (int i = 0; i < E; ++i) {
        float p = bias.get(i);
#pragma unroll
        for (int k = 0; k < W; ++k) p = __builtin_fmaf(taps.get(i * W + k), x[k].get(i), p);
        if (a.silu) p *= __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-p * kLog2e));
        out.set(i, live ? p : 0.f);
    }
    out.store(static_cast<T*>(a.y) + row * a.sy + c, vec, nv);
#pragma unroll
    for (int k = 0; k < W - 1; ++k) x[k + 1].store(st + (int64_t)k * a.C, vec, live ? nv : 0);
}

// Calls f with the element type and the tap count as compile-time constants.
template <int W> struct Taps { static constexpr int value = W; };
template <class F>
int by_taps(int W, F f) {
    switch (W) {
        case 1: return f(Taps<1>{});
        case 2: return f(Taps<2>{});
        case 3: return f(Taps<3>{});
        case 4: return f(Taps<4>{});
        case 5: return f(Taps<5>{});
        case 6: return f(Taps<6>{});
        case 7: return f(Taps<7>{});
        default: return f(Taps<8>{});
    }
}
template <class F>
int by_type(int dtype, F f) {
    if (dtype == WGRAD_BF16) return f(Bf16{});
    if (dtype == WGRAD_FP16) return f(Fp16{});
    return f(Fp32{});
}

}  // namespace

int launch_cconv(int dtype, const CconvArgs& a, void* stream) {
    return by_type(dtype, [&](auto t) {
        using T = decltype(t);
        return by_taps(a.W, [&](auto w) {
            constexpr int E = 16 / sizeof(T);
            constexpr int W = decltype(w)::value;
            const hipStream_t s = static_cast<hipStream_t>(stream);
            CconvArgs v = a;
            for_launches((int64_t)a.pc.count * a.cblks, [&](uint32_t first, uint32_t grid) {
                v.first = first;
                if (a.vec && a.silu)
                    cconv_kernel<T, E, W, true, true><<<grid, 256, 0, s>>>(v);
                else if (a.vec)
                    cconv_kernel<T, E, W, true, false><<<grid, 256, 0, s>>>(v);
                else if (a.silu)
                    cconv_kernel<T, E, W, false, true><<<grid, 256, 0, s>>>(v);
                else
                    cconv_kernel<T, E, W, false, false><<<grid, 256, 0, s>>>(v);
            });
            return (int)hipGetLastError();
        });
    });
}

int launch_cconv_bwd(int dtype, const CconvArgs& a, void* stream) {
    return by_type(dtype, [&](auto t) {
        using T = decltype(t);
        return by_taps(a.W, [&](auto w) {
            constexpr int E = kConvBwdVec, W = decltype(w)::value;
            const hipStream_t s = static_cast<hipStream_t>(stream);
            CconvArgs v = a;
            for_launches((int64_t)a.pc.count * a.cblks, [&](uint32_t first, uint32_t grid) {
                v.first = first;
                if (a.vec && a.silu)
                    cconv_bwd_kernel<T, E, W, true, true><<<grid, 256, 0, s>>>(v);
                else if (a.vec)
                    cconv_bwd_kernel<T, E, W, true, false><<<grid, 256, 0, s>>>(v);
                else if (a.silu)
                    cconv_bwd_kernel<T, E, W, false, true><<<grid, 256, 0, s>>>(v);
                else
                    cconv_bwd_kernel<T, E, W, false, false><<<grid, 256, 0, s>>>(v);
            });
            return (int)hipGetLastError();
        });
    });
}

int launch_cconv_reduce(const CconvReduceArgs& a, void* stream) {
    cconv_reduce_kernel<<<dim3((unsigned)((a.C + 31) / 32), (unsigned)(a.W + 1)), 256, 0,
                          static_cast<hipStream_t>(stream)>>>(a);
    return (int)hipGetLastError();
}

int launch_cconv_step(int dtype, const CconvStepArgs& a, void* stream) {
    return by_type(dtype, [&](auto t) {
        using T = decltype(t);
        return by_taps(a.W, [&](auto w) {
            constexpr int E = 16 / sizeof(T);
            const int64_t threads = a.rows * ((a.C + E - 1) / E);
            CconvStepArgs v = a;
            for_launches((threads + 255) / 256, [&](uint32_t first, uint32_t grid) {
                v.first = first;
                cconv_step_kernel<T, E, decltype(w)::value><<<grid, 256, 0, static_cast<hipStream_t>(stream)>>>(v);
            });
            return (int)hipGetLastError();
        });
    });
}

}  // namespace ssm
}  // namespace wgrad
