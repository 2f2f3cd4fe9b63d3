// Device helpers of the selective state space kernels (gfx950 only).
#pragma once

#include <hip/hip_runtime.h>

#include "device_common.hpp"
#include "ssm_internal.hpp"

namespace wgrad {
namespace ssm {

using dev::lds_barrier;
using dev::u32x2;
using dev::u32x4;

struct Bf16 { uint16_t b; };
struct Fp16 { uint16_t b; };
struct Fp32 { float f; };

// E adjacent elements of a row, as loaded.
template <class T, int E>
struct Pack {
    static constexpr int kBytes = E * (int)sizeof(T);
    static constexpr int kWords = (kBytes + 3) / 4;
    uint32_t w[kWords];

    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = 0;
    }
    __device__ __forceinline__ float get(int i) const {
        if constexpr (sizeof(T) == 4) {
            return __builtin_bit_cast(float, w[i]);
        } else {
            const uint32_t v = w[i >> 1];
            if constexpr (__is_same(T, Bf16))
                return __builtin_bit_cast(float, (i & 1) ? (v & 0xffff0000u) : (v << 16));
            else
                return (float)__builtin_bit_cast(_Float16, (uint16_t)((i & 1) ? (v >> 16) : v));
        }
    }
    // round to nearest even
    __device__ __forceinline__ void set(int i, float f) {
        if constexpr (sizeof(T) == 4) {
            w[i] = __builtin_bit_cast(uint32_t, f);
        } else {
            uint16_t h;
            if constexpr (__is_same(T, Bf16))
                h = dev::f32_to_bf16(f);
            else
                h = __builtin_bit_cast(uint16_t, (_Float16)f);
            if (i & 1)
                w[i >> 1] = (w[i >> 1] & 0xffffu) | ((uint32_t)h << 16);
            else
                w[i >> 1] = h;
        }
    }
    // Through a pointer, as the kernels for single tokens do, which choose by
    // alignment. vec: p is aligned to the pack (at most 16 bytes; 8 where the
    // pack is an odd number of 8-byte halves) and nv is E or <= 0;
    // otherwise elements from nv on are not touched (loaded as zeros)
    __device__ __forceinline__ void load(const T* p, bool vec, int nv) {
        zero();
        if (nv <= 0) return;
        if (vec) {
            if constexpr (kBytes % 16 == 0) {
#pragma unroll
                for (int i = 0; i < kBytes / 16; ++i) {
                    const u32x4 v = reinterpret_cast<const u32x4*>(p)[i];
                    w[4 * i] = v[0], w[4 * i + 1] = v[1], w[4 * i + 2] = v[2], w[4 * i + 3] = v[3];
                }
            } else if constexpr (kBytes % 8 == 0) {
#pragma unroll
                for (int i = 0; i < kBytes / 8; ++i) {
                    const u32x2 v = reinterpret_cast<const u32x2*>(p)[i];
                    w[2 * i] = v[0], w[2 * i + 1] = v[1];
                }
            } else if constexpr (kBytes == 4) {
                w[0] = *reinterpret_cast<const uint32_t*>(p);
            } else {
                w[0] = *reinterpret_cast<const uint16_t*>(p);
            }
        } else {
#pragma unroll
            for (int i = 0; i < E; ++i)
                if (i < nv) put_bits(i, p + i);
        }
    }
    // The same through a buffer descriptor, as the kernels for whole sequences
    // do, without a branch and at any alignment of the elements (the unaligned
    // access mode): off is the byte offset of element 0, accesses of elements
    // from nv on are sent out of the buffer's range (loads give 0, stores are
    // dropped).
    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, uint32_t off, bool vec, int nv) {
        if (vec) {
            off = nv > 0 ? off : dev::kBufOob;
            if constexpr (kBytes % 16 == 0) {
#pragma unroll
                for (int i = 0; i < kBytes / 16; ++i) {
                    const u32x4 v = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, off + 16 * i, 0, 0));
                    w[4 * i] = v[0], w[4 * i + 1] = v[1], w[4 * i + 2] = v[2], w[4 * i + 3] = v[3];
                }
            } else if constexpr (kBytes % 8 == 0) {
#pragma unroll
                for (int i = 0; i < kBytes / 8; ++i) {
                    const u32x2 v = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(r, off + 8 * i, 0, 0));
                    w[2 * i] = v[0], w[2 * i + 1] = v[1];
                }
            } else if constexpr (kBytes == 4) {
                w[0] = (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(r, off, 0, 0);
            } else {
                w[0] = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(r, off, 0, 0);
            }
        } else {
            zero();
#pragma unroll
            for (int i = 0; i < E; ++i) {
                const uint32_t o = i < nv ? off + i * (uint32_t)sizeof(T) : dev::kBufOob;
                if constexpr (sizeof(T) == 4)
                    w[i] = (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(r, o, 0, 0);
                else
                    w[i >> 1] |= (uint32_t)(uint16_t)__builtin_amdgcn_raw_buffer_load_b16(r, o, 0, 0) << (i & 1 ? 16 : 0);
            }
        }
    }
    __device__ __forceinline__ void store(__amdgpu_buffer_rsrc_t r, uint32_t off, bool vec, int nv) const {
        if (vec) {
            off = nv > 0 ? off : dev::kBufOob;
            if constexpr (kBytes % 16 == 0) {
#pragma unroll
                for (int i = 0; i < kBytes / 16; ++i)
                    __builtin_amdgcn_raw_buffer_store_b128(u32x4{w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]}, r, off + 16 * i, 0, 0);
            } else if constexpr (kBytes == 8) {
                __builtin_amdgcn_raw_buffer_store_b64(u32x2{w[0], w[1]}, r, off, 0, 0);
            } else if constexpr (kBytes == 4) {
                __builtin_amdgcn_raw_buffer_store_b32(w[0], r, off, 0, 0);
            } else {
                __builtin_amdgcn_raw_buffer_store_b16((uint16_t)w[0], r, off, 0, 0);
            }
        } else {
#pragma unroll
            for (int i = 0; i < E; ++i) {
                const uint32_t o = i < nv ? off + i * (uint32_t)sizeof(T) : dev::kBufOob;
                if constexpr (sizeof(T) == 4)
                    __builtin_amdgcn_raw_buffer_store_b32(w[i], r, o, 0, 0);
                else
                    __builtin_amdgcn_raw_buffer_store_b16((uint16_t)(i & 1 ? w[i >> 1] >> 16 : w[i >> 1]), r, o, 0, 0);
            }
        }
    }
    __device__ __forceinline__ void put_bits(int i, const T* p) {
        if constexpr (sizeof(T) == 4)
            w[i] = *reinterpret_cast<const uint32_t*>(p);
        else if (i & 1)
            w[i >> 1] |= (uint32_t)(*reinterpret_cast<const uint16_t*>(p)) << 16;
        else
            w[i >> 1] = *reinterpret_cast<const uint16_t*>(p);
    }
    __device__ __forceinline__ void store(T* p, bool vec, int nv) const {
        if (nv <= 0) return;
        if (vec) {
            if constexpr (kBytes % 16 == 0) {
#pragma unroll
                for (int i = 0; i < kBytes / 16; ++i)
                    reinterpret_cast<u32x4*>(p)[i] = u32x4{w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]};
            } else if constexpr (kBytes == 8) {
                *reinterpret_cast<u32x2*>(p) = u32x2{w[0], w[1]};
            } else if constexpr (kBytes == 4) {
                *reinterpret_cast<uint32_t*>(p) = w[0];
            } else {
                *reinterpret_cast<uint16_t*>(p) = (uint16_t)w[0];
            }
        } else {
#pragma unroll
            for (int i = 0; i < E; ++i)
                if (i < nv) {
                    if constexpr (sizeof(T) == 4)
                        *reinterpret_cast<uint32_t*>(p + i) = w[i];
                    else
                        *reinterpret_cast<uint16_t*>(p + i) = (uint16_t)((i & 1) ? (w[i >> 1] >> 16) : w[i >> 1]);
                }
        }
    }
};

// A row operand as the scan kernels walk it, tile by tile: the tile's first
// row (uniform over the workgroup) and the byte offset in it of a lane's first
// place; its NR places are RK rows apart, E channels each from channel c on.
// Offsets in a tile are below 2 GiB, since a tile has at most 32 rows and the
// plan's limits keep row strides to 2^23 elements. Lanes whose channels are
// past the end (nv <= 0) have offsets that no access reaches.
template <class T, int E, int NR, int RK, bool VEC>
struct Walk {
    const T* row;
    uint32_t off, step;   // step: from one place to the next (uniform)

    __device__ __forceinline__ void start(const void* base, int64_t first_row, int64_t stride, int et, int c, int nv) {
        row = static_cast<const T*>(base) + first_row * stride;
        step = (uint32_t)(RK * (int)stride * (int)sizeof(T));
        off = nv > 0 ? (uint32_t)((et * (int)stride + c) * (int)sizeof(T)) : dev::kBufOob;
    }
    // to the tile `rows` rows on (or back)
    __device__ __forceinline__ void move(int rows, int64_t stride) { row += (int64_t)rows * stride; }
    // live: how many rows of the tile there are (et: this lane's first)
    __device__ __forceinline__ void load(Pack<T, E> (&v)[NR], int live, int et, int nv) const {
        const auto r = dev::buf_rsrc(row, 0x7fffffffu);
        if (live >= RK * NR) {
#pragma unroll
            for (int k = 0; k < NR; ++k) v[k].load(r, off + k * step, VEC, VEC ? E : nv);
        } else {
#pragma unroll
            for (int k = 0; k < NR; ++k) v[k].load(r, off + k * step, VEC, et + k * RK < live ? nv : 0);
        }
    }
    __device__ __forceinline__ void store(const Pack<T, E> (&v)[NR], int live, int et, int nv) const {
        const auto r = dev::buf_rsrc(row, 0x7fffffffu);
        if (live >= RK * NR) {
#pragma unroll
            for (int k = 0; k < NR; ++k) v[k].store(r, off + k * step, VEC, VEC ? E : nv);
        } else {
#pragma unroll
            for (int k = 0; k < NR; ++k) v[k].store(r, off + k * step, VEC, et + k * RK < live ? nv : 0);
        }
    }
};

template <class T>
__device__ __forceinline__ __amdgpu_buffer_rsrc_t tile_rsrc(const void* base, int64_t row, int64_t stride) {
    return dev::buf_rsrc(static_cast<const T*>(base) + row * stride, 0x7fffffffu);
}

// What a piece id stands for (see Pieces).
struct Piece {
    int n, j;        // sequence, piece of it
    int row0, len;   // the sequence's first row and length
    int t0, rows;    // the piece's first position in the sequence and its rows (<= 0: none)
    bool last;       // the sequence ends with this piece
};

// Uniform over the workgroup (every lane of every wave computes the same).
__device__ __forceinline__ Piece find_piece(const Pieces& pc, int id) {
    Piece r;
    if (!pc.seq_start) {
        r.n = id / pc.per_seq;
        r.j = id - r.n * pc.per_seq;
        r.row0 = r.n * pc.L;
        r.len = pc.L;
    } else {
        // the last n with floor(start / rows) + n <= id, 64 sequences at a time
        const int lane = threadIdx.x & 63;
        int found = 0;
        for (int base = 0; base < pc.N; base += 64) {
            const int n = base + lane;
            const bool le = n < pc.N && min(max(pc.seq_start[n], 0), pc.T) / pc.rows + n <= id;
            const int k = __popcll(__ballot(le));
            found += k;
            if (k < 64) break;
        }
        r.n = __builtin_amdgcn_readfirstlane(max(found - 1, 0));
        const SeqRows q = packed_rows(pc.seq_start[r.n], pc.seq_start[r.n + 1], pc.T, pc.L);
        r.row0 = __builtin_amdgcn_readfirstlane(q.row0);
        r.len = __builtin_amdgcn_readfirstlane(q.len);
        r.j = id - (r.row0 / pc.rows + r.n);
    }
    const PieceRows p = piece_rows(r.j, r.len, pc.rows);    // ids between two sequences name no piece
    r.t0 = p.t0, r.rows = p.rows, r.last = p.last;
    return r;
}

constexpr float kLog2e = 1.44269504088896341f;
constexpr float kLog2eLo = 1.92596299112661746e-8f;   // log2(e) - kLog2e
constexpr float kLn2 = 0.693147180559945309f;

// exp(x) for x <= 0 with an error of about one unit in the last place: the
// hardware's 2^p, whose argument p = x log2(e) is rounded, times
// 1 + (rest of the argument) ln 2.
__device__ __forceinline__ float exp_neg(float x) {
    const float p = x * kLog2e;
    const float r = __builtin_fmaf(x, kLog2eLo, __builtin_fmaf(x, kLog2e, -p));
    const float e = __builtin_amdgcn_exp2f(p);
    return x < -87.f ? e : __builtin_fmaf(e, r * kLn2, e);   // below, p may be infinite and r not a number
}

// A state's rate, times log2(e) for the hardware's 2^x, at least the lowest
// finite number: times the step 0, which stands for the rows past a sequence's
// end, an infinite one would not be the decay 1 but not a number.
__device__ __forceinline__ float decay_rate(float A) {
    const float r = A * kLog2e;
    return r < -3.402823466e38f ? -3.402823466e38f : r;
}

// The gate's sigmoid: the argument of 2^x rounded as it is, an error of about
// |z| 2^-24 next to the exact form's 2^-24, at half its instructions.
__device__ __forceinline__ float gate_sigmoid(float z) {
    return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-z * kLog2e));
}

// softplus(v) = max(v, 0) + log(1 + e^-|v|) and its derivative sigmoid(v).
// log(1 + e) = 2 atanh(e / (2 + e)) by its series in s = e / (2 + e) <= 1/3,
// exact to fp32 after s^15 (next term 3e-9 of the sum), and without the
// cancellation of log(1 + e) for small e.
// EXACT: the exponential of exp_neg. Without it the argument's own rounding
// stays, |v| 2^-24 relative: well below the rounding of a 16-bit delta, and
// five instructions less.
template <bool EXACT>
__device__ __forceinline__ float softplus(float v, float& sig) {
    const float e = EXACT ? exp_neg(-__builtin_fabsf(v)) : __builtin_amdgcn_exp2f(-__builtin_fabsf(v) * kLog2e);
    const float r = __builtin_amdgcn_rcpf(1.f + e);
    sig = v >= 0.f ? r : e * r;
    const float s = e * __builtin_amdgcn_rcpf(2.f + e);
    const float q = s * s;
    float p = 1.f / 15.f;
    p = __builtin_fmaf(p, q, 1.f / 13.f);
    p = __builtin_fmaf(p, q, 1.f / 11.f);
    p = __builtin_fmaf(p, q, 1.f / 9.f);
    p = __builtin_fmaf(p, q, 1.f / 7.f);
    p = __builtin_fmaf(p, q, 1.f / 5.f);
    p = __builtin_fmaf(p, q, 1.f / 3.f);
    const float s2 = s + s;
    return __builtin_fmaxf(v, 0.f) + __builtin_fmaf(s2 * q, p, s2);
}

template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true));
}
constexpr int kQuadXor1 = 0xB1, kQuadXor2 = 0x4E;    // quad_perm [1,0,3,2] and [2,3,0,1]
constexpr int kRowShl4 = 0x104, kRowRor4 = 0x124, kRowRor8 = 0x128, kRowHalfMirror = 0x141, kRowMirror = 0x140;

// Sum over the LPC adjacent lanes that share a channel; every one of them
// gets it.
template <int LPC>
__device__ __forceinline__ float lanes_sum(float v) {
    v += dpp<kQuadXor1>(v);
    if constexpr (LPC >= 4) v += dpp<kQuadXor2>(v);
    if constexpr (LPC >= 8) v += dpp<kRowHalfMirror>(v);   // lane i of 8 gets 7 - i: the other four, which are equal by now
    if constexpr (LPC >= 16) v += dpp<kRowMirror>(v);
    return v;
}

// The sum of value(0) .. value(n - 1) in one order, in levels of 16: a running
// sum's roundings grow with the root of its terms, these with that of a few
// tens. Values are asked for 16, 8 and 4 at a time, so that their loads go out
// together.
template <int K, class F>
__device__ __forceinline__ void add_values(float& sum, int& at, F value) {
    float v[K];
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = value(at + k);
#pragma unroll
    for (int k = 0; k < K; ++k) sum += v[k];
    at += K;
}
template <class F>
__device__ __forceinline__ float sum_of(int n, F value) {
    float all = 0.f, some = 0.f, few = 0.f;
    int at = 0;
    while (n - at >= 16) {
        few = 0.f;
        add_values<16>(few, at, value);
        some += few;
        if (at % 256 == 0) all += some, some = 0.f;
    }
    few = 0.f;
    if (n - at >= 8) add_values<8>(few, at, value);
    if (n - at >= 4) add_values<4>(few, at, value);
    while (at < n) add_values<1>(few, at, value);
    return all + (some + few);
}

}  // namespace ssm
}  // namespace wgrad
