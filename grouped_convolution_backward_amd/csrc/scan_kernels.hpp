// Selective scan kernels, forward and backward (gfx950), instantiated for one
// element type by each of scan_bf16.hip, scan_fp16.hip and scan_fp32.hip.
//
//   d_t = softplus(delta_t + bias), u_t = d_t x_t, a_t[s] = exp(d_t A[s])
//   h_t[s] = a_t[s] h_{t-1}[s] + u_t B_t[s],  y_t = sum_s C_t[s] h_t[s] + D x_t
//
// The decays differ for every channel and state, so there is no matrix
// product in it: each (row, channel, state) costs one exponential (a quarter
// rate instruction) and four multiply-adds, and that work, not the rows'
// bytes, is the bound. Layout for it: LPC adjacent lanes share a channel and
// hold NS of its states each in registers (256 / LPC channels per workgroup),
// and the sum over a lane's own states is free of cross-lane traffic. All that
// is needed once per (row, channel) -- softplus, u, the D term, the gate --
// is done once, by one lane each, while a tile of rows passes through LDS in
// fp32; B and C rows are staged there once for all channels of the workgroup.
// States shared out over waves instead of lanes, with B and C as scalar loads
// from an fp32 copy, took as long (8 x 2048 x 4096: 375 against 378 us) and
// needed the copy.
//
// Long sequences with few channels do not fill the card: they are split into
// segments. Since the product of decays over a segment is exp(A sum d), a
// first kernel leaves each segment's final state from zero and its sum of d,
// and the main kernel folds the segments before its own into its first state.
// That costs the exponentials twice, so the plan splits only as far as the
// card has room (choose_segment_rows).
//
// Rates of this card (ns per wave instruction and SIMD): multiply-add 1.1,
// exp2 3.7; one state's step (two multiplies, exp2, two multiply-adds) 8.3, and
// 10.3 with its share of the LDS rows. By the latter, a forward pass over 8 x
// 2048 rows of 4096 channels with 16 states needs 169 us, while its rows need
// 108 at the rate of a large copy (5.0 TB/s).
#pragma once

#include "ssm_device.hpp"

namespace wgrad {
namespace ssm {
namespace scan {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

template <bool B> struct Bool { static constexpr bool value = B; };
constexpr int least(int a, int b) { return a < b ? a : b; }

template <class T, int NS, int LPC>
struct Form {
    static constexpr int SP = NS * LPC;                                // states, padded
    static constexpr int CT = 256 / LPC;                               // channels per workgroup
    // A lane stages E adjacent channels of NR rows of a tile (forward, TT rows)
    // or chunk (backward), in one access of up to 16 bytes: the address unit
    // takes four lanes a cycle whatever each asks for. With two channels a lane,
    // bf16, 16 x 512 x 4096, 16 states: forward 163 us, backward 483 us; with
    // eight and four: 146 and 430 us.
    static constexpr int TT = LPC == 2 ? 16 : 32;
    static constexpr int E = least(scan_unit(LPC), 16 / (int)sizeof(T)), NR = TT * CT / 256 / E;
    static constexpr int EB = least(E, kChunk * CT / 256), NRB = kChunk * CT / 256 / EB;
    static constexpr int NB = (TT * SP / 4 + 255) / 256;               // quads of B states, and of C's, a lane stages
    static constexpr int NBB = (kChunk * SP / 4 + 255) / 256;
};

// The channel block of a workgroup: a group's channels, in units of the most
// adjacent channels that a lane stages, are dealt evenly to its blocks, so that
// no block is left with less than a unit, which would make every block's
// accesses single elements (training pass of 2 x 333 rows of 518 channels in 2
// groups, fp32: 67 us with blocks of 128, 128 and 3 channels, 51 us dealt evenly).
struct Block {
    int g, c0, end, blk;    // group, first channel, end of the channels, block over all groups
};
template <int UNIT>
__device__ __forceinline__ Block channel_block(const ScanArgs& a, int blk) {
    Block b;
    b.blk = blk;
    b.g = blk / a.cblks_g;
    const int i = blk - b.g * a.cblks_g, at = i * a.units + min(i, a.units_more);
    b.c0 = b.g * a.Cg + at * UNIT;
    b.end = min(b.c0 + (a.units + (i < a.units_more)) * UNIT, (b.g + 1) * a.Cg);
    return b;
}

// The first of the E channels that a lane stages, in a block with `in` of them.
// VEC: 0 = single elements; 2 = `in` is a multiple of E; 1 = it is not, but no less:
// the last lane's are moved back until they end with the block, so that every
// lane has all E, and what it shares with the lane before it is staged, and
// stored, the same twice. Vector accesses need no more than the element's
// alignment (the unaligned access mode that this platform runs in); 2 is an
// instance of its own because it can write two channels to LDS at once and
// clamps nothing (bf16, 16 states, 8 x 2048 rows: 319 us forward and 856
// backward with 4096 channels, 361 and 905 with 4095).
template <int E, int VEC>
__device__ __forceinline__ int lane_channel(int at, int in) {
    return VEC == 1 && at < in ? min(at, in - E) : at;
}

// Places of a channel in a row of LDS. A lane that stages adjacent channels
// writes 64 bytes in four accesses, and every fourth lane of an access would
// meet the same banks: from the 33rd channel of a row on (the 17th for the
// backward kernel's 16-byte places), neighbouring 16 bytes change places.
__device__ __forceinline__ int place8(int ch) { return ch ^ (ch >> 4 & 2); }
__device__ __forceinline__ int place16(int ch) { return ch ^ (ch >> 4 & 1); }

// Writes (a[i], b[i]) of a lane's E adjacent channels to their places.
template <int E, int VEC>
__device__ __forceinline__ void write_pairs(f32x2* row, int ec, const float (&a)[E], const float (&b)[E]) {
    if constexpr (VEC == 2 && E % 2 == 0) {
#pragma unroll
        for (int i = 0; i < E; i += 2) *reinterpret_cast<f32x4*>(row + place8(ec + i)) = f32x4{a[i], b[i], a[i + 1], b[i + 1]};
    } else {
#pragma unroll
        for (int i = 0; i < E; ++i) row[place8(ec + i)] = f32x2{a[i], b[i]};
    }
}

// A lane's states' rates (decay_rate). Padding
// states have B = C = 0: they stay 0 and add nothing. Their rate is negative,
// so that an infinite step is a decay of 0 to them (with a rate of 0 it would
// be NaN, which 0 times it is too).
template <int NS>
__device__ __forceinline__ void load_rates(const ScanArgs& a, int c, bool ok, int s0, float (&A2)[NS]) {
#pragma unroll
    for (int i = 0; i < NS; ++i) A2[i] = ok && s0 + i < a.S ? decay_rate(a.A[(int64_t)c * a.S + s0 + i]) : -1.f;
}
template <int NS>
__device__ __forceinline__ void load_state(const ScanArgs& a, const float* p, int n, int c, bool ok, int s0, float (&h)[NS]) {
#pragma unroll
    for (int i = 0; i < NS; ++i)
        h[i] = p && ok && s0 + i < a.S ? p[((int64_t)n * a.channels + c) * a.S + s0 + i] : 0.f;
}
template <int NS>
__device__ __forceinline__ void store_state(const ScanArgs& a, float* p, int n, int c, bool ok, int s0, const float (&h)[NS]) {
#pragma unroll
    for (int i = 0; i < NS; ++i)
        if (ok && s0 + i < a.S) p[((int64_t)n * a.channels + c) * a.S + s0 + i] = h[i];
}
// fp32 records of SP states per channel (segment sums, saved states)
template <int NS>
__device__ __forceinline__ void load_quads(const float* p, float (&h)[NS]) {
#pragma unroll
    for (int i = 0; i < NS; i += 4) {
        const f32x4 v = *reinterpret_cast<const f32x4*>(p + i);
        h[i] = v[0], h[i + 1] = v[1], h[i + 2] = v[2], h[i + 3] = v[3];
    }
}
template <int NS>
__device__ __forceinline__ void store_quads(float* p, const float (&h)[NS]) {
#pragma unroll
    for (int i = 0; i < NS; i += 4) *reinterpret_cast<f32x4*>(p + i) = f32x4{h[i], h[i + 1], h[i + 2], h[i + 3]};
}

// A state h carried over a segment whose decays multiply to 2^p and whose own
// sum is s. The factor is applied in two halves, each finite: it may be beyond
// fp32 where the carried state is small enough, or 0, and its product is not
// (growing states). Beyond 2^255.98 any state but 0 overflows as it would row
// by row. p is not a number only if s is none either.
__device__ __forceinline__ float carry(float p, float h, float s) {
    const float f = __builtin_amdgcn_exp2f(__builtin_fminf(0.5f * p, 127.99f));
    return __builtin_fmaf(f * h, f, s);
}

// The record of the states before row t (a multiple of kChunk) of a sequence.
__device__ __forceinline__ int64_t saved_slot(const ScanArgs& a, const Piece& pc, int t) {
    const int base = a.pc.seq_start ? pc.row0 / kChunk + pc.n : pc.n * ((a.pc.L + kChunk - 1) / kChunk);
    return base + t / kChunk;
}

// Four adjacent states of B and of C for each lane: quad k * 256 + lane of a
// tile of TT rows of SP / 4 quads.
template <class T, int NQ>
struct QuadRegs { Pack<T, 4> b[NQ], c[NQ]; };
template <class T, int SP, int TT, int NQ>
__device__ __forceinline__ void load_quads_bc(const ScanArgs& a, QuadRegs<T, NQ>& r, int64_t row, int rows, int g) {
    const auto rb = tile_rsrc<T>(a.B, row, a.sB), rc = tile_rsrc<T>(a.C, row, a.sC);
    auto load = [&](auto vec) {
#pragma unroll
        for (int k = 0; k < NQ; ++k) {
            const int qd = k * 256 + (int)threadIdx.x;
            const int t = qd / (SP / 4), s = qd % (SP / 4) * 4;
            const int nv = t < min(rows, TT) ? a.S - s : 0;
            r.b[k].load(rb, (uint32_t)((t * (int)a.sB + g * a.S + s) * (int)sizeof(T)), decltype(vec)::value, nv);
            r.c[k].load(rc, (uint32_t)((t * (int)a.sC + g * a.S + s) * (int)sizeof(T)), decltype(vec)::value, nv);
        }
    };
    if (a.vec_s)
        load(Bool<true>{});
    else
        load(Bool<false>{});
}
template <class T, int SP, int TT, int NQ>
__device__ __forceinline__ void stage_quads_bc(const QuadRegs<T, NQ>& r, float (&sB)[TT][SP], float (&sC)[TT][SP]) {
#pragma unroll
    for (int k = 0; k < NQ; ++k) {
        const int qd = k * 256 + (int)threadIdx.x;
        const int t = qd / (SP / 4), s = qd % (SP / 4) * 4;
        if (TT * SP / 4 % 256 == 0 || t < TT) {
            *reinterpret_cast<f32x4*>(&sB[t][s]) = f32x4{r.b[k].get(0), r.b[k].get(1), r.b[k].get(2), r.b[k].get(3)};
            *reinterpret_cast<f32x4*>(&sC[t][s]) = f32x4{r.c[k].get(0), r.c[k].get(1), r.c[k].get(2), r.c[k].get(3)};
        }
    }
}

// Step sizes of N values, and the slopes of their softplus. One branch for all
// of them, so that their instructions interleave: an exponential or reciprocal
// is followed by a wait unless something independent stands between it and its
// use.
template <class T, int N>
__device__ __forceinline__ void step_sizes(const ScanArgs& a, const float (&raw)[N], float (&d)[N], float (&sig)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) d[i] = raw[i], sig[i] = 1.f;
    if (a.softplus) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float slope;
            d[i] = softplus<__is_same(T, Fp32)>(raw[i], slope);
            sig[i] = slope;
        }
    }
}

// Sums of LPC values over the LPC lanes of a channel: lane q gets that of
// v[q]. The steps halve the values a lane goes on with, half the additions of
// summing each for every lane.
template <int LPC>
__device__ __forceinline__ float deal_sum(const float (&v)[LPC], int q) {
    if constexpr (LPC == 2) {
        return (q & 1 ? v[1] : v[0]) + dpp<kQuadXor1>(q & 1 ? v[0] : v[1]);
    } else if constexpr (LPC == 4) {
        const float a = (q & 1 ? v[1] : v[0]) + dpp<kQuadXor1>(q & 1 ? v[0] : v[1]);
        const float b = (q & 1 ? v[3] : v[2]) + dpp<kQuadXor1>(q & 1 ? v[2] : v[3]);
        return (q & 2 ? b : a) + dpp<kQuadXor2>(q & 2 ? a : b);
    } else {
        float r = 0.f;
#pragma unroll
        for (int k = 0; k < LPC; ++k) {
            const float t = lanes_sum<LPC>(v[k]);
            r = k == q ? t : r;
        }
        return r;
    }
}

// Forward. SUM: the segment's state from zero and its sum of d only.
// bf16, 16 states, 8 x 2048 rows of 4096 channels: 319 us, half the rate that
// the instructions alone allow. The rest is the staging of a tile (a quarter of
// a workgroup's cycles: softplus, conversions, LDS writes), its loads and
// stores, and two or three waves a SIMD to cover them. As segments of one
// sequence, 1 x 16384 x 4096: 437 us, two fifths of them for the sums.
// Tiles of 32 rows (16 with 128 channels) cost two barriers each and leave room
// for five workgroups a CU.
template <class T, int NS, int LPC, int VEC, bool SUM>
__global__ __launch_bounds__(256) void fwd_kernel(const ScanArgs a) {
    using F = Form<T, NS, LPC>;
    constexpr int SP = F::SP, CT = F::CT, TT = F::TT, E = F::E, NR = F::NR, NB = F::NB;
    constexpr int U = LPC > 8 ? LPC : 8;        // rows between two checks for the end
    __shared__ __attribute__((aligned(16))) f32x2 sDU[TT][CT];         // d, u
    __shared__ float sY[SUM ? 1 : TT][CT];
    __shared__ float sBias[CT], sD[CT];
    __shared__ __attribute__((aligned(16))) float sB[TT][SP];
    __shared__ __attribute__((aligned(16))) float sC[TT][SP];

    const int nblk = a.cblks_g * a.G;
    const uint32_t group = a.first + blockIdx.x;
    const int id = group / nblk;
    const Block cb = channel_block<scan_unit(LPC)>(a, group - id * nblk);
    const Piece pc = find_piece(a.pc, id);
    if (SUM ? (pc.rows <= 0 || pc.last) : (pc.rows <= 0 && !pc.last)) return;

    const int tid = threadIdx.x, q = tid % LPC, ch = tid / LPC, s0 = q * NS, at = place8(ch);
    const int c = cb.c0 + ch;
    const bool ok = c < cb.end;
    float A2[NS], h[NS];
    load_rates<NS>(a, c, ok, s0, A2);
    if constexpr (SUM) {
#pragma unroll
        for (int i = 0; i < NS; ++i) h[i] = 0.f;
    } else {
        load_state<NS>(a, a.init_state, pc.n, c, ok, s0, h);
#pragma unroll 4
        for (int j = 0; j < pc.j; ++j) {
            const int64_t rec = (int64_t)(id - pc.j + j) * a.channels + (ok ? c : 0);
            const float sd = a.sum_d[rec];
            float s[NS];
            load_quads<NS>(a.sums + rec * SP + s0, s);
#pragma unroll
            for (int i = 0; i < NS; ++i) h[i] = carry(A2[i] * sd, h[i], s[i]);
        }
    }
    float sum_d = 0.f;

    // this lane's places in a tile when rows are staged and stored
    constexpr int RK = 256 / (CT / E);          // rows between them
    const int et = tid / (CT / E), ec = lane_channel<E, VEC>(tid % (CT / E) * E, cb.end - cb.c0);
    const int enc = min(cb.end - cb.c0 - ec, E);
    const int64_t row0 = (int64_t)pc.row0 + pc.t0;
    Walk<T, E, NR, RK, VEC != 0> wx, wd, wz, wy;
    wx.start(a.x, row0, a.sx, et, cb.c0 + ec, enc);
    wd.start(a.delta, row0, a.sdelta, et, cb.c0 + ec, enc);
    if constexpr (!SUM) {
        wz.start(a.z, row0, a.sz, et, cb.c0 + ec, enc);
        wy.start(a.y, row0, a.sy, et, cb.c0 + ec, enc);
    }
    Pack<T, E> bx[NR], bd[NR], bz[NR];          // the next tile, as loaded
    QuadRegs<T, NB> bq;
    auto fetch = [&](int t0) {                  // tiles in order
        wx.load(bx, pc.rows - t0, et, enc);
        wd.load(bd, pc.rows - t0, et, enc);
        wx.move(TT, a.sx);
        wd.move(TT, a.sdelta);
        if (!SUM && a.z) {
            wz.load(bz, pc.rows - t0, et, enc);
            wz.move(TT, a.sz);
        }
        load_quads_bc<T, SP, TT, NB>(a, bq, row0 + t0, pc.rows - t0, cb.g);
    };
    Pack<T, E> x[NR], z[NR];                    // of the tile in LDS
    auto stage = [&](int t0) {
        float raw[NR * E], d[NR * E], sig[NR * E];
#pragma unroll
        for (int k = 0; k < NR; ++k) {
            x[k] = bx[k], z[k] = bz[k];
#pragma unroll
            for (int i = 0; i < E; ++i) raw[k * E + i] = bd[k].get(i) + sBias[ec + i];
        }
        step_sizes<T, NR * E>(a, raw, d, sig);
#pragma unroll
        for (int k = 0; k < NR; ++k) {
            const int t = et + k * RK;
            const bool live = t0 + t < pc.rows;
            float dv[E], u[E];
#pragma unroll
            for (int i = 0; i < E; ++i) {
                // rows past the end: decay 1, nothing added (channels past the end have x 0)
                dv[i] = live ? d[k * E + i] : 0.f;
                u[i] = dv[i] * x[k].get(i);
            }
            write_pairs<E, VEC>(sDU[t], ec, dv, u);
        }
        stage_quads_bc<T, SP, TT, NB>(bq, sB, sC);
    };
    if (tid < CT) {
        const bool in = cb.c0 + tid < cb.end;
        sBias[tid] = a.delta_bias && in ? a.delta_bias[cb.c0 + tid] : 0.f;
        sD[tid] = !SUM && a.D && in ? a.D[cb.c0 + tid] : 0.f;
    }
    lds_barrier();
    if (pc.rows > 0) {
        fetch(0);
        stage(0);
        if (TT < pc.rows) fetch(TT);
    }
    for (int t0 = 0; t0 < pc.rows; t0 += TT) {
        lds_barrier();
        for (int tb = 0; tb < TT; tb += U) {
            if (t0 + tb >= pc.rows) break;
            if (!SUM && a.saved && (t0 + tb) % kChunk == 0 && ok)
                store_quads<NS>(a.saved + (saved_slot(a, pc, pc.t0 + t0 + tb) * a.channels + c) * SP + s0, h);
            float part[LPC];                    // a lane's shares of y of the last LPC rows
#pragma unroll
            for (int tu = 0; tu < U; ++tu) {
                const int t = tb + tu;
                const f32x2 du = sDU[t][at];
                float acc = 0.f;
#pragma unroll
                for (int i = 0; i < NS; ++i) {
                    const float ai = __builtin_amdgcn_exp2f(du[0] * A2[i]);
                    h[i] = __builtin_fmaf(ai, h[i], du[1] * sB[t][s0 + i]);
                    if (!SUM) acc = __builtin_fmaf(sC[t][s0 + i], h[i], acc);
                }
                if constexpr (SUM) {
                    sum_d += du[0];
                } else {
                    part[tu % LPC] = acc;
                    if (tu % LPC == LPC - 1) sY[t - (LPC - 1) + q][ch] = deal_sum<LPC>(part, q);
                }
            }
        }
        lds_barrier();
        // The next tile is staged before this one's rows are stored: loads and
        // stores retire in order, so a wait for the tile's loads behind fresh
        // stores would wait for those to reach memory.
        Pack<T, E> out[NR];
        if constexpr (!SUM) {
            float v[NR][E];
#pragma unroll
            for (int k = 0; k < NR; ++k)
#pragma unroll
                for (int i = 0; i < E; ++i) v[k][i] = __builtin_fmaf(sD[ec + i], x[k].get(i), sY[et + k * RK][ec + i]);
            if (a.z) {
#pragma unroll
                for (int k = 0; k < NR; ++k)
#pragma unroll
                    for (int i = 0; i < E; ++i) {
                        const float zz = z[k].get(i);
                        v[k][i] *= zz * gate_sigmoid(zz);
                    }
            }
#pragma unroll
            for (int k = 0; k < NR; ++k)
#pragma unroll
                for (int i = 0; i < E; ++i) out[k].set(i, v[k][i]);
        }
        if (t0 + TT < pc.rows) stage(t0 + TT);
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (!SUM) {
            wy.store(out, pc.rows - t0, et, enc);
            wy.move(TT, a.sy);
        }
        if (t0 + 2 * TT < pc.rows) fetch(t0 + 2 * TT);
    }
    if constexpr (SUM) {
        const int64_t rec = (int64_t)id * a.channels + c;
        if (ok) {
            store_quads<NS>(a.sums + rec * SP + s0, h);
            if (q == 0) a.sum_d[rec] = sum_d;
        }
    } else {
        if (a.final_state && pc.last) store_state<NS>(a, a.final_state, pc.n, c, ok, s0, h);
    }
}

// The gradient's sum of a segment: with e_t = C_t dy_t + a_{t+1} e_{t+1} and
// nothing behind the segment, what reaches the state before its first row.
template <class T, int NS, int LPC, int VEC>
__global__ __launch_bounds__(256) void bwd_sum_kernel(const ScanArgs a) {
    using F = Form<T, NS, LPC>;
    constexpr int SP = F::SP, CT = F::CT, TT = F::TT, E = F::E, NR = F::NR, NB = F::NB;
    __shared__ __attribute__((aligned(16))) f32x2 sDG[TT][CT];         // d, gated dy
    __shared__ float sBias[CT];
    __shared__ __attribute__((aligned(16))) float sB[TT][SP];
    __shared__ __attribute__((aligned(16))) float sC[TT][SP];

    const int nblk = a.cblks_g * a.G;
    const uint32_t group = a.first + blockIdx.x;
    const int id = group / nblk;
    const Block cb = channel_block<scan_unit(LPC)>(a, group - id * nblk);
    const Piece pc = find_piece(a.pc, id);
    if (pc.rows <= 0 || pc.j == 0) return;

    const int tid = threadIdx.x, q = tid % LPC, ch = tid / LPC, s0 = q * NS, at = place8(ch);
    const int c = cb.c0 + ch;
    const bool ok = c < cb.end;
    float A2[NS], e[NS];
    load_rates<NS>(a, c, ok, s0, A2);
#pragma unroll
    for (int i = 0; i < NS; ++i) e[i] = 0.f;
    float sum_d = 0.f;

    // this lane's places in a tile when rows are staged and stored
    constexpr int RK = 256 / (CT / E);          // rows between them
    const int et = tid / (CT / E), ec = lane_channel<E, VEC>(tid % (CT / E) * E, cb.end - cb.c0);
    const int enc = min(cb.end - cb.c0 - ec, E);
    const int64_t row0 = (int64_t)pc.row0 + pc.t0;
    const int last = (pc.rows - 1) / TT * TT;
    Walk<T, E, NR, RK, VEC != 0> wd, wg, wz;
    wd.start(a.delta, row0 + last, a.sdelta, et, cb.c0 + ec, enc);
    wg.start(a.dy, row0 + last, a.sdy, et, cb.c0 + ec, enc);
    wz.start(a.z, row0 + last, a.sz, et, cb.c0 + ec, enc);
    Pack<T, E> bd[NR], bg[NR], bz[NR];
    QuadRegs<T, NB> bq;
    auto fetch = [&](int t0) {                  // tiles in order, from the last
        wd.load(bd, pc.rows - t0, et, enc);
        wg.load(bg, pc.rows - t0, et, enc);
        wd.move(-TT, a.sdelta);
        wg.move(-TT, a.sdy);
        if (a.z) {
            wz.load(bz, pc.rows - t0, et, enc);
            wz.move(-TT, a.sz);
        }
        load_quads_bc<T, SP, TT, NB>(a, bq, row0 + t0, pc.rows - t0, cb.g);
    };
    if (tid < CT) sBias[tid] = a.delta_bias && cb.c0 + tid < cb.end ? a.delta_bias[cb.c0 + tid] : 0.f;
    fetch(last);
    for (int t0 = last; t0 >= 0; t0 -= TT) {
        lds_barrier();
        float raw[NR * E], d[NR * E], sig[NR * E], g[NR * E];
#pragma unroll
        for (int k = 0; k < NR; ++k)
#pragma unroll
            for (int i = 0; i < E; ++i) raw[k * E + i] = bd[k].get(i) + sBias[ec + i], g[k * E + i] = bg[k].get(i);
        step_sizes<T, NR * E>(a, raw, d, sig);
        if (a.z) {
#pragma unroll
            for (int k = 0; k < NR; ++k)
#pragma unroll
                for (int i = 0; i < E; ++i) {
                    const float zz = bz[k].get(i);
                    g[k * E + i] *= zz * gate_sigmoid(zz);
                }
        }
#pragma unroll
        for (int k = 0; k < NR; ++k) {
            const int t = et + k * RK;
            const bool live = t0 + t < pc.rows;
            float dv[E], gv[E];
#pragma unroll
            for (int i = 0; i < E; ++i) dv[i] = live ? d[k * E + i] : 0.f, gv[i] = live ? g[k * E + i] : 0.f;
            write_pairs<E, VEC>(sDG[t], ec, dv, gv);
        }
        stage_quads_bc<T, SP, TT, NB>(bq, sB, sC);
        if (t0 > 0) fetch(t0 - TT);
        lds_barrier();
        for (int tb = TT - 8; tb >= 0; tb -= 8) {
#pragma unroll
            for (int tu = 7; tu >= 0; --tu) {
                const int t = tb + tu;
                const f32x2 dg = sDG[t][at];
#pragma unroll
                for (int i = 0; i < NS; ++i)
                    e[i] = __builtin_amdgcn_exp2f(dg[0] * A2[i]) * __builtin_fmaf(sC[t][s0 + i], dg[1], e[i]);
                sum_d += dg[0];
            }
        }
    }
    if (ok) {
        const int64_t rec = (int64_t)id * a.channels + c;
        store_quads<NS>(a.sums + rec * SP + s0, e);
        if (q == 0) a.sum_d[rec] = sum_d;
    }
}

__device__ __forceinline__ void swap_add32(float& a, float b) {
    const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(int, a), __builtin_bit_cast(int, b), false, false);
    a = __builtin_bit_cast(float, (int)r[0]) + __builtin_bit_cast(float, (int)r[1]);
}
__device__ __forceinline__ void swap_add16(float& a, float b) {
    const auto r = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(int, a), __builtin_bit_cast(int, b), false, false);
    a = __builtin_bit_cast(float, (int)r[0]) + __builtin_bit_cast(float, (int)r[1]);
}
template <int CTRL>
__device__ __forceinline__ void pick_add(float& a, float b, bool upper) {
    const float keep = upper ? b : a, send = upper ? a : b;
    a = keep + dpp<CTRL>(send);
}

// Sums V values over the channels of a wave (lane bits from log2(LPC) up).
// Each step over one lane bit also halves the values a lane holds while there
// is more than one: lanes with the bit set go on with the upper half. After
// it a lane holds V / (values dealt out) sums, the first of which is value
// number `first`; lanes for which `writes` is false hold nothing of use.
template <int V, int LPC>
struct ChannelSum {
    static constexpr int kBits = LPC == 2 ? 5 : LPC == 4 ? 4 : LPC == 8 ? 3 : 2;
    static constexpr int kLog = V == 8 ? 3 : 4;
    static constexpr int kLeft = kBits >= kLog ? 1 : V >> kBits;
    int first;
    bool writes, up8;
    __device__ __forceinline__ explicit ChannelSum(int lane) {
        static_assert(V == 8 || V == 16, "values per lane");
        static_assert(V == 8 || LPC >= 8, "halving steps below lane bit 3 are not provided");
        first = (lane & 32 ? V / 2 : 0) + (lane & 16 ? V / 4 : 0);
        if (LPC <= 8) first += lane & 8 ? V / 8 : 0;
        up8 = lane & 8;
        writes = LPC >= 8 || (lane & (8 - LPC)) == 0;
    }
    __device__ __forceinline__ void sum(float (&v)[V]) const {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) swap_add32(v[i], v[i + V / 2]);
#pragma unroll
        for (int i = 0; i < V / 4; ++i) swap_add16(v[i], v[i + V / 4]);
        if constexpr (LPC <= 8) {
#pragma unroll
            for (int i = 0; i < V / 8; ++i) pick_add<kRowRor8>(v[i], v[i + V / 8], up8);
        }
        // V == 8 from here on: one value left
        if constexpr (LPC <= 4) v[0] += dpp<kRowShl4>(v[0]);
        if constexpr (LPC <= 2) v[0] += dpp<kQuadXor2>(v[0]);
    }
};

// Backward. A segment's rows are taken in chunks of kChunk from its end. For
// a chunk the lanes first run forward again from the saved state before it,
// keeping every decay and state in registers (no exponential is computed
// twice), then backward:
//   e_t = C_t dy_t + (a e)_{t+1},  dC_t = sum_c dy_t h_t,  dB_t = sum_c u_t e_t,
//   du_t = sum_s B_t e_t,  g = a_t e_t h_{t-1},  dA += d_t g,  dd_t = sum_s A g
// The sums over the channels of a wave deal their results out over the lanes
// as they go, about two instructions per value; the waves' shares are joined
// in LDS and leave one partial per channel block, which the reduce kernel adds
// in one order. GATE: z is there, so y is needed again for dz.
// bf16, 16 states, gated, 8 x 2048 rows of 4096 channels: 855 us. Of a chunk's
// cycles the forward run takes 24 %, the run back with its sums 42, staging 14,
// loads 10, stores 6, the rest 4: bound by instructions, at two waves a SIMD,
// since decays and states fill the registers. Chunks of 8 rows, with room for
// more waves, were slower (1046 us against 946 at the time) and doubled what
// forward saves. The saved states cost forward 3 %.
// The launch bound: four states a lane fit the 256 registers that two waves a
// SIMD leave each, some with scratch (17 to 32 states without a gate, 44 to 60
// bytes a lane; fp32 with 16 states and a gate, 8 or 16). Eight states a lane
// (S > 32) do not fit and run one wave a SIMD, with 150 to 205 AGPRs beyond
// them. So do two lanes a channel (S <= 8): up to 142 AGPRs, and with a gate the
// LDS of 128 channels, 101 (bf16) or 105 KB (fp32), has room for one workgroup.
// 4 x 2048 x 4096 bf16, us: 8 states 481, 16 states 510, 64 states 2213, 128
// states 4751.
template <class T, int NS, int LPC, int VEC, bool GATE>
__global__ __launch_bounds__(256, NS == 4 && LPC > 2 ? 2 : 1) void bwd_kernel(const ScanArgs a) {
    using F = Form<T, NS, LPC>;
    constexpr int SP = F::SP, CT = F::CT, E = F::EB, NR = F::NRB, NB = F::NBB, K = kChunk;
    using CS = ChannelSum<2 * NS, LPC>;
    __shared__ f32x4 sIn[K][CT];                 // d, u, gated dy, slope of softplus
    __shared__ float2 sOut[K][CT];               // du, dd
    __shared__ float sY[GATE ? K : 1][CT];       // sum_s C h
    __shared__ float sG[GATE ? K : 1][CT];       // sigmoid(z)
    constexpr int PW = Pack<T, E>::kWords;
    __shared__ uint32_t sPack[GATE ? 3 : 1][NR * PW][256];   // x, and dy and z, as loaded
    __shared__ float sBias[CT], sD[CT];
    __shared__ __attribute__((aligned(16))) float sB[K][SP];
    __shared__ __attribute__((aligned(16))) float sC[K][SP];
    __shared__ float sP[4][K][2 * SP + CS::kLeft];   // a row's last places: from lanes that hold nothing of use
    // Sums over rows that each lane keeps for itself. A running sum over a long
    // segment would round as often as it has chunks (dD over 16384 rows, fp32:
    // 5.2e-7 off); each 16 chunks' sums are added here instead (1.7e-7).
    __shared__ float sSum[2 * E][256];

    const int nblk = a.cblks_g * a.G;
    const uint32_t group = a.first + blockIdx.x;
    const int id = group / nblk;
    const Block cb = channel_block<scan_unit(LPC)>(a, group - id * nblk);
    const Piece pc = find_piece(a.pc, id);
    const int rows = max(pc.rows, 0);

    const int tid = threadIdx.x, q = tid % LPC, ch = tid / LPC, s0 = q * NS;
    const int lane = tid & 63, wave = tid >> 6;
    const int c = cb.c0 + ch;
    const bool ok = c < cb.end;
    float A2[NS], e[NS], dA[NS];
    load_rates<NS>(a, c, ok, s0, A2);
#pragma unroll
    for (int i = 0; i < NS; ++i) dA[i] = e[i] = 0.f;
    if (pc.last || rows > 0) {
        load_state<NS>(a, a.dfinal_state, pc.n, c, ok, s0, e);
        const int last_j = pc.len > 0 ? (pc.len - 1) / a.pc.rows : 0;
#pragma unroll 4
        for (int j = last_j; j > pc.j; --j) {
            const int64_t rec = (int64_t)(id - pc.j + j) * a.channels + (ok ? c : 0);
            const float sd = a.sum_d[rec];
            float s[NS];
            load_quads<NS>(a.sums + rec * SP + s0, s);
#pragma unroll
            for (int i = 0; i < NS; ++i) e[i] = carry(A2[i] * sd, e[i], s[i]);
        }
        // lanes past the block's last channel read another channel's records: their e enters the sums over channels, where 0
        // times it is not 0 if it is infinite
#pragma unroll
        for (int i = 0; i < NS; ++i) e[i] = ok ? e[i] : 0.f;
    }
    const CS cs(lane);
    // where this lane's first sum goes in a partial row
    const int pcol = cs.writes ? (cs.first >= NS ? SP : 0) + s0 + cs.first % NS : 2 * SP;

    // this lane's places in a chunk when rows are staged and stored
    constexpr int RK = 256 / (CT / E);          // rows between them
    const int et = tid / (CT / E), ec = lane_channel<E, VEC>(tid % (CT / E) * E, cb.end - cb.c0);
    const int enc = min(cb.end - cb.c0 - ec, E);
    const int64_t row0 = (int64_t)pc.row0 + pc.t0;
    float dD[E], dbias[E];
#pragma unroll
    for (int i = 0; i < E; ++i) dD[i] = dbias[i] = 0.f;
#pragma unroll
    for (int i = 0; i < 2 * E; ++i) sSum[i][tid] = 0.f;
    // channels past the end: no lane stages every one of them, all are summed over
    for (int i = tid; i < K * CT; i += 256) (&sIn[0][0])[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (tid < CT) {
        const bool in = cb.c0 + tid < cb.end;
        sBias[tid] = a.delta_bias && in ? a.delta_bias[cb.c0 + tid] : 0.f;
        sD[tid] = a.D && in ? a.D[cb.c0 + tid] : 0.f;
    }
    lds_barrier();
    const int last = rows > 0 ? (rows - 1) / K * K : -K;
    Walk<T, E, NR, RK, VEC != 0> wx, wd, wg, wz, ox, od, oz;
    wx.start(a.x, row0 + last, a.sx, et, cb.c0 + ec, enc);
    wd.start(a.delta, row0 + last, a.sdelta, et, cb.c0 + ec, enc);
    wg.start(a.dy, row0 + last, a.sdy, et, cb.c0 + ec, enc);
    ox.start(a.dx, row0 + last, a.sdx, et, cb.c0 + ec, enc);
    od.start(a.ddelta, row0 + last, a.sddelta, et, cb.c0 + ec, enc);
    if constexpr (GATE) {
        wz.start(a.z, row0 + last, a.sz, et, cb.c0 + ec, enc);
        oz.start(a.dz, row0 + last, a.sdz, et, cb.c0 + ec, enc);
    }
    Pack<T, E> bx[NR], bd[NR], bg[NR], bz[NR];   // the next chunk, as loaded
    QuadRegs<T, NB> bq;
    float h0[NS];
    auto fetch = [&](int t0) {                   // chunks in order, from the last
        wx.load(bx, rows - t0, et, enc);
        wd.load(bd, rows - t0, et, enc);
        wg.load(bg, rows - t0, et, enc);
        wx.move(-K, a.sx);
        wd.move(-K, a.sdelta);
        wg.move(-K, a.sdy);
        if constexpr (GATE) {
            wz.load(bz, rows - t0, et, enc);
            wz.move(-K, a.sz);
        }
        load_quads_bc<T, SP, K, NB>(a, bq, row0 + t0, rows - t0, cb.g);
        load_quads<NS>(a.saved + (saved_slot(a, pc, pc.t0 + t0) * a.channels + (ok ? c : 0)) * SP + s0, h0);
    };
    // What the epilogue needs of a row waits in LDS: the registers belong to
    // the decays and states.
    float hb[NS];
    auto stage = [&](int t0) {
        float raw[NR * E], d[NR * E], sg[NR * E];
#pragma unroll
        for (int k = 0; k < NR; ++k) {
#pragma unroll
            for (int w = 0; w < PW; ++w) {
                sPack[0][k * PW + w][tid] = bx[k].w[w];
                if constexpr (GATE) sPack[1][k * PW + w][tid] = bg[k].w[w], sPack[2][k * PW + w][tid] = bz[k].w[w];
            }
#pragma unroll
            for (int i = 0; i < E; ++i) raw[k * E + i] = bd[k].get(i) + sBias[ec + i];
        }
        step_sizes<T, NR * E>(a, raw, d, sg);
#pragma unroll
        for (int k = 0; k < NR; ++k) {
            const int t = et + k * RK;
            const bool live = t0 + t < rows;
#pragma unroll
            for (int i = 0; i < E; ++i) {
                // rows past the end: decay 1, nothing added (channels past the end have x and dy 0)
                const float dv = live ? d[k * E + i] : 0.f;
                float g = bg[k].get(i);
                if constexpr (GATE) {
                    const float z = bz[k].get(i), gs = gate_sigmoid(z);
                    sG[t][ec + i] = gs;
                    g *= z * gs;
                }
                sIn[t][place16(ec + i)] = f32x4{dv, dv * bx[k].get(i), live ? g : 0.f, sg[k * E + i]};
            }
        }
        stage_quads_bc<T, SP, K, NB>(bq, sB, sC);
#pragma unroll
        for (int i = 0; i < NS; ++i) hb[i] = ok ? h0[i] : 0.f;
    };
    if (rows > 0) {
        fetch(last);
        stage(last);
        if (last > 0) fetch(last - K);
    }
    for (int t0 = last; t0 >= 0; t0 -= K) {
        lds_barrier();
        float hs[K][NS], as[K][NS];
        // The LDS reads of a row are issued one row ahead and no further
        // (the barrier to the scheduler): hoisted all together they would
        // take the registers that the states are in.
        struct Row { f32x4 in; float b[NS], c[NS]; };
        auto read = [&](int t) {
            Row r;
            r.in = sIn[t][place16(ch)];
#pragma unroll
            for (int i = 0; i < NS; ++i) r.b[i] = sB[t][s0 + i], r.c[i] = sC[t][s0 + i];
            return r;
        };
        Row cur = read(0);
        float part[LPC];
#pragma unroll
        for (int t = 0; t < K; ++t) {
            const Row nx = t < K - 1 ? read(t + 1) : cur;
            float acc = 0.f;
#pragma unroll
            for (int i = 0; i < NS; ++i) {
                as[t][i] = __builtin_amdgcn_exp2f(cur.in[0] * A2[i]);
                hs[t][i] = __builtin_fmaf(as[t][i], t ? hs[t > 0 ? t - 1 : 0][i] : hb[i], cur.in[1] * cur.b[i]);
                if constexpr (GATE) acc = __builtin_fmaf(cur.c[i], hs[t][i], acc);
            }
            if constexpr (GATE) {
                part[t % LPC] = acc;
                if (t % LPC == LPC - 1) sY[t - (LPC - 1) + q][ch] = deal_sum<LPC>(part, q);
            }
            if (t < K - 1) cur = nx;
            __builtin_amdgcn_sched_barrier(0x207);
        }
        float dAc[NS], v[2 * NS];
#pragma unroll
        for (int i = 0; i < NS; ++i) dAc[i] = 0.f;
        // A row's sums over the channels are taken while the next row is
        // worked on: their steps depend on each other, and alone would leave
        // waits between them.
#pragma unroll
        for (int t = K - 1; t >= -1; --t) {
            const Row nx = t > 0 ? read(t > 0 ? t - 1 : 0) : cur;
            if (t < K - 1) {
                cs.sum(v);
#pragma unroll
                for (int i = 0; i < CS::kLeft; ++i) sP[wave][t + 1][pcol + i] = v[i];
            }
            if (t >= 0) {
                float du = 0.f, dd = 0.f, w[2 * NS];
#pragma unroll
                for (int i = 0; i < NS; ++i) {
                    e[i] = __builtin_fmaf(cur.c[i], cur.in[2], e[i]);
                    w[i] = cur.in[1] * e[i];
                    w[NS + i] = cur.in[2] * hs[t > 0 ? t : 0][i];
                    du = __builtin_fmaf(cur.b[i], e[i], du);
                    e[i] *= as[t > 0 ? t : 0][i];
                    const float gg = e[i] * (t > 0 ? hs[t > 0 ? t - 1 : 0][i] : hb[i]);
                    dd = __builtin_fmaf(A2[i], gg, dd);
                    dAc[i] = __builtin_fmaf(cur.in[0], gg, dAc[i]);
                }
                float o;                                   // even lanes write du, odd ones dd, some of them the same
                if constexpr (LPC == 8) {
                    du = lanes_sum<LPC>(du);
                    dd = lanes_sum<LPC>(dd);
                    o = q & 1 ? dd : du;
                } else {                                   // each sums its own of the two from the first step on
                    o = (q & 1 ? dd : du) + dpp<kQuadXor1>(q & 1 ? du : dd);
                    if constexpr (LPC >= 4) o += dpp<kQuadXor2>(o);
                    if constexpr (LPC >= 16) o += dpp<kRowRor4>(o);
                    if constexpr (LPC >= 16) o += dpp<kRowRor8>(o);
                }
                reinterpret_cast<float*>(&sOut[t > 0 ? t : 0][ch])[q & 1] = o;
#pragma unroll
                for (int i = 0; i < 2 * NS; ++i) v[i] = w[i];
            }
            cur = nx;
            __builtin_amdgcn_sched_barrier(0x207);
        }
#pragma unroll
        for (int i = 0; i < NS; ++i) dA[i] += dAc[i];
        lds_barrier();

        const int64_t row = row0 + t0;
        constexpr int NP = (K * 2 * SP + 255) / 256;
        float pv[NP];
#pragma unroll
        for (int w = 0; w < NP; ++w) {
            const int at = w * 256 + tid, t = at / (2 * SP) % K, s = at % (2 * SP);
            pv[w] = (sP[0][t][s] + sP[1][t][s]) + (sP[2][t][s] + sP[3][t][s]);
        }
        Pack<T, E> vx[NR], vd[NR], vz[NR];
#pragma unroll
        for (int k = 0; k < NR; ++k) {
            const int t = et + k * RK;
            const bool live = t0 + t < rows;
            Pack<T, E> px, pg, pz;
#pragma unroll
            for (int w = 0; w < PW; ++w) {
                px.w[w] = sPack[0][k * PW + w][tid];
                if constexpr (GATE) pg.w[w] = sPack[1][k * PW + w][tid], pz.w[w] = sPack[2][k * PW + w][tid];
            }
#pragma unroll
            for (int i = 0; i < E; ++i) {
                const float2 o = sOut[t][ec + i];
                const f32x4 in = sIn[t][place16(ec + i)];
                const float x = px.get(i), Dv = sD[ec + i];
                if constexpr (GATE) {
                    const float y = __builtin_fmaf(Dv, x, sY[t][ec + i]);
                    const float z = pz.get(i), gs = sG[t][ec + i];
                    vz[k].set(i, pg.get(i) * y * gs * __builtin_fmaf(z, 1.f - gs, 1.f));
                }
                const float dr = __builtin_fmaf(x, o.x, o.y * kLn2) * in[3];
                vx[k].set(i, __builtin_fmaf(in[0], o.x, Dv * in[2]));
                vd[k].set(i, dr);
                dD[i] += live ? in[2] * x : 0.f;
                dbias[i] += live ? dr : 0.f;
            }
        }
        if ((t0 / K) % 16 == 0) {                          // the last of them at t0 = 0
#pragma unroll
            for (int i = 0; i < E; ++i) {
                sSum[i][tid] += dD[i], dD[i] = 0.f;
                sSum[E + i][tid] += dbias[i], dbias[i] = 0.f;
            }
        }
        // The next chunk is staged before this one's rows are stored: loads and
        // stores retire in order, so a wait for the chunk's loads behind fresh
        // stores would wait for those to reach memory.
        if (t0 > 0) stage(t0 - K);
        __builtin_amdgcn_sched_barrier(0);
        const auto rp = dev::buf_rsrc(a.part_bc + ((int64_t)cb.blk * a.pc.T + row) * (2 * SP), 0x7fffffffu);
#pragma unroll
        for (int w = 0; w < NP; ++w) {
            const int at = w * 256 + tid;
            __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, pv[w]), rp,
                                                  at < min(K, rows - t0) * (2 * SP) ? (uint32_t)at * 4u : dev::kBufOob, 0, 0);
        }
        ox.store(vx, rows - t0, et, enc);
        od.store(vd, rows - t0, et, enc);
        ox.move(-K, a.sdx);
        od.move(-K, a.sddelta);
        if constexpr (GATE) {
            oz.store(vz, rows - t0, et, enc);
            oz.move(-K, a.sdz);
        }
        if (t0 > K) fetch(t0 - 2 * K);
    }

    if (ok) store_quads<NS>(a.part_a + ((int64_t)id * a.channels + c) * SP + s0, dA);
    if (a.dinit_state && pc.j == 0 && (pc.last || rows > 0)) store_state<NS>(a, a.dinit_state, pc.n, c, ok, s0, e);
    // dD and ddelta_bias: join the lanes of each channel in one order
    lds_barrier();
    float* const sR = reinterpret_cast<float*>(&sIn[0][0]);
#pragma unroll
    for (int i = 0; i < E; ++i) {
        sR[et * CT + ec + i] = sSum[i][tid];
        sR[(RK + et) * CT + ec + i] = sSum[E + i][tid];
    }
    lds_barrier();
    for (int w = tid; w < 2 * CT; w += 256) {
        const int which = w / CT, cc = w % CT;
        if (cb.c0 + cc < cb.end) {
            float v = 0.f;
            for (int t = 0; t < RK; ++t) v += sR[(which * RK + t) * CT + cc];
            a.part_d[((int64_t)id * 2 + which) * a.channels + cb.c0 + cc] = v;
        }
    }
}

// The sums of all segments go out before the kernels that fold them.
template <class F>
int launch_all(const ScanArgs& a, F launch) {
    ScanArgs v = a;
    for_launches((int64_t)a.pc.count * a.cblks_g * a.G, [&](uint32_t first, uint32_t grid) {
        v.first = first;
        launch(grid, v);
    });
    return (int)hipGetLastError();
}
template <class T, int NS, int LPC, int VEC>
int run_fwd(const ScanArgs& a, hipStream_t s) {
    if (a.split) launch_all(a, [&](uint32_t grid, const ScanArgs& v) { fwd_kernel<T, NS, LPC, VEC, true><<<grid, 256, 0, s>>>(v); });
    return launch_all(a, [&](uint32_t grid, const ScanArgs& v) { fwd_kernel<T, NS, LPC, VEC, false><<<grid, 256, 0, s>>>(v); });
}
template <class T, int NS, int LPC, int VEC>
int run_bwd(const ScanArgs& a, hipStream_t s) {
    if (a.split) launch_all(a, [&](uint32_t grid, const ScanArgs& v) { bwd_sum_kernel<T, NS, LPC, VEC><<<grid, 256, 0, s>>>(v); });
    return launch_all(a, [&](uint32_t grid, const ScanArgs& v) {
        if (a.z)
            bwd_kernel<T, NS, LPC, VEC, true><<<grid, 256, 0, s>>>(v);
        else
            bwd_kernel<T, NS, LPC, VEC, false><<<grid, 256, 0, s>>>(v);
    });
}

template <class T, int NS, int LPC>
int fwd(const ScanArgs& a, hipStream_t s) {
    return a.vec_c == 2 ? run_fwd<T, NS, LPC, 2>(a, s) : a.vec_c ? run_fwd<T, NS, LPC, 1>(a, s) : run_fwd<T, NS, LPC, 0>(a, s);
}
template <class T, int NS, int LPC>
int bwd(const ScanArgs& a, hipStream_t s) {
    return a.vec_c == 2 ? run_bwd<T, NS, LPC, 2>(a, s) : a.vec_c ? run_bwd<T, NS, LPC, 1>(a, s) : run_bwd<T, NS, LPC, 0>(a, s);
}

// form: index of kScanForms
template <class T>
int dispatch_fwd(int form, const ScanArgs& a, void* stream) {
    const hipStream_t s = static_cast<hipStream_t>(stream);
    switch (form) {
        case 0: return fwd<T, 4, 2>(a, s);
        case 1: return fwd<T, 4, 4>(a, s);
        case 2: return fwd<T, 4, 8>(a, s);
        case 3: return fwd<T, 8, 8>(a, s);
        default: return fwd<T, 8, 16>(a, s);
    }
}
template <class T>
int dispatch_bwd(int form, const ScanArgs& a, void* stream) {
    const hipStream_t s = static_cast<hipStream_t>(stream);
    switch (form) {
        case 0: return bwd<T, 4, 2>(a, s);
        case 1: return bwd<T, 4, 4>(a, s);
        case 2: return bwd<T, 4, 8>(a, s);
        case 3: return bwd<T, 8, 8>(a, s);
        default: return bwd<T, 8, 16>(a, s);
    }
}

}  // namespace scan

int scan_fwd_bf16(int form, const ScanArgs& a, void* stream);
int scan_bwd_bf16(int form, const ScanArgs& a, void* stream);
int scan_fwd_fp16(int form, const ScanArgs& a, void* stream);
int scan_bwd_fp16(int form, const ScanArgs& a, void* stream);
int scan_fwd_fp32(int form, const ScanArgs& a, void* stream);
int scan_bwd_fp32(int form, const ScanArgs& a, void* stream);

}  // namespace ssm
}  // namespace wgrad
