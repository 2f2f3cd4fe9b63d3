// Plans and kernel-argument blocks of the selective state space operators
// (causal convolution and selective scan). Not part of the public interface.
#pragma once

#include <cstdint>

#include "../../include/wgrad_ssm.h"

namespace wgrad {
namespace ssm {

// The rows of all sequences are cut into pieces of `rows` rows that never
// cross a sequence. A piece id names (sequence n, piece j of n). Dense: every
// sequence has `per_seq` pieces, id = n * per_seq + j. Packed: the pieces of
// sequence n start at id floor(seq_start[n] / rows) + n, which leaves each
// sequence at least max(1, ceil(length / rows)) ids of its own, so that
// floor(T / rows) + N ids cover everything and a kernel finds n from the id
// by comparing ids with seq_start, whatever the lengths are.
struct Pieces {
    const int32_t* seq_start;   // NULL: dense
    int32_t N, L, T;            // sequences, rows per sequence (packed: at most), rows in all
    int32_t rows;               // rows of a piece
    int32_t per_seq;            // dense: pieces per sequence
    int32_t count;              // piece ids in all
};

// The rows of a packed sequence from two neighbouring values of seq_start,
// whatever they are: 0 <= row0 <= row0 + len <= T and len <= L. No sum of two
// of the numbers is formed, since T and L go up to 2^30 each. Host and device.
struct SeqRows { int32_t row0, len; };
constexpr SeqRows packed_rows(int32_t from, int32_t to, int32_t T, int32_t L) {
    const int32_t s = from < 0 ? 0 : from > T ? T : from;
    const int32_t e = to < s ? s : to > T ? T : to;
    return {s, e - s < L ? e - s : L};
}

// Where piece j of a sequence of len rows lies in it, for any j: its first row
// and its rows (<= 0: none), and whether the sequence ends with it. A piece
// that the sequence does not have starts, without rows, at the sequence's end.
struct PieceRows { int32_t t0, rows; bool last; };
constexpr PieceRows piece_rows(int32_t j, int32_t len, int32_t rows) {
    const bool some = j >= 0 && j <= len / rows;
    const int32_t t0 = some ? j * rows : len;
    const int32_t left = len - t0;
    return {t0, left < rows ? left : rows, some && (j == 0 ? len <= rows : left > 0 && left <= rows)};
}

// Workgroups of 256 in one launch at most. Work items along an axis have to stay
// below 2^32, and a larger grid is cut off without an error, so that more of
// them go out as several launches, each with the number of its first workgroup.
// (As rows of a second axis, whose last is too long, every kernel would have to
// look whether its workgroup is one too many: single tokens, 256 rows of 4096
// channels, 30.5 us against 28.8.)
constexpr int64_t kLaunchGroups = int64_t(1) << 23;
// Calls launch(first, count) for them.
template <class F>
constexpr void for_launches(int64_t workgroups, F launch) {
    for (int64_t first = 0; first < workgroups; first += kLaunchGroups)
        launch((uint32_t)first, (uint32_t)(workgroups - first < kLaunchGroups ? workgroups - first : kLaunchGroups));
}

// The byte offset, from row `base` of a tensor on, of place `at` in row t. For
// rows that are not accessed (their offsets go out of range afterwards) it is
// any number, so it is formed modulo 2^32. Host and device.
constexpr uint32_t row_offset(int32_t t, int32_t base, int32_t row_bytes, int32_t at) {
    return ((uint32_t)t - (uint32_t)base) * (uint32_t)row_bytes + (uint32_t)at;
}

struct CconvArgs {
    const void *x, *w, *bias, *init, *dy, *dfinal;
    void *y, *final_state, *dx, *dinit;
    float* part;                // backward: [piece][W + 1][C] partial sums of dw (taps 0..W-1) and dbias (W)
    int64_t sx, sy, sdy, sdx;   // row strides in elements
    Pieces pc;
    int32_t C, W, silu;
    int32_t vec;                // rows are at least a vector long
    int32_t cl;                 // lanes of a workgroup along the channels (a power of two <= 256); 256 / cl runs of rows
    int32_t cblks;              // ceil(C / (cl * channels per lane))
    int32_t run;                // rows a lane walks; rows of a piece = run * 256 / cl
    uint32_t first;             // number of a launch's first workgroup (for_launches)
};

struct CconvReduceArgs {
    const float* part;
    float *dw, *dbias;          // dbias may be NULL
    int32_t pieces, C, W;
};

struct CconvStepArgs {
    const void *x, *w, *bias;
    void *y, *state;
    const int32_t* slots;
    int64_t sx, sy, rows, num_slots;
    int32_t C, W, silu, vec;
    uint32_t first;
};

struct ScanArgs {
    const void *x, *delta, *B, *C, *z, *dy;
    void *y, *dx, *ddelta, *dB, *dC, *dz;
    int64_t sx, sdelta, sB, sC, sz, sy, sdy, sdx, sddelta, sdB, sdC, sdz;
    const float *A, *D, *delta_bias, *init_state, *dfinal_state;
    float *final_state, *dinit_state, *saved;
    float *sums, *sum_d;        // split sequences: [piece][channels][SP] and [piece][channels]
    float *part_bc;             // backward: [channel block][row][2][SP] partial sums of dB and dC
    float *part_a, *part_d;     // backward: [piece][channels][SP] and [piece][2][channels] partial sums of dA and dD, ddelta_bias
    Pieces pc;                  // pieces of segment rows
    int32_t channels, G, Cg, S, softplus;
    int32_t cblks_g;            // channel blocks per group
    int32_t units, units_more;  // units of scan_unit() channels per block; the first units_more blocks have one more
    int32_t vec_c, vec_s;       // vector accesses along the channels (see lane_channel), and of four states of B and C
    int32_t split;              // sequences have more than one segment
    uint32_t first;             // number of a launch's first workgroup (for_launches)
};

struct ScanReduceArgs {
    const float *part_bc, *part_a, *part_d;
    void *dB, *dC;
    float *dA, *dD, *ddelta_bias;   // dD, ddelta_bias may be NULL
    int64_t sdB, sdC;
    int32_t rows, channels, G, S, SP, cblks_g, pieces;
    uint32_t first;
};

struct ScanStepArgs {
    const void *x, *delta, *B, *C, *z;
    void* y;
    const float *A, *D, *delta_bias;
    float* state;
    const int32_t* slots;
    int64_t sx, sdelta, sB, sC, sz, sy, rows, num_slots;
    int32_t channels, Cg, S, softplus, vec;
    uint32_t first;
};

// Rows between two saved states: the backward kernel keeps the decays and
// states of that many rows in registers (2 * 16 * 4 floats per lane).
constexpr int kChunk = 16;

// The lanes that share one channel's states, and the states each holds, for a
// state size S: the smallest pair whose product covers S. The index picks the
// kernel instance.
struct ScanForm { int lanes, per_lane; };
constexpr ScanForm kScanForms[] = {{2, 4}, {4, 4}, {8, 4}, {8, 8}, {16, 8}};

// The adjacent channels that a lane of the scan kernels stages at a time, at most.
constexpr int scan_unit(int lanes) { return lanes < 4 ? 8 : 32 / lanes; }

struct CconvPlan {
    wgrad_cconv_problem prob;
    CconvArgs fwd, bwd;         // launch shapes, pointers unset
    size_t ws_bytes;
};

struct ScanPlan {
    wgrad_scan_problem prob;
    wgrad_scan_plan_info info;
    int form;
    ScanArgs fwd, bwd;          // launch shapes, pointers unset
};

// Channels per lane of the convolution kernels: 16 bytes forward and for
// single tokens; four channels backward, whose lanes also hold a window of
// gradients and the sums of dw.
constexpr int conv_fwd_vec(int dtype) { return dtype == WGRAD_FP32 ? 4 : 8; }
constexpr int kConvBwdVec = 4;

// Launchers; each returns a hipError_t value (0 = success).
int launch_cconv(int dtype, const CconvArgs& a, void* stream);
int launch_cconv_bwd(int dtype, const CconvArgs& a, void* stream);
int launch_cconv_reduce(const CconvReduceArgs& a, void* stream);
int launch_cconv_step(int dtype, const CconvStepArgs& a, void* stream);
int launch_scan_fwd(int dtype, int form, const ScanArgs& a, void* stream);
int launch_scan_bwd(int dtype, int form, const ScanArgs& a, void* stream);
int launch_scan_reduce(int dtype, const ScanReduceArgs& a, void* stream);
int launch_scan_step(int dtype, int form, const ScanStepArgs& a, void* stream);

}  // namespace ssm
}  // namespace wgrad
