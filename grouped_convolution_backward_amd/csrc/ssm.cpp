// extern "C" entry points declared in include/wgrad_ssm.h, and the plans
// behind them (host only).
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <initializer_list>
#include <new>
#include <string>

#include <hip/hip_runtime.h>

#include "abi_internal.hpp"
#include "ssm_internal.hpp"

struct wgrad_cconv_plan_s {
    wgrad::ssm::CconvPlan plan;
};
struct wgrad_scan_plan_s {
    wgrad::ssm::ScanPlan plan;
};

namespace {

using namespace wgrad::ssm;
using wgrad::set_error;

constexpr int64_t kMaxRows = int64_t(1) << 30;
constexpr int64_t kMaxChannels = int64_t(1) << 23;   // and elements from one row to the next: 32 rows stay below 2 GiB
constexpr int64_t kConvChannels = int64_t(1) << 20;  // the same of a convolution, whose pieces have up to
constexpr int kConvPieceRows = 256;                  // this many rows (and a window on either side)
constexpr int64_t kSegmentRows = 32;                 // a tile of the forward kernel, whole chunks
constexpr int64_t kMaxGrid = (int64_t(1) << 31) - 1;

int invalid(const std::string& msg) { return set_error(WGRAD_ERR_INVALID_ARG, msg); }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t elem_bytes(int dtype) { return dtype == WGRAD_FP32 ? 4 : 2; }

// No exception leaves a C entry point: a host allocation that fails inside
// one (a reason string, a plan) ends as an error code, with the reason if
// there is memory for that.
int out_of_memory() noexcept {
    try {
        return invalid("out of host memory");
    } catch (...) {
        return WGRAD_ERR_INVALID_ARG;
    }
}
template <class F>
int guarded(F f) {
    try {
        wgrad::clear_error();
        return f();
    } catch (...) {
        return out_of_memory();
    }
}

int check_sequences(int packed, int64_t N, int64_t L, int64_t& T) {
    if (packed != 0 && packed != 1) return invalid("packed must be 0 or 1");
    if (N < 0 || L < 0 || T < 0) return invalid("N, L and T must not be negative");
    if (N > kMaxRows || L > kMaxRows || T > kMaxRows) return invalid("N, L and T must be at most 2^30");
    if (!packed) {
        const int64_t rows = N * L;   // at most 2^60
        if (rows > kMaxRows) return invalid("N * L must be at most 2^30");
        if (T != 0 && T != rows) return invalid("T must be 0 or N * L for dense sequences");
        T = rows;
    } else if (N == 0 && T != 0) {
        return invalid("packed rows without a sequence");
    } else if (T > N * L) {
        return invalid("T must be at most N * L: no sequence is longer than L");
    }
    return WGRAD_OK;
}

// Pieces of `rows` rows; rows <= 2^20 or one piece per sequence.
int make_pieces(Pieces& p, int packed, int64_t N, int64_t L, int64_t T, int64_t rows) {
    p.seq_start = nullptr;
    p.N = (int32_t)N, p.L = (int32_t)L, p.T = (int32_t)T, p.rows = (int32_t)rows;
    p.per_seq = (int32_t)(L > 0 ? ceil_div(L, rows) : 1);
    const int64_t count = packed ? (N ? T / rows + N : 0) : N * p.per_seq;
    if (count > kMaxGrid) return invalid("too many sequences for one launch");
    p.count = (int32_t)count;
    return WGRAD_OK;
}

bool aligned(const void* p, int64_t bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

// Whether every access of `bytes` adjacent bytes through these rows is aligned.
bool rows_aligned(std::initializer_list<const wgrad_rows*> list, int64_t elem, int64_t bytes) {
    for (const wgrad_rows* r : list)
        if (r->ptr && (!aligned(r->ptr, bytes) || (r->stride * elem) % bytes)) return false;
    return true;
}
bool all_aligned(std::initializer_list<const void*> list, int64_t bytes) {
    for (const void* p : list)
        if (!aligned(p, bytes)) return false;
    return true;
}

// A required row operand: present, its element alignment, rows that do not overlap.
int check_rows(const char* name, const wgrad_rows& r, int64_t width, int64_t elem, int64_t most = kMaxChannels) {
    if (!r.ptr) return invalid(std::string(name) + " must not be NULL");
    if (!aligned(r.ptr, elem)) return invalid(std::string(name) + " must be aligned to its element type");
    if (r.stride < width) return invalid(std::string(name) + ": row stride smaller than the row");
    if (r.stride > most) return invalid(std::string(name) + ": row stride above " + std::to_string(most) + " elements");
    return WGRAD_OK;
}
int check_ptr(const char* name, const void* p, int64_t elem, bool required) {
    if (!p) return required ? invalid(std::string(name) + " must not be NULL") : (int)WGRAD_OK;
    if (!aligned(p, elem)) return invalid(std::string(name) + " must be aligned to its element type");
    return WGRAD_OK;
}
int check_seq_start(int packed, const int32_t* p) {
    if (packed && !p) return invalid("seq_start must not be NULL for packed sequences");
    if (!packed && p) return invalid("seq_start given for dense sequences");
    return check_ptr("seq_start", p, 4, false);
}
int check_ws(const void* ws, size_t have, size_t need) {
    if (!need) return WGRAD_OK;
    if (!ws) return invalid("workspace is NULL but the plan needs " + std::to_string(need) + " bytes");
    if (have < need)
        return invalid("workspace of " + std::to_string(have) + " bytes is smaller than the " + std::to_string(need) + " needed");
    if (!aligned(ws, 16)) return invalid("workspace must be 16-byte aligned");
    return WGRAD_OK;
}
int check_slots(int64_t rows, int64_t num_slots, const int32_t* slots) {
    if (rows < 0 || num_slots < 0) return invalid("rows and num_slots must not be negative");
    if (rows > kMaxRows) return invalid("rows must be at most 2^30");
    if (!slots && rows > num_slots) return invalid("more rows than states");
    return check_ptr("slots", slots, 4, false);
}
int launched(int e, const char* what) {
    if (e == hipSuccess) return WGRAD_OK;
    return set_error(WGRAD_ERR_HIP, std::string(what) + " kernel launch: " + hipGetErrorString((hipError_t)e));
}

#define CHECK(expr)                \
    do {                           \
        const int rc_ = (expr);    \
        if (rc_) return rc_;       \
    } while (0)

// Lanes along the channels, rows per lane and pieces of a convolution launch.
int conv_shape(CconvArgs& a, const wgrad_cconv_problem& p, int64_t T, int vec, int64_t lanes_wanted, int run_most) {
    const int64_t cv = ceil_div(p.C, vec);
    int cl = 1;
    while (cl < cv && cl < 64) cl *= 2;
    a.cl = cl;
    a.cblks = (int32_t)ceil_div(cv, cl);
    a.C = (int32_t)p.C, a.W = p.W, a.silu = p.activation == WGRAD_ACT_SILU;
    // Long runs re-read fewer rows between runs and leave fewer partial sums;
    // short ones fill the card when there are few rows. Runs of 4 | 16 | 32 rows,
    // bf16, W = 4, us in a graph: forward 1 x 512 x 1024 4.1 | 6.9 | 10.5, 4 x 2048
    // x 4096 28.3 | 23.9 | 23.7; backward 1 x 512 x 1024 11.8 | 15.3 | 20.5, 1 x
    // 2048 x 4096 34.9 | 22.0 | 23.0, 4 x 2048 x 4096 104 | 54.8 | 47.5.
    int run = 4;
    while (run < run_most && T * cv / (2 * run) >= lanes_wanted) run *= 2;
    while (run * (256 / cl) > kConvPieceRows) run /= 2;
    a.run = run;
    CHECK(make_pieces(a.pc, p.packed, p.N, p.L, T, (int64_t)run * (256 / cl)));
    if ((int64_t)a.pc.count * a.cblks > kMaxGrid) return invalid("problem too large for one launch");
    return WGRAD_OK;
}

int build_cconv(const wgrad_cconv_problem& p, CconvPlan& out) {
    if (p.dtype != WGRAD_BF16 && p.dtype != WGRAD_FP16 && p.dtype != WGRAD_FP32) return invalid("dtype must be BF16, FP16 or FP32");
    if (p.activation != WGRAD_ACT_NONE && p.activation != WGRAD_ACT_SILU) return invalid("activation must be NONE or SILU");
    if (p.W < 1 || p.W > 8) return invalid("W must be 1 to 8");
    if (p.C < 1 || p.C > kConvChannels) return invalid("C must be 1 to 2^20");
    int64_t T = p.T;
    CHECK(check_sequences(p.packed, p.N, p.L, T));
    out.prob = p;
    out.prob.T = T;
    out.fwd = CconvArgs{};
    out.bwd = CconvArgs{};
    // lanes that longer runs have to leave: four waves per SIMD forward, three
    // per CU backward, where a run re-reads more and leaves partial sums
    CHECK(conv_shape(out.fwd, p, T, conv_fwd_vec(p.dtype), 1 << 18, 16));
    CHECK(conv_shape(out.bwd, p, T, kConvBwdVec, 3 << 14, 32));
    out.ws_bytes = (size_t)out.bwd.pc.count * (size_t)(p.W + 1) * (size_t)p.C * 4;
    return WGRAD_OK;
}

// Rows of the segments that sequences are cut into: all of L (no split) where
// whole sequences make enough workgroups of four waves, `enough`. A split
// computes the decays once more (forward; backward about a quarter more work)
// and wins it back by filling the card: eight workgroups a CU in all, in steps
// of kSegmentRows. Measured (bf16, 16 states, us whole -> split, forward with
// saved states and backward): 64 workgroups of 2048 rows 225 -> 74, 578 -> 154;
// 256 of 2048 rows 227 -> 219, 593 -> 510; 384 of 1024 rows 162 -> 178, 423 ->
// 414; 512 of 2048 rows 319 -> 411, 856 -> 975.
// A segment also folds the sums of all segments before it, one after another,
// so no more than about sqrt(L) segments pay: 1 x 16384 rows of 128 channels
// take 50 + 81 us in 128 segments, 97 + 136 in 512; 1 x 65536 rows 106 + 184 in
// 256, 296 + 442 in 1024.
int64_t choose_segment_rows(int64_t T, int64_t L, int64_t nblk, int64_t cus, int64_t enough) {
    if (L == 0 || ceil_div(T, L) * nblk >= enough) return L;   // T / L: packed sequences may be mostly short
    const int64_t least = std::max(ceil_div(T * nblk, 8 * cus), (int64_t)std::sqrt((double)L));
    const int64_t rows = ceil_div(least, kSegmentRows) * kSegmentRows;
    return rows < L ? rows : L;
}

int build_scan(const wgrad_scan_problem& p, const wgrad_scan_overrides* ov, const wgrad::DeviceModel& dev, ScanPlan& out) {
    if (p.dtype != WGRAD_BF16 && p.dtype != WGRAD_FP16 && p.dtype != WGRAD_FP32) return invalid("dtype must be BF16, FP16 or FP32");
    if (p.softplus != 0 && p.softplus != 1) return invalid("softplus must be 0 or 1");
    if (p.reserved != 0) return invalid("reserved must be 0");
    if (p.C < 1 || p.C > kMaxChannels) return invalid("C must be 1 to 2^23");
    if (p.G < 1 || p.G > p.C || p.C % p.G) return invalid("C must be a multiple of G");
    if (p.G * 128 > kMaxChannels) return invalid("G must be at most 2^16");
    if (p.S < 1 || p.S > 128) return invalid("S must be 1 to 128");
    if (ov && (ov->segments < 0 || ov->segments_backward < 0)) return invalid("segment overrides must not be negative");
    int64_t T = p.T;
    CHECK(check_sequences(p.packed, p.N, p.L, T));
    out.prob = p;
    out.prob.T = T;
    out.form = 0;
    while (kScanForms[out.form].lanes * kScanForms[out.form].per_lane < p.S) ++out.form;
    const ScanForm f = kScanForms[out.form];
    const int64_t SP = f.lanes * f.per_lane, CT = 256 / f.lanes, Cg = p.C / p.G;
    const int64_t cblks_g = ceil_div(Cg, CT), nblk = cblks_g * p.G;
    wgrad_scan_plan_info& info = out.info;
    info = wgrad_scan_plan_info{};
    info.lanes = f.lanes;
    info.states_per_lane = f.per_lane;
    info.chunk_rows = kChunk;

    for (int dir = 0; dir < 2; ++dir) {
        ScanArgs& a = dir ? out.bwd : out.fwd;
        a = ScanArgs{};
        a.channels = (int32_t)p.C, a.G = (int32_t)p.G, a.Cg = (int32_t)Cg, a.S = (int32_t)p.S;
        a.softplus = p.softplus, a.cblks_g = (int32_t)cblks_g;
        // Blocks of whole units, dealt evenly: of two or more blocks each has at least half of CT / E units.
        const int64_t E = scan_unit(f.lanes), units = ceil_div(Cg, E);
        a.units = (int32_t)(units / cblks_g), a.units_more = (int32_t)(units % cblks_g);
        a.vec_c = Cg % E == 0 ? 2 : Cg >= E;     // see lane_channel
        a.vec_s = p.S % 4 == 0;
        const int64_t seg = ov ? (dir ? ov->segments_backward : ov->segments) : 0;
        int64_t rows = seg ? ceil_div(ceil_div(p.L, seg), kSegmentRows) * kSegmentRows
                           : choose_segment_rows(T, p.L, nblk, dev.num_cus, dev.num_cus * (dir ? 7 : 5) / 4);
        if (rows < 1 || rows > p.L) rows = p.L;
        a.split = rows < p.L;
        CHECK(make_pieces(a.pc, p.packed, p.N, p.L, T, rows < 1 ? 1 : rows));
        if ((int64_t)a.pc.count * nblk > kMaxGrid) return invalid("problem too large for one launch");
        (dir ? info.segments_backward : info.segments) = a.pc.per_seq;
        (dir ? info.segment_rows_backward : info.segment_rows) = rows;
    }
    const int64_t chunks = p.packed ? (p.N ? T / kChunk + p.N : 0) : p.N * ceil_div(p.L, kChunk);
    info.saved_bytes = chunks * p.C * SP * 4;
    const int64_t sums = p.C * (SP + 1) * 4;
    if (ceil_div(T * p.G * 2 * SP + p.C * (SP + 2), 256) > kMaxGrid) return invalid("problem too large for one launch");
    // every part starts on 16 bytes: the quads (sums, part_bc, part_a) come first
    info.workspace_bytes = out.fwd.split ? (int64_t)out.fwd.pc.count * sums : 0;
    info.workspace_bytes_backward = nblk * T * 2 * SP * 4 + (int64_t)out.bwd.pc.count * (p.C * SP * 4 + 2 * p.C * 4) +
                                    (out.bwd.split ? (int64_t)out.bwd.pc.count * sums : 0);
    return WGRAD_OK;
}

// The checks forward and backward share.
int check_scan(const ScanPlan& P, const wgrad_scan_args& v) {
    const wgrad_scan_problem& p = P.prob;
    const int64_t e = elem_bytes(p.dtype);
    CHECK(check_seq_start(p.packed, v.seq_start));
    CHECK(check_ptr("A", v.A, 4, true));
    CHECK(check_ptr("D", v.D, 4, false));
    CHECK(check_ptr("delta_bias", v.delta_bias, 4, false));
    if (p.T == 0) return WGRAD_OK;
    CHECK(check_rows("x", v.x, p.C, e));
    CHECK(check_rows("delta", v.delta, p.C, e));
    CHECK(check_rows("B", v.B, p.G * p.S, e));
    CHECK(check_rows("C", v.C, p.G * p.S, e));
    if (v.z.ptr) CHECK(check_rows("z", v.z, p.C, e));
    return WGRAD_OK;
}

void fill_scan(ScanArgs& a, const wgrad_scan_args& v) {
    a.x = v.x.ptr, a.sx = v.x.stride;
    a.delta = v.delta.ptr, a.sdelta = v.delta.stride;
    a.B = v.B.ptr, a.sB = v.B.stride;
    a.C = v.C.ptr, a.sC = v.C.stride;
    a.z = v.z.ptr, a.sz = v.z.stride;
    a.A = v.A, a.D = v.D, a.delta_bias = v.delta_bias;
    a.pc.seq_start = v.seq_start;
}

}  // namespace

extern "C" {

int wgrad_cconv_plan(const wgrad_cconv_problem* problem, int hip_device, wgrad_cconv_plan_t** out) {
    return guarded([&]() -> int {
        if (!problem || !out) return invalid("problem and out must not be NULL");
        *out = nullptr;
        wgrad::DeviceModel dev{256, 8};
        CHECK(wgrad::device_model(hip_device, dev));
        CconvPlan plan;
        CHECK(build_cconv(*problem, plan));
        *out = new wgrad_cconv_plan_s{plan};
        return WGRAD_OK;
    });
}

void wgrad_cconv_plan_destroy(wgrad_cconv_plan_t* plan) { delete plan; }

size_t wgrad_cconv_workspace_bytes(const wgrad_cconv_plan_t* plan) { return plan ? plan->plan.ws_bytes : 0; }

int wgrad_cconv_run(const wgrad_cconv_plan_t* plan, const wgrad_cconv_args* args, void* stream) {
    return guarded([&]() -> int {
        if (!plan || !args) return invalid("plan and args must not be NULL");
        const CconvPlan& P = plan->plan;
        const wgrad_cconv_problem& p = P.prob;
        const wgrad_cconv_args& v = *args;
        const int64_t e = elem_bytes(p.dtype);
        CHECK(check_seq_start(p.packed, v.seq_start));
        CHECK(check_ptr("w", v.w, e, true));
        CHECK(check_ptr("bias", v.bias, e, false));
        CHECK(check_ptr("init_state", v.init_state, e, false));
        CHECK(check_ptr("final_state", v.final_state, e, false));
        if (p.T) {
            CHECK(check_rows("x", v.x, p.C, e, kConvChannels));
            CHECK(check_rows("y", v.y, p.C, e, kConvChannels));
        }
        CconvArgs a = P.fwd;
        if (a.pc.count == 0) return WGRAD_OK;
        a.x = v.x.ptr, a.sx = v.x.stride, a.y = v.y.ptr, a.sy = v.y.stride;
        a.w = v.w, a.bias = v.bias, a.init = v.init_state, a.final_state = p.W > 1 ? v.final_state : nullptr;
        a.pc.seq_start = v.seq_start;
        a.vec = p.C >= conv_fwd_vec(p.dtype);
        return launched(launch_cconv(p.dtype, a, stream), "causal convolution");
    });
}

int wgrad_cconv_backward_run(const wgrad_cconv_plan_t* plan, const wgrad_cconv_args* args, void* stream) {
    return guarded([&]() -> int {
        if (!plan || !args) return invalid("plan and args must not be NULL");
        const CconvPlan& P = plan->plan;
        const wgrad_cconv_problem& p = P.prob;
        const wgrad_cconv_args& v = *args;
        const int64_t e = elem_bytes(p.dtype);
        CHECK(check_seq_start(p.packed, v.seq_start));
        CHECK(check_ptr("w", v.w, e, true));
        CHECK(check_ptr("dw", v.dw, 4, true));
        CHECK(check_ptr("dbias", v.dbias, 4, false));
        CHECK(check_ptr("bias", v.bias, e, false));
        CHECK(check_ptr("init_state", v.init_state, e, false));
        CHECK(check_ptr("dfinal_state", v.dfinal_state, e, false));
        CHECK(check_ptr("dinit_state", v.dinit_state, e, false));
        if (p.T) {
            CHECK(check_rows("x", v.x, p.C, e, kConvChannels));
            CHECK(check_rows("dy", v.dy, p.C, e, kConvChannels));
            CHECK(check_rows("dx", v.dx, p.C, e, kConvChannels));
        }
        CHECK(check_ws(v.ws, v.ws_bytes, P.ws_bytes));
        CconvArgs a = P.bwd;
        a.x = v.x.ptr, a.sx = v.x.stride, a.dy = v.dy.ptr, a.sdy = v.dy.stride, a.dx = v.dx.ptr, a.sdx = v.dx.stride;
        a.w = v.w, a.bias = v.bias, a.init = v.init_state, a.dfinal = v.dfinal_state, a.dinit = v.dinit_state;
        a.pc.seq_start = v.seq_start;
        a.part = static_cast<float*>(v.ws);
        a.vec = p.C >= kConvBwdVec;
        if (a.pc.count) CHECK(launched(launch_cconv_bwd(p.dtype, a, stream), "causal convolution backward"));
        const CconvReduceArgs r{a.part, v.dw, v.dbias, a.pc.count, a.C, a.W};
        return launched(launch_cconv_reduce(r, stream), "causal convolution reduce");
    });
}

int wgrad_cconv_step_run(const wgrad_cconv_plan_t* plan, const wgrad_cconv_args* args, void* stream) {
    return guarded([&]() -> int {
        if (!plan || !args) return invalid("plan and args must not be NULL");
        const wgrad_cconv_problem& p = plan->plan.prob;
        const wgrad_cconv_args& v = *args;
        const int64_t e = elem_bytes(p.dtype);
        CHECK(check_slots(v.rows, v.num_slots, v.slots));
        if (v.rows == 0) return WGRAD_OK;
        CHECK(check_rows("x", v.x, p.C, e, kConvChannels));
        CHECK(check_rows("y", v.y, p.C, e, kConvChannels));
        CHECK(check_ptr("w", v.w, e, true));
        CHECK(check_ptr("bias", v.bias, e, false));
        CHECK(check_ptr("state", v.state, e, p.W > 1 && v.num_slots > 0));
        if (ceil_div(v.rows * ceil_div(p.C, conv_fwd_vec(p.dtype)), 256) > kMaxGrid) return invalid("too many rows for one launch");
        CconvStepArgs a{};
        a.x = v.x.ptr, a.sx = v.x.stride, a.y = v.y.ptr, a.sy = v.y.stride;
        a.w = v.w, a.bias = v.bias, a.state = v.state, a.slots = v.slots;
        a.rows = v.rows, a.num_slots = v.num_slots;
        a.C = (int32_t)p.C, a.W = p.W, a.silu = p.activation == WGRAD_ACT_SILU;
        a.vec = p.C % conv_fwd_vec(p.dtype) == 0 && rows_aligned({&v.x, &v.y}, e, 16) && all_aligned({v.w, v.bias, v.state}, 16);
        return launched(launch_cconv_step(p.dtype, a, stream), "causal convolution step");
    });
}

int wgrad_scan_plan(const wgrad_scan_problem* problem, const wgrad_scan_overrides* overrides, int hip_device,
                    wgrad_scan_plan_t** out) {
    return guarded([&]() -> int {
        if (!problem || !out) return invalid("problem and out must not be NULL");
        *out = nullptr;
        wgrad::DeviceModel dev{256, 8};
        CHECK(wgrad::device_model(hip_device, dev));
        ScanPlan plan;
        CHECK(build_scan(*problem, overrides, dev, plan));
        *out = new wgrad_scan_plan_s{plan};
        return WGRAD_OK;
    });
}

void wgrad_scan_plan_destroy(wgrad_scan_plan_t* plan) { delete plan; }

int wgrad_scan_plan_query(const wgrad_scan_plan_t* plan, wgrad_scan_plan_info* info) {
    return guarded([&]() -> int {
        if (!plan || !info) return invalid("plan and info must not be NULL");
        *info = plan->plan.info;
        return WGRAD_OK;
    });
}

size_t wgrad_scan_workspace_bytes(const wgrad_scan_plan_t* plan, int backward) {
    if (!plan) return 0;
    return (size_t)(backward ? plan->plan.info.workspace_bytes_backward : plan->plan.info.workspace_bytes);
}

size_t wgrad_scan_saved_bytes(const wgrad_scan_plan_t* plan) { return plan ? (size_t)plan->plan.info.saved_bytes : 0; }

int wgrad_scan_run(const wgrad_scan_plan_t* plan, const wgrad_scan_args* args, void* stream) {
    return guarded([&]() -> int {
        if (!plan || !args) return invalid("plan and args must not be NULL");
        const ScanPlan& P = plan->plan;
        const wgrad_scan_problem& p = P.prob;
        const wgrad_scan_args& v = *args;
        const int64_t e = elem_bytes(p.dtype);
        CHECK(check_scan(P, v));
        CHECK(check_ptr("init_state", v.init_state, 4, false));
        CHECK(check_ptr("final_state", v.final_state, 4, false));
        CHECK(check_ptr("saved", v.saved, 16, false));
        if (p.T) CHECK(check_rows("y", v.y, p.C, e));
        CHECK(check_ws(v.ws, v.ws_bytes, (size_t)P.info.workspace_bytes));
        ScanArgs a = P.fwd;
        if (a.pc.count == 0) return WGRAD_OK;
        fill_scan(a, v);
        a.y = v.y.ptr, a.sy = v.y.stride;
        a.init_state = v.init_state, a.final_state = v.final_state, a.saved = static_cast<float*>(v.saved);
        if (a.split) {
            a.sums = static_cast<float*>(v.ws);
            a.sum_d = a.sums + (int64_t)a.pc.count * p.C * (P.info.lanes * P.info.states_per_lane);
        }
        return launched(launch_scan_fwd(p.dtype, P.form, a, stream), "scan");
    });
}

int wgrad_scan_backward_run(const wgrad_scan_plan_t* plan, const wgrad_scan_args* args, void* stream) {
    return guarded([&]() -> int {
        if (!plan || !args) return invalid("plan and args must not be NULL");
        const ScanPlan& P = plan->plan;
        const wgrad_scan_problem& p = P.prob;
        const wgrad_scan_args& v = *args;
        const int64_t e = elem_bytes(p.dtype);
        CHECK(check_scan(P, v));
        CHECK(check_ptr("dA", v.dA, 4, true));
        CHECK(check_ptr("dD", v.dD, 4, false));
        CHECK(check_ptr("ddelta_bias", v.ddelta_bias, 4, false));
        CHECK(check_ptr("dfinal_state", v.dfinal_state, 4, false));
        CHECK(check_ptr("dinit_state", v.dinit_state, 4, false));
        if (p.T) {
            CHECK(check_ptr("saved", v.saved, 16, true));
            CHECK(check_rows("dy", v.dy, p.C, e));
            CHECK(check_rows("dx", v.dx, p.C, e));
            CHECK(check_rows("ddelta", v.ddelta, p.C, e));
            CHECK(check_rows("dB", v.dB, p.G * p.S, e));
            CHECK(check_rows("dC", v.dC, p.G * p.S, e));
            if (v.z.ptr) CHECK(check_rows("dz", v.dz, p.C, e));
        }
        CHECK(check_ws(v.ws, v.ws_bytes, (size_t)P.info.workspace_bytes_backward));
        ScanArgs a = P.bwd;
        fill_scan(a, v);
        a.dy = v.dy.ptr, a.sdy = v.dy.stride, a.dx = v.dx.ptr, a.sdx = v.dx.stride;
        a.ddelta = v.ddelta.ptr, a.sddelta = v.ddelta.stride, a.dz = v.dz.ptr, a.sdz = v.dz.stride;
        a.dfinal_state = v.dfinal_state, a.dinit_state = v.dinit_state, a.saved = static_cast<float*>(v.saved);
        const int64_t SP = (int64_t)P.info.lanes * P.info.states_per_lane, n = a.pc.count;
        a.part_bc = static_cast<float*>(v.ws);
        a.part_a = a.part_bc + (int64_t)a.cblks_g * a.G * p.T * 2 * SP;
        a.sums = a.part_a + n * p.C * SP;
        a.part_d = a.sums + (a.split ? n * p.C * SP : 0);
        a.sum_d = a.part_d + n * 2 * p.C;
        if (n) CHECK(launched(launch_scan_bwd(p.dtype, P.form, a, stream), "scan backward"));
        ScanReduceArgs r{};
        r.part_bc = a.part_bc, r.part_a = a.part_a, r.part_d = a.part_d;
        r.dB = v.dB.ptr, r.sdB = v.dB.stride, r.dC = v.dC.ptr, r.sdC = v.dC.stride;
        r.dA = v.dA, r.dD = v.dD, r.ddelta_bias = v.ddelta_bias;
        r.rows = (int32_t)p.T, r.channels = a.channels, r.G = a.G, r.S = a.S, r.SP = (int32_t)SP;
        r.cblks_g = a.cblks_g, r.pieces = a.pc.count;
        return launched(launch_scan_reduce(p.dtype, r, stream), "scan reduce");
    });
}

int wgrad_scan_step_run(const wgrad_scan_plan_t* plan, const wgrad_scan_args* args, void* stream) {
    return guarded([&]() -> int {
        if (!plan || !args) return invalid("plan and args must not be NULL");
        const ScanPlan& P = plan->plan;
        const wgrad_scan_problem& p = P.prob;
        const wgrad_scan_args& v = *args;
        const int64_t e = elem_bytes(p.dtype);
        CHECK(check_slots(v.rows, v.num_slots, v.slots));
        if (v.rows == 0) return WGRAD_OK;
        CHECK(check_ptr("A", v.A, 4, true));
        CHECK(check_ptr("D", v.D, 4, false));
        CHECK(check_ptr("delta_bias", v.delta_bias, 4, false));
        CHECK(check_rows("x", v.x, p.C, e));
        CHECK(check_rows("delta", v.delta, p.C, e));
        CHECK(check_rows("B", v.B, p.G * p.S, e));
        CHECK(check_rows("C", v.C, p.G * p.S, e));
        CHECK(check_rows("y", v.y, p.C, e));
        if (v.z.ptr) CHECK(check_rows("z", v.z, p.C, e));
        CHECK(check_ptr("state", v.state, 4, v.num_slots > 0));
        if (v.rows * ceil_div(p.C, 256 / P.info.lanes) > kMaxGrid) return invalid("too many rows for one launch");
        ScanStepArgs a{};
        a.x = v.x.ptr, a.sx = v.x.stride, a.delta = v.delta.ptr, a.sdelta = v.delta.stride;
        a.B = v.B.ptr, a.sB = v.B.stride, a.C = v.C.ptr, a.sC = v.C.stride;
        a.z = v.z.ptr, a.sz = v.z.stride, a.y = v.y.ptr, a.sy = v.y.stride;
        a.A = v.A, a.D = v.D, a.delta_bias = v.delta_bias, a.state = v.state, a.slots = v.slots;
        a.rows = v.rows, a.num_slots = v.num_slots;
        a.channels = (int32_t)p.C, a.Cg = (int32_t)(p.C / p.G), a.S = (int32_t)p.S, a.softplus = p.softplus;
        // a lane's 4 or 8 states: whole, and aligned to 16 bytes
        a.vec = p.S % P.info.states_per_lane == 0 && all_aligned({v.state, v.A}, 16) && rows_aligned({&v.B, &v.C}, e, 16);
        return launched(launch_scan_step(p.dtype, P.form, a, stream), "scan step");
    });
}

}  // extern "C"
