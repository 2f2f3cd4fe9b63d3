// The device's arithmetic on seq_start values (packed_rows, piece_rows) over
// valid and invalid ones, up to the largest problems a plan accepts. Built with
// UndefinedBehaviorSanitizer, which ends the program at the first overflow;
// the sums here are 64-bit. Likewise the offsets of rows in a piece of the
// convolution (row_offset), which its kernels also form for rows far outside
// it, and the launches of large grids (for_launches). Prints the number of combinations looked at.
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <initializer_list>

#include "../../grouped_convolution_backward_amd/csrc/ssm_internal.hpp"

using namespace wgrad::ssm;

namespace {
long long g_seen = 0;

void expect(bool ok, const char* what, int32_t from, int32_t to, int32_t T, int32_t L, int32_t rows, int32_t j) {
    ++g_seen;
    if (ok) return;
    std::printf("%s: seq_start %d, %d of T %d, L %d; rows %d, piece %d\n", what, from, to, T, L, rows, j);
    std::exit(1);
}
}  // namespace

int main() {
    constexpr int32_t big = 1 << 30;
    for (int32_t T : {0, 1, 31, 4096, big - 1, big})
        for (int32_t L : {0, 1, 31, 4096, big - 1, big})
            for (int32_t from : {INT32_MIN, INT32_MIN + 1, -big, -1, 0, 1, 30, T - 1, T, T + 1, big - 1, big, big + 1, INT32_MAX})
                for (int32_t to : {INT32_MIN, -1, 0, 1, 30, 31, T - 1, T, T + 1, big - 1, big, big + 1, INT32_MAX}) {
                    const SeqRows q = packed_rows(from, to, T, L);
                    const int64_t end = (int64_t)q.row0 + q.len;
                    expect(q.row0 >= 0 && q.len >= 0 && q.len <= L && end <= T, "rows out of range", from, to, T, L, 0, 0);
                    if (from >= 0 && from <= to && to <= T && (int64_t)to - from <= L)
                        expect(q.row0 == from && end == to, "a valid sequence changed", from, to, T, L, 0, 0);
                    for (int32_t rows : {1, 32, 96, 256, big}) {
                        for (int32_t j : {INT32_MIN, -1, 0, 1, 2, q.len / rows - 1, q.len / rows, q.len / rows + 1, big, INT32_MAX}) {
                            const PieceRows p = piece_rows(j, q.len, rows);
                            const int64_t n = p.rows > 0 ? p.rows : 0;
                            expect(p.t0 >= 0 && p.t0 + n <= q.len && n <= rows, "piece out of its sequence", from, to, T, L, rows, j);
                            const int64_t whole = q.len > 0 ? ((int64_t)q.len - 1) / rows : 0;   // the last piece
                            expect(p.last == (j == whole), "another last piece", from, to, T, L, rows, j);
                            const int64_t at = (int64_t)j * rows, have = q.len - at < rows ? q.len - at : rows;
                            expect(n == (j >= 0 && have > 0 ? have : 0), "another number of rows", from, to, T, L, rows, j);
                        }
                    }
                }
    for (int32_t row_bytes : {2, 4, 1 << 12, 1 << 21, 1 << 22})      // strides up to 2^20 elements of 4 bytes
        for (int32_t base : {-7, 0, 5, big - 300, big - 1})
            for (int64_t d : {-7, -1, 0, 1, 255, 263, 300, big - 300, big}) {
                const int32_t t = (int32_t)(base + d < big + 300 ? base + d : big);
                const uint32_t got = row_offset(t, base, row_bytes, 40);
                const int64_t want = ((int64_t)t - base) * row_bytes + 40;
                expect(got == (uint32_t)want, "another offset", t, base, row_bytes, 40, 0, 0);
                if (d >= 0 && d <= 263) expect((int64_t)got == want && want < (1LL << 31), "offset of a near row", t, base, row_bytes, 40, 0, 0);
            }
    constexpr int64_t most = (1LL << 31) - 1;                        // workgroups that a plan accepts
    for (int64_t n : std::initializer_list<int64_t>{0, 1, 255, kLaunchGroups - 1, kLaunchGroups, kLaunchGroups + 1, (1 << 24) - 1, 1 << 24,
                                                    (1 << 24) + 3, big + 1, most}) {
        int64_t next = 0;                                             // each workgroup once, in order
        for_launches(n, [&](uint32_t first, uint32_t count) {
            expect((int64_t)first == next && count > 0 && (int64_t)count * 256 < (1LL << 32), "launch", (int32_t)n, 0, 0, 0, 0, 0);
            next += count;
        });
        expect(next == n, "launches", (int32_t)n, 0, 0, 0, 0, 0);
    }
    std::printf("%lld\n", g_seen);
    return 0;
}
