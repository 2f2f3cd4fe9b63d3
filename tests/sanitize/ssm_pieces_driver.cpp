// The device's arithmetic on seq_start values (packed_rows, piece_rows) over
// valid and invalid ones, up to the largest problems a plan accepts. Built with
// UndefinedBehaviorSanitizer, which ends the program at the first overflow;
// the sums here are 64-bit. Prints the number of combinations looked at.
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
    std::printf("%lld\n", g_seen);
    return 0;
}
