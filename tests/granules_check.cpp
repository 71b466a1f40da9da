// Host-side brute-force check of granules.h (compiled and run by test_granules.py with the
// system C++ compiler): the reads of every row of narrow and odd matrices, at every base
// that their elements allow, as the row kernels make them.
#include <cstdio>

#include "granules.h"

int main() {
    for (int elem = 2; elem <= 4; elem += 2)
        for (uint64_t base = 1 << 20; base < (1 << 20) + 16; base += elem)
            for (int cols = 1; cols <= 40; ++cols)
                for (int ld = cols; ld <= cols + 9; ++ld)
                    for (int rows = 1; rows <= 20; ++rows)
                        for (int row = 0; row < rows; ++row) {
                            const uint64_t at = base + static_cast<uint64_t>(row) * ld * elem;
                            const uint64_t last = base + (static_cast<uint64_t>(rows - 1) * ld + cols) * elem;
                            const tg::Granules g = tg::granules(base, at - base, cols * elem);
                            const uint64_t first = at - g.skip;  // the granules, and what is read of them
                            bool ok = first % 16 == 0 && g.skip >= 0 && g.skip < 16 &&
                                      first + g.end == at + cols * elem && first + g.end <= last;
                            ok = ok && (g.outside ? g.skip > 0 : first >= base);
                            if (!ok) {
                                std::printf("FAIL elem %d base %d cols %d ld %d row %d: from %lld, outside %d\n", elem,
                                            static_cast<int>(base % 16), cols, ld, row,
                                            static_cast<long long>(first) - static_cast<long long>(base),
                                            static_cast<int>(g.outside));
                                return 1;
                            }
                        }
    std::printf("OK\n");
    return 0;
}
