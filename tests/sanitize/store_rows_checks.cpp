// store_rows_checks.cpp -- where the chunked pass of linear attention stores: the byte offsets of
// every lane and output at the narrowest and widest rows that the entry points allow, on the CPU.
// Test infrastructure only.  Exits 0 when every check holds.
#include <stdio.h>

#include "linattn.h"

int main() {
    long checks = 0, failed = 0;
    const int C = 64;
    // bytes of a row of all heads: bf16 and float32 outputs, and the gradients' float32 rows per head
    const int64_t rows[] = {2, 4, 256, 1 << 20, (1 << 24) - 4, int64_t(18300) * 256 * 4, int64_t(20000) * 248 * 4,
                            int64_t(32767) * 200 * 4, int64_t(32767) * 255 * 4, int64_t(32767) * 256 * 4};
    for (int64_t pitch : rows)
        for (int tokens : {1, 33, 64})
            for (int rev = 0; rev < 2; ++rev)
                for (int g4 = 0; g4 < 4; ++g4) {
                    const int64_t window = tokens * pitch;
                    const la::StoreRows to(pitch, rev, C, g4);
                    for (int it = 0; it < C / 16; ++it)
                        for (int r = 0; r < 4; ++r) {
                            const int row = 16 * it + 4 * g4 + r, token = rev ? C - 1 - row : row;
                            for (int at : {0, 2, int(pitch < 1024 ? pitch - 2 : 1020)}) {
                                const uint32_t on = to.first(true, at) + to.row(16 * it + r);
                                const uint32_t off = to.first(false, at) + to.row(16 * it + r);
                                ++checks;
                                // a column of the head: its own place, in the window as far as the tokens go
                                if (int64_t(on) != token * pitch + at) ++failed;
                                if (token >= tokens && int64_t(on) < window) ++failed;
                                // no column of the head: dropped, whichever the row
                                if (int64_t(off) < window) ++failed;
                            }
                        }
                }
    printf("%ld checks, %ld failed\n", checks, failed);
    return failed ? 1 : 0;
}
