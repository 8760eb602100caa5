// How many threads take a row of spec_residual_norm and spec_quantize_rows. Plain C++.
#pragma once
#include <algorithm>

namespace specs {

struct NormThreads {
    int slots;       // pieces of a thread
    int tpr, per;    // threads of a row, rows of a CTA
    long long room;  // threads of an SM, by registers
};

// `pieces` of a row, of 16 bytes (vec) or one value each; at most 512 x 4 and 512 x 16 of them. full: with a residual, a weight or a norm.
// Many rows: threads with four pieces, so that much is on its way. Few: halved as long as every row still has its place at once, and
// room for a warp more; to two pieces with codes, whose work is the most, without that room too. In us on 152 SMs, with and without room
// for a warp more (bf16): the norm to codes of 1500 rows of 512 3.7 and 3.3, 1216 of 1024 4.0 and 3.4, 608 of 2048 4.3 and 3.4; codes
// as they are, 2432 rows of 1024 5.1 and 3.8, 608 of 4096 5.0 and 4.0. To one piece it would be 1216 of 512 2.8 and 3.0, 500 of 1024 3.0
// and 3.2, 304 of 2048 3.0 and 3.1, and to two for 16-bit outputs 1000 of 1024 2.8 and 3.1, 500 of 2048 2.9 and 3.1.
inline NormThreads norm_threads(long long rows, int pieces, bool vec, bool codes, bool full, int sms) {
    NormThreads t = {vec ? 4 : 16, 0, 0, full ? 512 : 1024};
    auto fits = [&](int slots) {
        const int x = (pieces + slots - 1) / slots;
        return rows * (vec && codes && slots == 2 ? (x + 31) / 32 * 32 : x + 31) <= t.room * sms;
    };
    while (t.slots > 1 && 2 * pieces <= 512 * t.slots && fits(t.slots / 2)) t.slots /= 2;
    if (!vec && t.slots < 16) t.slots = t.slots < 4 ? 4 : t.slots == 8 ? 16 : t.slots;      // there are kernels of 4 and of 16
    t.tpr = ((pieces + t.slots - 1) / t.slots + 31) / 32 * 32;
    t.per = std::max(1, (rows > 4LL * sms ? 128 : 32) / t.tpr);
    return t;
}

}  // namespace specs
