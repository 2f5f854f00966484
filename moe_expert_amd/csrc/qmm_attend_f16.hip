// qmm_attend_f16.hip -- the attention's pass over a cache of binary16 keys (qmm_attend.h).
#include "qmm_attend.h"

namespace qmm {

void attend_f16(const AttendArgs& a, unsigned grid, int rt, hipStream_t st) {
    if (a.v.type == kKvF16) return attend_pair<kKvF16, kKvF16>(a, grid, rt, st);
    if (a.v.type == kKvQ8) return attend_pair<kKvF16, kKvQ8>(a, grid, rt, st);
    attend_pair<kKvF16, kKvIq4>(a, grid, rt, st);
}

}  // namespace qmm
