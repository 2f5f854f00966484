// qmm_attend_q8.hip -- the attention's pass over a cache of q8_0 keys (qmm_attend.h).
#include "qmm_attend.h"

namespace qmm {

void attend_q8(const AttendArgs& a, unsigned grid, int rt, hipStream_t st) {
    if (a.v.type == kKvQ8) return attend_pair<kKvQ8, kKvQ8>(a, grid, rt, st);
    attend_pair<kKvQ8, kKvIq4>(a, grid, rt, st);
}

}  // namespace qmm
