// qmm_attend_iq4.hip -- the attention's pass over a cache of iq4_nl keys (qmm_attend.h).
#include "qmm_attend.h"

namespace qmm {

void attend_iq4(const AttendArgs& a, unsigned grid, int rt, hipStream_t st) {
    attend_pair<kKvIq4, kKvIq4>(a, grid, rt, st);
}

}  // namespace qmm
