// decay_attn_pack_bwd: the walk that forms dq.
#include "decay_walk.h"

namespace ssmp {

int launch_decay_dq(const DecayArgs& a, int32_t dtype, hipStream_t s) {
    return a.dg ? launch_decay_walk<kDq, true>(a, dtype, s) : launch_decay_walk<kDq, false>(a, dtype, s);
}

}  // namespace ssmp
