// decay_attn_pack_bwd: the walk that forms dk.
#include "decay_walk.h"

namespace ssmp {

template <>
int launch_decay_walk<kDk>(const DecayArgs& a, int32_t dtype, hipStream_t s) {
    return a.dg ? launch_decay_walk_of<kDk, true>(a, dtype, s) : launch_decay_walk_of<kDk, false>(a, dtype, s);
}

}  // namespace ssmp
