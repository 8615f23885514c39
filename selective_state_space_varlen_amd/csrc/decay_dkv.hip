// decay_attn_pack_bwd: the walks that form dk and dv.
#include "decay_walk.h"

namespace ssmp {

int launch_decay_dkv(const DecayArgs& a, int32_t dtype, hipStream_t s) {
    return a.dg ? launch_decay_pair<kDk, true, kDv>(a, dtype, s) : launch_decay_pair<kDk, false, kDv>(a, dtype, s);
}

}  // namespace ssmp
