// muon_launch.hpp -- the launchers of muon.hip, for the entry points of api.cpp.
#pragma once

#include <hip/hip_runtime.h>

#include "muon.hpp"

namespace adamw {

// One call over a plan already on the device.
struct NsCall {
    NsKind kind;
    const DevMatrix* mats;
    const DevTile* tiles;
    char* ws;
    adamw_newton_schulz ns;
    NsScales scales;
    // a step's
    adamw_muon_hparams hp;
    ClipRule clip;
    int32_t* step;
    const int32_t* found_inf;
    const adamw_loss_scale_state* amp;
};
// `last`: the list's last batch, which advances a step's counter
hipError_t launch_ns_batch(const NsCall& call, const NsBatch& batch, bool last, hipStream_t stream);
// A step over an empty list: the counter alone.
hipError_t launch_ns_count(const NsCall& call, hipStream_t stream);

}  // namespace adamw
