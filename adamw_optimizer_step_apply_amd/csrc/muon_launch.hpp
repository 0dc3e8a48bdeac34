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
    adamw_muon_hparams hp;   // a step's
};
hipError_t launch_ns_prologue(const adamw_muon_hparams& hp, const ClipRule& clip, int32_t* d_step,
                              const int32_t* d_found_inf, const adamw_loss_scale_state* d_amp, char* ws,
                              hipStream_t stream);
hipError_t launch_ns_batch(const NsCall& call, const NsBatch& batch, hipStream_t stream);

}  // namespace adamw
