// Per-thread state of the C ABI (muon_set_stream, muon_set_workspace,
// muon_set_step_options, muon_last_error), shared by its translation units.
#pragma once

#include <hip/hip_runtime_api.h>

#include <string>

#include "muon.h"

namespace muon {

struct State {
  hipStream_t stream = nullptr;
  void *ws = nullptr;
  size_t ws_bytes = 0;
  int32_t iters = 5;
  float coeffs[3] = {3.4445f, -4.7750f, 2.0315f};
  float eps = 1e-7f;
  uint32_t mode = MUON_NS_FULL | MUON_PACK_COST | MUON_AA_PLAIN;
  std::string err;
};

State &thread_state();  // api.cpp

}  // namespace muon
