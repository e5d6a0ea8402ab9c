// The MLP block's handle, shared by its entry points' files.
#pragma once
#include "host_common.cuh"

struct tp_mlp_handle {
  tpmlp::host::HandleCore core;
  tp_mlp_config cfg;
  unsigned long long drop_seed = 0, drop_offset = 0;
  bool ln_prologue = true;   // tp_mlp_set_ln_prologue
  int* fp4_status = nullptr; // tp_fp4_mlp_set_status
};
