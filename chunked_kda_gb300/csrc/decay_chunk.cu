// Linear attention with a decay for each head, the form for prompts.
#include "common.cuh"
#include "kda_internal.h"

namespace kda {

size_t decay_chunk_workspace_bytes(bool, int, int, int, int, int, int, bool) { return 0; }

cudaError_t launch_decay_chunk(const DecayArgs& a) { return launch_decay_recurrent(a); }

}  // namespace kda
