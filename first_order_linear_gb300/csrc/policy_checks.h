// policy_checks.h -- the workspace query of the policy-update operators
// (policy_api.cu), as rlca_workspace_size (api.cu) calls it.
#pragma once

#include <cstddef>
#include <cstdint>

namespace rlca {

// whether `estimator` is one of theirs
bool policy_estimator(int estimator);
// its workspace in *bytes; RLCA_OK or an error status
int policy_workspace_size(int estimator, int64_t E, int64_t T, int32_t num_actions, uint32_t flags, size_t* bytes);

}  // namespace rlca
