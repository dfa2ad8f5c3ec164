// policy_checks.h -- what the entry points of the policy-update operators and
// of a recurrent policy's trunk share, and their workspace query
// (policy_api.cu), as rlca_workspace_size (api.cu) calls it.
#pragma once

#include <cstddef>
#include <cstdint>

#include "policy.h"
#include "rlca.h"

namespace rlca {

// largest row count, width and vocabulary: products of any two, times the
// element size and a tile's rounding, stay well inside 63 bits
constexpr int64_t kMaxRows = INT32_MAX;
constexpr int64_t kMaxWidth = int64_t(1) << 30;
constexpr int64_t kMaxStride = int64_t(1) << 31;

inline size_t ebytes(uint32_t flags) { return (flags & RLCA_BF16) ? 2 : 4; }

// status of a finished sequence of launches
inline int launched(cudaError_t e, cudaStream_t s) { return e == cudaSuccess ? checked_build_status(s) : RLCA_ERR_CUDA; }

// whether `estimator` is one of theirs
bool policy_estimator(int estimator);
// its workspace in *bytes; RLCA_OK or an error status
int policy_workspace_size(int estimator, int64_t E, int64_t T, int32_t num_actions, uint32_t flags, size_t* bytes);

}  // namespace rlca
