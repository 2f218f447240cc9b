// Host-side helpers shared by the library's translation units (defined in mfa_decode.cu).
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <cstdint>

#include "mfa.h"

namespace mfa {

// Records the text of a CUDA failure for mfa_last_cuda_error() and returns MFA_ERR_CUDA.
mfa_status cuda_fail(cudaError_t e, const char* where);
// The same for a failure with a text of its own (a static string).
mfa_status cuda_fail_msg(const char* msg);

// The driver's cuTensorMapEncodeTiled, or null.
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();

// Shape, dtype and range checks of a problem description (MFA_OK, or the error to return).
mfa_status check_problem(const mfa_problem* pr);

// The attention shape of a problem that check_problem accepts: 0 MFA, 1 grouped heads,
// 2 shared latent.
int problem_shape(const mfa_problem* pr);

// Shape, dtype and range checks of a problem over a block-scaled cache with 1 to most_tokens new tokens a
// sequence (MFA_OK, or the error).
mfa_status check_block_problem(const mfa_problem* pr, int scale_tokens, int most_tokens = 4);

// Shape and range checks of a rope's description (MFA_OK, or the error).
mfa_status check_rope(const mfa_rope_config* c);

// Whether two sets of rows share memory: `rows` rows of `len` elements of esz bytes each, `stride` apart.
bool rows_share(const void* a, int64_t a_stride, int64_t a_len, const void* b, int64_t b_stride, int64_t b_len, int rows,
                int esz);

// True when p is a multiple of a bytes.
bool aligned(const void* p, uintptr_t a);

}  // namespace mfa
