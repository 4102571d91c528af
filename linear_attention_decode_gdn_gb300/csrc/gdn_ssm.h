// gdn_ssm.h -- launch parameters of the selective state space layers' calls, shared by the C-ABI
// layer and the kernels. Not part of the public interface (include/gdn.h is).
#pragma once

#include <cstddef>
#include <cstdint>

#include <cuda_runtime_api.h>

#include "gdn.h"
#include "gdn_kv.h"

namespace gdn {

constexpr int kMaxNormWidth = 16384;
constexpr int kNormGroup = 128;  // channels of a scale, where a row has several

struct SsmParams {
  gdn_ssm s;
  int32_t* status;
};

struct ConvParams {
  gdn_conv c;
  int32_t* status;
};

cudaError_t launch_add_rms_norm(const gdn_norm& p, cudaStream_t stream);
cudaError_t launch_causal_conv(const ConvParams& p, cudaStream_t stream);
size_t ssm_workspace_bytes(int32_t batch, int32_t tokens, int32_t channels, int32_t state_size);
bool ssm_scan_in_parts(const gdn_ssm& s);  // whether the call uses its workspace
cudaError_t launch_ssm_scan(const SsmParams& p, void* workspace, cudaStream_t stream);
cudaError_t launch_ssm_step(const SsmParams& p, cudaStream_t stream);

}  // namespace gdn
