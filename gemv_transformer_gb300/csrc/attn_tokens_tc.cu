#include "attn_tokens.cuh"
namespace wq {
namespace tok {
bool tokens_tc_takes(const KvView &, int) { return false; }
void tokens_tc_shape(int, int, int, int, int, int &rt, int &kt, int &dp) { rt = kt = dp = 0; }
cudaError_t launch_tokens_tc(const TokensArgs &, const KvView &, const DeviceInfo &, cudaStream_t) { return cudaErrorNotSupported; }
}
}
