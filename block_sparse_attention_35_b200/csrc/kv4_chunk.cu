#include "kv4_attn.cuh"
namespace pbsa {
bool chunk_takes(const pbsa_kv4_config& c, int R) { return false; }
cudaError_t launch_chunk_attn(const AttnArgs& a, cudaStream_t st) { return cudaErrorNotSupported; }
cudaError_t launch_chunk_mass(const AttnArgs& a, cudaStream_t st) { return cudaErrorNotSupported; }
}
