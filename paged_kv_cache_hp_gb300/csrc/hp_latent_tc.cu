#include "hp_latent.cuh"
namespace hp {
bool latent_tc_fits(uint32_t, uint64_t, uint64_t, uint64_t) { return false; }
int launch_latent_tc(const LatentArgs&, void*) { return HP_ERR_CUDA; }
bool latent_prefill_tc_fits(uint32_t, uint64_t, uint32_t, uint32_t, uint64_t, uint64_t, uint32_t) { return false; }
int launch_latent_prefill_tc(const LatentPrefillArgs&, void*) { return HP_ERR_CUDA; }
}
