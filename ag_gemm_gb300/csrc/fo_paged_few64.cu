// Attention of a few new tokens over a paged cache, heads of 64.
#include "fo_paged_few.cuh"

fo_status fo_ops::attend_few_64(FewParams& k, int eights, bool eight, int sms, cudaStream_t s) {
  return launch_for<64>(k, eights, eight, sms, s);
}
