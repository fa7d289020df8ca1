// Attention of a few new tokens over a paged cache, heads of 128.
#include "fo_paged_few.cuh"

fo_status fo_ops::attend_few_128(FewParams& k, int eights, bool eight, int sms, cudaStream_t s) {
  return launch_for<128>(k, eights, eight, sms, s);
}
