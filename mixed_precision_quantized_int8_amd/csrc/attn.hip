// Causal attention over the 8-bit key/value cache: the kernels of attn.h.
#include "attn.h"

namespace i8l {

size_t attention_partials(int B, int H, int G, int D, int max_q, int max_len, int window) {
  const Plan p = plan(B, H, G, D, max_q, max_len, window);
  const size_t count = (size_t)B * H * G * max_q * p.n_split;
  return p.n_split == 1 ? 0 : part_head(count) + count * D;
}

hipError_t launch_attention(const AttnArgs& a, hipStream_t stream) {
  return launch_planned<false>(a, stream);
}

}  // namespace i8l
