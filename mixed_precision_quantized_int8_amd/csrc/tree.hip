// Trees of drafted tokens: their positions and masks, attention for them (attn.h's
// kernels), and the path that the model's choices accept.
//
// Draft j of a sequence follows draft parents[j] < j, or the cached text (-1, or any
// entry that is no earlier draft).  Plan and verdict are bound by latency: a workgroup,
// or a wave, a sequence, the tree in LDS.
#include "attn.h"

namespace i8l {

struct DraftSpan {
  int64_t c0;
  int n;
};
__device__ __forceinline__ DraftSpan drafts_of(const TreeRows& r, int b) {
  int64_t c0 = r.cu ? r.cu[b] : b, c1 = r.cu ? r.cu[b + 1] : b + 1;
  c0 = min(max(c0, (int64_t)0), r.rows);
  c1 = min(max(c1, c0), r.rows);
  return DraftSpan{c0, (int)min(c1 - c0, (int64_t)r.max_q)};
}

// A thread walks from its draft to the text: each step one bit of its mask, one of its
// depth.  Ancestors come in descending order, so the words do too.
__global__ __launch_bounds__(256) void tree_plan_kernel(TreeRows r, int32_t* __restrict__ positions,
                                                        uint64_t* __restrict__ masks, int words) {
  __shared__ int s_parent[kMaxDrafts];
  const DraftSpan d = drafts_of(r, blockIdx.x);
  for (int j = threadIdx.x; j < d.n; j += 256) {
    const int p = r.parents[d.c0 + j];
    s_parent[j] = p >= 0 && p < j ? p : -1;
  }
  const int len = max(r.lengths[blockIdx.x], 0);
  __syncthreads();
  for (int j = threadIdx.x; j < d.n; j += 256) {
    uint64_t* row = masks + (d.c0 + j) * words;
    int p = j, depth = -1;
    for (int w = words - 1; w >= 0; --w) {
      uint64_t bits = 0;
      for (; p >= 64 * w; p = s_parent[p], ++depth) bits |= 1ull << (p & 63);   // (-1: below any)
      row[w] = bits;
    }
    positions[d.c0 + j] = len + depth;
  }
}

// A wave a sequence: from the accepted draft `cur` on, the first of its children whose
// token is what the model chose after it; 64 drafts a step are looked at together.
__global__ __launch_bounds__(64) void tree_accept_kernel(
    TreeRows r, const int64_t* __restrict__ tokens, const int64_t* __restrict__ choices,
    const int64_t* __restrict__ first, int32_t* __restrict__ path, int32_t* __restrict__ counts,
    int32_t* __restrict__ new_lengths, int64_t* __restrict__ next) {
  __shared__ int64_t s_token[kMaxDrafts], s_choice[kMaxDrafts];
  __shared__ int s_parent[kMaxDrafts], s_path[kMaxDrafts];
  const int b = blockIdx.x, lane = threadIdx.x;
  const DraftSpan d = drafts_of(r, b);
  for (int j = lane; j < d.n; j += 64) {
    const int p = r.parents[d.c0 + j];
    s_parent[j] = p >= 0 && p < j ? p : -1;
    s_token[j] = tokens[d.c0 + j];
    s_choice[j] = choices[d.c0 + j];
  }
  const int len = max(r.lengths[b], 0);
  int cur = -1, count = 0;
  int64_t want = first ? first[b] : -1;
  __syncthreads();
  if (!first && d.n > 0) {   // the first draft is known
    cur = 0;
    want = s_choice[0];
    if (lane == 0) s_path[0] = 0;
    count = 1;
  }
  for (bool more = first || d.n > 0; more;) {   // cur rises with every turn
    more = false;
    for (int j0 = (cur + 1) & ~63; j0 < d.n; j0 += 64) {
      const int j = j0 + lane;
      const uint64_t hit = __ballot(j < d.n && s_parent[j] == cur && s_token[j] == want);
      if (hit) {
        cur = j0 + __builtin_ctzll(hit);
        want = s_choice[cur];
        if (lane == 0) s_path[count] = cur;
        ++count;
        more = true;
        break;
      }
    }
  }
  __syncthreads();
  for (int j = lane; j < d.n; j += 64) path[d.c0 + j] = j < count ? (int32_t)(d.c0 + s_path[j]) : -1;
  if (lane == 0) {
    counts[b] = count;
    new_lengths[b] = len + count;
    next[b] = want;
  }
}

hipError_t launch_tree_plan(const TreeRows& r, int32_t* positions, uint64_t* masks, int words,
                            hipStream_t stream) {
  hipLaunchKernelGGL(tree_plan_kernel, dim3(r.n), dim3(256), 0, stream, r, positions, masks, words);
  return hipGetLastError();
}

hipError_t launch_tree_accept(const TreeRows& r, const int64_t* tokens, const int64_t* choices,
                              const int64_t* first, int32_t* path, int32_t* counts,
                              int32_t* new_lengths, int64_t* next, hipStream_t stream) {
  hipLaunchKernelGGL(tree_accept_kernel, dim3(r.n), dim3(64), 0, stream, r, tokens, choices, first, path,
                     counts, new_lengths, next);
  return hipGetLastError();
}

size_t tree_partials(int B, int H, int G, int D, int max_q, int max_len, int window) {
  const Plan p = plan(B, H, G, D, max_q, max_len, window);
  if (const int n = tree_shares(p, B, H, G, max_q, max_len, window))
    return kShareHead + 2 * (size_t)n * H * p.rows * (D + 2);
  const size_t count = (size_t)B * H * G * max_q * p.n_split;
  return p.n_split == 1 ? 0 : part_head(count) + count * D;
}

hipError_t launch_tree_attention(const TreeArgs& a, hipStream_t stream) {
  return launch_planned<true>(a, stream);
}

}  // namespace i8l
