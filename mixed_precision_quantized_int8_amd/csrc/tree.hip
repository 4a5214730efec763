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

// A thread has draft t, or t and t + BS (kMaxDrafts): its mask and depth cover the ancestors up to
// some distance, and each step takes those of the ancestor at that distance as well: twice as
// far, until every draft has come to the text.  (A walk from parent to parent took 6.8 us
// for 64 trees of 256 drafts, a step an LDS read behind the other.)
template <int W, int BS>
__global__ __launch_bounds__(BS) void tree_plan_kernel(TreeRows r, int32_t* __restrict__ positions,
                                                        uint64_t* __restrict__ masks, int words) {
  constexpr int NJ = (64 * W + BS - 1) / BS;   // drafts a thread
  __shared__ uint64_t s_mask[64 * W][W];
  __shared__ int s_up[64 * W], s_depth[64 * W];
  const DraftSpan d = drafts_of(r, blockIdx.x);
  const int len = max(r.lengths[blockIdx.x], 0), t = threadIdx.x;
  uint64_t mask[NJ][W];
  int up[NJ], depth[NJ];
#pragma unroll
  for (int n = 0; n < NJ; ++n) {
    const int j = t + BS * n;
    up[n] = -1;
    if (j < d.n) {
      const int p = r.parents[d.c0 + j];
      up[n] = p >= 0 && p < j ? p : -1;
    }
    depth[n] = up[n] >= 0;
#pragma unroll
    for (int w = 0; w < W; ++w) mask[n][w] = w == j >> 6 ? 1ull << (j & 63) : 0ull;
  }
  for (;;) {
    bool more = false;
#pragma unroll
    for (int n = 0; n < NJ; ++n) {
      const int j = t + BS * n;
      if (j < d.n) {
#pragma unroll
        for (int w = 0; w < W; ++w) s_mask[j][w] = mask[n][w];
        s_up[j] = up[n];
        s_depth[j] = depth[n];
      }
      more |= up[n] >= 0;
    }
    if (!__syncthreads_or(more)) break;
#pragma unroll
    for (int n = 0; n < NJ; ++n)
      if (const int p = up[n]; p >= 0) {
#pragma unroll
        for (int w = 0; w < W; ++w) mask[n][w] |= s_mask[p][w];
        depth[n] += s_depth[p];
        up[n] = s_up[p];
      }
    __syncthreads();
  }
#pragma unroll
  for (int n = 0; n < NJ; ++n) {
    const int j = t + BS * n;
    if (j >= d.n) continue;
    uint64_t* row = masks + (d.c0 + j) * words;
#pragma unroll
    for (int w = 0; w < W; ++w)
      if (w < words) row[w] = mask[n][w];
    for (int w = W; w < words; ++w) row[w] = 0;
    positions[d.c0 + j] = len + depth[n];
  }
}

// A workgroup a sequence (one wave for up to 64 drafts); its first wave walks: from the accepted draft `cur` on, the first
// of its children whose token is what the model chose after it, 64 drafts looked at
// together.
template <int BS>
__global__ __launch_bounds__(BS) void tree_accept_kernel(
    TreeRows r, const int64_t* __restrict__ tokens, const int64_t* __restrict__ choices,
    const int64_t* __restrict__ first, int32_t* __restrict__ path, int32_t* __restrict__ counts,
    int32_t* __restrict__ new_lengths, int64_t* __restrict__ next) {
  __shared__ int64_t s_token[kMaxDrafts], s_choice[kMaxDrafts];
  __shared__ int s_parent[kMaxDrafts], s_path[kMaxDrafts], s_count;
  const int b = blockIdx.x, t = threadIdx.x;
  const DraftSpan d = drafts_of(r, b);
  for (int j = t; j < d.n; j += BS) {
    const int p = r.parents[d.c0 + j];
    s_parent[j] = p >= 0 && p < j ? p : -1;
    s_token[j] = tokens[d.c0 + j];
    s_choice[j] = choices[d.c0 + j];
  }
  __syncthreads();
  if (t < 64) {
    int cur = -1, count = 0;
    int64_t want = first ? first[b] : -1;
    if (!first && d.n > 0) {   // the first draft is known
      cur = 0;
      want = s_choice[0];
      if (t == 0) s_path[0] = 0;
      count = 1;
    }
    for (bool more = first || d.n > 0; more;) {   // cur rises with every turn
      more = false;
      for (int j0 = (cur + 1) & ~63; j0 < d.n; j0 += 64) {
        const int j = j0 + t;
        const uint64_t hit = __ballot(j < d.n && s_parent[j] == cur && s_token[j] == want);
        if (hit) {
          cur = j0 + __builtin_ctzll(hit);
          want = s_choice[cur];
          if (t == 0) s_path[count] = cur;
          ++count;
          more = true;
          break;
        }
      }
    }
    if (t == 0) {
      s_count = count;
      counts[b] = count;
      new_lengths[b] = max(r.lengths[b], 0) + count;
      next[b] = want;
    }
  }
  __syncthreads();
  for (int j = t; j < d.n; j += BS) path[d.c0 + j] = j < s_count ? (int32_t)(d.c0 + s_path[j]) : -1;
}

hipError_t launch_tree_plan(const TreeRows& r, int32_t* positions, uint64_t* masks, int words,
                            hipStream_t stream) {
  // (the drafts that max_q allows, in words)
#define I8L_PLAN(W, BS)                                                                        \
  hipLaunchKernelGGL((tree_plan_kernel<W, BS>), dim3(r.n), dim3(BS), 0, stream, r, positions,  \
                     masks, words)
  if (r.max_q <= 64) I8L_PLAN(1, 64);
  else if (r.max_q <= 256) I8L_PLAN(4, 256);
  else I8L_PLAN(8, 256);
#undef I8L_PLAN
  return hipGetLastError();
}

hipError_t launch_tree_accept(const TreeRows& r, const int64_t* tokens, const int64_t* choices,
                              const int64_t* first, int32_t* path, int32_t* counts,
                              int32_t* new_lengths, int64_t* next, hipStream_t stream) {
#define I8L_ACCEPT(BS)                                                                           \
  hipLaunchKernelGGL((tree_accept_kernel<BS>), dim3(r.n), dim3(BS), 0, stream, r, tokens, choices, \
                     first, path, counts, new_lengths, next)
  if (r.max_q <= 64) I8L_ACCEPT(64);
  else I8L_ACCEPT(256);
#undef I8L_ACCEPT
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
