// tree.cu -- a step's drafted trees: who sees whom, and the path that the model's picks confirm.
//
// Whole numbers over some hundred drafts a sequence: a few microseconds of dependent reads whatever is done, so both
// kernels are written for few steps in a row, a sequence's drafts in shared memory and one launch for the batch.
#include "page.cuh"

namespace kvc {
namespace {

constexpr int kMaskThreads = 128;

// Drafts of sequence b, and whether every parent is one of the drafts before it (block-wide).
__device__ __forceinline__ int drafts_of(const int32_t* n_q, int b, int T) { return n_q ? min(max(n_q[b], 0), T) : T; }

// A CTA a sequence, a thread a draft. Parents have lower numbers, so a walk up the tree meets the words of a row from
// its own down: the word in hand is written when the walk leaves it, and the words it passes over are zero.
__global__ void __launch_bounds__(kMaskThreads) tree_mask_kernel(int T, const int32_t* parent, const int32_t* n_q,
                                                                int window, uint32_t* mask, int32_t* depth,
                                                                int32_t* status) {
  __shared__ int16_t par[KVC_TREE_MAX];
  griddep_launch();
  griddep_wait();
  const int b = blockIdx.x, n = drafts_of(n_q, b, T), words = (T + 31) / 32;
  bool bad = false;
  for (int i = threadIdx.x; i < n; i += kMaskThreads) {
    const int p = parent[(size_t)b * T + i];
    bad |= p < -1 || p >= i;
    par[i] = (int16_t)p;
  }
  bad = __syncthreads_or(bad);
  if (bad && threadIdx.x == 0) status_or(status, KVC_STATUS_BAD_INDEX);
  for (int i = threadIdx.x; i < T; i += kMaskThreads) {
    uint32_t* row = mask + ((size_t)b * T + i) * words;
    int d = 0, w = words - 1;
    uint32_t bits = 0u;
    if (i < n && !bad)
      for (int j = i; j >= 0; j = par[j], ++d)
        if (window == 0 || d < window) {
          for (; w > j >> 5; --w) {
            row[w] = bits;
            bits = 0u;
          }
          bits |= 1u << (j & 31);
        }
    for (; w >= 0; --w) {
      row[w] = bits;
      bits = 0u;
    }
    if (depth) depth[(size_t)b * T + i] = max(d - 1, 0);
  }
}

// A warp a sequence, one sweep over its drafts 32 at a time: children come behind their parents, so the next kept
// draft is the first lane behind the last one whose parent that is and whose token the model picked there.
constexpr int kVerifyWarps = 4;
__global__ void __launch_bounds__(32 * kVerifyWarps) tree_verify_kernel(int B, int T, const int32_t* parent,
                                                                       const int32_t* draft, const int32_t* target,
                                                                       const int32_t* n_q, int32_t* path, int32_t* n_path,
                                                                       int32_t* next, int32_t* status) {
  griddep_launch();
  griddep_wait();
  const int b = blockIdx.x * kVerifyWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (b >= B) return;
  const int n = drafts_of(n_q, b, T);
  const size_t row = (size_t)b * T;
  bool bad = false;
  for (int i = lane; i < n; i += 32) {
    const int p = parent[row + i];
    bad |= p < -1 || p >= i;
  }
  bad = __any_sync(kFull, bad);
  if (bad && lane == 0) status_or(status, KVC_STATUS_BAD_INDEX);
  int last = -1, want = -1, k = 0;  // the last kept draft and the model's pick behind it
  if (n > 0 && !bad) {
    if (lane == 0) path[row] = 0;
    last = 0, k = 1;
    want = target[row];
    for (int i0 = 0; i0 < n; i0 += 32) {
      const int i = i0 + lane;
      const int p = i < n ? parent[row + i] : -1, d = i < n ? draft[row + i] : 0, t = i < n ? target[row + i] : 0;
      for (;;) {
        const unsigned hit = __ballot_sync(kFull, i > last && p == last && d == want);
        if (!hit) break;
        const int j = __ffs(hit) - 1;
        last = i0 + j;
        want = __shfl_sync(kFull, t, j);
        if (lane == 0) path[row + k] = last;
        ++k;
      }
    }
  }
  for (int i = k + lane; i < T; i += 32) path[row + i] = -1;
  if (lane == 0) {
    n_path[b] = k;
    if (next) next[b] = want;
  }
}

}  // namespace

int launch_tree_mask(int B, int T, const int32_t* parent, const int32_t* n_q, int window, uint32_t* mask, int32_t* depth,
                     int32_t* status, cudaStream_t s) {
  return launch_pdl(tree_mask_kernel, dim3(B), dim3(kMaskThreads), 0, s, false, T, parent, n_q, window, mask, depth,
                    status) == cudaSuccess
             ? KVC_OK
             : KVC_ERR_LAUNCH;
}

int launch_tree_verify(int B, int T, const int32_t* parent, const int32_t* draft, const int32_t* target,
                       const int32_t* n_q, int32_t* path, int32_t* n_path, int32_t* next, int32_t* status,
                       cudaStream_t s) {
  return launch_pdl(tree_verify_kernel, dim3((B + kVerifyWarps - 1) / kVerifyWarps), dim3(32 * kVerifyWarps), 0, s, false,
                    B, T, parent, draft, target, n_q, path, n_path, next, status) == cudaSuccess
             ? KVC_OK
             : KVC_ERR_LAUNCH;
}

}  // namespace kvc
