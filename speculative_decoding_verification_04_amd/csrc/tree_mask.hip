// Positions and visibility bits of a candidate tree's nodes, from its links
// (gfx950).
//
// Node i of a sequence's tree attends the sequence's cached rows and the nodes
// on the path from the root to i, and stands at position n_b + depth(i).  Both
// follow from parent(i): the path of i is {i} and the path of parent(i).
//
// Design.  One workgroup per tree, one lane per node, everything in
// LDS.  Parents: the first child of i knows i; a later sibling finds its
// parent through the run of siblings before it, by pointer jumping.  Paths:
// sets of 256 bits, doubled along the parents (path of i |= path of the
// ancestor at distance 2^t), so a chain of 255 links takes 8 rounds and not
// 255.  Bound by its barriers and LDS round trips: one tree of 16 nodes 2.5 us, 256
// trees of 255 nodes 6.5 us (2.9 MB read and written).
#include "cache_view.h"

namespace specv {
namespace {

constexpr int kTreeThreads = 256;
constexpr int kWords = SPEC_TREE_MAX_N / 32;
constexpr int kRounds = 12;   // log2(SPEC_TREE_MAX_N) and the last, empty one, and some

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

struct TreeMaskParams {
  int N, words;
  const int32_t *first_child, *next_sibling, *kv_len;
  int32_t *positions;
  uint32_t *mask;
  int32_t *status;
};

__global__ __launch_bounds__(kTreeThreads) void tree_mask_kernel(TreeMaskParams P) {
  __shared__ int refs[SPEC_TREE_MAX_N];                   // links that point to a node
  __shared__ int up[2][SPEC_TREE_MAX_N];                  // parent + N, or the sibling before; then ancestors
  __shared__ u32x4 path[2][SPEC_TREE_MAX_N][kWords / 4];
  __shared__ int more[2][kRounds];                        // whether a round has work, by phase
  __shared__ int bad;
  const int b = blockIdx.x, i = threadIdx.x, N = P.N;
  const bool in = i < N;
  refs[i] = 0;
  up[0][i] = -1;
  if (i == 0) bad = 0;
  if (i < 2 * kRounds) more[i / kRounds][i % kRounds] = 0;
  const int fc = in ? P.first_child[static_cast<long long>(b) * N + i] : -1;
  const int ns = in ? P.next_sibling[static_cast<long long>(b) * N + i] : -1;
  const int n = P.kv_len[b];
  __syncthreads();
  bool ok = true;
  if (fc != -1) {
    ok = fc > i && fc < N;
    if (ok) {
      atomicAdd(&refs[fc], 1);
      up[0][fc] = N + i;                                  // its parent
    }
  }
  if (ns != -1) {
    const bool good = ns > i && ns < N;
    ok = ok && good;
    if (good) {
      atomicAdd(&refs[ns], 1);
      up[0][ns] = i;                                      // the sibling before it
    }
  }
  if (!ok) bad = 1;
  __syncthreads();
  if (refs[i] > 1) bad = 1;                               // two links to one node: two paths
  // Siblings to parents: after round t an entry has skipped 2^t siblings.  A
  // node that no link reaches, and its later siblings, end with none (-1);
  // so do the root's siblings.
  // Every link points forward, so N entries settle in log2 N rounds; a round
  // that finds nothing left to do is the last.
  int cur = 0, x = up[0][i];
  for (int r = 0; r < kRounds; ++r) {
    if (x >= 0 && x < N) more[0][r] = 1;
    __syncthreads();
    if (!more[0][r]) break;
    if (x >= 0 && x < N) x = up[cur][x];
    cur ^= 1;
    up[cur][i] = x;
  }
  // Paths, doubled along the parents.  anc: the ancestor 2^t above, or -1.
  int anc = x >= N ? x - N : -1;
  u32x4 w[kWords / 4];
#pragma unroll
  for (int k = 0; k < kWords; ++k) w[k / 4][k % 4] = (i >> 5) == k && in ? 1u << (i & 31) : 0u;
  for (int r = 0; r < kRounds; ++r) {
    cur ^= 1;
    up[cur][i] = anc;
    path[cur][i][0] = w[0];
    if (P.words > 4) path[cur][i][1] = w[1];
    if (anc >= 0) more[1][r] = 1;
    __syncthreads();
    if (!more[1][r]) break;
    if (anc >= 0) {
      w[0] |= path[cur][anc][0];
      if (P.words > 4) w[1] |= path[cur][anc][1];
      anc = up[cur][anc];
    }
  }
  // A path that does not start at the root belongs to no branch of the tree.
  const bool linked = in && (w[0][0] & 1u) && !bad;
  int depth = -1;
#pragma unroll
  for (int k = 0; k < kWords; ++k) depth += __popc(w[k / 4][k % 4]);
  if (in) {
    const long long node = static_cast<long long>(b) * N + i;
    P.positions[node] = n + (linked ? depth : 0);
#pragma unroll
    for (int k = 0; k < kWords; ++k)
      if (k < P.words) P.mask[node * P.words + k] = linked ? w[k / 4][k % 4] : 0u;
  }
  if (i == 0 && P.status) P.status[b] = bad || n < 0 ? SPEC_ST_BAD_STATE : 0;
}

}  // namespace
}  // namespace specv

using namespace specv;

extern "C" int spec_tree_mask(int B, int N, const int32_t *first_child, const int32_t *next_sibling,
                              const int32_t *kv_len, int32_t *positions, uint32_t *mask, int32_t *status,
                              spec_stream_t stream) {
  if (!first_child || !next_sibling || !kv_len || !positions || !mask) return SPEC_EINVAL;
  if (B < 1 || N < 1) return SPEC_EINVAL;
  if (N > SPEC_TREE_MAX_N) return SPEC_ECAPACITY;
  const int threads = static_cast<int>(round_up(N, kWave));
  if (!launchable(B, threads)) return SPEC_EINVAL;
  const int words = (N + 31) / 32;
  const size_t b4 = static_cast<size_t>(B) * 4, bn4 = b4 * N;
  const void *ins[] = {first_child, next_sibling, kv_len};
  const size_t in_n[] = {bn4, bn4, b4};
  const void *outs[] = {positions, mask, status};
  const size_t out_n[] = {bn4, bn4 * words, b4};
  for (int o = 0; o < 3; ++o) {
    if (outs[o] && !aligned(outs[o], 4)) return SPEC_EINVAL;
    for (int j = 0; j < 3; ++j)
      if (overlaps(outs[o], out_n[o], ins[j], in_n[j])) return SPEC_EINVAL;
    for (int j = o + 1; j < 3; ++j)
      if (overlaps(outs[o], out_n[o], outs[j], out_n[j])) return SPEC_EINVAL;
  }
  TreeMaskParams P{N, words, first_child, next_sibling, kv_len, positions, mask, status};
  (void)hipGetLastError();
  hipLaunchKernelGGL(tree_mask_kernel, dim3(B), dim3(threads), 0, static_cast<hipStream_t>(stream), P);
  return launch_status();
}
