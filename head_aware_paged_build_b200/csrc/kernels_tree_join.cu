// Joining the pieces of row groups that tree attention split over CTAs.
//
// With m_i, l_i, acc_i the running maximum (log2 domain), sum and unnormalised
// output of piece i:  M = max m_i,  O = sum 2^(m_i - M) acc_i / sum 2^(m_i - M) l_i,
// pieces in line order, so the same inputs give the same bits.
//
// A programmatic dependent launch: its blocks are placed while the attention's
// last CTAs run and wait for that grid on the device.  (The last CTA of a row
// group joining it instead was 3 to 10 times slower on the 8K and 32K layers:
// one SM reads what a dozen wrote, 64 KB for each piece of 128 rows.)  Every
// block lists the split groups (the CTA a group starts in left its description),
// and they share out the rows: eight rows an item, a warp each, or two rows an
// item, four warps each, when there are few rows and so probably many pieces.
// Bound by L2 latency: a warp keeps eight pieces' loads in flight.
#include "kernels.h"
#include "tree_common.cuh"

namespace sp {
namespace {

constexpr int kJoinThreads = 256;
constexpr int kJoinWarps = kJoinThreads / 32;

template <typename T, int D>
__global__ void __launch_bounds__(kJoinThreads) tree_join_kernel(TreeLaunch a) {
  constexpr int V = D / 32;  // columns of a lane
  __shared__ int s_end[kTreeMaxCtas];  // items up to and with each CTA's group
  __shared__ float s_acc[kJoinWarps][D];
  __shared__ float s_l[kJoinWarps];
  __shared__ int s_few;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int c = threadIdx.x; c < a.n_ctas; c += kJoinThreads)
    s_end[c] = a.joins[c].n_pieces > 0 ? a.joins[c].rows : 0;
  __syncthreads();
  if (warp == 0) {
    constexpr int PER = kTreeMaxCtas / 32;
    int rows = 0;
    for (int i = 0; i < PER; ++i) rows += lane * PER + i < a.n_ctas ? s_end[lane * PER + i] : 0;
    const int all = __reduce_add_sync(0xffffffffu, rows);
    const bool few = all <= 4 * int(gridDim.x);
    const int per = few ? 2 : kJoinWarps;
    int items = 0;
    for (int i = 0; i < PER; ++i)
      if (lane * PER + i < a.n_ctas) {
        items += (s_end[lane * PER + i] + per - 1) / per;
        s_end[lane * PER + i] = items;
      }
    int upto = items;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += x;
    }
    for (int i = 0; i < PER; ++i)
      if (lane * PER + i < a.n_ctas) s_end[lane * PER + i] += upto - items;
    if (lane == 0) s_few = few;
  }
  __syncthreads();
  const bool few = s_few;
  const int rows_max = a.nodes_per_group * a.group;
  const int64_t stride = tree_slot_floats(a);
  const int total = s_end[a.n_ctas - 1];
  for (int item = blockIdx.x; item < total; item += gridDim.x) {
    int lo = 0, hi = a.n_ctas - 1;  // the first CTA whose items reach past this one
    while (lo < hi) {
      const int mid = (lo + hi) / 2;
      if (s_end[mid] > item) hi = mid;
      else lo = mid + 1;
    }
    const TreeJoin jn = a.joins[lo];
    const int in_group = item - (lo ? s_end[lo - 1] : 0);
    const int W = few ? 4 : 1;  // warps a row
    const int row = few ? in_group * 2 + warp / 4 : in_group * kJoinWarps + warp, part = few ? warp % 4 : 0;
    auto slot = [&](int i) { return a.partial + int64_t(i == 0 ? jn.first_slot : 2 * (lo + i)) * stride; };
    float M = -INFINITY, l = 0.f, acc[V];
#pragma unroll
    for (int v = 0; v < V; ++v) acc[v] = 0.f;
    if (row < jn.rows) {
      for (int i = lane; i < jn.n_pieces; i += 32) M = fmaxf(M, __ldcg(slot(i) + rows_max * D + 2 * row));
#pragma unroll
      for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
      const float base = M == -INFINITY ? 0.f : M;
      constexpr int B = 8;  // pieces in flight
      for (int i0 = part; i0 < jn.n_pieces; i0 += B * W) {
        float2 ml[B];
        float x[B][V];
#pragma unroll
        for (int u = 0; u < B; ++u) {
          const int i = i0 + u * W;
          ml[u] = make_float2(-INFINITY, 0.f);
#pragma unroll
          for (int v = 0; v < V; ++v) x[u][v] = 0.f;
          if (i >= jn.n_pieces) continue;
          const float* s = slot(i);
          ml[u] = __ldcg(reinterpret_cast<const float2*>(s + rows_max * D + 2 * row));
          if constexpr (V == 4)
            *reinterpret_cast<float4*>(x[u]) = __ldcg(reinterpret_cast<const float4*>(s + row * D + lane * V));
          else
            *reinterpret_cast<float2*>(x[u]) = __ldcg(reinterpret_cast<const float2*>(s + row * D + lane * V));
        }
#pragma unroll
        for (int u = 0; u < B; ++u) {
          const float f = exp2f(ml[u].x - base);
          l += f * ml[u].y;
#pragma unroll
          for (int v = 0; v < V; ++v) acc[v] += f * x[u][v];
        }
      }
    }
    if (few) {  // the row's four warps, in order
      __syncthreads();
#pragma unroll
      for (int v = 0; v < V; ++v) s_acc[warp][lane * V + v] = acc[v];
      if (lane == 0) s_l[warp] = l;
      __syncthreads();
      if (part != 0) continue;
#pragma unroll
      for (int w = 1; w < 4; ++w) {
        l += s_l[warp + w];
#pragma unroll
        for (int v = 0; v < V; ++v) acc[v] += s_acc[warp + w][lane * V + v];
      }
    }
    if (row >= jn.rows) continue;
    const int64_t at =
        (int64_t(jn.b) * a.T + jn.node0 + row / a.group) * a.num_q_heads + jn.kv * a.group + row % a.group;
    const float inv = a.v_scale / l;
    T* dst = static_cast<T*>(a.out) + at * D + lane * V;
    if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int v = 0; v < V; v += 2)
        reinterpret_cast<uint32_t*>(dst)[v / 2] = pack_bf16x2(acc[v] * inv, acc[v + 1] * inv);
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) dst[v] = acc[v] * inv;
    }
    if (lane == 0 && a.lse) a.lse[at] = (M + log2f(l)) * kTreeLn2;
  }
}

template <typename T, int D>
cudaError_t launch(const TreeLaunch& a, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(4 * 148);
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, tree_join_kernel<T, D>, a);
}

}  // namespace

cudaError_t launch_tree_join(const TreeLaunch& a, cudaStream_t s) {
  if (a.bf16) return a.D == 128 ? launch<__nv_bfloat16, 128>(a, s) : launch<__nv_bfloat16, 64>(a, s);
  return a.D == 128 ? launch<float, 128>(a, s) : launch<float, 64>(a, s);
}

}  // namespace sp
