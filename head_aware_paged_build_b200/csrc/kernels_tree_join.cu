// Joining the pieces of row groups that tree attention split over CTAs.
//
// A programmatic dependent launch: its blocks are placed while the attention's
// last CTAs run and wait for that grid on the device.  (The last CTA of a row
// group joining it instead was 3 to 10 times slower on the 8K and 32K layers:
// one SM reads what a dozen wrote, 64 KB for each piece of 128 rows.)  Every
// block lists the split groups (the CTA a group starts in left its description)
// and takes its share of items.  A thread holds a row's 16 columns over a part
// of the pieces; a group of many pieces is divided into 4 or 16 parts, which
// meet in shared memory.  Bound by L2 latency.
#include "kernels.h"
#include "tree_common.cuh"

namespace sp {
namespace {

constexpr int kJoinThreads = 256;
constexpr int kCols = kJoinCols;

// Parts a group's pieces are divided into: one while a batch holds them.
__device__ __forceinline__ int join_parts(int n_pieces) {
  return n_pieces <= kJoinBatch ? 1 : n_pieces <= 4 * kJoinBatch ? 4 : 16;
}

template <typename T, int D>
__global__ void __launch_bounds__(kJoinThreads) tree_join_kernel(TreeLaunch a) {
  constexpr int CG = D / kCols;           // column groups of a row
  constexpr int R1 = kJoinThreads / CG;   // rows of an item in one part
  constexpr int PER = kTreeMaxCtas / 32;
  __shared__ int s_end[kTreeMaxCtas];  // items up to and with each CTA's group
  __shared__ TreeJoin s_join[kTreeMaxCtas];
  __shared__ float s_part[kJoinThreads][kCols + 1];
  __shared__ float s_m[kJoinThreads], s_l[kJoinThreads];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int tid = threadIdx.x, lane = tid & 31;
  for (int c = tid; c < kTreeMaxCtas; c += kJoinThreads) {
    int4 head = make_int4(0, 0, 0, 0), rest = head;  // n_pieces, first_slot, rows, b; the others
    if (c < a.n_ctas) {
      head = __ldcg(reinterpret_cast<const int4*>(a.joins + c));
      rest = __ldcg(reinterpret_cast<const int4*>(a.joins + c) + 1);
    }
    const int per = R1 / join_parts(head.x);
    s_end[c] = head.x > 0 ? (head.z + per - 1) / per : 0;
    reinterpret_cast<int4*>(s_join + c)[0] = head;
    reinterpret_cast<int4*>(s_join + c)[1] = rest;
  }
  __syncthreads();
  if (tid < 32) {  // a lane takes a run of CTAs
    int items[PER], sum = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) items[i] = s_end[lane * PER + i];
#pragma unroll
    for (int i = 0; i < PER; ++i) items[i] = sum += items[i];
    int upto = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += x;
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) s_end[lane * PER + i] = items[i] + upto - sum;
  }
  __syncthreads();
  const int total = s_end[a.n_ctas - 1];
  for (int item = blockIdx.x; item < total; item += gridDim.x) {
    int lo = 0, hi = a.n_ctas - 1;  // the first CTA whose items reach past this one
    while (lo < hi) {
      const int mid = (lo + hi) / 2;
      if (s_end[mid] > item) hi = mid;
      else lo = mid + 1;
    }
    const TreeJoin& jn = s_join[lo];
    const int parts = join_parts(jn.n_pieces), R = R1 / parts;
    const int row0 = (item - (lo ? s_end[lo - 1] : 0)) * R;
    // thread = (part, column group, row of the item)
    const int row = row0 + tid % R, cg = tid / R % CG, part = tid / (R * CG);
    float m = -INFINITY, l = 0.f, acc[kCols] = {};
    if (row < jn.rows) tree_sum_pieces<D>(a, jn.n_pieces, jn.first_slot, lo, row, cg, part, parts, m, l, acc);
    auto out_row = [&](int r) { return tree_out_row(a, jn.b, jn.kv, jn.node0, r); };
    if (parts == 1) {
      if (row < jn.rows) tree_finish_row<T, D>(a, out_row(row), cg, m, l, acc);
      continue;
    }
    // the parts meet: each brings its sums to the common maximum, then a thread adds up single columns in order
    s_m[tid] = m;
    __syncthreads();  // (also: the previous item's sums are read)
    float M = -INFINITY;
    for (int p = 0; p < parts; ++p) M = fmaxf(M, s_m[p * R * CG + cg * R + tid % R]);
    const float f = exp2f(m - (M == -INFINITY ? 0.f : M));
#pragma unroll
    for (int e = 0; e < kCols; ++e) s_part[tid][e] = acc[e] * f;
    s_l[tid] = l * f;
    __syncthreads();
    for (int e = tid; e < R * D; e += kJoinThreads) {
      const int r = e / D, col = e % D, at0 = col / kCols * R + r;  // the thread of part 0
      float L = 0.f, x = 0.f;
      for (int p = 0; p < parts; ++p) {
        L += s_l[p * R * CG + at0];
        x += s_part[p * R * CG + at0][col % kCols];
      }
      if (row0 + r >= jn.rows) continue;
      const int64_t at = out_row(row0 + r);
      x *= a.v_scale / L;
      if constexpr (sizeof(T) == 2) static_cast<__nv_bfloat16*>(a.out)[at * D + col] = __float2bfloat16_rn(x);
      else static_cast<float*>(a.out)[at * D + col] = x;
    }
    if (part == 0 && cg == 0 && row < jn.rows && a.lse) {
      float L = 0.f;
      for (int p = 0; p < parts; ++p) L += s_l[p * R * CG + tid % R];
      a.lse[out_row(row)] = (M + log2f(L)) * kTreeLn2;
    }
  }
}

template <typename T, int D>
cudaError_t launch(const TreeLaunch& a, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * 148);
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
