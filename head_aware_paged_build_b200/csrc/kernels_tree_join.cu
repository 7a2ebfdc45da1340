// Joining the pieces of row groups that tree attention split over CTAs.
//
// With m_i, l_i, acc_i the running maximum (log2 domain), sum and unnormalised
// output of piece i:  M = max m_i,  O = sum 2^(m_i - M) acc_i / sum 2^(m_i - M) l_i,
// in an order that the pieces' numbers fix, so the same inputs give the same bits.
//
// A programmatic dependent launch: its blocks are placed while the attention's
// last CTAs run and wait for that grid on the device.  (The last CTA of a row
// group joining it instead was 3 to 10 times slower on the 8K and 32K layers:
// one SM reads what a dozen wrote, 64 KB for each piece of 128 rows.)  Every
// block lists the split groups (the CTA a group starts in left its description)
// and takes its share of items.  A thread holds a row's 16 columns over a part
// of the pieces; a group of many pieces is divided into 4 or 16 parts, which
// meet in shared memory.  Bound by L2 latency: a thread asks for kBatch pieces
// (maximum, sum and columns) at once and rescales once a batch.
#include "kernels.h"
#include "tree_common.cuh"

namespace sp {
namespace {

constexpr int kJoinThreads = 256;
constexpr int kBatch = 4;
constexpr int kCols = 16;

// Parts a group's pieces are divided into: one while a batch holds them.
__device__ __forceinline__ int join_parts(int n_pieces) {
  return n_pieces <= kBatch ? 1 : n_pieces <= 4 * kBatch ? 4 : 16;
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
    const TreeJoin& jn = s_join[lo];
    const int parts = join_parts(jn.n_pieces), R = R1 / parts;
    const int row0 = (item - (lo ? s_end[lo - 1] : 0)) * R;
    // thread = (part, column group, row of the item)
    const int row = row0 + tid % R, cg = tid / R % CG, part = tid / (R * CG);
    float m = -INFINITY, l = 0.f, acc[kCols];
#pragma unroll
    for (int e = 0; e < kCols; ++e) acc[e] = 0.f;
    if (row < jn.rows) {
      for (int i0 = part; i0 < jn.n_pieces; i0 += kBatch * parts) {
        float2 ml[kBatch];
        float4 x[kBatch][kCols / 4];
        float top = m;
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
          const int i = i0 + u * parts;
          ml[u] = make_float2(-INFINITY, 0.f);
          if (i >= jn.n_pieces) continue;
          const float* s = a.partial + int64_t(i == 0 ? jn.first_slot : 2 * (lo + i)) * stride;
          ml[u] = __ldcg(reinterpret_cast<const float2*>(s + rows_max * D + 2 * row));
#pragma unroll
          for (int c = 0; c < kCols / 4; ++c)
            x[u][c] = __ldcg(reinterpret_cast<const float4*>(s + tree_acc_at(row, cg * kCols + 4 * c, rows_max)));
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) top = fmaxf(top, ml[u].x);
        const float base = top == -INFINITY ? 0.f : top, f0 = exp2f(m - base);
        m = top;
        l *= f0;
#pragma unroll
        for (int e = 0; e < kCols; ++e) acc[e] *= f0;
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
          if (i0 + u * parts >= jn.n_pieces) continue;
          const float f = exp2f(ml[u].x - base);
          l += f * ml[u].y;
#pragma unroll
          for (int c = 0; c < kCols / 4; ++c) {
            acc[4 * c] += f * x[u][c].x, acc[4 * c + 1] += f * x[u][c].y;
            acc[4 * c + 2] += f * x[u][c].z, acc[4 * c + 3] += f * x[u][c].w;
          }
        }
      }
    }
    auto out_row = [&](int r) {
      return (int64_t(jn.b) * a.T + jn.node0 + r / a.group) * a.num_q_heads + jn.kv * a.group + r % a.group;
    };
    if (parts == 1) {
      if (row >= jn.rows) continue;
      const int64_t at = out_row(row);
      const float inv = a.v_scale / l;
      T* dst = static_cast<T*>(a.out) + at * D + cg * kCols;
      if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int e = 0; e < kCols; e += 8)
          reinterpret_cast<uint4*>(dst)[e / 8] = make_uint4(
              pack_bf16x2(acc[e] * inv, acc[e + 1] * inv), pack_bf16x2(acc[e + 2] * inv, acc[e + 3] * inv),
              pack_bf16x2(acc[e + 4] * inv, acc[e + 5] * inv), pack_bf16x2(acc[e + 6] * inv, acc[e + 7] * inv));
      } else {
#pragma unroll
        for (int e = 0; e < kCols; e += 4)
          reinterpret_cast<float4*>(dst)[e / 4] =
              make_float4(acc[e] * inv, acc[e + 1] * inv, acc[e + 2] * inv, acc[e + 3] * inv);
      }
      if (cg == 0 && a.lse) a.lse[at] = (m + log2f(l)) * kTreeLn2;
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
