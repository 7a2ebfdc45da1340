// Reorder: sequence b's cache becomes that of sequence parents[b], in place.
//
// A ring plan's records sit at the same index for the same positions in every
// sequence of one layout, and no token of a page moves, so the copy is page by
// page: one CTA per (kv-head, record index) holds that record of every
// sequence, copies the pages and rewrites the records (each keeps its own
// physical page).  The CTA alone touches them, so the in-place hazards are its
// own: it lists the moves so that a page is written only when nobody still has
// to read it (pages nobody reads first, peeled off round by round; what is
// left are pure cycles, whose first page waits in registers), and every thread
// runs the list on its 16-byte columns, eight loads in flight: of eight moves,
// or of four moves on two columns where the list is short.  Bound by HBM: each
// moved page is read and written once (a page with several readers is re-read
// from cache).  Measured: four of eight 32K sequences 77 us, 4.8 TB/s; sixteen
// rotated 4K sequences 38 us, 5.1 TB/s (84 us with 256 threads and four moves).
#include <type_traits>

#include "append_common.cuh"
#include "kernels.h"

namespace sp {
namespace {

constexpr int kReorderThreads = 512;
constexpr int kSaved = -1;  // move source: the page a cycle saved

struct Move {
  int16_t dst, src;  // sequences; src kSaved: the saved page
  int16_t save;      // >= 0: save this sequence's page before the move
  int16_t pad;
};

__global__ void __launch_bounds__(kReorderThreads) reorder_kernel(const __grid_constant__ ReorderLaunch a) {
  extern __shared__ __align__(16) uint8_t smem[];
  const int B = a.batch;
  PageDesc* rec = reinterpret_cast<PageDesc*>(smem);    // [B] records of this index, as they were
  Move* moves = reinterpret_cast<Move*>(rec + B);       // [B]
  int32_t* phys = reinterpret_cast<int32_t*>(moves + B);  // [B] page of each sequence's record
  int32_t* readers = phys + B;                          // [B] moves that still read this sequence
  int16_t* from = reinterpret_cast<int16_t*>(readers + B);  // [B] source sequence (b: stays)
  uint8_t* copy = reinterpret_cast<uint8_t*>(from + B);     // [B] the page's bytes move too
  uint8_t* listed = copy + B;                               // [B]
  __shared__ int s_kv, s_count;
  const int tid = threadIdx.x;

  for (int kv = tid; kv < a.num_kv_heads; kv += kReorderThreads)
    if (int(blockIdx.x) >= a.rec_begin[kv] && int(blockIdx.x) < a.rec_begin[kv + 1]) s_kv = kv;
  if (tid == 0) s_count = 0;
  for (int b = tid; b < B; b += kReorderThreads) readers[b] = 0;
  __syncthreads();
  const int kv = s_kv, index = int(blockIdx.x) - a.rec_begin[kv];
  int moved = 0;
  for (int b = tid; b < B; b += kReorderThreads) {
    int p = a.parents[b];
    if (p < 0 || p >= B || a.layout[p] != a.layout[b]) {
      if (blockIdx.x == 0) record_error(a.status, kDevBadParent);
      p = b;  // that sequence stays as it is
    }
    const HeadDesc* hd = a.heads + int64_t(b) * a.num_kv_heads + kv;
    if (index >= hd->n_vpages) p = b;  // this layout has no such record
    from[b] = int16_t(p);
    listed[b] = p == b;
    if (p != b) atomicAdd(&readers[p], 1), ++moved;
    rec[b] = index < hd->n_vpages ? a.pages[hd->vpage_begin + index] : PageDesc{kNoPage, 0, 0, 0};
  }
  const int any = __syncthreads_or(moved);
  if (!any) return;

  // Which moves copy bytes; a destination without a page takes one.
  for (int b = tid; b < B; b += kReorderThreads) {
    phys[b] = rec[b].phys;
    copy[b] = 0;
    if (from[b] == b) continue;
    const PageDesc src = rec[from[b]];
    if (slot_hi(src) <= slot_lo(src)) continue;
    if (src.phys < 0 || src.phys >= a.pool_pages) {
      record_error(a.status, kDevBadPage);
      continue;
    }
    bool fresh = false;
    if (phys[b] == kNoPage) {
      PageDesc taken = rec[b];
      phys[b] = append_take_page(&taken, a.free_pool, a.status);
      fresh = true;
    }
    if (phys[b] == kNoPage) continue;  // the spare pool is empty (reported)
    if (phys[b] < 0 || phys[b] >= a.pool_pages) {
      record_error(a.status, kDevBadPage);
      continue;
    }
    // No copy where all that the source's page holds is known to be equal, and this page still holds it (a
    // ring that has gone on further holds other positions, or has let some of these go).
    const PageDesc dst = rec[b];
    const bool held = !fresh && dst.abs_start == src.abs_start && slot_lo(dst) <= slot_lo(src) &&
                      slot_hi(dst) >= slot_hi(src);
    copy[b] = !held || !a.common_len || src.abs_start + slot_hi(src) > a.common_len[b];
  }
  __syncthreads();

  // The list.  A round takes every sequence that nobody still reads.
  int last = 0;
  for (;;) {
    for (int b = tid; b < B; b += kReorderThreads)
      if (!listed[b] && readers[b] == 0) {
        listed[b] = 2;
        moves[atomicAdd(&s_count, 1)] = Move{int16_t(b), from[b], -1, 0};
      }
    __syncthreads();
    const int count = s_count;
    for (int i = last + tid; i < count; i += kReorderThreads) atomicSub(&readers[moves[i].src], 1);
    __syncthreads();
    if (count == last) break;
    last = count;
  }
  // What is left are cycles; the smallest member of each lists it.
  for (int b = tid; b < B; b += kReorderThreads) {
    if (listed[b]) continue;
    int len = 1, low = b;
    for (int x = from[b]; x != b; x = from[x]) ++len, low = min(low, x);
    if (low != b) continue;
    int at = atomicAdd(&s_count, len);
    // b <- f(b) <- ... : each is written after its only reader has read it; b itself is saved
    for (int x = b, i = 0; i < len; x = from[x], ++i)
      moves[at + i] = Move{int16_t(x), int16_t(i == len - 1 ? kSaved : from[x]), int16_t(i == 0 ? b : -1), 0};
  }
  __syncthreads();

  const int count = s_count;
  // M moves at a time, on C of the thread's columns
  auto run = [&](auto m_, auto c_) {
    constexpr int M = decltype(m_)::value, C = decltype(c_)::value;
    const int chunks = int(a.page_bytes / 16);
    for (int e0 = tid; e0 < 2 * chunks; e0 += kReorderThreads * C) {
      auto at = [&](int b, int c) {
        const int e = e0 + c * kReorderThreads;
        uint8_t* pool = e < chunks ? a.kpool : a.vpool;
        return reinterpret_cast<uint4*>(pool + int64_t(phys[b]) * a.page_bytes +
                                        int64_t(e < chunks ? e : e - chunks) * 16);
      };
      auto in = [&](int c) { return e0 + c * kReorderThreads < 2 * chunks; };
      uint4 saved[C];
#pragma unroll
      for (int c = 0; c < C; ++c) saved[c] = make_uint4(0, 0, 0, 0);
      for (int i = 0; i < count; i += M) {
        uint4 v[M][C];
#pragma unroll
        for (int u = 0; u < M; ++u) {
          if (i + u >= count) continue;
          const Move mv = moves[i + u];
          const bool keep = mv.save >= 0 && rec[mv.save].phys >= 0 && rec[mv.save].phys < a.pool_pages;
          const bool read = mv.src != kSaved && copy[mv.dst];
#pragma unroll
          for (int c = 0; c < C; ++c) {
            v[u][c] = saved[c];
            if (keep && in(c)) saved[c] = *at(mv.save, c);
            if (read && in(c)) v[u][c] = *at(mv.src, c);
          }
        }
#pragma unroll
        for (int u = 0; u < M; ++u)
          if (i + u < count && copy[moves[i + u].dst])
#pragma unroll
            for (int c = 0; c < C; ++c)
              if (in(c)) *at(moves[i + u].dst, c) = v[u][c];
      }
    }
  };
  if (count <= 4) run(std::integral_constant<int, 4>{}, std::integral_constant<int, 2>{});
  else run(std::integral_constant<int, 8>{}, std::integral_constant<int, 1>{});
  // Records: the source's positions and span on the sequence's own page.
  for (int b = tid; b < B; b += kReorderThreads) {
    if (from[b] == b) continue;
    const int64_t head = int64_t(b) * a.num_kv_heads + kv;
    PageDesc r = rec[from[b]];
    r.phys = phys[b];
    r.head = rec[b].head;
    if (r.phys == kNoPage) r.span = 0;
    a.pages[a.heads[head].vpage_begin + index] = r;
  }
  // Context lengths: the CTA of the head's first record (nobody else reads them).
  if (index == 0) {
    int32_t* len = readers;
    __syncthreads();
    for (int b = tid; b < B; b += kReorderThreads)
      len[b] = a.heads[int64_t(from[b]) * a.num_kv_heads + kv].ctx_len;
    __syncthreads();
    for (int b = tid; b < B; b += kReorderThreads) {
      if (from[b] == b) continue;
      HeadDesc* hd = a.heads + int64_t(b) * a.num_kv_heads + kv;
      hd->ctx_len = len[b];
      hd->q_start = len[b] - 1;
    }
  }
}

}  // namespace

cudaError_t launch_reorder(const ReorderLaunch& a, cudaStream_t s) {
  const int n = a.rec_begin[a.num_kv_heads];
  if (n == 0) return cudaSuccess;
  const int bytes = (a.batch * (16 + 8 + 4 + 4 + 2 + 1 + 1) + 15) / 16 * 16;
  const cudaError_t e = cudaFuncSetAttribute(reorder_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  reorder_kernel<<<n, kReorderThreads, bytes, s>>>(a);
  return cudaGetLastError();
}

}  // namespace sp
