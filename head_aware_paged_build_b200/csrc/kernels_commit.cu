// Tree commit: the accepted path of each sequence's draft joins a ring plan's
// cache, in place, with the bytes and records that one append per token would
// leave (append_common.cuh).
//
// One CTA per (sequence, kv-head).  A path of n tokens at positions L ... L+n-1
// touches few page records: its targets' blocks, and the blocks of the tokens
// that leave a LOCAL window, positions up to e = L + n - 1 - w.  What the
// appends would do to a record has a closed form, because a ring page's old run
// has left the window before its new run's first token arrives: with run start
// B (a multiple of P), the run's tokens end at hi, and lo moves up behind the
// last of its evicted positions.  So a lane takes a record each, whatever the
// path's length; only pages are taken from the pool in order, by one lane (at
// most one a block).  Then all threads copy the rows, a few loads in flight
// each.  Latency-bound: four dependent reads (head, path, records, rows).  (One
// thread walking the tokens, a warp copying a row at a time: 47 us for 64 tokens
// where this takes 13 us; a path of 4 takes 5.)
#include <type_traits>

#include "append_common.cuh"
#include "kernels.h"

namespace sp {
namespace {

constexpr int kCommitThreads = 256;

// The record after the window moved past position e: the run at abs_start loses its positions up to e.
template <int P>
__device__ __forceinline__ void commit_evict(PageDesc& r, int e_first, int e) {
  const int last = min(e, r.abs_start + P - 1);
  if (last < max(e_first, r.abs_start)) return;
  const int lo = max(slot_lo(r), last - r.abs_start + 1), hi = slot_hi(r);
  r.span = lo < hi ? (make_span(lo, hi) | (r.span & kSpanCausal)) : 0;
}

// 16-bit and fp32 rows as they are; E4M3 pages: the codes an append would write.
template <typename T, int D, int P, bool FP8>
__global__ void __launch_bounds__(kCommitThreads) commit_kernel(CommitLaunch a) {
  // blocks of P positions a path of kMaxTreeNodes tokens can touch
  constexpr int kBlocks = 8;
  static_assert((P - 1 + kMaxTreeNodes - 1) / P + 1 <= kBlocks, "candidate records of a path");
  __shared__ PageDesc recs[3 * kBlocks];
  __shared__ int64_t s_page[kMaxTreeNodes];  // token -> byte offset of its page, -1: a later token takes its slot
  __shared__ int s_slot[kMaxTreeNodes];
  __shared__ int s_node[kMaxTreeNodes];
  __shared__ int s_lead[3 * kBlocks];
  __shared__ int s_n;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int b = blockIdx.x / a.num_kv_heads;  // heads are in (sequence, kv-head) order
  const HeadDesc h = a.heads[blockIdx.x];
  int n = a.path_len[b];
  bool good = n >= 0 && n <= a.max_path;
  if (tid < a.max_path) {
    const int node = a.path[int64_t(b) * a.max_path + tid];
    s_node[tid] = node;
    if (tid < n) good = good && node >= 0 && node < a.n_nodes;
  }
  if (!__syncthreads_and(good)) {  // the same verdict for every head of the sequence
    if (tid == 0) record_error(a.status, kDevBadTree);
    return;
  }
  if (n == 0) return;

  const int L = h.ctx_len;
  const bool local = h.kind == 1;
  const int nsink = local ? (h.sink + P - 1) / P : 0;
  const int R = local ? int((int64_t(h.window) + P - 1) / P + 1) : 1;
  const int b0 = L / P, b1 = (L + n - 1) / P;
  const int e_first = max(h.sink, L - h.window);  // positions e_first ... L + n - 1 - window leave the window
  if (warp == 0) {
    // lanes 0-7: sink and GLOBAL targets; 8-15: ring targets; 16-23: evictions
    const int part = lane / kBlocks, block = (part == 2 ? e_first / P : b0) + lane % kBlocks;
    const int e_path = L + n - 1 - h.window;
    int vp = -1;
    if (part == 0 && block <= b1 && (local ? block < nsink : block < h.n_vpages)) vp = block;
    if (part == 1 && local && block <= b1) vp = nsink + block % R;
    if (part == 2 && local && e_path >= e_first && block <= e_path / P) vp = nsink + block % R;
    const uint32_t same = __match_any_sync(0xffffffffu, vp < 0 ? -1 - lane : vp);
    const bool leads = vp >= 0 && __ffs(same) - 1 == lane;
    PageDesc r{};
    if (leads) r = a.pages[h.vpage_begin + vp];
    if (lane < 3 * kBlocks) recs[lane] = r, s_lead[lane] = __ffs(same) - 1;
    __syncwarp();
    if (lane == 0) {
      // how many tokens fit, and pages for the blocks they reach, in order
      const int room = local ? n : int(min(int64_t(n), int64_t(h.n_vpages) * P - L));
      int done = room;
      for (int at = L; at < L + done;) {
        const bool ring = local && at >= h.sink;
        int end = (at / P + 1) * P;  // of this record's run
        if (local && !ring) end = min(end, h.sink);
        PageDesc* pg = recs + s_lead[(ring ? kBlocks : 0) + at / P - b0];
        const int32_t phys = append_take_page(pg, a.free_pool, a.status);
        if (phys < 0 || phys >= a.pool_pages) {
          if (phys != kNoPage) record_error(a.status, kDevBadPage);  // corrupted table: nothing is written there
          done = at - L;
          break;
        }
        at = end;
      }
      if (done == room && room < n) record_error(a.status, kDevAppendFull);
      s_n = done;
    }
    __syncwarp();
    n = s_n;
    if (leads && n > 0) {
      r = recs[lane];
      const int e = local ? L + n - 1 - h.window : -1;
      const int first = local && vp >= nsink ? max(L, h.sink) : L;               // the record's kind of tokens
      const int last = local && vp < nsink ? min(L + n, h.sink) - 1 : L + n - 1;
      if (local && vp >= nsink) commit_evict<P>(r, e_first, e);
      for (int c = b0; c <= b1; ++c) {
        if (local && vp >= nsink ? nsink + c % R != vp : c != vp) continue;
        const int from = max(first, c * P), to = min(last, c * P + P - 1);
        if (from > to) continue;
        int lo = slot_lo(r);
        if (slot_hi(r) <= lo || r.abs_start != c * P) r.abs_start = c * P, lo = from - c * P;
        r.span = make_span(lo, to - c * P + 1) | (r.span & kSpanCausal);
        if (local && vp >= nsink) commit_evict<P>(r, e_first, e);
      }
      a.pages[h.vpage_begin + vp] = r;
      recs[lane] = r;
    }
    if (lane == 0 && n > 0) {
      a.heads[blockIdx.x].ctx_len = L + n;
      a.heads[blockIdx.x].q_start = L + n - 1;
    }
  }
  __syncthreads();
  n = s_n;
  if (tid < n) {
    const int pos = L + tid;
    const bool ring = local && pos >= h.sink;
    // a ring smaller than the path (16-token pages): a later token takes this one's slot
    const bool gone = ring && int64_t(tid) + int64_t(R) * P < n;
    s_page[tid] = gone ? -1 : int64_t(recs[s_lead[(ring ? kBlocks : 0) + pos / P - b0]].phys) * a.page_bytes;
    s_slot[tid] = pos % P;  // ring slots too: a ring is whole pages
  }
  __syncthreads();
  const int64_t base = int64_t(b) * a.ds_seq + int64_t(h.kv) * a.ds_head;
  const T* kd = static_cast<const T*>(a.k_draft) + base;
  const T* vd = static_cast<const T*>(a.v_draft) + base;
  uint8_t *kpool = static_cast<uint8_t*>(a.kpool), *vpool = static_cast<uint8_t*>(a.vpool);
  constexpr int CR = D * int(sizeof(T)) / 16, VR = D / 2, B = 4;  // 16-byte chunks, value pairs of a row; in flight
  for (int u0 = tid; u0 < n * CR; u0 += kCommitThreads * B) {
    uint4 v[B];
#pragma unroll
    for (int i = 0; i < B; ++i) {
      const int u = u0 + i * kCommitThreads;
      if (u < n * CR) v[i] = reinterpret_cast<const uint4*>(kd + int64_t(s_node[u / CR]) * a.ds_tok)[u % CR];
    }
#pragma unroll
    for (int i = 0; i < B; ++i) {
      const int u = u0 + i * kCommitThreads, t = u / CR, c = u % CR;
      if (u < n * CR && s_page[t] >= 0)
        append_store_k<T, D, P, FP8>(kpool + s_page[t], s_slot[t], c, v[i], a.k_inv);
    }
  }
  using V2 = typename std::conditional<sizeof(T) == 2, uint32_t, uint2>::type;  // two values
  for (int u0 = tid; u0 < n * VR; u0 += kCommitThreads * B) {
    V2 v[B];
#pragma unroll
    for (int i = 0; i < B; ++i) {
      const int u = u0 + i * kCommitThreads;
      if (u < n * VR) v[i] = reinterpret_cast<const V2*>(vd + int64_t(s_node[u / VR]) * a.ds_tok)[u % VR];
    }
#pragma unroll
    for (int i = 0; i < B; ++i) {
      const int u = u0 + i * kCommitThreads, t = u / VR, d = u % VR * 2;
      if (u >= n * VR || s_page[t] < 0) continue;
      const T* x = reinterpret_cast<const T*>(&v[i]);
      append_store_v<T, P, FP8>(vpool + s_page[t], s_slot[t], d, x[0], a.v_inv);
      append_store_v<T, P, FP8>(vpool + s_page[t], s_slot[t], d + 1, x[1], a.v_inv);
    }
  }
}

template <typename T, int D, int P, bool FP8 = false>
cudaError_t launch(const CommitLaunch& a, cudaStream_t s) {
  commit_kernel<T, D, P, FP8><<<a.n_heads, kCommitThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_commit(const CommitLaunch& a, cudaStream_t s) {
  const bool wide = a.D == 128;
  if (a.fp8) return wide ? launch<__nv_bfloat16, 128, 64, true>(a, s) : launch<__nv_bfloat16, 64, 64, true>(a, s);
  if (a.bf16) return wide ? launch<__nv_bfloat16, 128, 64>(a, s) : launch<__nv_bfloat16, 64, 64>(a, s);
  if (a.P == 16) return wide ? launch<float, 128, 16>(a, s) : launch<float, 64, 16>(a, s);
  return wide ? launch<float, 128, 64>(a, s) : launch<float, 64, 64>(a, s);
}

}  // namespace sp
