// Tree commit: the accepted path of each sequence's draft joins a ring plan's
// cache, in place, with the bytes and records that one append per token would
// leave (append_common.cuh makes the record changes of both).
//
// One CTA per (sequence, kv-head).  Warp 0 brings the few page records the
// path can touch into shared memory together (its targets' blocks, and the
// blocks of the tokens that leave a LOCAL window), one thread walks the tokens
// over them, and the rows are copied by all warps, a token each, once every
// token's page and slot are known.  Latency-bound: a step moves a few KB a head.
#include "append_common.cuh"
#include "kernels.h"

namespace sp {
namespace {

constexpr int kCommitWarps = 8;

template <typename T, int D, int P, bool FP8 = false>
__global__ void __launch_bounds__(kCommitWarps * 32) commit_kernel(CommitLaunch a) {
  // blocks of P positions a path of kMaxTreeNodes tokens can touch
  constexpr int kBlocks = 8;
  static_assert((P - 1 + kMaxTreeNodes - 1) / P + 1 <= kBlocks, "candidate records of a path");
  __shared__ PageDesc recs[3 * kBlocks];
  __shared__ int lead[3 * kBlocks];       // candidate -> the candidate that holds its record
  __shared__ int64_t s_page[kMaxTreeNodes];  // token -> byte offset of its page
  __shared__ int s_slot[kMaxTreeNodes];
  __shared__ int s_node[kMaxTreeNodes];
  __shared__ int s_n;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const HeadDesc h = a.heads[blockIdx.x];
  const int n = a.path_len[h.b];
  bool good = n >= 0 && n <= a.max_path;
  if (good && int(threadIdx.x) < n) {
    const int node = a.path[int64_t(h.b) * a.max_path + threadIdx.x];
    s_node[threadIdx.x] = node;
    good = node >= 0 && node < a.n_nodes;
  }
  if (!__syncthreads_and(good)) {  // the same verdict for every head of the sequence
    if (threadIdx.x == 0) record_error(a.status, kDevBadTree);
    return;
  }
  if (n == 0) return;

  const int L = h.ctx_len;
  const bool local = h.kind == 1;
  const int nsink = local ? (h.sink + P - 1) / P : 0;
  const int R = local ? int((int64_t(h.window) + P - 1) / P + 1) : 1;
  const int b0 = L / P, b1 = (L + n - 1) / P;
  const int e0 = max(h.sink, L - h.window) / P, e1 = L + n - 1 - h.window;  // evicted: positions up to e1
  if (warp == 0) {
    // lanes 0-7: sink and GLOBAL targets; 8-15: ring targets; 16-23: evictions
    const int part = lane / kBlocks, block = (part == 2 ? e0 : b0) + lane % kBlocks;
    int vp = -1;
    if (part == 0 && block <= b1 && (local ? block < nsink : block < h.n_vpages)) vp = block;
    if (part == 1 && local && block <= b1) vp = nsink + block % R;
    if (part == 2 && local && e1 >= h.sink && block <= e1 / P) vp = nsink + block % R;
    const uint32_t same = __match_any_sync(0xffffffffu, vp < 0 ? -1 - lane : vp);
    const int leader = __ffs(same) - 1;
    if (lane < 3 * kBlocks) {
      lead[lane] = leader;
      if (vp >= 0 && leader == lane) recs[lane] = a.pages[h.vpage_begin + vp];
    }
    __syncwarp();
    if (lane == 0) {
      HeadDesc now = h;
      int done = 0;
      for (; done < n; ++done) {
        const int pos = L + done;
        now.ctx_len = pos;
        int tvp, slot;
        append_target<P>(now, tvp, slot);
        if (tvp >= h.n_vpages) {  // no reserved page left
          record_error(a.status, kDevAppendFull);
          break;
        }
        PageDesc* pg = recs + lead[(local && pos >= h.sink ? kBlocks : 0) + pos / P - b0];
        const int32_t phys = append_take_page(pg, a.free_pool, a.status);
        if (phys == kNoPage) break;
        if (phys < 0 || phys >= a.pool_pages) {  // corrupted table: nothing is written there
          record_error(a.status, kDevBadPage);
          break;
        }
        s_page[done] = int64_t(phys) * a.page_bytes;
        s_slot[done] = slot;
        append_update_target(pg, pos, slot);
        int evp, eslot, epos;
        append_eviction<P>(now, evp, eslot, epos);
        if (evp >= 0) append_update_eviction(recs + lead[2 * kBlocks + epos / P - e0], epos, eslot);
      }
      s_n = done;
    }
    __syncwarp();
    if (vp >= 0 && leader == lane) a.pages[h.vpage_begin + vp] = recs[lane];
    if (lane == 0 && s_n > 0) {
      a.heads[blockIdx.x].ctx_len = L + s_n;
      a.heads[blockIdx.x].q_start = L + s_n - 1;
    }
  }
  __syncthreads();
  const int done = s_n;
  const T* kd = static_cast<const T*>(a.k_draft) + int64_t(h.b) * a.ds_seq + int64_t(h.kv) * a.ds_head;
  const T* vd = static_cast<const T*>(a.v_draft) + int64_t(h.b) * a.ds_seq + int64_t(h.kv) * a.ds_head;
  for (int i = warp; i < done; i += kCommitWarps) {
    // a ring smaller than the path (16-token pages): a later token takes this one's slot
    if (local && L + i >= h.sink && int64_t(i) + int64_t(R) * P < done) continue;
    const int64_t from = int64_t(s_node[i]) * a.ds_tok;
    append_write_token<T, D, P, FP8>(kd + from, vd + from, static_cast<uint8_t*>(a.kpool) + s_page[i],
                                     static_cast<uint8_t*>(a.vpool) + s_page[i], s_slot[i], a.k_inv, a.v_inv, lane,
                                     32);
  }
}

}  // namespace

cudaError_t launch_commit(const CommitLaunch& a, cudaStream_t s) {
  constexpr int kThreads = kCommitWarps * 32;
  if (a.fp8) {
    if (a.D == 128) commit_kernel<__nv_bfloat16, 128, 64, true><<<a.n_heads, kThreads, 0, s>>>(a);
    else commit_kernel<__nv_bfloat16, 64, 64, true><<<a.n_heads, kThreads, 0, s>>>(a);
  } else if (a.bf16) {
    if (a.D == 128) commit_kernel<__nv_bfloat16, 128, 64><<<a.n_heads, kThreads, 0, s>>>(a);
    else commit_kernel<__nv_bfloat16, 64, 64><<<a.n_heads, kThreads, 0, s>>>(a);
  } else if (a.P == 16) {
    if (a.D == 128) commit_kernel<float, 128, 16><<<a.n_heads, kThreads, 0, s>>>(a);
    else commit_kernel<float, 64, 16><<<a.n_heads, kThreads, 0, s>>>(a);
  } else {
    if (a.D == 128) commit_kernel<float, 128, 64><<<a.n_heads, kThreads, 0, s>>>(a);
    else commit_kernel<float, 64, 64><<<a.n_heads, kThreads, 0, s>>>(a);
  }
  return cudaGetLastError();
}

}  // namespace sp
