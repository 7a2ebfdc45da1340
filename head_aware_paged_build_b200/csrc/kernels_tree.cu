// Attention of a drafted tree over the paged cache: the mma.sync kernel
// (up to 32 rows a kv-head) and the fp32 kernel.
//
// mma.sync kernel: a producer warp walks the CTA's pieces, hands each to the
// others a slot ahead (its table entries, parents and Q rows) and streams its
// pages into a ring of shared-memory stages with bulk copies, as decode does;
// one or two more warps write the draft's rows as one more page of the same
// layout (E4M3 pages: quantised as an append would, so a node sees exactly the
// codes the cache will hold once the node is committed).  WR x 4 consumer
// warps: warp (wr, wt) holds rows 16 wr .. 16 wr + 15 of the row group and
// takes tokens 16 wt ... of each page: S = Q K^T, online softmax with a lazy
// rescale, O += P V on m16n8k16 fragments.  Scores, sums and O are
// fp32; P is rounded to the type of the pages' operands (bf16, or f16 over
// widened E4M3 codes, lifted: kWeightLift), V's own type, while the sums use the
// unrounded weights.
#include <algorithm>

#include "tree_common.cuh"

namespace sp {
namespace {

constexpr float kLazyLog2 = 8.f;

template <int D, bool FP8, int WR>
struct TreeMma {
  static constexpr int WT = 4;  // warps over a page's tokens
  static constexpr int kConsumers = WR * WT;
  // 16-row form: two CTAs an SM, whose 12 warps may have 168 registers a thread; a 14th would cost 40 of them, so
  // the producer writes the draft's K
  static constexpr int kDraftWarps = WR > 1 ? 2 : 1;
  static constexpr int kThreads = (kConsumers + 1 + kDraftWarps) * 32;
  static constexpr int kRows = 16 * WR;
  static constexpr int kPageBytes = 64 * D * (FP8 ? 1 : 2);
  static constexpr int kRing = (WR > 1 ? 128 : 64) * 1024 / (2 * kPageBytes);
  static constexpr int kStages = kRing < 8 ? kRing : 8;
  static constexpr int kPitch = D + 8;
  static constexpr int kQPitch = D * 2 + 16;  // bytes; the 8 rows of a fragment load fall on distinct banks
  static constexpr int kMergeOff = kStages * 2 * kPageBytes;
  static constexpr int kMlOff = kMergeOff + (WT - 1) * kRows * kPitch * 4;
  static constexpr int kQOff = kMlOff + (WT - 1) * kRows * 2 * 4;
  static constexpr int kDescOff = kQOff + 2 * kRows * kQPitch;
  static constexpr int kBarOff = kDescOff + kStages * 16;
  static constexpr int kScanOff = kBarOff + (2 * kStages + 6) * 8;
  static constexpr int kInfoOff = kScanOff + ((kThreads / 32 + 2) * 8 + 15) / 16 * 16;
  using Split = TreeSplit<7, 2>;
  using Info = TreePieceInfo<typename Split::Piece>;
  static_assert(kMlOff % 8 == 0 && kQOff % 16 == 0 && kDescOff % 16 == 0 && kBarOff % 8 == 0 && kScanOff % 8 == 0 &&
                    kInfoOff % alignof(Info) == 0,
                "alignment of the shared-memory parts");
  static_assert(alignof(TreeJoinsHere) <= alignof(Info), "the list behind the pieces");
  static constexpr int kBytes = kInfoOff + 2 * int(sizeof(Info)) + int(sizeof(TreeJoinsHere));
};

// HERE: the CTAs join split groups themselves (tree_joins_here).  A form of its
// own: the join's registers cost the page loop of long calls 5 to 9 %.
template <int D, bool FP8, int WR, bool HERE>
__global__ void __launch_bounds__(TreeMma<D, FP8, WR>::kThreads, WR > 1 ? 1 : 2) tree_mma_kernel(TreeLaunch a) {
  using C = TreeMma<D, FP8, WR>;
  using Split = typename C::Split;
  using Info = typename C::Info;
  constexpr int P = 64, PB = C::kPageBytes, NST = C::kStages, NC = C::kConsumers, ND = C::kDraftWarps;
  constexpr int KSTEPS = D / 16, NT = D / 8, WT = C::WT;
  constexpr uint32_t kAll = 0xffffffffu;
  constexpr DraftForm FORM = FP8 ? kDraftE4m3 : kDraftBf16;
  constexpr float kLift = FP8 ? kWeightLift : 0.f;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* stage = smem;
  float* mbuf = reinterpret_cast<float*>(smem + C::kMergeOff);
  float* mlbuf = reinterpret_cast<float*>(smem + C::kMlOff);
  uint8_t* qbuf = smem + C::kQOff;
  PageDesc* sdesc = reinterpret_cast<PageDesc*>(smem + C::kDescOff);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kBarOff);
  uint64_t *empty = full + NST, *piece_full = empty + NST, *piece_free = piece_full + 2, *draft_go = piece_free + 2;
  int64_t* scratch = reinterpret_cast<int64_t*>(smem + C::kScanOff);
  Info* info = reinterpret_cast<Info*>(smem + C::kInfoOff);
  TreeJoinsHere* here = reinterpret_cast<TreeJoinsHere*>(info + 2);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    here->n = 0;
    for (int s = 0; s < NST; ++s) {
      mbar_init(&full[s], 1 + ND);  // the producer and the draft's writers (it arrives for them on cached pages)
      mbar_init(&empty[s], NC);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&piece_full[s], 1);
      mbar_init(&piece_free[s], NC + ND);
      mbar_init(&draft_go[s], 1);
    }
    fence_barrier_init();
  }
  Split split;
  if (!split.template init<C::kThreads>(a, scratch)) return;  // its barriers order the mbarriers' init too
  const int G = a.group;
  int k = 0;  // pages streamed so far

  if (warp == NC) {
    // ------------------------------ producer ------------------------------
    typename Split::Walk walk = split.walk();
    typename Split::Piece pc;
    const uint8_t* kpool = static_cast<const uint8_t*>(a.kpool);
    const uint8_t* vpool = static_cast<const uint8_t*>(a.vpool);
    bool ok = true;
    int pi = 0;
    auto piece_slot = [&] {  // the next piece's slot, once it is free
      const int ps = pi & 1;
      ok = pi < 2 || __shfl_sync(kAll, int(lane == 0 && mbar_wait(&piece_free[ps], ((pi >> 1) - 1) & 1)), 0);
      if (!ok && lane == 0) record_error(a.status, kDevTimeoutEmpty);
      return ps;
    };
    while (ok && split.next(a, walk, pc)) {
      const PageDesc* rec = a.pages + pc.hd.vpage_begin;
      int4 mine = make_int4(0, 0, 0, 0);
      if (pc.p0 + lane < pc.live) mine = *reinterpret_cast<const int4*>(rec + pc.p0 + lane);
      const int ps = piece_slot();
      if (!ok) break;
      tree_publish(a, pc, k, lane, info[ps]);
      const int rows = pc.nodes * G;
      if (lane == 0) {
        mbar_arrive_expect_tx(&piece_full[ps], rows * D * 2);
        if (pc.p1 <= pc.live) mbar_arrive(&draft_go[ps]);  // no draft page in this piece
      }
      __syncwarp();
      const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q);
      for (int r = lane; r < rows; r += 32)
        bulk_g2s(qbuf + (ps * C::kRows + r) * C::kQPitch,
                 q + ((int64_t(pc.hd.b) * a.T + pc.node0 + r / G) * a.num_q_heads + pc.hd.kv * G + r % G) * D, D * 2,
                 &piece_full[ps]);
      ++pi;
      for (int p = pc.p0; p < pc.p1; ++p, ++k) {
        const int i = (p - pc.p0) & 31;
        if (i == 0 && p > pc.p0 && p + lane < pc.live) mine = *reinterpret_cast<const int4*>(rec + p + lane);
        PageDesc pg;
        pg.phys = __shfl_sync(kAll, mine.x, i);
        pg.abs_start = __shfl_sync(kAll, mine.y, i);
        pg.span = __shfl_sync(kAll, mine.z, i);
        pg.head = pc.head;
        const int s = k % NST;
        ok = k < NST || __shfl_sync(kAll, int(lane == 0 && mbar_wait(&empty[s], ((k / NST) & 1) ^ 1)), 0);
        if (!ok) {
          if (lane == 0) record_error(a.status, kDevTimeoutEmpty);
          break;
        }
        uint8_t* kd = stage + s * 2 * PB;
        if (p >= pc.live) {  // the draft's page: its writers arrive when they have filled it
          if (lane == 0) {
            sdesc[s] = PageDesc{kDraftPage, 0, 0, pc.head};
            mbar_arrive(&draft_go[ps]);  // the stage is free
          }
          if constexpr (ND == 1) {
            tree_draft_k<D, FORM>(a, pc.hd, pc.n, kd, lane);
            fence_proxy_async_smem();  // before a later bulk copy into this stage
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&full[s]);
          continue;
        }
        if (lane == 0) {
          if (slot_hi(pg) > slot_lo(pg) && (pg.phys < 0 || pg.phys >= a.pool_pages)) {
            record_error(a.status, kDevBadPage);  // corrupted table: report, read nothing
            pg.span = 0;
          }
          sdesc[s] = pg;
          if (slot_hi(pg) > slot_lo(pg)) {
            mbar_arrive_expect_tx(&full[s], 2 * PB);
            bulk_g2s(kd, kpool + int64_t(pg.phys) * a.page_bytes, PB, &full[s]);
            bulk_g2s(kd + PB, vpool + int64_t(pg.phys) * a.page_bytes, PB, &full[s]);
          } else {
            mbar_arrive(&full[s]);  // an empty record: nothing to read
          }
#pragma unroll
          for (int w = 0; w < ND; ++w) mbar_arrive(&full[s]);
        }
      }
    }
    // never leave with copies in flight
    const int last = pi;
    if (ok) {
      const int ps = piece_slot();
      if (ok && lane == 0) {
        info[ps].pc.head = -1;
        mbar_arrive(&piece_full[ps]);
      }
    }
    if (lane == 0) {
      // Q rows: the end mark took the slot of the last piece but one, after its readers
      for (int j = max(0, last - (ok ? 1 : 2)); j < last; ++j)
        if (!mbar_wait(&piece_full[j & 1], (j >> 1) & 1)) break;
      for (int j = (k > NST ? k - NST : 0); j < k; ++j)
        if (!mbar_wait(&full[j % NST], (j / NST) & 1)) break;
    }
    return;
  }

  if (warp > NC) {
    // ------------------------------ draft page ------------------------------
    const bool does_k = ND == 2 && warp == NC + 1, does_v = warp == NC + ND;
    for (int pi = 0;; ++pi) {
      const int ps = pi & 1;
      if (!__all_sync(kAll, mbar_wait(&piece_full[ps], (pi >> 1) & 1))) break;
      const Info& in = info[ps];
      if (in.pc.head < 0) break;
      if (in.pc.p1 > in.pc.live) {
        const int kd = in.stage0 + in.pc.p1 - 1 - in.pc.p0, s = kd % NST;
        // the producer has seen the stage free (a wait on the stage's own barrier could be phases ahead of it)
        if (!__all_sync(kAll, mbar_wait(&draft_go[ps], (pi >> 1) & 1))) break;
        uint8_t* page = stage + s * 2 * PB;
        if (does_k) tree_draft_k<D, FORM>(a, in.pc.hd, in.pc.n, page, lane);
        if (does_v) tree_draft_v<D, FORM>(a, in.pc.hd, in.pc.n, page + PB, lane);
        fence_proxy_async_smem();  // before a later bulk copy into this stage
        __syncwarp();
        if (lane == 0) mbar_arrive(&full[s]);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&piece_free[ps]);
    }
    return;
  }

  // ------------------------------ consumers ------------------------------
  auto bar = [] { asm volatile("bar.sync 1, %0;" ::"n"(NC * 32) : "memory"); };
  const int wr = warp / WT, wt = warp % WT;
  const int grp = lane >> 2, tq = lane & 3, mi = lane >> 3, rr = lane & 7;
  const int row[2] = {wr * 16 + grp, wr * 16 + grp + 8};
  bool ok = true;
  for (int pi = 0;; ++pi) {
    const int ps = pi & 1;
    // all consumers go on, or none (a barrier waits for every one of them); also: the previous piece's buffers are read
    const bool got = ok && __all_sync(kAll, mbar_wait(&piece_full[ps], (pi >> 1) & 1));
    if (ok && !got) record_error(a.status, kDevTimeoutFull);
    if (!bar_red_and(1, NC * 32, got)) break;
    const Info& in = info[ps];
    if (in.pc.head < 0) break;
    const typename Split::Piece pc = in.pc;
    uint64_t nodes[2];
    tree_ancestors(in.up[lane], in.up[lane + 32], lane, nodes);
    const int rows = pc.nodes * G;
    const int p_last = pc.hd.ctx_len + pc.n - 1;
    int pos[2] = {0, 0};
    uint64_t anc[2] = {0, 0};
    uint32_t qa[KSTEPS][4];
    const uint8_t* qrow[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const uint64_t mask = tree_mask_of(nodes, min(pc.node0 + row[x] / G, kMaxTreeNodes - 1));
      if (row[x] < rows) {
        anc[x] = tree_visible(mask, pc.hd);
        pos[x] = pc.hd.ctx_len + __popcll(mask) - 1;
      }
      qrow[x] = qbuf + (ps * C::kRows + row[x]) * C::kQPitch;  // rows behind the last hold anything: never written out
    }
    if constexpr (FP8) {  // k-steps 2j, 2j+1 cover dims 32j .. 32j+31 in the K loads' order
#pragma unroll
      for (int j = 0; j < D / 32; ++j) {
        const uint4 x0 = *reinterpret_cast<const uint4*>(qrow[0] + (j * 32 + tq * 8) * 2);
        const uint4 x1 = *reinterpret_cast<const uint4*>(qrow[1] + (j * 32 + tq * 8) * 2);
        qa[2 * j][0] = bf16x2_to_f16x2(x0.x), qa[2 * j][2] = bf16x2_to_f16x2(x0.y);
        qa[2 * j + 1][0] = bf16x2_to_f16x2(x0.z), qa[2 * j + 1][2] = bf16x2_to_f16x2(x0.w);
        qa[2 * j][1] = bf16x2_to_f16x2(x1.x), qa[2 * j][3] = bf16x2_to_f16x2(x1.y);
        qa[2 * j + 1][1] = bf16x2_to_f16x2(x1.z), qa[2 * j + 1][3] = bf16x2_to_f16x2(x1.w);
      }
    } else {
#pragma unroll
      for (int kk = 0; kk < KSTEPS; ++kk)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          qa[kk][x] = *reinterpret_cast<const uint32_t*>(qrow[x] + (kk * 16 + tq * 2) * 2);
          qa[kk][x + 2] = *reinterpret_cast<const uint32_t*>(qrow[x] + (kk * 16 + tq * 2 + 8) * 2);
        }
    }
    float o[NT][4];
#pragma unroll
    for (int j = 0; j < NT; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

    for (int p = pc.p0; p < pc.p1; ++p, ++k) {
      const int s = k % NST;
      // the wait's outcome is voted: ldmatrix and mma.sync need the whole warp
      if (ok && !__all_sync(0xffffffffu, mbar_wait(&full[s], (k / NST) & 1))) {
        record_error(a.status, kDevTimeoutFull);
        ok = false;
      }
      const PageDesc pg = sdesc[s];
      const bool draft = pg.phys == kDraftPage;
      const bool all = !draft && tree_page_full(pg, pc.hd, p_last);
      uint64_t vis[2];
#pragma unroll
      for (int x = 0; x < 2; ++x)
        vis[x] = row[x] >= rows ? 0 : all ? ~uint64_t(0) : draft ? anc[x] : tree_page_mask(pg, pc.hd, pos[x]);
      const uint32_t kst = smem_u32(stage + s * 2 * PB), vst = kst + PB;
      const uint8_t* kp8 = stage + s * 2 * PB;
      const int tok0 = wt * 16;
      const uint32_t v0 = uint32_t(vis[0] >> tok0) & 0xffffu, v1 = uint32_t(vis[1] >> tok0) & 0xffffu;
      if (ok && __any_sync(0xffffffffu, v0 | v1)) {
        float sc[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
        if constexpr (FP8) {
#pragma unroll
          for (int j = 0; j < D / 32; ++j)
#pragma unroll
            for (int n = 0; n < 2; ++n) {
              const uint2 u =
                  *reinterpret_cast<const uint2*>(kp8 + fp8_kpage_offset(tok0 + n * 8 + grp, j * 32 + tq * 8, D));
              mma_f16_16816(sc[n], qa[2 * j], e4m3x2_to_f16x2(uint16_t(u.x)), e4m3x2_to_f16x2(uint16_t(u.x >> 16)));
              mma_f16_16816(sc[n], qa[2 * j + 1], e4m3x2_to_f16x2(uint16_t(u.y)),
                            e4m3x2_to_f16x2(uint16_t(u.y >> 16)));
            }
        } else {
          // all fragments first (a product waits for its own load, and nothing passes it), and two sums a score,
          // for chains of half the length
          const int ktok = tok0 + (mi >> 1) * 8 + rr;
          uint32_t kb[KSTEPS][4];
#pragma unroll
          for (int kk = 0; kk < KSTEPS; ++kk)
            ldmatrix_x4(kb[kk][0], kb[kk][1], kb[kk][2], kb[kk][3],
                        kst + uint32_t(kpage_chunk_offset_bf16(ktok, 2 * kk + (mi & 1), P)));
          float sd[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
          for (int kk = 0; kk < KSTEPS; kk += 2) {
            mma_bf16_16816(sc[0], qa[kk], kb[kk][0], kb[kk][1]);
            mma_bf16_16816(sc[1], qa[kk], kb[kk][2], kb[kk][3]);
            mma_bf16_16816(sd[0], qa[kk + 1], kb[kk + 1][0], kb[kk + 1][1]);
            mma_bf16_16816(sd[1], qa[kk + 1], kb[kk + 1][2], kb[kk + 1][3]);
          }
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) sc[n][e] += sd[n][e];
        }
        // V's first fragments come while the weights are made
        constexpr int VB = 4;
        uint32_t vb[VB][4];
        const int vc = (tok0 >> 3) + (mi & 1);
        auto load_v = [&](int j0) {
#pragma unroll
          for (int j = 0; j < VB; ++j)
            ldmatrix_x4(vb[j][0], vb[j][1], vb[j][2], vb[j][3],
                        vst + uint32_t(vpage_chunk_offset_bf16((2 * (j0 + j) + (mi >> 1)) * 8 + rr, vc)));
        };
        if constexpr (!FP8) load_v(0);
        float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const bool see = ((e < 2 ? v0 : v1) >> (n * 8 + tq * 2 + (e & 1))) & 1;
            sc[n][e] = see ? sc[n][e] * a.scale_log2 : -INFINITY;
            mx[e >> 1] = fmaxf(mx[e >> 1], sc[n][e]);
          }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          mx[x] = fmaxf(mx[x], __shfl_xor_sync(0xffffffffu, mx[x], 1));
          mx[x] = fmaxf(mx[x], __shfl_xor_sync(0xffffffffu, mx[x], 2));
        }
        if (__any_sync(0xffffffffu, mx[0] > m[0] + kLazyLog2 || mx[1] > m[1] + kLazyLog2)) {
          float al[2];
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const float mn = mx[x] > m[x] + kLazyLog2 ? mx[x] : m[x];
            al[x] = mn == m[x] ? 1.f : fast_exp2(m[x] - mn);
            l[x] *= al[x], m[x] = mn;
          }
#pragma unroll
          for (int j = 0; j < NT; ++j) o[j][0] *= al[0], o[j][1] *= al[0], o[j][2] *= al[1], o[j][3] *= al[1];
        }
        const float b0 = m[0] == -INFINITY ? 0.f : m[0] - kLift, b1 = m[1] == -INFINITY ? 0.f : m[1] - kLift;
        float pr[2][4];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          pr[n][0] = fast_exp2(sc[n][0] - b0), pr[n][1] = fast_exp2(sc[n][1] - b0);
          pr[n][2] = fast_exp2(sc[n][2] - b1), pr[n][3] = fast_exp2(sc[n][3] - b1);
        }
        l[0] += (pr[0][0] + pr[0][1]) + (pr[1][0] + pr[1][1]);
        l[1] += (pr[0][2] + pr[0][3]) + (pr[1][2] + pr[1][3]);
        uint32_t pa[4];
        if constexpr (FP8) {
#pragma unroll
          for (int n = 0; n < 2; ++n)
            pa[2 * n] = pack_f16x2(pr[n][0], pr[n][1]), pa[2 * n + 1] = pack_f16x2(pr[n][2], pr[n][3]);
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            const uint32_t u =
                *reinterpret_cast<const uint32_t*>(kp8 + PB + fp8_vpage_offset(j * 8 + grp, tok0 + tq * 4));
            mma_f16_16816(o[j], pa, e4m3x2_to_f16x2(uint16_t(u)), e4m3x2_to_f16x2(uint16_t(u >> 16)));
          }
        } else {
#pragma unroll
          for (int n = 0; n < 2; ++n)
            pa[2 * n] = pack_bf16x2(pr[n][0], pr[n][1]), pa[2 * n + 1] = pack_bf16x2(pr[n][2], pr[n][3]);
#pragma unroll
          for (int j0 = 0; j0 < NT / 2; j0 += VB) {
            if (j0) load_v(j0);
#pragma unroll
            for (int j = 0; j < VB; ++j) {
              mma_bf16_16816(o[2 * (j0 + j)], pa, vb[j][0], vb[j][1]);
              mma_bf16_16816(o[2 * (j0 + j) + 1], pa, vb[j][2], vb[j][3]);
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[s]);
    }

    // ---- the row's WT warps join, in warp order ----
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      l[x] += __shfl_xor_sync(0xffffffffu, l[x], 1);
      l[x] += __shfl_xor_sync(0xffffffffu, l[x], 2);
      m[x] -= kLift;  // what l and o are relative to
    }
    if (wt > 0) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int at = (wt - 1) * C::kRows + row[x];
        if (tq == 0) mlbuf[at * 2] = m[x], mlbuf[at * 2 + 1] = l[x];
#pragma unroll
        for (int j = 0; j < NT; ++j)
          *reinterpret_cast<float2*>(mbuf + at * C::kPitch + j * 8 + tq * 2) =
              make_float2(o[j][2 * x], o[j][2 * x + 1]);
      }
    }
    bar();
    if (wt == 0) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        float M = m[x], f[WT];
#pragma unroll
        for (int w = 1; w < WT; ++w) M = fmaxf(M, mlbuf[((w - 1) * C::kRows + row[x]) * 2]);
        const float base = M == -INFINITY ? 0.f : M;
        f[0] = fast_exp2(m[x] - base);
        l[x] *= f[0];
#pragma unroll
        for (int w = 1; w < WT; ++w) {
          const float* ml = mlbuf + ((w - 1) * C::kRows + row[x]) * 2;
          f[w] = fast_exp2(ml[0] - base);
          l[x] += f[w] * ml[1];
        }
        m[x] = M;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          o[j][2 * x] *= f[0], o[j][2 * x + 1] *= f[0];
#pragma unroll
          for (int w = 1; w < WT; ++w) {
            const float2 v = *reinterpret_cast<const float2*>(
                mbuf + ((w - 1) * C::kRows + row[x]) * C::kPitch + j * 8 + tq * 2);
            o[j][2 * x] += f[w] * v.x, o[j][2 * x + 1] += f[w] * v.y;
          }
        }
      }
    }
    // ---- whole row group: the result; else a partial ----
    if (wt == 0) {
      const int rows_max = a.nodes_per_group * G;
      float* slot = a.partial + int64_t(pc.slot) * tree_slot_floats(a);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        if (row[x] >= rows) continue;
        if (pc.n_pieces == 1) {
          const float inv = a.v_scale / l[x];
          const int64_t at = (int64_t(pc.hd.b) * a.T + pc.node0 + row[x] / G) * a.num_q_heads + pc.hd.kv * G +
                             row[x] % G;
          uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(a.out) + at * D);
#pragma unroll
          for (int j = 0; j < NT; ++j) dst[j * 4 + tq] = pack_bf16x2(o[j][2 * x] * inv, o[j][2 * x + 1] * inv);
          if (tq == 0 && a.lse) a.lse[at] = (m[x] + log2f(l[x])) * kTreeLn2;
        } else {
#pragma unroll
          for (int j = 0; j < NT; ++j)
            *reinterpret_cast<float2*>(slot + tree_acc_at(row[x], j * 8 + tq * 2, rows_max)) =
                make_float2(o[j][2 * x], o[j][2 * x + 1]);
          if (tq == 0)
            *reinterpret_cast<float2*>(slot + rows_max * D + 2 * row[x]) = make_float2(m[x], l[x]);
        }
      }
    }
    if constexpr (!HERE) {
      if (threadIdx.x == 0) tree_note_join(a, pc);
    } else if (pc.n_pieces > 1) {
      __threadfence();
      bar();
      if (threadIdx.x == 0) tree_take_ticket(a, pc, here);
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&piece_free[ps]);
  }
  // (the loop ended behind a barrier: every thread sees the list)
  if constexpr (HERE) tree_join_here<__nv_bfloat16, D>(a, *here, threadIdx.x, NC * 32);
}

// ---------------------------------------------------------------------------
// fp32 pages: SIMT, FP32 FMA only.  At most 16 rows a group.  Pages are copied
// asynchronously into two stages, rows padded by 16 bytes so that the 128-bit
// reads of eight lanes (tokens of K, dimensions of V) fall on distinct banks;
// each K (V) read serves all the rows a thread works for.
// ---------------------------------------------------------------------------
constexpr int kF32Threads = 128;
constexpr int kF32Rows = 16;

template <int D, int P>
struct TreeF32 {
  static constexpr int kKPitch = D + 4, kVPitch = P + 4;  // floats
  static constexpr int kStage = P * kKPitch + D * kVPitch;
  static constexpr int kBytes = (2 * kStage + kF32Rows * kKPitch + kF32Rows * kVPitch + 3 * kF32Rows) * 4;
};

__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ float dot4(float4 a, float4 b, float s) {
  return fmaf(a.w, b.w, fmaf(a.z, b.z, fmaf(a.y, b.y, fmaf(a.x, b.x, s))));
}

template <int D, int P, bool HERE>
__global__ void __launch_bounds__(kF32Threads) tree_f32_kernel(TreeLaunch a) {
  using Split = TreeSplit<4, 2>;
  using C = TreeF32<D, P>;
  constexpr int KP = C::kKPitch, VP = C::kVPitch;
  constexpr int SR = kF32Rows * P / kF32Threads;  // rows a thread scores (of one token)
  constexpr int OR = kF32Rows * D / kF32Threads;  // rows a thread accumulates (of one dimension)
  extern __shared__ __align__(1024) uint8_t smem[];
  float* stage = reinterpret_cast<float*>(smem);  // 2 x (K [P][KP], V [D][VP])
  float* qs = stage + 2 * C::kStage;              // [rows][KP]
  float* sc = qs + kF32Rows * KP;                 // [rows][VP]
  float* st = sc + kF32Rows * VP;                 // alpha, m, l of each row
  __shared__ int64_t scratch[kF32Threads / 32 + 2];
  __shared__ int pos[kF32Rows];
  __shared__ uint64_t anc[kF32Rows];
  __shared__ TreeJoinsHere here;
  const int tid = threadIdx.x, G = a.group;
  if (tid == 0) here.n = 0;
  Split split;
  if (!split.template init<kF32Threads>(a, scratch)) return;
  typename Split::Walk walk = split.walk();
  typename Split::Piece pc;
  while (split.next(a, walk, pc)) {
    const int rows = pc.nodes * G, rows_max = a.nodes_per_group * G;
    const int64_t q0 = int64_t(pc.hd.b) * a.T + pc.node0;
    auto at_row = [&](int r) { return (q0 + r / G) * a.num_q_heads + pc.hd.kv * G + r % G; };
    // a page's record (span 0: nothing to see there), and its copy into a stage
    auto record = [&](int p) {
      PageDesc pg{};
      if (p >= pc.live) return pg;
      pg = a.pages[pc.hd.vpage_begin + p];
      if (slot_hi(pg) > slot_lo(pg) && (pg.phys < 0 || pg.phys >= a.pool_pages)) {
        if (tid == 0) record_error(a.status, kDevBadPage);
        pg.span = 0;
      }
      return pg;
    };
    auto load = [&](int p) {
      float* kp = stage + (p - pc.p0 & 1) * C::kStage;
      float* vp = kp + P * KP;
      if (p < pc.live) {
        const PageDesc pg = record(p);
        if (slot_hi(pg) > slot_lo(pg)) {
          const float* ks = reinterpret_cast<const float*>(static_cast<const uint8_t*>(a.kpool) +
                                                           int64_t(pg.phys) * a.page_bytes);
          const float* vs = reinterpret_cast<const float*>(static_cast<const uint8_t*>(a.vpool) +
                                                           int64_t(pg.phys) * a.page_bytes);
          for (int e = tid; e < P * D / 4; e += kF32Threads) {
            cp_async16(kp + e / (D / 4) * KP + e % (D / 4) * 4, ks + e * 4);
            cp_async16(vp + e / (P / 4) * VP + e % (P / 4) * 4, vs + e * 4);
          }
        }
      } else {
        const int first = (p - pc.live) * P;
        const int64_t base = int64_t(pc.hd.b) * a.ds_seq + int64_t(pc.hd.kv) * a.ds_head;
        for (int e = tid; e < P * D; e += kF32Threads) {
          const int t = e / D, i = e % D;
          const int64_t from = base + (first + t) * a.ds_tok + i;
          const bool in = first + t < pc.n;
          kp[t * KP + i] = in ? static_cast<const float*>(a.k_draft)[from] : 0.f;
          vp[i * VP + t] = in ? static_cast<const float*>(a.v_draft)[from] : 0.f;
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    __syncthreads();  // the previous piece's buffers are read
    load(pc.p0);
    if (tid < 32) {  // one warp holds all rows' nodes
      uint64_t nodes[2];
      tree_ancestors(tree_parent(a, pc.hd.b, pc.n, tid), tree_parent(a, pc.hd.b, pc.n, tid + 32), tid, nodes);
      const uint64_t mask = tree_mask_of(nodes, min(pc.node0 + tid / G, kMaxTreeNodes - 1));
      if (tid < kF32Rows) {
        anc[tid] = tid < rows ? tree_visible(mask, pc.hd) : 0;
        pos[tid] = pc.hd.ctx_len + __popcll(mask) - 1;
        st[kF32Rows + tid] = -INFINITY, st[2 * kF32Rows + tid] = 0.f;
      }
    }
    for (int e = tid; e < kF32Rows * D / 4; e += kF32Threads) {
      const int r = e / (D / 4), c = e % (D / 4) * 4;
      *reinterpret_cast<float4*>(qs + r * KP + c) =
          r < rows ? *reinterpret_cast<const float4*>(static_cast<const float*>(a.q) + at_row(r) * D + c)
                   : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    float acc[OR];
#pragma unroll
    for (int j = 0; j < OR; ++j) acc[j] = 0.f;
    for (int p = pc.p0; p < pc.p1; ++p) {
      if (p + 1 < pc.p1) load(p + 1);
      else asm volatile("cp.async.commit_group;" ::: "memory");
      asm volatile("cp.async.wait_group 1;" ::: "memory");
      __syncthreads();
      const bool draft = p >= pc.live;
      const int first = (p - pc.live) * P;  // draft: the page's first node
      const PageDesc pg = record(p);
      const float* kp = stage + (p - pc.p0 & 1) * C::kStage;
      const float* vp = kp + P * KP;
      if (draft || slot_hi(pg) > slot_lo(pg)) {
        {
          const int t = tid % P, r0 = tid / P;  // rows r0, r0 + 128 / P, ...
          float s[SR];
#pragma unroll
          for (int j = 0; j < SR; ++j) s[j] = 0.f;
#pragma unroll 4
          for (int i = 0; i < D; i += 4) {
            const float4 kv = *reinterpret_cast<const float4*>(kp + t * KP + i);
#pragma unroll
            for (int j = 0; j < SR; ++j)
              s[j] = dot4(*reinterpret_cast<const float4*>(qs + (r0 + j * (kF32Threads / P)) * KP + i), kv, s[j]);
          }
#pragma unroll
          for (int j = 0; j < SR; ++j) {
            const int r = r0 + j * (kF32Threads / P);
            const uint64_t vis = draft ? anc[r] >> first : tree_page_mask(pg, pc.hd, pos[r]);
            sc[r * VP + t] = (vis >> t) & 1 ? s[j] * a.scale_log2 : -INFINITY;
          }
        }
        __syncthreads();
        {  // eight threads a row
          const int r = tid / 8, sub = tid % 8;
          float x[P / 8], mx = -INFINITY, sum = 0.f;
#pragma unroll
          for (int k = 0; k < P / 8; ++k) mx = fmaxf(mx, x[k] = sc[r * VP + sub + 8 * k]);
#pragma unroll
          for (int o = 1; o < 8; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
          const float mo = st[kF32Rows + r], mn = fmaxf(mo, mx), base = mn == -INFINITY ? 0.f : mn;
#pragma unroll
          for (int k = 0; k < P / 8; ++k) {
            const float e = exp2f(x[k] - base);
            sc[r * VP + sub + 8 * k] = e;
            sum += e;
          }
#pragma unroll
          for (int o = 1; o < 8; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
          const float al = exp2f(mo - base);
          __syncwarp();
          if (sub == 0) st[r] = al, st[kF32Rows + r] = mn, st[2 * kF32Rows + r] = st[2 * kF32Rows + r] * al + sum;
        }
        __syncthreads();
        {
          const int col = tid % D, r0 = tid / D;  // rows r0, r0 + 128 / D, ...
#pragma unroll
          for (int j = 0; j < OR; ++j) acc[j] *= st[r0 + j * (kF32Threads / D)];
#pragma unroll 4
          for (int t = 0; t < P; t += 4) {
            const float4 vv = *reinterpret_cast<const float4*>(vp + col * VP + t);
#pragma unroll
            for (int j = 0; j < OR; ++j)
              acc[j] = dot4(*reinterpret_cast<const float4*>(sc + (r0 + j * (kF32Threads / D)) * VP + t), vv, acc[j]);
          }
        }
      }
      __syncthreads();  // the stage, the weights and alpha are read
    }
    const int col = tid % D, r0 = tid / D;
#pragma unroll
    for (int j = 0; j < OR; ++j) {
      const int r = r0 + j * (kF32Threads / D);
      if (r >= rows) continue;
      const float M = st[kF32Rows + r], L = st[2 * kF32Rows + r];
      if (pc.n_pieces == 1) {
        static_cast<float*>(a.out)[at_row(r) * D + col] = acc[j] / L;
        if (col == 0 && a.lse) a.lse[at_row(r)] = (M + log2f(L)) * kTreeLn2;
      } else {
        float* slot = a.partial + int64_t(pc.slot) * tree_slot_floats(a);
        slot[tree_acc_at(r, col, rows_max)] = acc[j];
        if (col == 0) slot[rows_max * D + 2 * r] = M, slot[rows_max * D + 2 * r + 1] = L;
      }
    }
    if constexpr (!HERE) {
      if (tid == 0) tree_note_join(a, pc);
    } else if (pc.n_pieces > 1) {
      __threadfence();
      __syncthreads();
      if (tid == 0) tree_take_ticket(a, pc, &here);
    }
  }
  if constexpr (HERE) {
    __syncthreads();
    tree_join_here<float, D>(a, here, tid, kF32Threads);
  }
}

template <int D, bool FP8, int WR, bool HERE>
cudaError_t launch_mma(const TreeLaunch& a, cudaStream_t s) {
  using C = TreeMma<D, FP8, WR>;
  const cudaError_t e = allow_smem<tree_mma_kernel<D, FP8, WR, HERE>>(C::kBytes);
  if (e != cudaSuccess) return e;
  tree_mma_kernel<D, FP8, WR, HERE><<<a.n_ctas, C::kThreads, C::kBytes, s>>>(a);
  return cudaGetLastError();
}

template <int D, int P, bool HERE>
cudaError_t launch_f32_form(const TreeLaunch& a, cudaStream_t s) {
  constexpr int bytes = TreeF32<D, P>::kBytes;
  const cudaError_t e = allow_smem<tree_f32_kernel<D, P, HERE>>(bytes);
  if (e != cudaSuccess) return e;
  tree_f32_kernel<D, P, HERE><<<a.n_ctas, kF32Threads, bytes, s>>>(a);
  return cudaGetLastError();
}

template <int D, int P>
cudaError_t launch_f32(const TreeLaunch& a, cudaStream_t s) {
  return a.tickets ? launch_f32_form<D, P, true>(a, s) : launch_f32_form<D, P, false>(a, s);
}

template <int D, bool FP8>
cudaError_t launch_rows(const TreeLaunch& a, cudaStream_t s) {
  if (a.nodes_per_group * a.group <= 16)
    return a.tickets ? launch_mma<D, FP8, 1, true>(a, s) : launch_mma<D, FP8, 1, false>(a, s);
  return a.tickets ? launch_mma<D, FP8, 2, true>(a, s) : launch_mma<D, FP8, 2, false>(a, s);
}

}  // namespace

// A call of few heads and few pieces joins its split groups itself: the CTA of a
// group's last piece reads the others' from L2 in less time than a second launch
// takes (one user, 5 nodes, group 4, bf16: 13.7 us against 15.3 at 400 tokens,
// 15.9 against 17.4 at 1600; 64 heads, 8 nodes, 1600 tokens: 17.7 against 20.7).
// Groups are split at two units or more (TreeSplit's MIN_UNITS), so a head of n
// pages makes at most n / 2 + 2 pieces a group: up to 16, four batches of loads;
// beyond, the rows are shared out over the GPU.  With more heads the CTAs have
// pages enough that the page loop's registers count (128 heads, 1000 tokens:
// 28.0 us against 27.1).
constexpr int kPiecesHere = 16;
static bool tree_joins_here(const sp_plan* plan) {
  if (plan->hdr.n_heads > kTreeHeadsHere) return false;
  int32_t most = 0;
  for (const HeadDesc& h : plan->heads) most = std::max(most, h.n_vpages);
  const int draft = (kMaxTreeNodes + plan->prob.page_size - 1) / plan->prob.page_size;
  return (most + draft) / 2 + 2 <= kPiecesHere;
}

// Rows of a group: 16 or 32 while a sequence's rows fit; more rows of 16-bit and
// E4M3 pages go to the tensor cores (kernels_tree_tc.cu) in tiles of 128, two at
// a time where a sequence has more.  fp32 pages: 16.
TreeConfig tree_config(const sp_plan* plan, int32_t nodes) {
  const int g = plan->group, all = nodes * g;
  TreeConfig c{};
  c.tensor = plan->prob.dtype == SP_BF16 && all > 32;
  c.nodes_per_tile = 128 / g;
  int most;
  if (c.tensor) {
    most = (all > 128 ? 2 : 1) * c.nodes_per_tile;
    c.n_ctas = 148;
  } else {
    const int rows = plan->prob.dtype == SP_F32 || all <= 16 ? 16 : 32;
    most = rows / g;
    c.n_ctas = rows == 16 ? 2 * 148 : 148;
  }
  c.nodes_per_group = std::min(most, nodes);
  c.rows_per_group = c.nodes_per_group * g;
  c.joins_here = !c.tensor && tree_joins_here(plan);
  return c;
}

cudaError_t launch_tree(const TreeLaunch& a, const TreeConfig& c, cudaStream_t s) {
  if (c.tensor) return launch_tree_tc(a, s);
  if (!a.bf16) {
    if (a.P == 16) return a.D == 128 ? launch_f32<128, 16>(a, s) : launch_f32<64, 16>(a, s);
    return a.D == 128 ? launch_f32<128, 64>(a, s) : launch_f32<64, 64>(a, s);
  }
  if (a.fp8) return a.D == 128 ? launch_rows<128, true>(a, s) : launch_rows<64, true>(a, s);
  return a.D == 128 ? launch_rows<128, false>(a, s) : launch_rows<64, false>(a, s);
}

}  // namespace sp
