// Attention of a drafted tree on 5th-generation tensor cores (tcgen05, sm_100a):
// the many-row form, over bf16 and E4M3 pages.
//
// One persistent CTA an SM walks its pieces of the work line (tree_common.cuh).
// A query tile is up to 128 rows (nodes x the group's q-heads, TMEM lane = row),
// a KV tile one page, 64 tokens.  Two softmax streams share the tensor core:
//   one query tile a piece       stream x takes the pages of parity x with its own
//                                running maximum, sum and O; the streams' results
//                                join at the end of the piece;
//   two query tiles (WIDE)       stream x takes query tile x over every page, so one
//                                staged page feeds 256 rows (a piece with rows for one
//                                tile leaves stream 1 idle).
// A barrier's phase is waited for by parity, so a waiter must not be a phase ahead
// or behind: every role waits for every phase of a barrier it uses, or for all of
// the barriers it owns.  Hence pages alternate by their number in the CTA, not in
// the piece, over rings of even length: a place of a ring belongs to one stream.
// A stream has two S buffers of 64 columns: while its softmax works on one page's
// scores, the tensor core makes the next page's S and the last one's O += P V.
// (With one buffer of 128 tokens a stream, a softmax waited for its own two
// products: 251 us where this form takes 221 on 64 nodes of the 32K layer.)
// One query tile reads its K/V once and is bound by HBM (bf16, d = 128: 0.82 us a
// page and CTA, 5.9 TB/s); two tiles a CTA double the products on the same bytes:
// 1.3 us a page, 2500 to 2650 cycles, of which the products' issue takes 2030.
//
// Warp roles (384 threads):
//   warp 0     walks the CTA's pieces and hands each to the others a slot ahead; Q
//              tiles by TMA (128-byte swizzle), K pages by bulk copies into a ring
//              (pool pages are stored as the tensor cores' operands), the draft's K
//              rows written as one more page
//   warps 1, 3 MMA issuers of the two streams (one thread each), so that one
//              stream's waits and commits pass while the other's products run;
//              warp 1 owns the TMEM
//   warp 2     V pages, and the draft's V rows, into a ring of their own: a K page is
//              free after S, a V page only a softmax and O += P V later
//   warps 4-7  softmax of stream 0, warps 8-11 of stream 1: a thread a row; lazy
//              rescale of O (only when the row's maximum grows by more than 2^8), P
//              written in 16 bits over the page's own S
//   warps 12-15  E4M3 pages only: the codes arrive in rings of their own (warps 0, 2)
//              and two warps each widen K and V into the operand rings, once a page,
//              as f16, which holds every code; Q is rewritten as f16 in place
// Sums, maxima and O are fp32; P is rounded to the operands' type: bf16, V's own, or
// f16 over widened codes (lifted: kWeightLift).
// Every wait is bounded; one that runs out records a status code, and the CTA
// drains its copies and MMAs, frees its TMEM and returns.
#include <cuda.h>

#include "kernels.h"
#include "tc_ptx.cuh"
#include "tensor_map.h"
#include "tree_common.cuh"

namespace sp {
namespace {

constexpr int kSoftmaxThreads = 256;
// E4M3 form, 512 threads: 128 registers at launch (65536); 80 x 256 + 168 x 256 = 63488.
constexpr int kRegsMove = 80, kRegsSoftmax = 168;
constexpr uint32_t kTmemCols = 512;
constexpr float kRescaleLog2 = 8.f;
constexpr uint32_t kAll = 0xffffffffu;
// Page descriptions in flight: a K page's place is free once its S is made, so
// the producer is at most KS pages ahead of S, and S four pages ahead of the
// softmax that reads the description.
constexpr int kDescs = 16;

template <int D, bool WIDE, bool FP8>
struct TreeTc {
  static constexpr int kThreads = FP8 ? 512 : 384;
  static constexpr int kQ = D / 64 * 16384;  // a query tile: [D/64][128 rows][128 B]
  static constexpr int kPage = 64 * D * 2;   // a K page [D/64][64 tokens][128 B], a V page [D rows][128 B]
  static constexpr int kRaw = 64 * D;        // a page of codes
  static constexpr int kQTiles = WIDE ? 2 : 1;
  // the 224 KB that Q leaves, in pages: K waits for its copy alone, V for a softmax too
  static constexpr int KS = D == 128 ? (WIDE && !FP8 ? 3 : 4) : (FP8 ? 6 : 8);
  static constexpr int VS = D == 128 ? (FP8 ? 4 : WIDE ? 5 : 8) : (FP8 ? 8 : 12);
  static constexpr int RS = !FP8 ? 0 : D == 128 ? (WIDE ? 2 : 4) : 6;  // pages of codes, K and V each
  static_assert(!FP8 || (KS % 2 == 0 && VS % 2 == 0 && RS % 2 == 0), "a place of a ring belongs to one widening warp");
  static constexpr int kOffK = kQTiles * kQ;
  static constexpr int kOffV = kOffK + KS * kPage;
  static constexpr int kOffRaw = kOffV + VS * kPage;     // K codes, then V codes
  static constexpr int kOffMl = kOffRaw + 2 * RS * kRaw;  // (m, l) of each row and stream
  static constexpr int kOffDesc = kOffMl + 2 * 128 * 8;
  static constexpr int kOffInfo = kOffDesc + kDescs * 8;
  using Split = TreeSplit<6, 8>;
  using Info = TreePieceInfo<typename Split::Piece>;
  static constexpr int kOffBar = kOffInfo + (2 * int(sizeof(Info)) + 7) / 8 * 8;
  static constexpr int kBytes = kOffBar + (22 + 2 * KS + 2 * VS + 4 * RS) * 8 + 8 + 8 * (RS > 0);
  static_assert(WIDE || (KS % 2 == 0 && VS % 2 == 0), "a place of a ring belongs to one stream");
  static_assert(KS + RS + 4 <= kDescs, "page descriptions");
  static_assert(kBytes <= 232448, "shared memory of a CTA");
  static_assert(kOffK % 1024 == 0 && kPage % 1024 == 0 && kRaw % 1024 == 0 && kOffMl % 8 == 0 && kOffDesc % 8 == 0 &&
                    kOffInfo % alignof(Info) == 0 && kOffBar % 8 == 0,
                "alignment of the shared-memory parts");
  static_assert((kThreads / 32 + 2) * 8 <= 2 * 128 * 8, "the split's scratch lies in the statistics' place");
};

// What the softmax needs of a page: its first position and its valid slots
// (lo | hi << 16); 0: no slot is seen.
struct PageSlots {
  int32_t abs_start;
  int32_t span;
};
constexpr int32_t kSlotsAll = -1;    // every row sees every slot
constexpr int32_t kSlotsDraft = -2;  // the draft's page

// E4M3 form: parked, so that its sixteen warps poll less (its 32K layer of 16 nodes takes 85 us, polling 95); the
// bf16 form is 3 % faster without.
template <bool PARKED>
__device__ __forceinline__ bool tc_wait(uint64_t* bar, uint32_t parity) {
  return PARKED ? mbar_wait_parked(bar, parity) : mbar_wait(bar, parity);
}

// A page of codes to f16, by one warp.  K: a lane is a token (then the token 32
// behind), a step 16 dimensions; V: a lane is a dimension (of 32, then the next
// 32), a step 16 positions or the dimension 64 behind.  Both layouts swizzle by
// XOR, so a step's address is an XOR of the lane's first one.  Four steps at a
// time in a rolled loop: all unrolled, with addresses made afresh, the page took
// 4300 cycles where this takes 1800.
template <int D, bool K>
__device__ __forceinline__ void widen_page(uint32_t src, uint32_t dst, int lane) {
  constexpr bool kHalves = D == 128 && !K;  // dimensions 64 ... 127 as every other step
#pragma unroll 1
  for (int it = 0; it < D / 32; ++it) {
    const int id = lane + it % 2 * 32, i0 = it / 2 * 4;
    const uint32_t from = src + (K ? fp8_kpage_offset(id, 0, D) : fp8_vpage_offset(id, 0));
    uint4 c[4], o[2];
#pragma unroll
    for (int u = 0; u < 4; ++u)
      c[u] = lds128(kHalves ? (from ^ ((i0 / 2 + u / 2) << 4)) + u % 2 * 4096 : from ^ ((i0 + u) << 4));
    const uint32_t to = dst + id * 128 + ((id & 7) << 4), at = K ? to + i0 / 4 * 8192 : to ^ (i0 << 4);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      widen16(c[u], o[0], o[1]);
#pragma unroll
      for (int h = 0; h < 2; ++h)
        sts128(kHalves ? (at ^ ((u / 2 * 2 + h) << 4)) + u % 2 * 8192 : at ^ ((2 * u + h) << 4), o[h]);
    }
  }
}

// E4M3 form: the draft's rows of K or V on their way to L1, asked for when a piece is handed out: its last page is
// written a ring of stages later, and would wait for them then (85 us where it takes 88 without; the bf16 forms, whose
// producers write the page well ahead of its turn, lose 1 to 2 % by it).
template <int D>
__device__ __forceinline__ void prefetch_draft(const TreeLaunch& a, const void* draft, const HeadDesc& hd, int n,
                                               int lane) {
  const char* row0 = reinterpret_cast<const char*>(static_cast<const __nv_bfloat16*>(draft) +
                                                   int64_t(hd.b) * a.ds_seq + int64_t(hd.kv) * a.ds_head);
  constexpr int LINES = D * 2 / 128;
  for (int u = lane; u < n * LINES; u += 32)
    asm volatile("prefetch.global.L1 [%0];" ::"l"(row0 + (u / LINES) * a.ds_tok * 2 + u % LINES * 128));
}

template <int D, bool WIDE, bool FP8>
__global__ void __launch_bounds__(TreeTc<D, WIDE, FP8>::kThreads, 1)
    tree_tc_kernel(const __grid_constant__ CUtensorMap qmap, TreeLaunch a) {
  using C = TreeTc<D, WIDE, FP8>;
  using Split = typename C::Split;
  using Info = typename C::Info;
  constexpr int kThreads = C::kThreads;
  constexpr int KS = C::KS, VS = C::VS, RS = C::RS, kUses = WIDE ? 2 : 1;
  constexpr float kLift = FP8 ? kWeightLift : 0.f;
  // the rings that the copies fill
  constexpr int KR = FP8 ? RS : KS, VR = FP8 ? RS : VS, kCopy = FP8 ? C::kRaw : C::kPage;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t *k_ring = smem + C::kOffK, *v_ring = smem + C::kOffV;
  float2* ml_s = reinterpret_cast<float2*>(smem + C::kOffMl);
  PageSlots* slots_s = reinterpret_cast<PageSlots*>(smem + C::kOffDesc);
  Info* info = reinterpret_cast<Info*>(smem + C::kOffInfo);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  uint64_t *q_full = bars, *q_free = bars + 1, *done = bars + 2, *piece_full = bars + 4, *piece_free = bars + 6;
  // [stream][buffer]: a softmax warp without rows may be a buffer ahead of the others, not two
  uint64_t *s_full = bars + 8, *p_full = bars + 12;
  uint64_t *pv_done = bars + 16, *o_done = bars + 18;  // a piece's last but one O += P V of a stream, and its last
  uint64_t* q_ready = bars + 20;                                   // E4M3: Q is f16
  uint64_t *k_full = bars + 22, *k_free = k_full + KS, *v_full = k_free + KS, *v_free = v_full + VS;
  // the rings that the copies fill
  uint8_t *kr_ring = FP8 ? smem + C::kOffRaw : k_ring, *vr_ring = FP8 ? kr_ring + RS * C::kRaw : v_ring;
  uint64_t *kr_full = FP8 ? v_free + VS : k_full, *kr_free = FP8 ? kr_full + RS : k_free;
  uint64_t *vr_full = FP8 ? kr_free + RS : v_full, *vr_free = FP8 ? vr_full + RS : v_free;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(v_free + VS + 4 * RS);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int8_t* v_kind = reinterpret_cast<volatile int8_t*>(tmem_slot + 2);  // E4M3: what a place of V's codes holds

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    mbar_init(q_full, 1);
    mbar_init(q_free, 2);
    for (int x = 0; x < 2; ++x) {
      mbar_init(&done[x], 1);
      mbar_init(&s_full[2 * x], 1), mbar_init(&s_full[2 * x + 1], 1);
      mbar_init(&p_full[2 * x], 4), mbar_init(&p_full[2 * x + 1], 4);
      mbar_init(&pv_done[x], 1);
      mbar_init(&o_done[x], 1);
      mbar_init(&piece_full[x], 1);
      mbar_init(&piece_free[x], 8 + 3 + (FP8 ? 4 : 0));  // softmax warps; MMA issuers, V producer; widening warps
    }
    // a page of two query tiles is free when both issuers' products have read it
    for (int s = 0; s < KS; ++s) mbar_init(&k_full[s], 1), mbar_init(&k_free[s], kUses);
    for (int s = 0; s < VS; ++s) mbar_init(&v_full[s], 1), mbar_init(&v_free[s], kUses);
    if constexpr (FP8) {
      mbar_init(q_ready, 2);
      for (int s = 0; s < RS; ++s) {
        mbar_init(&kr_full[s], 1), mbar_init(&kr_free[s], 1);
        mbar_init(&vr_full[s], 1), mbar_init(&vr_free[s], 1);
      }
    }
    *abort_flag = 0;
    fence_barrier_init();
    tc::prefetch_tensormap(&qmap);
  }
  Split split;
  if (!split.template init<kThreads>(a, reinterpret_cast<int64_t*>(ml_s))) return;
  if (warp == 1) {
    tc::tmem_alloc(tmem_slot, kTmemCols);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  // TMEM columns: S / P buffer b of stream x at 128 x + 64 b; O at 256 + x D
  auto t_s = [&](int x, int b) { return tmem + uint32_t(128 * x + 64 * b); };
  auto t_o = [&](int x) { return tmem + uint32_t(256 + x * D); };
  auto fail = [&](int32_t code) {
    record_error(a.status, code);
    *abort_flag = 1;
  };
  const int G = a.group, npt = a.nodes_per_tile;
  int k = 0;   // pages of the earlier pieces
  int pi = 0;  // pieces so far
  bool ok = true;

  if (warp < 4) {
    if constexpr (FP8) tc::reg_dealloc<kRegsMove>();
    if (warp == 0 || warp == 2) {
      // A producer's pages: records fetched 32 at a time, a lane each; kDraftPage for the draft's, kNoPage for an
      // empty record or a page id outside the pool.
      int4 mine = make_int4(0, 0, 0, 0);
      auto fetch = [&](const typename Split::Piece& pc, int p) {
        if (p + lane < min(pc.live, pc.p1))
          mine = *reinterpret_cast<const int4*>(a.pages + pc.hd.vpage_begin + p + lane);
      };
      auto page = [&](const typename Split::Piece& pc, int p) {
        const int i = (p - pc.p0) & 31;
        if (i == 0 && p > pc.p0) fetch(pc, p);
        const PageDesc rec{__shfl_sync(kAll, mine.x, i), __shfl_sync(kAll, mine.y, i), __shfl_sync(kAll, mine.z, i), 0};
        if (p >= pc.live) return PageDesc{kDraftPage, 0, 0, 0};
        if (slot_hi(rec) <= slot_lo(rec)) return PageDesc{kNoPage, 0, 0, 0};
        if (rec.phys >= 0 && rec.phys < a.pool_pages) return rec;
        if (lane == 0) record_error(a.status, kDevBadPage);  // corrupted table: report, read nothing there
        return PageDesc{kNoPage, 0, 0, 0};
      };
      // a wait by lane 0, its outcome for the warp
      auto wait0 = [&](uint64_t* bar, int parity, int32_t code) {
        ok = __shfl_sync(kAll, int(lane == 0 && tc_wait<FP8>(bar, parity)), 0);
        if (!ok && lane == 0) fail(code);
        return ok;
      };
      if (warp == 0) {
        // ------------------------------ pieces, Q and K ------------------------------
        const uint8_t* kpool = static_cast<const uint8_t*>(a.kpool);
        typename Split::Walk walk = split.walk();
        typename Split::Piece pc;
        auto slot_free = [&] { return pi < 2 || wait0(&piece_free[pi & 1], ((pi >> 1) - 1) & 1, kDevTimeoutEmpty); };
        while (ok && split.next(a, walk, pc)) {
          const int tiles = WIDE && pc.nodes > npt ? 2 : 1;
          fetch(pc, pc.p0);
          if (!slot_free()) break;
          tree_publish(a, pc, k, lane, info[pi & 1]);
          if (lane == 0) mbar_arrive(&piece_full[pi & 1]);
          if (FP8 && pc.p1 > pc.live) prefetch_draft<D>(a, a.k_draft, pc.hd, pc.n, lane);
          const int p_last = pc.hd.ctx_len + pc.n - 1;
          for (int p = pc.p0; p < pc.p1; ++p, ++k) {
            const int st = k % KR;
            uint8_t* k_s = kr_ring + st * kCopy;
            const PageDesc pg = page(pc, p);
            if (k >= KR && !wait0(&kr_free[st], ((k / KR) - 1) & 1, kDevTimeoutEmpty)) break;
            if (!FP8 && pg.phys == kDraftPage) {
              tree_draft_k<D, kDraftBf16>(a, pc.hd, pc.n, k_s, lane);
              fence_proxy_async_smem();
              __syncwarp();
            }
            if (lane == 0) {
              slots_s[k % kDescs] =
                  PageSlots{pg.abs_start, pg.phys == kDraftPage                                      ? kSlotsDraft
                                          : pg.phys >= 0 && tree_page_full(pg, pc.hd, p_last) ? kSlotsAll
                                                                                              : pg.span};
              if (pg.phys >= 0) {
                mbar_arrive_expect_tx(&kr_full[st], kCopy);
                bulk_g2s(k_s, kpool + int64_t(pg.phys) * a.page_bytes, kCopy, &kr_full[st]);
              } else {
                mbar_arrive(&kr_full[st]);
              }
            }
            __syncwarp();
            if (p == pc.p0) {  // behind the first K page: Q's place is free only after the previous piece's last S
              if (pi > 0 && !wait0(q_free, (pi - 1) & 1, kDevTimeoutMma)) break;
              if (lane == 0) {
                mbar_arrive_expect_tx(q_full, tiles * (D / 64) * npt * G * 128);
                for (int x = 0; x < tiles; ++x)
#pragma unroll
                  for (int h = 0; h < D / 64; ++h)
                    tc::tma_load_3d(smem + x * C::kQ + h * 16384, &qmap, h * 64, pc.hd.kv * G,
                                    pc.hd.b * a.T + pc.node0 + x * npt, q_full);
              }
              __syncwarp();
              ++pi;
            }
          }
        }
        if (ok && slot_free() && lane == 0) {
          info[pi & 1].pc.head = -1;
          mbar_arrive(&piece_full[pi & 1]);
        }
        // drain: never leave with copies still writing this CTA's shared memory
        if (lane == 0) {
          if (pi > 0) tc_wait<FP8>(q_full, (pi - 1) & 1);
          for (int j = (k > KR ? k - KR : 0); j < k; ++j)
            if (!tc_wait<FP8>(&kr_full[j % KR], (j / KR) & 1)) break;
        }
      } else {
        // ------------------------------ V ------------------------------
        const uint8_t* vpool = static_cast<const uint8_t*>(a.vpool);
        for (; ok; ++pi) {
          const int ps = pi & 1;
          if (!wait0(&piece_full[ps], (pi >> 1) & 1, kDevTimeoutFull) || info[ps].pc.head < 0) break;
          const typename Split::Piece pc = info[ps].pc;
          __syncwarp();
          if (lane == 0) mbar_arrive(&piece_free[ps]);
          fetch(pc, pc.p0);
          if (FP8 && pc.p1 > pc.live) prefetch_draft<D>(a, a.v_draft, pc.hd, pc.n, lane);
          for (int p = pc.p0; p < pc.p1; ++p, ++k) {
            const int st = k % VR;
            uint8_t* v_s = vr_ring + st * kCopy;
            const PageDesc pg = page(pc, p);
            if (k >= VR && !wait0(&vr_free[st], ((k / VR) - 1) & 1, kDevTimeoutEmpty)) break;
            if (!FP8 && pg.phys < 0) {
              if (pg.phys == kDraftPage) {
                tree_draft_v<D, kDraftBf16>(a, pc.hd, pc.n, v_s, lane);
              } else {  // no page: weights of zero meet values of zero
                for (int e = lane; e < C::kPage / 16; e += 32)
                  reinterpret_cast<uint4*>(v_s)[e] = make_uint4(0, 0, 0, 0);
              }
              fence_proxy_async_smem();
              __syncwarp();
            }
            if (lane == 0) {
              if (FP8) v_kind[st] = int8_t(min(pg.phys, 0));
              if (pg.phys >= 0) {
                mbar_arrive_expect_tx(&vr_full[st], kCopy);
                bulk_g2s(v_s, vpool + int64_t(pg.phys) * a.page_bytes, kCopy, &vr_full[st]);
              } else {
                mbar_arrive(&vr_full[st]);
              }
            }
            __syncwarp();
          }
        }
        if (lane == 0)
          for (int j = (k > VR ? k - VR : 0); j < k; ++j)
            if (!tc_wait<FP8>(&vr_full[j % VR], (j / VR) & 1)) break;
      }
    } else {
      if (lane == 0) {
        // ------------------------------ MMA issuers ------------------------------
        const int x = warp >> 1;  // stream
        constexpr uint32_t idesc_s = FP8 ? tc::idesc_f16_f32(128, 64) : tc::idesc_bf16_f32(128, 64);
        constexpr uint32_t idesc_o = FP8 ? tc::idesc_f16_f32(128, D) : tc::idesc_bf16_f32(128, D);
        const uint32_t q_addr = smem_u32(smem), k_addr = smem_u32(k_ring), v_addr = smem_u32(v_ring);
        uint32_t phase = 0;  // bit b: parity of the phase of the stream's P buffer b
        auto wait = [&](uint64_t* bar, int parity, int32_t code) {
          ok = tc_wait<FP8>(bar, parity);
          if (!ok) fail(code);
          return ok;
        };
        while (ok) {
          const int ps = pi & 1;
          if (!wait(&piece_full[ps], (pi >> 1) & 1, kDevTimeoutFull) || info[ps].pc.head < 0) break;
          const int np = info[ps].pc.p1 - info[ps].pc.p0, j0 = (x - k) & 1;
          const bool lone = WIDE && info[ps].pc.nodes <= npt;  // rows for one tile
          const int U = !WIDE ? (np + 1 - j0) / 2 : lone && x == 1 ? 0 : np;
          mbar_arrive(&piece_free[ps]);
          auto page_of = [&](int u) { return k + (WIDE ? u : 2 * u + j0); };
          const uint64_t qd = tc::smem_desc_sw128(q_addr + (WIDE ? x : 0) * C::kQ);
          auto wait_k = [&](int u) {
            const int pg = page_of(u);
            return wait(&k_full[pg % KS], (pg / KS) & 1, kDevTimeoutFull);
          };
          auto issue_s = [&](int u) {
            const int pg = page_of(u);
            const uint64_t kd = tc::smem_desc_sw128(k_addr + (pg % KS) * C::kPage);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
              tc::mma_f16_ss(t_s(x, u & 1), qd + (((kk >> 2) * 16384 + (kk & 3) * 32) >> 4),
                              kd + (((kk >> 2) * 8192 + (kk & 3) * 32) >> 4), idesc_s, kk > 0);
            tc::commit(&s_full[2 * x + (u & 1)]);
            tc::commit(&k_free[pg % KS]);
            if (u == U - 1) tc::commit(q_free);
          };
          if (!wait(FP8 ? q_ready : q_full, pi & 1, kDevTimeoutFull)) break;
          if (U == 0) {
            mbar_arrive(q_free);
            for (int j = 0; WIDE && j < np; ++j) {  // the pages pass it by
              const int pg = k + j;
              if (!wait(&k_full[pg % KS], (pg / KS) & 1, kDevTimeoutFull)) break;
              mbar_arrive(&k_free[pg % KS]);
              if (!wait(&v_full[pg % VS], (pg / VS) & 1, kDevTimeoutFull)) break;
              mbar_arrive(&v_free[pg % VS]);
            }
          } else {
            for (int u = 0; u < min(2, U) && wait_k(u); ++u) {
              tc::fence_after_sync();
              issue_s(u);
            }
            for (int u = 0; ok && u < U; ++u) {
              const int pg = page_of(u);
              if (!wait(&v_full[pg % VS], (pg / VS) & 1, kDevTimeoutFull)) break;
              if (u + 2 < U && !wait_k(u + 2)) break;  // ahead of P: a wait costs 100 cycles even when it is over
              if (!wait(&p_full[2 * x + (u & 1)], phase >> (u & 1) & 1, kDevTimeoutSoftmax)) break;
              phase ^= 1u << (u & 1);
              tc::fence_after_sync();
              const uint64_t vd = tc::smem_desc_sw128(v_addr + (pg % VS) * C::kPage);
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                tc::mma_f16_ts(t_o(x), t_s(x, u & 1) + kk * 8, vd + ((kk * 32) >> 4), idesc_o,
                                (u > 0 || kk > 0) ? 1u : 0u);
              // the next S also says that this product is done; the last two have no next S
              if (u + 2 < U) issue_s(u + 2);
              else tc::commit(u + 1 < U ? &pv_done[x] : &o_done[x]);
              tc::commit(&v_free[pg % VS]);
            }
          }
          if (*abort_flag) break;
          k += np, ++pi;
        }
        // all MMAs issued by this thread complete before TMEM is released
        tc::commit(&done[x]);
        tc_wait<FP8>(&done[x], 0);
      }
    }
  } else if (FP8 && warp >= 12) {
    if constexpr (FP8) {
      // ------------------------------ widening ------------------------------
      tc::reg_dealloc<kRegsMove>();
      const bool is_k = warp < 14;
      const int odd = warp & 1;  // the pages it takes: even ones or odd ones
      uint8_t *raw = is_k ? kr_ring : vr_ring, *wide = is_k ? k_ring : v_ring;
      uint64_t *raw_full = is_k ? kr_full : vr_full, *raw_free = is_k ? kr_free : vr_free;
      uint64_t *wide_full = is_k ? k_full : v_full, *wide_free = is_k ? k_free : v_free;
      const int WS = is_k ? KS : VS;
      auto wait = [&](uint64_t* bar, int parity) {
        ok = __all_sync(kAll, tc_wait<FP8>(bar, parity));
        if (!ok) fail(kDevTimeoutFull);
        return ok;
      };
      for (; ok; ++pi) {
        const int ps = pi & 1;
        if (!wait(&piece_full[ps], (pi >> 1) & 1)) break;
        const Info& in = info[ps];
        if (in.pc.head < 0) break;
        if (!is_k) {  // Q to f16, in place: the same swizzled chunks
          if (!wait(q_full, pi & 1)) break;
          const int bytes = (WIDE && in.pc.nodes > npt ? 2 : 1) * C::kQ;
#pragma unroll 4
          for (int e = odd * 32 + lane; e < bytes / 16; e += 64) {
            uint4* q = reinterpret_cast<uint4*>(smem) + e;
            const uint4 v = *q;
            *q = make_uint4(bf16x2_to_f16x2(v.x), bf16x2_to_f16x2(v.y), bf16x2_to_f16x2(v.z), bf16x2_to_f16x2(v.w));
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(q_ready);
        }
        const int np = in.pc.p1 - in.pc.p0;
        for (int j = 0; j < np; ++j, ++k) {
          if ((k & 1) != odd) continue;
          const int rs = k % RS, ws = k % WS;
          if (!wait(&raw_full[rs], (k / RS) & 1)) break;
          if (k >= WS && !wait(&wide_free[ws], ((k / WS) - 1) & 1)) break;
          const uint8_t* src = raw + rs * C::kRaw;
          uint8_t* dst = wide + ws * C::kPage;
          const int kind = is_k ? (slots_s[k % kDescs].span == kSlotsDraft ? kDraftPage : 0) : v_kind[rs];
          if (kind == kDraftPage) {
            if (is_k) tree_draft_k<D, kDraftWide>(a, in.pc.hd, in.pc.n, dst, lane);
            else tree_draft_v<D, kDraftWide>(a, in.pc.hd, in.pc.n, dst, lane);
          } else if (kind == kNoPage) {  // V: weights of zero meet values of zero
            for (int e = lane; e < C::kPage / 16; e += 32)
              reinterpret_cast<uint4*>(dst)[e] = make_uint4(0, 0, 0, 0);
          } else {
            if (is_k) widen_page<D, true>(smem_u32(src), smem_u32(dst), lane);
            else widen_page<D, false>(smem_u32(src), smem_u32(dst), lane);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&wide_full[ws]);
            mbar_arrive(&raw_free[rs]);
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&piece_free[ps]);
      }
    }
  } else {
    if constexpr (FP8) tc::reg_alloc<kRegsSoftmax>();
    // ------------------------------ softmax ------------------------------
    const int x = (warp - 4) >> 2;
    const int quarter = warp & 3;  // TMEM lane quarter this warp may access
    const int r = quarter * 32 + lane;
    const uint32_t lane_off = uint32_t(quarter * 32) << 16;
    const uint32_t to = t_o(x) + lane_off;
    const int t256 = threadIdx.x - 128;
    const float sl2 = a.scale_log2;
    uint32_t phase = 0;  // parities: bits 0, 1 of the stream's S buffers, 2 of pv_done, 3 of o_done
    auto bar = [] { asm volatile("bar.sync 1, %0;" ::"n"(kSoftmaxThreads) : "memory"); };
    // waits are voted: tcgen05.ld / st need the whole warp
    auto wait = [&](uint64_t* bar, int bit) {
      if (ok && !__all_sync(kAll, tc_wait<FP8>(bar, phase >> bit & 1))) {
        fail(kDevTimeoutMma);
        ok = false;
      }
    };
    for (;; ++pi) {
      const int ps = pi & 1;
      // all softmax warps go on, or none: the barriers wait for every one of them
      const bool got = ok && __all_sync(kAll, tc_wait<FP8>(&piece_full[ps], (pi >> 1) & 1));
      if (ok && !got) fail(kDevTimeoutFull);
      if (!bar_red_and(1, kSoftmaxThreads, got)) break;
      if (info[ps].pc.head < 0) break;
      const typename Split::Piece& pc = info[ps].pc;
      const HeadDesc hd = pc.hd;
      const int first_node = pc.node0 + (WIDE ? x * npt : 0);
      const int rows = min(npt, pc.node0 + pc.nodes - first_node) * G;
      const int np = pc.p1 - pc.p0, j0 = (x - k) & 1;
      const int U = !WIDE ? (np + 1 - j0) / 2 : rows > 0 ? np : 0;
      const bool busy = quarter * 32 < rows;  // any row in this warp
      uint64_t nodes[2];
      tree_ancestors(info[ps].up[lane], info[ps].up[lane + 32], lane, nodes);
      const uint64_t mask = tree_mask_of(nodes, min(first_node + r / G, kMaxTreeNodes - 1));
      const uint64_t anc = tree_visible(mask, hd);
      const int pos = hd.ctx_len + __popcll(mask) - 1;
      float m = -INFINITY, l = 0.f;
      auto page_scores = [&](int u, int b) {
        const PageSlots sl = slots_s[(k + (WIDE ? u : 2 * u + j0)) % kDescs];
        const uint32_t ts = t_s(x, b) + lane_off;
        tc::fence_after_sync();
        // two passes over the scores, which stay in TMEM.  The E4M3 form rolls the halves: unrolled, the loops of its
        // roles outgrow the instruction cache (97 us where it takes 85); the bf16 form is 3 % faster unrolled
        float mts = -INFINITY;
#pragma unroll(FP8 ? 1 : 2)
        for (int c = 0; c < 2; ++c) {
          float w[32], m8[8];
          tc::tmem_ld32(ts + 32 * c, w);
          tc::tmem_wait_ld();
          if (sl.span != kSlotsAll) {
            const uint64_t vis = sl.span == kSlotsDraft ? anc : tree_page_mask({0, sl.abs_start, sl.span, 0}, hd, pos);
            const uint32_t bits = uint32_t(vis >> (32 * c));
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (!((bits >> e) & 1)) w[e] = -INFINITY;
            tc::tmem_st32(ts + 32 * c, w);
            tc::tmem_wait_st();
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) m8[i] = fmax3(w[i], w[i + 8], w[i + 16]);
#pragma unroll
          for (int i = 0; i < 8; ++i) m8[i] = fmaxf(m8[i], w[i + 24]);
          mts = fmaxf(fmax3(fmax3(m8[0], m8[1], m8[2]), m8[3], m8[4]), fmax3(fmax3(m8[5], m8[6], m8[7]), mts, mts));
        }
        mts *= sl2;
        // the running reference nearly always holds; where a row of the warp has outgrown it, it moves, and O
        // follows once the previous product is done (the next page's S says so)
        float alpha = 1.f;
        if (__any_sync(kAll, mts > m + kRescaleLog2)) {
          if (mts > m + kRescaleLog2) {
            alpha = fast_exp2(m - mts);
            m = mts;
          }
          if (u > 0) {
            if (u + 1 < U) wait(&s_full[2 * x + (b ^ 1)], b ^ 1);
            else wait(&pv_done[x], 2);
            if (!ok) return;
            tc::fence_after_sync();
#pragma unroll
            for (int c = 0; c < D / 16; ++c) {
              uint32_t o[16];
              tc::tmem_ld16(to + c * 16, o);
              tc::tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
              tc::tmem_st16(to + c * 16, o);
            }
          }
        }
        const float base = m == -INFINITY ? 0.f : m - kLift;
        const uint64_t nbase2 = f2_pack(-base, -base), scale2 = f2_pack(sl2, sl2);
        uint64_t s2[2] = {f2_pack(0.f, 0.f), f2_pack(0.f, 0.f)};
#pragma unroll(FP8 ? 1 : 2)
        for (int c = 0; c < 2; ++c) {  // P of columns 32 c ... goes where those of 16 c ... were
          float w[32], e0[16], e1[16];  // e0, e1: of pairs of tokens
          tc::tmem_ld32(ts + 32 * c, w);
          tc::tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            float x0, x1;
            f2_unpack(f2_fma(f2_pack(w[2 * e], w[2 * e + 1]), scale2, nbase2), x0, x1);
            e0[e] = fast_exp2(x0), e1[e] = fast_exp2(x1);
            s2[e & 1] = f2_add(s2[e & 1], f2_pack(e0[e], e1[e]));
          }
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            // E4M3: the order of the page's positions (pairs of tokens 0 4 1 5 2 6 3 7 of every 16 tokens)
            if constexpr (FP8) pk[(e & 8) | (e & 3) << 1 | (e >> 2 & 1)] = pack_f16x2(e0[e], e1[e]);
            else pk[e] = pack_bf16x2(e0[e], e1[e]);
          }
          tc::tmem_st16(ts + 16 * c, pk);
        }
        float a0, a1;
        f2_unpack(f2_add(s2[0], s2[1]), a0, a1);
        l = l * alpha + (a0 + a1);
        tc::tmem_wait_st();
      };
      for (int u = 0; u < U; ++u) {
        const int b = u & 1;
        wait(&s_full[2 * x + b], b);
        phase ^= 1u << b;
        if (ok && busy) page_scores(u, b);
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[2 * x + b]);
      }
      // ------------------------------ end of the piece ------------------------------
      m -= kLift;  // what l and O are relative to
      if (U > 1) phase ^= 1u << 2;
      if (U > 0) {
        wait(&o_done[x], 3);
        phase ^= 1u << 3;
      }
      tc::fence_after_sync();
      const int row_in_group = WIDE ? x * npt * G + r : r;
      const bool valid = r < rows;
      const bool whole = pc.n_pieces == 1;
      float* slot = a.partial + int64_t(pc.slot) * tree_slot_floats(a);
      const int rows_max = a.nodes_per_group * G;
      const int64_t at = (int64_t(hd.b) * a.T + first_node + r / G) * a.num_q_heads + hd.kv * G + r % G;
      // 32 columns of the row's accumulator, scaled, to the output or the partial slot
      auto put = [&](const float (&o)[32], int col, float inv) {
        if (!valid) return;
        if (whole) {
          uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + at * D + col);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            dst[e] = make_uint4(pack_bf16x2(o[8 * e] * inv, o[8 * e + 1] * inv),
                                pack_bf16x2(o[8 * e + 2] * inv, o[8 * e + 3] * inv),
                                pack_bf16x2(o[8 * e + 4] * inv, o[8 * e + 5] * inv),
                                pack_bf16x2(o[8 * e + 6] * inv, o[8 * e + 7] * inv));
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            *reinterpret_cast<float4*>(slot + tree_acc_at(row_in_group, col + 4 * e, rows_max)) =
                make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
        }
      };
      auto put_ml = [&](float mm, float ll) {
        if (!valid) return;
        if (!whole) *reinterpret_cast<float2*>(slot + rows_max * D + 2 * row_in_group) = make_float2(mm, ll);
        else if (a.lse) a.lse[at] = (mm + log2f(ll)) * kTreeLn2;
      };
      if constexpr (WIDE) {
        if (ok && busy) {
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            float o[32];
            tc::tmem_ld32(to + 32 * c, o);
            tc::tmem_wait_ld();
            put(o, 32 * c, a.v_scale / l);
          }
          put_ml(m, l);
        }
      } else {  // join the two streams: each thread takes half of the row's columns
        ml_s[x * 128 + r] = make_float2(m, l);
        tc::fence_before_sync();
        bar();
        tc::fence_after_sync();
        if (ok && busy) {
          const float2 o_ml = ml_s[(1 - x) * 128 + r];
          const float M = fmaxf(m, o_ml.x), base = M == -INFINITY ? 0.f : M;
          const float own = fast_exp2(m - base), other = fast_exp2(o_ml.x - base);
          const float L = own * l + other * o_ml.y;
          const float f0 = x == 0 ? own : other, f1 = x == 0 ? other : own;
#pragma unroll
          for (int c = 0; c < D / 64; ++c) {
            const int col = x * (D / 2) + 32 * c;
            float o[32] = {};
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              if ((np + 1 - ((y - k) & 1)) / 2 == 0) continue;  // stream y had no page
              float v[32];
              tc::tmem_ld32(t_o(y) + lane_off + col, v);
              tc::tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] += (y ? f1 : f0) * v[e];
            }
            put(o, col, a.v_scale / L);
          }
          if (x == 0) put_ml(M, L);
        }
      }
      tc::fence_before_sync();
      if (t256 == 0) tree_note_join(a, pc);
      k += np;
      bar();  // both streams have read O, the exchanged statistics and the piece
      if (lane == 0) mbar_arrive(&piece_free[ps]);
    }
  }

  tc::fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, kTmemCols);
  }
}

template <int D, bool WIDE, bool FP8>
cudaError_t launch(const TreeLaunch& a, int64_t total_rows, cudaStream_t s) {
  using C = TreeTc<D, WIDE, FP8>;
  CUtensorMap qmap;
  cudaError_t e = encode_query_map(&qmap, a.q, D, a.num_q_heads, total_rows, a.group, a.nodes_per_tile);
  if (e != cudaSuccess) return e;
  e = allow_smem<tree_tc_kernel<D, WIDE, FP8>>(C::kBytes);
  if (e != cudaSuccess) return e;
  tree_tc_kernel<D, WIDE, FP8><<<a.n_ctas, C::kThreads, C::kBytes, s>>>(qmap, a);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_form(const TreeLaunch& a, cudaStream_t s) {
  const int64_t total_rows = int64_t(a.n_heads / a.num_kv_heads) * a.T;
  const bool wide = a.nodes_per_group > a.nodes_per_tile;
  if (a.fp8) return wide ? launch<D, true, true>(a, total_rows, s) : launch<D, false, true>(a, total_rows, s);
  return wide ? launch<D, true, false>(a, total_rows, s) : launch<D, false, false>(a, total_rows, s);
}

}  // namespace

cudaError_t launch_tree_tc(const TreeLaunch& a, cudaStream_t s) {
  return a.D == 128 ? launch_form<128>(a, s) : launch_form<64>(a, s);
}

}  // namespace sp
