// Attention of a drafted tree over bf16 pages on 5th-generation tensor cores
// (tcgen05, sm_100a): the many-row form.
//
// One persistent CTA an SM walks its pieces of the work line (tree_common.cuh).
// A query tile is up to 128 rows (nodes x the group's q-heads, TMEM lane = row),
// a KV tile two pages, 128 tokens.  Two softmax streams share the tensor core:
//   a piece of one query tile   stream x takes KV tiles x, x + 2, ... with its own
//                               running maximum, sum and O; the streams' results
//                               join at the end of the piece;
//   a piece of two query tiles  (kWide) stream x takes query tile x over every
//                               KV tile, so one staged tile feeds 256 rows.
// Either way the tensor core works for one stream while the other's softmax runs:
//   S_x = Q K^T, then  O_x += P_x V, S_x (next), O_1-x += ..., alternating.
// One query tile reads its K/V once and is bound by HBM (64 KB a tile take
// 1.5 us of an SM's share, its two products 0.75 us); two tiles a CTA double the
// products on the same bytes.
//
// Warp roles (384 threads; the first warpgroup's spare registers go to the
// softmax threads):
//   warp 0     producer: walks the CTA's pieces and hands each to the others a slot
//              ahead; Q tiles by TMA (128-byte swizzle), K and V pages by bulk copies
//              into a ring of stages (pool pages are stored as the tensor cores' operands)
//   warp 1     TMEM owner and MMA issuer (one thread)
//   warps 2, 3 the draft's K and V rows, written as one more page of a stage
//   warps 4-7  softmax of stream 0, warps 8-11 of stream 1: a thread a row, the
//              whole 128-score row in registers; lazy rescale of O (only when the
//              row's maximum grows by more than 2^8), P written as bf16 over S
// The commit that signals S_x(j) also covers stream x's earlier O += P V, so a
// softmax thread that holds S_x(j) may rescale O_x with no further wait.
// Sums, maxima and O are fp32; P is rounded to bf16, V's own type.
// Every wait is bounded; one that runs out records a status code, and the CTA
// drains its copies and MMAs, frees its TMEM and returns.
#include <cuda.h>

#include "kernels.h"
#include "tc_ptx.cuh"
#include "tensor_map.h"
#include "tree_common.cuh"

namespace sp {
namespace {

constexpr int kThreads = 384;
// Registers a thread: 168 at launch (x 384 threads = 64512); 88 x 128 + 208 x 256 = 64512.
constexpr int kRegsIssue = 88, kRegsSoftmax = 208;
constexpr int kSoftmaxThreads = 256;
constexpr uint32_t kTmemCols = 512;
constexpr float kRescaleLog2 = 8.f;
constexpr uint32_t kAll = 0xffffffffu;
// One exponent pair in every kPolyPeriod is computed on the FMA pipe.
constexpr int kPolyPeriod = 8;

template <int D, bool WIDE>
struct TreeTc {
  static constexpr int kQ = D / 64 * 16384;  // a query tile: [D/64][128 rows][128 B]
  static constexpr int kK = D / 64 * 16384;  // [D/64][128 tokens][128 B]
  static constexpr int kV = 2 * D * 128;     // [2 pages][D rows][64 tokens * 2 B]
  static constexpr int kStage = kK + kV;
  static constexpr int kQTiles = WIDE ? 2 : 1;
  static constexpr int NS = (D == 128 ? 3 : 6) - (WIDE ? 1 : 0);
  static constexpr int kOffStage = kQTiles * kQ;
  static constexpr int kOffMl = kOffStage + NS * kStage;  // (m, l) of each row and stream
  static constexpr int kOffDesc = kOffMl + 2 * 128 * 8;
  static constexpr int kOffInfo = kOffDesc + NS * 2 * 16;
  using Split = TreeSplit<2, 2, 3>;
  using Info = TreePieceInfo<typename Split::Piece>;
  static constexpr int kOffBar = kOffInfo + (2 * int(sizeof(Info)) + 7) / 8 * 8;
  static constexpr int kBytes = kOffBar + (14 + 2 * NS) * 8 + 8;
  static_assert(kBytes <= 232448, "shared memory of a CTA");
  static_assert(kOffStage % 1024 == 0 && kStage % 1024 == 0 && kOffMl % 8 == 0 && kOffDesc % 16 == 0 &&
                    kOffInfo % alignof(Info) == 0 && kOffBar % 8 == 0,
                "alignment of the shared-memory parts");
  static_assert((kThreads / 32 + 2) * 8 <= 2 * 128 * 8, "the split's scratch lies in the statistics' place");
};

template <int D, bool WIDE>
__global__ void __launch_bounds__(kThreads, 1) tree_tc_kernel(const __grid_constant__ CUtensorMap qmap, TreeLaunch a) {
  using C = TreeTc<D, WIDE>;
  using Split = typename C::Split;
  using Info = typename C::Info;
  constexpr int NS = C::NS;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* stage_s = smem + C::kOffStage;
  float2* ml_s = reinterpret_cast<float2*>(smem + C::kOffMl);
  PageDesc* sdesc = reinterpret_cast<PageDesc*>(smem + C::kOffDesc);
  Info* info = reinterpret_cast<Info*>(smem + C::kOffInfo);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  uint64_t *q_full = bars, *q_free = bars + 1, *o_done = bars + 2, *done = bars + 3;
  uint64_t *s_full = bars + 4, *p_full = bars + 6, *piece_full = bars + 8, *piece_free = bars + 10;
  uint64_t *draft_go = bars + 12, *kv_full = bars + 14, *kv_free = kv_full + NS;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(kv_free + NS);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    mbar_init(q_full, 1);
    mbar_init(q_free, 1);
    mbar_init(o_done, 1);
    mbar_init(done, 1);
    for (int x = 0; x < 2; ++x) {
      mbar_init(&s_full[x], 1);
      mbar_init(&p_full[x], 128);
      mbar_init(&piece_full[x], 1);
      mbar_init(&draft_go[x], 1);
      mbar_init(&piece_free[x], 8 + 1 + 2);  // softmax warps, MMA issuer, draft warps
    }
    for (int s = 0; s < NS; ++s) {
      mbar_init(&kv_full[s], 3);  // the producer and the draft's two writers (without a draft it arrives for them)
      mbar_init(&kv_free[s], 1);
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
  // TMEM columns: S / P of stream x at [128 x, 128 x + 128); O at 256 + x D
  auto t_s = [&](int x) { return tmem + uint32_t(128 * x); };
  auto t_o = [&](int x) { return tmem + uint32_t(256 + x * D); };
  auto fail = [&](int32_t code) {
    record_error(a.status, code);
    *abort_flag = 1;
  };
  const int G = a.group, npt = a.nodes_per_tile;
  int k = 0;   // KV tiles of the earlier pieces
  int pi = 0;  // pieces so far
  bool ok = true;

  if (warp < 4) {
    tc::reg_dealloc<kRegsIssue>();
    if (warp == 0) {
      // ------------------------------ producer ------------------------------
      const uint8_t* kpool = static_cast<const uint8_t*>(a.kpool);
      const uint8_t* vpool = static_cast<const uint8_t*>(a.vpool);
      typename Split::Walk walk = split.walk();
      typename Split::Piece pc;
      auto piece_slot = [&] {  // the next piece's slot, once it is free
        const int ps = pi & 1;
        ok = pi < 2 || __shfl_sync(kAll, int(lane == 0 && mbar_wait(&piece_free[ps], ((pi >> 1) - 1) & 1)), 0);
        if (!ok && lane == 0) fail(kDevTimeoutEmpty);
        return ps;
      };
      while (ok && split.next(a, walk, pc)) {
        const bool two = WIDE && pc.nodes > npt;
        const PageDesc* rec = a.pages + pc.hd.vpage_begin;
        int4 mine = make_int4(0, 0, 0, 0);
        if (pc.p0 + lane < pc.live) mine = *reinterpret_cast<const int4*>(rec + pc.p0 + lane);
        const int ps = piece_slot();
        if (!ok) break;
        tree_publish(a, pc, k, lane, info[ps]);
        if (lane == 0) {
          mbar_arrive(&piece_full[ps]);
          if (pc.p1 <= pc.live) mbar_arrive(&draft_go[ps]);  // no draft page in this piece
        }
        auto load_q = [&] {  // behind the first KV tiles: its place is free only after the previous piece's last S
          if (lane == 0) {
            ok = pi == 0 || mbar_wait(q_free, (pi - 1) & 1);
            if (ok) {
              mbar_arrive_expect_tx(q_full, (two ? 2 : 1) * (D / 64) * npt * G * 128);
              for (int x = 0; x < (two ? 2 : 1); ++x)
#pragma unroll
                for (int h = 0; h < D / 64; ++h)
                  tc::tma_load_3d(smem + x * C::kQ + h * 16384, &qmap, h * 64, pc.hd.kv * G,
                                  pc.hd.b * a.T + pc.node0 + x * npt, q_full);
            } else {
              fail(kDevTimeoutMma);
            }
          }
          ok = __shfl_sync(kAll, int(ok), 0);
        };
        const int nt = (pc.p1 - pc.p0 + 1) / 2;
        for (int j = 0; ok && j < nt; ++j, ++k) {
          const int st = k % NS;
          uint8_t* k_s = stage_s + st * C::kStage;
          uint8_t* v_s = k_s + C::kK;
          PageDesc pg[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int p = pc.p0 + 2 * j + h, i = (2 * j + h) & 31;
            if (i == 0 && p > pc.p0 && p + lane < pc.live) mine = *reinterpret_cast<const int4*>(rec + p + lane);
            pg[h] = PageDesc{__shfl_sync(kAll, mine.x, i), __shfl_sync(kAll, mine.y, i), __shfl_sync(kAll, mine.z, i),
                             0};
            if (p >= pc.live) pg[h] = PageDesc{p == pc.live && p < pc.p1 ? kDraftPage : kNoPage, 0, 0, 0};
            else if (p >= pc.p1 || slot_hi(pg[h]) <= slot_lo(pg[h])) pg[h] = PageDesc{kNoPage, 0, 0, 0};
            else if (pg[h].phys < 0 || pg[h].phys >= a.pool_pages) {
              if (lane == 0) record_error(a.status, kDevBadPage);  // corrupted table: read nothing there
              pg[h] = PageDesc{kNoPage, 0, 0, 0};
            }
          }
          if (k >= NS) ok = __shfl_sync(kAll, int(lane == 0 && mbar_wait(&kv_free[st], ((k / NS) - 1) & 1)), 0);
          if (!ok) {
            if (lane == 0) fail(kDevTimeoutEmpty);
            break;
          }
          int bytes = 0;
          bool draft = false;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (pg[h].phys >= 0) bytes += (C::kK + C::kV) / 2;
            else if (pg[h].phys == kDraftPage) draft = true;
            else {  // no page: weights of zero meet values of zero
              for (int e = lane; e < D * 8; e += 32)
                reinterpret_cast<uint4*>(v_s + h * (D * 128))[e] = make_uint4(0, 0, 0, 0);
              fence_proxy_async_smem();
            }
          }
          __syncwarp();
          if (lane == 0) {
            sdesc[2 * st] = pg[0], sdesc[2 * st + 1] = pg[1];
            mbar_arrive_expect_tx(&kv_full[st], bytes);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              if (pg[h].phys < 0) continue;
              const int64_t off = int64_t(pg[h].phys) * a.page_bytes;
#pragma unroll
              for (int c = 0; c < D / 64; ++c)
                bulk_g2s(k_s + c * 16384 + h * 8192, kpool + off + c * 8192, 8192, &kv_full[st]);
              bulk_g2s(v_s + h * (D * 128), vpool + off, D * 128, &kv_full[st]);
            }
            if (draft) mbar_arrive(&draft_go[ps]);  // the stage is free
            else mbar_arrive(&kv_full[st]), mbar_arrive(&kv_full[st]);
          }
          __syncwarp();
          if (j == min(1, nt - 1)) {
            load_q();
            if (ok) ++pi;
          }
        }
      }
      if (ok) {
        const int ps = piece_slot();
        if (ok && lane == 0) {
          info[ps].pc.head = -1;
          mbar_arrive(&piece_full[ps]);
        }
      }
      // drain: never leave with copies still writing this CTA's shared memory
      if (lane == 0) {
        if (pi > 0) mbar_wait(q_full, (pi - 1) & 1);
        for (int j = (k > NS ? k - NS : 0); j < k; ++j)
          if (!mbar_wait(&kv_full[j % NS], (j / NS) & 1)) break;
      }
    } else if (warp == 1) {
      // ------------------------------ MMA issuer ------------------------------
      if (lane == 0) {
        constexpr uint32_t idesc_s = tc::idesc_bf16_f32(128, 128);
        constexpr uint32_t idesc_o = tc::idesc_bf16_f32(128, D);
        const uint32_t q_addr = smem_u32(smem), st_addr = smem_u32(stage_s);
        uint32_t turn[2] = {0, 0};  // P tiles taken of each stream
        auto wait_kv = [&](int tile) {
          if (mbar_wait(&kv_full[tile % NS], (tile / NS) & 1)) return true;
          fail(kDevTimeoutFull);
          return false;
        };
        auto issue_s = [&](int x, int q, int tile) {
          const uint64_t qd = tc::smem_desc_sw128(q_addr + q * C::kQ);
          const uint64_t kd = tc::smem_desc_sw128(st_addr + (tile % NS) * C::kStage);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = ((kk >> 2) * 16384 + (kk & 3) * 32) >> 4;
            tc::mma_bf16_ss(t_s(x), qd + off, kd + off, idesc_s, kk > 0);
          }
          tc::commit(&s_full[x]);
        };
        auto issue_pv = [&](int x, int tile, bool acc) {
          const uint64_t vd = tc::smem_desc_sw128(st_addr + (tile % NS) * C::kStage + C::kK);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            tc::mma_bf16_ts(t_o(x), t_s(x) + kk * 8, vd + (((kk >> 2) * (D * 128) + (kk & 3) * 32) >> 4), idesc_o,
                            (acc || kk > 0) ? 1u : 0u);
        };
        while (ok) {
          const int ps = pi & 1;
          if (!mbar_wait(&piece_full[ps], (pi >> 1) & 1)) {
            fail(kDevTimeoutFull);
            break;
          }
          if (info[ps].pc.head < 0) break;
          const bool two = WIDE && info[ps].pc.nodes > npt;
          const int nt = (info[ps].pc.p1 - info[ps].pc.p0 + 1) / 2, U = two ? 2 * nt : nt;
          mbar_arrive(&piece_free[ps]);
          auto tile_of = [&](int u) { return k + (two ? u >> 1 : u); };
          if (!mbar_wait(q_full, pi & 1)) {
            fail(kDevTimeoutFull);
            break;
          }
          for (int u = 0; ok && u < min(2, U); ++u) {
            ok = wait_kv(tile_of(u));
            if (!ok) break;
            tc::fence_after_sync();
            issue_s(u, two ? u : 0, tile_of(u));
          }
          if (ok && U <= 2) tc::commit(q_free);
          for (int u = 0; ok && u < U; ++u) {
            const int x = u & 1;
            if (*abort_flag || !mbar_wait(&p_full[x], turn[x] & 1)) {
              fail(kDevTimeoutSoftmax);
              ok = false;
              break;
            }
            ++turn[x];
            tc::fence_after_sync();
            issue_pv(x, tile_of(u), u >= 2);
            if (!two || x == 1) tc::commit(&kv_free[tile_of(u) % NS]);
            if (u + 2 < U) {
              ok = wait_kv(tile_of(u + 2));
              if (!ok) break;
              tc::fence_after_sync();
              issue_s(x, two ? x : 0, tile_of(u + 2));
              if (u + 3 == U) tc::commit(q_free);
            }
          }
          if (!ok) break;
          tc::commit(o_done);
          k += nt, ++pi;
        }
        // all MMAs issued by this thread complete before TMEM is released
        tc::commit(done);
        mbar_wait(done, 0);
      }
      __syncwarp();
    } else {
      // ------------------------------ draft page ------------------------------
      for (;; ++pi) {
        const int ps = pi & 1;
        if (!__all_sync(kAll, mbar_wait(&piece_full[ps], (pi >> 1) & 1))) break;
        const Info& in = info[ps];
        if (in.pc.head < 0) break;
        if (in.pc.p1 > in.pc.live) {
          const int at = in.pc.p1 - 1 - in.pc.p0, tile = in.stage0 + at / 2, h = at & 1, st = tile % NS;
          // the producer has seen the stage free (a wait on the stage's own barrier could be phases ahead of it)
          if (!__all_sync(kAll, mbar_wait(&draft_go[ps], (pi >> 1) & 1))) break;
          uint8_t* k_s = stage_s + st * C::kStage;
          if (warp == 2) tree_draft_k<D, false>(a, in.pc.hd, in.pc.n, k_s + h * 8192, 16384, lane);
          else tree_draft_v<D, false>(a, in.pc.hd, in.pc.n, k_s + C::kK + h * (D * 128), lane);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&kv_full[st]);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&piece_free[ps]);
      }
    }
  } else {
    tc::reg_alloc<kRegsSoftmax>();
    // ------------------------------ softmax ------------------------------
    const int x = (warp - 4) >> 2;
    const int quarter = warp & 3;  // TMEM lane quarter this warp may access
    const int r = quarter * 32 + lane;
    const uint32_t lane_off = uint32_t(quarter * 32) << 16;
    const int t256 = threadIdx.x - 128;
    const float sl2 = a.scale_log2;
    uint32_t turn = 0;  // tiles of this stream so far
    auto bar = [] { asm volatile("bar.sync 1, %0;" ::"n"(kSoftmaxThreads) : "memory"); };
    for (;; ++pi) {
      const int ps = pi & 1;
      // all softmax warps go on, or none: the barriers wait for every one of them
      const bool got = ok && __all_sync(kAll, mbar_wait(&piece_full[ps], (pi >> 1) & 1));
      if (ok && !got) fail(kDevTimeoutFull);
      if (!bar_red_and(1, kSoftmaxThreads, got)) break;
      if (info[ps].pc.head < 0) break;
      const typename Split::Piece pc = info[ps].pc;
      const bool two = WIDE && pc.nodes > npt;
      const int nt = (pc.p1 - pc.p0 + 1) / 2, U = two ? 2 * nt : nt;
      const int first_node = pc.node0 + (two ? x * npt : 0);
      const int rows = min(npt, pc.node0 + pc.nodes - first_node) * G;
      const bool busy = quarter * 32 < rows;  // any row in this warp
      uint64_t nodes[2];
      tree_ancestors(info[ps].up[lane], info[ps].up[lane + 32], lane, nodes);
      const uint64_t mask = tree_mask_of(nodes, min(first_node + r / G, kMaxTreeNodes - 1));
      const uint64_t anc = tree_visible(mask, pc.hd);
      const int pos = pc.hd.ctx_len + __popcll(mask) - 1;
      const int p_last = pc.hd.ctx_len + pc.n - 1;
      float m = -INFINITY, l = 0.f;
      for (int u = x; u < U; u += 2, ++turn) {
        const int tile = k + (two ? u >> 1 : u), st = tile % NS;
        // waits are voted: tcgen05.ld / st need the whole warp
        // (S_x first: then the stage's phase is this tile's, and its descriptors are read behind that barrier too)
        if (ok && !__all_sync(kAll, mbar_wait(&s_full[x], turn & 1) && mbar_wait(&kv_full[st], (tile / NS) & 1))) {
          fail(kDevTimeoutMma);
          ok = false;
        }
        if (ok && busy) {
          uint64_t vis[2];
          bool all = true;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const PageDesc pg = sdesc[2 * st + h];
            if (pg.phys >= 0 && tree_page_full(pg, pc.hd, p_last)) {
              vis[h] = ~uint64_t(0);
            } else {
              vis[h] = pg.phys == kDraftPage ? anc : pg.phys < 0 ? 0 : tree_page_mask(pg, pc.hd, pos);
              all = false;
            }
          }
          tc::fence_after_sync();
          float w[128];
          auto chunk = [&](int c) -> float(&)[32] { return *reinterpret_cast<float(*)[32]>(w + 32 * c); };
#pragma unroll
          for (int c = 0; c < 4; ++c) tc::tmem_ld32(t_s(x) + lane_off + 32 * c, chunk(c));
          tc::tmem_wait_ld();
          if (!all) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const uint32_t bits = uint32_t(vis[c >> 1] >> (32 * (c & 1)));
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (!((bits >> e) & 1)) w[32 * c + e] = -INFINITY;
            }
          }
          float m4[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) m4[i] = fmaxf(w[i], w[i + 4]);
#pragma unroll
          for (int e = 8; e < 128; e += 8)
#pragma unroll
            for (int i = 0; i < 4; ++i) m4[i] = fmax3(m4[i], w[e + i], w[e + 4 + i]);
          const float mts = fmax3(fmaxf(m4[0], m4[1]), m4[2], m4[3]) * sl2;
          float alpha = 1.f;
          bool need = false;
          if (mts > m + kRescaleLog2) {
            alpha = fast_exp2(m - mts);
            need = m != -INFINITY;
            m = mts;
          }
          if (__any_sync(kAll, need)) {
#pragma unroll
            for (int c = 0; c < D / 16; ++c) {
              uint32_t o[16];
              tc::tmem_ld16(t_o(x) + lane_off + c * 16, o);
              tc::tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
              tc::tmem_st16(t_o(x) + lane_off + c * 16, o);
            }
          }
          const float base = m == -INFINITY ? 0.f : m;
          const uint64_t nbase2 = f2_pack(-base, -base), scale2 = f2_pack(sl2, sl2);
          uint64_t s2[2] = {f2_pack(0.f, 0.f), f2_pack(0.f, 0.f)};
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t pk[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const uint64_t x2 = f2_fma(f2_pack(w[32 * c + 2 * e], w[32 * c + 2 * e + 1]), scale2, nbase2);
              float e0, e1;
              if (e % kPolyPeriod == kPolyPeriod - 1) {
                exp2_poly_pair(x2, e0, e1);
              } else {
                float x0, x1;
                f2_unpack(x2, x0, x1);
                e0 = fast_exp2(x0), e1 = fast_exp2(x1);
              }
              s2[e & 1] = f2_add(s2[e & 1], f2_pack(e0, e1));
              pk[e] = pack_bf16x2(e0, e1);
            }
            tc::tmem_st16(t_s(x) + lane_off + 16 * c, pk);
          }
          float a0, a1;
          f2_unpack(f2_add(s2[0], s2[1]), a0, a1);
          l = l * alpha + (a0 + a1);
          tc::tmem_wait_st();
        }
        tc::fence_before_sync();
        mbar_arrive(&p_full[x]);
      }
      // ------------------------------ end of the piece ------------------------------
      if (ok && !__all_sync(kAll, mbar_wait(o_done, pi & 1))) {
        fail(kDevTimeoutMma);
        ok = false;
      }
      tc::fence_after_sync();
      const int row_in_group = two ? x * npt * G + r : r;
      const bool valid = r < rows;
      const bool whole = pc.n_pieces == 1;
      float* slot = a.partial + int64_t(pc.slot) * tree_slot_floats(a);
      const int rows_max = a.nodes_per_group * G;
      const int64_t at =
          (int64_t(pc.hd.b) * a.T + first_node + r / G) * a.num_q_heads + pc.hd.kv * G + r % G;
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
      if (two) {
        if (ok && busy) {
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            float o[32];
            tc::tmem_ld32(t_o(x) + lane_off + 32 * c, o);
            tc::tmem_wait_ld();
            put(o, 32 * c, a.v_scale / l);
          }
          put_ml(m, l);
        }
      } else {  // join the two streams: each thread takes half of the row's columns
        ml_s[x * 128 + r] = make_float2(m, l);
        bar();
        if (ok && busy) {
          const float2 o_ml = ml_s[(1 - x) * 128 + r];
          const float M = fmaxf(m, o_ml.x), base = M == -INFINITY ? 0.f : M;
          const float own = fast_exp2(m - base), other = fast_exp2(o_ml.x - base);
          const float L = own * l + other * o_ml.y;
          const float f0 = x == 0 ? own : other, f1 = x == 0 ? other : own;
#pragma unroll
          for (int c = 0; c < D / 64; ++c) {
            const int col = x * (D / 2) + 32 * c;
            float o[32];
            tc::tmem_ld32(t_o(0) + lane_off + col, o);
            tc::tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] *= f0;
            if (nt > 1) {  // stream 1 had a tile
              float o1[32];
              tc::tmem_ld32(t_o(1) + lane_off + col, o1);
              tc::tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] += f1 * o1[e];
            }
            put(o, col, a.v_scale / L);
          }
          if (x == 0) put_ml(M, L);
        }
      }
      tc::fence_before_sync();
      bar();  // both streams have read O and the exchanged statistics
      if (t256 == 0) tree_note_join(a, pc);
      __syncwarp();
      if (lane == 0) mbar_arrive(&piece_free[ps]);
      k += nt;
    }
  }

  tc::fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, kTmemCols);
  }
}

template <int D, bool WIDE>
cudaError_t launch(const TreeLaunch& a, int64_t total_rows, cudaStream_t s) {
  using C = TreeTc<D, WIDE>;
  CUtensorMap qmap;
  cudaError_t e = encode_query_map(&qmap, a.q, D, a.num_q_heads, total_rows, a.group, a.nodes_per_tile);
  if (e != cudaSuccess) return e;
  auto kern = tree_tc_kernel<D, WIDE>;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kBytes);
  if (e != cudaSuccess) return e;
  kern<<<a.n_ctas, kThreads, C::kBytes, s>>>(qmap, a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_tree_tc(const TreeLaunch& a, cudaStream_t s) {
  const int64_t total_rows = int64_t(a.n_heads / a.num_kv_heads) * a.T;
  const bool wide = a.nodes_per_group > a.nodes_per_tile;
  if (a.D == 128) return wide ? launch<128, true>(a, total_rows, s) : launch<128, false>(a, total_rows, s);
  return wide ? launch<64, true>(a, total_rows, s) : launch<64, false>(a, total_rows, s);
}

}  // namespace sp
