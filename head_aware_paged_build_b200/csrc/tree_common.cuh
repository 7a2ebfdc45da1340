// Work split, visibility and merge of tree attention, shared by its kernels.
//
// A sequence's draft is a forest of n <= 64 nodes (parent[i] < i); node i at
// depth d sits at position p = L + d, L the sequence's context length.  With
// s the sink and w the window of a LOCAL head it sees, of the cache, the
// positions j < s or j > p - w (a GLOBAL head: all; a RETRIEVAL head: its kept
// blocks' pages too, which carry kSpanCausal), and of the draft itself
// and its ancestors, by the same rule at their positions.  A kv-head's rows
// are its nodes times its group's q-heads, node-major.
//
// Split.  A head's work is its live pages, then the draft's page(s), once for
// each row group, plus a fixed cost per group in pages (START: loading Q,
// publishing or writing the rows).  Laid end to end
// over the heads this is a line of U units; CTA c of G takes [cU/G, (c+1)U/G).
// Every CTA works the line out from the table itself (a block-wide sum over
// the heads), so the split follows the lengths as the cache grows and needs no
// host work and no list: which CTAs share a row group, and which workspace
// slot each of them wrote (its first piece: 2c, a later one: 2c + 1; pieces
// between cover their group and need none) are arithmetic on (U, G).  A group
// in one CTA is written there; the others' pieces are joined by a second,
// dependent kernel, or in short calls by the CTA of a group's last piece.
#pragma once

#include "append_common.cuh"
#include "kernels.h"

namespace sp {

constexpr int kDraftPage = -2;  // phys of the draft's page in a stage's record
constexpr float kTreeLn2 = 0.6931471805599453f;

// E4M3 pages: softmax weights are f16 operands, taken 2^7 times larger.  The
// lazy rescale lets a weight reach 2^8 times the running maximum's, so 2^15 of
// f16's 65504 is used, and a weight's rounding, half a subnormal step of 2^-24,
// is 2^-32 of the maximum's.  (Without the lift 2^-25: beside a dominant key,
// 32768 others below that, up to a thousandth of the row together, would vanish.)
constexpr float kWeightLift = 7.f;

// Bits [x, y) of a 64-bit word (any x, y).
__device__ __forceinline__ uint64_t bit_range(int x, int y) {
  x = max(x, 0), y = min(y, 64);
  return y <= x ? 0 : (~uint64_t(0) >> (64 - (y - x))) << x;
}

// Slots of a cached page that a row at position p sees (p is behind the cache: no causal bound).
__device__ __forceinline__ uint64_t tree_page_mask(const PageDesc& pg, const HeadDesc& hd, int p) {
  const int lo = slot_lo(pg), hi = slot_hi(pg);
  if (hd.kind == 0 || page_causal(pg)) return bit_range(lo, hi);
  return bit_range(lo, min(hi, hd.sink - pg.abs_start)) | bit_range(max(lo, p - hd.window + 1 - pg.abs_start), hi);
}
// Does every row at a position <= p_last see all 64 slots of this page?
__device__ __forceinline__ bool tree_page_full(const PageDesc& pg, const HeadDesc& hd, int p_last) {
  if (slot_lo(pg) != 0 || slot_hi(pg) != 64) return false;
  if (hd.kind == 0 || page_causal(pg)) return true;
  return pg.abs_start + 63 < hd.sink || pg.abs_start > p_last - hd.window;
}

// Node count of sequence b, bounded; *bad reports one outside [0, T].
__device__ __forceinline__ int tree_nodes(const TreeLaunch& a, int b, bool* bad = nullptr) {
  if (!a.num_nodes) return a.T;
  const int n = a.num_nodes[b];
  if (bad && (n < 0 || n > a.T)) *bad = true;
  return min(max(n, 0), a.T);
}

// One parent entry, checked: one outside [-1, own index) is reported and counts as a root.
__device__ __forceinline__ int tree_parent(const TreeLaunch& a, int b, int n, int i) {
  if (i >= n) return -1;
  const int p = a.parents[int64_t(b) * a.T + i];
  if (p >= -1 && p < i) return p;
  record_error(a.status, kDevBadTree);
  return -1;
}
// Ancestor masks (each node itself included) by one warp: lane x holds nodes x
// and x + 32, up[] their parents.  Pointer doubling: a round joins each node's
// mask with that of the farthest ancestor reached so far and jumps there, so a
// chain of 64 takes six rounds and a shallow tree two or three.
__device__ __forceinline__ void tree_ancestors(int up0, int up1, int lane, uint64_t (&anc)[2]) {
  int up[2] = {up0, up1};
  anc[0] = uint64_t(1) << lane, anc[1] = uint64_t(1) << (lane + 32);
  while (__any_sync(0xffffffffu, up[0] >= 0 || up[1] >= 0)) {
    uint64_t m[2];
    int next[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int from = up[x] & 31;
      const uint64_t m0 = __shfl_sync(0xffffffffu, anc[0], from), m1 = __shfl_sync(0xffffffffu, anc[1], from);
      const int u0 = __shfl_sync(0xffffffffu, up[0], from), u1 = __shfl_sync(0xffffffffu, up[1], from);
      m[x] = up[x] < 0 ? 0 : up[x] >= 32 ? m1 : m0;
      next[x] = up[x] < 0 ? -1 : up[x] >= 32 ? u1 : u0;
    }
#pragma unroll
    for (int x = 0; x < 2; ++x) anc[x] |= m[x], up[x] = next[x];
  }
}
// Node i's mask out of the warp's (all lanes call; i may differ by lane).
__device__ __forceinline__ uint64_t tree_mask_of(const uint64_t (&anc)[2], int i) {
  const uint64_t m0 = __shfl_sync(0xffffffffu, anc[0], i & 31), m1 = __shfl_sync(0xffffffffu, anc[1], i & 31);
  return i >= 32 ? m1 : m0;
}
// The ancestors a node sees: a node's index is above its parent's, so the k-th
// set bit is the ancestor at depth k, and a LOCAL head hides the lowest bits
// that are neither in the window nor among the sink positions.
__device__ __forceinline__ uint64_t tree_visible(uint64_t mask, const HeadDesc& hd) {
  const int depth = __popcll(mask) - 1;
  if (hd.kind == 0 || hd.window > depth) return mask;
  uint64_t left = mask, hidden = 0;
  for (int d = 0; d <= depth - hd.window; ++d) {
    const uint64_t bit = left & (0 - left);
    left ^= bit;
    if (hd.ctx_len + d >= hd.sink) hidden |= bit;
  }
  return mask & ~hidden;
}

// 16 E4M3 codes to two 16-byte chunks of f16, which holds each of them exactly.
__device__ __forceinline__ void widen16(const uint4& c, uint4& lo, uint4& hi) {
  lo = make_uint4(e4m3x2_to_f16x2(uint16_t(c.x)), e4m3x2_to_f16x2(uint16_t(c.x >> 16)),
                  e4m3x2_to_f16x2(uint16_t(c.y)), e4m3x2_to_f16x2(uint16_t(c.y >> 16)));
  hi = make_uint4(e4m3x2_to_f16x2(uint16_t(c.z)), e4m3x2_to_f16x2(uint16_t(c.z >> 16)),
                  e4m3x2_to_f16x2(uint16_t(c.w)), e4m3x2_to_f16x2(uint16_t(c.w >> 16)));
}

// Forms of the draft's page: as an append lays out bf16 and E4M3 pages, and the
// E4M3 codes widened to f16 in the bf16 pages' layout (V's tokens in the order
// of the E4M3 pages' positions).
enum DraftForm { kDraftBf16, kDraftE4m3, kDraftWide };

// The draft's n rows as a page of 64 slots in shared memory; one warp each for K
// and V (transposed).  Slots behind n hold zeros in V
// (their weights are zero, and 0 x garbage must stay 0) and are left as they are
// in K (their scores are masked).  Loads go out in batches: the rows come from
// global memory, and one row at a time would cost its latency up to 64 times.
template <int D, DraftForm FORM>
__device__ __forceinline__ void tree_draft_k(const TreeLaunch& a, const HeadDesc& hd, int n, uint8_t* kdst, int lane) {
  const __nv_bfloat16* kn =
      static_cast<const __nv_bfloat16*>(a.k_draft) + int64_t(hd.b) * a.ds_seq + int64_t(hd.kv) * a.ds_head;
  constexpr int CR = D / 8, KB = 8;  // 16-byte chunks of a K row; loads in flight
  for (int u0 = lane; u0 < n * CR; u0 += 32 * KB) {
    uint4 v[KB];
#pragma unroll
    for (int i = 0; i < KB; ++i) {
      const int u = u0 + 32 * i;
      if (u < n * CR) v[i] = *reinterpret_cast<const uint4*>(kn + (u / CR) * a.ds_tok + (u % CR) * 8);
    }
#pragma unroll
    for (int i = 0; i < KB; ++i) {
      const int u = u0 + 32 * i, t = u / CR, c = u % CR;
      if (u >= n * CR) continue;
      if constexpr (FORM == kDraftBf16) {
        *reinterpret_cast<uint4*>(kdst + kpage_chunk_offset_bf16(t, c, 64)) = v[i];
      } else {
        const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
        uint16_t q[4];
#pragma unroll
        for (int h = 0; h < 4; ++h)
          q[h] = pack_e4m3x2(__uint_as_float(w[h] << 16) * a.k_inv, __uint_as_float(w[h] & 0xffff0000u) * a.k_inv);
        if constexpr (FORM == kDraftE4m3)
          *reinterpret_cast<uint2*>(kdst + fp8_kpage_offset(t, c * 8, D)) =
              make_uint2(uint32_t(q[0]) | uint32_t(q[1]) << 16, uint32_t(q[2]) | uint32_t(q[3]) << 16);
        else
          *reinterpret_cast<uint4*>(kdst + kpage_chunk_offset_bf16(t, c, 64)) = make_uint4(
              e4m3x2_to_f16x2(q[0]), e4m3x2_to_f16x2(q[1]), e4m3x2_to_f16x2(q[2]), e4m3x2_to_f16x2(q[3]));
      }
    }
  }
}
template <int D, DraftForm FORM>
__device__ __forceinline__ void tree_draft_v(const TreeLaunch& a, const HeadDesc& hd, int n, uint8_t* vdst, int lane) {
  const __nv_bfloat16* vn =
      static_cast<const __nv_bfloat16*>(a.v_draft) + int64_t(hd.b) * a.ds_seq + int64_t(hd.kv) * a.ds_head;
  // A lane takes two dimensions of eight positions and writes a chunk of each, two such runs at a time: the loads'
  // latency counts (24 nodes over 64 heads: 47 us, one at a time 56).  In the E4M3 tcgen05 form, whose roles fill the
  // instruction cache, code that runs once or twice a CTA has to be short: one at a time its 32K layer takes 85 us, two
  // runs of sixteen positions 105.
  constexpr bool FP8 = FORM != kDraftBf16;
  constexpr int DP = D / 2;
#pragma unroll(FORM == kDraftWide ? 1 : 2)
  for (int u = lane; u < DP * 8; u += 32) {
    const int i = (u % DP) * 2, g = u / DP;
    const int t0 = FP8 ? (g >> 1) * 16 + (g & 1) * 4 : g * 8;  // E4M3: positions 8 ... 15 of 16 are 4 tokens behind
    uint32_t x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int t = t0 + (FP8 ? fp8_vpos_tok(e) : e);
      x[e] = t < n ? *reinterpret_cast<const uint32_t*>(vn + t * a.ds_tok + i) : 0u;
    }
#pragma unroll
    for (int y = 0; y < 2; ++y) {  // dimension i, dimension i + 1
      uint32_t w[4];
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        const uint32_t p = x[2 * h], r = x[2 * h + 1];
        if constexpr (FP8)
          w[h] = pack_e4m3x2(__uint_as_float(y ? p & 0xffff0000u : p << 16) * a.v_inv,
                             __uint_as_float(y ? r & 0xffff0000u : r << 16) * a.v_inv);
        else
          w[h] = __byte_perm(p, r, y ? 0x7632 : 0x5410);
      }
      if constexpr (FORM == kDraftE4m3)
        *reinterpret_cast<uint2*>(vdst + fp8_vpage_offset(i + y, g * 8)) =
            make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
      else if constexpr (FORM == kDraftWide)
        *reinterpret_cast<uint4*>(vdst + vpage_chunk_offset_bf16(i + y, g)) =
            make_uint4(e4m3x2_to_f16x2(uint16_t(w[0])), e4m3x2_to_f16x2(uint16_t(w[1])),
                       e4m3x2_to_f16x2(uint16_t(w[2])), e4m3x2_to_f16x2(uint16_t(w[3])));
      else
        *reinterpret_cast<uint4*>(vdst + vpage_chunk_offset_bf16(i + y, g)) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

template <int START, int MIN_UNITS>
struct TreeSplit {
  int64_t units;                             // U
  int32_t ctas;                              // G, <= the grid
  int32_t head;                              // head the CTA's range starts in ...
  int64_t head_unit;                         // ... and that head's first unit

  struct Weight {
    int32_t n;       // nodes of the sequence
    int32_t live;    // cached page records to visit
    int32_t pages;   // live + the draft's pages
    int32_t groups;  // row groups
    int64_t per;     // units of one row group
  };
  __device__ __forceinline__ static Weight weight(const TreeLaunch& a, int kind, int ctx_len, int n_vpages, int b,
                                                   bool* bad = nullptr) {
    Weight w;
    w.n = tree_nodes(a, b, bad);
    w.live = kind == 0 ? min(n_vpages, (ctx_len + a.P - 1) / a.P) : n_vpages;
    w.pages = w.live + (w.n + a.P - 1) / a.P;
    w.groups = (w.n + a.nodes_per_group - 1) / a.nodes_per_group;
    w.per = w.pages + START;
    return w;
  }
  __device__ __forceinline__ static int64_t head_units(const TreeLaunch& a, int h) {
    const HeadDesc* d = a.heads + h;
    const int b = h / a.num_kv_heads;  // heads are in (sequence, kv-head) order
    bool bad = false;
    const Weight w = weight(a, d->kind, d->ctx_len, d->n_vpages, b, &bad);
    if (bad && blockIdx.x == 0) record_error(a.status, kDevBadTree);
    return w.per * w.groups;
  }
  // (32-bit divisions where the line is short enough: a small call makes a dozen of them one after another)
  __device__ __forceinline__ bool small() const { return units < (1 << 22); }  // units x CTAs, and units more: < 2^32
  __device__ __forceinline__ int64_t cut(int64_t c) const {
    return small() ? int64_t(uint32_t(c) * uint32_t(units) / uint32_t(ctas)) : c * units / ctas;
  }
  __device__ __forceinline__ int cta_of(int64_t u) const {
    if (small()) return int((uint32_t(u + 1) * uint32_t(ctas) + uint32_t(units) - 1) / uint32_t(units)) - 1;
    return int(((u + 1) * ctas + units - 1) / units) - 1;
  }

  // All NT threads of the block.  scratch: NT / 32 + 2 int64 in shared memory.
  // Returns false when this CTA has no work.  Also lets the joining kernel's blocks be placed.
  template <int NT>
  __device__ bool init(const TreeLaunch& a, int64_t* scratch) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (threadIdx.x == 0) a.joins[blockIdx.x].n_pieces = 0;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr int NW = NT / 32;
    auto scan = [&](int64_t v, int64_t& total) {  // inclusive sum over the block
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += x;
      }
      if (lane == 31) scratch[warp] = v;
      __syncthreads();
      int64_t before = 0;
      total = 0;
#pragma unroll
      for (int i = 0; i < NW; ++i) {
        if (i < warp) before += scratch[i];
        total += scratch[i];
      }
      __syncthreads();
      return v + before;
    };
    // each thread takes a run of heads: one scan, and the thread whose run holds the CTA's first unit walks it again
    const int per = (a.n_heads + NT - 1) / NT, h0 = min(a.n_heads, int(threadIdx.x) * per),
              h1 = min(a.n_heads, h0 + per);
    int64_t mine = 0;
#pragma unroll 4
    for (int h = h0; h < h1; ++h) mine += head_units(a, h);
    const int64_t upto = scan(mine, units);
    ctas = int(min(int64_t(gridDim.x), max(int64_t(1), units / MIN_UNITS)));
    if (units == 0 || int(blockIdx.x) >= ctas) return false;
    const int64_t u0 = cut(blockIdx.x);
    if (u0 < upto && u0 >= upto - mine) {
      int64_t u = upto - mine;
      for (int h = h0; h < h1; ++h) {
        const int64_t w = head_units(a, h);
        if (u0 < u + w) {
          scratch[NW] = h, scratch[NW + 1] = u;
          break;
        }
        u += w;
      }
    }
    __syncthreads();
    head = int32_t(scratch[NW]);
    head_unit = scratch[NW + 1];
    return true;
  }

  struct Piece {
    HeadDesc hd;
    int32_t head, group;
    int32_t n;             // nodes of the sequence
    int32_t node0, nodes;  // the row group's nodes
    int32_t live;          // cached records; page index >= live: draft page
    int32_t p0, p1;        // pages [p0, p1) of live + draft
    int32_t n_pieces;      // CTAs sharing the row group
    int32_t first_cta;     // the first of them
    int32_t first_slot;    // its slot
    int32_t slot;          // this piece's slot
  };
  struct Walk {
    int64_t u, u1, head_unit;
    int32_t head;
  };
  __device__ __forceinline__ Walk walk() const {
    return Walk{cut(blockIdx.x), cut(blockIdx.x + 1), head_unit, head};
  }
  // The CTA's next piece (uniform over the threads); false: no more.
  __device__ __forceinline__ bool next(const TreeLaunch& a, Walk& w, Piece& pc) const {
    while (w.u < w.u1) {
      pc.hd = a.heads[w.head];
      const Weight g = weight(a, pc.hd.kind, pc.hd.ctx_len, pc.hd.n_vpages, pc.hd.b);
      const int64_t local = w.u - w.head_unit, end = g.per * g.groups;
      if (local >= end) {
        w.head_unit += end;
        ++w.head;
        continue;
      }
      const int32_t group = int32_t(local / g.per);
      const int64_t x = local - group * g.per, y = min(g.per, x + (w.u1 - w.u));
      const int64_t at = w.u - x;  // the row group's first unit
      w.u += y - x;
      if (y <= START) continue;  // only the fixed cost falls into this CTA: the next one takes all pages
      pc.head = w.head;
      pc.group = group;
      pc.n = g.n;
      pc.node0 = group * a.nodes_per_group;
      pc.nodes = min(a.nodes_per_group, g.n - pc.node0);
      pc.live = g.live;
      pc.p0 = int32_t(max(int64_t(0), x - START));
      pc.p1 = int32_t(y - START);
      pc.first_cta = cta_of(at + START);
      pc.n_pieces = cta_of(at + g.per - 1) - pc.first_cta + 1;
      pc.first_slot = 2 * pc.first_cta + (cut(pc.first_cta) < at ? 1 : 0);
      pc.slot = int(blockIdx.x) == pc.first_cta ? pc.first_slot : 2 * int(blockIdx.x);
      return true;
    }
    return false;
  }
};

// A partial slot: the accumulators in chunks of four columns, [D / 4][rows][4],
// then (m, l) of each row.  (A thread holds a row, or eight lanes hold eight: in
// row order a warp's store would touch a line a row.)  16-byte aligned.
__device__ __forceinline__ int64_t tree_slot_floats(const TreeLaunch& a) {
  return partial_slot_floats(a.nodes_per_group * a.group, a.D);
}
__device__ __forceinline__ int64_t tree_acc_at(int row, int col, int rows_max) {
  return (int64_t(col >> 2) * rows_max + row) * 4 + (col & 3);
}

// A piece as the producer warp hands it to the others, a slot ahead, so that
// nobody else waits for the table: the table's entries, the sequence's checked
// parents and the number of ring stages used before it.  head < 0: no more.
template <typename Piece>
struct TreePieceInfo {
  Piece pc;
  int32_t stage0;
  int8_t up[kMaxTreeNodes];
};
// The producer warp's writing of it (the caller signals it).
template <typename Piece>
__device__ __forceinline__ void tree_publish(const TreeLaunch& a, const Piece& pc, int stage0, int lane,
                                             TreePieceInfo<Piece>& out) {
#pragma unroll
  for (int x = 0; x < 2; ++x)
    out.up[lane + 32 * x] = int8_t(tree_parent(a, pc.hd.b, pc.n, lane + 32 * x));
  if (lane == 0) out.pc = pc, out.stage0 = stage0;
  __syncwarp();
}

// What the joining kernel needs of this CTA: the row group that starts in it
// and goes on in the next one (a CTA starts one such group at most: its last
// piece's).  One thread, at every piece; n_pieces 0: none.
template <typename Piece>
__device__ __forceinline__ void tree_note_join(const TreeLaunch& a, const Piece& pc) {
  if (pc.n_pieces == 1 || pc.first_cta != int(blockIdx.x)) return;
  a.joins[blockIdx.x] =
      TreeJoin{pc.n_pieces, pc.first_slot, pc.nodes * a.group, pc.hd.b, pc.hd.kv, pc.node0, {0, 0}};
}

// ---- joining pieces ---------------------------------------------------------
// With m_i, l_i, acc_i the running maximum (log2 domain), sum and unnormalised
// output of piece i:  M = max m_i,  O = sum 2^(m_i - M) acc_i / sum 2^(m_i - M) l_i,
// in an order that the pieces' numbers fix, so the same inputs give the same bits.
constexpr int kJoinBatch = 4;  // pieces a thread asks for at once
constexpr int kJoinCols = 16;  // columns of a thread

// Pieces part, part + parts, ... of a row's columns 16 cg ...: a batch's loads go out together, one rescale a batch.
template <int D>
__device__ __forceinline__ void tree_sum_pieces(const TreeLaunch& a, int n_pieces, int first_slot, int first_cta,
                                                int row, int cg, int part, int parts, float& m, float& l,
                                                float (&acc)[kJoinCols]) {
  const int rows_max = a.nodes_per_group * a.group;
  const int64_t stride = tree_slot_floats(a);
  m = -INFINITY, l = 0.f;
#pragma unroll
  for (int e = 0; e < kJoinCols; ++e) acc[e] = 0.f;
  for (int i0 = part; i0 < n_pieces; i0 += kJoinBatch * parts) {
    float2 ml[kJoinBatch];
    float4 x[kJoinBatch][kJoinCols / 4];
    float top = m;
#pragma unroll
    for (int u = 0; u < kJoinBatch; ++u) {
      const int i = i0 + u * parts;
      ml[u] = make_float2(-INFINITY, 0.f);
      if (i >= n_pieces) continue;
      const float* s = a.partial + int64_t(i == 0 ? first_slot : 2 * (first_cta + i)) * stride;
      ml[u] = __ldcg(reinterpret_cast<const float2*>(s + rows_max * D + 2 * row));
#pragma unroll
      for (int c = 0; c < kJoinCols / 4; ++c)
        x[u][c] = __ldcg(reinterpret_cast<const float4*>(s + tree_acc_at(row, cg * kJoinCols + 4 * c, rows_max)));
    }
#pragma unroll
    for (int u = 0; u < kJoinBatch; ++u) top = fmaxf(top, ml[u].x);
    const float base = top == -INFINITY ? 0.f : top, f0 = exp2f(m - base);
    m = top;
    l *= f0;
#pragma unroll
    for (int e = 0; e < kJoinCols; ++e) acc[e] *= f0;
#pragma unroll
    for (int u = 0; u < kJoinBatch; ++u) {
      if (i0 + u * parts >= n_pieces) continue;
      const float f = exp2f(ml[u].x - base);
      l += f * ml[u].y;
#pragma unroll
      for (int c = 0; c < kJoinCols / 4; ++c) {
        acc[4 * c] += f * x[u][c].x, acc[4 * c + 1] += f * x[u][c].y;
        acc[4 * c + 2] += f * x[u][c].z, acc[4 * c + 3] += f * x[u][c].w;
      }
    }
  }
}

// Output row of row `row` of a group that starts at node node0 of (b, kv).
__device__ __forceinline__ int64_t tree_out_row(const TreeLaunch& a, int b, int kv, int node0, int row) {
  return (int64_t(b) * a.T + node0 + row / a.group) * a.num_q_heads + kv * a.group + row % a.group;
}
// A finished row's columns 16 cg ..., and with the first of them its LSE.
template <typename T, int D>
__device__ __forceinline__ void tree_finish_row(const TreeLaunch& a, int64_t at, int cg, float m, float l,
                                                const float (&acc)[kJoinCols]) {
  const float inv = a.v_scale / l;
  T* dst = static_cast<T*>(a.out) + at * D + cg * kJoinCols;
  if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int e = 0; e < kJoinCols; e += 8)
      reinterpret_cast<uint4*>(dst)[e / 8] = make_uint4(
          pack_bf16x2(acc[e] * inv, acc[e + 1] * inv), pack_bf16x2(acc[e + 2] * inv, acc[e + 3] * inv),
          pack_bf16x2(acc[e + 4] * inv, acc[e + 5] * inv), pack_bf16x2(acc[e + 6] * inv, acc[e + 7] * inv));
  } else {
#pragma unroll
    for (int e = 0; e < kJoinCols; e += 4)
      reinterpret_cast<float4*>(dst)[e / 4] =
          make_float4(acc[e] * inv, acc[e + 1] * inv, acc[e + 2] * inv, acc[e + 3] * inv);
  }
  if (cg == 0 && a.lse) a.lse[at] = (m + log2f(l)) * kTreeLn2;
}

// Short calls (TreeLaunch::tickets): the CTA that publishes a group's last piece
// joins it, behind its own pieces, of which two at most are parts of a group.
struct TreeJoinsHere {
  int n;
  int first_cta[2];
  TreeJoin join[2];
};
// One thread, behind a fence and a barrier of the block's stores; also returns the counter to zero.
template <typename Piece>
__device__ __forceinline__ void tree_take_ticket(const TreeLaunch& a, const Piece& pc, TreeJoinsHere* here) {
  int32_t* c = a.tickets + int64_t(pc.head) * kMaxTreeNodes + pc.group;
  if (atomicAdd(c, 1) != pc.n_pieces - 1) return;
  *c = 0;
  const int i = here->n++;
  here->first_cta[i] = pc.first_cta;
  here->join[i] = TreeJoin{pc.n_pieces, pc.first_slot, pc.nodes * a.group, pc.hd.b, pc.hd.kv, pc.node0, {0, 0}};
}
template <typename T, int D>
__device__ __forceinline__ void tree_join_here(const TreeLaunch& a, const TreeJoinsHere& here, int tid, int threads) {
  __threadfence();
  for (int i = 0; i < here.n; ++i) {
    const TreeJoin& jn = here.join[i];
    for (int e = tid; e < jn.rows * (D / kJoinCols); e += threads) {
      const int row = e % jn.rows, cg = e / jn.rows;
      float m, l, acc[kJoinCols];
      tree_sum_pieces<D>(a, jn.n_pieces, jn.first_slot, here.first_cta[i], row, cg, 0, 1, m, l, acc);
      tree_finish_row<T, D>(a, tree_out_row(a, jn.b, jn.kv, jn.node0, row), cg, m, l, acc);
    }
  }
}

}  // namespace sp
