// Device entry points that decode several candidates at once: tree attention,
// tree commit and reorder.  As in api.cu, every argument is checked on the
// host before anything is launched.
#include <algorithm>
#include <limits>
#include <string>

#include "kernels.h"
#include "sp_internal.h"

namespace sp {
namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

sp_status cuda_fail(cudaError_t e, const char* what) {
  return fail(SP_ERR_CUDA, std::string(what) + ": " + cudaGetErrorString(e));
}

template <typename T>
T* section(const void* d_table, int64_t off) {
  return reinterpret_cast<T*>(const_cast<uint8_t*>(static_cast<const uint8_t*>(d_table)) + off);
}

// Workspace: status block | descriptions of split row groups, one a CTA |
// tickets (the same place whatever the tree's size, so that calls of different
// sizes leave each other's at zero) | two partial slots a CTA.
constexpr int64_t kTreeTicketOffset = kStatusBytes + (kTreeMaxCtas * int64_t(sizeof(TreeJoin)) + 255) / 256 * 256;
constexpr int64_t kTreePartialOffset = kTreeTicketOffset + kTreeHeadsHere * kMaxTreeNodes * 4;

int64_t tree_workspace_bytes(const sp_plan* plan, int32_t nodes) {
  const TreeConfig c = tree_config(plan, nodes);
  const int64_t slot = partial_slot_floats(c.rows_per_group, plan->prob.head_dim) * 4;
  return kTreePartialOffset + (2 * int64_t(c.n_ctas) * slot + 255) / 256 * 256;
}

sp_status check_tree_plan(const sp_plan* plan, int32_t nodes) {
  if (!plan) return fail(SP_ERR_INVALID_ARG, "plan is NULL");
  if (!plan->sizes.is_decode) return fail(SP_ERR_INVALID_ARG, "tree attention needs a decode plan");
  if (nodes < 1) return fail(SP_ERR_INVALID_ARG, "a tree needs at least one node");
  if (nodes > kMaxTreeNodes)
    return fail(SP_ERR_UNSUPPORTED, "at most " + std::to_string(kMaxTreeNodes) + " nodes a tree");
  if (int64_t(plan->prob.batch) * nodes > std::numeric_limits<int32_t>::max())
    return fail(SP_ERR_UNSUPPORTED, "batch * nodes above 2^31");
  return SP_OK;
}

sp_status check_draft(const sp_plan* plan, const void* k, const void* v, int64_t ss, int64_t st, int64_t sh) {
  if (!k || !v || !aligned(k, 16) || !aligned(v, 16))
    return fail(SP_ERR_INVALID_ARG, "k_draft and v_draft must be non-NULL and 16-byte aligned");
  const int64_t eb = plan->elem_bytes;
  if (ss < 0 || st < 0 || sh < 0 || (ss * eb) % 16 || (st * eb) % 16 || (sh * eb) % 16)
    return fail(SP_ERR_INVALID_ARG, "draft strides must be >= 0 and give 16-byte aligned rows");
  return SP_OK;
}

}  // namespace
}  // namespace sp

extern "C" {

sp_status segpaged_tree_workspace(const sp_plan* plan, int32_t max_nodes, size_t* bytes) {
  using namespace sp;
  if (!bytes) return fail(SP_ERR_INVALID_ARG, "bytes must be non-NULL");
  const sp_status st = check_tree_plan(plan, max_nodes);
  if (st != SP_OK) return st;
  int64_t need = 0;  // row groups grow with the tree, but not evenly: the largest of all smaller trees too
  for (int32_t n = 1; n <= max_nodes; ++n) need = std::max(need, tree_workspace_bytes(plan, n));
  *bytes = size_t(need);
  return SP_OK;
}

sp_status segpaged_tree_attention(const sp_plan* plan, const void* d_table, const void* k_pool, const void* v_pool,
                                  const void* q, const void* k_draft, const void* v_draft, int64_t stride_seq,
                                  int64_t stride_tok, int64_t stride_head, const int32_t* parents,
                                  const int32_t* num_nodes, int32_t nodes, void* out, float* lse, float softmax_scale,
                                  void* workspace, size_t workspace_bytes, void* stream) {
  using namespace sp;
  sp_status st = check_tree_plan(plan, nodes);
  if (st != SP_OK) return st;
  st = check_attention_args(plan, d_table, k_pool, v_pool, q, out, lse, softmax_scale);
  if (st != SP_OK) return st;
  st = check_draft(plan, k_draft, v_draft, stride_seq, stride_tok, stride_head);
  if (st != SP_OK) return st;
  if (!parents || !aligned(parents, 4) || !aligned(num_nodes, 4))
    return fail(SP_ERR_INVALID_ARG, "parents must be non-NULL; parents and num_nodes 4-byte aligned");
  if (!workspace || !aligned(workspace, 256)) return fail(SP_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  if (int64_t(workspace_bytes) < tree_workspace_bytes(plan, nodes))
    return fail(SP_ERR_WORKSPACE, "workspace smaller than segpaged_tree_workspace gives");
  const TreeConfig c = tree_config(plan, nodes);
  TreeLaunch L{};
  L.heads = section<HeadDesc>(d_table, plan->hdr.off_heads);
  L.pages = section<PageDesc>(d_table, plan->hdr.off_pages);
  L.n_heads = plan->hdr.n_heads;
  L.num_kv_heads = plan->prob.num_kv_heads, L.num_q_heads = plan->prob.num_q_heads, L.group = plan->group;
  L.D = plan->prob.head_dim, L.P = plan->prob.page_size;
  L.bf16 = plan->prob.dtype == SP_BF16, L.fp8 = plan->fp8;
  L.page_bytes = plan->sizes.page_bytes, L.pool_pages = plan->sizes.pool_pages;
  L.kpool = k_pool, L.vpool = v_pool, L.q = q, L.k_draft = k_draft, L.v_draft = v_draft;
  L.ds_seq = stride_seq, L.ds_tok = stride_tok, L.ds_head = stride_head;
  L.parents = parents, L.num_nodes = num_nodes, L.T = nodes;
  L.out = out, L.lse = lse;
  L.scale_log2 = softmax_scale_of(plan, softmax_scale) * 1.4426950408889634f * plan->k_scale;
  L.v_scale = plan->v_scale;
  L.k_inv = 1.0f / plan->k_scale, L.v_inv = 1.0f / plan->v_scale;
  L.nodes_per_group = c.nodes_per_group, L.nodes_per_tile = c.nodes_per_tile, L.n_ctas = c.n_ctas;
  L.partial = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kTreePartialOffset);
  L.joins = reinterpret_cast<TreeJoin*>(static_cast<uint8_t*>(workspace) + kStatusBytes);
  if (c.joins_here) L.tickets = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(workspace) + kTreeTicketOffset);
  L.status = static_cast<int32_t*>(workspace);
  cudaError_t e = launch_tree(L, c, static_cast<cudaStream_t>(stream));
  if (e == cudaSuccess && !c.joins_here) e = launch_tree_join(L, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? SP_OK : cuda_fail(e, "segpaged_tree_attention launch");
}

sp_status segpaged_tree_commit(const sp_plan* plan, void* d_table, const void* k_draft, const void* v_draft,
                               int64_t stride_seq, int64_t stride_tok, int64_t stride_head, int32_t nodes,
                               const int32_t* path, const int32_t* path_len, int32_t max_path, void* k_pool,
                               void* v_pool, void* workspace, void* stream) {
  using namespace sp;
  sp_status st = check_table(plan, d_table);
  if (st != SP_OK) return st;
  if (!(plan->prob.flags & SP_FLAG_RING)) return fail(SP_ERR_INVALID_ARG, "segpaged_tree_commit needs a ring plan");
  if (nodes < 1 || max_path < 1) return fail(SP_ERR_INVALID_ARG, "nodes and max_path must be >= 1");
  if (nodes > kMaxTreeNodes || max_path > kMaxTreeNodes)
    return fail(SP_ERR_UNSUPPORTED, "at most " + std::to_string(kMaxTreeNodes) + " nodes a tree or path");
  st = check_draft(plan, k_draft, v_draft, stride_seq, stride_tok, stride_head);
  if (st != SP_OK) return st;
  if (!path || !path_len || !aligned(path, 4) || !aligned(path_len, 4))
    return fail(SP_ERR_INVALID_ARG, "path and path_len must be non-NULL and 4-byte aligned");
  if (!k_pool || !v_pool || !aligned(k_pool, 16) || !aligned(v_pool, 16))
    return fail(SP_ERR_INVALID_ARG, "pools must be non-NULL and 16-byte aligned");
  if (!workspace || !aligned(workspace, 256)) return fail(SP_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  CommitLaunch L{};
  L.heads = section<HeadDesc>(d_table, plan->hdr.off_heads);
  L.pages = section<PageDesc>(d_table, plan->hdr.off_pages);
  L.n_heads = plan->hdr.n_heads, L.num_kv_heads = plan->prob.num_kv_heads;
  L.D = plan->prob.head_dim, L.P = plan->prob.page_size;
  L.bf16 = plan->prob.dtype == SP_BF16, L.fp8 = plan->fp8;
  L.k_inv = 1.0f / plan->k_scale, L.v_inv = 1.0f / plan->v_scale;
  L.ds_seq = stride_seq, L.ds_tok = stride_tok, L.ds_head = stride_head;
  L.page_bytes = plan->sizes.page_bytes, L.pool_pages = plan->sizes.pool_pages;
  L.k_draft = k_draft, L.v_draft = v_draft;
  L.path = path, L.path_len = path_len, L.max_path = max_path, L.n_nodes = nodes;
  L.kpool = k_pool, L.vpool = v_pool;
  L.status = static_cast<int32_t*>(workspace);
  L.free_pool = section<int32_t>(d_table, plan->hdr.off_free);
  const cudaError_t e = launch_commit(L, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? SP_OK : cuda_fail(e, "segpaged_tree_commit launch");
}

sp_status segpaged_reorder(const sp_plan* plan, void* d_table, const int32_t* parents, const int32_t* common_len,
                           void* k_pool, void* v_pool, void* workspace, void* stream) {
  using namespace sp;
  sp_status st = check_table(plan, d_table);
  if (st != SP_OK) return st;
  if (!(plan->prob.flags & SP_FLAG_RING)) return fail(SP_ERR_INVALID_ARG, "segpaged_reorder needs a ring plan");
  if (!parents || !aligned(parents, 4) || !aligned(common_len, 4))
    return fail(SP_ERR_INVALID_ARG, "parents must be non-NULL; parents and common_len 4-byte aligned");
  if (!k_pool || !v_pool || !aligned(k_pool, 16) || !aligned(v_pool, 16))
    return fail(SP_ERR_INVALID_ARG, "pools must be non-NULL and 16-byte aligned");
  if (!workspace || !aligned(workspace, 256)) return fail(SP_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  const int B = plan->prob.batch, H = plan->prob.num_kv_heads;
  if (B > kReorderMaxBatch || H > kReorderMaxKvHeads)
    return fail(SP_ERR_UNSUPPORTED, "reorder: at most " + std::to_string(kReorderMaxBatch) + " sequences and " +
                                        std::to_string(kReorderMaxKvHeads) + " kv-heads");
  ReorderLaunch L{};
  L.heads = section<HeadDesc>(d_table, plan->hdr.off_heads);
  L.pages = section<PageDesc>(d_table, plan->hdr.off_pages);
  L.batch = B, L.num_kv_heads = H;
  L.page_bytes = plan->sizes.page_bytes, L.pool_pages = plan->sizes.pool_pages;
  L.parents = parents, L.common_len = common_len;
  L.kpool = static_cast<uint8_t*>(k_pool), L.vpool = static_cast<uint8_t*>(v_pool);
  L.status = static_cast<int32_t*>(workspace);
  L.free_pool = section<int32_t>(d_table, plan->hdr.off_free);
  int64_t recs = 0;
  for (int kv = 0; kv < H; ++kv) {
    int32_t most = 0;
    for (int b = 0; b < B; ++b) most = std::max(most, plan->heads[b * H + kv].n_vpages);
    L.rec_begin[kv] = int32_t(recs);
    recs += most;
    if (recs > std::numeric_limits<int32_t>::max()) return fail(SP_ERR_UNSUPPORTED, "more than 2^31 records");
  }
  L.rec_begin[H] = int32_t(recs);
  for (int b = 0; b < B; ++b) L.layout[b] = uint16_t(plan->layout[b]);
  const cudaError_t e = launch_reorder(L, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? SP_OK : cuda_fail(e, "segpaged_reorder launch");
}

}  // extern "C"
