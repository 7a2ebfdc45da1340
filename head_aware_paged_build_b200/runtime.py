"""PyTorch-facing wrapper of one SegPaged layer (buffers + calls, nothing else).

``SegPagedLayer`` owns the device buffers a plan needs (table blob, K/V
pools, workspace) as PyTorch tensors and forwards to the C ABI.  It performs
no arithmetic of the method: planning, packing and attention all run in
libsegpaged.so.
"""
from __future__ import annotations

from typing import Sequence

import torch

from . import segpaged as S


def _on(device: torch.device, stream):
    """Context: ``stream`` (a torch stream, a raw handle, or None: the device's current stream) is current."""
    if stream is None:
        return torch.cuda.stream(torch.cuda.current_stream(device))
    return torch.cuda.stream(stream if isinstance(stream, torch.cuda.Stream) else
                             torch.cuda.ExternalStream(int(stream), device=device))


def _stream(stream) -> int:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _current_raw_stream(index: int) -> int:
    """Handle of device ``index``'s current stream, without building a stream object (5 us a call)."""
    return torch._C._cuda_getCurrentRawStream(index)


class SegPagedLayer:
    """Plan + device buffers of one attention layer's batch.

    ``policy`` holds ``(kind, sink, window)`` per (sequence, kv-head) with kind
    in {"global", "local", "dense"}, or ``("retrieval", sink, window, top_p)``;
    ``block_mass`` gives each retrieval head's importance per page-size block
    (None for other heads); ``q_start[b]`` is the position of the first query
    of sequence b (``ctx_len[b] - 1`` for decode).
    """

    def __init__(self, *, batch: int, num_q_heads: int, num_kv_heads: int, head_dim: int, page_size: int,
                 dtype: str, ctx_len: Sequence[int], q_start: Sequence[int],
                 policy: Sequence[tuple], device="cuda", flags: int = 0,
                 page_ids: Sequence[int] | None = None, first_page: int = 0, target_ctas: int = 0,
                 append_capacity: int = 0, pools: tuple[torch.Tensor, torch.Tensor] | None = None,
                 kv_dtype: str | None = None, k_scale: float = 1.0, v_scale: float = 1.0,
                 block_mass: Sequence | None = None, spare_pages: int = 0):
        self.dtype = dtype
        self.torch_dtype = {"f32": torch.float32, "bf16": torch.bfloat16}[dtype]
        self.num_q_heads, self.num_kv_heads, self.head_dim = num_q_heads, num_kv_heads, head_dim
        self.device = torch.device(device)
        self.problem = S.make_problem(batch, num_q_heads, num_kv_heads, head_dim, page_size, dtype, ctx_len,
                                      q_start, policy, first_page, page_ids, target_ctas, flags, append_capacity,
                                      kv_dtype, k_scale, v_scale, block_mass, spare_pages)
        self.kv_dtype = kv_dtype or dtype
        self.batch = batch
        self.ctx_len = [int(x) for x in ctx_len]
        self.plan = S.segpaged_plan_create(self.problem)
        self.sizes = S.segpaged_plan_sizes(self.plan)
        z = self.sizes
        self.table = torch.empty(z.table_bytes, dtype=torch.uint8, device=self.device)
        S.segpaged_table_write(self.plan, self.table.data_ptr(), z.table_bytes, _stream(None))
        if pools is None:
            nbytes = z.pool_pages * z.page_bytes
            self.k_pool = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=self.device)
            self.v_pool = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=self.device)
        else:
            self.k_pool, self.v_pool = pools
        self.workspace = torch.zeros(z.workspace_bytes, dtype=torch.uint8, device=self.device)
        self.index = self.k_pool.device.index
        self.tree_workspaces: list[torch.Tensor] = []  # of tree_attention; the last is in use
        self.tree_nodes = 0  # nodes the last of them covers

    # -- argument checks (the C ABI sees only pointers and strides) ------------
    def _check_tensor(self, t: torch.Tensor, what: str, dtype: torch.dtype) -> None:
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{what} must be a torch.Tensor")
        if t.dtype != dtype:
            raise TypeError(f"{what} must be {dtype}, got {t.dtype}")
        if t.device != self.k_pool.device:
            raise ValueError(f"{what} is on {t.device}, the layer's buffers on {self.k_pool.device}")

    def _check_dense(self, k: torch.Tensor, v: torch.Tensor, varlen: bool, what: str,
                     dtype: torch.dtype | None = None) -> None:
        """Dense K/V (or gather targets): every row the plan reads or writes must lie inside."""
        dtype = dtype or self.torch_dtype
        self._check_tensor(k, f"{what} K", dtype)
        self._check_tensor(v, f"{what} V", dtype)
        if k.shape != v.shape or k.stride() != v.stride() or k.stride(-1) != 1:
            raise ValueError(f"{what}: K and V need the same shape and strides, head_dim contiguous")
        d, hkv = self.head_dim, self.num_kv_heads
        if varlen:
            ok = k.dim() == 3 and k.shape[0] >= sum(self.ctx_len) and k.shape[1] >= hkv and k.shape[2] == d
            want = f"[>= {sum(self.ctx_len)}, >= {hkv}, {d}]"
        else:
            ok = (k.dim() == 4 and k.shape[0] >= self.batch and k.shape[1] >= hkv and
                  k.shape[2] >= max(self.ctx_len) and k.shape[3] == d)
            want = f"[>= {self.batch}, >= {hkv}, >= {max(self.ctx_len)}, {d}]"
        if not ok:
            raise ValueError(f"{what}: K/V shape {tuple(k.shape)} does not cover {want}")

    # -- calls --------------------------------------------------------------
    def build(self, k_dense: torch.Tensor, v_dense: torch.Tensor, varlen: bool = False, stream=None) -> None:
        """Pack dense K/V ([B, Hkv, Lmax, d], or varlen [sum L, Hkv, d] with varlen=True)."""
        self._check_dense(k_dense, v_dense, varlen, "build")
        if varlen:
            ss, sh, st = S.SP_VARLEN, k_dense.stride(1), k_dense.stride(0)
        else:
            ss, sh, st = k_dense.stride(0), k_dense.stride(1), k_dense.stride(2)
        S.build_segpaged_cache(self.plan, self.table.data_ptr(), k_dense.data_ptr(), v_dense.data_ptr(), ss, sh,
                               st, self.k_pool.data_ptr(), self.v_pool.data_ptr(), _stream(stream))

    def gather(self, k_out: torch.Tensor, v_out: torch.Tensor, varlen: bool = False, stream=None) -> None:
        """Write every stored row back to its dense position (the inverse of build).

        E4M3 pages give their 1-byte codes: k_out / v_out are then torch.uint8."""
        self._check_dense(k_out, v_out, varlen, "gather", torch.uint8 if self.kv_dtype == "e4m3" else None)
        if varlen:
            ss, sh, st = S.SP_VARLEN, k_out.stride(1), k_out.stride(0)
        else:
            ss, sh, st = k_out.stride(0), k_out.stride(1), k_out.stride(2)
        S.segpaged_gather(self.plan, self.table.data_ptr(), self.k_pool.data_ptr(), self.v_pool.data_ptr(),
                          k_out.data_ptr(), v_out.data_ptr(), ss, sh, st, _stream(stream))

    def attention(self, q: torch.Tensor, out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                  scale: float = 0.0, with_lse: bool = True, stream=None):
        """q: [sum C_b, Hq, d] contiguous; returns (out, lse)."""
        rows = (self.sizes.num_queries, self.num_q_heads)
        self._check_tensor(q, "q", self.torch_dtype)
        if tuple(q.shape) != rows + (self.head_dim,) or not q.is_contiguous():
            raise ValueError(f"q must be contiguous {rows + (self.head_dim,)}, got {tuple(q.shape)}")
        if out is None:
            out = torch.empty_like(q)
        self._check_tensor(out, "out", self.torch_dtype)
        if out.shape != q.shape or not out.is_contiguous():
            raise ValueError(f"out must be contiguous {tuple(q.shape)}, got {tuple(out.shape)}")
        if lse is None and with_lse:
            lse = torch.empty(q.shape[0], q.shape[1], dtype=torch.float32, device=q.device)
        if lse is not None:
            self._check_tensor(lse, "lse", torch.float32)
            if tuple(lse.shape) != rows or not lse.is_contiguous():
                raise ValueError(f"lse must be contiguous {rows}, got {tuple(lse.shape)}")
        S.segpaged_attention(self.plan, self.table.data_ptr(), self.k_pool.data_ptr(), self.v_pool.data_ptr(),
                             q.data_ptr(), out.data_ptr(), lse.data_ptr() if lse is not None else None, scale,
                             self.workspace.data_ptr(), self.workspace.numel(), _stream(stream))
        return out, lse

    def _check_new_rows(self, k_new: torch.Tensor, v_new: torch.Tensor) -> None:
        self._check_tensor(k_new, "k_new", self.torch_dtype)
        self._check_tensor(v_new, "v_new", self.torch_dtype)
        if (k_new.dim() != 3 or k_new.shape != v_new.shape or k_new.stride() != v_new.stride() or
                k_new.stride(-1) != 1 or k_new.shape[0] < self.batch or k_new.shape[1] < self.num_kv_heads or
                k_new.shape[2] != self.head_dim):
            raise ValueError(f"k_new / v_new must be [{self.batch}, {self.num_kv_heads}, {self.head_dim}] "
                             f"with the same strides, head_dim contiguous; got {tuple(k_new.shape)}")

    def append(self, k_new: torch.Tensor, v_new: torch.Tensor, stream=None) -> None:
        """Ring plans: add one token per sequence (k_new, v_new: [B, Hkv, d])."""
        self._check_new_rows(k_new, v_new)
        S.segpaged_decode_append(self.plan, self.table.data_ptr(), k_new.data_ptr(), v_new.data_ptr(),
                                 k_new.stride(0), k_new.stride(1), self.k_pool.data_ptr(), self.v_pool.data_ptr(),
                                 self.workspace.data_ptr(), _stream(stream))

    def decode_step(self, k_new: torch.Tensor, v_new: torch.Tensor, q: torch.Tensor, out: torch.Tensor | None = None,
                    lse: torch.Tensor | None = None, scale: float = 0.0, stream=None):
        """Ring plans: append one token per sequence and attend with its queries (q: [B, Hq, d]) in one call;
        the same results as ``append`` followed by ``attention``.  Returns (out, lse)."""
        self._check_new_rows(k_new, v_new)
        rows = (self.sizes.num_queries, self.num_q_heads)
        self._check_tensor(q, "q", self.torch_dtype)
        if tuple(q.shape) != rows + (self.head_dim,) or not q.is_contiguous():
            raise ValueError(f"q must be contiguous {rows + (self.head_dim,)}, got {tuple(q.shape)}")
        out = torch.empty_like(q) if out is None else out
        self._check_tensor(out, "out", self.torch_dtype)
        if out.shape != q.shape or not out.is_contiguous():
            raise ValueError(f"out must be contiguous {tuple(q.shape)}, got {tuple(out.shape)}")
        lse = torch.empty(rows, dtype=torch.float32, device=q.device) if lse is None else lse
        self._check_tensor(lse, "lse", torch.float32)
        if tuple(lse.shape) != rows or not lse.is_contiguous():
            raise ValueError(f"lse must be contiguous {rows}, got {tuple(lse.shape)}")
        S.segpaged_decode_step(self.plan, self.table.data_ptr(), k_new.data_ptr(), v_new.data_ptr(), k_new.stride(0),
                               k_new.stride(1), self.k_pool.data_ptr(), self.v_pool.data_ptr(), q.data_ptr(),
                               out.data_ptr(), lse.data_ptr(), scale, self.workspace.data_ptr(),
                               self.workspace.numel(), _stream(stream))
        return out, lse

    # -- several candidates a sequence -------------------------------------------
    def prepare_tree(self, max_nodes: int, workspace: torch.Tensor | None = None) -> None:
        """Allocate the workspace of ``tree_attention`` for trees of up to ``max_nodes`` nodes, or take ``workspace``.

        A call makes it when it is missing; a CUDA graph capture needs it made before.  Workspaces
        that a larger one replaced are kept: a captured graph may hold their addresses.  Layers whose calls
        never overlap on the GPU, as those of one model, can use one: ``workspace`` is a zero-filled
        uint8 tensor, or another layer's ``tree_workspaces[-1]`` (the layers then share its status too)."""
        if workspace is not None:
            self._check_tensor(workspace, "workspace", torch.uint8)
            need = S.segpaged_tree_workspace(self.plan, max_nodes)
            if not workspace.is_contiguous() or workspace.data_ptr() % 256 or workspace.numel() < need:
                raise ValueError(f"workspace must be contiguous, 256-byte aligned and hold {need} bytes for "
                                 f"{max_nodes} nodes, got {workspace.numel()}")
            if not any(workspace is ws for ws in self.tree_workspaces[-1:]):
                self.tree_workspaces.append(workspace)
            self.tree_nodes = max_nodes
            return
        if 1 <= max_nodes <= self.tree_nodes:
            return
        if 1 <= max_nodes <= S.SP_TREE_MAX_NODES:  # trees that grow node by node need few workspaces
            max_nodes = (max_nodes + 15) // 16 * 16
        need = S.segpaged_tree_workspace(self.plan, max_nodes)
        if not self.tree_workspaces or self.tree_workspaces[-1].numel() < need:  # larger trees may need no more bytes
            if torch.cuda.is_current_stream_capturing():
                raise RuntimeError("call prepare_tree(max_nodes) before a CUDA graph capture")
            device = self.k_pool.device
            self.tree_workspaces.append(torch.zeros(need, dtype=torch.uint8, device=device))
            torch.cuda.current_stream(device).synchronize()  # zeroed before any stream's call uses it
        self.tree_nodes = max_nodes

    def _elsewhere(self, stream) -> bool:
        """Does a call have to be made under another current device or stream?"""
        if isinstance(stream, torch.cuda.Stream) and stream.device != self.k_pool.device:
            raise ValueError(f"the stream is on {stream.device}, the layer's buffers on {self.k_pool.device}")
        return stream is not None or torch.cuda.current_device() != self.index

    def _check_draft(self, k: torch.Tensor, v: torch.Tensor, nodes: int) -> None:
        self._check_tensor(k, "k_draft", self.torch_dtype)
        self._check_tensor(v, "v_draft", self.torch_dtype)
        want = (self.batch, nodes, self.num_kv_heads, self.head_dim)
        strides = k.stride()
        if k.shape != want or v.shape != want or strides != v.stride() or strides[-1] != 1:
            raise ValueError(f"k_draft / v_draft must be {want} with the same strides, head_dim contiguous; got "
                             f"{tuple(k.shape)} and {tuple(v.shape)}")

    def _check_index(self, t: torch.Tensor, what: str, *shape: int) -> None:
        self._check_tensor(t, what, torch.int32)
        if t.shape != shape or not t.is_contiguous():
            raise ValueError(f"{what} must be contiguous {shape}, got {tuple(t.shape)}")

    def tree_attention(self, q: torch.Tensor, k_draft: torch.Tensor, v_draft: torch.Tensor, parents: torch.Tensor,
                       num_nodes: torch.Tensor | None = None, out: torch.Tensor | None = None,
                       lse: torch.Tensor | None = None, scale: float = 0.0, stream=None):
        """Attention of a drafted tree a sequence over the cache and over the draft itself.

        ``q``: contiguous [B, T, Hq, d], one row a node; ``k_draft`` / ``v_draft``: [B, T, Hkv, d], the
        nodes' own keys and values (not in the cache); ``parents``: int32 [B, T], -1 for a root, else an
        earlier node; ``num_nodes``: int32 [B] or None (T each).  Node i at depth d stands at position
        L + d and sees the cache by its head's rule, its ancestors and itself.  Returns (out, lse); rows
        behind ``num_nodes[b]`` are left as they were (in fresh outputs: zero).  T is at most 64.  The
        layer's calls share its workspaces: they must not overlap on the GPU.  After a device status of a
        wait that ran out (codes 1 to 4) call ``clear_device_status`` before the next one."""
        self._check_tensor(q, "q", self.torch_dtype)
        T = q.shape[1] if q.dim() == 4 else 0
        if not 1 <= T <= S.SP_TREE_MAX_NODES or not q.is_contiguous() or \
                q.shape != (self.batch, T, self.num_q_heads, self.head_dim):
            raise ValueError(f"q must be contiguous [{self.batch}, 1 .. {S.SP_TREE_MAX_NODES}, {self.num_q_heads}, "
                             f"{self.head_dim}], got {tuple(q.shape)}")
        rows = (self.batch, T, self.num_q_heads)
        self._check_draft(k_draft, v_draft, T)
        self._check_index(parents, "parents", self.batch, T)
        if num_nodes is not None:
            self._check_index(num_nodes, "num_nodes", self.batch)
        if out is not None:
            self._check_tensor(out, "out", self.torch_dtype)
            if out.shape != q.shape or not out.is_contiguous():
                raise ValueError(f"out must be contiguous {tuple(q.shape)}, got {tuple(out.shape)}")
        if lse is not None:
            self._check_tensor(lse, "lse", torch.float32)
            if lse.shape != rows or not lse.is_contiguous():
                raise ValueError(f"lse must be contiguous {rows}, got {tuple(lse.shape)}")
        if self._elsewhere(stream):  # fresh outputs and workspaces belong to the call's stream
            with _on(self.k_pool.device, stream):
                return self.tree_attention(q, k_draft, v_draft, parents, num_nodes, out, lse, scale)
        fresh = torch.empty if num_nodes is None else torch.zeros
        if out is None:
            out = fresh(q.shape, dtype=q.dtype, device=q.device)
        if lse is None:
            lse = fresh(rows, dtype=torch.float32, device=q.device)
        self.prepare_tree(T)
        ws = self.tree_workspaces[-1]
        S.segpaged_tree_attention(self.plan, self.table.data_ptr(), self.k_pool.data_ptr(), self.v_pool.data_ptr(),
                                  q.data_ptr(), k_draft.data_ptr(), v_draft.data_ptr(), k_draft.stride(0),
                                  k_draft.stride(1), k_draft.stride(2), parents.data_ptr(),
                                  num_nodes.data_ptr() if num_nodes is not None else None, T, out.data_ptr(),
                                  lse.data_ptr(), scale, ws.data_ptr(), ws.numel(), _current_raw_stream(self.index))
        return out, lse

    def tree_commit(self, k_draft: torch.Tensor, v_draft: torch.Tensor, path: torch.Tensor, path_len: torch.Tensor,
                    stream=None) -> None:
        """Ring plans: append the accepted nodes ``path[b, :path_len[b]]`` of the draft to each sequence.

        ``k_draft`` / ``v_draft`` as in ``tree_attention``; ``path``: int32 [B, M], ``path_len``: int32 [B]
        in [0, M].  The cache ends as after that many ``append`` calls."""
        if not isinstance(k_draft, torch.Tensor) or k_draft.dim() != 4:
            raise ValueError("k_draft must be a [B, T, Hkv, d] tensor")
        self._check_draft(k_draft, v_draft, k_draft.shape[1])
        if not isinstance(path, torch.Tensor) or path.dim() != 2:
            raise ValueError("path must be an int32 [B, M] tensor")
        self._check_index(path, "path", self.batch, path.shape[1])
        self._check_index(path_len, "path_len", self.batch)
        if self._elsewhere(stream):
            with _on(self.k_pool.device, stream):
                return self.tree_commit(k_draft, v_draft, path, path_len)
        S.segpaged_tree_commit(self.plan, self.table.data_ptr(), k_draft.data_ptr(), v_draft.data_ptr(),
                               k_draft.stride(0), k_draft.stride(1), k_draft.stride(2), k_draft.shape[1],
                               path.data_ptr(), path_len.data_ptr(), path.shape[1], self.k_pool.data_ptr(),
                               self.v_pool.data_ptr(), self.workspace.data_ptr(), _current_raw_stream(self.index))

    def reorder(self, parents: torch.Tensor, common_len: torch.Tensor | None = None, stream=None) -> None:
        """Ring plans: sequence b goes on with the cache of sequence ``parents[b]`` (int32 [B]), in place.

        Forks, beam reorderings, any map; ``common_len`` (int32 [B]): positions below it are known equal in
        both and not copied.  b and ``parents[b]`` need the same policies and ``ctx_len`` page counts."""
        self._check_index(parents, "parents", self.batch)
        if common_len is not None:
            self._check_index(common_len, "common_len", self.batch)
        if self._elsewhere(stream):
            with _on(self.k_pool.device, stream):
                return self.reorder(parents, common_len)
        S.segpaged_reorder(self.plan, self.table.data_ptr(), parents.data_ptr(),
                           common_len.data_ptr() if common_len is not None else None, self.k_pool.data_ptr(),
                           self.v_pool.data_ptr(), self.workspace.data_ptr(), _current_raw_stream(self.index))

    def device_status(self, stream=None) -> int:
        """The first recorded code of the layer's workspaces (0: none)."""
        code = S.segpaged_read_device_status(self.workspace.data_ptr(), _stream(stream))
        for ws in self.tree_workspaces:
            code = code or S.segpaged_read_device_status(ws.data_ptr(), _stream(stream))
        return code

    def clear_device_status(self, stream=None) -> None:
        """Zero the layer's workspaces: the recorded codes, and the counters that a wait which ran out may have
        left behind (``segpaged_clear_device_status`` clears the code of one workspace alone).  None of the
        layer's calls may be running on another stream."""
        with _on(self.k_pool.device, stream):
            for ws in (self.workspace, *self.tree_workspaces):
                ws.zero_()

    def close(self) -> None:
        if getattr(self, "plan", None):
            S.segpaged_plan_destroy(self.plan)
            self.plan = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def layer_for(prob, device="cuda", flags: int = 0, **kw) -> SegPagedLayer:
    """A SegPagedLayer for a ``workloads.Problem``."""
    wl = prob.wl
    if "block_mass" not in kw and wl.has_retrieval:
        kw["block_mass"] = prob.block_masses()
    return SegPagedLayer(batch=wl.batch, num_q_heads=wl.num_q_heads, num_kv_heads=wl.num_kv_heads,
                         head_dim=wl.head_dim, page_size=wl.page_size, dtype=wl.dtype, ctx_len=prob.ctx_lens,
                         q_start=prob.q_starts, policy=wl.policy, device=device, flags=flags, **kw)


def block_mass(k_dense: torch.Tensor, q: torch.Tensor, ctx_len: Sequence[int], page_size: int = 64,
               scale: float = 0.0, stream=None) -> torch.Tensor:
    """The attention mass per page-size block of each (sequence, kv-head): the importance a retrieval
    head's top-p selection reads (``segpaged_block_mass``).

    ``k_dense``: bf16 [B, Hkv, Lmax, d] (d contiguous, rows 16-byte aligned); ``q``: bf16 [B, Hq, d]
    contiguous, each sequence's queries at its last position ``ctx_len[b] - 1``.  Returns fp32
    [B, Hkv, ceil(Lmax / page_size)] on k's device; row (b, kv) holds ceil(ctx_len[b] / page_size)
    masses summing to 1, zeros after them.  ``[m[b, kv, :n].tolist() ...]`` are the ``block_mass``
    entries a plan takes.
    """
    B, hkv, lmax, d = k_dense.shape
    if k_dense.dtype != torch.bfloat16 or q.dtype != torch.bfloat16:
        raise ValueError("block_mass: bf16 keys and queries")
    if k_dense.stride(-1) != 1 or not q.is_contiguous() or tuple(q.shape[::2]) != (B, d) or q.shape[1] % hkv:
        raise ValueError(f"block_mass: q must be contiguous [{B}, Hq, {d}] with Hq a multiple of {hkv}")
    if len(ctx_len) != B or max(ctx_len) > lmax or min(ctx_len) < 1:
        raise ValueError("block_mass: one ctx_len in [1, Lmax] per sequence")
    hq = q.shape[1]
    prob = S.make_problem(B, hq, hkv, d, page_size, "bf16", ctx_len, [L - 1 for L in ctx_len],
                          [("global", 0, 0)] * (B * hkv))
    nb = -(-lmax // page_size)
    out = torch.zeros(B, hkv, nb, dtype=torch.float32, device=k_dense.device)
    ws = torch.empty(S.segpaged_block_mass_workspace(prob), dtype=torch.uint8, device=k_dense.device)
    S.segpaged_block_mass(prob, k_dense.data_ptr(), k_dense.stride(0), k_dense.stride(1), k_dense.stride(2),
                          q.data_ptr(), scale, out.data_ptr(), nb, ws.data_ptr(), ws.numel(), _stream(stream))
    return out


def build_layers(layers: Sequence[SegPagedLayer], k_dense: Sequence[torch.Tensor], v_dense: Sequence[torch.Tensor],
                 varlen: bool = False, stream=None) -> None:
    """Pack several layers that share one pair of pools with a single launch.

    ``layers[i]`` packs ``k_dense[i]`` / ``v_dense[i]`` (all with the same strides); the
    layers must hold the same pools (``pools=`` at construction, distinct ``first_page``).
    """
    if not (len(layers) == len(k_dense) == len(v_dense)) or not layers:
        raise ValueError("build_layers: one dense K and one dense V per layer, at least one layer")
    k0 = k_dense[0]
    if varlen:
        ss, sh, st = S.SP_VARLEN, k0.stride(1), k0.stride(0)
    else:
        ss, sh, st = k0.stride(0), k0.stride(1), k0.stride(2)
    for lay, k, v in zip(layers, k_dense, v_dense):
        lay._check_dense(k, v, varlen, "build_layers")
        if k.stride() != k0.stride():
            raise ValueError("build_layers: every layer's dense K/V needs the same strides")
        if (lay.k_pool.data_ptr() != layers[0].k_pool.data_ptr() or
                lay.v_pool.data_ptr() != layers[0].v_pool.data_ptr()):
            raise ValueError("build_layers: the layers must share the pools")
    S.build_segpaged_cache_layers([lay.plan for lay in layers], [lay.table.data_ptr() for lay in layers],
                                  [k.data_ptr() for k in k_dense], [v.data_ptr() for v in v_dense], ss, sh, st,
                                  layers[0].k_pool.data_ptr(), layers[0].v_pool.data_ptr(), _stream(stream))


class DecodeStepGraph:
    """One serving decode step of a ring-plan layer, captured once in a CUDA graph.

    A step copies the new token's K and V rows ([B, Hkv, d]) and its queries
    ([B, Hq, d]) from the pinned host buffers ``k_in``, ``v_in``, ``q_in``,
    appends the token and runs decode attention (``segpaged_decode_step``: one
    launch on bf16 pages; with ``fused=False`` the two calls
    ``segpaged_decode_append`` and ``segpaged_attention``) and copies O and
    LSE into the pinned host buffers ``out`` and ``lse``.  The caller refills
    the inputs, then calls ``replay()``; every replay appends one more token
    (the device table advances in place).  The graph holds the same library
    calls an eager step makes; it removes the per-call launch gaps between them.
    """

    def __init__(self, layer: SegPagedLayer, stream: torch.cuda.Stream | None = None, fused: bool = True):
        if layer.problem.flags & S.SP_FLAG_RING == 0:
            raise ValueError("DecodeStepGraph needs a ring plan (flags=SP_FLAG_RING)")
        if not layer.sizes.is_decode:
            raise ValueError("DecodeStepGraph needs a decode plan")
        B, Hkv, Hq, d = layer.problem.batch, layer.num_kv_heads, layer.num_q_heads, layer.head_dim
        dt, dev = layer.torch_dtype, layer.device
        self.layer = layer
        # Inputs and outputs each live in one staging buffer (host and device), so a
        # step moves them with one copy each way; the named tensors are views.
        eb = torch.empty((), dtype=dt).element_size()
        kb, qb = B * Hkv * d * eb, B * Hq * d * eb
        self._host_in = torch.empty(2 * kb + qb, dtype=torch.uint8).pin_memory()
        self._dev_in = torch.empty(2 * kb + qb, dtype=torch.uint8, device=dev)
        self._host_out = torch.empty(qb + B * Hq * 4, dtype=torch.uint8).pin_memory()
        self._dev_out = torch.empty(qb + B * Hq * 4, dtype=torch.uint8, device=dev)

        def views(buf, shapes):
            out, off = [], 0
            for shape, t in shapes:
                n = int(torch.Size(shape).numel()) * torch.empty((), dtype=t).element_size()
                out.append(buf[off:off + n].view(t).view(shape))
                off += n
            return out

        ins = [((B, Hkv, d), dt), ((B, Hkv, d), dt), ((B, Hq, d), dt)]
        outs = [((B, Hq, d), dt), ((B, Hq), torch.float32)]
        self.k_in, self.v_in, self.q_in = views(self._host_in, ins)
        self._k, self._v, self._q = views(self._dev_in, ins)
        self.out, self.lse = views(self._host_out, outs)
        self._o, self._lse = views(self._dev_out, outs)
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph, stream=stream):
            self._dev_in.copy_(self._host_in, non_blocking=True)
            if fused:
                layer.decode_step(self._k, self._v, self._q, self._o, self._lse)
            else:
                layer.append(self._k, self._v)
                layer.attention(self._q, self._o, self._lse)
            self._host_out.copy_(self._dev_out, non_blocking=True)

    def replay(self) -> None:
        self.graph.replay()
