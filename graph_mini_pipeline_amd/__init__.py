"""graph_mini_pipeline_amd -- Python binding of libgnnmb.so, the MI355X (gfx950) GNN mini-batch path.

Argument marshalling only: torch tensors become device pointers and the current torch stream
becomes the hipStream_t.  Every step of the path (sampling, relabel, gather, aggregation) runs in
the library's HIP kernels; torch supplies device memory and streams.  The functions carry the C
names of include/gnnmb.h and raise GnnError on a negative status.
"""
from __future__ import annotations

import contextlib
import ctypes
from dataclasses import dataclass, field
from typing import List, Optional, Sequence

import torch

from . import _abi
from ._abi import (GNN_ERR_CAPACITY, GNN_ERR_HIP, GNN_ERR_INTERNAL, GNN_ERR_INVALID_ARG,  # noqa
                   GNN_ERR_OUT_OF_RANGE, GNN_ERR_UNSUPPORTED, GNN_MAX_HOPS, GNN_OK, GNN_SYNC,
                   GNN_SUPERBATCH_COMPACT, GNN_SUPERBATCH_FULL, GNN_GATHER_BATCHED,
                   GNN_NOALLOC_MAX_IDS, GNN_NOALLOC_SCRATCH_BYTES, GNN_RELABEL_SORT, GNN_RELABEL_BITMAP, GNN_SAMPLE_EXACT_RANK,
                   GNN_GATHER_INTERLEAVED,
                   GNN_TIMER_STAGES)

__all__ = [
    "GnnError", "DeviceGraph", "Blocks", "MinibatchOut", "FeatureStore", "Timer", "Options",
    "gnn_status_string", "gnn_batch_seed", "gnn_capacity", "gnn_workspace_size", "gnn_sample_khop",
    "gnn_unique_relabel", "gnn_relabel_workspace_size", "gnn_feature_store_create",
    "gnn_feature_store_destroy", "gnn_gather_features", "gnn_mean_aggregate", "gnn_sage_layer",
    "gnn_sage_update", "gnn_minibatch", "gnn_unique_relabel_noalloc", "AdjacencyCache", "gnn_adjacency_cache_create",
    "gnn_host_mapped_pointer",
    "gnn_embedding_lookup", "gnn_embedding_grad", "gnn_embedding_grad_rows",
    "gnn_embedding_grad_workspace_size", "gnn_orthogonalize", "gnn_orthogonalize_workspace_size",
    "gnn_cross_attention", "gnn_cross_attention_backward", "gnn_cross_attention_workspace_size",
    "gnn_layer_norm", "gnn_layer_norm_backward", "gnn_layer_norm_workspace_size",
    "gnn_linear", "gnn_linear_backward", "gnn_linear_workspace_size",
    "gnn_gated_linear", "gnn_gated_linear_backward", "gnn_gated_linear_workspace_size",
    "gnn_read_device_status", "gnn_timer_create", "gnn_timer_destroy", "gnn_timer_reset",
    "gnn_timer_elapsed", "gnn_copy_probe", "gnn_copy_probe_host", "gnn_hash_probe", "lib",
]

lib = _abi.lib


class GnnError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = status
        super().__init__(f"{what}: {gnn_status_string(status)} ({status})")


def _ok(status: int, what: str) -> None:
    if status != GNN_OK:
        raise GnnError(status, what)


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    return ctypes.c_void_p(t.data_ptr())


# The current stream's handle without a Stream object around it (3 us of a short call), where torch has it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        device = torch.cuda.current_device()      # initialises the device, or says why it cannot
        if _raw_stream is not None:
            return ctypes.c_void_p(_raw_stream(device))
        stream = torch.cuda.current_stream(device)
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


def _need(t: torch.Tensor, dtype, name: str, device=True) -> None:
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    if device and not t.is_cuda:
        raise ValueError(f"{name}: must be a device tensor")


def gnn_status_string(status: int) -> str:
    return lib().gnn_status_string(status).decode()


def gnn_batch_seed(rng_seed: int, b: int) -> int:
    return int(lib().gnn_batch_seed(rng_seed & 0xFFFFFFFFFFFFFFFF, b))


@dataclass
class Options:
    group_max_deg: int = 0
    wave_max_deg: int = 0
    sync: bool = False
    superbatch: str = "auto"    # super-batch relabel: "auto", "full" or "compact"
    gather: str = "auto"        # gather and outermost mean: "auto", "interleaved" or "batched"
    relabel: str = "auto"       # short id lists: "auto", "sort" (whenever eligible) or "bitmap"
    exact_rank: bool = False    # rank every node's candidates by the full (key, position) order
    d_hits: Optional[torch.Tensor] = None   # int64 [1] device: rows read from the HBM caches

    def c(self) -> _abi.gnn_options:
        o = _abi.gnn_options()
        if self.d_hits is not None:
            _need(self.d_hits, torch.int64, "d_hits")
            o.d_hits = self.d_hits.data_ptr()
        o.group_max_deg = self.group_max_deg
        o.wave_max_deg = self.wave_max_deg
        modes = {"auto": 0, "full": GNN_SUPERBATCH_FULL, "compact": GNN_SUPERBATCH_COMPACT}
        if self.superbatch not in modes:
            raise ValueError(f"superbatch must be one of {sorted(modes)}")
        gmodes = {"auto": 0, "interleaved": GNN_GATHER_INTERLEAVED, "batched": GNN_GATHER_BATCHED}
        if self.gather not in gmodes:
            raise ValueError(f"gather must be one of {sorted(gmodes)}")
        rmodes = {"auto": 0, "sort": GNN_RELABEL_SORT, "bitmap": GNN_RELABEL_BITMAP}
        if self.relabel not in rmodes:
            raise ValueError(f"relabel must be one of {sorted(rmodes)}")
        o.flags = (GNN_SYNC if self.sync else 0) | modes[self.superbatch] | gmodes[self.gather] | \
            rmodes[self.relabel] | (GNN_SAMPLE_EXACT_RANK if self.exact_rank else 0)
        return o


def gnn_host_mapped_pointer(t: torch.Tensor) -> int:
    """The device address of a pinned host tensor's memory."""
    if t.is_cuda or not t.is_pinned():
        raise ValueError("expected a pinned host tensor")
    out = ctypes.c_void_p()
    _ok(lib().gnn_host_mapped_pointer(_ptr(t), ctypes.byref(out)), "gnn_host_mapped_pointer")
    return int(out.value)


@dataclass
class DeviceGraph:
    """CSR by destination: indptr (int32 or int64) in device memory; indices (int32) in device
    memory or in pinned host memory (read in place); optionally an HBM adjacency cache."""
    num_nodes: int
    indptr: torch.Tensor
    indices: torch.Tensor
    adjacency: Optional["AdjacencyCache"] = None

    def c(self) -> _abi.gnn_graph:
        host = not self.indices.is_cuda
        _need(self.indices, torch.int32, "indices", device=not host)
        if host and self.indices.numel() and not self.indices.is_pinned():
            raise ValueError("host-resident indices must be pinned")
        if self.indptr.dtype not in (torch.int32, torch.int64) or not self.indptr.is_cuda:
            raise TypeError("indptr: int32 or int64 device tensor")
        g = _abi.gnn_graph()
        g.num_nodes = self.num_nodes
        g.num_edges = self.indices.numel()
        g.indptr = self.indptr.data_ptr()
        g.indptr_bytes = self.indptr.element_size()
        if not self.indices.numel():
            g.indices = None
        elif host:
            g.indices = gnn_host_mapped_pointer(self.indices)
        else:
            g.indices = self.indices.data_ptr()
        if self.adjacency is not None:
            _ok(lib().gnn_adjacency_cache_attach(self.adjacency.handle, ctypes.byref(g)),
                "gnn_adjacency_cache_attach")
        return g


class AdjacencyCache:
    """Owns a gnn_adjacency_cache handle (the HBM copies of hot adjacency rows)."""

    def __init__(self, handle: ctypes.c_void_p, rows: int, entries: int):
        self.handle = handle
        self.rows = rows
        self.entries = entries

    def close(self):
        if self.handle:
            lib().gnn_adjacency_cache_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def gnn_adjacency_cache_create(graph: DeviceGraph, hot_order: torch.Tensor,
                               max_entries: int) -> AdjacencyCache:
    """HBM copies of the rows of hot_order (device int32, hottest first) that fit max_entries
    neighbour ids; attach it with DeviceGraph(..., adjacency=cache)."""
    _need(hot_order, torch.int32, "hot_order")
    bare = DeviceGraph(graph.num_nodes, graph.indptr, graph.indices)
    g = bare.c()
    h = ctypes.c_void_p()
    rows, entries = ctypes.c_int64(), ctypes.c_int64()
    _ok(lib().gnn_adjacency_cache_create(ctypes.byref(g), _ptr(hot_order), hot_order.numel(),
                                         max_entries, ctypes.byref(h), ctypes.byref(rows),
                                         ctypes.byref(entries)),
        "gnn_adjacency_cache_create")
    return AdjacencyCache(h, rows.value, entries.value)


def gnn_capacity(n_seeds: int, fanouts: Sequence[int], num_nodes: int) -> _abi.gnn_caps:
    caps = _abi.gnn_caps()
    fo = (ctypes.c_int32 * len(fanouts))(*fanouts)
    _ok(lib().gnn_capacity(n_seeds, fo, len(fanouts), num_nodes, ctypes.byref(caps)), "gnn_capacity")
    return caps


def gnn_workspace_size(caps: _abi.gnn_caps, num_nodes: int, group: int = 1) -> int:
    n = ctypes.c_size_t(0)
    _ok(lib().gnn_workspace_size(ctypes.byref(caps), num_nodes, group, ctypes.byref(n)),
        "gnn_workspace_size")
    return int(n.value)


def gnn_relabel_workspace_size(id_bound: int) -> int:
    n = ctypes.c_size_t(0)
    _ok(lib().gnn_relabel_workspace_size(id_bound, ctypes.byref(n)), "gnn_relabel_workspace_size")
    return int(n.value)


class Blocks:
    """Device buffers of the K blocks of one batch, allocated at the given caps."""

    def __init__(self, caps: _abi.gnn_caps, device="cuda", stream=None):
        """`stream`: the stream the blocks are first written on.  The counts are zeroed by a kernel
        queued on it, so that the zeroing is ordered before that stream's calls (queued on the
        current stream instead, it could run after the counts of a call on a non-blocking side
        stream, and wipe them)."""
        self.caps = caps
        K = caps.num_hops
        i32 = torch.int32
        with torch.cuda.stream(stream) if stream is not None else contextlib.nullcontext():
            self.counts = torch.zeros(2 * K, dtype=torch.int64, device=device)
            self.indptr, self.gid, self.lid, self.dst_lid, self.nodes = [], [], [], [], []
            for l in range(K):
                self.indptr.append(torch.empty(caps.frontier[l] + 1, dtype=i32, device=device))
                self.gid.append(torch.empty(max(caps.edges[l], 1), dtype=i32, device=device))
                self.lid.append(torch.empty(max(caps.edges[l], 1), dtype=i32, device=device))
                self.dst_lid.append(torch.empty(max(caps.frontier[l], 1), dtype=i32, device=device))
                self.nodes.append(torch.empty(max(caps.nodes[l], 1), dtype=i32, device=device))

    def c(self) -> _abi.gnn_blocks:
        b = _abi.gnn_blocks()
        b.caps = self.caps
        for l in range(self.caps.num_hops):
            h = b.hop[l]
            h.indptr = self.indptr[l].data_ptr()
            h.gid = self.gid[l].data_ptr()
            h.lid = self.lid[l].data_ptr()
            h.dst_lid = self.dst_lid[l].data_ptr()
            h.nodes = self.nodes[l].data_ptr()
        b.counts = self.counts.data_ptr()
        return b

    def host(self):
        """Per-hop (indptr, gid, lid, dst_lid, nodes) trimmed to the device counts (syncs)."""
        cnt = self.counts.cpu().tolist()
        out = []
        F = self.caps.n_seeds
        for l in range(self.caps.num_hops):
            E, V = cnt[2 * l], cnt[2 * l + 1]
            out.append((self.indptr[l][:F + 1].cpu().numpy(), self.gid[l][:E].cpu().numpy(),
                        self.lid[l][:E].cpu().numpy(), self.dst_lid[l][:F].cpu().numpy(),
                        self.nodes[l][:V].cpu().numpy()))
            F = V
        return out


def gnn_sample_khop(graph: DeviceGraph, seeds: torch.Tensor, fanouts: Sequence[int], seed64: int,
                    blocks: Blocks, ws: torch.Tensor, opts: Optional[Options] = None,
                    stream=None) -> int:
    _need(seeds, torch.int32, "seeds")
    g = graph.c()
    b = blocks.c()
    fo = (ctypes.c_int32 * len(fanouts))(*fanouts)
    o = opts.c() if opts else None
    st = lib().gnn_sample_khop(ctypes.byref(g), _ptr(seeds) if seeds.numel() else None,
                               seeds.numel(), fo, len(fanouts), seed64 & 0xFFFFFFFFFFFFFFFF,
                               ctypes.byref(b), _ptr(ws), ws.numel() * ws.element_size(),
                               ctypes.byref(o) if o else None, _stream(stream))
    _ok(st, "gnn_sample_khop")
    return st


def gnn_unique_relabel(keep: torch.Tensor, add: torch.Tensor, id_bound: int, uniq: torch.Tensor,
                       d_n_uniq: torch.Tensor, add_lid: torch.Tensor, keep_lid: torch.Tensor,
                       ws: torch.Tensor, d_n_add: Optional[torch.Tensor] = None,
                       stream=None) -> None:
    for t, n in ((keep, "keep"), (add, "add"), (uniq, "uniq"), (add_lid, "add_lid"),
                 (keep_lid, "keep_lid")):
        _need(t, torch.int32, n)
    _need(d_n_uniq, torch.int64, "d_n_uniq")
    if add_lid.numel() < add.numel() or keep_lid.numel() < keep.numel():
        raise ValueError("add_lid / keep_lid shorter than add / keep")
    st = lib().gnn_unique_relabel(_ptr(keep), keep.numel(), _ptr(add), _ptr(d_n_add), add.numel(),
                                  id_bound, _ptr(uniq), uniq.numel(), _ptr(d_n_uniq), _ptr(add_lid),
                                  _ptr(keep_lid), _ptr(ws), ws.numel() * ws.element_size(),
                                  _stream(stream))
    _ok(st, "gnn_unique_relabel")


def gnn_unique_relabel_noalloc(keep: torch.Tensor, add: torch.Tensor, id_bound: int,
                               uniq: torch.Tensor, d_n_uniq: torch.Tensor, add_lid: torch.Tensor,
                               keep_lid: torch.Tensor, d_status: Optional[torch.Tensor] = None,
                               d_n_add: Optional[torch.Tensor] = None, stream=None) -> None:
    """gnn_unique_relabel on the library's fixed per-GPU scratch (no workspace, no allocation;
    id_bound <= GNN_NOALLOC_MAX_IDS; calls that overlap on one GPU race)."""
    for t, n in ((keep, "keep"), (add, "add"), (uniq, "uniq"), (add_lid, "add_lid"),
                 (keep_lid, "keep_lid")):
        _need(t, torch.int32, n)
    _need(d_n_uniq, torch.int64, "d_n_uniq")
    if d_status is not None:
        _need(d_status, torch.int32, "d_status")
    if add_lid.numel() < add.numel() or keep_lid.numel() < keep.numel():
        raise ValueError("add_lid / keep_lid shorter than add / keep")
    st = lib().gnn_unique_relabel_noalloc(_ptr(keep), keep.numel(), _ptr(add), _ptr(d_n_add),
                                          add.numel(), id_bound, _ptr(uniq), uniq.numel(),
                                          _ptr(d_n_uniq), _ptr(add_lid), _ptr(keep_lid),
                                          _ptr(d_status), _stream(stream))
    _ok(st, "gnn_unique_relabel_noalloc")


class FeatureStore:
    """Owns a gnn_feature_store handle; keeps the table (and hot order) tensors alive."""

    def __init__(self, handle: ctypes.c_void_p, table: torch.Tensor, d: int, ld: int):
        self.handle = handle
        self.table = table
        self.d = d
        self.ld = ld

    def close(self):
        if self.handle:
            lib().gnn_feature_store_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def gnn_feature_store_create(table: torch.Tensor, d: int, cache_rows: int = 0,
                             hot_order: Optional[torch.Tensor] = None) -> FeatureStore:
    """table: float32 [N, ld] on the device, or pinned host memory (table.is_pinned())."""
    on_host = not table.is_cuda
    if on_host and not table.is_pinned():
        raise ValueError("a host feature table must be pinned")
    _need(table, torch.float32, "table", device=not on_host)
    if hot_order is not None:
        _need(hot_order, torch.int32, "hot_order")
    h = ctypes.c_void_p()
    st = lib().gnn_feature_store_create(_ptr(table), 1 if on_host else 0, table.shape[0], d,
                                        table.shape[1], cache_rows, _ptr(hot_order),
                                        ctypes.byref(h))
    _ok(st, "gnn_feature_store_create")
    return FeatureStore(h, table, d, table.shape[1])


def gnn_feature_store_destroy(fs: FeatureStore) -> None:
    fs.close()


def gnn_feature_store_enable_dynamic(fs: FeatureStore, gamma: float, k_dyn: int, t_update: int,
                                     max_refreshes: int = 0, auto: bool = False) -> None:
    """GARDEN's Dynamic-Cache on the store: k_dyn more HBM rows for residual hot rows, ranked by
    the EWMA of their accesses (decay gamma) and refreshed every t_update mini-batches; frozen
    after max_refreshes refreshes (0: never).  auto: gathers refresh when due, on their stream."""
    p = _abi.gnn_dyn_cache_params(float(gamma), int(k_dyn), int(t_update), int(max_refreshes),
                                  _abi.GNN_DYN_AUTO if auto else 0)
    _ok(lib().gnn_feature_store_enable_dynamic(fs.handle, ctypes.byref(p)),
        "gnn_feature_store_enable_dynamic")
    fs.dynamic = dict(gamma=float(gamma), k_dyn=int(k_dyn), t_update=int(t_update),
                      max_refreshes=int(max_refreshes), auto=bool(auto))


def gnn_dyn_cache_update(fs: FeatureStore, d_status: Optional[torch.Tensor] = None,
                         stream=None) -> bool:
    """Refresh the Dynamic-Cache on the stream if one is due; True if it ran."""
    r = ctypes.c_int32(0)
    _ok(lib().gnn_dyn_cache_update(fs.handle, ctypes.byref(r), _ptr(d_status), _stream(stream)),
        "gnn_dyn_cache_update")
    return bool(r.value)


def gnn_dyn_cache_query(fs: FeatureStore) -> dict:
    """Dynamic-Cache counters (synchronises the device)."""
    info = _abi.gnn_dyn_cache_info()
    _ok(lib().gnn_dyn_cache_query(fs.handle, ctypes.byref(info)), "gnn_dyn_cache_query")
    return {name: getattr(info, name) for name, _ in info._fields_ if name != "reserved"}


def gnn_dyn_cache_state(fs: FeatureStore, score: Optional[torch.Tensor] = None,
                        member: Optional[torch.Tensor] = None, stream=None) -> None:
    """score: float64 [N] device (Score(v, t) after the last observed mini-batch); member: uint8
    [N] device (1: holds a Dynamic-Cache row)."""
    n = fs.table.shape[0]
    if score is not None:
        _need(score, torch.float64, "score")
        if score.numel() < n:
            raise ValueError("score: [num_nodes]")
    if member is not None:
        _need(member, torch.uint8, "member")
        if member.numel() < n:
            raise ValueError("member: [num_nodes]")
    _ok(lib().gnn_dyn_cache_state(fs.handle, _ptr(score), _ptr(member), _stream(stream)),
        "gnn_dyn_cache_state")


def gnn_gather_features(fs: FeatureStore, ids: torch.Tensor, out: torch.Tensor,
                        d_n: Optional[torch.Tensor] = None, d_hits: Optional[torch.Tensor] = None,
                        d_status: Optional[torch.Tensor] = None, stream=None) -> None:
    _need(ids, torch.int32, "ids")
    _need(out, torch.float32, "out")
    if out.dim() != 2 or out.shape[0] < ids.numel():
        raise ValueError("out: [>= len(ids), ld_out]")
    st = lib().gnn_gather_features(fs.handle, _ptr(ids), _ptr(d_n), ids.numel(), _ptr(out),
                                   out.shape[1], _ptr(d_hits), _ptr(d_status), _stream(stream))
    _ok(st, "gnn_gather_features")


def gnn_gather_features_match(fs: FeatureStore, ids: torch.Tensor, out: torch.Tensor,
                              prev_ids: torch.Tensor, prev_x: torch.Tensor, match: torch.Tensor,
                              d_n: Optional[torch.Tensor] = None,
                              d_prev_n: Optional[torch.Tensor] = None,
                              d_matched: Optional[torch.Tensor] = None,
                              d_hits: Optional[torch.Tensor] = None,
                              d_status: Optional[torch.Tensor] = None, stream=None) -> None:
    """gnn_gather_features, with the rows whose ids are in prev_ids (strictly ascending) copied from
    prev_x (row p = features of prev_ids[p]); match[i] receives p or -1."""
    _need(ids, torch.int32, "ids")
    _need(out, torch.float32, "out")
    _need(prev_ids, torch.int32, "prev_ids")
    _need(prev_x, torch.float32, "prev_x")
    _need(match, torch.int32, "match")
    if out.dim() != 2 or out.shape[0] < ids.numel() or match.numel() < ids.numel():
        raise ValueError("out: [>= len(ids), ld_out]; match: [>= len(ids)]")
    if prev_x.dim() != 2 or prev_x.shape[0] < prev_ids.numel():
        raise ValueError("prev_x: [>= len(prev_ids), ld_prev]")
    st = lib().gnn_gather_features_match(fs.handle, _ptr(ids), _ptr(d_n), ids.numel(), _ptr(out),
                                         out.shape[1], _ptr(prev_ids), _ptr(d_prev_n),
                                         prev_ids.numel(), _ptr(prev_x), prev_x.shape[1],
                                         _ptr(match), _ptr(d_matched), _ptr(d_hits),
                                         _ptr(d_status), _stream(stream))
    _ok(st, "gnn_gather_features_match")


def gnn_batch_overlap(lists: Sequence[torch.Tensor], out: torch.Tensor,
                      counts: Optional[Sequence[Optional[torch.Tensor]]] = None,
                      stream=None) -> None:
    """out[a * B + b] = |lists[a] ∩ lists[b]| (device int64 [B * B]); each list strictly ascending,
    counts[a] (device int64 [1]) its actual length if given, else the whole tensor."""
    B = len(lists)
    _need(out, torch.int64, "out")
    if out.numel() < B * B:
        raise ValueError("out: [B * B]")
    for t in lists:
        _need(t, torch.int32, "lists")
    ids = (ctypes.c_void_p * B)(*[t.data_ptr() if t.numel() else None for t in lists])
    dn = None
    if counts is not None:
        dn = (ctypes.c_void_p * B)(*[c.data_ptr() if c is not None else None for c in counts])
    n = (ctypes.c_int64 * B)(*[t.numel() for t in lists])
    _ok(lib().gnn_batch_overlap(ids, dn, n, B, _ptr(out), _stream(stream)), "gnn_batch_overlap")


def gnn_greedy_order(overlap, first: int = 0) -> List[int]:
    """Nearest-overlap-first order of B batches from their overlap matrix (host array-like B x B)."""
    import numpy as np
    m = np.ascontiguousarray(np.asarray(overlap, dtype=np.int64))
    B = m.shape[0]
    if m.shape != (B, B):
        raise ValueError("overlap: B x B")
    order = (ctypes.c_int32 * B)()
    _ok(lib().gnn_greedy_order(m.ctypes.data_as(ctypes.POINTER(ctypes.c_int64)), B, first, order),
        "gnn_greedy_order")
    return list(order)


def gnn_mean_aggregate(indptr: torch.Tensor, lid: torch.Tensor, src: torch.Tensor, d: int,
                       out: torch.Tensor, d_n_dst: Optional[torch.Tensor] = None,
                       d_status: Optional[torch.Tensor] = None, stream=None) -> None:
    _need(indptr, torch.int32, "indptr")
    _need(lid, torch.int32, "lid")
    _need(src, torch.float32, "src")
    _need(out, torch.float32, "out")
    n_dst = indptr.numel() - 1
    if out.shape[0] < n_dst:
        raise ValueError("out has fewer rows than destinations")
    st = lib().gnn_mean_aggregate(_ptr(indptr), _ptr(lid), lid.numel(), _ptr(d_n_dst), n_dst,
                                  _ptr(src), src.shape[1], src.shape[0], d, _ptr(out),
                                  out.shape[1], _ptr(d_status), _stream(stream))
    _ok(st, "gnn_mean_aggregate")


def gnn_sage_layer(indptr: torch.Tensor, lid: torch.Tensor, dst_lid: torch.Tensor,
                   src: torch.Tensor, d: int, W: torch.Tensor, bias: Optional[torch.Tensor],
                   relu: bool, agg: torch.Tensor, out: torch.Tensor,
                   d_n_dst: Optional[torch.Tensor] = None, d_status: Optional[torch.Tensor] = None,
                   stream=None) -> None:
    """One GraphSAGE-mean layer: agg = block means, out = act([src[dst_lid] || agg] @ W + bias).
    W: float32 [2d, d_out] contiguous; agg: [n_dst, >= d]; out: [n_dst, >= d_out]."""
    for t, n in ((indptr, "indptr"), (lid, "lid"), (dst_lid, "dst_lid")):
        _need(t, torch.int32, n)
    for t, n in ((src, "src"), (W, "W"), (agg, "agg"), (out, "out")):
        _need(t, torch.float32, n)
    if bias is not None:
        _need(bias, torch.float32, "bias")
    n_dst = indptr.numel() - 1
    if W.dim() != 2 or W.shape[0] != 2 * d or not W.is_contiguous():
        raise ValueError("W must be a contiguous [2d, d_out] tensor")
    d_out = W.shape[1]
    if bias is not None and bias.numel() < d_out:
        raise ValueError("bias shorter than d_out")
    if dst_lid.numel() < n_dst or agg.shape[0] < n_dst or out.shape[0] < n_dst:
        raise ValueError("dst_lid / agg / out have fewer rows than destinations")
    st = lib().gnn_sage_layer(_ptr(indptr), _ptr(lid), lid.numel(), _ptr(dst_lid), _ptr(d_n_dst),
                              n_dst, _ptr(src), src.shape[1], src.shape[0], d, _ptr(W),
                              _ptr(bias), d_out, 1 if relu else 0, _ptr(agg), agg.shape[1],
                              _ptr(out), out.shape[1], _ptr(d_status), _stream(stream))
    _ok(st, "gnn_sage_layer")


def gnn_sage_update(dst_lid: torch.Tensor, src: torch.Tensor, d: int, agg: torch.Tensor,
                    W: torch.Tensor, bias: Optional[torch.Tensor], relu: bool, out: torch.Tensor,
                    n_dst: Optional[int] = None, d_n_dst: Optional[torch.Tensor] = None,
                    d_status: Optional[torch.Tensor] = None, stream=None) -> None:
    """The UPDATE alone: out = act([src[dst_lid] || agg] @ W + bias) for n_dst rows (default:
    dst_lid.numel()); agg holds the means."""
    _need(dst_lid, torch.int32, "dst_lid")
    for t, n in ((src, "src"), (W, "W"), (agg, "agg"), (out, "out")):
        _need(t, torch.float32, n)
    if bias is not None:
        _need(bias, torch.float32, "bias")
    n = dst_lid.numel() if n_dst is None else n_dst
    if W.dim() != 2 or W.shape[0] != 2 * d or not W.is_contiguous():
        raise ValueError("W must be a contiguous [2d, d_out] tensor")
    d_out = W.shape[1]
    if bias is not None and bias.numel() < d_out:
        raise ValueError("bias shorter than d_out")
    if dst_lid.numel() < n or agg.shape[0] < n or out.shape[0] < n:
        raise ValueError("dst_lid / agg / out have fewer rows than destinations")
    st = lib().gnn_sage_update(_ptr(dst_lid), _ptr(d_n_dst), n, _ptr(src), src.shape[1],
                               src.shape[0], d, _ptr(agg), agg.shape[1], _ptr(W), _ptr(bias), d_out,
                               1 if relu else 0, _ptr(out), out.shape[1], _ptr(d_status),
                               _stream(stream))
    _ok(st, "gnn_sage_update")


class MinibatchOut:
    """Blocks plus X and h_0..h_{K-1} of one (sub-)batch."""

    def __init__(self, caps: _abi.gnn_caps, d: int, ld_h: Optional[int] = None, device="cuda",
                 stream=None):
        """`stream`: the stream the outputs are first written on (as for Blocks)."""
        self.blocks = Blocks(caps, device, stream)
        self.d = d
        self.ld_h = ld_h if ld_h is not None else (d + 3) // 4 * 4
        K = caps.num_hops
        f32 = torch.float32
        with torch.cuda.stream(stream) if stream is not None else contextlib.nullcontext():
            self.x = torch.empty(max(caps.nodes[K - 1], 1), self.ld_h, dtype=f32, device=device)
            self.h = [torch.empty(max(caps.n_seeds if l == 0 else caps.nodes[l - 1], 1), self.ld_h,
                                  dtype=f32, device=device) for l in range(K)]

    def c(self) -> _abi.gnn_minibatch_out:
        m = _abi.gnn_minibatch_out()
        m.blocks = self.blocks.c()
        m.x = self.x.data_ptr()
        for l, t in enumerate(self.h):
            m.h[l] = t.data_ptr()
        m.ld_h = self.ld_h
        return m


class Timer:
    def __init__(self, n_records: int):
        h = ctypes.c_void_p()
        _ok(lib().gnn_timer_create(n_records, ctypes.byref(h)), "gnn_timer_create")
        self.handle = h
        self.n_records = n_records

    def reset(self):
        _ok(lib().gnn_timer_reset(self.handle), "gnn_timer_reset")

    def elapsed(self):
        """List of per-call stage times in ms: [sample+relabel, gather, outer mean, other means]."""
        n = ctypes.c_int32(0)
        buf = (ctypes.c_float * (self.n_records * GNN_TIMER_STAGES))()
        _ok(lib().gnn_timer_elapsed(self.handle, ctypes.byref(n), buf), "gnn_timer_elapsed")
        k = GNN_TIMER_STAGES
        return [list(buf[r * k:(r + 1) * k]) for r in range(n.value)]

    def close(self):
        if self.handle:
            lib().gnn_timer_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def gnn_timer_create(n_records: int) -> Timer:
    return Timer(n_records)


def gnn_timer_destroy(t: Timer) -> None:
    t.close()


def gnn_timer_reset(t: Timer) -> None:
    t.reset()


def gnn_timer_elapsed(t: Timer):
    return t.elapsed()


def gnn_minibatch(graph: DeviceGraph, fs: FeatureStore, seeds: torch.Tensor,
                  batch_ptr: Sequence[int], fanouts: Sequence[int], seed64: int,
                  outs: List[MinibatchOut], ws: torch.Tensor, opts: Optional[Options] = None,
                  stream=None, timer: Optional[Timer] = None) -> int:
    _need(seeds, torch.int32, "seeds")
    G = len(batch_ptr) - 1
    if len(outs) != G:
        raise ValueError("one MinibatchOut per sub-batch")
    g = graph.c()
    bp = (ctypes.c_int64 * (G + 1))(*batch_ptr)
    fo = (ctypes.c_int32 * len(fanouts))(*fanouts)
    mo = (_abi.gnn_minibatch_out * G)(*[o.c() for o in outs])
    o = opts.c() if opts else None
    st = lib().gnn_minibatch(ctypes.byref(g), fs.handle, _ptr(seeds) if seeds.numel() else None,
                             bp, G, fo, len(fanouts), seed64 & 0xFFFFFFFFFFFFFFFF, mo, _ptr(ws),
                             ws.numel() * ws.element_size(), ctypes.byref(o) if o else None,
                             _stream(stream), timer.handle if timer else None)
    _ok(st, "gnn_minibatch")
    return st


_TYPES = {torch.float32: _abi.GNN_F32, torch.bfloat16: _abi.GNN_BF16}


def _type(dtype, name: str) -> int:
    t = _TYPES.get(dtype)
    if t is None:
        raise TypeError(f"{name}: expected float32 or bfloat16, got {dtype}")
    return t


def _need_rows(t: torch.Tensor, name: str) -> int:
    """Checks a device matrix of float32 or bfloat16 whose rows are contiguous; its element type."""
    kind = _type(t.dtype, name)
    if not t.is_cuda:
        raise ValueError(f"{name}: must be a device tensor")
    shape, stride = t.shape, t.stride()
    if len(shape) != 2 or (shape[1] > 1 and stride[1] != 1) or \
            (shape[0] > 1 and stride[0] < shape[1]):
        raise ValueError(f"{name}: must be a matrix with contiguous rows that do not overlap")
    return kind


def _ld(t: torch.Tensor) -> int:
    """Elements from one row of a matrix to the next."""
    shape = t.shape
    return t.stride()[0] if shape[0] > 1 else shape[1]


def gnn_embedding_lookup(table: torch.Tensor, ids: torch.Tensor, scale: float, out: torch.Tensor,
                         pad_id: int = -1, d_n: Optional[torch.Tensor] = None,
                         d_status: Optional[torch.Tensor] = None, stream=None) -> None:
    """out[i] = scale * table[ids[i]], a zero row where ids[i] == pad_id.  table: [num_rows, d],
    out: [>= len(ids), d], float32 or bfloat16 each."""
    _need(ids, torch.int32, "ids")
    tt, ot = _need_rows(table, "table"), _need_rows(out, "out")
    n, d = ids.numel(), table.shape[1]
    if out.shape[0] < n or out.shape[1] != d:
        raise ValueError("out: [>= len(ids), d]")
    if d_n is not None:
        _need(d_n, torch.int64, "d_n")
    if d_status is not None:
        _need(d_status, torch.int32, "d_status")
    _ok(lib().gnn_embedding_lookup(table.data_ptr(), tt, table.shape[0], d, _ld(table),
                                   ids.data_ptr(), _ptr(d_n), n, scale, pad_id, out.data_ptr(), ot,
                                   _ld(out), _ptr(d_status), _stream(stream)),
        "gnn_embedding_lookup")


def gnn_embedding_grad_workspace_size(n: int, num_rows: int, d: int) -> int:
    b = ctypes.c_size_t(0)
    _ok(lib().gnn_embedding_grad_workspace_size(n, num_rows, d, ctypes.byref(b)),
        "gnn_embedding_grad_workspace_size")
    return int(b.value)


def _need_grad(ids, dout, grad, d_n, d_status, ws):
    _need(ids, torch.int32, "ids")
    dt, gt = _need_rows(dout, "dout"), _need_rows(grad, "grad")
    if dout.shape[0] < ids.numel() or grad.shape[1] != dout.shape[1]:
        raise ValueError("dout: [>= len(ids), d]; grad: [*, d]")
    if d_n is not None:
        _need(d_n, torch.int64, "d_n")
    if d_status is not None:
        _need(d_status, torch.int32, "d_status")
    if not ws.is_cuda or not ws.is_contiguous():
        raise ValueError("ws: must be a contiguous device tensor")
    return dt, gt


def gnn_embedding_grad(ids: torch.Tensor, dout: torch.Tensor, scale: float, grad: torch.Tensor,
                       ws: torch.Tensor, pad_id: int = -1, accumulate: bool = False,
                       d_n: Optional[torch.Tensor] = None,
                       d_status: Optional[torch.Tensor] = None, stream=None) -> None:
    """grad[t] = scale * sum of dout[i] over ids[i] == t (accumulate: added to grad's rows), for the
    whole table grad [num_rows, d]."""
    dt, gt = _need_grad(ids, dout, grad, d_n, d_status, ws)
    _ok(lib().gnn_embedding_grad(ids.data_ptr(), _ptr(d_n), ids.numel(), dout.data_ptr(), dt,
                                 _ld(dout), scale, pad_id, grad.shape[0], grad.shape[1],
                                 grad.data_ptr(), gt, _ld(grad), 1 if accumulate else 0,
                                 _ptr(d_status), ws.data_ptr(), ws.numel() * ws.element_size(),
                                 _stream(stream)), "gnn_embedding_grad")


def gnn_embedding_grad_rows(ids: torch.Tensor, dout: torch.Tensor, scale: float, num_rows: int,
                            uniq: torch.Tensor, d_n_uniq: torch.Tensor, grad: torch.Tensor,
                            ws: torch.Tensor, pad_id: int = -1,
                            d_n: Optional[torch.Tensor] = None,
                            d_status: Optional[torch.Tensor] = None, stream=None) -> None:
    """The gradient rows of the distinct ids only: uniq (int32, ascending), d_n_uniq (int64 [1])
    their number, grad[p] the row of uniq[p]."""
    dt, gt = _need_grad(ids, dout, grad, d_n, d_status, ws)
    _need(uniq, torch.int32, "uniq")
    _need(d_n_uniq, torch.int64, "d_n_uniq")
    if grad.shape[0] < uniq.numel() or d_n_uniq.numel() < 1:
        raise ValueError("grad: [>= len(uniq), d]; d_n_uniq: [1]")
    _ok(lib().gnn_embedding_grad_rows(ids.data_ptr(), _ptr(d_n), ids.numel(), dout.data_ptr(), dt,
                                      _ld(dout), scale, pad_id, num_rows, grad.shape[1],
                                      uniq.data_ptr(), uniq.numel(), d_n_uniq.data_ptr(),
                                      grad.data_ptr(), gt, _ld(grad), _ptr(d_status),
                                      ws.data_ptr(), ws.numel() * ws.element_size(),
                                      _stream(stream)), "gnn_embedding_grad_rows")


def gnn_cross_attention_workspace_size(n_seq: int, n_q: int, n_k: int, max_q: int, max_k: int,
                                       heads: int, kv_heads: int, head_dim: int, dtype,
                                       backward: bool = False) -> int:
    x = _abi.gnn_attention(_type(dtype, "dtype"), heads, kv_heads, head_dim, n_seq, n_q, n_k, max_q,
                           max_k)
    b = ctypes.c_size_t(0)
    _ok(lib().gnn_cross_attention_workspace_size(ctypes.byref(x), 1 if backward else 0,
                                                 ctypes.byref(b)),
        "gnn_cross_attention_workspace_size")
    return int(b.value)


def _head_rows(t: torch.Tensor, dtype, heads: int, head_dim: int, name: str) -> int:
    """Checks a [rows, heads, head_dim] device tensor whose rows are contiguous; its row stride."""
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name}: must be a device tensor")
    if t.dim() != 3 or t.shape[1] != heads or t.shape[2] != head_dim or \
            (head_dim > 1 and t.stride(2) != 1) or (heads > 1 and t.stride(1) != head_dim):
        raise ValueError(f"{name}: must be [rows, {heads}, {head_dim}] with contiguous rows")
    return t.stride(0) if t.shape[0] > 1 else heads * head_dim


def _attention(q, k, v, q_indptr, k_indptr, max_q, max_k, scale, out, lse, k_count, d_status):
    if q.dim() != 3 or k.dim() != 3:
        raise ValueError("q: [n_q, heads, head_dim]; k: [n_k, kv_heads, head_dim]")
    heads, d, kv = q.shape[1], q.shape[2], k.shape[1]
    kind = _type(q.dtype, "q")
    ld_q = _head_rows(q, q.dtype, heads, d, "q")
    ld_k = _head_rows(k, q.dtype, kv, d, "k")
    ld_v = _head_rows(v, q.dtype, kv, d, "v")
    ld_out = _head_rows(out, q.dtype, heads, d, "out")
    _need(q_indptr, torch.int32, "q_indptr")
    _need(k_indptr, torch.int32, "k_indptr")
    n_seq = q_indptr.numel() - 1
    if n_seq < 0 or k_indptr.numel() != n_seq + 1:
        raise ValueError("q_indptr, k_indptr: [n_seq + 1] each")
    if v.shape[0] != k.shape[0] or out.shape[0] != q.shape[0]:
        raise ValueError("v: as many rows as k; out: as many rows as q")
    if k_count is not None:
        _need(k_count, torch.int64, "k_count")
        if k_count.numel() != n_seq:
            raise ValueError("k_count: [n_seq]")
    if lse is not None:
        _need(lse, torch.float32, "lse")
        if lse.numel() != q.shape[0] * heads:
            raise ValueError("lse: [n_q, heads]")
    if d_status is not None:
        _need(d_status, torch.int32, "d_status")
    return _abi.gnn_attention(
        kind, heads, kv, d, n_seq, q.shape[0], k.shape[0], max_q, max_k, scale, q_indptr.data_ptr(),
        k_indptr.data_ptr(), None if k_count is None else k_count.data_ptr(), q.data_ptr(),
        k.data_ptr(), v.data_ptr(), ld_q, ld_k, ld_v, out.data_ptr(), ld_out,
        None if lse is None else lse.data_ptr(), None if d_status is None else d_status.data_ptr())


def gnn_cross_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, q_indptr: torch.Tensor,
                        k_indptr: torch.Tensor, max_q: int, max_k: int, scale: float,
                        out: torch.Tensor, ws: torch.Tensor, lse: Optional[torch.Tensor] = None,
                        k_count: Optional[torch.Tensor] = None,
                        d_status: Optional[torch.Tensor] = None, stream=None) -> None:
    """out[i, h] = softmax(scale q[i, h] . k) v over the states of i's sequence; lse [n_q, heads] the
    log of the weights' sum.  q, out: [n_q, heads, head_dim]; k, v: [n_k, kv_heads, head_dim]."""
    x = _attention(q, k, v, q_indptr, k_indptr, max_q, max_k, scale, out, lse, k_count, d_status)
    if not ws.is_cuda or not ws.is_contiguous():
        raise ValueError("ws: must be a contiguous device tensor")
    _ok(lib().gnn_cross_attention(ctypes.byref(x), ws.data_ptr(), ws.numel() * ws.element_size(),
                                  _stream(stream)), "gnn_cross_attention")


def gnn_cross_attention_backward(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                                 q_indptr: torch.Tensor, k_indptr: torch.Tensor, max_q: int,
                                 max_k: int, scale: float, out: torch.Tensor, lse: torch.Tensor,
                                 dout: torch.Tensor, dq: torch.Tensor, dk: torch.Tensor,
                                 dv: torch.Tensor, ws: torch.Tensor,
                                 k_count: Optional[torch.Tensor] = None,
                                 d_status: Optional[torch.Tensor] = None, stream=None) -> None:
    """dq, dk, dv of gnn_cross_attention from its out and lse and the gradient dout of out."""
    x = _attention(q, k, v, q_indptr, k_indptr, max_q, max_k, scale, out, lse, k_count, d_status)
    if not ws.is_cuda or not ws.is_contiguous():
        raise ValueError("ws: must be a contiguous device tensor")
    heads, d, kv = q.shape[1], q.shape[2], k.shape[1]
    g = _abi.gnn_attention_grad(
        dout.data_ptr(), _head_rows(dout, q.dtype, heads, d, "dout"), dq.data_ptr(), dk.data_ptr(),
        dv.data_ptr(), _head_rows(dq, q.dtype, heads, d, "dq"),
        _head_rows(dk, q.dtype, kv, d, "dk"), _head_rows(dv, q.dtype, kv, d, "dv"))
    if dout.shape[0] != q.shape[0] or dq.shape[0] != q.shape[0] or dk.shape[0] != k.shape[0] or \
            dv.shape[0] != k.shape[0]:
        raise ValueError("dout, dq: as many rows as q; dk, dv: as many rows as k")
    _ok(lib().gnn_cross_attention_backward(ctypes.byref(x), ctypes.byref(g), ws.data_ptr(),
                                           ws.numel() * ws.element_size(), _stream(stream)),
        "gnn_cross_attention_backward")


def gnn_orthogonalize_workspace_size(batch: int, rows: int, cols: int, dtype) -> int:
    b = ctypes.c_size_t(0)
    _ok(lib().gnn_orthogonalize_workspace_size(batch, rows, cols, _type(dtype, "dtype"),
                                               ctypes.byref(b)),
        "gnn_orthogonalize_workspace_size")
    return int(b.value)


def _matrices(t: torch.Tensor, name: str):
    """(type, batch, rows, cols, row stride, matrix stride) of a device matrix or batch of them."""
    kind = _type(t.dtype, name)
    if not t.is_cuda:
        raise ValueError(f"{name}: must be a device tensor")
    if t.dim() == 2:
        t = t.unsqueeze(0)
    if t.dim() != 3 or (t.shape[2] > 1 and t.stride(2) != 1):
        raise ValueError(f"{name}: must be [rows, cols] or [batch, rows, cols] with contiguous rows")
    b, m, n = t.shape
    ld = t.stride(1) if m > 1 else n
    return kind, b, m, n, ld, t.stride(0) if b > 1 else m * ld


def gnn_orthogonalize(g: torch.Tensor, out: torch.Tensor, ws: torch.Tensor, steps: int = 5,
                      coefs: Optional[Sequence[float]] = None, eps: float = 1e-7,
                      scale: float = 1.0, stream=None) -> None:
    """out = scale * X after `steps` Newton-Schulz steps X <- (c0 I + c1 A + c2 A^2) X, A = X X^T, from
    X = g / (|g|_F + eps).  g, out: [rows, cols] or [batch, rows, cols], float32 or bfloat16."""
    kind, b, m, n, ld, stride = _matrices(g, "g")
    okind, ob, om, on, old, ostride = _matrices(out, "out")
    if okind != kind or (ob, om, on) != (b, m, n):
        raise ValueError("out: g's shape and type")
    if not ws.is_cuda or not ws.is_contiguous():
        raise ValueError("ws: must be a contiguous device tensor")
    c = None
    if coefs is not None:
        if len(coefs) != 3:
            raise ValueError("coefs: three numbers")
        c = (ctypes.c_float * 3)(*coefs)
    _ok(lib().gnn_orthogonalize(g.data_ptr(), kind, b, m, n, ld, stride, steps, c, eps, scale,
                                out.data_ptr(), old, ostride, ws.data_ptr(),
                                ws.numel() * ws.element_size(), _stream(stream)),
        "gnn_orthogonalize")


def _on(t: torch.Tensor, device: int, name: str) -> None:
    """Refuses a tensor that is on another device than the call (-1: the host)."""
    if t.get_device() < 0:
        raise ValueError(f"{name}: must be a device tensor")
    raise ValueError(f"{name}: is on device {t.get_device()}, the call on device {device}")


def _device_of(x: torch.Tensor, stream) -> int:
    """The device that a call on x runs on: the stream's (a handle's is the current one)."""
    device = stream.device_index if isinstance(stream, torch.cuda.Stream) else torch.cuda.current_device() \
        if x.is_cuda else -1
    if device < 0 or x.get_device() != device:
        _on(x, device, "x")
    return device


def _matrix(t: Optional[torch.Tensor], dtype, rows: int, cols: int, name: str, device: int):
    """(pointer, row stride) of a [>= rows, cols] matrix of this type on the device; (None, 0) of None."""
    if t is None:
        return None, 0
    if t.dtype is not dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.get_device() != device:
        _on(t, device, name)
    shape, stride = t.shape, t.stride()
    if len(shape) != 2 or shape[0] < rows or shape[1] != cols or (cols > 1 and stride[1] != 1) or \
            (shape[0] > 1 and stride[0] < cols):
        raise ValueError(f"{name}: must be [{rows}, {cols}] with contiguous rows that do not overlap")
    return t.data_ptr(), stride[0] if shape[0] > 1 else cols


def _vector(t: Optional[torch.Tensor], dtype, n: int, name: str, device: int):
    """The pointer of a contiguous tensor of n elements on the device; None of None."""
    if t is None:
        return None
    if t.dtype is not dtype or not t.is_contiguous():
        _need(t, dtype, name)
    if t.get_device() != device:
        _on(t, device, name)
    if t.numel() != n:
        raise ValueError(f"{name}: [{n}]")
    return t.data_ptr()


def _space(ws: torch.Tensor, device: int):
    if ws.get_device() != device:
        _on(ws, device, "ws")
    if not ws.is_contiguous():
        raise ValueError("ws: must be a contiguous device tensor")
    return ws.data_ptr(), ws.numel() * ws.element_size()


def _rows_of(x: torch.Tensor):
    shape = x.shape
    if len(shape) != 2:
        raise ValueError("x: must be a matrix")
    return shape


def gnn_layer_norm(x: torch.Tensor, weight: Optional[torch.Tensor], bias: Optional[torch.Tensor],
                   eps: float, out: torch.Tensor, mean: Optional[torch.Tensor] = None,
                   rstd: Optional[torch.Tensor] = None, d_n: Optional[torch.Tensor] = None,
                   stream=None) -> None:
    """out = (x - mean) * rstd * weight + bias over the rows of x [n, d], mean and rstd (float32 [n])
    those of each row, rstd = 1 / sqrt(variance + eps).  x, out and weight with bias: float32 or
    bfloat16 each; None for weight: ones, for bias: zeros."""
    n, d = _rows_of(x)
    dev = _device_of(x, stream)
    xt, ot = x.dtype, out.dtype
    pt = weight.dtype if weight is not None else xt if bias is None else bias.dtype
    px, ld_x = _matrix(x, xt, n, d, "x", dev)
    po, ld_out = _matrix(out, ot, n, d, "out", dev)
    a = _abi.gnn_norm(_type(xt, "x"), _type(ot, "out"), _type(pt, "weight"), eps, n, d,
                      _vector(d_n, torch.int64, 1, "d_n", dev), px, ld_x, _vector(weight, pt, d, "weight", dev),
                      _vector(bias, pt, d, "bias", dev), po, ld_out, _vector(mean, torch.float32, n, "mean", dev),
                      _vector(rstd, torch.float32, n, "rstd", dev))
    _ok(lib().gnn_layer_norm(ctypes.byref(a), _stream(stream)), "gnn_layer_norm")


def gnn_layer_norm_workspace_size(n: int, d: int) -> int:
    b = ctypes.c_size_t(0)
    _ok(lib().gnn_layer_norm_workspace_size(n, d, ctypes.byref(b)), "gnn_layer_norm_workspace_size")
    return int(b.value)


def gnn_layer_norm_backward(x: torch.Tensor, weight: Optional[torch.Tensor], mean: torch.Tensor,
                            rstd: torch.Tensor, dout: torch.Tensor, dx: Optional[torch.Tensor],
                            ws: torch.Tensor, dweight: Optional[torch.Tensor] = None,
                            dbias: Optional[torch.Tensor] = None,
                            residual_grad: Optional[torch.Tensor] = None,
                            d_n: Optional[torch.Tensor] = None, stream=None) -> None:
    """dx, dweight and dbias (those that are not None) of gnn_layer_norm from its mean and rstd and the
    gradient dout of out; residual_grad, the gradient that reaches x past the norm, is added to dx."""
    n, d = _rows_of(x)
    dev = _device_of(x, stream)
    xt, ot = x.dtype, dout.dtype
    pt = next((t.dtype for t in (weight, dweight, dbias) if t is not None), xt)
    px, ld_x = _matrix(x, xt, n, d, "x", dev)
    a = _abi.gnn_norm(_type(xt, "x"), _type(ot, "dout"), _type(pt, "weight"), 0.0, n, d,
                      _vector(d_n, torch.int64, 1, "d_n", dev), px, ld_x, _vector(weight, pt, d, "weight", dev), None,
                      None, d, _vector(mean, torch.float32, n, "mean", dev), _vector(rstd, torch.float32, n, "rstd", dev))
    pdy, ld_dy = _matrix(dout, ot, n, d, "dout", dev)
    pr, ld_r = _matrix(residual_grad, xt, n, d, "residual_grad", dev)
    pdx, ld_dx = _matrix(dx, xt, n, d, "dx", dev)
    g = _abi.gnn_norm_grad(pdy, ld_dy, pr, ld_r, pdx, ld_dx, _vector(dweight, pt, d, "dweight", dev),
                           _vector(dbias, pt, d, "dbias", dev))
    p, size = _space(ws, dev)
    _ok(lib().gnn_layer_norm_backward(ctypes.byref(a), ctypes.byref(g), p, size, _stream(stream)),
        "gnn_layer_norm_backward")


#: The activations of the dense layers, by name.
ACTIVATIONS = {"none": _abi.GNN_ACT_NONE, "relu": _abi.GNN_ACT_RELU, "gelu": _abi.GNN_ACT_GELU,
               "gelu_tanh": _abi.GNN_ACT_GELU_TANH, "silu": _abi.GNN_ACT_SILU,
               "sigmoid": _abi.GNN_ACT_SIGMOID}


def _activation(name: str) -> int:
    a = ACTIVATIONS.get(name)
    if a is None:
        raise ValueError(f"activation must be one of {sorted(ACTIVATIONS)}")
    return a


def _layer(x, w, activation, d_n, stream):
    """(type, activation, n, d_in, d_out, d_n, x, ld_x) of a layer, and its device; w: any of its weights."""
    n, d_in = _rows_of(x)
    shape = w.shape
    if len(shape) != 2:
        raise ValueError("weights: must be matrices")
    dt = x.dtype
    kind, act, dev = _type(dt, "x"), _activation(activation), _device_of(x, stream)
    return (kind, act, n, d_in, shape[1], _vector(d_n, torch.int64, 1, "d_n", dev),
            *_matrix(x, dt, n, d_in, "x", dev)), dev


def _same_stride(first, second, names: str):
    """One row stride of two matrices, either of which may be missing."""
    (p, ld), (q, ld2) = first, second
    if p is not None and q is not None and ld != ld2:
        raise ValueError(f"{names}: must have one row stride")
    return p, q, ld if p is not None else ld2


def _layer_size(layer, call, n, d_in, d_out, dtype, backward):
    a = layer(_type(dtype, "dtype"), _abi.GNN_ACT_NONE, n, d_in, d_out)
    b = ctypes.c_size_t(0)
    _ok(getattr(lib(), call)(ctypes.byref(a), 1 if backward else 0, ctypes.byref(b)), call)
    return int(b.value)


def gnn_linear_workspace_size(n: int, d_in: int, d_out: int, dtype, backward: bool = False) -> int:
    """Bytes of ws for gnn_linear (or its backward pass) over up to n rows."""
    return _layer_size(_abi.gnn_dense, "gnn_linear_workspace_size", n, d_in, d_out, dtype, backward)


def gnn_linear(x: torch.Tensor, w: torch.Tensor, out: torch.Tensor, ws: torch.Tensor,
               bias: Optional[torch.Tensor] = None, activation: str = "none",
               residual: Optional[torch.Tensor] = None, pre: Optional[torch.Tensor] = None,
               d_n: Optional[torch.Tensor] = None, stream=None) -> None:
    """out = act(x w + bias) + residual; pre, if given, receives x w + bias for the backward pass.
    x: [n, d_in], w: [d_in, d_out], the others [n, d_out] and [d_out], one type, float32 or bfloat16."""
    head, dev = _layer(x, w, activation, d_n, stream)
    n, d_in, d_out, dt = head[2], head[3], head[4], x.dtype
    a = _abi.gnn_dense(*head, *_matrix(w, dt, d_in, d_out, "w", dev), _vector(bias, dt, d_out, "bias", dev),
                       *_matrix(residual, dt, n, d_out, "residual", dev), *_matrix(out, dt, n, d_out, "out", dev),
                       *_matrix(pre, dt, n, d_out, "pre", dev))
    p, size = _space(ws, dev)
    _ok(lib().gnn_linear(ctypes.byref(a), p, size, _stream(stream)), "gnn_linear")


def gnn_linear_backward(x: torch.Tensor, w: torch.Tensor, dout: torch.Tensor, ws: torch.Tensor,
                        activation: str = "none", pre: Optional[torch.Tensor] = None,
                        dx: Optional[torch.Tensor] = None, dw: Optional[torch.Tensor] = None,
                        dbias: Optional[torch.Tensor] = None, d_n: Optional[torch.Tensor] = None,
                        stream=None) -> None:
    """Those of dx, dw and dbias that are given, from the gradient dout of gnn_linear's out and, where
    there is an activation, its pre.  (The residual's gradient is dout.)"""
    head, dev = _layer(x, w, activation, d_n, stream)
    n, d_in, d_out, dt = head[2], head[3], head[4], x.dtype
    a = _abi.gnn_dense(*head, *_matrix(w, dt, d_in, d_out, "w", dev), None, None, 0, None, 0,
                       *_matrix(pre, dt, n, d_out, "pre", dev))
    g = _abi.gnn_dense_grad(*_matrix(dout, dt, n, d_out, "dout", dev), *_matrix(dx, dt, n, d_in, "dx", dev),
                            *_matrix(dw, dt, d_in, d_out, "dw", dev), _vector(dbias, dt, d_out, "dbias", dev))
    p, size = _space(ws, dev)
    _ok(lib().gnn_linear_backward(ctypes.byref(a), ctypes.byref(g), p, size, _stream(stream)),
        "gnn_linear_backward")


def gnn_gated_linear_workspace_size(n: int, d_in: int, d_out: int, dtype, backward: bool = False) -> int:
    """Bytes of ws for gnn_gated_linear (or its backward pass) over up to n rows."""
    return _layer_size(_abi.gnn_gated, "gnn_gated_linear_workspace_size", n, d_in, d_out, dtype, backward)


def gnn_gated_linear(x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor, out: torch.Tensor,
                     ws: torch.Tensor, bias_gate: Optional[torch.Tensor] = None,
                     bias_up: Optional[torch.Tensor] = None, activation: str = "silu",
                     gate: Optional[torch.Tensor] = None, up: Optional[torch.Tensor] = None,
                     d_n: Optional[torch.Tensor] = None, stream=None) -> None:
    """out = act(x w_gate + bias_gate) * (x w_up + bias_up); gate and up, if given, receive the two sums for
    the backward pass.  x: [n, d_in], weights: [d_in, d_out] of one row stride (halves of one matrix, for
    instance), the others [n, d_out] and [d_out], one type, float32 or bfloat16."""
    head, dev = _layer(x, w_gate, activation, d_n, stream)
    n, d_in, d_out, dt = head[2], head[3], head[4], x.dtype
    w = _same_stride(_matrix(w_gate, dt, d_in, d_out, "w_gate", dev), _matrix(w_up, dt, d_in, d_out, "w_up", dev),
                     "w_gate, w_up")
    pre = _same_stride(_matrix(gate, dt, n, d_out, "gate", dev), _matrix(up, dt, n, d_out, "up", dev), "gate, up")
    a = _abi.gnn_gated(*head, *w, _vector(bias_gate, dt, d_out, "bias_gate", dev),
                       _vector(bias_up, dt, d_out, "bias_up", dev), *_matrix(out, dt, n, d_out, "out", dev), *pre)
    p, size = _space(ws, dev)
    _ok(lib().gnn_gated_linear(ctypes.byref(a), p, size, _stream(stream)), "gnn_gated_linear")


def gnn_gated_linear_backward(x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor,
                              gate: torch.Tensor, up: torch.Tensor, dout: torch.Tensor,
                              ws: torch.Tensor, activation: str = "silu",
                              dx: Optional[torch.Tensor] = None, dw_gate: Optional[torch.Tensor] = None,
                              dw_up: Optional[torch.Tensor] = None,
                              dbias_gate: Optional[torch.Tensor] = None,
                              dbias_up: Optional[torch.Tensor] = None,
                              d_n: Optional[torch.Tensor] = None, stream=None) -> None:
    """Those of dx, dw_gate, dw_up, dbias_gate and dbias_up that are given, from the gradient dout of
    gnn_gated_linear's out and its gate and up.  dw_gate and dw_up have one row stride, like gate and up."""
    head, dev = _layer(x, w_gate, activation, d_n, stream)
    n, d_in, d_out, dt = head[2], head[3], head[4], x.dtype
    w = _same_stride(_matrix(w_gate, dt, d_in, d_out, "w_gate", dev), _matrix(w_up, dt, d_in, d_out, "w_up", dev),
                     "w_gate, w_up")
    pre = _same_stride(_matrix(gate, dt, n, d_out, "gate", dev), _matrix(up, dt, n, d_out, "up", dev), "gate, up")
    a = _abi.gnn_gated(*head, *w, None, None, None, 0, *pre)
    dw = _same_stride(_matrix(dw_gate, dt, d_in, d_out, "dw_gate", dev), _matrix(dw_up, dt, d_in, d_out, "dw_up", dev),
                      "dw_gate, dw_up")
    g = _abi.gnn_gated_grad(*_matrix(dout, dt, n, d_out, "dout", dev), *_matrix(dx, dt, n, d_in, "dx", dev), *dw,
                            _vector(dbias_gate, dt, d_out, "dbias_gate", dev),
                            _vector(dbias_up, dt, d_out, "dbias_up", dev))
    p, size = _space(ws, dev)
    _ok(lib().gnn_gated_linear_backward(ctypes.byref(a), ctypes.byref(g), p, size, _stream(stream)),
        "gnn_gated_linear_backward")


def gnn_copy_probe(src: torch.Tensor, dst: torch.Tensor, stream=None) -> None:
    """Plain device copy of src into dst (same byte size) by k_copy_probe; calibrates counters."""
    nbytes = src.numel() * src.element_size()
    if dst.numel() * dst.element_size() != nbytes:
        raise ValueError("src and dst differ in size")
    _ok(lib().gnn_copy_probe(_ptr(src), _ptr(dst), nbytes, _stream(stream)), "gnn_copy_probe")


def gnn_copy_probe_host(src: torch.Tensor, dst: torch.Tensor, stream=None) -> None:
    """The same copy with src in pinned host memory, read in place over the host link."""
    if src.is_cuda or not src.is_pinned():
        raise ValueError("src must be a pinned host tensor")
    nbytes = src.numel() * src.element_size()
    if dst.numel() * dst.element_size() != nbytes:
        raise ValueError("src and dst differ in size")
    _ok(lib().gnn_copy_probe_host(_ptr(src), _ptr(dst), nbytes, _stream(stream)),
        "gnn_copy_probe_host")


def gnn_hash_probe(seed: int, tau: int, lanes: int, per_lane: int, d_count: torch.Tensor,
                   stream=None) -> None:
    """lanes * per_lane sampling keys (mix64 of a stepped counter); adds the keys <= tau to d_count."""
    _need(d_count, torch.int64, "d_count")
    _ok(lib().gnn_hash_probe(seed, tau, lanes, per_lane, _ptr(d_count), _stream(stream)),
        "gnn_hash_probe")


def gnn_read_device_status(ws: torch.Tensor, stream=None) -> int:
    out = ctypes.c_int32(0)
    _ok(lib().gnn_read_device_status(_ptr(ws), _stream(stream), ctypes.byref(out)),
        "gnn_read_device_status")
    return int(out.value)
