"""ctypes binding of ``libmpk.so`` (include/mpk.h).  Argument marshalling
only: every step of the decode path runs in the library's kernels.  Loading
fails loudly when the library is missing; there is no fallback.

Functions keep the C names (``mpk_build_tgraph``, ``mpk_decode_step``, ...).
``Graph`` wraps a graph handle for convenience; ``Weights`` and ``KVCache``
hold the device tensors a step borrows (torch tensors are used for device
memory and streams only)."""
from __future__ import annotations

import ctypes
import os
from typing import Dict, Optional, Sequence

import numpy as np

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmpk.so")

MPK_OK = 0
STATUS_NAMES = {
    0: "MPK_OK", 1: "MPK_ERR_INVALID_ARG", 2: "MPK_ERR_UNSUPPORTED",
    3: "MPK_ERR_CUDA", 4: "MPK_ERR_OOM", 5: "MPK_ERR_NOT_CORESIDENT",
    6: "MPK_ERR_TIMEOUT", 7: "MPK_ERR_KV_PAGE", 8: "MPK_ERR_QUEUE_OVERFLOW",
    9: "MPK_ERR_GRAPH_INVALID", 10: "MPK_ERR_NOT_BOUND"}
globals().update({v: k for k, v in STATUS_NAMES.items()})

TASK_KINDS = ["empty", "qkv", "attn", "o", "gateup", "down", "lm_head",
              "argmax", "chain_up", "chain_down"]
MODE_MEGAKERNEL, MODE_KPO, MODE_KPO_GRAPH = 0, 1, 2
LAYER_TENSORS = ["ln1", "wqkv", "q_norm", "k_norm", "wo", "ln2", "wgu", "wd"]


class MpkError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS_NAMES.get(status, status)}")


class ModelShape(ctypes.Structure):
    _fields_ = [("n_layers", ctypes.c_int), ("hidden", ctypes.c_int),
                ("n_q_heads", ctypes.c_int), ("n_kv_heads", ctypes.c_int),
                ("head_dim", ctypes.c_int), ("ffn", ctypes.c_int),
                ("vocab", ctypes.c_int), ("rms_eps", ctypes.c_float),
                ("rope_theta", ctypes.c_float), ("qk_norm", ctypes.c_int),
                ("chain_ffn", ctypes.c_int), ("page_size", ctypes.c_int),
                ("max_pages_per_seq", ctypes.c_int)]


class TileSizes(ctypes.Structure):
    _fields_ = [("num_workers", ctypes.c_int),
                ("gemv_rows_per_task", ctypes.c_int),
                ("mma_rows_per_task", ctypes.c_int),
                ("attn_chunks", ctypes.c_int),
                ("num_sched_sms", ctypes.c_int),
                ("sched_warps_per_sm", ctypes.c_int),
                ("smem_pages", ctypes.c_int),
                ("coarse_events", ctypes.c_int)]


class _Weights(ctypes.Structure):
    _fields_ = [("embed", ctypes.c_void_p), ("final_norm", ctypes.c_void_p),
                ("lm_head", ctypes.c_void_p),
                ("layers", ctypes.POINTER(ctypes.c_void_p)),
                ("chain_w1", ctypes.c_void_p), ("chain_w2", ctypes.c_void_p)]


class _KVCache(ctypes.Structure):
    _fields_ = [("k_pool", ctypes.c_void_p), ("v_pool", ctypes.c_void_p),
                ("page_table", ctypes.c_void_p), ("seq_lens", ctypes.c_void_p),
                ("num_pages", ctypes.c_int)]


_P32 = ctypes.POINTER(ctypes.c_int32)


class SimReport(ctypes.Structure):
    _fields_ = [("tasks_run", ctypes.c_int64),
                ("order_violations", ctypes.c_int64),
                ("duplicate_runs", ctypes.c_int64),
                ("missing_runs", ctypes.c_int64),
                ("deadlocked", ctypes.c_int32),
                ("steps_completed", ctypes.c_int32),
                ("seconds", ctypes.c_double)]


class GraphExport(ctypes.Structure):
    _fields_ = [("n_tasks", ctypes.c_int), ("n_events", ctypes.c_int),
                ("n_ops", ctypes.c_int), ("n_empty", ctypes.c_int),
                ("n_workers", ctypes.c_int), ("attn_chunks", ctypes.c_int)] + [
        (n, _P32) for n in (
            "task_kind", "task_op", "task_layer", "task_tile", "task_row0",
            "task_row1", "task_b", "task_g", "task_c", "task_dep",
            "task_trig", "task_launch", "task_worker", "task_pre_id",
            "event_count", "event_first", "event_last", "op_kind",
            "op_layer", "op_n_tasks")] + [
        ("n_raw_events", ctypes.c_int64), ("n_fused_events", ctypes.c_int64),
        ("n_sched_sms", ctypes.c_int), ("sched_warps_per_sm", ctypes.c_int)]


class AttnShape(ctypes.Structure):
    _fields_ = [("n_q_heads", ctypes.c_int), ("n_kv_heads", ctypes.c_int),
                ("head_dim", ctypes.c_int), ("page_size", ctypes.c_int),
                ("max_pages_per_seq", ctypes.c_int)]


class TokenBatch(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int), ("n_tokens", ctypes.c_int),
                ("q_start", ctypes.c_void_p),
                ("tokens_per_seq", ctypes.c_int)]


class _Rope(ctypes.Structure):
    _fields_ = [("table", ctypes.c_void_p), ("n_pos", ctypes.c_int),
                ("rotary_dim", ctypes.c_int), ("interleaved", ctypes.c_int)]


class RopeScaling(ctypes.Structure):
    _fields_ = [("rotary_dim", ctypes.c_int), ("theta", ctypes.c_double),
                ("scaling", ctypes.c_int), ("factor", ctypes.c_double),
                ("low", ctypes.c_double), ("high", ctypes.c_double),
                ("old_ctx", ctypes.c_double),
                ("attn_factor", ctypes.c_double)]


class PrefixGroups(ctypes.Structure):
    _fields_ = [("n_groups", ctypes.c_int), ("group_start", ctypes.c_void_p),
                ("prefix_len", ctypes.c_void_p)]


class VerifyArgs(ctypes.Structure):
    _fields_ = [("vocab", ctypes.c_int), ("max_out", ctypes.c_int),
                ("tokens", ctypes.c_void_p), ("logits", ctypes.c_void_p),
                ("logits_stride", ctypes.c_int64),
                ("draft", ctypes.c_void_p), ("draft_stride", ctypes.c_int64),
                ("draft_is_logits", ctypes.c_int),
                ("temperature", ctypes.c_void_p),
                ("uniform", ctypes.c_void_p), ("noise", ctypes.c_void_p),
                ("noise_stride", ctypes.c_int64),
                ("n_accepted", ctypes.c_void_p),
                ("out_tokens", ctypes.c_void_p),
                ("logprobs", ctypes.c_void_p),
                ("next_tokens", ctypes.c_void_p),
                ("seq_lens", ctypes.c_void_p),
                ("seq_lens_out", ctypes.c_void_p)]


ROPE_PLAIN, ROPE_LINEAR, ROPE_BANDS, ROPE_RAMP = 0, 1, 2, 3

_lib = None


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libmpk.so (once).  Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(
            f"{path} is missing: build it with "
            "`python -m task_graph_runtime_gb300.build` (no fallback exists)")
    lib = ctypes.CDLL(path)
    vp, i, st = ctypes.c_void_p, ctypes.c_int, ctypes.c_int
    i64 = ctypes.c_int64
    sig = {
        "mpk_build_tgraph": ([ctypes.POINTER(ModelShape),
                              ctypes.POINTER(TileSizes), i,
                              ctypes.POINTER(vp)], st),
        "mpk_bind_weights": ([vp, ctypes.POINTER(_Weights)], st),
        "mpk_decode_step": ([vp, vp, ctypes.POINTER(_KVCache), vp, vp, vp],
                            st),
        "mpk_decode_steps": ([vp, vp, ctypes.POINTER(_KVCache), vp, vp, i,
                              vp], st),
        "mpk_get_status": ([vp], st),
        "mpk_set_mode": ([vp, i], st),
        "mpk_export_tgraph": ([vp, ctypes.POINTER(GraphExport)], st),
        "mpk_reset": ([vp], st),
        "mpk_destroy_tgraph": ([vp], None),
        "mpk_status_string": ([i], ctypes.c_char_p),
        "mpk_debug_set_wait_timeout_ms": ([vp, i], st),
        "mpk_debug_add_event_count": ([vp, i, i], st),
        "mpk_debug_set_trace": ([vp, i], st),
        "mpk_debug_read_trace": ([vp, vp, i, ctypes.POINTER(i)], st),
        "mpk_debug_read_hidden": ([vp, i, vp], st),
        "mpk_debug_simulate": ([vp, i, ctypes.c_uint32, i, i,
                                ctypes.POINTER(SimReport)], st),
        "mpk_decode_step_noalloc": ([vp, ctypes.POINTER(_Weights), vp,
                                     ctypes.POINTER(_KVCache), vp, vp, vp,
                                     vp], st),
        "mpk_rope_table": ([ctypes.POINTER(RopeScaling), i64, i, vp, vp], st),
        "mpk_kv_append": ([ctypes.POINTER(AttnShape),
                           ctypes.POINTER(TokenBatch),
                           ctypes.POINTER(_KVCache), i, vp, i64, vp, i64, vp,
                           i64, vp, vp, ctypes.c_float,
                           ctypes.POINTER(_Rope), vp, i64, vp, vp], st),
        "mpk_prefix_attention_workspace": ([ctypes.POINTER(AttnShape),
                                            ctypes.POINTER(TokenBatch), i],
                                           ctypes.c_size_t),
        "mpk_prefix_attention": ([ctypes.POINTER(AttnShape),
                                  ctypes.POINTER(TokenBatch),
                                  ctypes.POINTER(PrefixGroups),
                                  ctypes.POINTER(_KVCache), i, vp, i64,
                                  ctypes.c_float, vp, i64, vp, vp,
                                  ctypes.c_size_t, vp, vp], st),
        "mpk_verify_drafts_workspace": ([ctypes.POINTER(TokenBatch), i],
                                        ctypes.c_size_t),
        "mpk_verify_step_workspace": ([vp, ctypes.POINTER(TokenBatch), i],
                                      ctypes.c_size_t),
        "mpk_verify_step": ([vp, ctypes.POINTER(TokenBatch),
                             ctypes.POINTER(PrefixGroups),
                             ctypes.POINTER(_KVCache),
                             ctypes.POINTER(VerifyArgs), vp, vp,
                             ctypes.c_size_t, vp], st),
        "mpk_verify_drafts": ([ctypes.POINTER(TokenBatch),
                               ctypes.POINTER(VerifyArgs), vp,
                               ctypes.c_size_t, vp, vp], st),
    }
    for name, (args, res) in sig.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = res
    _lib = lib
    return lib


def _check(status: int, where: str):
    if status != MPK_OK:
        raise MpkError(status, where)


def model_shape(shape, page_size: int = 16, max_pages_per_seq: int = 1
                ) -> ModelShape:
    """ModelShape from a ``synth.ModelShape``-like object."""
    return ModelShape(shape.n_layers, shape.hidden, shape.n_q_heads,
                      shape.n_kv_heads, shape.head_dim, shape.ffn,
                      shape.vocab, shape.rms_eps, shape.rope_theta,
                      int(shape.qk_norm), shape.chain_ffn, page_size,
                      max_pages_per_seq)


# --------------------------------------------------------- C-named calls
def mpk_build_tgraph(shape: ModelShape, tiles: Optional[TileSizes],
                     batch: int) -> int:
    lib = load_library()
    h = ctypes.c_void_p()
    _check(lib.mpk_build_tgraph(ctypes.byref(shape),
                                ctypes.byref(tiles) if tiles else None,
                                batch, ctypes.byref(h)), "mpk_build_tgraph")
    return h.value


def mpk_export_tgraph(handle: int) -> Dict[str, np.ndarray]:
    lib = load_library()
    ex = GraphExport()
    _check(lib.mpk_export_tgraph(handle, ctypes.byref(ex)),
           "mpk_export_tgraph")

    def arr(ptr, n):
        return np.ctypeslib.as_array(ptr, shape=(n,)).copy() if n else \
            np.zeros(0, np.int32)
    out = {k: getattr(ex, k) for k in ("n_tasks", "n_events", "n_ops",
                                        "n_empty", "n_workers", "attn_chunks",
                                        "n_raw_events", "n_fused_events",
                                        "n_sched_sms", "sched_warps_per_sm")}
    for k in ("task_kind", "task_op", "task_layer", "task_tile", "task_row0",
              "task_row1", "task_b", "task_g", "task_c", "task_dep",
              "task_trig", "task_launch", "task_worker", "task_pre_id"):
        out[k] = arr(getattr(ex, k), ex.n_tasks)
    for k in ("event_count", "event_first", "event_last"):
        out[k] = arr(getattr(ex, k), ex.n_events)
    for k in ("op_kind", "op_layer", "op_n_tasks"):
        out[k] = arr(getattr(ex, k), ex.n_ops)
    return out


def mpk_destroy_tgraph(handle: int):
    if handle:
        load_library().mpk_destroy_tgraph(handle)


def mpk_status_string(status: int) -> str:
    return load_library().mpk_status_string(status).decode()


# -------------------------------------------------------------- wrappers
class Weights:
    """Device weight tensors (torch.bfloat16, caller-owned)."""

    def __init__(self, tensors: Dict[str, "object"], shape):
        self.tensors = tensors
        self.shape = shape

    def c_struct(self):
        t = self.tensors
        s = self.shape
        ptr = lambda name: t[name].data_ptr() if name in t else None
        if s.chain_ffn > 0:
            layers = (ctypes.c_void_p * 1)()
            st = _Weights(ptr("embed"), ptr("final_norm"), ptr("lm_head"),
                          ctypes.cast(layers, ctypes.POINTER(ctypes.c_void_p)),
                          ptr("chain_w1"), ptr("chain_w2"))
            return st, layers
        layers = (ctypes.c_void_p * (s.n_layers * len(LAYER_TENSORS)))()
        for l in range(s.n_layers):
            for k, name in enumerate(LAYER_TENSORS):
                layers[l * len(LAYER_TENSORS) + k] = ptr(f"layer{l}.{name}")
        st = _Weights(ptr("embed"), ptr("final_norm"), ptr("lm_head"),
                      ctypes.cast(layers, ctypes.POINTER(ctypes.c_void_p)),
                      None, None)
        return st, layers


class KVCache:
    """Paged KV cache on the device (caller-owned torch tensors)."""

    def __init__(self, k_pool, v_pool, page_table, seq_lens):
        self.k_pool, self.v_pool = k_pool, v_pool
        self.page_table, self.seq_lens = page_table, seq_lens

    def c_struct(self) -> _KVCache:
        return _KVCache(self.k_pool.data_ptr(), self.v_pool.data_ptr(),
                        self.page_table.data_ptr(), self.seq_lens.data_ptr(),
                        int(self.k_pool.shape[1]))


class Graph:
    """A built tGraph (owns the library handle)."""

    def __init__(self, shape, batch: int, num_workers: int = 0,
                 gemv_rows_per_task: int = 0, attn_chunks: int = 0,
                 num_sched_sms: int = 0, sched_warps_per_sm: int = 0,
                 smem_pages: int = 0, page_size: int = 16,
                 max_pages_per_seq: int = 1, mma_rows_per_task: int = 0,
                 coarse_events: int = 0):
        self.shape = shape
        self.batch = batch
        self.c_shape = model_shape(shape, page_size, max_pages_per_seq)
        self.tiles = TileSizes(num_workers, gemv_rows_per_task,
                               mma_rows_per_task, attn_chunks, num_sched_sms,
                               sched_warps_per_sm, smem_pages,
                               coarse_events)
        self.handle = mpk_build_tgraph(self.c_shape, self.tiles, batch)
        self._keep = None
        self._ws = None            # verify_step's

    def export(self) -> Dict[str, np.ndarray]:
        return mpk_export_tgraph(self.handle)

    def bind(self, weights: Weights):
        st, layers = weights.c_struct()
        self._keep = (weights, layers)
        _check(load_library().mpk_bind_weights(self.handle, ctypes.byref(st)),
               "mpk_bind_weights")

    def set_mode(self, mode: int):
        _check(load_library().mpk_set_mode(self.handle, mode), "mpk_set_mode")

    def decode_step(self, tokens, kv: Optional[KVCache], logits, next_tokens,
                    stream=None):
        """Enqueue one step on ``stream`` (a torch.cuda.Stream, a raw
        cudaStream_t int, or None for torch's current stream)."""
        import torch
        if stream is None:
            s = torch.cuda.current_stream().cuda_stream
        elif isinstance(stream, int):
            s = stream
        else:
            s = stream.cuda_stream
        kvs = kv.c_struct() if kv is not None else None
        _check(load_library().mpk_decode_step(
            self.handle, tokens.data_ptr(),
            ctypes.byref(kvs) if kvs is not None else None,
            logits.data_ptr(), next_tokens.data_ptr(), s), "mpk_decode_step")

    def decode_steps(self, tokens, kv: Optional[KVCache], logits,
                     next_tokens, n_steps: int, stream=None):
        """Enqueue ``n_steps`` greedy steps in one launch (megakernel mode);
        ``next_tokens`` is int32 [n_steps, batch], ``logits`` receives the
        last step's."""
        import torch
        if stream is None:
            s = torch.cuda.current_stream().cuda_stream
        elif isinstance(stream, int):
            s = stream
        else:
            s = stream.cuda_stream
        kvs = kv.c_struct() if kv is not None else None
        _check(load_library().mpk_decode_steps(
            self.handle, tokens.data_ptr(),
            ctypes.byref(kvs) if kvs is not None else None,
            logits.data_ptr(), next_tokens.data_ptr(), n_steps, s),
            "mpk_decode_steps")

    def verify_step(self, tokens, kv: KVCache, logits, uniform, noise,
                    n_accepted, out_tokens, q_start=None, group_start=None,
                    prefix_len=None, draft=None, draft_is_logits=False,
                    temperature=None, logprobs=None, next_tokens=None,
                    advance: bool = True, stream=None):
        """One step of drafted decoding (mpk_verify_step): this graph's batch
        is the number of rows, the page table's rows are the sequences.
        Arguments as for ``DraftVerifier.verify`` and ``PagedBatch``;
        ``advance`` moves kv.seq_lens past the accepted tokens.  The workspace
        is the graph's own and grows with the first call of a shape."""
        import torch
        w = "Graph.verify_step"
        lib, i32, f32 = load_library(), torch.int32, torch.float32
        dev = _OnDevice()
        dev._on(_cuda_device(kv.page_table, w))
        rows, V = self.batch, self.shape.vocab
        B = int(kv.page_table.shape[0])
        if out_tokens.dim() != 2 or B < 1 or B > rows:
            _refuse(w, "out_tokens must be [sequences, max_out], and the "
                       "sequences no more than the graph's batch")
        if q_start is None and rows % B:
            _refuse(w, "the graph's batch must be a multiple of the "
                       "sequences without q_start")
        if tuple(kv.page_table.shape) != (
                B, self.c_shape.max_pages_per_seq):
            _refuse(w, "page_table must be [sequences, max_pages_per_seq]")
        want = (self.shape.n_layers, self.shape.n_kv_heads,
                self.c_shape.page_size, self.shape.head_dim)
        for pool in (kv.k_pool, kv.v_pool):
            if (pool.dtype is not torch.bfloat16 or pool.dim() != 5 or
                    not pool.is_contiguous() or
                    pool.get_device() != dev._index or
                    (pool.shape[0], *pool.shape[2:]) != want or
                    pool.shape != kv.k_pool.shape):
                _refuse(w, "k_pool and v_pool must be the graph's")
        mo = int(out_tokens.shape[1])
        vec = dev._vec
        vec(kv.page_table, 0, i32, w, "page_table")
        seq = vec(kv.seq_lens, B, i32, w, "seq_lens")
        tok = TokenBatch(B, rows, vec(q_start, B + 1, i32, w, "q_start"),
                         rows // B)
        groups = None
        if (group_start is None) != (prefix_len is None):
            _refuse(w, "group_start and prefix_len come together")
        if prefix_len is not None:
            n = int(prefix_len.numel())
            groups = PrefixGroups(
                n, vec(group_start, n + 1, i32, w, "group_start"),
                vec(prefix_len, n, i32, w, "prefix_len"))

        def matrix(t, n, name):
            if t is None:
                return None, 0
            if (t.dtype is not f32 or t.get_device() != dev._index or
                    t.dim() != 2 or t.shape[0] < n or t.shape[1] != V or
                    (V > 1 and t.stride(1) != 1)):
                _refuse(w, f"{name} must be float32 [{n}, {V}]")
            return t.data_ptr(), (t.stride(0) if n > 1 else V)
        dp, ds = matrix(draft, rows, "draft")
        np_, ns = matrix(noise, B, "noise")
        a = VerifyArgs(
            vocab=V, max_out=mo, tokens=vec(tokens, rows, i32, w, "tokens"),
            draft=dp, draft_stride=ds, draft_is_logits=int(draft_is_logits),
            temperature=vec(temperature, B, f32, w, "temperature"),
            uniform=vec(uniform, rows, f32, w, "uniform"), noise=np_,
            noise_stride=ns,
            n_accepted=vec(n_accepted, B, i32, w, "n_accepted"),
            out_tokens=vec(out_tokens, B * mo, i32, w, "out_tokens"),
            logprobs=vec(logprobs, B * mo, f32, w, "logprobs"),
            next_tokens=vec(next_tokens, B, i32, w, "next_tokens"),
            seq_lens_out=seq if advance else None)
        lg = vec(logits, rows * V, f32, w, "logits")
        need = lib.mpk_verify_step_workspace(
            self.handle, ctypes.byref(tok), groups.n_groups if groups else 0)
        if self._ws is None or self._ws.numel() < need:
            self._ws = torch.empty(max(need, 1), dtype=torch.uint8,
                                   device=dev.device)
        kvs = kv.c_struct()
        _check(dev._call(
            lib.mpk_verify_step, self.handle, ctypes.byref(tok),
            ctypes.byref(groups) if groups else None, ctypes.byref(kvs),
            ctypes.byref(a), lg, self._ws.data_ptr(), self._ws.numel(),
            dev._stream(stream)), "mpk_verify_step")

    def status(self) -> int:
        return load_library().mpk_get_status(self.handle)

    def reset(self):
        _check(load_library().mpk_reset(self.handle), "mpk_reset")

    def set_wait_timeout_ms(self, ms: int):
        _check(load_library().mpk_debug_set_wait_timeout_ms(self.handle, ms),
               "mpk_debug_set_wait_timeout_ms")

    def add_event_count(self, event: int, delta: int):
        _check(load_library().mpk_debug_add_event_count(self.handle, event,
                                                        delta),
               "mpk_debug_add_event_count")

    def set_trace(self, capacity: int):
        _check(load_library().mpk_debug_set_trace(self.handle, capacity),
               "mpk_debug_set_trace")

    def read_trace(self, capacity: int) -> np.ndarray:
        """uint64 [n, 8]: task | worker << 32, looked, ready, staged, pages
        done, body done, triggered (ns; 0 where not recorded), 0."""
        buf = np.zeros((capacity, 8), np.uint64)
        n = ctypes.c_int(0)
        _check(load_library().mpk_debug_read_trace(
            self.handle, buf.ctypes.data, capacity, ctypes.byref(n)),
            "mpk_debug_read_trace")
        return buf[:n.value]

    def simulate(self, steps: int = 2, seed: int = 0, max_delay_us: int = 20,
                 timeout_ms: int = 20000) -> Dict[str, float]:
        """CPU model of the runtime protocol on this graph's encoding
        (mpk_debug_simulate): host threads for workers and scheduler warps,
        random task delays."""
        rep = SimReport()
        _check(load_library().mpk_debug_simulate(
            self.handle, steps, seed, max_delay_us, timeout_ms,
            ctypes.byref(rep)), "mpk_debug_simulate")
        return {k: getattr(rep, k) for k, _ in SimReport._fields_}

    def read_hidden(self, layer: int) -> np.ndarray:
        """bf16 bits [batch, hidden] of the residual stream entering decoder
        layer ``layer`` (``n_layers``: the final RMSNorm's input) in the last
        step."""
        out = np.zeros((self.batch, self.shape.hidden), np.uint16)
        _check(load_library().mpk_debug_read_hidden(
            self.handle, layer, out.ctypes.data), "mpk_debug_read_hidden")
        return out

    def close(self):
        if self.handle:
            mpk_destroy_tgraph(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def mpk_decode_step_noalloc(graph: "Graph", weights: Weights, tokens, kv,
                            logits, next_tokens, status=None, stream=None):
    """One decode step with every piece of scratch in the library's static
    device array (no device allocation); see include/mpk.h."""
    import torch
    s = (torch.cuda.current_stream().cuda_stream if stream is None
         else stream if isinstance(stream, int) else stream.cuda_stream)
    st, layers = weights.c_struct()
    kvs = kv.c_struct() if kv is not None else None
    _check(load_library().mpk_decode_step_noalloc(
        graph.handle, ctypes.byref(st), tokens.data_ptr(),
        ctypes.byref(kvs) if kvs is not None else None, logits.data_ptr(),
        next_tokens.data_ptr(),
        status.data_ptr() if status is not None else None, s),
        "mpk_decode_step_noalloc")
    return layers          # keep the host pointer array alive until here


# ------------------------------------------------------- serving operators
# These calls take a few microseconds on the GPU at small batches, so what
# Python does around them counts: arguments are checked by value, the
# structures that do not change are built once, and torch is asked for the
# current device and stream by its shortest way.
def _refuse(where: str, what: str):
    raise MpkError(MPK_ERR_INVALID_ARG, f"{where}: {what}")


def _failed(st, where: str, call: str):
    """The answer of a call through _binding: a refusal's text, or a status."""
    if isinstance(st, str):
        _refuse(where, st)
    raise MpkError(st, call)


def _native():
    """The module that checks the serving calls' tensors (csrc/binding.cpp)."""
    load_library()
    import torch  # noqa: F401  (its libraries have to be there first)
    try:
        from . import _binding
    except ImportError as e:
        raise RuntimeError(
            "the binding of the serving calls is missing or of another torch:"
            " build it with `python -m task_graph_runtime_gb300.build` (no "
            "fallback exists)") from e
    return _binding


class _OnDevice:
    """Calls go to the tensors' own device, whichever one is current."""

    def _on(self, device):
        import torch
        self.device = device
        self._index = device.index
        self._bf16, self._f32, self._i32 = (torch.bfloat16, torch.float32,
                                            torch.int32)
        self._current = torch._C._cuda_getDevice
        self._raw_stream = torch._C._cuda_getCurrentRawStream

    def _stream(self, stream):
        if stream is None:
            return self._raw_stream(self._index)
        return stream if isinstance(stream, int) else stream.cuda_stream

    def _call(self, fn, *args):
        if self._current() == self._index:
            return fn(*args)
        import torch
        with torch.cuda.device(self.device):
            return fn(*args)

    def _vec(self, t, n, dtype, where, name):
        """Device pointer of a contiguous vector of at least n values."""
        if t is None:
            return None
        if (t.dtype is not dtype or t.get_device() != self._index or
                t.numel() < n or not t.is_contiguous()):
            _refuse(where, f"{name} must be a contiguous {dtype} tensor of "
                           f"{n} values on {self.device}")
        return t.data_ptr()


def _cuda_device(t, where):
    if t.device.type != "cuda":
        _refuse(where, f"tensors must be on a CUDA device, not {t.device}")
    return t.device


def mpk_rope_table(rotary_dim: int, n_pos: int, theta: float,
                   first_pos: int = 0, scaling: int = ROPE_PLAIN,
                   factor: float = 1.0, low: float = 1.0, high: float = 4.0,
                   old_ctx: float = 8192.0, attn_factor: float = 1.0,
                   device="cuda", stream=None):
    """fp32 [n_pos, rotary_dim // 2, 2] table of (cos, sin) for positions
    first_pos, first_pos + 1, ...; see include/mpk.h for the scalings."""
    import torch
    out = torch.empty(max(n_pos, 0), max(rotary_dim, 0) // 2, 2,
                      dtype=torch.float32, device=device)
    dev = _cuda_device(out, "mpk_rope_table")
    s = RopeScaling(rotary_dim, theta, scaling, factor, low, high, old_ctx,
                    attn_factor)
    with torch.cuda.device(dev):
        _check(load_library().mpk_rope_table(
            ctypes.byref(s), first_pos, n_pos, out.data_ptr() or None,
            torch.cuda.current_stream(dev).cuda_stream if stream is None
            else stream if isinstance(stream, int) else stream.cuda_stream),
            "mpk_rope_table")
    return out


class Rope:
    """A rotation table (``mpk_rope_table``) and how heads use it."""

    def __init__(self, table, rotary_dim: int, interleaved: bool = False):
        import torch
        dev = _cuda_device(table, "Rope")
        if (table.dtype is not torch.float32 or not table.is_contiguous() or
                table.dim() != 3 or tuple(table.shape[1:]) !=
                (rotary_dim // 2, 2)):
            _refuse("Rope", "table must be contiguous float32 "
                            "[n_pos, rotary_dim // 2, 2]")
        self.table = table
        self.device = dev
        self.c = _Rope(table.data_ptr(), int(table.shape[0]), rotary_dim,
                       int(bool(interleaved)))
        self._address = ctypes.addressof(self.c)


class PagedBatch(_OnDevice):
    """New tokens of a batch over a paged cache: what a server keeps while
    the batch's composition stays.  ``q_start`` (int32 [batch + 1]) gives each
    sequence's rows; without it every sequence has n_tokens // batch.
    ``group_start`` / ``prefix_len`` name the sequences that share a prefix
    (include/mpk.h: mpk_prefix_groups).  The arrays are read on the device by
    every call, so their contents may change between calls.  ``status``
    (int32 [1], optional) keeps the first error the kernels find.  The
    workspace is this object's own, allocated by the first ``attend``: calls
    of one object must not overlap on the GPU."""

    def __init__(self, kv: KVCache, n_q_heads: int, n_tokens: int,
                 q_start=None, group_start=None, prefix_len=None,
                 status=None):
        import torch
        w = "PagedBatch"
        k, v = kv.k_pool, kv.v_pool
        self._on(_cuda_device(k, w))
        if (k.dim() != 5 or k.dtype is not torch.bfloat16 or
                v.dtype is not torch.bfloat16 or v.shape != k.shape or
                not k.is_contiguous() or not v.is_contiguous() or
                v.device != self.device):
            _refuse(w, "k_pool and v_pool must be contiguous bfloat16 "
                       "[layers, pages, kv_heads, page_size, head_dim]")
        if kv.page_table.dim() != 2:
            _refuse(w, "page_table must be [batch, max_pages_per_seq]")
        batch, cols = (int(x) for x in kv.page_table.shape)
        self._vec(kv.page_table, 0, torch.int32, w, "page_table")
        self._vec(kv.seq_lens, batch, torch.int32, w, "seq_lens")
        qs = self._vec(q_start, batch + 1, torch.int32, w, "q_start")
        if batch < 1 or n_tokens < 0 or (qs is None and n_tokens % batch):
            _refuse(w, "n_tokens must be a multiple of the batch without "
                       "q_start")
        st = self._vec(status, 1, torch.int32, w, "status")
        self.kv, self.n_layers = kv, int(k.shape[0])
        self.n_tokens, self.batch = n_tokens, batch
        self.q_width = n_q_heads * int(k.shape[4])
        self.kv_width = int(k.shape[2]) * int(k.shape[4])
        self.n_q_heads, self.head_dim = n_q_heads, int(k.shape[4])
        self._shape = AttnShape(n_q_heads, int(k.shape[2]), int(k.shape[4]),
                                int(k.shape[3]), cols)
        self._tok = TokenBatch(batch, n_tokens, qs, n_tokens // batch)
        self._kv = kv.c_struct()
        self._groups = None
        if (group_start is None) != (prefix_len is None):
            _refuse(w, "group_start and prefix_len come together")
        if prefix_len is not None:
            n = int(prefix_len.numel())
            self._groups = PrefixGroups(
                n, self._vec(group_start, n + 1, torch.int32, w,
                             "group_start"),
                self._vec(prefix_len, n, torch.int32, w, "prefix_len"))
            if n < 1 or n > batch:
                _refuse(w, "1 to batch groups")
        # (the pointers of these very tensors are used, whatever kv's
        # attributes are set to later)
        self._keep = (q_start, group_start, prefix_len, status, k, v,
                      kv.page_table, kv.seq_lens)
        self._st = st
        native = _native()
        at = ctypes.addressof
        self._plan = native.paged(
            at(self._shape), at(self._tok), at(self._kv),
            at(self._groups) if self._groups else None, st, self.n_layers,
            self._index)
        self._append, self._attend = native.append, native.attend
        self._ws = None

    def append(self, layer: int, q, k, v, rope: Optional[Rope] = None,
               q_out=None, q_norm=None, k_norm=None, eps: float = 1e-6,
               stream=None):
        """mpk_kv_append: norm and rotate q and k, append k and v.  q may be
        None when q_out is."""
        at = None
        if rope is not None:
            if rope.device != self.device:
                _refuse("PagedBatch.append", "rope is on another device")
            at = rope._address
        st = self._append(self._plan, layer, q, k, v, at, q_out, q_norm,
                          k_norm, eps, stream)
        if st:
            _failed(st, "PagedBatch.append", "mpk_kv_append")

    def attend(self, layer: int, q, out, lse=None, scale: float = 0.0,
               stream=None):
        """mpk_prefix_attention of the new tokens over the cache."""
        if self._ws is None:
            import torch
            n = load_library().mpk_prefix_attention_workspace(
                ctypes.byref(self._shape), ctypes.byref(self._tok),
                self._groups.n_groups if self._groups else 0)
            self._ws = torch.empty(max(n, 1), dtype=torch.uint8,
                                   device=self.device)
            self._ws_args = (self._ws.data_ptr(), self._ws.numel())
        st = self._attend(self._plan, layer, q, out, lse, scale,
                          *self._ws_args, stream)
        if st:
            _failed(st, "PagedBatch.attend", "mpk_prefix_attention")


class DraftVerifier(_OnDevice):
    """mpk_verify_drafts with a workspace of its own (calls of one object must
    not overlap on the GPU).  ``n_tokens`` rows of ``batch`` sequences, at most
    ``max_out`` rows each."""

    def __init__(self, batch: int, n_tokens: int, vocab: int, max_out: int,
                 device="cuda", status=None):
        import torch
        w = "DraftVerifier"
        probe = torch.empty(0, dtype=torch.uint8, device=device)
        self._on(_cuda_device(probe, w))
        self.batch, self.n_tokens = batch, n_tokens
        self.vocab, self.max_out = vocab, max_out
        tok = TokenBatch(batch, n_tokens, None, n_tokens // max(batch, 1))
        n = load_library().mpk_verify_drafts_workspace(ctypes.byref(tok),
                                                       vocab)
        if n == 0 or not 1 <= max_out <= 128:
            raise MpkError(MPK_ERR_UNSUPPORTED if max_out > 128 else
                           MPK_ERR_INVALID_ARG, w)
        self._ws = torch.empty(n, dtype=torch.uint8, device=self.device)
        self._status = status
        native = _native()
        self._judge = native.judge(
            batch, n_tokens, vocab, max_out,
            self._vec(status, 1, torch.int32, w, "status"),
            self._ws.data_ptr(), n, self._index)
        self._verify = native.verify

    def verify(self, tokens, logits, uniform, noise, n_accepted, out_tokens,
               q_start=None, draft=None, draft_is_logits: bool = False,
               temperature=None, logprobs=None, next_tokens=None,
               seq_lens=None, seq_lens_out=None, stream=None):
        """Accept or refuse the drafts and sample the next tokens; arguments
        and outputs as in include/mpk.h (mpk_verify_args)."""
        st = self._verify(self._judge, tokens, logits, uniform, noise,
                          n_accepted, out_tokens, q_start, draft,
                          draft_is_logits, temperature, logprobs, next_tokens,
                          seq_lens, seq_lens_out, stream)
        if st:
            _failed(st, "DraftVerifier.verify", "mpk_verify_drafts")
