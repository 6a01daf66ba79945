"""Python binding of libdsaidx, the B200 DSA lightning-indexer library.

Argument marshalling only: every step of the indexer runs in the library's
CUDA kernels.  Tensors are torch CUDA tensors (PyTorch supplies device
memory and the current stream); the library itself allocates nothing, so
outputs and workspaces are allocated here with torch and handed over as raw
pointers.  There is no CPU fallback: importing this package fails loudly
when the compiled library is missing.

Calls go to the current stream, or to `stream` where one is given; its work then
has to come after what made the arguments.  No call records autograd history:
tensors that require a gradient are read as they are, results are detached, and
a torch.autograd.Function of the user's joins an operator and its backward pass.
Backward calls give all their gradients here; the C interface takes NULL for
one that is not wanted.

Entry points mirror include/dsa_index.h:
  index_scores, index_topk, index_topk_host, index_layers, pivot_group_index,
  pivot_refine_candidates, hisa_pool_keys, hisa_index, device_check, the
  operators an indexer is trained with (layer_norm, layer_norm_backward,
  list_scores, list_scores_backward, distill_topk), plus the *_workspace
  size queries.
"""
from __future__ import annotations

import ctypes
import functools
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
# DSA_LIBRARY=checked loads the build whose kernels verify their device-side indices; every entry
# point then also reads the workspace status word after its work (synchronising) and raises on a
# recorded error.
CHECKED = os.environ.get("DSA_LIBRARY", "") == "checked"
LIB_PATH = os.path.join(_HERE, "libdsaidx_checked.so" if CHECKED else "libdsaidx.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: build it with `python sparse_attention_indexer_04_b200/build.py` "
                      "(or __graft_entry__.build()); there is no fallback path")
_lib = ctypes.CDLL(LIB_PATH)

STATUS = {0: "ok", 1: "invalid argument", 2: "unsupported shape", 3: "workspace", 4: "CUDA error",
          5: "device check"}
REUSE, REFINE = 0, 1
BF16, FP32 = 0, 1                            # element types
TEACHER_LOGITS, TEACHER_WEIGHTS = 0, 1       # what a teacher's values are


class DsaError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {_lib.dsa_status_string(status).decode()} (status {status})")


class _Batch(ctypes.Structure):
    _fields_ = [("num_seqs", ctypes.c_int32), ("num_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("num_queries", ctypes.c_int32), ("num_keys", ctypes.c_int32),
                ("q_offsets", ctypes.c_void_p), ("k_offsets", ctypes.c_void_p), ("q_pos", ctypes.c_void_p),
                ("q_offsets_host", ctypes.c_void_p), ("k_offsets_host", ctypes.c_void_p)]


_P = ctypes.c_void_p
_B = ctypes.POINTER(_Batch)
_I32, _I64, _SZ = ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t


def _sig(name, res, *args):
    f = getattr(_lib, name)
    f.restype = res
    f.argtypes = list(args)
    return f


_sig("dsa_status_string", ctypes.c_char_p, ctypes.c_int)
_sig("dsa_version", _I32)
_sig("dsa_index_scores_workspace", _SZ, _B)
_sig("dsa_index_scores", ctypes.c_int, _B, _P, _P, _P, _P, _I64, _P, _SZ, _P)
_sig("dsa_index_topk_workspace", _SZ, _B, _I32)
_sig("dsa_index_topk", ctypes.c_int, _B, _P, _P, _P, _I32, _P, _P, _P, _SZ, _P)
_sig("dsa_index_topk_host_workspace", _SZ, _B, _I32)
_sig("dsa_index_topk_host", ctypes.c_int, _B, _P, _P, _P, _P, _I32, _P, _P, _SZ, _P, _P, _P)
_sig("pivot_num_groups", _I32, _B, _I32)
_sig("pivot_group_index_workspace", _SZ, _B, _I32, _I32, _I32, _I32)
_sig("pivot_group_index", ctypes.c_int, _B, _P, _P, _P, _I32, _I32, _I32, _I32, _P, _P, _P, _SZ, _P)
_sig("pivot_refine_candidates_workspace", _SZ, _B, _I32, _I32, _I32)
_sig("pivot_refine_candidates", ctypes.c_int, _B, _P, _P, _P, _I32, _I32, _I32, _P, _P, _P, _SZ, _P)
_sig("hisa_num_blocks", _I64, _B, _I32)
_sig("hisa_pool_keys", ctypes.c_int, _B, _P, _I32, _P, _P)
_sig("hisa_index_workspace", _SZ, _B, _I32, _I32, _I32)
_sig("hisa_index", ctypes.c_int, _B, _P, _P, _P, _P, _I32, _I32, _I32, _P, _P, _P, _SZ, _P)
_sig("dsa_device_check", ctypes.c_int, _P, _P, ctypes.POINTER(ctypes.c_uint32))
_sig("dsa_selftest_wait_timeout", ctypes.c_int, ctypes.c_uint32, _P, _SZ, _P)
_sig("dsa_index_topk_static_capacity", _SZ)
_sig("dsa_index_topk_static", ctypes.c_int, _B, _P, _P, _P, _I32, _P, _P, _P)
_sig("dsa_index_layers_source", _I32, _I32, _I32, _I32)
_sig("dsa_index_layers_workspace", _SZ, _B, _I32)
_sig("dsa_index_layers", ctypes.c_int, _B, _I32, ctypes.POINTER(_P), ctypes.POINTER(_P), ctypes.POINTER(_P), _I32,
     _I32, _I32, ctypes.POINTER(_P), ctypes.POINTER(_P), _P, _SZ, _P, _P)
_sig("dsa_layer_norm", ctypes.c_int, _I64, _I32, _P, _I32, _I64, _P, _P, ctypes.c_float, _P, _I32, _I64, _P, _P, _P)
_sig("dsa_layer_norm_backward_workspace", _SZ, _I64, _I32)
_sig("dsa_layer_norm_backward", ctypes.c_int, _I64, _I32, _P, _I32, _I64, _P, _I32, _I64, _P, _P, _P, _P, _I64, _P,
     _P, _P, _SZ, _P)
_sig("dsa_distill_topk", ctypes.c_int, _I32, _I32, _P, _I64, _P, _I64, _P, _I32, _I64, _I32, ctypes.c_float, _P, _P,
     _P, _I64, _P)
_sig("dsa_list_scores_workspace", _SZ, _B, _I32)
_sig("dsa_list_scores", ctypes.c_int, _B, _P, _P, _P, _I32, _P, _P, _P, _SZ, _P)
_sig("dsa_list_scores_backward_workspace", _SZ, _B, _I32)
_sig("dsa_list_scores_backward", ctypes.c_int, _B, _P, _P, _P, _I32, _P, _P, _P, _P, _P, _P, _SZ, _P)
_sig("dsa_profile_enable", None, _I32)
_sig("dsa_launch_count", ctypes.c_uint64)
_sig("dsa_profile_kind_name", ctypes.c_char_p, _I32)
_sig("dsa_profile_read", _I32, ctypes.POINTER(ctypes.c_float), ctypes.POINTER(ctypes.c_int32), _I32)


def library():
    return _lib


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _check(status: int, where: str):
    if status != 0:
        raise DsaError(status, where)


ERR_BAD_INDEX = 4   # status-word code of the checked build: a device-side index outside its buffer


def _after(ws, where: str, stream=None):
    """Checked build only: wait for the call's work and raise if a kernel recorded an index error in
    the workspace status word (other codes are left for device_check)."""
    if not CHECKED:
        return
    torch.cuda.synchronize()   # every stream the call used
    code, detail = (int(x) for x in ws[:8].view(torch.int32).cpu())
    if code == ERR_BAD_INDEX:
        raise DsaError(5, f"{where}: device index check failed at site {detail}")


class Layout:
    """Sequence layout of a batch: offsets and positions on the device plus host copies.

    q_offsets / k_offsets: [B+1] row offsets of each sequence's queries / keys;
    q_pos: [n_q] sequence-local position of each query.
    """

    def __init__(self, q_offsets, k_offsets, q_pos, num_heads: int, head_dim: int, device="cuda"):
        self.q_off_host = torch.as_tensor(q_offsets, dtype=torch.int32).cpu().contiguous()
        self.k_off_host = torch.as_tensor(k_offsets, dtype=torch.int32).cpu().contiguous()
        self.q_off = self.q_off_host.to(device)
        self.k_off = self.k_off_host.to(device)
        self.q_pos = torch.as_tensor(q_pos, dtype=torch.int32).to(device).contiguous()
        self.num_heads, self.head_dim = int(num_heads), int(head_dim)
        self.device = torch.device(device)
        self.c = _Batch(int(self.q_off_host.numel() - 1), self.num_heads, self.head_dim,
                        int(self.q_off_host[-1]), int(self.k_off_host[-1]),
                        self.q_off.data_ptr(), self.k_off.data_ptr(),
                        self.q_pos.data_ptr() if self.q_pos.numel() else None,
                        self.q_off_host.data_ptr(), self.k_off_host.data_ptr())

    @classmethod
    def from_batch(cls, b, device="cuda"):
        return cls(b.q_offsets, b.k_offsets, b.q_pos, b.H, b.d, device)

    @property
    def num_queries(self):
        return self.c.num_queries

    @property
    def max_keys(self):
        ko = self.k_off_host
        return int((ko[1:] - ko[:-1]).max()) if ko.numel() > 1 else 0

    def ref(self):
        return ctypes.byref(self.c)


def _workspace(nbytes: int, device, ws=None):
    if ws is not None:
        return ws
    # 256-byte aligned: torch's caching allocator returns 512-byte aligned blocks
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)


def _bytes(ws):
    return ctypes.c_size_t(ws.numel() * ws.element_size())


def _tensors(x):
    """The CUDA tensors of an argument or a result."""
    if isinstance(x, torch.Tensor):
        return [x] if x.is_cuda else []
    if isinstance(x, Layout):
        return _tensors([x.q_off, x.k_off, x.q_pos])
    return [t for y in x for t in _tensors(y)] if isinstance(x, (list, tuple)) else []


def _on_stream(stream, index, call, *args):
    """call(*args) with `stream`, of the CUDA device `index`, as the current one.  Outputs and workspaces are then
    made from that stream's memory: from the caller's stream's, they could be blocks that work pending there still
    uses.  The allocator learns that the arguments are in use on `stream` and the results on the caller's."""
    if stream.device.index != index:
        raise ValueError(f"the stream is on {stream.device}, the tensors on cuda:{index}")
    caller = torch.cuda.current_stream(index)
    with torch.cuda.stream(stream):
        out = call(*args)
    for t in _tensors(args):
        t.record_stream(stream)
    for t in _tensors(out):
        t.record_stream(stream)
        t.record_stream(caller)
    return out


# ------------------------------------------------------------------- dense

def index_scores_workspace(layout: Layout) -> int:
    return int(_lib.dsa_index_scores_workspace(layout.ref()))


def index_scores(layout: Layout, Q, K, W, S=None, ws=None, stream=None):
    """Dense indexer scores: S [n_q, ld] fp32, -inf where the key is not eligible."""
    if stream is not None:
        return _on_stream(stream, layout.q_off.get_device(), index_scores, layout, Q, K, W, S, ws)
    if S is None:
        S = torch.empty(layout.num_queries, max(layout.max_keys, 1), dtype=torch.float32, device=layout.device)
    ws = _workspace(index_scores_workspace(layout), layout.device, ws)
    _check(_lib.dsa_index_scores(layout.ref(), _ptr(Q), _ptr(K), _ptr(W), _ptr(S), S.stride(0), _ptr(ws),
                                 _bytes(ws), _stream()), "dsa_index_scores")
    _after(ws, "dsa_index_scores")
    return S


def index_topk_workspace(layout: Layout, k: int) -> int:
    return int(_lib.dsa_index_topk_workspace(layout.ref(), k))


def index_topk(layout: Layout, Q, K, W, k: int, idx=None, scores=None, want_scores=False, ws=None, stream=None):
    """Dense indexer top-k: idx [n_q, k] int32 (ascending, -1 padded), optional scores [n_q, k]."""
    if stream is not None:
        return _on_stream(stream, layout.q_off.get_device(), index_topk, layout, Q, K, W, k, idx, scores,
                          want_scores, ws)
    if idx is None:
        idx = torch.empty(layout.num_queries, k, dtype=torch.int32, device=layout.device)
    if want_scores and scores is None:
        scores = torch.empty(layout.num_queries, k, dtype=torch.float32, device=layout.device)
    ws = _workspace(index_topk_workspace(layout, k), layout.device, ws)
    _check(_lib.dsa_index_topk(layout.ref(), _ptr(Q), _ptr(K), _ptr(W), k, _ptr(idx), _ptr(scores), _ptr(ws),
                               _bytes(ws), _stream()), "dsa_index_topk")
    _after(ws, "dsa_index_topk")
    return (idx, scores) if want_scores else idx


def index_layers_source(layer: int, retain_every: int, lag: int) -> int:
    """The layer whose indexer run gives `layer` its selection (-1 for invalid arguments)."""
    return int(_lib.dsa_index_layers_source(layer, retain_every, lag))


def index_layers(layout: Layout, Qs, Ks, Ws, k: int, retain_every: int = 1, lag: int = 0, idx=None, events=None,
                 ws=None, stream=None, side_stream=None):
    """Selections of len(Qs) layers (dsa_index_layers): idx[l] [n_q, k] int32 for layer l.  `events`: optional
    torch.cuda.Event per layer, recorded once idx[l] is complete (then `stream` is not made to wait)."""
    if stream is not None:
        return _on_stream(stream, layout.q_off.get_device(), index_layers, layout, Qs, Ks, Ws, k, retain_every, lag,
                          idx, events, ws, None, side_stream)
    n = len(Qs)
    if not (len(Ks) == len(Ws) == n):
        raise ValueError("one Q, K and W per layer")
    if idx is None:
        idx = [torch.empty(layout.num_queries, k, dtype=torch.int32, device=layout.device) for _ in range(n)]
    if side_stream is None:
        raise ValueError("index_layers needs a side stream distinct from the compute stream")
    arr = lambda ts: (_P * n)(*[t.data_ptr() for t in ts])
    ev = None
    if events is not None:
        for e in events:
            e.record()   # creates the event
        ev = (_P * n)(*[e.cuda_event for e in events])
    ws = _workspace(int(_lib.dsa_index_layers_workspace(layout.ref(), k)), layout.device, ws)
    _check(_lib.dsa_index_layers(layout.ref(), n, arr(Qs), arr(Ks), arr(Ws), k, retain_every, lag, arr(idx), ev,
                                 _ptr(ws), _bytes(ws), _stream(), _stream(side_stream)), "dsa_index_layers")
    _after(ws, "dsa_index_layers")
    if events is not None:   # (else this stream waits for the side stream, and later work here comes after it)
        for t in _tensors([layout, Qs, Ks, Ws, ws, idx]):
            t.record_stream(side_stream)
    return idx


def index_topk_host_workspace(layout: Layout, k: int) -> int:
    return int(_lib.dsa_index_topk_host_workspace(layout.ref(), k))


def index_topk_host(layout: Layout, q_pos, Q, K, W, k: int, idx, ws, stream=None, in_stream=None, out_stream=None):
    """dsa_index_topk on HOST tensors (pinned for overlap): Q, K, W, q_pos (CPU) in, idx [n_q, k] (CPU,
    int32) out.  The copies run on in_stream / out_stream (torch.cuda.Stream) overlapped with the
    work on `stream`; idx is complete once `stream` has passed the call."""
    for t in (q_pos, Q, K, W, idx):
        if t.is_cuda or not t.is_contiguous():
            raise ValueError("index_topk_host takes contiguous host tensors")
    if in_stream is None or out_stream is None:
        raise ValueError("index_topk_host needs copy streams distinct from the compute stream")
    _check(_lib.dsa_index_topk_host(layout.ref(), _ptr(q_pos), _ptr(Q), _ptr(K), _ptr(W), k, _ptr(idx), _ptr(ws),
                                    _bytes(ws), _stream(stream), _stream(in_stream), _stream(out_stream)),
           "dsa_index_topk_host")
    _after(ws, "dsa_index_topk_host", stream)
    return idx


def index_topk_static(layout: Layout, Q, K, W, k: int, idx=None, scores=None, want_scores=False, stream=None):
    """dsa_index_topk with the library's built-in device scratch instead of a workspace (allocates nothing
    in the library; for callers that cannot allocate).  Calls on one device must not overlap on the GPU."""
    if stream is not None:
        return _on_stream(stream, layout.q_off.get_device(), index_topk_static, layout, Q, K, W, k, idx, scores,
                          want_scores)
    if idx is None:
        idx = torch.empty(layout.num_queries, k, dtype=torch.int32, device=layout.device)
    if want_scores and scores is None:
        scores = torch.empty(layout.num_queries, k, dtype=torch.float32, device=layout.device)
    _check(_lib.dsa_index_topk_static(layout.ref(), _ptr(Q), _ptr(K), _ptr(W), k, _ptr(idx), _ptr(scores),
                                      _stream()), "dsa_index_topk_static")
    return (idx, scores) if want_scores else idx


def index_topk_static_capacity() -> int:
    return int(_lib.dsa_index_topk_static_capacity())


# ------------------------------------------------------------------- PIVOT

def pivot_num_groups(layout: Layout, group: int) -> int:
    return int(_lib.pivot_num_groups(layout.ref(), group))


def pivot_group_index_workspace(layout: Layout, k: int, group: int, n_cand: int, mode: int) -> int:
    return int(_lib.pivot_group_index_workspace(layout.ref(), k, group, n_cand, mode))


def pivot_group_index(layout: Layout, Q, K, W, k: int, group: int, n_cand: int, mode: int, idx=None, cand=None,
                      want_cand=False, ws=None, stream=None):
    """PIVOT Reuse (mode 0) / Refine (mode 1): idx [n_q, k]; optional cand [n_groups, n_cand]."""
    if stream is not None:
        return _on_stream(stream, layout.q_off.get_device(), pivot_group_index, layout, Q, K, W, k, group, n_cand,
                          mode, idx, cand, want_cand, ws)
    if idx is None:
        idx = torch.empty(layout.num_queries, k, dtype=torch.int32, device=layout.device)
    if want_cand and cand is None:
        cand = torch.empty(max(pivot_num_groups(layout, group), 0), n_cand, dtype=torch.int32, device=layout.device)
    ws = _workspace(pivot_group_index_workspace(layout, k, group, n_cand, mode), layout.device, ws)
    _check(_lib.pivot_group_index(layout.ref(), _ptr(Q), _ptr(K), _ptr(W), k, group, n_cand, mode, _ptr(idx),
                                  _ptr(cand), _ptr(ws), _bytes(ws), _stream()), "pivot_group_index")
    _after(ws, "pivot_group_index")
    return (idx, cand) if want_cand else idx


def pivot_refine_candidates_workspace(layout: Layout, k: int, group: int, n_cand: int) -> int:
    return int(_lib.pivot_refine_candidates_workspace(layout.ref(), k, group, n_cand))


def pivot_refine_candidates(layout: Layout, Q, K, W, k: int, group: int, cand, idx=None, ws=None, stream=None):
    """Refine on supplied candidates: cand [n_groups, n_cand] int32 (ascending, -1 padded) -> idx [n_q, k]."""
    if stream is not None:
        return _on_stream(stream, layout.q_off.get_device(), pivot_refine_candidates, layout, Q, K, W, k, group,
                          cand, idx, ws)
    n_cand = int(cand.shape[1])
    if idx is None:
        idx = torch.empty(layout.num_queries, k, dtype=torch.int32, device=layout.device)
    ws = _workspace(pivot_refine_candidates_workspace(layout, k, group, n_cand), layout.device, ws)
    _check(_lib.pivot_refine_candidates(layout.ref(), _ptr(Q), _ptr(K), _ptr(W), k, group, n_cand, _ptr(cand),
                                        _ptr(idx), _ptr(ws), _bytes(ws), _stream()), "pivot_refine_candidates")
    _after(ws, "pivot_refine_candidates")
    return idx


# -------------------------------------------------------------------- HISA

def hisa_num_blocks(layout: Layout, block: int) -> int:
    return int(_lib.hisa_num_blocks(layout.ref(), block))


def hisa_pool_keys(layout: Layout, K, block: int, pooled=None, stream=None):
    """Mean-pooled block keys [n_blocks, d] fp32."""
    if stream is not None:
        return _on_stream(stream, layout.q_off.get_device(), hisa_pool_keys, layout, K, block, pooled)
    if pooled is None:
        pooled = torch.empty(max(hisa_num_blocks(layout, block), 0), layout.head_dim, dtype=torch.float32,
                             device=layout.device)
    _check(_lib.hisa_pool_keys(layout.ref(), _ptr(K), block, _ptr(pooled), _stream()), "hisa_pool_keys")
    return pooled


def hisa_index_workspace(layout: Layout, k: int, block: int, keep: int) -> int:
    return int(_lib.hisa_index_workspace(layout.ref(), k, block, keep))


def hisa_index(layout: Layout, Q, K, W, pooled, k: int, block: int, keep: int, idx=None, kept=None,
               want_kept=False, ws=None, stream=None):
    """HISA top-k: idx [n_q, k]; optional kept [n_q, keep+2] block lists."""
    if stream is not None:
        return _on_stream(stream, layout.q_off.get_device(), hisa_index, layout, Q, K, W, pooled, k, block, keep,
                          idx, kept, want_kept, ws)
    if idx is None:
        idx = torch.empty(layout.num_queries, k, dtype=torch.int32, device=layout.device)
    if want_kept and kept is None:
        kept = torch.empty(layout.num_queries, keep + 2, dtype=torch.int32, device=layout.device)
    ws = _workspace(hisa_index_workspace(layout, k, block, keep), layout.device, ws)
    _check(_lib.hisa_index(layout.ref(), _ptr(Q), _ptr(K), _ptr(W), _ptr(pooled), k, block, keep, _ptr(idx),
                           _ptr(kept), _ptr(ws), _bytes(ws), _stream()), "hisa_index")
    _after(ws, "hisa_index")
    return (idx, kept) if want_kept else idx


# ---------------------------------------------------------------- training

_TYPES = {torch.bfloat16: BF16, torch.float32: FP32}
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


_I32_MAX = 2 ** 31 - 1


def _rows(t, name, index, n=None, d=None, dtype=None):
    """Row stride of a 2-D matrix that the library can read in place: adjacent values along a row, on the
    CUDA device `index`."""
    shape = t.shape
    if len(shape) != 2 or (n is not None and (shape[0] != n or shape[1] != d)):
        raise ValueError(f"{name}: expected a 2-D tensor{'' if n is None else f' of shape {(n, d)}'}, "
                         f"got {tuple(shape)}")
    if shape[1] > _I32_MAX:   # (the library counts them in 32 bits, and ctypes would cut the number)
        raise ValueError(f"{name}: rows of {shape[1]} values are too long")
    if t.dtype not in _TYPES if dtype is None else t.dtype != dtype:
        raise ValueError(f"{name}: {t.dtype} is not supported here")
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, expected cuda:{index}")
    ld, unit = t.stride()
    if shape[1] > 1 and unit != 1:
        raise ValueError(f"{name}: values of a row must be adjacent")
    if shape[0] <= 1:
        return shape[1]
    if ld < shape[1]:
        raise ValueError(f"{name}: rows overlap")
    return ld


def _dense(t, name, index, shape, dtype):
    """Address of a contiguous tensor of the given shape and type on the CUDA device `index`; None passes."""
    if t is None:
        return None
    if t.shape != shape or t.dtype != dtype or t.get_device() != index or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous {dtype} tensor of shape {tuple(shape)} on cuda:{index}, got "
                         f"{t.dtype} {tuple(t.shape)} on {t.device}")
    return t.data_ptr()


def _device(t):
    """The CUDA device index of a tensor (the library has no CPU path)."""
    if not t.is_cuda:
        raise ValueError("expected CUDA tensors")
    return t.get_device()


def _on(index, call, *args):
    """call(*args, stream) with the CUDA device `index` current and that device's current stream."""
    if index != torch.cuda.current_device():
        with torch.cuda.device(index):
            return _on(index, call, *args)
    if _raw_stream is not None:
        raw = _raw_stream(index)
    else:
        raw = torch.cuda.current_stream(index).cuda_stream
    return call(*args, raw)


def layer_norm(x, weight=None, bias=None, eps: float = 1e-6, out=None, out_dtype=None, want_stats=False, stream=None):
    """Layer norm of the rows of x [n, d] (bf16 or fp32; rows may be a slice of a wider matrix): y [n, d] of
    out_dtype (x's by default); with want_stats also mean and rstd [n] fp32, which the backward pass takes."""
    if stream is not None:
        return _on_stream(stream, _device(x), layer_norm, x, weight, bias, eps, out, out_dtype, want_stats)
    dev = _device(x)
    ld_x = _rows(x, "x", dev)
    n, d = x.shape
    w, b = _dense(weight, "weight", dev, (d,), torch.float32), _dense(bias, "bias", dev, (d,), torch.float32)
    if out is None:
        out = x.new_empty((n, d), dtype=out_dtype)
    ld_y = _rows(out, "out", dev, n, d)
    mean = rstd = mp = rp = None
    if want_stats:
        mean, rstd = x.new_empty(n, dtype=torch.float32), x.new_empty(n, dtype=torch.float32)
        mp, rp = mean.data_ptr(), rstd.data_ptr()
    _check(_on(dev, _lib.dsa_layer_norm, n, d, x.data_ptr(), _TYPES[x.dtype], ld_x, w, b, eps, out.data_ptr(),
               _TYPES[out.dtype], ld_y, mp, rp), "dsa_layer_norm")
    return (out, mean, rstd) if want_stats else out


@functools.lru_cache(maxsize=256)
def layer_norm_backward_workspace(n: int, d: int) -> int:
    return int(_lib.dsa_layer_norm_backward_workspace(n, d))


def layer_norm_backward(dy, x, weight, mean, rstd, dx=None, ws=None, stream=None):
    """Backward pass of layer_norm: (dx [n, d] of x's type, dweight [d], dbias [d] fp32)."""
    if stream is not None:
        return _on_stream(stream, _device(x), layer_norm_backward, dy, x, weight, mean, rstd, dx, ws)
    dev = _device(x)
    ld_x = _rows(x, "x", dev)
    n, d = x.shape
    ld_dy = _rows(dy, "dy", dev, n, d)
    w = _dense(weight, "weight", dev, (d,), torch.float32)
    mp, rp = _dense(mean, "mean", dev, (n,), torch.float32), _dense(rstd, "rstd", dev, (n,), torch.float32)
    if dx is None:
        dx = x.new_empty((n, d))
    ld_dx = _rows(dx, "dx", dev, n, d, x.dtype)
    dw, db = x.new_empty(d, dtype=torch.float32), x.new_empty(d, dtype=torch.float32)
    if ws is None:
        ws = _workspace(layer_norm_backward_workspace(n, d), x.device)
    _check(_on(dev, _lib.dsa_layer_norm_backward, n, d, dy.data_ptr(), _TYPES[dy.dtype], ld_dy, x.data_ptr(),
               _TYPES[x.dtype], ld_x, w, mp, rp, dx.data_ptr(), ld_dx, dw.data_ptr(), db.data_ptr(), ws.data_ptr(),
               ws.numel() * ws.element_size()), "dsa_layer_norm_backward")
    return dx, dw, db


def distill_topk(scores, teacher, lists=None, kind: int = TEACHER_LOGITS, temperature: float = 1.0, grad_loss=None,
                 loss=None, dscores=None, stream=None):
    """Distillation loss of each row's scores [n, k] from a teacher's logits or weights on the same places, and
    its gradient: (loss [n], dscores [n, k]).  Places with a negative entry in `lists` or a score of -inf do not
    count.  grad_loss [n]: the gradient of each row's loss (ones by default)."""
    if stream is not None:
        return _on_stream(stream, _device(scores), distill_topk, scores, teacher, lists, kind, temperature,
                          grad_loss, loss, dscores)
    dev = _device(scores)
    ld_s = _rows(scores, "scores", dev, dtype=torch.float32)
    n, k = scores.shape
    if n > _I32_MAX:
        raise ValueError(f"scores: {n} rows are too many")
    ld_t = _rows(teacher, "teacher", dev, n, k)
    lp, ld_l = (None, 0) if lists is None else (lists.data_ptr(), _rows(lists, "lists", dev, n, k, torch.int32))
    g = _dense(grad_loss, "grad_loss", dev, (n,), torch.float32)
    if loss is None:
        loss = scores.new_empty(n)
    if dscores is None:
        dscores = scores.new_empty((n, k))
    ld_d = _rows(dscores, "dscores", dev, n, k, torch.float32)
    _check(_on(dev, _lib.dsa_distill_topk, n, k, scores.data_ptr(), ld_s, lp, ld_l, teacher.data_ptr(),
               _TYPES[teacher.dtype], ld_t, kind, temperature, g, _dense(loss, "loss", dev, (n,), torch.float32),
               dscores.data_ptr(), ld_d), "dsa_distill_topk")
    return loss, dscores


def _list_inputs(layout, Q, K, W, lists):
    """Device index, list length, and the addresses of Q, K, W and lists."""
    dev = _device(Q)
    c = layout.c
    H, d, n_q = c.num_heads, c.head_dim, c.num_queries
    if layout.q_off.get_device() != dev:
        raise ValueError(f"Q is on {Q.device}, the layout on {layout.q_off.device}")
    if lists.dim() != 2:
        raise ValueError("lists: expected [n_q, k]")
    k = lists.shape[1]
    return (dev, k, _dense(Q, "Q", dev, (n_q, H, d), torch.bfloat16),
            _dense(K, "K", dev, (c.num_keys, d), torch.bfloat16), _dense(W, "W", dev, (n_q, H), torch.float32),
            _dense(lists, "lists", dev, (n_q, k), torch.int32))


def list_scores_workspace(layout: Layout, k: int) -> int:
    return int(_lib.dsa_list_scores_workspace(layout.ref(), k))


def list_scores(layout: Layout, Q, K, W, lists, scores=None, ws=None, stream=None):
    """Indexer scores at listed keys: lists [n_q, k] int32 (ascending, -1 padded) -> scores [n_q, k] fp32, -inf
    where a place is empty or its key is not in the query's prefix."""
    if stream is not None:
        return _on_stream(stream, _device(Q), list_scores, layout, Q, K, W, lists, scores, ws)
    dev, k, q, kk, w, l = _list_inputs(layout, Q, K, W, lists)
    if scores is None:
        scores = W.new_empty(lists.shape)
    if ws is None:
        ws = _workspace(list_scores_workspace(layout, k), Q.device)
    _check(_on(dev, _lib.dsa_list_scores, layout.ref(), q, kk, w, k, l,
               _dense(scores, "scores", dev, lists.shape, torch.float32), ws.data_ptr(), ws.numel() * ws.element_size()),
           "dsa_list_scores")
    _after(ws, "dsa_list_scores")
    return scores


def list_scores_backward_workspace(layout: Layout, k: int) -> int:
    return int(_lib.dsa_list_scores_backward_workspace(layout.ref(), k))


def list_scores_backward(layout: Layout, Q, K, W, lists, dscores, dQ=None, dK=None, dW=None, ws=None, stream=None):
    """Backward pass of list_scores: (dQ [n_q, H, d] bf16, dK [n_k, d] bf16, dW [n_q, H] fp32)."""
    if stream is not None:
        return _on_stream(stream, _device(Q), list_scores_backward, layout, Q, K, W, lists, dscores, dQ, dK, dW, ws)
    dev, k, q, kk, w, l = _list_inputs(layout, Q, K, W, lists)
    ds = _dense(dscores, "dscores", dev, lists.shape, torch.float32)
    dQ = torch.empty_like(Q) if dQ is None else dQ
    dK = torch.empty_like(K) if dK is None else dK
    dW = torch.empty_like(W) if dW is None else dW
    if ws is None:
        ws = _workspace(list_scores_backward_workspace(layout, k), Q.device)
    _check(_on(dev, _lib.dsa_list_scores_backward, layout.ref(), q, kk, w, k, l, ds,
               _dense(dQ, "dQ", dev, Q.shape, torch.bfloat16), _dense(dK, "dK", dev, K.shape, torch.bfloat16),
               _dense(dW, "dW", dev, W.shape, torch.float32), ws.data_ptr(), ws.numel() * ws.element_size()),
           "dsa_list_scores_backward")
    _after(ws, "dsa_list_scores_backward")
    return dQ, dK, dW


def launch_count() -> int:
    """Kernels this library has launched since it was loaded."""
    return int(_lib.dsa_launch_count())


def profile_enable(on: bool = True):
    """Bracket every later launch with CUDA events on its own stream (see profile_read)."""
    _lib.dsa_profile_enable(1 if on else 0)


def profile_read():
    """{kernel kind: (total ms, launches)} since the last read; synchronises the recorded events."""
    cap = 32
    ms = (ctypes.c_float * cap)()
    n = (ctypes.c_int32 * cap)()
    kinds = _lib.dsa_profile_read(ms, n, cap)
    if kinds < 0:
        raise DsaError(4, "dsa_profile_read")
    return {_lib.dsa_profile_kind_name(i).decode(): (float(ms[i]), int(n[i])) for i in range(kinds) if n[i]}


def selftest_wait_timeout(limit_us: int, ws, stream=None):
    """Launch the bounded-wait self-test: a wait nothing completes runs out after limit_us and records
    code 1 in ws's status word (read it with device_check)."""
    _check(_lib.dsa_selftest_wait_timeout(limit_us, _ptr(ws), _bytes(ws), _stream(stream)),
           "dsa_selftest_wait_timeout")


def device_check(ws, stream=None) -> int:
    """Status word recorded by kernels in a workspace (0 = none); synchronises the stream."""
    detail = ctypes.c_uint32(0)
    st = _lib.dsa_device_check(_ptr(ws), _stream(stream), ctypes.byref(detail))
    if st not in (0, 5):
        raise DsaError(st, "dsa_device_check")
    return int(detail.value) if st == 5 else 0
