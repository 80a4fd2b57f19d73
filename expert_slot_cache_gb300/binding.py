"""ctypes binding of libmoeslot.so (argument marshalling only).

Every computation runs in the library's CUDA kernels; this module allocates
output tensors with PyTorch, passes raw pointers and the current CUDA stream,
and turns a negative status into an exception.  There is no fallback: if the
library is missing, importing this module raises.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import inspect
import os
from ctypes import POINTER, c_float, c_int, c_int32, c_size_t, c_void_p
from dataclasses import dataclass
from typing import NamedTuple, Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_lib", "libmoeslot.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is not built; run `python __graft_entry__.py` "
        "(or __graft_entry__.build()) first")

lib = ctypes.CDLL(LIB_PATH)

MODE_RESIDENT, MODE_GATHER, MODE_ZERO_RETURN = 0, 1, 2
POLICY_LRU, POLICY_LFU, POLICY_STATIC = 0, 1, 2
DEV_BAD_EXPERT, DEV_BAD_SLOT = 1, 2


PROF_CLASSES = ("route", "permute", "manage", "gather", "ffn_gateup", "ffn_down", "combine", "ffn_rows")


class Prof(ctypes.Structure):
    _fields_ = [("events", POINTER(c_void_p)), ("capacity", c_int32), ("used", c_int32),
                ("tags", POINTER(c_int32))]


class LayerArgs(ctypes.Structure):
    _fields_ = [("T", c_int32), ("H", c_int32), ("E", c_int32), ("k", c_int32), ("I", c_int32), ("S", c_int32),
                ("mode", c_int32), ("policy", c_int32),
                ("x", c_void_p), ("w_router", c_void_p), ("logit_offset", c_void_p), ("sel_bias", c_void_p),
                ("pool", c_void_p), ("host_slabs", c_void_p),
                ("e2s", c_void_p), ("s2e", c_void_p), ("prio", c_void_p), ("stamp", c_void_p),
                ("ids", c_void_p), ("w", c_void_p), ("out", c_void_p), ("out_res", c_void_p),
                ("out_miss", c_void_p), ("stats", c_void_p), ("dev_status", c_void_p),
                ("workspace", c_void_p), ("workspace_bytes", c_size_t), ("prof", POINTER(Prof)),
                ("affinity", c_float), ("route_flags", c_int32), ("window_counts", c_void_p), ("quant", c_int32),
                ("schedule", c_int32), ("decode_kernels", c_int32), ("quant_group", c_int32)]


def _sig(name, argtypes, restype=c_int):
    f = getattr(lib, name)
    f.argtypes = argtypes
    f.restype = restype
    return f


V = c_void_p
I32 = c_int
_status_str = _sig("moe_status_str", [c_int], ctypes.c_char_p)
_bias_table = _sig("moe_bias_table", [V, I32, I32, c_float, V, V])
_bias_table_mode = _sig("moe_bias_table_mode", [V, I32, I32, I32, c_float, V, V])
_route = _sig("moe_route", [V, V, V, V, V, c_float, I32, I32, I32, I32, V, V, V, V, V])
_route_ex = _sig("moe_route_ex", [V, V, V, V, V, c_float, I32, I32, I32, I32, I32, V, V, V, V, V])

BIAS_GRADED, BIAS_FLAT, BIAS_HARD = 0, 1, 2
SCHED_CHUNKS, SCHED_WAVES = 0, 1
ROUTE_SIGMOID, ROUTE_DAMPED, ROUTE_GROUP_MAX, ROUTE_RAW = 1, 2, 4, 8
_route_scratch = _sig("moe_route_scratch_bytes", [I32, I32, I32], c_size_t)
_permute = _sig("moe_permute", [V, I32, I32, V, V, V, V, V, V, V, V, V])
_permute_scratch = _sig("moe_permute_scratch_bytes", [I32, I32], c_size_t)
_manage = _sig("moe_cache_manage", [V, I32, I32, I32, I32, V, V, V, V, V, V, V, V, V, V, V, V])
_gather = _sig("moe_cache_gather", [V, V, c_size_t, I32, I32, V, V, V, I32, V, V])
_count = _sig("moe_cache_count", [V, I32, I32, V, V, V])
_q8_slab = _sig("moe_q8_slab_bytes", [I32, I32], c_size_t)
_quantize = _sig("moe_quantize_slabs", [V, I32, I32, I32, V, V])
_ffn_q8_ws = _sig("moe_ffn_q8_workspace_bytes", [I32, I32, I32, I32], c_size_t)
_ffn_q8 = _sig("moe_expert_ffn_q8", [V, I32, I32, I32, I32, I32, V, V, V, V, I32, V, I32, V, V, V, c_size_t, V, V])
_repick = _sig("moe_cache_repick", [V, I32, I32, V, V, V, V, V, V])
_ffn = _sig("moe_expert_ffn", [V, I32, I32, I32, I32, I32, V, V, V, V, I32, V, I32, V, V, V, V, c_size_t, V, V])
_ffn_ws = _sig("moe_ffn_workspace_bytes", [I32, I32, I32, I32], c_size_t)
_combine = _sig("moe_combine", [V, V, V, V, V, I32, I32, I32, I32, I32, V, V, V, V])
LL = ctypes.c_longlong
_w4_bytes = _sig("moe_w4_bytes", [I32, I32, I32], c_size_t)
_w4_slab = _sig("moe_w4_slab_bytes", [I32, I32, I32], c_size_t)
_w4_pack = _sig("moe_w4_pack", [V, V, I32, I32, I32, I32, V, V])
_w4_quantize = _sig("moe_w4_quantize", [V, I32, I32, I32, I32, V, V])
_w4_pack_slabs = _sig("moe_w4_pack_slabs", [V, V, I32, I32, I32, I32, V, V])
_w4_quantize_slabs = _sig("moe_w4_quantize_slabs", [V, I32, I32, I32, I32, V, V])
_w4_linear_ws = _sig("moe_w4_linear_workspace_bytes", [I32, I32, I32, I32], c_size_t)
_w4_linear = _sig("moe_w4_linear", [V, LL, I32, I32, I32, I32, V, V, LL, I32, V, c_size_t, V, V])
_ffn_w4_ws = _sig("moe_ffn_w4_workspace_bytes", [I32, I32, I32, I32], c_size_t)
_ffn_w4 = _sig("moe_expert_ffn_w4", [V, I32, I32, I32, I32, I32, I32, V, V, V, V, I32, V, I32, V, V, V, c_size_t, V, V])
_experts_w4_ws = _sig("moe_experts_w4_workspace_bytes", [I32, I32, I32, I32, I32], c_size_t)
_experts_w4 = _sig("moe_experts_w4", [V, V, V, I32, I32, I32, I32, I32, I32, V, I32, V, V, V, c_size_t, V, V])
_balance_ws = _sig("moe_balance_workspace_bytes", [I32, I32, I32], c_size_t)
_balance = _sig("moe_balance_loss", [V, I32, V, V, V, I32, I32, I32, I32, I32, c_float, V, V, V, V, V, c_size_t, V, V])
_route_groups = _sig("moe_route_groups", [V, I32, V, V, I32, I32, I32, I32, I32, I32, c_float, V, V, V])
_route_groups_grad = _sig("moe_route_groups_grad", [V, I32, V, V, I32, I32, I32, I32, c_float, V, V, V])
_adapters = _sig("moe_adapters", [V, LL, V, LL, I32, I32, I32, I32, I32, V, V, V, V, V, I32, V, LL, I32, V, V, V])
_adapters_grad_ws = _sig("moe_adapters_grad_workspace_bytes", [I32, I32], c_size_t)
_adapters_grad = _sig("moe_adapters_grad", [V, LL, V, LL, V, V, LL, I32, I32, I32, I32, I32, V, V, V, V, V, I32, V, LL, V, V,
                                            V, c_size_t, V, V])
_layer = _sig("moe_layer_forward", [POINTER(LayerArgs), V, V])
_layer_ws = _sig("moe_layer_workspace_bytes", [I32, I32, I32, I32, I32, I32], c_size_t)


class MoeError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {status_str(code)} ({code})")


def status_str(code: int) -> str:
    return _status_str(code).decode()


def _ck(rc: int, where: str) -> None:
    if rc != 0:
        raise MoeError(rc, where)


def _p(t: Optional[torch.Tensor]):
    return None if t is None else c_void_p(t.data_ptr())


def _ptr(t: Optional[torch.Tensor]) -> int:
    return 0 if t is None else t.data_ptr()


def _s(stream=None):
    s = torch.cuda.current_stream() if stream is None else stream
    return c_void_p(s.cuda_stream)


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _here(index: int, stream=None) -> int:
    """The handle of ``stream``, or of the current stream of CUDA device ``index``."""
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None:
        return _raw_stream(index)
    return torch.cuda.current_stream(index).cuda_stream


def _on(dev: torch.device, **tensors) -> None:
    """Refuses tensors that are not all on the CUDA device ``dev``: the kernels get their addresses as they are."""
    if dev.type != "cuda":
        raise ValueError(f"need tensors on a CUDA device, got {dev}")
    index = dev.index
    for name, t in tensors.items():
        if t is not None and t.get_device() != index:
            raise ValueError(f"{name}: on {t.device}, the call runs on {dev}")


def _for_its_stream(call):
    """A call given a ``stream`` allocates its temporaries and results for that stream.  From the current stream's pool
    a temporary, free again on return, could go to the current stream's next work while the kernels still use it."""
    at = list(inspect.signature(call).parameters).index("stream")

    @functools.wraps(call)
    def on(*args, **kwargs):
        stream = args[at] if len(args) > at else kwargs.get("stream")
        if stream is None:
            return call(*args, **kwargs)
        with torch.cuda.stream(stream):
            return call(*args, **kwargs)
    return on


_AS_IT_IS = contextlib.nullcontext()


def _current(dev: torch.device):
    """Makes a device the current one, where it is not: the library launches on the current device."""
    return _AS_IT_IS if dev.index == _current_device() else torch.cuda.device(dev)


def _result(stream, *shape, dtype, device) -> torch.Tensor:
    """A result of a call on ``stream`` (None: the current one), allocated for it."""
    if stream is None:
        return torch.empty(*shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(*shape, dtype=dtype, device=device)


# ---------------------------------------------------------------------------
# Single calls
# ---------------------------------------------------------------------------

@_for_its_stream
def bias_table(b: torch.Tensor, n_hot: int, cap: float, stream=None, mode: int = BIAS_GRADED) -> torch.Tensor:
    out = torch.empty_like(b)
    if mode == BIAS_GRADED:
        _ck(_bias_table(_p(b), b.numel(), n_hot, cap, _p(out), _s(stream)), "moe_bias_table")
    else:
        _ck(_bias_table_mode(_p(b), b.numel(), n_hot, mode, cap, _p(out), _s(stream)), "moe_bias_table_mode")
    return out


@_for_its_stream
def route(x, w_router, k, logit_offset=None, sel_bias=None, return_logits=False, stream=None, blocked=True,
          e2s=None, affinity=0.0, rflags=0):
    T, H = x.shape
    E = w_router.shape[1]
    ids = torch.empty(T, k, dtype=torch.int32, device=x.device)
    w = torch.empty(T, k, dtype=torch.float32, device=x.device)
    logits = torch.empty(T, E, dtype=torch.float32, device=x.device)
    nb = int(_route_scratch(T, H, E)) if blocked else 0
    scratch = torch.empty(max(nb // 4, 1), dtype=torch.float32, device=x.device) if nb else None
    if rflags:
        _ck(_route_ex(_p(x), _p(w_router), _p(logit_offset), _p(sel_bias), _p(e2s), affinity, rflags, T, H, E, k,
                      _p(logits), _p(scratch), _p(ids), _p(w), _s(stream)), "moe_route_ex")
    else:
        _ck(_route(_p(x), _p(w_router), _p(logit_offset), _p(sel_bias), _p(e2s), affinity, T, H, E, k,
                   _p(logits), _p(scratch), _p(ids), _p(w), _s(stream)), "moe_route")
    return (ids, w, logits) if return_logits else (ids, w)


@dataclass
class Groups:
    count: torch.Tensor
    offset: torch.Tensor
    rows: torch.Tensor
    pos: torch.Tensor
    act_e: torch.Tensor
    n_act: torch.Tensor


@_for_its_stream
def permute(ids: torch.Tensor, E: int, dev_status: Optional[torch.Tensor] = None, stream=None,
            chunked: bool = True) -> Groups:
    n = ids.numel()
    i32 = dict(dtype=torch.int32, device=ids.device)
    g = Groups(torch.empty(E, **i32), torch.empty(E + 1, **i32), torch.empty(n, **i32), torch.empty(n, **i32),
               torch.empty(E, **i32), torch.empty(1, **i32))
    nb = int(_permute_scratch(n, E)) if chunked else 0
    scratch = torch.empty(max(nb // 4, 1), **i32) if nb else None
    _ck(_permute(_p(ids), n, E, _p(g.count), _p(g.offset), _p(g.rows), _p(g.pos), _p(g.act_e), _p(g.n_act),
                 _p(scratch), _p(dev_status), _s(stream)), "moe_permute")
    return g


@dataclass
class CacheState:
    e2s: torch.Tensor    # int32 [E]
    s2e: torch.Tensor    # int32 [S]
    prio: torch.Tensor   # uint32 [S], held as int32
    stamp: torch.Tensor  # uint32 [1], held as int32

    @staticmethod
    def from_slots(s2e, E: int, device="cuda") -> "CacheState":
        s2e_t = torch.as_tensor(s2e, dtype=torch.int32).clone().cpu()
        e2s = torch.full((E,), -1, dtype=torch.int32)
        for s, e in enumerate(s2e_t.tolist()):
            if e >= 0:
                e2s[e] = s
        S = s2e_t.numel()
        return CacheState(e2s.to(device), s2e_t.to(device), torch.zeros(S, dtype=torch.int32, device=device),
                          torch.zeros(1, dtype=torch.int32, device=device))

    def clone(self) -> "CacheState":
        return CacheState(self.e2s.clone(), self.s2e.clone(), self.prio.clone(), self.stamp.clone())


@dataclass
class ManageOut:
    miss_e: torch.Tensor
    miss_s: torch.Tensor
    n_miss: torch.Tensor
    hit_e: torch.Tensor
    n_hit: torch.Tensor
    sid: torch.Tensor


@_for_its_stream
def cache_manage(ids: torch.Tensor, state: CacheState, policy: int, dev_status=None, stream=None) -> ManageOut:
    n = ids.numel()
    E, S = state.e2s.numel(), state.s2e.numel()
    lmax = min(n, E)
    i32 = dict(dtype=torch.int32, device=ids.device)
    o = ManageOut(torch.empty(lmax, **i32), torch.empty(lmax, **i32), torch.empty(1, **i32),
                  torch.empty(lmax, **i32), torch.empty(1, **i32), torch.empty(ids.shape, **i32))
    _ck(_manage(_p(ids), n, E, S, policy, _p(state.e2s), _p(state.s2e), _p(state.prio), _p(state.stamp),
                _p(o.miss_e), _p(o.miss_s), _p(o.n_miss), _p(o.hit_e), _p(o.n_hit), _p(o.sid), _p(dev_status),
                _s(stream)), "moe_cache_manage")
    return o


def cache_gather(host_slabs, pool, miss_e, miss_s, n_miss, max_miss, dev_status=None, stream=None) -> None:
    E = host_slabs.shape[0]
    S = pool.shape[0]
    slab_bytes = pool[0].numel() * pool.element_size()
    _ck(_gather(_p(host_slabs), _p(pool), slab_bytes, E, S, _p(miss_e), _p(miss_s), _p(n_miss), max_miss,
                _p(dev_status), _s(stream)), "moe_cache_gather")


def cache_count(ids, E, counts, dev_status=None, stream=None) -> None:
    """counts[e] += number of routings of expert e in ``ids`` (window counts for a re-pick)."""
    _ck(_count(_p(ids), ids.numel(), E, _p(counts), _p(dev_status), _s(stream)), "moe_cache_count")


@dataclass
class RepickResult:
    miss_e: torch.Tensor
    miss_s: torch.Tensor
    n_miss: torch.Tensor


@_for_its_stream
def cache_repick(counts, state: "CacheState", stream=None) -> RepickResult:
    """Re-pick a STATIC pool's resident set from the window counts (clears them)."""
    E, S = state.e2s.numel(), state.s2e.numel()
    i32 = dict(dtype=torch.int32, device=counts.device)
    r = RepickResult(torch.empty(min(S, E), **i32), torch.empty(min(S, E), **i32), torch.zeros(1, **i32))
    _ck(_repick(_p(counts), E, S, _p(state.e2s), _p(state.s2e), _p(r.miss_e), _p(r.miss_s), _p(r.n_miss),
                _s(stream)), "moe_cache_repick")
    return r


def q8_slab_bytes(H: int, I: int) -> int:
    return int(_q8_slab(H, I))


@_for_its_stream
def quantize_slabs(slabs: torch.Tensor, H: int, I: int, stream=None) -> torch.Tensor:
    """bf16 slabs [n][3HI] (device) -> W8A8 slabs uint8 [n][q8_slab_bytes] (device)."""
    n = slabs.shape[0]
    out = torch.empty(n, q8_slab_bytes(H, I), dtype=torch.uint8, device=slabs.device)
    _ck(_quantize(_p(slabs), n, H, I, _p(out), _s(stream)), "moe_quantize_slabs")
    return out


@_for_its_stream
def expert_ffn_q8(x, k, I, E, offset, rows, list_e, n_list, max_list, pool_q, e2s=None, y=None, workspace=None,
                  dev_status=None, stream=None) -> torch.Tensor:
    T, H = x.shape
    if y is None:
        y = torch.zeros(T * k, H, dtype=torch.float32, device=x.device)
    if workspace is None:
        workspace = torch.empty(int(_ffn_q8_ws(T, H, k, I)), dtype=torch.uint8, device=x.device)
    _ck(_ffn_q8(_p(x), T, H, I, k, E, _p(offset), _p(rows), _p(list_e), _p(n_list), max_list, _p(pool_q),
                pool_q.shape[0], _p(e2s), _p(y), _p(workspace), workspace.numel(), _p(dev_status), _s(stream)),
        "moe_expert_ffn_q8")
    return y


# ---------------------------------------------------------------------------
# 4-bit weights with group scales
# ---------------------------------------------------------------------------

def w4_bytes(K: int, N: int, group: int) -> int:
    """Bytes of a packed K x N matrix (0: shape out of range)."""
    return int(_w4_bytes(K, N, group))


def w4_slab_bytes(H: int, I: int, group: int) -> int:
    return int(_w4_slab(H, I, group))


def _want(t: torch.Tensor, what: str, dtype, shape=None) -> None:
    if t.dtype != dtype or not t.is_contiguous() or (shape is not None and tuple(t.shape) != tuple(shape)):
        raise ValueError(f"{what}: need a contiguous {dtype} tensor" + (f" of shape {tuple(shape)}" if shape is not None else "")
                         + f", got {t.dtype} {tuple(t.shape)}")


def _want_status(t: torch.Tensor, dev: torch.device) -> None:
    if t.dtype != torch.int32 or t.numel() < 1:
        raise ValueError(f"dev_status: need int32 [1], got {t.dtype} {tuple(t.shape)}")
    if t.device != dev:
        raise ValueError(f"dev_status: on {t.device}, the call runs on {dev}")


@_for_its_stream
def w4_pack(codes: torch.Tensor, scales: torch.Tensor, group: int, stream=None) -> torch.Tensor:
    """codes uint8 [..., K, N] (0..15), scales bf16 [..., ceil(K / group), N] -> packed uint8 [..., w4_bytes]."""
    K, N = codes.shape[-2:]
    _want(codes, "codes", torch.uint8)
    _want(scales, "scales", torch.bfloat16, (*codes.shape[:-2], -(-K // group) if group > 0 else 0, N))
    _on(codes.device, scales=scales)
    with _current(codes.device):
        out = torch.empty(*codes.shape[:-2], w4_bytes(K, N, group), dtype=torch.uint8, device=codes.device)
        _ck(_w4_pack(_p(codes), _p(scales), codes[..., 0, 0].numel(), K, N, group, _p(out), _s(stream)), "moe_w4_pack")
    return out


@_for_its_stream
def w4_quantize(w: torch.Tensor, group: int, stream=None) -> torch.Tensor:
    """bf16 [..., K, N] -> packed uint8 [..., w4_bytes]."""
    K, N = w.shape[-2:]
    _want(w, "w", torch.bfloat16)
    _on(w.device)
    with _current(w.device):
        out = torch.empty(*w.shape[:-2], w4_bytes(K, N, group), dtype=torch.uint8, device=w.device)
        _ck(_w4_quantize(_p(w), w[..., 0, 0].numel(), K, N, group, _p(out), _s(stream)), "moe_w4_quantize")
    return out


@_for_its_stream
def w4_pack_slabs(codes: torch.Tensor, scales: torch.Tensor, H: int, I: int, group: int, stream=None) -> torch.Tensor:
    """Expert slabs: codes uint8 [n][3HI], scales bf16 [n][2 ceil(H/group) I + ceil(I/group) H] -> [n][w4_slab_bytes]."""
    n = codes.shape[0]
    _want(codes, "codes", torch.uint8, (n, 3 * H * I))
    if group > 0:
        _want(scales, "scales", torch.bfloat16, (n, 2 * -(-H // group) * I + -(-I // group) * H))
    _on(codes.device, scales=scales)
    with _current(codes.device):
        out = torch.empty(n, w4_slab_bytes(H, I, group), dtype=torch.uint8, device=codes.device)
        _ck(_w4_pack_slabs(_p(codes), _p(scales), n, H, I, group, _p(out), _s(stream)), "moe_w4_pack_slabs")
    return out


@_for_its_stream
def w4_quantize_slabs(slabs: torch.Tensor, H: int, I: int, group: int, stream=None) -> torch.Tensor:
    """bf16 slabs [n][3HI] (device) -> packed 4-bit slabs uint8 [n][w4_slab_bytes] (device)."""
    n = slabs.shape[0]
    _want(slabs, "slabs", torch.bfloat16, (n, 3 * H * I))
    _on(slabs.device)
    with _current(slabs.device):
        out = torch.empty(n, w4_slab_bytes(H, I, group), dtype=torch.uint8, device=slabs.device)
        _ck(_w4_quantize_slabs(_p(slabs), n, H, I, group, _p(out), _s(stream)), "moe_w4_quantize_slabs")
    return out


class W4Linear:
    """y = x W with a packed 4-bit matrix (w4_pack, w4_quantize) of K inputs and N outputs, for up to max_tokens rows.

    x may be a row-strided view (last dimension contiguous).  One call at a time: calls share the workspace.  Forward
    only: the result carries no gradient.

    ``forward(x, adapters=, adapter_ids=, seq_start=)`` adds the low-rank part of each request's adapter (``Adapters``)
    to the result, in place: a bf16 result is rounded once as the projection's and once more as the sum (a layer with
    ``out_dtype=torch.float32`` keeps the sum in fp32).
    """

    def __init__(self, packed: torch.Tensor, K: int, N: int, group: int, max_tokens: int = 1,
                 out_dtype=torch.bfloat16):
        if w4_bytes(K, N, group) == 0:
            raise MoeError(-1, "W4Linear")
        _want(packed, "packed", torch.uint8, (w4_bytes(K, N, group),))
        if out_dtype not in (torch.bfloat16, torch.float32):
            raise ValueError(f"out_dtype: bfloat16 or float32, got {out_dtype}")
        self.packed, self.K, self.N, self.group = packed, K, N, group
        self.max_tokens, self.out_dtype = max_tokens, out_dtype
        self.device, self._index = packed.device, packed.get_device()
        self.dev_status = torch.zeros(1, dtype=torch.int32, device=packed.device)
        self.workspace = torch.empty(int(_w4_linear_ws(max_tokens, K, N, group)), dtype=torch.uint8,
                                     device=packed.device)
        self._packed, self._status = packed.data_ptr(), self.dev_status.data_ptr()
        self._ws, self._ws_bytes, self._f32 = self.workspace.data_ptr(), self.workspace.numel(), out_dtype == torch.float32

    def forward(self, x: torch.Tensor, out: Optional[torch.Tensor] = None, stream=None,
                adapters: Optional["Adapters"] = None, adapter_ids: Optional[torch.Tensor] = None,
                seq_start: Optional[torch.Tensor] = None) -> torch.Tensor:
        if adapters is not None:
            if (adapters.K, adapters.N) != (self.K, self.N) or adapter_ids is None:
                raise ValueError(f"adapters: need {self.K} inputs, {self.N} outputs and adapter_ids")
            adapters.check(x, adapter_ids, seq_start, self.out_dtype, out)  # nothing is written where the second call refuses
            out = self.forward(x, out, stream)
            return adapters.forward(x, adapter_ids, out, seq_start, out, stream=stream)
        if adapter_ids is not None or seq_start is not None:
            raise ValueError("adapter_ids, seq_start: given without adapters")
        T, K = x.shape
        if T > self.max_tokens or K != self.K:
            raise ValueError(f"x is {T} x {K}; the layer takes up to {self.max_tokens} rows of {self.K}")
        if x.dtype != torch.bfloat16 or x.stride(1) != 1:
            raise ValueError("x: need bf16 rows with a contiguous last dimension")
        if out is not None and (out.dtype != self.out_dtype or out.shape != (T, self.N) or out.stride(1) != 1):
            raise ValueError(f"out: need {self.out_dtype} ({T}, {self.N}) with a contiguous last dimension")
        dev = self._index
        if dev < 0 or x.get_device() != dev or (out is not None and out.get_device() != dev):
            _on(self.device, x=x, out=out)
        if _current_device() != dev:
            with torch.cuda.device(self.device):
                return self.forward(x, out, stream)
        if out is None:
            out = _result(stream, T, self.N, dtype=self.out_dtype, device=self.device)
        _ck(_w4_linear(x.data_ptr(), x.stride(0) if T > 1 else K, T, K, self.N, self.group, self._packed,
                       out.data_ptr(), out.stride(0) if T > 1 else self.N, self._f32, self._ws, self._ws_bytes,
                       self._status, _here(dev, stream)), "moe_w4_linear")
        return out


# ---------------------------------------------------------------------------
# Low-rank adapters beside a projection
# ---------------------------------------------------------------------------

def _rows_apart(x: torch.Tensor, y: torch.Tensor) -> bool:
    """Whether two matrices of as many rows have no byte in common: apart, or side by side in rows of one stride."""
    (p, ld, n), (q, le, m) = ((t.data_ptr(), t.stride(0) * t.element_size(), t.shape[1] * t.element_size()) for t in (x, y))
    T = x.shape[0]
    if p + (T - 1) * ld + n <= q or q + (T - 1) * le + m <= p:
        return True
    return T > 1 and ld == le and (q - p) % ld >= n and (q - p) % ld + m <= ld


class AdapterGrads(NamedTuple):
    dx: Optional[torch.Tensor]  # bf16 [T][K]
    da: Optional[torch.Tensor]  # fp32 [L][R][K]
    db: Optional[torch.Tensor]  # fp32 [L][R][N]


class Adapters:
    """L low-rank adapters of rank R for a projection of K inputs and N outputs: out = base + scale_l (x A_l^T) B_l.

    ``a`` bf16 [L][R][K], ``b`` bf16 [L][R][N] and ``scale`` fp32 [L] are read where they are: what is written into them
    counts from the next call on.  Sequence q of a batch is the rows [seq_start[q], seq_start[q + 1]) with the adapter
    ids[q] (int32, -1: none); without ``seq_start`` every row is a sequence of its own.  Rows may be row-strided views
    on 16 bytes.  ``AdapterAdd`` is the form for autograd; forward and grad carry no gradient themselves.  Errors found on
    the device are recorded in ``dev_status`` (int32 [1]; the caller's, or one of its own).
    """

    def __init__(self, a: torch.Tensor, b: torch.Tensor, scale: torch.Tensor, dev_status: Optional[torch.Tensor] = None, *,
                 _record: bool = True):
        if a.dim() != 3 or b.dim() != 3 or a.shape[:2] != b.shape[:2]:
            raise ValueError(f"a, b: need [L][R][K] and [L][R][N], got {tuple(a.shape)} and {tuple(b.shape)}")
        _want(a, "a", torch.bfloat16)
        _want(b, "b", torch.bfloat16)
        _want(scale, "scale", torch.float32, (a.shape[0],))
        self.a, self.b, self.scale = a, b, scale
        (self.L, self.R, self.K), self.N = a.shape, b.shape[2]
        if not (1 <= self.L <= 65535 and 1 <= self.R <= 128) or any(n % 8 or not 8 <= n <= 1 << 17 for n in (self.K, self.N)):
            raise ValueError(f"a, b: 1..65535 adapters of rank 1..128, 8..131072 features in eights, got "
                             f"{tuple(a.shape)} and {tuple(b.shape)}")
        self.device, self._index = a.device, a.get_device()
        if b.device != a.device or scale.device != a.device:
            raise ValueError(f"a, b, scale: on {a.device}, {b.device} and {scale.device}")
        if dev_status is not None:
            _want_status(dev_status, a.device)
        elif _record:
            dev_status = torch.zeros(1, dtype=torch.int32, device=a.device)
        self.dev_status = dev_status
        self._a, self._b, self._scale = a.data_ptr(), b.data_ptr(), scale.data_ptr()
        self._status = None if dev_status is None else dev_status.data_ptr()

    def _sequences(self, T, ids, seq_start):
        n = T if seq_start is None else seq_start.numel() - 1
        if ids.dtype is not torch.int32 or ids.shape != (n,) or not ids.is_contiguous():
            raise ValueError(f"ids: need contiguous int32 [{n}], got {ids.dtype} {tuple(ids.shape)}")
        if seq_start is not None:
            _want(seq_start, "seq_start", torch.int32, (n + 1,))
        return n

    @staticmethod
    def _rows(t, what, T, n, dtype):
        if t.dtype is not dtype or t.shape != (T, n) or t.stride(1) != 1:
            raise ValueError(f"{what}: need {dtype} ({T}, {n}) with a contiguous last dimension, got {t.dtype} "
                             f"{tuple(t.shape)}")
        return t.data_ptr(), t.stride(0) if T > 1 else n

    def check(self, x, ids, seq_start, dtype, out) -> None:
        """Refuses what forward would refuse."""
        T = x.shape[0]
        if self._sequences(T, ids, seq_start) < 1:
            raise MoeError(-1, "Adapters (no sequence)")
        for what, t, n, kind in (("x", x, self.K, torch.bfloat16), ("out", out, self.N, dtype)):
            if t is not None:
                at, ld = self._rows(t, what, T, n, kind)
                if ld < n:
                    raise MoeError(-1, f"Adapters ({what})")
                if at % 16 or ld * t.element_size() % 16:
                    raise MoeError(-3, f"Adapters ({what})")
        if out is not None and not _rows_apart(x, out):
            raise MoeError(-1, "Adapters (out over x)")
        _on(self.device, x=x, ids=ids, seq_start=seq_start, out=out)

    def forward(self, x: torch.Tensor, ids: torch.Tensor, base: Optional[torch.Tensor] = None,
                seq_start: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                out_dtype=torch.bfloat16, kept: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """base + the adapters' part, in a new tensor or in ``out`` (base itself, if need be), of the type of base or
        out (neither: ``out_dtype``).  ``kept`` (fp32 [T][R]) receives scale_l x A_l^T for the gradient."""
        T = x.shape[0]
        px, ldx = self._rows(x, "x", T, self.K, torch.bfloat16)
        n = self._sequences(T, ids, seq_start)
        dtype = base.dtype if base is not None else out.dtype if out is not None else out_dtype
        f32 = dtype == torch.float32
        if not f32 and dtype != torch.bfloat16:
            raise ValueError(f"base, out: bfloat16 or float32, got {dtype}")
        pb, ldb = (None, 0) if base is None else self._rows(base, "base", T, self.N, dtype)
        if kept is not None:
            _want(kept, "kept", torch.float32, (T, self.R))
        dev = self._index
        if (dev < 0 or x.get_device() != dev or ids.get_device() != dev or _elsewhere(base, dev)
                or _elsewhere(seq_start, dev) or _elsewhere(out, dev) or _elsewhere(kept, dev)):
            _on(self.device, x=x, ids=ids, base=base, seq_start=seq_start, out=out, kept=kept)
        if _current_device() != dev:
            with torch.cuda.device(self.device):
                return self.forward(x, ids, base, seq_start, out, out_dtype, kept, stream)
        if out is None:
            out = _result(stream, T, self.N, dtype=dtype, device=self.device)
            po, ldo = out.data_ptr(), self.N
        else:
            po, ldo = (pb, ldb) if out is base else self._rows(out, "out", T, self.N, dtype)
        rc = _adapters(px, ldx, pb, ldb, T, self.K, self.N, self.R, self.L, self._a, self._b, self._scale, ids.data_ptr(),
                       None if seq_start is None else seq_start.data_ptr(), n, po, ldo, f32,
                       None if kept is None else kept.data_ptr(), self._status, _here(dev, stream))
        if rc:
            _ck(rc, "moe_adapters")
        return out

    def grad(self, dy: torch.Tensor, x: Optional[torch.Tensor], kept: Optional[torch.Tensor], ids: torch.Tensor,
             base: Optional[torch.Tensor] = None, seq_start: Optional[torch.Tensor] = None, with_dx: bool = True,
             with_weights: bool = True, stream=None) -> AdapterGrads:
        """The gradients in x (plus ``base``), a and b, from that in out; ``kept`` as the forward pass left it."""
        if stream is not None:
            with torch.cuda.stream(stream):
                return self.grad(dy, x, kept, ids, base, seq_start, with_dx, with_weights)
        T = dy.shape[0]
        pdy, ldy = self._rows(dy, "dy", T, self.N, torch.bfloat16)
        n = self._sequences(T, ids, seq_start)
        px = ldx = pk = None
        if with_weights:
            if x is None or kept is None:
                raise ValueError("x, kept: needed for the gradients in a and b")
            px, ldx = self._rows(x, "x", T, self.K, torch.bfloat16)
            _want(kept, "kept", torch.float32, (T, self.R))
            pk = kept.data_ptr()
        pb, ldb = (None, 0) if base is None else self._rows(base, "base", T, self.K, torch.bfloat16)
        dev = self._index
        if (dev < 0 or dy.get_device() != dev or ids.get_device() != dev or _elsewhere(x, dev) or _elsewhere(kept, dev)
                or _elsewhere(base, dev) or _elsewhere(seq_start, dev)):
            _on(self.device, dy=dy, x=x, kept=kept, ids=ids, base=base, seq_start=seq_start)
        if _current_device() != dev:
            with torch.cuda.device(self.device):
                return self.grad(dy, x, kept, ids, base, seq_start, with_dx, with_weights)
        dx = torch.empty((T, self.K), dtype=torch.bfloat16, device=self.device) if with_dx else None
        da = torch.empty(self.a.shape, dtype=torch.float32, device=self.device) if with_weights else None
        db = torch.empty(self.b.shape, dtype=torch.float32, device=self.device) if with_weights else None
        nws = _adapters_grad_ws(T, self.R)
        ws = torch.empty(nws, dtype=torch.uint8, device=self.device)
        _ck(_adapters_grad(pdy, ldy, px, ldx or 0, pk, pb, ldb, T, self.K, self.N, self.R, self.L, self._a, self._b,
                           self._scale, ids.data_ptr(), None if seq_start is None else seq_start.data_ptr(), n,
                           None if dx is None else dx.data_ptr(), self.K, None if da is None else da.data_ptr(),
                           None if db is None else db.data_ptr(), ws.data_ptr(), nws, self._status, _here(dev)),
            "moe_adapters_grad")
        return AdapterGrads(dx, da, db)


class AdapterAdd(torch.autograd.Function):
    """Adapters for autograd: ``out = AdapterAdd.apply(x, a, b, scale, ids, base, seq_start, dev_status)``, bf16.

    Gradients in x, a, b and base (none in scale).  Errors found on the device in either pass are recorded in
    ``dev_status`` (int32 [1]), where it is given.  There is no second derivative: differentiating the gradient again
    raises.
    """

    @staticmethod
    def forward(ctx, x, a, b, scale, ids, base=None, seq_start=None, dev_status=None):
        if base is not None and base.dtype != torch.bfloat16:
            raise ValueError(f"base: bfloat16 where a gradient is wanted, got {base.dtype}")
        need = any(ctx.needs_input_grad[1:3])
        op = Adapters(a, b, scale, dev_status, _record=False)
        kept = torch.empty((x.shape[0], op.R), dtype=torch.float32, device=x.device) if need else None
        out = op.forward(x, ids, base, seq_start, kept=kept)
        ctx.save_for_backward(x if need else None, a, b, scale, ids, seq_start, kept)
        ctx.dev_status = dev_status
        return out

    @staticmethod
    def backward(ctx, dy):
        x, a, b, scale, ids, seq_start, kept = ctx.saved_tensors
        op = Adapters(a.detach(), b.detach(), scale.detach(), ctx.dev_status, _record=False)
        need_x, need_a, need_b = ctx.needs_input_grad[:3]
        rows = dy.detach()
        if rows.stride(1) != 1 or rows.stride(0) % 8 or rows.stride(0) < op.N or rows.data_ptr() % 16:
            rows = rows.clone(memory_format=torch.contiguous_format)  # (contiguous() leaves a contiguous one on its address)
        dx = da = db = None
        if need_x or need_a or need_b:
            g = op.grad(rows, x, kept, ids, None, seq_start, need_x, need_a or need_b)
            dx = g.dx
            da = g.da.to(a.dtype) if need_a else None
            db = g.db.to(b.dtype) if need_b else None
            if torch.is_grad_enabled():
                dx, da, db = _FirstGrad.apply("AdapterAdd", 3, dx, da, db, dy, x, a, b)
        return dx, da, db, None, None, dy if ctx.needs_input_grad[5] else None, None, None


@_for_its_stream
def expert_ffn_w4(x, k, I, E, group, offset, rows, list_e, n_list, max_list, pool, e2s=None, y=None, workspace=None,
                  dev_status=None, stream=None) -> torch.Tensor:
    T, H = x.shape
    _on(x.device, offset=offset, rows=rows, list_e=list_e, n_list=n_list, pool=pool, e2s=e2s, y=y, workspace=workspace,
        dev_status=dev_status)
    with _current(x.device):
        if y is None:
            y = torch.zeros(T * k, H, dtype=torch.float32, device=x.device)
        if workspace is None:
            workspace = torch.empty(int(_ffn_w4_ws(T, H, k, I)), dtype=torch.uint8, device=x.device)
        _ck(_ffn_w4(_p(x), T, H, I, k, E, group, _p(offset), _p(rows), _p(list_e), _p(n_list), max_list, _p(pool),
                    pool.shape[0], _p(e2s), _p(y), _p(workspace), workspace.numel(), _p(dev_status), _s(stream)),
            "moe_expert_ffn_w4")
    return y


class W4Experts:
    """The routed experts of one layer over a pool of packed 4-bit slabs ([S][w4_slab_bytes] uint8, device).

    forward(x, ids, w) -> bf16 [T][H]: sum_j w[t][j] * FFN_{ids[t][j]}(x[t]).  One call at a time: calls share the
    workspace.  Forward only: the result carries no gradient.
    """

    def __init__(self, pool: torch.Tensor, H: int, I: int, k: int, E: int, group: int,
                 e2s: Optional[torch.Tensor] = None, max_tokens: int = 64):
        if w4_slab_bytes(H, I, group) == 0 or int(_experts_w4_ws(max_tokens, H, I, k, E)) == 0:
            raise MoeError(-1, "W4Experts")
        _want(pool, "pool", torch.uint8, (pool.shape[0], w4_slab_bytes(H, I, group)))
        if e2s is not None:
            _want(e2s, "e2s", torch.int32, (E,))
        self.pool, self.H, self.I, self.k, self.E, self.group, self.e2s = pool, H, I, k, E, group, e2s
        self.S, self.max_tokens = pool.shape[0], max_tokens
        self.device, self._index = pool.device, pool.get_device()
        if e2s is not None and e2s.device != pool.device:
            raise ValueError(f"e2s: on {e2s.device}, the pool is on {pool.device}")
        self.dev_status = torch.zeros(1, dtype=torch.int32, device=pool.device)
        self.workspace = torch.empty(int(_experts_w4_ws(max_tokens, H, I, k, E)), dtype=torch.uint8,
                                     device=pool.device)
        self._pool, self._e2s = pool.data_ptr(), None if e2s is None else e2s.data_ptr()
        self._status, self._ws, self._ws_bytes = self.dev_status.data_ptr(), self.workspace.data_ptr(), self.workspace.numel()

    def forward(self, x: torch.Tensor, ids: torch.Tensor, w: torch.Tensor, out: Optional[torch.Tensor] = None,
                stream=None) -> torch.Tensor:
        T = x.shape[0]
        if T > self.max_tokens:
            raise ValueError(f"T={T} > max_tokens={self.max_tokens}")
        if x.dtype != torch.bfloat16 or x.shape != (T, self.H) or not x.is_contiguous():
            raise ValueError(f"x: need contiguous bf16 [{T}][{self.H}]")
        if ids.dtype != torch.int32 or ids.shape != (T, self.k) or not ids.is_contiguous():
            raise ValueError(f"ids: need contiguous int32 [{T}][{self.k}]")
        if w.dtype != torch.float32 or w.shape != (T, self.k) or not w.is_contiguous():
            raise ValueError(f"w: need contiguous fp32 [{T}][{self.k}]")
        if out is not None:
            _want(out, "out", torch.bfloat16, (T, self.H))
        dev = self._index
        if (dev < 0 or x.get_device() != dev or ids.get_device() != dev or w.get_device() != dev
                or (out is not None and out.get_device() != dev)):
            _on(self.device, x=x, ids=ids, w=w, out=out)
        if _current_device() != dev:
            with torch.cuda.device(self.device):
                return self.forward(x, ids, w, out, stream)
        if out is None:
            out = _result(stream, T, self.H, dtype=torch.bfloat16, device=self.device)
        _ck(_experts_w4(x.data_ptr(), ids.data_ptr(), w.data_ptr(), T, self.H, self.I, self.k, self.E, self.group,
                        self._pool, self.S, self._e2s, out.data_ptr(), self._ws, self._ws_bytes, self._status,
                        _here(dev, stream)), "moe_experts_w4")
        return out


# ---------------------------------------------------------------------------
# The router's balance loss
# ---------------------------------------------------------------------------

class Balance(NamedTuple):
    loss: Optional[torch.Tensor]   # fp32 scalar
    counts: torch.Tensor           # int32 [n_seq][E]
    grad: Optional[torch.Tensor]   # [T][E], the type of the logits


def balance_loss(logits: torch.Tensor, ids: torch.Tensor, coef: float, seq_start: Optional[torch.Tensor] = None,
                 token_mask: Optional[torch.Tensor] = None, sigmoid: bool = False, with_loss: bool = True,
                 with_grad: bool = False, grad_loss: Optional[torch.Tensor] = None, dev_status=None,
                 stream=None) -> Balance:
    """Loss, per-sequence expert counts and (with_grad) the gradient in the logits times ``grad_loss`` (1 if None)."""
    T, E = logits.shape
    bf16 = logits.dtype == torch.bfloat16
    if not (bf16 or logits.dtype == torch.float32) or not logits.is_contiguous():
        raise ValueError(f"logits: need contiguous fp32 or bf16, got {logits.dtype}")
    k = ids.shape[-1]
    if ids.dtype != torch.int32 or ids.shape != (T, k) or not ids.is_contiguous():
        raise ValueError(f"ids: need contiguous int32 [{T}][k], got {ids.dtype} {tuple(ids.shape)}")
    if token_mask is not None:
        _want(token_mask, "token_mask", torch.bool if token_mask.dtype == torch.bool else torch.uint8, (T,))
    n_seq = 1
    if seq_start is not None:
        _want(seq_start, "seq_start", torch.int32)
        n_seq = seq_start.numel() - 1
    if grad_loss is not None and (grad_loss.dtype != torch.float32 or grad_loss.numel() != 1):
        raise ValueError("grad_loss: need one fp32 value")
    dev, index = logits.device, logits.get_device()
    if index < 0 or any(t is not None and t.get_device() != index for t in (ids, seq_start, token_mask, grad_loss, dev_status)):
        _on(dev, ids=ids, seq_start=seq_start, token_mask=token_mask, grad_loss=grad_loss, dev_status=dev_status)
    if stream is not None or _current_device() != index:  # temporaries and results for the stream that the kernels run on
        with torch.cuda.device(dev) if stream is None else torch.cuda.stream(stream):
            return balance_loss(logits, ids, coef, seq_start, token_mask, sigmoid, with_loss, with_grad, grad_loss, dev_status)
    loss = torch.empty((), dtype=torch.float32, device=dev) if with_loss else None
    counts = torch.empty((max(n_seq, 0), E), dtype=torch.int32, device=dev)
    grad = torch.empty_like(logits) if with_grad else None
    nws = _balance_ws(T, E, n_seq)
    ws = torch.empty(nws, dtype=torch.uint8, device=dev)
    _ck(_balance(logits.data_ptr(), bf16, ids.data_ptr(), None if token_mask is None else token_mask.data_ptr(),
                 None if seq_start is None else seq_start.data_ptr(), n_seq, T, E, k, ROUTE_SIGMOID if sigmoid else 0,
                 coef, None if grad_loss is None else grad_loss.data_ptr(), counts.data_ptr(),
                 loss.data_ptr() if with_loss else None, grad.data_ptr() if with_grad else None, ws.data_ptr(), nws,
                 None if dev_status is None else dev_status.data_ptr(), _here(index)), "moe_balance_loss")
    return Balance(loss, counts, grad)


class _BalanceGrad(torch.autograd.Function):
    """The gradient as a function of what it came from: to differentiate it again is an error, it is not a constant."""

    @staticmethod
    def forward(ctx, grad, logits, grad_loss):
        return grad.view_as(grad)

    @staticmethod
    def backward(ctx, _):
        raise RuntimeError("BalanceLoss has no second derivative")


class BalanceLoss(torch.autograd.Function):
    """balance_loss for autograd: ``loss, counts = BalanceLoss.apply(logits, ids, coef, seq_start, token_mask, sigmoid)``.

    It has no second derivative: differentiating the gradient again raises.
    """

    @staticmethod
    def forward(ctx, logits, ids, coef, seq_start=None, token_mask=None, sigmoid=False):
        r = balance_loss(logits, ids, coef, seq_start, token_mask, sigmoid)
        ctx.save_for_backward(logits, ids, seq_start, token_mask)
        ctx.coef, ctx.sigmoid = coef, sigmoid
        ctx.mark_non_differentiable(r.counts)
        return r.loss, r.counts

    @staticmethod
    def backward(ctx, grad_loss, _):
        logits, ids, seq_start, token_mask = ctx.saved_tensors
        r = balance_loss(logits, ids, ctx.coef, seq_start, token_mask, ctx.sigmoid, with_loss=False, with_grad=True,
                         grad_loss=grad_loss.detach().float().contiguous())
        grad = _BalanceGrad.apply(r.grad, logits, grad_loss) if torch.is_grad_enabled() else r.grad
        return grad, None, None, None, None, None


# ---------------------------------------------------------------------------
# Group-limited routing
# ---------------------------------------------------------------------------

class GroupRoute(NamedTuple):
    ids: torch.Tensor  # int32 [T][k]
    w: torch.Tensor    # fp32 [T][k]


def _logits_ok(logits: torch.Tensor) -> bool:
    """Whether the logits are bf16; refuses what is neither bf16 nor fp32."""
    bf16 = logits.dtype is torch.bfloat16
    if not (bf16 or logits.dtype is torch.float32) or logits.dim() != 2 or not logits.is_contiguous():
        raise ValueError(f"logits: need contiguous fp32 or bf16 [T][E], got {logits.dtype} {tuple(logits.shape)}")
    return bf16


def _elsewhere(t: Optional[torch.Tensor], index: int) -> bool:
    return t is not None and t.get_device() != index


def route_groups(logits: torch.Tensor, k: int, n_group: int = 1, topk_group: int = 1,
                 sel_bias: Optional[torch.Tensor] = None, token_mask: Optional[torch.Tensor] = None,
                 sigmoid: bool = False, group_max: bool = False, renormalise: bool = True, scale: float = 1.0,
                 stream=None) -> GroupRoute:
    """Picks and weights of each token from its ``topk_group`` best of ``n_group`` groups of experts.

    Forward only; ``RouteGroups`` carries the gradient of the weights.
    """
    bf16 = _logits_ok(logits)
    T, E = logits.shape
    bias = mask = None
    if sel_bias is not None:
        if sel_bias.dtype is not torch.float32 or sel_bias.shape != (E,) or not sel_bias.is_contiguous():
            _want(sel_bias, "sel_bias", torch.float32, (E,))
        bias = sel_bias.data_ptr()
    if token_mask is not None:
        _want(token_mask, "token_mask", torch.bool if token_mask.dtype is torch.bool else torch.uint8, (T,))
        mask = token_mask.data_ptr()
    dev, index = logits.device, logits.get_device()
    if index < 0 or _elsewhere(sel_bias, index) or _elsewhere(token_mask, index):
        _on(dev, sel_bias=sel_bias, token_mask=token_mask)
    if stream is not None or _current_device() != index:  # results for the stream that the kernel runs on
        with torch.cuda.device(dev) if stream is None else torch.cuda.stream(stream):
            return route_groups(logits, k, n_group, topk_group, sel_bias, token_mask, sigmoid, group_max, renormalise,
                                scale)
    if k < 1:
        raise MoeError(-1, "moe_route_groups")
    ids = torch.empty((T, k), dtype=torch.int32, device=dev)
    w = torch.empty((T, k), dtype=torch.float32, device=dev)
    flags = (ROUTE_SIGMOID if sigmoid else 0) | (ROUTE_GROUP_MAX if group_max else 0) | (0 if renormalise else ROUTE_RAW)
    rc = _route_groups(logits.data_ptr(), bf16, bias, mask, T, E, k, n_group, topk_group, flags, scale, ids.data_ptr(),
                       w.data_ptr(), _here(index))
    if rc:
        _ck(rc, "moe_route_groups")
    return GroupRoute(ids, w)


def route_groups_grad(logits: torch.Tensor, ids: torch.Tensor, grad_w: torch.Tensor, sigmoid: bool = False,
                      renormalise: bool = True, scale: float = 1.0, dev_status=None, stream=None) -> torch.Tensor:
    """The gradient in the logits of the weights of ``route_groups``, for the picks ``ids``."""
    bf16 = _logits_ok(logits)
    T, E = logits.shape
    k = ids.shape[-1]
    if ids.dtype != torch.int32 or ids.shape != (T, k) or not ids.is_contiguous():
        raise ValueError(f"ids: need contiguous int32 [{T}][k], got {ids.dtype} {tuple(ids.shape)}")
    _want(grad_w, "grad_w", torch.float32, (T, k))
    if dev_status is not None:
        _want_status(dev_status, logits.device)
    dev, index = logits.device, logits.get_device()
    if index < 0 or ids.get_device() != index or grad_w.get_device() != index:
        _on(dev, ids=ids, grad_w=grad_w)
    if stream is not None or _current_device() != index:
        with torch.cuda.device(dev) if stream is None else torch.cuda.stream(stream):
            return route_groups_grad(logits, ids, grad_w, sigmoid, renormalise, scale, dev_status)
    grad = torch.empty_like(logits)
    flags = (ROUTE_SIGMOID if sigmoid else 0) | (0 if renormalise else ROUTE_RAW)
    _ck(_route_groups_grad(logits.data_ptr(), bf16, ids.data_ptr(), grad_w.data_ptr(), T, E, k, flags, scale,
                           grad.data_ptr(), None if dev_status is None else dev_status.data_ptr(), _here(index)),
        "moe_route_groups_grad")
    return grad


class _FirstGrad(torch.autograd.Function):
    """Gradients as a function of what they came from: to differentiate them again is an error, they are no constants."""

    @staticmethod
    def forward(ctx, name, n, *args):
        ctx.name = name
        return tuple(None if g is None else g.view_as(g) for g in args[:n])

    @staticmethod
    def backward(ctx, *_):
        raise RuntimeError(f"{ctx.name} has no second derivative")


class RouteGroups(torch.autograd.Function):
    """route_groups for autograd: ``ids, w = RouteGroups.apply(logits, k, n_group, topk_group, sel_bias, token_mask,
    sigmoid, group_max, renormalise, scale, dev_status)``.

    The weights have a gradient in the logits, the picks none (nor has the bias).  Errors that the backward pass finds on
    the device are recorded in ``dev_status`` (int32 [1]), where it is given.  There is no second derivative:
    differentiating the gradient again raises.
    """

    @staticmethod
    def forward(ctx, logits, k, n_group=1, topk_group=1, sel_bias=None, token_mask=None, sigmoid=False, group_max=False,
                renormalise=True, scale=1.0, dev_status=None):
        if dev_status is not None:
            _want_status(dev_status, logits.device)
        r = route_groups(logits, k, n_group, topk_group, sel_bias, token_mask, sigmoid, group_max, renormalise, scale)
        ctx.save_for_backward(logits, r.ids)
        ctx.args = sigmoid, renormalise, scale, dev_status
        ctx.mark_non_differentiable(r.ids)
        return r.ids, r.w

    @staticmethod
    def backward(ctx, _, grad_w):
        logits, ids = ctx.saved_tensors
        grad = route_groups_grad(logits, ids, grad_w.detach().float().contiguous(), *ctx.args)
        if torch.is_grad_enabled():
            grad = _FirstGrad.apply("RouteGroups", 1, grad, logits, grad_w)[0]
        return (grad,) + (None,) * 10


def ffn_workspace_bytes(T: int, H: int, k: int, I: int) -> int:
    return int(_ffn_ws(T, H, k, I))


@_for_its_stream
def expert_ffn(x, k, I, E, offset, rows, list_e, n_list, max_list, pool, e2s=None, host_slabs=None,
               y=None, workspace=None, dev_status=None, stream=None) -> torch.Tensor:
    T, H = x.shape
    if y is None:
        y = torch.zeros(T * k, H, dtype=torch.float32, device=x.device)
    if workspace is None:
        workspace = torch.empty(ffn_workspace_bytes(T, H, k, I), dtype=torch.uint8, device=x.device)
    _ck(_ffn(_p(x), T, H, I, k, E, _p(offset), _p(rows), _p(list_e), _p(n_list), max_list, _p(pool),
             pool.shape[0], _p(e2s),
             _p(host_slabs), _p(y), _p(workspace), workspace.numel(), _p(dev_status), _s(stream)),
        "moe_expert_ffn")
    return y


@_for_its_stream
def combine(y, w, pos, T, k, E, ids=None, e2s=None, split=False, stream=None):
    H = y.shape[1]
    out = torch.empty(T, H, dtype=torch.bfloat16, device=y.device)
    out_res = torch.empty(T, H, dtype=torch.float32, device=y.device) if split else None
    out_miss = torch.empty(T, H, dtype=torch.float32, device=y.device) if split else None
    _ck(_combine(_p(y), _p(w), _p(pos), _p(ids), _p(e2s), T, k, H, E, int(split), _p(out), _p(out_res),
                 _p(out_miss), _s(stream)), "moe_combine")
    return (out, out_res, out_miss) if split else out


def layer_workspace_bytes(T, H, E, k, I, S) -> int:
    return int(_layer_ws(T, H, E, k, I, S))


# ---------------------------------------------------------------------------
# Whole layer
# ---------------------------------------------------------------------------

class SlotCachedMoELayer:
    """One layer's router, slot pool, host store, cache state and workspace.

    ``host_slabs`` (pinned host, [E][3HI] bf16) is the authoritative copy of
    every expert; ``pool`` ([S][3HI] bf16, device) holds the slot contents.
    In RESIDENT mode the pool holds every expert and no host store is needed.
    """

    def __init__(self, w_router, pool, k, I, mode, policy=POLICY_LRU, host_slabs=None, state=None,
                 logit_offset=None, sel_bias=None, max_tokens=64, side_stream=True, affinity=0.0,
                 route_flags=0, window_counts=None, quant=0, schedule=0, decode_kernels=0, quant_group=0):
        if w_router.dtype != torch.bfloat16:
            raise ValueError(f"w_router: need bfloat16 [H][E], got {w_router.dtype}")
        self.w_router, self.pool, self.k, self.I = w_router, pool, k, I
        self.H, self.E = w_router.shape
        self.S = pool.shape[0]
        self.mode, self.policy = mode, policy
        self.host_slabs, self.state = host_slabs, state
        self.logit_offset, self.sel_bias = logit_offset, sel_bias
        self.affinity = float(affinity)
        self.route_flags = int(route_flags)
        self.window_counts = window_counts
        self.quant = int(quant)  # pool / host hold W8A8 slabs (1: quantize_slabs) or 4-bit slabs (2: w4_pack_slabs)
        self.quant_group = int(quant_group)  # inputs per scale group of 4-bit slabs
        self.schedule = int(schedule)  # SCHED_CHUNKS or SCHED_WAVES (GATHER steps larger than the pool)
        self.decode_kernels = int(decode_kernels)  # 0: persistent decode kernel where it applies, 1: separate
        dev = pool.device
        self.stats = torch.zeros(4, dtype=torch.int64, device=dev)
        self.dev_status = torch.zeros(1, dtype=torch.int32, device=dev)
        self.max_tokens = max_tokens
        # zero-filled once: the persistent decode kernel's counters live at its start
        self.workspace = torch.zeros(layer_workspace_bytes(max_tokens, self.H, self.E, k, I, self.S),
                                     dtype=torch.uint8, device=dev)
        self.side = torch.cuda.Stream(device=dev) if side_stream else None

    @_for_its_stream
    def forward(self, x, out=None, ids=None, w=None, out_res=None, out_miss=None, stream=None, prof=None):
        T = x.shape[0]
        if T > self.max_tokens:
            raise ValueError(f"T={T} > max_tokens={self.max_tokens}")
        dev = x.device
        ids = torch.empty(T, self.k, dtype=torch.int32, device=dev) if ids is None else ids
        w = torch.empty(T, self.k, dtype=torch.float32, device=dev) if w is None else w
        out = torch.empty(T, self.H, dtype=torch.bfloat16, device=dev) if out is None else out
        if self.mode == MODE_ZERO_RETURN:
            out_res = torch.empty(T, self.H, dtype=torch.float32, device=dev) if out_res is None else out_res
            out_miss = torch.empty(T, self.H, dtype=torch.float32, device=dev) if out_miss is None else out_miss
        st = self.state
        a = LayerArgs(T, self.H, self.E, self.k, self.I, self.S, self.mode, self.policy,
                      x.data_ptr(), self.w_router.data_ptr(), _ptr(self.logit_offset), _ptr(self.sel_bias),
                      self.pool.data_ptr(), _ptr(self.host_slabs),
                      _ptr(st.e2s if st else None), _ptr(st.s2e if st else None),
                      _ptr(st.prio if st else None), _ptr(st.stamp if st else None),
                      ids.data_ptr(), w.data_ptr(), out.data_ptr(), _ptr(out_res), _ptr(out_miss),
                      self.stats.data_ptr(), self.dev_status.data_ptr(), self.workspace.data_ptr(),
                      self.workspace.numel(), ctypes.pointer(prof) if prof is not None else None, self.affinity,
                      self.route_flags, _ptr(self.window_counts), self.quant, self.schedule,
                      self.decode_kernels, self.quant_group)
        main = torch.cuda.current_stream() if stream is None else stream
        # the library forks to and joins back from the side stream itself
        _ck(_layer(ctypes.byref(a), c_void_p(main.cuda_stream),
                   c_void_p(self.side.cuda_stream) if self.side is not None else None), "moe_layer_forward")
        res = {"out": out, "ids": ids, "w": w}
        if self.mode == MODE_ZERO_RETURN:
            res["out_res"], res["out_miss"] = out_res, out_miss
        return res

    def repick(self, stream=None) -> RepickResult:
        """Re-pick the resident set from ``window_counts`` and copy the new members into their slots."""
        r = cache_repick(self.window_counts, self.state, stream)
        cache_gather(self.host_slabs, self.pool, r.miss_e, r.miss_s, r.n_miss, r.miss_e.numel(), self.dev_status,
                     stream)
        return r


class LayerStack:
    """Several layers' forwards replayed as one CUDA graph.

    "Betelgeuse ... on an RTX 3060", "What it actually does under the hood":
    with hits resolved on the device and no host sync inside a layer, a whole
    decode pass over all layers replays as a single CUDA graph.  Each layer
    reads its own input buffer ``xs[l]`` and writes ``outs[l]``; the caller
    refreshes the inputs between replays.  Cache state and slot pools evolve
    on the device across replays.
    """

    def __init__(self, layers, T: int):
        self.layers = layers
        dev = layers[0].pool.device
        H = layers[0].H
        # one contiguous [L][T][H] input block, so a step's inputs arrive in one copy
        self.x_all = torch.zeros(len(layers), T, H, dtype=torch.bfloat16, device=dev)
        self.xs = list(self.x_all.unbind(0))
        self.out_all = torch.empty(len(layers), T, H, dtype=torch.bfloat16, device=dev)
        self.outs = list(self.out_all.unbind(0))
        self.ids = [torch.empty(T, l.k, dtype=torch.int32, device=dev) for l in layers]
        self.ws = [torch.empty(T, l.k, dtype=torch.float32, device=dev) for l in layers]
        self.graph = None

    def _run(self, prof=None):
        for i, l in enumerate(self.layers):
            l.forward(self.xs[i], out=self.outs[i], ids=self.ids[i], w=self.ws[i],
                      prof=None if prof is None else prof[i])

    def capture(self, prof=None):
        """Capture one pass over all layers (run one eager pass first to set up)."""
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph, capture_error_mode="relaxed"):
            self._run(prof)
        return self.graph

    def replay(self):
        if self.graph is None:
            raise RuntimeError("capture() first")
        self.graph.replay()
