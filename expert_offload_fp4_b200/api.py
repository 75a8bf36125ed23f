"""Thin Python binding of libmoe_fp4.so: argument marshalling only.

Device buffers are torch tensors (their data_ptr is passed); streams are
torch.cuda.Stream objects (their cuda_stream handle is passed).  Every step of
the MoE layer runs in the library's kernels.
"""
from __future__ import annotations

import ctypes as C
import functools
from dataclasses import dataclass

import numpy as np
import torch

from . import _lib as L

FMT = {"mxfp4": L.MOE_MXFP4, "nvfp4": L.MOE_NVFP4}


def _p(t):
    return None if t is None else C.c_void_p(t.data_ptr())


def _s(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return C.c_void_p(stream.cuda_stream)


def _np(a, dt):
    a = np.ascontiguousarray(a, dtype=dt)
    return a, a.ctypes.data_as(C.c_void_p)


class Pool:
    """The library-owned expert store: pinned host blocks, HBM slots, LRU state."""

    def __init__(self, H, I, E, k, L_layers, fmt, n_slots, max_tokens=8, host_layers=0):
        self.lib = L.load()
        self.cfg = L.MoeConfig(H, I, E, k, L_layers, FMT[fmt], n_slots, max_tokens, host_layers)
        self.H, self.I, self.E, self.k, self.L = H, I, E, k, L_layers
        self.fmt, self.n_slots, self.max_tokens = fmt, n_slots, max_tokens
        self.n_active = n_slots
        self.host_layers = host_layers or L_layers
        h = C.c_void_p()
        L.check("moe_pool_create", self.lib.moe_pool_create(C.byref(self.cfg), C.byref(h)))
        self.handle = h
        self.block_bytes = self.lib.moe_expert_block_bytes(C.byref(self.cfg))

    def close(self):
        if getattr(self, "handle", None):
            self.lib.moe_pool_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def load_expert(self, layer, expert, tensors):
        """tensors: {"gate"|"up"|"down": (codes uint8, scales uint8, tensor_scale)}"""
        src = L.ExpertSrc()
        keep = []
        for i, name in enumerate(("gate", "up", "down")):
            c, s, ts = tensors[name]
            c, cp = _np(c, np.uint8)
            s, sp = _np(s, np.uint8)
            keep += [c, s]
            src.codes_h[i] = cp.value
            src.scales_h[i] = sp.value
            src.tensor_scale[i] = float(ts)
        L.check("moe_pool_load_expert",
                self.lib.moe_pool_load_expert(self.handle, int(layer), int(expert), C.byref(src)))

    def reset(self, n_active_slots=None):
        """Empty the pool and use only the first n_active_slots slots from now on."""
        n = self.n_slots if n_active_slots is None else int(n_active_slots)
        L.check("moe_pool_reset", self.lib.moe_pool_reset(self.handle, n))
        self.n_active = n

    def resize(self, n_active_slots):
        """Resize the slot pool at run time, keeping the LRU state (moe_pool_resize)."""
        L.check("moe_pool_resize", self.lib.moe_pool_resize(self.handle, int(n_active_slots)))
        self.n_active = int(n_active_slots)

    def set_copy_mode(self, mode):
        """"sm" (a kernel reads the mapped host block over PCIe) or "dma" (copy engine)."""
        m = {"sm": L.MOE_COPY_SM, "dma": L.MOE_COPY_DMA}[mode]
        L.check("moe_pool_set_copy_mode", self.lib.moe_pool_set_copy_mode(self.handle, m))

    def read_state(self):
        sk = np.empty(self.n_slots, np.int32)
        sc = np.empty(self.n_slots, np.uint64)
        ks = np.empty(self.L * self.E, np.int32)
        g = np.zeros(1, np.uint64)
        L.check("moe_pool_read_state", self.lib.moe_pool_read_state(
            self.handle, sk.ctypes.data_as(C.c_void_p), sc.ctypes.data_as(C.c_void_p),
            ks.ctypes.data_as(C.c_void_p), g.ctypes.data_as(C.c_void_p)))
        return dict(slot_key=sk, slot_clock=sc, key_slot=ks, clock=int(g[0]))

    def stats(self):
        st = L.Stats()
        L.check("moe_pool_stats", self.lib.moe_pool_stats(self.handle, C.byref(st)))
        return {f: getattr(st, f) for f, _ in L.Stats._fields_}

    def slot_ptr(self, slot):
        p, n = C.c_void_p(), C.c_size_t()
        L.check("moe_pool_slot_ptr", self.lib.moe_pool_slot_ptr(self.handle, int(slot), C.byref(p), C.byref(n)))
        return p.value, n.value


def route_workspace_bytes(T, E):
    return L.load().moe_route_workspace_bytes(int(T), int(E))


def route(x, wr, bias, k, renormalize, idx, w, workspace, stream=None):
    T, H = x.shape
    E = wr.shape[0]
    L.check("moe_route", L.load().moe_route(
        _p(x), _p(wr), _p(bias), T, H, E, int(k), int(renormalize), _p(idx), _p(w),
        _p(workspace), workspace.numel() * workspace.element_size(), _s(stream)))


def route_noalloc(x, wr, bias, k, renormalize, idx, w, stream=None):
    """moe_route_noalloc: the router with its scratch in a static device array of
    the library (for callers that cannot allocate device memory)."""
    T, H = x.shape
    E = wr.shape[0]
    L.check("moe_route_noalloc", L.load().moe_route_noalloc(
        _p(x), _p(wr), _p(bias), T, H, E, int(k), int(renormalize), _p(idx), _p(w), _s(stream)))


def _need(ok, what):
    if not ok:
        raise ValueError(what)


def _rows(t, dtypes, rows, cols, what):
    """Checks a 2-D tensor with contiguous rows; returns its row stride in elements."""
    if t.dtype not in dtypes or t.shape != (rows, cols):
        raise ValueError(f"{what} must be [{rows}, {cols}] of {' or '.join(map(str, dtypes))}")
    ld, inner = t.stride()
    if inner != 1 and cols != 1:
        raise ValueError(f"{what} must have contiguous rows")
    return ld if rows > 1 else cols


_functions = {}


def _call(name, tensors, stream, *args):
    """Library call on the device that holds all of `tensors`, on `stream` or that
    device's current stream."""
    dev = tensors[0].get_device()
    for t in tensors:
        if t is not None and t.get_device() != dev or dev < 0:
            raise ValueError(f"{name}: all tensors must be on one CUDA device")
    if stream is None:
        handle = torch._C._cuda_getCurrentRawStream(dev)
    elif stream.device.index != dev:
        raise ValueError(f"{name}: the stream belongs to another device than the tensors")
    else:
        handle = stream.cuda_stream
    fn = _functions.get(name)
    if fn is None:
        fn = _functions[name] = getattr(L.load(), name)
    if torch._C._cuda_getDevice() == dev:
        rc = fn(*args, handle)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, handle)
    if rc:
        L.check(name, rc)


@dataclass(frozen=True)
class GroupedRouting:
    """How a layer chooses its experts (the options of route_grouped)."""
    score: str = "sigmoid"
    n_group: int = 1
    topk_group: int = 1
    group_top: int = 1
    renormalize: bool = True
    scale: float = 1.0


_SCORE = {"softmax": L.MOE_SCORE_SOFTMAX, "sigmoid": L.MOE_SCORE_SIGMOID}
_TYPE = {torch.bfloat16: L.MOE_BF16, torch.float32: L.MOE_F32}


@functools.lru_cache(maxsize=64)
def _choice(k, score, n_group, topk_group, group_top, renormalize, scale):
    _need(score in _SCORE, f"score must be one of {sorted(_SCORE)}")
    return L.RouteChoice(k, _SCORE[score], n_group, topk_group, group_top, int(renormalize), scale)


def _choice_outputs(T, E, idx, w, bias):
    k = idx.shape[-1]
    _need(idx.dtype == torch.int32 and idx.shape == (T, k) and idx.is_contiguous(),
          "idx must be a contiguous int32 [T, k]")
    _need(w.dtype == torch.float32 and w.shape == (T, k) and w.is_contiguous(),
          "w must be a contiguous float32 [T, k]")
    _need(bias is None or (bias.dtype == torch.float32 and bias.shape == (E,) and bias.is_contiguous()),
          "bias must be a contiguous float32 [E]")
    return k


def route_grouped_workspace_bytes(T, E):
    return L.load().moe_route_grouped_workspace_bytes(int(T), int(E))


def route_grouped(x, wr, idx, w, workspace, *, score="sigmoid", bias=None, n_group=1, topk_group=1, group_top=1,
                  renormalize=True, scale=1.0, stream=None):
    """moe_route_grouped: x [T, H] and wr [E, H] bf16 -> idx [T, k] int32 and w [T, k]
    fp32.  Experts are chosen by sigmoid or softmax score + bias [E] fp32 (which does
    not enter the weights; -inf masks an expert) within the topk_group best of n_group
    groups, a group counting its group_top (1 or 2) best; w = scale * score, over the
    chosen scores' sum if renormalize.  workspace: route_grouped_workspace_bytes(T, E)
    bytes (enough for fewer tokens, too), zeroed before its first use."""
    _need(x.dim() == 2 and wr.dim() == 2 and x.dtype == wr.dtype == torch.bfloat16 and x.shape[1] == wr.shape[1]
          and x.is_contiguous() and wr.is_contiguous(), "x [T, H] and wr [E, H] must be contiguous bfloat16")
    T, H = x.shape
    E = wr.shape[0]
    k = _choice_outputs(T, E, idx, w, bias)
    _need(workspace.is_contiguous(), "the workspace must be contiguous")
    _call("moe_route_grouped", (x, wr, idx, w, workspace, bias), stream, x.data_ptr(), wr.data_ptr(),
          None if bias is None else bias.data_ptr(), T, H, E,
          C.byref(_choice(k, score, n_group, topk_group, group_top, bool(renormalize), float(scale))), idx.data_ptr(),
          w.data_ptr(), workspace.data_ptr(), workspace.numel() * workspace.element_size())


def route_select(logits, idx, w, *, score="sigmoid", bias=None, n_group=1, topk_group=1, group_top=1,
                 renormalize=True, scale=1.0, stream=None):
    """moe_route_select: route_grouped's choice on given logits [T, E], bf16 or fp32
    with any row stride (a logit of -inf masks its expert)."""
    _need(logits.dim() == 2, "logits must be [T, E]")
    T, E = logits.shape
    ld = _rows(logits, _TYPE, T, E, "logits")
    k = _choice_outputs(T, E, idx, w, bias)
    _call("moe_route_select", (logits, idx, w, bias), stream, logits.data_ptr(), _TYPE[logits.dtype], ld,
          None if bias is None else bias.data_ptr(), T, E,
          C.byref(_choice(k, score, n_group, topk_group, group_top, bool(renormalize), float(scale))), idx.data_ptr(),
          w.data_ptr())


def _status(t):
    _need(t.dtype == torch.int32 and t.numel() >= 1, "status must be an int32 tensor")
    return t.data_ptr()


class FP4Weight:
    """A 4-bit matrix [N, K] on the device (moe_fp4_weight): codes [N, K/2] uint8 (the
    lower index in the low nibble), block scales [N, K/32] (mxfp4, E8M0) or [N, K/16]
    (nvfp4, E4M3) uint8, and NVFP4's tensor scale.  Keeps the tensors."""

    def __init__(self, codes, scales, fmt, tensor_scale=1.0):
        _need(fmt in FMT, f"fmt must be one of {sorted(FMT)}")
        _need(codes.dim() == 2 and scales.dim() == 2 and codes.dtype == scales.dtype == torch.uint8
              and codes.is_contiguous() and scales.is_contiguous(), "codes and scales must be contiguous 2-D uint8")
        N, K = codes.shape[0], codes.shape[1] * 2
        _need(K % 32 == 0 and K > 0 and N > 0, "K must be a positive multiple of 32, N positive")
        _need(tuple(scales.shape) == (N, K // (32 if fmt == "mxfp4" else 16)),
              "scales must be [N, K/32] (mxfp4) or [N, K/16] (nvfp4)")
        _need(codes.device.type == "cuda" and codes.device == scales.device,
              "codes and scales must be on one CUDA device")
        self.codes, self.scales, self.fmt, self.tensor_scale = codes, scales, fmt, float(tensor_scale)
        self.N, self.K = N, K
        self._desc = L.Fp4WeightDesc(codes.data_ptr(), scales.data_ptr(), self.tensor_scale, N, K, FMT[fmt])
        self.ref = C.byref(self._desc)


def fp4_linear(x, weight, y, status, add=None, stream=None):
    """moe_fp4_linear: y [T, N] (bf16 or fp32) = add + x W^T for x [T, K] (bf16 or fp32),
    T <= 16.  add: None or like y (it may be y itself).  Row strides are free."""
    _need(x.dim() == 2, "x must be [T, K]")
    T = x.shape[0]
    ldx = _rows(x, _TYPE, T, weight.K, "x")
    ldy = _rows(y, _TYPE, T, weight.N, "y")
    lda = 0 if add is None else _rows(add, (y.dtype,), T, weight.N, "add")
    _call("moe_fp4_linear", (x, weight.codes, y, status, add), stream, weight.ref, x.data_ptr(), _TYPE[x.dtype], ldx,
          T, None if add is None else add.data_ptr(), lda, y.data_ptr(), _TYPE[y.dtype], ldy, _status(status))


def fp4_swiglu(x, gate, up, h, status, stream=None):
    """moe_fp4_swiglu: h [T, N] fp32 = silu(x W_gate^T) * (x W_up^T), T <= 16."""
    _need(x.dim() == 2, "x must be [T, K]")
    T = x.shape[0]
    ldx = _rows(x, _TYPE, T, gate.K, "x")
    ldh = _rows(h, (torch.float32,), T, gate.N, "h")
    _call("moe_fp4_swiglu", (x, gate.codes, up.codes, h, status), stream, gate.ref, up.ref, x.data_ptr(),
          _TYPE[x.dtype], ldx, T, h.data_ptr(), ldh, _status(status))


class SharedExpert:
    """The always-active SwiGLU expert beside a layer's routed ones: gate and up [I, H],
    down [H, I] as FP4Weight."""

    def __init__(self, gate, up, down):
        _need((gate.N, gate.K, gate.fmt) == (up.N, up.K, up.fmt), "gate and up must have one shape and format")
        _need((down.N, down.K) == (gate.K, gate.N), "down must be [H, I] for gate and up [I, H]")
        self.gate, self.up, self.down = gate, up, down
        self.I, self.H = gate.N, gate.K

    def hidden(self, x, h, status, stream=None):
        """h [T, I] fp32 = silu(x W_gate^T) * (x W_up^T) for x [T, H] bf16."""
        fp4_swiglu(x, self.gate, self.up, h, status, stream=stream)

    def add_down(self, h, y, status, stream=None):
        """y [T, H] bf16 += h W_down^T."""
        fp4_linear(h, self.down, y, status, add=y, stream=stream)

    def add_to(self, x, h, y, status, stream=None):
        """y [T, H] bf16 += the expert's output for x [T, H] bf16; h [T, I] fp32 scratch."""
        self.hidden(x, h, status, stream)
        self.add_down(h, y, status, stream)


class Lookup:
    """Host-side result of one slot lookup (arrays sized for the call)."""

    def __init__(self, cap):
        self.uniq = np.zeros(cap, np.int32)
        self.is_hit = np.zeros(cap, np.int32)
        self.misses = (L.Miss * cap)()
        self.res = L.LookupResult(0, 0, self.uniq.ctypes.data_as(C.POINTER(C.c_int32)),
                                  self.is_hit.ctypes.data_as(C.POINTER(C.c_int32)), self.misses)

    @property
    def n_uniq(self):
        return self.res.n_uniq

    @property
    def n_miss(self):
        return self.res.n_miss

    def miss_list(self):
        return [(m.expert, m.slot, m.ticket, m.evicted_key) for m in self.misses[:self.res.n_miss]]


def slot_lookup(pool, layer, idx, slot_of, result=None, stream=None):
    T, k = idx.shape
    if result is None:
        result = Lookup(min(T * k, pool.E))
    L.check("moe_slot_lookup", pool.lib.moe_slot_lookup(
        pool.handle, int(layer), _p(idx), T, k, _p(slot_of), C.byref(result.res), _s(stream)))
    return result


def slot_lookup_launch(pool, layer, idx, slot_of, stream=None):
    T, k = idx.shape
    L.check("moe_slot_lookup_launch", pool.lib.moe_slot_lookup_launch(
        pool.handle, int(layer), _p(idx), T, k, _p(slot_of), _s(stream)))


def slot_lookup_result(pool, result):
    L.check("moe_slot_lookup_result", pool.lib.moe_slot_lookup_result(pool.handle, C.byref(result.res)))
    return result


def stream_misses(pool, layer, lookup, copy_stream):
    L.check("moe_stream_misses", pool.lib.moe_stream_misses(
        pool.handle, int(layer), lookup.misses, lookup.res.n_miss, _s(copy_stream)))


def expert_ffn(pool, layer, x, idx, w, slot_of, y_part, status, y=None, stream=None):
    """moe_expert_ffn: y_part [T, k, H] fp32; with y [T, H] bf16 also the fused combine."""
    T = x.shape[0]
    L.check("moe_expert_ffn", pool.lib.moe_expert_ffn(
        pool.handle, int(layer), _p(x), T, _p(idx), _p(w), _p(slot_of), _p(y_part), _p(y), _p(status),
        _s(stream)))


def ffn_launch_info(pool, T):
    """moe_ffn_launch_info: the decode FFN's launch shape for T tokens on this pool."""
    c, st, sb, sm = C.c_int(), C.c_int(), C.c_int(), C.c_int()
    L.check("moe_ffn_launch_info", pool.lib.moe_ffn_launch_info(
        pool.handle, int(T), C.byref(c), C.byref(st), C.byref(sb), C.byref(sm)))
    return dict(ctas=c.value, stages=st.value, stage_bytes=sb.value, smem_bytes=sm.value)


def decode_layer(pool, layer, x, wr, bias, renormalize, idx, w, slot_of, y_part, y, status, ws,
                 lookup=None, copy_events=None, overlap=True, stream=None, copy_stream=None):
    """moe_decode_layer: route, lookup, FFN, miss copies and combine of one layer."""
    T = x.shape[0]
    if copy_stream is None:
        raise ValueError("decode_layer needs a copy_stream of its own (torch.cuda.Stream())")
    cs = copy_stream
    ev0, ev1 = (None, None) if copy_events is None else (C.c_void_p(copy_events[0].cuda_event),
                                                        C.c_void_p(copy_events[1].cuda_event))
    L.check("moe_decode_layer", pool.lib.moe_decode_layer(
        pool.handle, int(layer), _p(x), T, _p(wr), _p(bias), int(renormalize), _p(idx), _p(w),
        _p(slot_of), _p(y_part), _p(y), _p(status), _p(ws), ws.numel(),
        C.byref(lookup.res) if lookup is not None else None, ev0, ev1, 1 if overlap else 0,
        _s(stream), _s(cs)))


def decode_layer_routed(pool, layer, x, idx, w, slot_of, y_part, y, status, lookup=None, copy_events=None,
                        overlap=True, stream=None, copy_stream=None):
    """moe_decode_layer_routed: lookup, FFN, miss copies and combine of one layer for
    idx and w that another router wrote on the same stream."""
    if copy_stream is None:
        raise ValueError("decode_layer_routed needs a copy_stream of its own (torch.cuda.Stream())")
    T = x.shape[0]
    _need(idx.dtype == torch.int32 and idx.shape == (T, pool.k) and idx.is_contiguous(),
          "idx must be a contiguous int32 [T, k], k the pool's")
    _need(w.dtype == torch.float32 and w.shape == (T, pool.k) and w.is_contiguous(),
          "w must be a contiguous float32 [T, k], k the pool's")
    _need(idx.is_cuda and idx.device == w.device == x.device, "x, idx and w must be on one CUDA device")
    ev0, ev1 = (None, None) if copy_events is None else (C.c_void_p(copy_events[0].cuda_event),
                                                        C.c_void_p(copy_events[1].cuda_event))
    L.check("moe_decode_layer_routed", pool.lib.moe_decode_layer_routed(
        pool.handle, int(layer), _p(x), x.shape[0], _p(idx), _p(w), _p(slot_of), _p(y_part), _p(y), _p(status),
        C.byref(lookup.res) if lookup is not None else None, ev0, ev1, 1 if overlap else 0, _s(stream),
        _s(copy_stream)))


def decode_resident(pool, layer0, x, wr, bias, renormalize, idx, w, slot_of, y_part, y, status, stream=None):
    """moe_decode_resident: one FFN launch per layer with the router, the resident
    lookup and the combine fused in, for x.shape[0] consecutive layers from
    layer0, with no host wait (capturable in a CUDA graph).  x, y: [n_layers, T, H]
    bf16; wr: list of n_layers [E, H] bf16; bias: list of n_layers [E] fp32
    (entries may be None) or None."""
    n, T = x.shape[0], x.shape[1]
    if len(wr) != n or (bias is not None and len(bias) != n):
        raise ValueError("decode_resident: one router weight (and bias) per layer")
    wr_arr = (C.c_void_p * n)(*[t.data_ptr() for t in wr])
    b_arr = None if bias is None else (C.c_void_p * n)(*[None if b is None else b.data_ptr() for b in bias])
    L.check("moe_decode_resident", pool.lib.moe_decode_resident(
        pool.handle, int(layer0), n, _p(x), T, wr_arr, b_arr, int(renormalize), _p(idx), _p(w), _p(slot_of),
        _p(y_part), _p(y), _p(status), _s(stream)))


def combine(y_part, y, stream=None):
    T, k, H = y_part.shape
    L.check("moe_combine", L.load().moe_combine(_p(y_part), T, k, H, _p(y), _s(stream)))


def lru_plan_resize(slot_key, slot_clock, n_new):
    """moe_lru_plan_resize on host arrays: (evicted slots, [(from, to) moves])."""
    sk = np.ascontiguousarray(slot_key, np.int32)
    sc = np.ascontiguousarray(slot_clock, np.uint64)
    n_old = len(sk)
    ev, mf, mt = (np.zeros(n_old, np.int32) for _ in range(3))
    ne, nm = C.c_int(), C.c_int()
    L.check("moe_lru_plan_resize", L.load().moe_lru_plan_resize(
        sk.ctypes.data_as(C.c_void_p), sc.ctypes.data_as(C.c_void_p), n_old, int(n_new),
        ev.ctypes.data_as(C.c_void_p), C.byref(ne), mf.ctypes.data_as(C.c_void_p),
        mt.ctypes.data_as(C.c_void_p), C.byref(nm)))
    return ev[:ne.value].tolist(), list(zip(mf[:nm.value].tolist(), mt[:nm.value].tolist()))


class BandwidthEstimate:
    """Moving estimates of PCIe and host-memory bandwidth (GB/s) and the q* split
    recomputed from them (moe_bw_init / moe_bw_observe / moe_bw_qstar)."""

    def __init__(self, alpha=0.25, b_pcie=0.0, b_host=0.0):
        self.est = L.BwEstimate()
        L.check("moe_bw_init", L.load().moe_bw_init(C.byref(self.est), float(alpha), float(b_pcie),
                                                     float(b_host)))

    def observe(self, link, nbytes, seconds):
        """link: "pcie" or "host"."""
        which = {"pcie": L.MOE_BW_PCIE, "host": L.MOE_BW_HOST}[link]
        L.check("moe_bw_observe", L.load().moe_bw_observe(C.byref(self.est), which, float(nbytes),
                                                           float(seconds)))

    @property
    def b_pcie(self):
        return self.est.b_pcie

    @property
    def b_host(self):
        return self.est.b_host

    def qstar(self, m):
        qg, qc, r = C.c_int(), C.c_int(), C.c_double()
        L.check("moe_bw_qstar", L.load().moe_bw_qstar(C.byref(self.est), int(m), C.byref(qg), C.byref(qc),
                                                       C.byref(r)))
        return qg.value, qc.value, r.value


def qstar_split(m, b_pcie, b_host):
    qg, qc, r = C.c_int(), C.c_int(), C.c_double()
    L.check("qstar_split", L.load().qstar_split(int(m), float(b_pcie), float(b_host),
                                                C.byref(qg), C.byref(qc), C.byref(r)))
    return qg.value, qc.value, r.value


def dequant_slot(pool, slot, key, which, out, stream=None):
    L.check("moe_dequant_slot", pool.lib.moe_dequant_slot(
        pool.handle, int(slot), int(key), int(which), _p(out), _s(stream)))


def nvfp4_gemm(a_codes, a_scales, b_codes, b_scales, D, status, stream=None):
    """D [M, N] fp32 = dq(A) dq(B)^T for NVFP4 A [M, K] and B [N, K] (codes uint8
    [rows, K/2], E4M3 scales uint8 [rows, K/16]), on the tcgen05 tensor cores."""
    M, N, K = a_codes.shape[0], b_codes.shape[0], a_codes.shape[1] * 2
    L.check("moe_nvfp4_gemm", L.load().moe_nvfp4_gemm(
        _p(a_codes), _p(a_scales), _p(b_codes), _p(b_scales), M, N, K, _p(D), _p(status), _s(stream)))


def nvfp4_quantize(x, codes, scales, sx, stream=None):
    """Per-token NVFP4 quantisation of x [T, H] bf16 (the prefill A operand)."""
    T, H = x.shape
    L.check("moe_nvfp4_quantize", L.load().moe_nvfp4_quantize(
        _p(x), T, H, _p(codes), _p(scales), _p(sx), _s(stream)))


def prefill_workspace_bytes(pool, T):
    return pool.lib.moe_prefill_workspace_bytes(pool.handle, int(T))


def prefill_ffn(pool, layer, x, idx, w, slot_of, y, workspace, status, stream=None):
    """y: y_part [T, k, H] fp32, every row written: the routed experts' FFN outputs
    times their routing weights, one row per (token, rank); sum and round them in
    rank order with combine(y, y_bf16)."""
    T = x.shape[0]
    L.check("moe_prefill_ffn", pool.lib.moe_prefill_ffn(
        pool.handle, int(layer), _p(x), T, _p(idx), _p(w), _p(slot_of), _p(y), _p(workspace),
        workspace.numel() * workspace.element_size(), _p(status), _s(stream)))


def set_wait_limits(ready_ms, dep_ms, pipe_ms):
    L.check("moe_set_wait_limits", L.load().moe_set_wait_limits(float(ready_ms), float(dep_ms),
                                                                 float(pipe_ms)))
