"""ctypes binding of libmoefp8.so (the C ABI declared in include/moefp8.h).

Argument marshalling only: every step of the layer runs in the library's
CUDA kernels.  Functions keep the C names; tensors are torch tensors on the
current CUDA device (their data pointers are passed), and `stream` defaults to
torch's current stream.  A non-zero status raises MoeError.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libmoefp8.so")

MOE_OK = 0
MOE_EPI_F32 = 0
MOE_EPI_BF16 = 1
MOE_EPI_SWIGLU_QUANT = 2
MOE_DEV_TIMEOUT = 1
MOE_T_F32 = 0
MOE_T_BF16 = 1
MOE_T_F16 = 2
MOE_T_CKPT = 3


class MoeError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn} failed: status {status} ({status_string(status)})")


class MoeShape(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int), ("d", ctypes.c_int), ("n_routed", ctypes.c_int),
                ("n_groups", ctypes.c_int), ("topk_groups", ctypes.c_int),
                ("topk", ctypes.c_int), ("inter", ctypes.c_int), ("gamma", ctypes.c_float)]


class MoeWeights(ctypes.Structure):
    _fields_ = [("w13", ctypes.c_void_p), ("w13_scales", ctypes.c_void_p),
                ("w2", ctypes.c_void_p), ("w2_scales", ctypes.c_void_p),
                ("router_w", ctypes.c_void_p)]


class MoeWeightsMx(ctypes.Structure):
    _fields_ = [("w13", ctypes.c_void_p), ("w13_sf", ctypes.c_void_p),
                ("w2", ctypes.c_void_p), ("w2_sf", ctypes.c_void_p),
                ("router_w", ctypes.c_void_p)]


class MoeRouting(ctypes.Structure):
    _fields_ = [("topk_idx", ctypes.c_void_p), ("topk_gate", ctypes.c_void_p),
                ("expert_counts", ctypes.c_void_p), ("expert_offsets", ctypes.c_void_p),
                ("row_of_pair", ctypes.c_void_p)]


_L = None


def lib() -> ctypes.CDLL:
    """Load libmoefp8.so (built in-tree by __graft_entry__.build()).  Raises
    if it is missing: there is no fallback implementation."""
    global _L
    if _L is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing; build it with "
                              "`python -c 'import __graft_entry__ as g; g.build()'`")
        L = ctypes.CDLL(LIB_PATH)
        P, I, I64, SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
        SP = ctypes.POINTER(MoeShape)
        sig = {
            "moe_version": (I, []),
            "moe_status_string": (ctypes.c_char_p, [I]),
            "moe_read_status": (I, [P, P, P]),
            "moe_route_workspace_size": (SZ, [SP]),
            "moe_route": (I, [SP, P, P, P, P, P, P, P, P, SZ, P, P]),
            "moe_route_scores": (I, [SP, P, P, P, P, P, P, P, P, P, SZ, P, P]),
            "fp8_transpose_w_128x128": (I, [P, P, I64, I64, I64, P, P, P, P]),
            "moe_combine_backward_quant": (I, [SP, P, P, P, P, P, P, P]),
            "moe_swiglu_backward_quant": (I, [P, P, I64, I, I64, P, P, P, P]),
            "moe_gate_backward": (I, [SP, P, P, P, P, P, P, P, P]),
            "moe_router_backward_workspace_size": (SZ, [SP]),
            "moe_router_backward": (I, [SP, P, P, P, P, P, P, P, P, P, P, SZ, P, P]),
            "moe_dx_combine": (I, [SP, P, P, P, P, P, P]),
            "moe_wgrad_max_blocks": (I, [I64, I]),
            "moe_wgrad_layout": (I, [I, P, I, P, P, P, P]),
            "moe_wgrad_quant_x": (I, [SP, P, P, P, I, P, P, P, P]),
            "moe_wgrad_quant_do": (I, [SP, P, P, P, P, I, P, P, P, P]),
            "moe_wgrad_quant_h": (I, [P, I, P, I, P, P, P, P]),
            "moe_wgrad_quant_dac": (I, [P, P, I, P, I, P, P, P, P]),
            "moe_grouped_gemm_wgrad": (I, [I, P, I, P, P, I, P, P, I, P, P, P]),
            "fp8_quant_act_1x128": (I, [P, I64, I64, P, P, I, P, P]),
            "fp8_quant_w_128x128": (I, [P, I64, I64, P, P, P, P]),
            "moe_permute_workspace_size": (SZ, [SP]),
            "moe_permute": (I, [SP, P, P, P, P, P, P, P, P, P, SZ, P, P]),
            "moe_permute_static_ws": (I, [SP, P, P, P, P, P, P, P, P, P, P]),
            "moe_quant_permute": (I, [SP, P, P, P, P, P, P, P, P, SZ, P, P]),
            "moe_grouped_gemm_fp8": (I, [I, P, I, P, P, I, P, P, I, I, P, P, P, P]),
            "moe_grouped_gemm_form": (I, [I, I, I, I]),
            "fp8_quant_act_1x128_ue8m0": (I, [P, I64, I64, P, P, I, P, P]),
            "fp8_quant_w_128x128_ue8m0": (I, [P, I64, I64, P, P, P, P]),
            "moe_grouped_gemm_mxfp8": (I, [I, P, I, P, P, I, P, P, I, I, P, P, P, P]),
            "moe_grouped_gemm_fp8_indexed": (I, [I, P, P, I, I, P, P, I, P, P, I, I, P, P, P,
                                                 P]),
            "moe_plan_redundant_experts": (I, [P, I, I, P, P]),
            "moe_quant_permute_ue8m0": (I, [SP, P, P, P, P, P, P, P, P, SZ, P, P]),
            "moe_ep_row_bytes": (SZ, [SP]),
            "moe_ep_workspace_size": (SZ, [SP, I, I]),
            "moe_ep_dispatch_plan": (I, [SP, I, P, P, P, P, P, SZ, P, P]),
            "moe_ep_pack": (I, [SP, I, P, P, P, P, P, P, P]),
            "moe_ep_local_permute": (I, [SP, I, P, I, P, P, I, P, P, P, SZ, P, P]),
            "moe_ep_partial_combine": (I, [SP, I, P, I, P, P, P, P, P]),
            "moe_ep_final_combine": (I, [SP, I, P, P, P, P, P, P]),
            "moe_layer_mx_workspace_size": (SZ, [SP]),
            "moe_layer_forward_mx": (I, [SP, ctypes.POINTER(MoeWeightsMx), P, P, P,
                                         ctypes.POINTER(MoeRouting), P, I, P, SZ, P, P]),
            "moe_layernorm_forward": (I, [P, I, I64, I, P, P, ctypes.c_float, P, P, P, P, P]),
            "moe_layernorm_backward_workspace_size": (SZ, [I64, I]),
            "moe_layernorm_backward": (I, [P, I, P, I, P, I64, I, P, P, P, P, P, P, P, SZ, P, P]),
            "moe_ckpt_row_bytes": (I64, [I64]),
            "moe_ckpt_pack": (I, [P, I, I64, I64, P, P, P, P]),
            "moe_ckpt_unpack": (I, [P, P, I64, I64, P, I, P, P]),
            "moe_grouped_gemm_fp8_ckpt": (I, [I, P, I, P, P, I, P, P, I, P, P, P, P, P, P]),
            "moe_swiglu_backward_quant_ckpt": (I, [P, P, P, I64, I, I64, P, P, P, P]),
            "moe_wgrad_quant_h_ckpt": (I, [P, P, I64, I, P, I, P, P, P, P]),
            "moe_wgrad_quant_dac_ckpt": (I, [P, P, P, I64, I, P, I, P, P, P, P]),
            "moe_gate_backward_ckpt": (I, [SP, P, P, P, P, P, P, P, P, P]),
            "moe_ffn_forward": (I, [P, P, P, I, I64, I, I, P, P, P, I, P, P, P]),
            "moe_ffn_backward": (I, [P, P, P, P, P, I, P, I, I64, I, I, P, P, P, P, P, P, P]),
            "moe_split_groups": (I, [SP, P, P, P, P, I, P, P, P, P]),
            "moe_combine": (I, [SP, P, P, P, P, P, P, P]),
            "moe_update_bias": (I, [SP, P, P, P, P]),
            "moe_layer_workspace_size": (SZ, [SP]),
            "moe_layer_forward": (I, [SP, ctypes.POINTER(MoeWeights), P, P, P,
                                      ctypes.POINTER(MoeRouting), P, I, P, SZ, P, P]),
            "moe_layer_host_workspace_size": (SZ, [SP]),
            "moe_layer_forward_host": (I, [SP, ctypes.POINTER(MoeWeights), P, P, P,
                                           ctypes.POINTER(MoeRouting), P, I, P, SZ, P, P]),
            "moe_layer_host_batches_workspace_size": (SZ, [SP]),
            "moe_layer_forward_host_batches": (I, [SP, ctypes.POINTER(MoeWeights), P, I, P, P,
                                                   ctypes.POINTER(MoeRouting), P, I, P, SZ, P,
                                                   P]),
        }
        for name, (res, args) in sig.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _L = L
    return _L


def status_string(status: int) -> str:
    return lib().moe_status_string(int(status)).decode()


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        c = _get_torch()._C
        return c._cuda_getCurrentRawStream(c._cuda_getDevice())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(name: str, rc: int) -> None:
    if rc != MOE_OK:
        raise MoeError(name, rc)


def make_shape(T, d, n_routed, n_groups, topk_groups, topk, inter, gamma=0.001) -> MoeShape:
    return MoeShape(int(T), int(d), int(n_routed), int(n_groups), int(topk_groups), int(topk),
                    int(inter), float(gamma))


def moe_version() -> int:
    return lib().moe_version()


def moe_read_status(dev_status, stream=None) -> int:
    out = ctypes.c_int(0)
    _check("moe_read_status", lib().moe_read_status(_ptr(dev_status), ctypes.addressof(out),
                                                    _stream(stream)))
    return out.value


def moe_route_workspace_size(shape: MoeShape) -> int:
    return lib().moe_route_workspace_size(ctypes.byref(shape))


def moe_route(shape, x, router_w, bias, logit_offset, topk_idx, topk_gate, expert_counts,
              ws, dev_status=None, stream=None) -> None:
    nbytes = ws.numel() * ws.element_size() if ws is not None else 0
    _check("moe_route", lib().moe_route(
        ctypes.byref(shape), _ptr(x), _ptr(router_w), _ptr(bias), _ptr(logit_offset),
        _ptr(topk_idx), _ptr(topk_gate), _ptr(expert_counts), _ptr(ws), nbytes,
        _ptr(dev_status), _stream(stream)))


def moe_route_scores(shape, x, router_w, bias, logit_offset, topk_idx, topk_gate, topk_score,
                     expert_counts, ws, dev_status=None, stream=None) -> None:
    """moe_route that also returns the chosen unbiased affinities (topk_score)."""
    nbytes = ws.numel() * ws.element_size() if ws is not None else 0
    _check("moe_route_scores", lib().moe_route_scores(
        ctypes.byref(shape), _ptr(x), _ptr(router_w), _ptr(bias), _ptr(logit_offset),
        _ptr(topk_idx), _ptr(topk_gate), _ptr(topk_score), _ptr(expert_counts), _ptr(ws),
        nbytes, _ptr(dev_status), _stream(stream)))


def fp8_quant_act_1x128(x, q, scales, scales_kb_major=False, dev_status=None, stream=None):
    rows, cols = x.shape
    _check("fp8_quant_act_1x128", lib().fp8_quant_act_1x128(
        _ptr(x), rows, cols, _ptr(q), _ptr(scales), int(bool(scales_kb_major)),
        _ptr(dev_status), _stream(stream)))


def fp8_quant_w_128x128(w, q, scales, dev_status=None, stream=None):
    rows, cols = w.shape
    _check("fp8_quant_w_128x128", lib().fp8_quant_w_128x128(
        _ptr(w), rows, cols, _ptr(q), _ptr(scales), _ptr(dev_status), _stream(stream)))


def moe_permute_workspace_size(shape: MoeShape) -> int:
    return lib().moe_permute_workspace_size(ctypes.byref(shape))


def moe_permute(shape, topk_idx, expert_counts, xq, xs, xq_perm, xs_perm, expert_offsets,
                row_of_pair, ws, dev_status=None, stream=None):
    nbytes = ws.numel() * ws.element_size() if ws is not None else 0
    _check("moe_permute", lib().moe_permute(
        ctypes.byref(shape), _ptr(topk_idx), _ptr(expert_counts), _ptr(xq), _ptr(xs),
        _ptr(xq_perm), _ptr(xs_perm), _ptr(expert_offsets), _ptr(row_of_pair), _ptr(ws), nbytes,
        _ptr(dev_status), _stream(stream)))


def moe_quant_permute(shape, x, topk_idx, expert_counts, xq_perm, xs_perm, expert_offsets,
                      row_of_pair, ws, dev_status=None, stream=None):
    """fp8_quant_act_1x128 of x (bf16 [T, d]) fused with moe_permute."""
    nbytes = ws.numel() * ws.element_size() if ws is not None else 0
    _check("moe_quant_permute", lib().moe_quant_permute(
        ctypes.byref(shape), _ptr(x), _ptr(topk_idx), _ptr(expert_counts), _ptr(xq_perm),
        _ptr(xs_perm), _ptr(expert_offsets), _ptr(row_of_pair), _ptr(ws), nbytes,
        _ptr(dev_status), _stream(stream)))


def moe_permute_static_ws(shape, topk_idx, expert_counts, xq, xs, xq_perm, xs_perm,
                          expert_offsets, row_of_pair, dev_status=None, stream=None):
    """moe_permute for callers that cannot allocate device memory while they
    run: no workspace argument; the library's own fixed 1 MiB device array
    is used instead (ceil(T/64) * N_r <= 262144).  Calls that overlap on the
    GPU share that array and race."""
    _check("moe_permute_static_ws", lib().moe_permute_static_ws(
        ctypes.byref(shape), _ptr(topk_idx), _ptr(expert_counts), _ptr(xq), _ptr(xs),
        _ptr(xq_perm), _ptr(xs_perm), _ptr(expert_offsets), _ptr(row_of_pair),
        _ptr(dev_status), _stream(stream)))


def moe_grouped_gemm_fp8(n_groups, group_offsets, max_rows, a, a_scales, k, w, w_scales, n,
                         epilogue, out, out_scales=None, dev_status=None, stream=None):
    _check("moe_grouped_gemm_fp8", lib().moe_grouped_gemm_fp8(
        int(n_groups), _ptr(group_offsets), int(max_rows), _ptr(a), _ptr(a_scales), int(k),
        _ptr(w), _ptr(w_scales), int(n), int(epilogue), _ptr(out), _ptr(out_scales),
        _ptr(dev_status), _stream(stream)))


def moe_grouped_gemm_form(n_groups, max_rows, n, epilogue) -> int:
    """CTAs per tile moe_grouped_gemm_fp8 uses for these arguments on the
    current device: 1 (single CTAs), 2 (CTA pairs), 0 (invalid arguments)."""
    return int(lib().moe_grouped_gemm_form(int(n_groups), int(max_rows), int(n), int(epilogue)))


def moe_combine(shape, expert_out, expert_offsets, row_of_pair, topk_gate, y,
                dev_status=None, stream=None):
    _check("moe_combine", lib().moe_combine(
        ctypes.byref(shape), _ptr(expert_out), _ptr(expert_offsets), _ptr(row_of_pair),
        _ptr(topk_gate), _ptr(y), _ptr(dev_status), _stream(stream)))


def moe_update_bias(shape, expert_counts, bias, dev_status=None, stream=None):
    _check("moe_update_bias", lib().moe_update_bias(
        ctypes.byref(shape), _ptr(expert_counts), _ptr(bias), _ptr(dev_status),
        _stream(stream)))


def moe_layer_workspace_size(shape: MoeShape) -> int:
    return lib().moe_layer_workspace_size(ctypes.byref(shape))


def moe_layer_host_workspace_size(shape: MoeShape) -> int:
    return lib().moe_layer_host_workspace_size(ctypes.byref(shape))


def make_weights(w13, w13_scales, w2, w2_scales, router_w) -> MoeWeights:
    return MoeWeights(_ptr(w13), _ptr(w13_scales), _ptr(w2), _ptr(w2_scales), _ptr(router_w))


def make_routing(topk_idx, topk_gate, expert_counts, expert_offsets, row_of_pair) -> MoeRouting:
    return MoeRouting(_ptr(topk_idx), _ptr(topk_gate), _ptr(expert_counts),
                      _ptr(expert_offsets), _ptr(row_of_pair))


def moe_layer_forward(shape, weights: MoeWeights, x, bias, logit_offset, routing: MoeRouting,
                      y, update_bias, ws, dev_status=None, stream=None):
    nbytes = ws.numel() * ws.element_size()
    _check("moe_layer_forward", lib().moe_layer_forward(
        ctypes.byref(shape), ctypes.byref(weights), _ptr(x), _ptr(bias), _ptr(logit_offset),
        ctypes.byref(routing), _ptr(y), int(bool(update_bias)), _ptr(ws), nbytes,
        _ptr(dev_status), _stream(stream)))


def moe_layer_forward_host(shape, weights: MoeWeights, x_host, bias, logit_offset,
                           routing: MoeRouting, y_host, update_bias, ws, dev_status=None,
                           stream=None):
    nbytes = ws.numel() * ws.element_size()
    _check("moe_layer_forward_host", lib().moe_layer_forward_host(
        ctypes.byref(shape), ctypes.byref(weights), _ptr(x_host), _ptr(bias),
        _ptr(logit_offset), ctypes.byref(routing), _ptr(y_host), int(bool(update_bias)),
        _ptr(ws), nbytes, _ptr(dev_status), _stream(stream)))


def moe_layer_host_batches_workspace_size(shape: MoeShape) -> int:
    return lib().moe_layer_host_batches_workspace_size(ctypes.byref(shape))


def moe_layer_forward_host_batches(shape, weights: MoeWeights, x_host, n_batches, bias,
                                   logit_offset, routing: MoeRouting, y_host, update_bias, ws,
                                   dev_status=None, stream=None):
    """n_batches successive batches, x_host / y_host pinned [n_batches, T, d]."""
    nbytes = ws.numel() * ws.element_size()
    _check("moe_layer_forward_host_batches", lib().moe_layer_forward_host_batches(
        ctypes.byref(shape), ctypes.byref(weights), _ptr(x_host), int(n_batches), _ptr(bias),
        _ptr(logit_offset), ctypes.byref(routing), _ptr(y_host), int(bool(update_bias)),
        _ptr(ws), nbytes, _ptr(dev_status), _stream(stream)))


# ------------------------------------------- power-of-two scale option
def fp8_quant_act_1x128_ue8m0(x, q, sf, sf_kb_major=False, dev_status=None, stream=None):
    """1x128 tiles with power-of-two scales; sf: uint8 UE8M0 bytes."""
    rows, cols = x.shape
    _check("fp8_quant_act_1x128_ue8m0", lib().fp8_quant_act_1x128_ue8m0(
        _ptr(x), rows, cols, _ptr(q), _ptr(sf), int(bool(sf_kb_major)), _ptr(dev_status),
        _stream(stream)))


def fp8_quant_w_128x128_ue8m0(w, q, sf, dev_status=None, stream=None):
    rows, cols = w.shape
    _check("fp8_quant_w_128x128_ue8m0", lib().fp8_quant_w_128x128_ue8m0(
        _ptr(w), rows, cols, _ptr(q), _ptr(sf), _ptr(dev_status), _stream(stream)))


def moe_grouped_gemm_mxfp8(n_groups, group_offsets, max_rows, a, a_sf, k, w, w_sf, n, epilogue,
                           out, out_sf=None, dev_status=None, stream=None):
    _check("moe_grouped_gemm_mxfp8", lib().moe_grouped_gemm_mxfp8(
        int(n_groups), _ptr(group_offsets), int(max_rows), _ptr(a), _ptr(a_sf), int(k), _ptr(w),
        _ptr(w_sf), int(n), int(epilogue), _ptr(out), _ptr(out_sf), _ptr(dev_status),
        _stream(stream)))


# ----------------------------------------------------- redundant experts
def moe_grouped_gemm_fp8_indexed(n_groups, group_offsets, group_weight, n_weights, max_rows, a,
                                 a_scales, k, w, w_scales, n, epilogue, out, out_scales=None,
                                 dev_status=None, stream=None):
    _check("moe_grouped_gemm_fp8_indexed", lib().moe_grouped_gemm_fp8_indexed(
        int(n_groups), _ptr(group_offsets), _ptr(group_weight), int(n_weights), int(max_rows),
        _ptr(a), _ptr(a_scales), int(k), _ptr(w), _ptr(w_scales), int(n), int(epilogue),
        _ptr(out), _ptr(out_scales), _ptr(dev_status), _stream(stream)))


def moe_plan_redundant_experts(counts, n_extra):
    """Host planner: counts (sequence of ints) -> (replicas, slot_expert) as
    numpy int32 arrays."""
    import numpy as np
    c = np.ascontiguousarray(np.asarray(counts, dtype=np.int32))
    rep = np.empty(c.size, dtype=np.int32)
    slots = np.empty(c.size + int(n_extra), dtype=np.int32)
    _check("moe_plan_redundant_experts", lib().moe_plan_redundant_experts(
        c.ctypes.data, int(c.size), int(n_extra), rep.ctypes.data, slots.ctypes.data))
    return rep, slots


def moe_split_groups(shape, expert_offsets, replicas, slot_expert, first_slot, n_extra,
                     slot_offsets, slot_weight, dev_status=None, stream=None):
    _check("moe_split_groups", lib().moe_split_groups(
        ctypes.byref(shape), _ptr(expert_offsets), _ptr(replicas), _ptr(slot_expert),
        _ptr(first_slot), int(n_extra), _ptr(slot_offsets), _ptr(slot_weight), _ptr(dev_status),
        _stream(stream)))


def moe_quant_permute_ue8m0(shape, x, topk_idx, expert_counts, xq_perm, xsf_perm,
                            expert_offsets, row_of_pair, ws, dev_status=None, stream=None):
    """moe_quant_permute with power-of-two scales (xsf_perm: uint8 UE8M0)."""
    nbytes = ws.numel() * ws.element_size() if ws is not None else 0
    _check("moe_quant_permute_ue8m0", lib().moe_quant_permute_ue8m0(
        ctypes.byref(shape), _ptr(x), _ptr(topk_idx), _ptr(expert_counts), _ptr(xq_perm),
        _ptr(xsf_perm), _ptr(expert_offsets), _ptr(row_of_pair), _ptr(ws), nbytes,
        _ptr(dev_status), _stream(stream)))


def moe_layer_mx_workspace_size(shape: MoeShape) -> int:
    return lib().moe_layer_mx_workspace_size(ctypes.byref(shape))


def make_weights_mx(w13, w13_sf, w2, w2_sf, router_w) -> MoeWeightsMx:
    return MoeWeightsMx(_ptr(w13), _ptr(w13_sf), _ptr(w2), _ptr(w2_sf), _ptr(router_w))


def moe_layer_forward_mx(shape, weights: MoeWeightsMx, x, bias, logit_offset,
                         routing: MoeRouting, y, update_bias, ws, dev_status=None, stream=None):
    nbytes = ws.numel() * ws.element_size()
    _check("moe_layer_forward_mx", lib().moe_layer_forward_mx(
        ctypes.byref(shape), ctypes.byref(weights), _ptr(x), _ptr(bias), _ptr(logit_offset),
        ctypes.byref(routing), _ptr(y), int(bool(update_bias)), _ptr(ws), nbytes,
        _ptr(dev_status), _stream(stream)))


# -------------------------------------------------- expert parallelism
def moe_ep_row_bytes(shape) -> int:
    return int(lib().moe_ep_row_bytes(ctypes.byref(shape)))


def moe_ep_workspace_size(shape, n_ranks, max_recv_rows) -> int:
    return int(lib().moe_ep_workspace_size(ctypes.byref(shape), int(n_ranks),
                                           int(max_recv_rows)))


def moe_ep_dispatch_plan(shape, n_ranks, topk_idx, send_counts, send_offsets, send_row, ws,
                         dev_status=None, stream=None):
    nbytes = ws.numel() * ws.element_size()
    _check("moe_ep_dispatch_plan", lib().moe_ep_dispatch_plan(
        ctypes.byref(shape), int(n_ranks), _ptr(topk_idx), _ptr(send_counts),
        _ptr(send_offsets), _ptr(send_row), _ptr(ws), nbytes, _ptr(dev_status),
        _stream(stream)))


def moe_ep_pack(shape, n_ranks, x, topk_idx, topk_gate, send_row, send_buf, dev_status=None,
                stream=None):
    _check("moe_ep_pack", lib().moe_ep_pack(
        ctypes.byref(shape), int(n_ranks), _ptr(x), _ptr(topk_idx), _ptr(topk_gate),
        _ptr(send_row), _ptr(send_buf), _ptr(dev_status), _stream(stream)))


def moe_ep_local_permute(shape, n_ranks, recv_buf, n_recv, xq_perm, xs_perm, max_rows,
                         local_offsets, pair_row, ws, dev_status=None, stream=None):
    nbytes = ws.numel() * ws.element_size()
    _check("moe_ep_local_permute", lib().moe_ep_local_permute(
        ctypes.byref(shape), int(n_ranks), _ptr(recv_buf), int(n_recv), _ptr(xq_perm),
        _ptr(xs_perm), int(max_rows), _ptr(local_offsets), _ptr(pair_row), _ptr(ws), nbytes,
        _ptr(dev_status), _stream(stream)))


def moe_ep_partial_combine(shape, n_ranks, recv_buf, n_recv, pair_row, expert_out, back_buf,
                           dev_status=None, stream=None):
    _check("moe_ep_partial_combine", lib().moe_ep_partial_combine(
        ctypes.byref(shape), int(n_ranks), _ptr(recv_buf), int(n_recv), _ptr(pair_row),
        _ptr(expert_out), _ptr(back_buf), _ptr(dev_status), _stream(stream)))


def moe_ep_final_combine(shape, n_ranks, shared_out, back_recv, send_row, y, dev_status=None,
                         stream=None):
    _check("moe_ep_final_combine", lib().moe_ep_final_combine(
        ctypes.byref(shape), int(n_ranks), _ptr(shared_out), _ptr(back_recv), _ptr(send_row),
        _ptr(y), _ptr(dev_status), _stream(stream)))


# ------------------------------------------------------------- backward
def fp8_transpose_w_128x128(q, scales, qt, scales_t, dev_status=None, stream=None):
    """q uint8 [mats, rows, cols] (or [rows, cols]), scales fp32
    [mats, rows/128, cols/128] -> the transposed codes and scales."""
    rows, cols = q.shape[-2], q.shape[-1]
    mats = q.numel() // max(rows * cols, 1) if rows * cols else 0
    _check("fp8_transpose_w_128x128", lib().fp8_transpose_w_128x128(
        _ptr(q), _ptr(scales), int(mats), int(rows), int(cols), _ptr(qt), _ptr(scales_t),
        _ptr(dev_status), _stream(stream)))


def moe_combine_backward_quant(shape, dy, row_of_pair, topk_gate, do_q, do_scales,
                               dev_status=None, stream=None):
    _check("moe_combine_backward_quant", lib().moe_combine_backward_quant(
        ctypes.byref(shape), _ptr(dy), _ptr(row_of_pair), _ptr(topk_gate), _ptr(do_q),
        _ptr(do_scales), _ptr(dev_status), _stream(stream)))


def moe_swiglu_backward_quant(dh, ac, rows, inter, rows_total, q, q_scales, dev_status=None,
                              stream=None):
    _check("moe_swiglu_backward_quant", lib().moe_swiglu_backward_quant(
        _ptr(dh), _ptr(ac), int(rows), int(inter), int(rows_total), _ptr(q), _ptr(q_scales),
        _ptr(dev_status), _stream(stream)))


def moe_gate_backward(shape, dy, expert_out, row_of_pair, topk_score, dgate, du,
                      dev_status=None, stream=None):
    _check("moe_gate_backward", lib().moe_gate_backward(
        ctypes.byref(shape), _ptr(dy), _ptr(expert_out), _ptr(row_of_pair), _ptr(topk_score),
        _ptr(dgate), _ptr(du), _ptr(dev_status), _stream(stream)))


def moe_router_backward_workspace_size(shape) -> int:
    return int(lib().moe_router_backward_workspace_size(ctypes.byref(shape)))


def moe_router_backward(shape, x, router_w, du, topk_idx, expert_offsets, row_of_pair,
                        pair_scratch, dx_router, d_router_w, ws, dev_status=None, stream=None):
    nbytes = ws.numel() * ws.element_size() if ws is not None else 0
    _check("moe_router_backward", lib().moe_router_backward(
        ctypes.byref(shape), _ptr(x), _ptr(router_w), _ptr(du), _ptr(topk_idx),
        _ptr(expert_offsets), _ptr(row_of_pair), _ptr(pair_scratch), _ptr(dx_router),
        _ptr(d_router_w), _ptr(ws), nbytes, _ptr(dev_status), _stream(stream)))


def moe_dx_combine(shape, dx_rows, dx_router, row_of_pair, dx, dev_status=None, stream=None):
    _check("moe_dx_combine", lib().moe_dx_combine(
        ctypes.byref(shape), _ptr(dx_rows), _ptr(dx_router), _ptr(row_of_pair), _ptr(dx),
        _ptr(dev_status), _stream(stream)))


# ------------------------------------------------------- weight gradients
def moe_wgrad_max_blocks(rows, n_groups) -> int:
    return int(lib().moe_wgrad_max_blocks(int(rows), int(n_groups)))


def moe_wgrad_layout(n_groups, row_offsets, kb_offsets, blocks, dev_status=None, stream=None):
    """blocks: int32 [max_blocks, 2]."""
    _check("moe_wgrad_layout", lib().moe_wgrad_layout(
        int(n_groups), _ptr(row_offsets), int(blocks.shape[0]), _ptr(kb_offsets), _ptr(blocks),
        _ptr(dev_status), _stream(stream)))


def moe_wgrad_quant_x(shape, x, pair_of_row, blocks, xt, xt_scales, dev_status=None,
                      stream=None):
    _check("moe_wgrad_quant_x", lib().moe_wgrad_quant_x(
        ctypes.byref(shape), _ptr(x), _ptr(pair_of_row), _ptr(blocks), int(blocks.shape[0]),
        _ptr(xt), _ptr(xt_scales), _ptr(dev_status), _stream(stream)))


def moe_wgrad_quant_do(shape, dy, topk_gate, pair_of_row, blocks, dot, dot_scales,
                       dev_status=None, stream=None):
    _check("moe_wgrad_quant_do", lib().moe_wgrad_quant_do(
        ctypes.byref(shape), _ptr(dy), _ptr(topk_gate), _ptr(pair_of_row), _ptr(blocks),
        int(blocks.shape[0]), _ptr(dot), _ptr(dot_scales), _ptr(dev_status), _stream(stream)))


def moe_wgrad_quant_h(ac, inter, blocks, ht, ht_scales, dev_status=None, stream=None):
    _check("moe_wgrad_quant_h", lib().moe_wgrad_quant_h(
        _ptr(ac), int(inter), _ptr(blocks), int(blocks.shape[0]), _ptr(ht), _ptr(ht_scales),
        _ptr(dev_status), _stream(stream)))


def moe_wgrad_quant_dac(dh, ac, inter, blocks, dact, dact_scales, dev_status=None, stream=None):
    _check("moe_wgrad_quant_dac", lib().moe_wgrad_quant_dac(
        _ptr(dh), _ptr(ac), int(inter), _ptr(blocks), int(blocks.shape[0]), _ptr(dact),
        _ptr(dact_scales), _ptr(dev_status), _stream(stream)))


def moe_grouped_gemm_wgrad(n_groups, kb_offsets, nkb_total, a_t, a_scales, m, b_t, b_scales, n,
                           out, dev_status=None, stream=None):
    _check("moe_grouped_gemm_wgrad", lib().moe_grouped_gemm_wgrad(
        int(n_groups), _ptr(kb_offsets), int(nkb_total), _ptr(a_t), _ptr(a_scales), int(m),
        _ptr(b_t), _ptr(b_scales), int(n), _ptr(out), _ptr(dev_status), _stream(stream)))


# --------------------------------- layer norm, 8-bit checkpoints, dense block
_TYPES = {}


def _type(t, name, kept=False) -> int:
    """Type code of a tensor; uint8 is a checkpoint's codes where `kept`."""
    code = _types().get(t.dtype)
    if code is None or (code == MOE_T_CKPT and not kept):
        raise ValueError(f"{name}: unsupported dtype {t.dtype}")
    return code


def _types():
    if not _TYPES:
        import torch
        _TYPES.update({torch.float32: MOE_T_F32, torch.bfloat16: MOE_T_BF16,
                       torch.float16: MOE_T_F16, torch.uint8: MOE_T_CKPT})
    return _TYPES


def _mat(name, t, shape, dtype=None):
    """Checks one tensor argument (None passes): on the current CUDA device,
    contiguous, of this shape (and dtype): the library sees only its address."""
    if t is None:
        return
    import torch
    if not t.is_cuda or t.device.index != torch.cuda.current_device():
        raise ValueError(f"{name}: needs a tensor on the current CUDA device, got {t.device}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: not contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {dtype}")


def _mats(first, *specs):
    """_mat for (name, tensor, shape, dtype) of a whole call, in the few
    attribute reads that a call of some microseconds can afford: the first
    tensor's device is compared with the current one, the others' with its.
    Returns the tensors' addresses (None for None)."""
    name, t, shape, dtype = first
    dev = t.get_device()
    if (dev < 0 or dev != _current_device() or t.dtype is not dtype or t.shape != shape
            or not t.is_contiguous()):
        _mat(name, t, shape, dtype)
    at = [t.data_ptr()]
    for name, t, shape, dtype in specs:
        if t is None:
            at.append(None)
            continue
        if (t.get_device() != dev or t.dtype is not dtype or t.shape != shape
                or not t.is_contiguous()):
            _mat(name, t, shape, dtype)
        at.append(t.data_ptr())
    return at


def _scratch(name, t, dev):
    """Address of a workspace or status word of any shape (None for None; an
    address passes): on device `dev`, in one piece."""
    if t is None or isinstance(t, int):
        return t
    if t.get_device() != dev or not t.is_contiguous():
        _mat(name, t, t.shape)
    return t.data_ptr()


def _current_device() -> int:
    return _get_torch()._C._cuda_getDevice()


_torch = None


def _get_torch():
    global _torch
    if _torch is None:
        import torch
        _torch = torch
    return _torch


def _f32():
    return _get_torch().float32


def _u8():
    return _get_torch().uint8


def _tiles(n) -> int:
    return (n + 127) // 128


def _wide(n) -> int:
    return (n + 127) // 128 * 128


def moe_layernorm_forward(x, weight, bias, eps, y, mean=None, rstd=None, dev_status=None,
                          stream=None):
    """y = layer norm of x [rows, cols]; weight, bias fp32 [cols] or None;
    mean, rstd fp32 [rows] out or None."""
    ty, f32 = _type(x, "x"), _f32()
    rows, cols = x.shape
    px, py, pw, pb, pm, pr = _mats(
        ("x", x, (rows, cols), x.dtype), ("y", y, (rows, cols), x.dtype),
        ("weight", weight, (cols,), f32), ("bias", bias, (cols,), f32),
        ("mean", mean, (rows,), f32), ("rstd", rstd, (rows,), f32))
    _check("moe_layernorm_forward", lib().moe_layernorm_forward(
        px, ty, rows, cols, pw, pb, eps, py, pm, pr,
        _scratch("dev_status", dev_status, x.get_device()), _stream(stream)))


def moe_layernorm_backward_workspace_size(rows, cols) -> int:
    return int(lib().moe_layernorm_backward_workspace_size(int(rows), int(cols)))


def moe_layernorm_backward(dy, x, x_scales, weight, mean, rstd, dx, dweight, dbias, ws,
                           dev_status=None, stream=None):
    """Gradients of moe_layernorm_forward.  x as the forward pass had it
    (x_scales None), or kept in 8 bits (uint8 codes and their x_scales)."""
    ty, xt, f32 = _type(dy, "dy"), _type(x, "x", kept=True), _f32()
    rows, cols = dy.shape
    kept = xt == MOE_T_CKPT
    if kept == (x_scales is None):
        raise ValueError("x_scales goes with x kept in 8 bits")
    pdy, px, ps, pw, pm, pr, pdx, pdw, pdb = _mats(
        ("dy", dy, (rows, cols), dy.dtype),
        ("x", x, (rows, _wide(cols) if kept else cols), x.dtype),
        ("x_scales", x_scales, (_tiles(cols), rows), f32), ("weight", weight, (cols,), f32),
        ("mean", mean, (rows,), f32), ("rstd", rstd, (rows,), f32),
        ("dx", dx, (rows, cols), dy.dtype), ("dweight", dweight, (cols,), f32),
        ("dbias", dbias, (cols,), f32))
    nbytes = ws.numel() * ws.element_size() if ws is not None else 0
    dev = dy.get_device()
    _check("moe_layernorm_backward", lib().moe_layernorm_backward(
        pdy, ty, px, xt, ps, rows, cols, pw, pm, pr, pdx, pdw, pdb, _scratch("ws", ws, dev), nbytes,
        _scratch("dev_status", dev_status, dev), _stream(stream)))


def moe_ckpt_row_bytes(cols) -> int:
    return int(lib().moe_ckpt_row_bytes(int(cols)))


def moe_ckpt_pack(x, q, scales, dev_status=None, stream=None):
    """x [rows, cols] -> q uint8 [rows, moe_ckpt_row_bytes(cols)], scales fp32
    [ceil(cols / 128), rows]."""
    ty = _type(x, "x")
    rows, cols = x.shape
    px, pq, ps = _mats(("x", x, (rows, cols), x.dtype), ("q", q, (rows, _wide(cols)), _u8()),
                       ("scales", scales, (_tiles(cols), rows), _f32()))
    _check("moe_ckpt_pack", lib().moe_ckpt_pack(
        px, ty, rows, cols, pq, ps, _scratch("dev_status", dev_status, x.get_device()),
        _stream(stream)))


def moe_ckpt_unpack(q, scales, y, dev_status=None, stream=None):
    """The kept values as y [rows, cols] (its dtype)."""
    ty = _type(y, "y")
    rows, cols = y.shape
    py, pq, ps = _mats(("y", y, (rows, cols), y.dtype), ("q", q, (rows, _wide(cols)), _u8()),
                       ("scales", scales, (_tiles(cols), rows), _f32()))
    _check("moe_ckpt_unpack", lib().moe_ckpt_unpack(
        pq, ps, rows, cols, py, ty, _scratch("dev_status", dev_status, y.get_device()),
        _stream(stream)))


def moe_grouped_gemm_fp8_ckpt(n_groups, group_offsets, max_rows, a, a_scales, k, w, w_scales, n,
                              out, out_scales, ac_q, ac_scales, dev_status=None, stream=None):
    """moe_grouped_gemm_fp8 with MOE_EPI_SWIGLU_QUANT that also keeps gate and
    up in 8 bits."""
    _check("moe_grouped_gemm_fp8_ckpt", lib().moe_grouped_gemm_fp8_ckpt(
        int(n_groups), _ptr(group_offsets), int(max_rows), _ptr(a), _ptr(a_scales), int(k),
        _ptr(w), _ptr(w_scales), int(n), _ptr(out), _ptr(out_scales), _ptr(ac_q),
        _ptr(ac_scales), _ptr(dev_status), _stream(stream)))


def moe_swiglu_backward_quant_ckpt(dh, ac_q, ac_scales, rows, inter, rows_total, q, q_scales,
                                   dev_status=None, stream=None):
    """moe_swiglu_backward_quant from [a | c] kept in 8 bits; dh [>= rows,
    inter], the others rows_total rows."""
    f32, u8, n = _f32(), _u8(), 2 * inter
    pa, ps, ph, pq, pqs = _mats(
        ("ac_q", ac_q, (rows_total, n), u8), ("ac_scales", ac_scales, (n // 128, rows_total), f32),
        ("dh", dh, (dh.shape[0], inter), f32), ("q", q, (rows_total, n), u8),
        ("q_scales", q_scales, (n // 128, rows_total), f32))
    if dh.shape[0] < rows:
        raise ValueError("dh: fewer rows than the call's")
    _check("moe_swiglu_backward_quant_ckpt", lib().moe_swiglu_backward_quant_ckpt(
        ph, pa, ps, rows, inter, rows_total, pq, pqs,
        _scratch("dev_status", dev_status, ac_q.get_device()), _stream(stream)))


def moe_wgrad_quant_h_ckpt(ac_q, ac_scales, inter, blocks, ht, ht_scales, dev_status=None,
                           stream=None):
    """moe_wgrad_quant_h from [a | c] kept in 8 bits."""
    _check("moe_wgrad_quant_h_ckpt", lib().moe_wgrad_quant_h_ckpt(
        _ptr(ac_q), _ptr(ac_scales), int(ac_scales.shape[1]), int(inter), _ptr(blocks),
        int(blocks.shape[0]), _ptr(ht), _ptr(ht_scales), _ptr(dev_status), _stream(stream)))


def moe_wgrad_quant_dac_ckpt(dh, ac_q, ac_scales, inter, blocks, dact, dact_scales,
                             dev_status=None, stream=None):
    """moe_wgrad_quant_dac from [a | c] kept in 8 bits."""
    _check("moe_wgrad_quant_dac_ckpt", lib().moe_wgrad_quant_dac_ckpt(
        _ptr(dh), _ptr(ac_q), _ptr(ac_scales), int(ac_scales.shape[1]), int(inter), _ptr(blocks),
        int(blocks.shape[0]), _ptr(dact), _ptr(dact_scales), _ptr(dev_status), _stream(stream)))


def moe_gate_backward_ckpt(shape, dy, o_q, o_scales, row_of_pair, topk_score, dgate, du,
                           dev_status=None, stream=None):
    """moe_gate_backward from expert outputs kept in 8 bits."""
    _check("moe_gate_backward_ckpt", lib().moe_gate_backward_ckpt(
        ctypes.byref(shape), _ptr(dy), _ptr(o_q), _ptr(o_scales), _ptr(row_of_pair),
        _ptr(topk_score), _ptr(dgate), _ptr(du), _ptr(dev_status), _stream(stream)))


def _kept_ac(ac, ac_scales, dtype, T, inter):
    """Type code of a and c kept by moe_ffn_forward, and what to check of them."""
    if ac is None:
        if ac_scales is not None:
            raise ValueError("ac_scales goes with ac in 8 bits")
        return MOE_T_CKPT, (("ac", None, None, None), ("ac_scales", None, None, None))
    kept = ac.dtype is _u8()
    if kept == (ac_scales is None):
        raise ValueError("ac_scales goes with ac in 8 bits")
    if not kept:
        return _type(ac, "ac"), (("ac", ac, (T, 2 * inter), dtype),
                                 ("ac_scales", None, None, None))
    return MOE_T_CKPT, (("ac", ac, (T, 2 * _wide(inter)), ac.dtype),
                        ("ac_scales", ac_scales, (2 * _tiles(inter), T), _f32()))


def moe_ffn_forward(x, w13, w2, h, y, ac=None, ac_scales=None, dev_status=None, stream=None):
    """y = (silu(x W1^T) (x W3^T)) W2^T for x [T, d], w13 [2 inter, d], w2
    [d, inter]; h [T, inter] out; ac, ac_scales: a and c kept for
    moe_ffn_backward, in 8 bits (uint8 and scales) or in x's type."""
    T, d = x.shape
    inter = w2.shape[1]
    ty, t = _type(x, "x"), x.dtype
    at, kept = _kept_ac(ac, ac_scales, t, T, inter)
    px, p13, p2, ph, py, pac, ps = _mats(
        ("x", x, (T, d), t), ("w13", w13, (2 * inter, d), t), ("w2", w2, (d, inter), t),
        ("h", h, (T, inter), t), ("y", y, (T, d), t), *kept)
    _check("moe_ffn_forward", lib().moe_ffn_forward(
        px, p13, p2, ty, T, d, inter, ph, py, pac, at, ps,
        _scratch("dev_status", dev_status, x.get_device()), _stream(stream)))


def moe_ffn_backward(dy, x, w13, w2, ac, ac_scales, dac, h, dx=None, dw13=None, dw2=None,
                     dev_status=None, stream=None):
    """Gradients of moe_ffn_forward from the kept a and c; dac [T, 2 inter]
    and h [T, inter] are written on the way; dx, dw13, dw2 may be None."""
    T, d = dy.shape
    inter = w2.shape[1]
    ty, t = _type(dy, "dy"), dy.dtype
    if ac is None:
        raise ValueError("moe_ffn_backward needs the kept ac")
    at, kept = _kept_ac(ac, ac_scales, t, T, inter)
    pdy, px, p13, p2, pdac, ph, pdx, pd13, pd2, pac, ps = _mats(
        ("dy", dy, (T, d), t), ("x", x, (T, d), t), ("w13", w13, (2 * inter, d), t),
        ("w2", w2, (d, inter), t), ("dac", dac, (T, 2 * inter), t), ("h", h, (T, inter), t),
        ("dx", dx, (T, d), t), ("dw13", dw13, (2 * inter, d), t), ("dw2", dw2, (d, inter), t),
        *kept)
    _check("moe_ffn_backward", lib().moe_ffn_backward(
        pdy, px, p13, p2, pac, at, ps, ty, T, d, inter, pdac, ph, pdx, pd13, pd2,
        _scratch("dev_status", dev_status, dy.get_device()), _stream(stream)))
