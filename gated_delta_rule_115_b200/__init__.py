"""Python binding of libmuir, the Muir gated delta rule on one NVIDIA B200.

Argument marshalling only (ctypes; a native module for the softmax-attention layer):
every step of the computation runs in the CUDA kernels of ``libmuir.so`` (built in-tree
by ``gated_delta_rule_115_b200.build``) behind the C ABI declared in ``include/muir.h``.  PyTorch supplies device
memory and the current CUDA stream.  There is no CPU fallback: if the library
is missing or a call fails, an exception is raised.

Recurrence (arXiv 2611.08376, wolonglab.org page, "Methodology", eq:gdn2 and
eq:ours), per batch and head, state S in R^{dk x dv} with rows = key channels:

    S_t = diag(exp g_t) S_{t-1} - (e_t*k_t)(k_t^T diag(exp g_t) S_{t-1}) + k_t (w_t*v_t)^T
    o_t = S_t^T (gamma_t * q_t)

Per-token tensors are ``[B, T, H, d]``; states ``[B, H, dk, dv]`` float32.
"""
from __future__ import annotations

import ctypes
import math
import operator
import os

import torch

__all__ = [
    "MuirError", "lib", "chunk_fwd", "chunk_bwd", "chunk_fwd_varlen", "chunk_bwd_varlen",
    "recurrent_step", "qk_prologue", "chunk_fwd_fused", "chunk_bwd_fused", "MuirFusion",
    "qk_prologue_bwd", "rotary", "rotary_frequencies", "attn_fwd", "attn_bwd",
    "attn_fwd_varlen", "attn_bwd_varlen", "MuirRotaryFunction", "MuirAttentionFunction",
    "kv_cache", "kv_append", "attn_step",
    "fwd_workspace_bytes", "bwd_workspace_bytes", "MuirChunkFunction",
    "LIB_PATH",
]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmuir.so")

MUIR_BF16, MUIR_FP32 = 0, 1
_STATUS = {0: "MUIR_OK", 1: "MUIR_ERR_INVALID_ARG", 2: "MUIR_ERR_UNSUPPORTED",
           3: "MUIR_ERR_WORKSPACE", 4: "MUIR_ERR_CUDA", 5: "MUIR_ERR_DEVICE_TIMEOUT"}


class MuirError(RuntimeError):
    def __init__(self, fn: str, code: int):
        self.code = code
        msg = _lib.muir_status_string(code).decode() if _lib is not None else _STATUS.get(code)
        super().__init__(f"{fn} failed: {msg}")


class MuirShape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("T", ctypes.c_int), ("H", ctypes.c_int),
                ("dk", ctypes.c_int), ("dv", ctypes.c_int), ("chunk", ctypes.c_int),
                ("in_dtype", ctypes.c_int), ("out_dtype", ctypes.c_int)]


class MuirGateFamily(ctypes.Structure):
    _fields_ = [("off", ctypes.c_int), ("rank", ctypes.c_int), ("U", ctypes.c_void_p),
                ("bias", ctypes.c_void_p)]


class MuirFusion(ctypes.Structure):
    _fields_ = [("z_out", ctypes.c_void_p), ("qk_raw", ctypes.c_int),
                ("latent", ctypes.c_void_p), ("R", ctypes.c_int), ("fam", MuirGateFamily * 5)]


class MuirFusionGrads(ctypes.Structure):
    _fields_ = [("dlatent", ctypes.c_void_p), ("dU", ctypes.c_void_p * 5),
                ("dbias", ctypes.c_void_p * 5)]


class MuirAttnShape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("Tq", ctypes.c_int), ("Tk", ctypes.c_int),
                ("Hq", ctypes.c_int), ("Hk", ctypes.c_int), ("d", ctypes.c_int),
                ("causal", ctypes.c_int), ("window", ctypes.c_int), ("scale", ctypes.c_float),
                ("q_ld", ctypes.c_longlong), ("k_ld", ctypes.c_longlong),
                ("v_ld", ctypes.c_longlong)]


class MuirKvCache(ctypes.Structure):
    _fields_ = [("Hk", ctypes.c_int), ("d", ctypes.c_int), ("page", ctypes.c_int),
                ("num_pages", ctypes.c_int), ("max_pages", ctypes.c_int),
                ("k_pages", ctypes.c_void_p), ("v_pages", ctypes.c_void_p),
                ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
                ("table", ctypes.c_void_p)]


# gate families of the fused projection, in the latent's column order
GATE_FAMILIES = ("f", "b", "g", "w", "q")


_lib = None


def lib():
    """The loaded ``libmuir.so`` (ctypes).  Raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: run `python -m gated_delta_rule_115_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        P, I, S = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
        SP = ctypes.POINTER(MuirShape)
        L.muir_selftest_expired_wait.argtypes = [I, P]
        L.muir_selftest_expired_wait.restype = I
        L.muir_device_wait_status.argtypes = []
        L.muir_device_wait_status.restype = I
        L.muir_status_string.argtypes = [I]
        L.muir_status_string.restype = ctypes.c_char_p
        L.muir_chunk_aux_floats.argtypes = [SP]
        L.muir_chunk_aux_floats.restype = ctypes.c_size_t
        L.muir_chunk_fwd_workspace.argtypes = [SP]
        L.muir_chunk_fwd_workspace.restype = S
        L.muir_chunk_bwd_workspace.argtypes = [SP]
        L.muir_chunk_bwd_workspace.restype = S
        L.muir_chunk_fwd.argtypes = [SP] + [P] * 14 + [S, P]
        L.muir_chunk_fwd.restype = I
        L.muir_chunk_bwd.argtypes = [SP] + [P] * 22 + [S, P]
        L.muir_chunk_bwd.restype = I
        L.muir_recurrent_step.argtypes = [I, I, I, I, I, I] + [P] * 7 + [I, P, P, P]
        L.muir_recurrent_step.restype = I
        LLP = ctypes.POINTER(ctypes.c_longlong)
        L.muir_chunk_varlen_workspace.argtypes = [SP, I, LLP, I]
        L.muir_chunk_varlen_workspace.restype = S
        L.muir_chunk_fwd_varlen.argtypes = [SP, I, LLP] + [P] * 11 + [S, P]
        L.muir_chunk_fwd_varlen.restype = I
        L.muir_chunk_bwd_varlen.argtypes = [SP, I, LLP] + [P] * 19 + [S, P]
        L.muir_chunk_bwd_varlen.restype = I
        L.muir_qk_prologue.argtypes = [ctypes.c_longlong, I, I, P, P, P]
        L.muir_qk_prologue.restype = I
        L.muir_qk_prologue_bwd.argtypes = [ctypes.c_longlong, I, I, P, P, P, P]
        L.muir_qk_prologue_bwd.restype = I
        FP = ctypes.POINTER(MuirFusion)
        L.muir_chunk_fused_workspace.argtypes = [SP, FP, I]
        L.muir_chunk_fused_workspace.restype = S
        L.muir_chunk_fwd_fused.argtypes = [SP, FP] + [P] * 15 + [S, P]
        L.muir_chunk_fwd_fused.restype = I
        L.muir_chunk_bwd_fused.argtypes = [SP, FP] + [P] * 25 + [S, P]
        L.muir_chunk_bwd_fused.restype = I
        L.muir_chunk_fwd_noalloc.argtypes = [SP] + [P] * 10 + [P]
        L.muir_chunk_fwd_noalloc.restype = I
        LL, F, CP = ctypes.c_longlong, ctypes.c_float, ctypes.POINTER(MuirKvCache)
        L.muir_rotary.argtypes = [I] * 7 + [P, LL, P, LL, P, P, F, I, I, P, LL, P, LL, P]
        L.muir_rotary.restype = I
        AP, LLA = ctypes.POINTER(MuirAttnShape), ctypes.POINTER(ctypes.c_longlong)
        L.muir_attn_fwd.argtypes = [AP] + [P] * 6
        L.muir_attn_fwd.restype = I
        L.muir_attn_bwd_workspace.argtypes = [AP]
        L.muir_attn_bwd_workspace.restype = S
        L.muir_attn_bwd.argtypes = [AP] + [P] * 10 + [S, P]
        L.muir_attn_bwd.restype = I
        L.muir_attn_fwd_varlen.argtypes = [AP, I, LLA, LLA] + [P] * 6
        L.muir_attn_fwd_varlen.restype = I
        L.muir_attn_bwd_varlen.argtypes = [AP, I, LLA, LLA] + [P] * 10 + [S, P]
        L.muir_attn_bwd_varlen.restype = I
        L.muir_kv_append.argtypes = [I, I, I, P, LL, P, LL, CP, P, P, P]
        L.muir_kv_append.restype = I
        L.muir_attn_step_workspace.argtypes = [I, I, CP]
        L.muir_attn_step_workspace.restype = S
        L.muir_attn_step.argtypes = [I, I, CP, P, P, F, I, P, P, S, P]
        L.muir_attn_step.restype = I
        L.muir_profile_enable.argtypes = [I]
        L.muir_profile_enable.restype = None
        L.muir_profile_reset.argtypes = []
        L.muir_profile_reset.restype = None
        L.muir_profile_collect.argtypes = []
        L.muir_profile_collect.restype = I
        L.muir_profile_count.argtypes = []
        L.muir_profile_count.restype = I
        L.muir_profile_name.argtypes = [I]
        L.muir_profile_name.restype = ctypes.c_char_p
        L.muir_profile_total_ms.argtypes = [I]
        L.muir_profile_total_ms.restype = ctypes.c_double
        L.muir_profile_launches.argtypes = [I]
        L.muir_profile_launches.restype = ctypes.c_longlong
        _lib = L
    return _lib


def _dt(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return MUIR_BF16
    if t.dtype == torch.float32:
        return MUIR_FP32
    raise TypeError(f"unsupported dtype {t.dtype} (bfloat16 or float32)")


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("libmuir takes CUDA tensors only")
    if not t.is_contiguous():
        raise ValueError("libmuir takes contiguous tensors")
    return ctypes.c_void_p(t.data_ptr())


def _stream(dev):
    return ctypes.c_void_p(torch.cuda.current_stream(dev).cuda_stream)


def _check(fn, rc):
    if rc != 0:
        raise MuirError(fn, rc)


def _shape(q, v, chunk, out_dtype):
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    od = _dt(q) if out_dtype is None else (MUIR_BF16 if out_dtype == torch.bfloat16 else MUIR_FP32)
    return MuirShape(B, T, H, dk, dv, chunk, _dt(q), od)


def device_wait_status() -> None:
    """Synchronise the device and raise MuirError if a bounded wait inside a
    chunk kernel expired since the previous check (muir_device_wait_status)."""
    _check("muir_device_wait_status", lib().muir_device_wait_status())


def fwd_workspace_bytes(B, T, H, d, chunk, dtype=torch.bfloat16) -> int:
    s = MuirShape(B, T, H, d, d, chunk, MUIR_BF16 if dtype == torch.bfloat16 else MUIR_FP32, 0)
    return int(lib().muir_chunk_fwd_workspace(ctypes.byref(s)))


def bwd_workspace_bytes(B, T, H, d, chunk, dtype=torch.bfloat16) -> int:
    s = MuirShape(B, T, H, d, d, chunk, MUIR_BF16 if dtype == torch.bfloat16 else MUIR_FP32, 0)
    return int(lib().muir_chunk_bwd_workspace(ctypes.byref(s)))


def _workspace(nbytes, dev, ws):
    if nbytes == 0:
        return None
    if ws is not None and ws.numel() >= nbytes:
        return ws
    return torch.empty(nbytes, dtype=torch.uint8, device=dev)


def chunk_fwd(q, k, v, g, e, w, gamma, S0=None, chunk=64, out_dtype=None,
              return_chunk_states=False, return_saved=False, save_aux=False, ws=None):
    """Chunkwise forward.  Returns ``(o, S_final)``; with ``return_chunk_states``
    ``(o, S_final, S_chunks)`` where ``S_chunks[b,h,n]`` is the state at the start
    of chunk ``n``; with ``return_saved`` ``(o, S_final, S_chunks, M_chunks)``
    where ``M_chunks[b,h,n]`` is chunk n's transition, and with ``save_aux`` as
    well a fifth element ``aux``, the per-chunk intermediates
    (``muir_chunk_aux_floats``).  All are reusable by :func:`chunk_bwd`."""
    L = lib()
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    shp = _shape(q, v, chunk, out_dtype)
    od = torch.bfloat16 if shp.out_dtype == MUIR_BF16 else torch.float32
    o = torch.empty(B, T, H, dv, dtype=od, device=q.device)
    S_final = torch.empty(B, H, dk, dv, dtype=torch.float32, device=q.device)
    Sc = (torch.empty(B, H, -(-T // chunk), dk, dv, dtype=torch.float32, device=q.device)
          if (return_chunk_states or return_saved) else None)
    Mc = (torch.empty(B, H, -(-T // chunk), dk, dk, dtype=torch.float32, device=q.device)
          if return_saved else None)
    aux = None
    if return_saved and save_aux:
        aux = torch.empty(int(L.muir_chunk_aux_floats(ctypes.byref(shp))), dtype=torch.float32,
                          device=q.device)
    need = int(L.muir_chunk_fwd_workspace(ctypes.byref(shp)))
    wsb = _workspace(need, q.device, ws)
    rc = L.muir_chunk_fwd(ctypes.byref(shp), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(e),
                          _ptr(w), _ptr(gamma), _ptr(S0), _ptr(o), _ptr(S_final), _ptr(Sc),
                          _ptr(Mc), _ptr(aux), _ptr(wsb),
                          ctypes.c_size_t(0 if wsb is None else wsb.numel()), _stream(q.device))
    _check("muir_chunk_fwd", rc)
    if return_saved:
        return (o, S_final, Sc, Mc, aux) if save_aux else (o, S_final, Sc, Mc)
    return (o, S_final, Sc) if return_chunk_states else (o, S_final)


def chunk_bwd(q, k, v, g, e, w, gamma, S0, dO, dS_final=None, chunk=64, S_chunks=None,
              M_chunks=None, aux=None, ws=None):
    """Gradients of ``sum(o*dO) + sum(S_final*dS_final)``.  Returns a dict with
    ``dq, dk, dv, dg, de, dw, dgamma`` (input dtype) and ``dS0`` (float32).
    ``S_chunks`` / ``M_chunks`` / ``aux`` from :func:`chunk_fwd` skip
    recomputation (``aux`` only together with ``S_chunks``)."""
    L = lib()
    shp = _shape(q, v, chunk, None)
    grads = {n: torch.empty_like(x) for n, x in
             dict(dq=q, dk=k, dv=v, dg=g, de=e, dw=w, dgamma=gamma).items()}
    B, T, H, dk = q.shape
    grads["dS0"] = torch.empty(B, H, dk, v.shape[-1], dtype=torch.float32, device=q.device)
    need = int(L.muir_chunk_bwd_workspace(ctypes.byref(shp)))
    wsb = _workspace(need, q.device, ws)
    rc = L.muir_chunk_bwd(ctypes.byref(shp), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(e),
                          _ptr(w), _ptr(gamma), _ptr(S0), _ptr(S_chunks), _ptr(M_chunks), _ptr(aux),
                          _ptr(dO),
                          _ptr(dS_final), _ptr(grads["dq"]), _ptr(grads["dk"]),
                          _ptr(grads["dv"]), _ptr(grads["dg"]), _ptr(grads["de"]),
                          _ptr(grads["dw"]), _ptr(grads["dgamma"]), _ptr(grads["dS0"]),
                          _ptr(wsb), ctypes.c_size_t(0 if wsb is None else wsb.numel()),
                          _stream(q.device))
    _check("muir_chunk_bwd", rc)
    return grads


def _fusion(z_out, qk_raw, latent=None, proj=None):
    """``proj`` maps a family name (``GATE_FAMILIES``) to ``(offset, U, bias)``:
    U [rank, H*dk] bf16, bias [H*dk] float32."""
    f = MuirFusion()
    f.z_out = None if z_out is None else _ptr(z_out).value
    f.qk_raw = int(bool(qk_raw))
    if latent is not None:
        f.latent = _ptr(latent).value
        f.R = latent.shape[-1]
        for name, (off, U, bias) in (proj or {}).items():
            fam = f.fam[GATE_FAMILIES.index(name)]
            fam.off, fam.rank = int(off), U.shape[0]
            fam.U, fam.bias = _ptr(U).value, _ptr(bias).value
    return f


def chunk_fwd_fused(q, k, v, g, e, w, gamma, S0=None, z_out=None, qk_raw=False, chunk=128,
                    out_dtype=None, save=True, ws=None, latent=None, proj=None):
    """Forward with the fused stages (``muir_chunk_fwd_fused``): ``qk_raw``
    means q and k are the raw pre-activations (SiLU and the unit L2 norm are
    applied in the kernels); ``z_out`` is the output gate's pre-activation
    (the output is ``o * sigmoid(z_out)``); ``latent`` [B, T, R] with ``proj``
    (family -> (offset, U, bias)) projects those families' gates from the
    latent (their tensor arguments may be None).  Returns ``(o, S_final, saved)``;
    ``saved`` (None unless ``save``) holds what :func:`chunk_bwd_fused` reuses:
    ``S_chunks``, ``M_chunks``, ``aux`` and, with a gate, ``o_pre``."""
    L = lib()
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    shp = _shape(q, v, chunk, out_dtype)
    fu = _fusion(z_out, qk_raw, latent, proj)
    od = torch.bfloat16 if shp.out_dtype == MUIR_BF16 else torch.float32
    o = torch.empty(B, T, H, dv, dtype=od, device=q.device)
    gated = z_out is not None or (proj is not None and "g" in proj)
    o_pre = torch.empty_like(o) if gated else None
    S_final = torch.empty(B, H, dk, dv, dtype=torch.float32, device=q.device)
    Sc = Mc = aux = None
    if save:
        n = -(-T // chunk)
        Sc = torch.empty(B, H, n, dk, dv, dtype=torch.float32, device=q.device)
        Mc = torch.empty(B, H, n, dk, dk, dtype=torch.float32, device=q.device)
        aux = torch.empty(int(L.muir_chunk_aux_floats(ctypes.byref(shp))), dtype=torch.float32,
                          device=q.device)
    need = int(L.muir_chunk_fused_workspace(ctypes.byref(shp), ctypes.byref(fu), 0))
    if need == 0:
        raise MuirError("muir_chunk_fused_workspace", 2)
    wsb = _workspace(need, q.device, ws)
    rc = L.muir_chunk_fwd_fused(ctypes.byref(shp), ctypes.byref(fu), _ptr(q), _ptr(k), _ptr(v),
                                _ptr(g), _ptr(e), _ptr(w), _ptr(gamma), _ptr(S0), _ptr(o),
                                _ptr(o_pre), _ptr(S_final), _ptr(Sc), _ptr(Mc), _ptr(aux),
                                _ptr(wsb), ctypes.c_size_t(wsb.numel()), _stream(q.device))
    _check("muir_chunk_fwd_fused", rc)
    saved = dict(S_chunks=Sc, M_chunks=Mc, aux=aux, o_pre=o_pre) if save else None
    return o, S_final, saved


def chunk_bwd_fused(q, k, v, g, e, w, gamma, S0, dO, dS_final=None, z_out=None, qk_raw=False,
                    o_pre=None, saved=None, chunk=128, ws=None, latent=None, proj=None):
    """Gradients through :func:`chunk_fwd_fused` (``muir_chunk_bwd_fused``):
    ``dO`` is the gradient of the (gated) output.  Returns the dict of
    :func:`chunk_bwd` plus ``dz_out`` with a gate; dq and dk are with respect
    to the raw q and k when ``qk_raw``.  ``saved`` from the forward skips
    recomputation; with a gate, ``o_pre`` (or ``saved["o_pre"]``) is required."""
    L = lib()
    shp = _shape(q, v, chunk, None)
    if saved is not None and o_pre is None:
        o_pre = saved.get("o_pre")
    if o_pre is not None:
        shp.out_dtype = MUIR_BF16 if o_pre.dtype == torch.bfloat16 else MUIR_FP32
    fu = _fusion(z_out, qk_raw, latent, proj)
    grads = {n: (torch.empty_like(x) if x is not None else None) for n, x in
             dict(dq=q, dk=k, dv=v, dg=g, de=e, dw=w, dgamma=gamma).items()}
    B, T, H, dk = q.shape
    grads["dS0"] = torch.empty(B, H, dk, v.shape[-1], dtype=torch.float32, device=q.device)
    dz = torch.empty_like(z_out) if z_out is not None else None
    fg = None
    if latent is not None:
        fg = MuirFusionGrads()
        grads["dlatent"] = torch.empty_like(latent)
        fg.dlatent = _ptr(grads["dlatent"]).value
        for name, (off, U, bias) in proj.items():
            i = GATE_FAMILIES.index(name)
            grads["dU_" + name] = torch.empty(U.shape, dtype=torch.float32, device=q.device)
            grads["dbias_" + name] = torch.empty(bias.shape, dtype=torch.float32, device=q.device)
            fg.dU[i] = _ptr(grads["dU_" + name]).value
            fg.dbias[i] = _ptr(grads["dbias_" + name]).value
    Sc, Mc, aux = ((saved["S_chunks"], saved["M_chunks"], saved["aux"]) if saved is not None
                   else (None, None, None))
    need = int(L.muir_chunk_fused_workspace(ctypes.byref(shp), ctypes.byref(fu), 1))
    if need == 0:
        raise MuirError("muir_chunk_fused_workspace", 2)
    wsb = _workspace(need, q.device, ws)
    rc = L.muir_chunk_bwd_fused(ctypes.byref(shp), ctypes.byref(fu), _ptr(q), _ptr(k), _ptr(v),
                                _ptr(g), _ptr(e), _ptr(w), _ptr(gamma), _ptr(S0), _ptr(Sc),
                                _ptr(Mc), _ptr(aux), _ptr(o_pre), _ptr(dO), _ptr(dS_final),
                                *[_ptr(grads[n]) for n in ("dq", "dk", "dv", "dg", "de", "dw",
                                                           "dgamma")],
                                _ptr(dz), _ptr(grads["dS0"]),
                                ctypes.byref(fg) if fg is not None else None, _ptr(wsb),
                                ctypes.c_size_t(wsb.numel()), _stream(q.device))
    _check("muir_chunk_bwd_fused", rc)
    for n in ("dg", "de", "dw", "dgamma"):
        if grads[n] is None:
            del grads[n]
    if dz is not None:
        grads["dz_out"] = dz
    return grads


def recurrent_step(q, k, v, g, e, w, gamma, S, gamma_static=False, out_dtype=None, o=None):
    """One decode token for every (b, h); ``S`` ([B,H,dk,dv] float32) is
    updated in place.  ``gamma`` is ``[B,H,dk]``, ``[H,dk]`` with
    ``gamma_static=True``, or None.  Returns ``o`` ([B,H,dv])."""
    L = lib()
    B, H, dk = q.shape
    dv = v.shape[-1]
    od = q.dtype if out_dtype is None else out_dtype
    if o is None:
        o = torch.empty(B, H, dv, dtype=od, device=q.device)
    rc = L.muir_recurrent_step(B, H, dk, dv, _dt(q), _dt(o), _ptr(q), _ptr(k), _ptr(v),
                               _ptr(g), _ptr(e), _ptr(w), _ptr(gamma), int(bool(gamma_static)),
                               _ptr(S), _ptr(o), _stream(q.device))
    _check("muir_recurrent_step", rc)
    return o


def _cu(cu_seqlens):
    vals = [int(c) for c in (cu_seqlens.tolist() if hasattr(cu_seqlens, "tolist") else cu_seqlens)]
    return len(vals) - 1, (ctypes.c_longlong * len(vals))(*vals)


def chunk_fwd_varlen(q, k, v, g, e, w, gamma, cu_seqlens, S0=None, chunk=64, out_dtype=None,
                     ws=None):
    """Forward over packed sequences: per-token tensors ``[1, T, H, d]`` with
    sequence i at rows ``cu_seqlens[i]:cu_seqlens[i+1]`` (a host list or CPU
    tensor).  ``S0`` is ``[num_seqs, H, dk, dv]`` or None.  Returns
    ``(o, S_final)`` with ``S_final`` of shape ``[num_seqs, H, dk, dv]``."""
    L = lib()
    n, cu = _cu(cu_seqlens)
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    shp = _shape(q, v, chunk, out_dtype)
    od = torch.bfloat16 if shp.out_dtype == MUIR_BF16 else torch.float32
    o = torch.empty(B, T, H, dv, dtype=od, device=q.device)
    S_final = torch.empty(n, H, dk, dv, dtype=torch.float32, device=q.device)
    need = int(L.muir_chunk_varlen_workspace(ctypes.byref(shp), n, cu, 0))
    wsb = _workspace(need, q.device, ws)
    rc = L.muir_chunk_fwd_varlen(ctypes.byref(shp), n, cu, _ptr(q), _ptr(k), _ptr(v), _ptr(g),
                                 _ptr(e), _ptr(w), _ptr(gamma), _ptr(S0), _ptr(o), _ptr(S_final),
                                 _ptr(wsb), ctypes.c_size_t(0 if wsb is None else wsb.numel()),
                                 _stream(q.device))
    _check("muir_chunk_fwd_varlen", rc)
    return o, S_final


def chunk_bwd_varlen(q, k, v, g, e, w, gamma, cu_seqlens, S0, dO, dS_final=None, chunk=64,
                     ws=None):
    """Gradients of ``sum(o*dO) + sum(S_final*dS_final)`` over packed sequences
    (see :func:`chunk_fwd_varlen`); returns the dict of :func:`chunk_bwd` with
    ``dS0`` of shape ``[num_seqs, H, dk, dv]``."""
    L = lib()
    n, cu = _cu(cu_seqlens)
    shp = _shape(q, v, chunk, None)
    grads = {nm: torch.empty_like(x) for nm, x in
             dict(dq=q, dk=k, dv=v, dg=g, de=e, dw=w, dgamma=gamma).items()}
    _, _, H, dk = q.shape
    grads["dS0"] = torch.empty(n, H, dk, v.shape[-1], dtype=torch.float32, device=q.device)
    need = int(L.muir_chunk_varlen_workspace(ctypes.byref(shp), n, cu, 1))
    wsb = _workspace(need, q.device, ws)
    rc = L.muir_chunk_bwd_varlen(ctypes.byref(shp), n, cu, _ptr(q), _ptr(k), _ptr(v), _ptr(g),
                                 _ptr(e), _ptr(w), _ptr(gamma), _ptr(S0), _ptr(dO),
                                 _ptr(dS_final), *[_ptr(grads[nm]) for nm in
                                                   ("dq", "dk", "dv", "dg", "de", "dw", "dgamma")],
                                 _ptr(grads["dS0"]), _ptr(wsb),
                                 ctypes.c_size_t(0 if wsb is None else wsb.numel()),
                                 _stream(q.device))
    _check("muir_chunk_bwd_varlen", rc)
    return grads


def qk_prologue(x, out=None):
    """``SiLU(x) / max(||SiLU(x)||, 1e-12)`` over the last dim (64 or 128) of a
    contiguous bf16/float32 tensor; ``out`` may be ``x`` (in place)."""
    L = lib()
    if out is None:
        out = torch.empty_like(x)
    d = x.shape[-1]
    rc = L.muir_qk_prologue(x.numel() // d, d, _dt(x), _ptr(x), _ptr(out), _stream(x.device))
    _check("muir_qk_prologue", rc)
    return out


def qk_prologue_bwd(x, dy, out=None):
    """Gradient of :func:`qk_prologue` with respect to ``x`` for upstream ``dy``."""
    L = lib()
    if out is None:
        out = torch.empty_like(x)
    d = x.shape[-1]
    rc = L.muir_qk_prologue_bwd(x.numel() // d, d, _dt(x), _ptr(x), _ptr(dy), _ptr(out),
                                _stream(x.device))
    _check("muir_qk_prologue_bwd", rc)
    return out


# ------------------------------------------------------------------ softmax-attention layers


_nat = None


def _native():
    """The native half of this binding (``_attn``, built from ``csrc/torch_binding.cpp``):
    these operators are called once a token and layer, where ctypes marshalling would take
    longer than the kernels."""
    global _nat
    if _nat is None:
        lib()
        try:
            from . import _attn
        except ImportError as e:
            raise ImportError("the native binding is missing or was built for another torch: run "
                              "`python -m gated_delta_rule_115_b200.build`") from e
        _attn.load(LIB_PATH, MuirError)
        _nat = _attn
    return _nat


def rotary_frequencies(rot, base=10000.0, scaling=None, factor=1.0, original_length=2048,
                       beta_fast=32.0, beta_slow=1.0, device="cuda"):
    """``(inv_freq, mscale)`` for :func:`rotary`: radians per position of the ``rot // 2``
    pairs (float64 on ``device``) and the factor on the rotated values.

    ``scaling`` stretches them for contexts ``factor`` times ``original_length``: ``"linear"``
    divides every frequency by ``factor``; ``"ntk"`` raises the base so that the slowest
    pair slows down by ``factor`` and the fastest keeps its speed; ``"yarn"`` (arXiv
    2309.00071) keeps pairs that turn more than ``beta_fast`` times within the original
    length, divides those that turn fewer than ``beta_slow`` times by ``factor``, blends
    between, and scales the values by ``0.1 ln(factor) + 1``."""
    if rot < 2 or rot % 2:
        raise ValueError("rot must be a positive even number")
    if scaling not in (None, "linear", "ntk", "yarn"):
        raise ValueError(f"unknown scaling {scaling!r}")
    if not (base > 1.0 and factor > 0.0):
        raise ValueError("base must exceed 1 and factor 0")
    mscale = 1.0
    if scaling == "ntk" and rot > 2:
        base = base * factor ** (rot / (rot - 2))
    f = base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    if scaling == "linear":
        f = f / factor
    elif scaling == "yarn":
        def pair_with(turns):
            return rot * math.log(original_length / (turns * 2 * math.pi)) / (2 * math.log(base))
        low = max(math.floor(pair_with(beta_fast)), 0)
        high = min(math.ceil(pair_with(beta_slow)), rot - 1)
        ramp = ((torch.arange(rot // 2, dtype=torch.float64) - low) / max(high - low, 0.001)).clamp(0, 1)
        f = f / factor * ramp + f * (1 - ramp)
        mscale = 0.1 * math.log(factor) + 1.0 if factor > 1.0 else 1.0
    return f.to(device), mscale


def rotary(q, k=None, positions=None, inv_freq=None, interleaved=False, mscale=1.0,
           inverse=False, q_out=None, k_out=None):
    """Rotary positions (``muir_rotary``) of ``q [B, T, Hq, d]`` and, in the same launch,
    ``k [B, T, Hk, d]`` (bfloat16 or float32; parts of a packed projection are taken as they
    lie).  ``positions`` is int32 ``[B, T]`` (None: 0 .. T-1), ``inv_freq`` float64
    ``[rot / 2]`` (see :func:`rotary_frequencies`) and fixes the rotated channels.
    ``inverse`` applies the transpose, which maps an output gradient to the input's.
    ``q_out`` / ``k_out`` may be the inputs (in place).  Returns ``(q_out, k_out)``, or
    ``q_out`` alone without ``k``.  Records nothing with autograd, and refuses tensors that
    require a gradient while gradients are enabled: :class:`MuirRotaryFunction` takes those."""
    return (_nat or _native()).rotary(q, k, positions, inv_freq, interleaved, mscale, inverse, q_out, k_out)


def attn_fwd(q, k, v, causal=True, window=0, scale=None):
    """Softmax attention (``muir_attn_fwd``) of bfloat16 ``q [B, Tq, Hq, d]`` over
    ``k, v [B, Tk, Hk, d]`` (parts of a packed projection are taken as they lie).  Query i
    stands at key position ``i + Tk - Tq``; ``causal`` hides later keys, ``window`` all but
    the last ``window``.  ``scale`` defaults to ``d ** -0.5``.  Returns ``(o, lse)`` with
    ``o [B, Tq, Hq, d]`` and float32 ``lse [B, Hq, Tq]``."""
    return (_nat or _native()).attn_fwd(q, k, v, None, None, causal, window, scale)


def attn_bwd(q, k, v, o, lse, dO, causal=True, window=0, scale=None, ws=None):
    """Gradients of ``sum(o * dO)`` (``muir_attn_bwd``) from :func:`attn_fwd`'s ``o`` and
    ``lse``; the probabilities are recomputed.  Returns a dict with ``dq, dk, dv``."""
    return (_nat or _native()).attn_bwd(q, k, v, o, lse, dO, None, None, causal, window, scale, ws)


def _offsets(cu):
    """A copy of host offsets (a list or a tensor), None kept."""
    if cu is None:
        return None
    return tuple(cu.to("cpu", torch.long).tolist() if torch.is_tensor(cu) else map(operator.index, cu))


def _given(cu):
    """The native calls take None for a dense batch: packed rows would run as one sequence."""
    if cu is None:
        raise ValueError("packed sequences need cu_seqlens")
    return cu


def attn_fwd_varlen(q, k, v, cu_seqlens, cu_seqlens_k=None, causal=True, window=0, scale=None):
    """:func:`attn_fwd` over packed sequences: ``q [1, T, Hq, d]``, ``k, v [1, Tk, Hk, d]`` with
    sequence i at rows ``cu_seqlens[i]:cu_seqlens[i+1]`` (a host list or CPU tensor;
    ``cu_seqlens_k`` for the keys where they differ).  ``lse`` is ``[1, Hq, T]``."""
    return (_nat or _native()).attn_fwd(q, k, v, _given(cu_seqlens), cu_seqlens_k, causal, window, scale)


def attn_bwd_varlen(q, k, v, o, lse, dO, cu_seqlens, cu_seqlens_k=None, causal=True, window=0,
                    scale=None, ws=None):
    """Gradients through :func:`attn_fwd_varlen`; returns the dict of :func:`attn_bwd`."""
    return (_nat or _native()).attn_bwd(q, k, v, o, lse, dO, _given(cu_seqlens), cu_seqlens_k, causal,
                                        window, scale, ws)


def kv_cache(num_pages, Hk, page, d, device="cuda"):
    """Fresh cache tensors ``(k_pages, v_pages, k_scale, v_scale)``: float8_e4m3fn codes
    ``[num_pages, Hk, page, d]`` and float32 scales ``[num_pages, Hk]``."""
    z = [torch.zeros(num_pages, Hk, page, d, dtype=torch.uint8, device=device).view(torch.float8_e4m3fn)
         for _ in range(2)]
    return z[0], z[1], *[torch.ones(num_pages, Hk, dtype=torch.float32, device=device) for _ in range(2)]


def kv_append(k, v, k_pages, v_pages, k_scale, v_scale, page_table, start, count=None):
    """Writes the tokens of ``k, v [B, T, Hk, d]`` (bfloat16 or float32) into the cache
    (:func:`kv_cache`), in place (``muir_kv_append``): token t of sequence b to position
    ``start[b] + t`` for t below ``count[b]`` (None: T).  ``page_table`` is int32
    ``[B, max_pages]``, ``start`` and ``count`` int32 ``[B]``, all on the device.  The new
    tokens' entries of the table must not name a page twice."""
    (_nat or _native()).kv_append(k, v, k_pages, v_pages, k_scale, v_scale, page_table, start, count)


def attn_step(q, k_pages, v_pages, k_scale, v_scale, page_table, lens, scale=None, window=0,
              o=None, ws=None):
    """One bfloat16 query token of every sequence, ``q [B, Hq, d]`` (contiguous), attends over
    its first ``lens[b]`` cached tokens, or the last ``window`` of them (``muir_attn_step``).
    ``scale`` defaults to ``d ** -0.5``.  Work is split by the width of ``page_table``: one
    much wider than the longest sequence costs time.  Returns ``o [B, Hq, d]``."""
    return (_nat or _native()).attn_step(q, k_pages, v_pages, k_scale, v_scale, page_table, lens, scale,
                                         window, o, ws)


class _Once(torch.autograd.Function):
    """``apply(n, *tensors)``: the first n, gradients without a derivative of their own, as results
    of the others, which they were formed from.  Differentiating them again raises, where it
    would leave that part out (with ``once_differentiable`` it still would, wherever the
    incoming gradient is a constant: that looks at the arguments, not at what was saved)."""

    @staticmethod
    def forward(ctx, n, *tensors):
        return tuple(None if t is None else t.view_as(t) for t in tensors[:n])

    @staticmethod
    def backward(ctx, *grads):
        raise RuntimeError("this backward pass is a kernel without a derivative: its gradients cannot be "
                           "differentiated again")


class MuirChunkFunction(torch.autograd.Function):
    """Autograd wrapper: forward saves the chunk states, backward reuses them."""

    @staticmethod
    def forward(ctx, q, k, v, g, e, w, gamma, S0, chunk):
        o, S_final, Sc, Mc, aux = chunk_fwd(q, k, v, g, e, w, gamma, S0, chunk=chunk,
                                            return_saved=True, save_aux=True)
        ctx.save_for_backward(q, k, v, g, e, w, gamma, S0, Sc, Mc, aux)
        ctx.chunk = chunk
        return o, S_final

    @staticmethod
    def backward(ctx, dO, dS_final):
        q, k, v, g, e, w, gamma, S0, Sc, Mc, aux = ctx.saved_tensors
        gr = chunk_bwd(q, k, v, g, e, w, gamma, S0, dO.contiguous().to(q.dtype),
                       None if dS_final is None else dS_final.contiguous().float(),
                       chunk=ctx.chunk, S_chunks=Sc, M_chunks=Mc, aux=aux)
        out = (gr["dq"], gr["dk"], gr["dv"], gr["dg"], gr["de"], gr["dw"], gr["dgamma"],
               gr["dS0"] if S0 is not None else None)
        if torch.is_grad_enabled():  # create_graph
            out = _Once.apply(len(out), *out, q, k, v, g, e, w, gamma, S0, dO, dS_final)
        return *out, None


class MuirRotaryFunction(torch.autograd.Function):
    """Autograd wrapper of :func:`rotary`: ``apply(q, k, positions, inv_freq, interleaved,
    mscale, inverse, inplace)`` returns what it does.  The map is linear: its gradient is the
    call with ``inverse`` turned over, and differentiable in its turn.

    ``inplace`` writes over ``q`` and ``k``.  Autograd takes neither leaves for that, nor views
    in a call that returns two tensors: parts of one projection, as slices of it, are rotated in
    a call each.  (Pieces from ``split`` or ``unbind`` it refuses too, once they are written.)"""

    @staticmethod
    def forward(ctx, q, k=None, positions=None, inv_freq=None, interleaved=False, mscale=1.0, inverse=False,
                inplace=False):
        ctx.set_materialize_grads(False)
        ctx.args = (interleaved, mscale, not inverse)
        ctx.save_for_backward(positions, inv_freq)
        if not inplace:
            return rotary(q, k, positions, inv_freq, interleaved, mscale, inverse)
        both = (q,) if k is None else (q, k)
        if any(ctx.needs_input_grad[:2]):  # autograd would refuse these after they are written
            if any(t.is_leaf and t.requires_grad for t in both):
                raise ValueError("a leaf that requires a gradient cannot be rotated in place")
            if len(both) > 1 and any(t._is_view() for t in both):
                raise ValueError("views of a larger tensor are rotated in place in a call each")
        ctx.mark_dirty(*both)
        rotary(q, k, positions, inv_freq, interleaved, mscale, inverse, q_out=q, k_out=k)
        return q if k is None else both

    @staticmethod
    def backward(ctx, *grads):
        rest = *ctx.saved_tensors, *ctx.args
        had = [g.contiguous() for g in grads if g is not None]
        if len(had) == 2:
            d = MuirRotaryFunction.apply(*had, *rest)
        else:
            one = MuirRotaryFunction.apply(had[0], None, *rest) if had else None
            d = [None if g is None else one for g in (*grads, None)[:2]]
        return (*d, None, None, None, None, None, None)


class MuirAttentionFunction(torch.autograd.Function):
    """Autograd wrapper of :func:`attn_fwd` / :func:`attn_bwd`, or of the varlen forms with
    ``cu_seqlens``, which is copied: its owner may refill it before the backward pass.
    Returns ``o``."""

    @staticmethod
    def forward(ctx, q, k, v, causal=True, window=0, scale=None, cu_seqlens=None, cu_seqlens_k=None):
        ctx.args = dict(causal=causal, window=window, scale=scale)
        ctx.cu = (None if cu_seqlens is None and cu_seqlens_k is None
                  else dict(cu_seqlens=_offsets(cu_seqlens), cu_seqlens_k=_offsets(cu_seqlens_k)))
        o, lse = (attn_fwd(q, k, v, **ctx.args) if ctx.cu is None
                  else attn_fwd_varlen(q, k, v, **ctx.cu, **ctx.args))
        ctx.save_for_backward(q, k, v, o, lse)
        return o

    @staticmethod
    def backward(ctx, dO):
        saved = ctx.saved_tensors
        dO = dO.contiguous().to(torch.bfloat16)
        g = (attn_bwd(*saved, dO, **ctx.args) if ctx.cu is None
             else attn_bwd_varlen(*saved, dO, **ctx.cu, **ctx.args))
        out = g["dq"], g["dk"], g["dv"]
        if torch.is_grad_enabled():  # create_graph
            out = _Once.apply(len(out), *out, *saved[:3], dO)
        return *out, None, None, None, None, None
