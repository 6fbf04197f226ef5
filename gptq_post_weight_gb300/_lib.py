"""ctypes binding of libgptqfold.so (include/gptq_fold.h).

Argument marshalling only: every step runs in the library's CUDA kernels.
The wrappers take torch CUDA tensors (device memory and the current stream
come from PyTorch) and raise ``GptqError`` on a non-zero status.  There is
no fallback: without the built library every call fails loudly.
"""
from __future__ import annotations

import ctypes
import math
import os
import threading

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libgptqfold.so")

STATUS = {0: "GPTQ_OK", 1: "GPTQ_ERR_ARG", 2: "GPTQ_ERR_SHAPE", 3: "GPTQ_ERR_NOMEM",
          4: "GPTQ_ERR_NOT_SPD", 5: "GPTQ_ERR_CUDA", 6: "GPTQ_ERR_TIMEOUT"}

# name -> (restype, argtypes); the full exported surface of the header.
_P, _I, _D, _S = ctypes.c_void_p, ctypes.c_int, ctypes.c_double, ctypes.c_size_t
_L, _F = ctypes.c_longlong, ctypes.c_float
SIGNATURES = {
    "gptq_status_string": (ctypes.c_char_p, [_I]),
    "gptq_fold_workspace_bytes": (_S, [_I]),
    "gptq_fold": (_I, [_P, _I, _D, _P, _P, _P, _P, _P, _S, _P]),
    "gptq_ladder": (_I, [_P, _I, _I, _P, _P, _P]),
    "gptq_sweep_workspace_bytes": (_S, [_I, _I]),
    "gptq_q4tp_sweep": (_I, [_P, _I, _I, _P, _P, _P, _P, _P, _P, _P, _P, _S, _P]),
    "gptq_q4tp_group": (_I, [_P, _I, _P, _P, _P, _P, _P, _P, _P, _P, _P]),
    "gptq_q4tp_sweep_noalloc": (_I, [_P, _I, _I, _P, _P, _P, _P, _P, _P, _P, _P]),
    "gptq_group_workspace_bytes": (_S, [_I, _I]),
    "gptq_quantize_group": (_I, [_P, _I, _D, _P, _I, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _S, _P]),
    "gptq_build_equilibrated": (_I, [_P, _I, _D, _P, _P, _P, _S, _P]),
    "gptq_act_order_perm": (_I, [_P, _I, _P, _P]),
    "gptq_fold_permuted": (_I, [_P, _I, _D, _P, _P, _P, _P, _P, _P, _S, _P]),
    "gptq_static_rungs": (_I, [_P, _I, _I, _P, _P, _P, _P, _P]),
    "gptq_sweep_act_order_workspace_bytes": (_S, [_I, _I]),
    "gptq_q4tp_sweep_act_order": (_I, [_P, _I, _I, _P, _P, _P, _P, _P, _P, _S, _P]),
    "gptq_group_act_order_workspace_bytes": (_S, [_I, _I]),
    "gptq_quantize_group_act_order": (_I, [_P, _I, _D, _P, _I, _P, _P, _P, _P, _P, _P, _P, _S, _P]),
    "gptq_q2tp_place": (_I, [_P, _I, _I, _P, _P, _P, _P, _P]),
    "gptq_q2tp_group": (_I, [_P, _I, _P, _P, _P, _P, _P, _P, _P, _P]),
    "gptq_q2tp_sweep": (_I, [_P, _I, _I, _P, _P, _P, _P, _P, _P, _P, _S, _P]),
    "gptq_quantize_group_q2tp": (_I, [_P, _I, _D, _P, _I, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _S, _P]),
    "gptq_debias_workspace_bytes": (_S, [_I, _I]),
    "gptq_debias": (_I, [_I, _P, _I, _I, _P, _P, _P, _P, _P, _P, _P, _P, _S, _P]),
    "gptq_gram_workspace_bytes": (_S, [_I]),
    "gptq_gram_add": (_I, [_P, _I, _P, _I, _P, _S, _P]),
    "gptq_q4tp_linear": (_I, [_I, _P, _L, _I, _P, _P, _P, _I, _I, _P, _I, _P, _L, _P, _L, _P, _P]),
    "gptq_q4tp_gated_workspace_bytes": (_S, [_I, _I, _I]),
    "gptq_q4tp_gated": (_I, [_I, _P, _L, _I, _P, _P, _P, _I, _I, _P, _I, _P, _L, _P, _S, _P, _P]),
    "gptq_kv4_write": (_I, [_I, _P, _L, _I, _I, _I, _P, _P, _L, _L, _L, _L, _P, _I, _P]),
    "gptq_rotary": (_I, [_I, _P, _L, _L, _I, _I, _I, _I, _I, _P, _P, _F, _P, _L, _L, _P]),
    "gptq_kv4_write_rotary": (_I, [_I, _P, _L, _I, _I, _I, _P, _L, _L, _I, _P, _P, _L, _L, _L, _L, _P, _I, _I, _I, _P, _P,
                                   _F, _P, _L, _L, _P]),
    "gptq_kv4_read": (_I, [_I, _P, _L, _I, _I, _I, _P, _I, _P, _P, _P]),
    "gptq_kv4_attention_workspace_bytes": (_S, [_I, _I, _I]),
    "gptq_kv4_attention_call_bytes": (_S, [_I, _I, _I, _I, _I, _I, _L]),
    "gptq_kv4_attention_lse": (_I, [_I, _P, _L, _L, _I, _P, _L, _I, _I, _I, _I, _P, _I, _P, _P, _I, _I, _F, _P, _P, _P,
                                    _S, _P, _P]),
    "gptq_kv4_attention_weights_workspace_bytes": (_S, [_I, _I, _I, _I, _I, _L]),
    "gptq_kv4_attention_weights": (_I, [_I, _P, _L, _L, _I, _P, _P, _L, _I, _I, _I, _I, _P, _I, _P, _P, _I, _I, _F, _P,
                                        _P, _S, _P, _P]),
    "gptq_kv4_evict": (_I, [_P, _L, _I, _I, _I, _P, _I, _P, _I, _P, _I, _P, _I, _I, _P, _P, _P, _P]),
    "gptq_kv4_attention": (_I, [_I, _P, _L, _L, _I, _P, _L, _I, _I, _I, _I, _P, _I, _P, _P, _I, _I, _F, _P, _P,
                                _S, _P, _P]),
    "gptq_launch_count": (ctypes.c_longlong, []),
    "gptq_kernel_kinds": (_I, []),
    "gptq_kernel_kind_name": (ctypes.c_char_p, [_I]),
    "gptq_profile_select": (None, [ctypes.c_uint]),
    "gptq_profile_start": (_I, [_I]),
    "gptq_profile_stop": (_I, [_P, _P, _I]),
    "gptq_test_set_wait": (_I, [ctypes.c_ulonglong, _I]),
}


class GptqError(RuntimeError):
    def __init__(self, fn, code):
        self.code = code
        super().__init__(f"{fn}: {STATUS.get(code, code)}")


_lib = None


def load(path: str = LIB_PATH):
    """Load the library (built by ``gptq_post_weight_gb300.build``)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with `python -m gptq_post_weight_gb300.build`")
    lib = ctypes.CDLL(path)
    for name, (res, args) in SIGNATURES.items():
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args
    _lib = lib
    return lib


def _ptr(t):
    """Device address of a CUDA tensor (None -> NULL).  Taken when the
    library call's arguments are built, after every size check."""
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"tensor arguments must be CUDA tensors, got one on {t.device}")
    return ctypes.c_void_p(t.data_ptr())


def _stream(torch, stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _check(fn, code):
    if code != 0:
        raise GptqError(fn, code)


def _need(t, name, dtype=None, numel=None, device=None):
    """Raise ValueError unless ``t`` is a contiguous tensor of ``dtype``
    (default float32) with ``numel`` elements on ``device``.  The kernels
    index every buffer by the sizes the call states, so a buffer of another
    size is refused here, before anything is launched (that it lives on the
    GPU is checked by ``_ptr``)."""
    import torch

    dtype = torch.float32 if dtype is None else dtype
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a torch tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if numel is not None and t.numel() != numel:
        raise ValueError(f"{name} must have {numel} elements, got {t.numel()} (shape {tuple(t.shape)})")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, the call's data on {device}")


def _matrix(w, name="w", n=None):
    """rows, n of a 2-D float32 matrix (n checked when given)."""
    _need(w, name)
    if w.dim() != 2:
        raise ValueError(f"{name} must be 2-D [rows, n], got shape {tuple(w.shape)}")
    if n is not None and w.shape[1] != n:
        raise ValueError(f"{name} has {w.shape[1]} columns, n = {n}")
    return w.shape[0], w.shape[1]


def _packed(h_packed, n, device=None):
    _need(h_packed, "h_packed", numel=n * (n + 1) // 2 if n > 0 else None, device=device)


def _ws(ws, device):
    import torch

    _need(ws, "ws", dtype=torch.uint8, device=device)


def _check_outs(out, names, sizes, dtypes, device):
    if len(out) != len(names):
        raise ValueError(f"out must hold {len(names)} tensors ({', '.join(names)})")
    for t, nm, k, dt in zip(out, names, sizes, dtypes):
        _need(t, nm, dtype=dt, numel=k, device=device)


def workspace(nbytes: int, device):
    import torch

    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)


def fold(h_packed, n: int, lam: float = 0.01, ws=None, stream=None, want_d=True):
    """U [n, n], D [n], hdiag [n], lambda_used.  Raises GptqError(NOT_SPD)."""
    import torch

    lib = load()
    _packed(h_packed, n)
    dev = h_packed.device
    u = torch.empty(n, n, dtype=torch.float32, device=dev)
    d = torch.empty(n, dtype=torch.float32, device=dev) if want_d else None
    hd = torch.empty(n, dtype=torch.float32, device=dev)
    need = lib.gptq_fold_workspace_bytes(n)
    if ws is None:
        ws = workspace(need, dev)
    _ws(ws, dev)
    lam_used = ctypes.c_double(0.0)
    code = lib.gptq_fold(_ptr(h_packed), n, float(lam), _ptr(u), _ptr(d), _ptr(hd),
                         ctypes.byref(lam_used), _ptr(ws), ws.numel(), _stream(torch, stream))
    _check("gptq_fold", code)
    return u, d, hd, lam_used.value


def build_equilibrated(h_packed, n: int, lam: float = 0.01):
    import torch

    lib = load()
    _packed(h_packed, n)
    dev = h_packed.device
    a = torch.zeros(n, n, dtype=torch.float32, device=dev)
    d = torch.empty(n, dtype=torch.float32, device=dev)
    ws = workspace(lib.gptq_fold_workspace_bytes(n), dev)
    code = lib.gptq_build_equilibrated(_ptr(h_packed), n, float(lam), _ptr(a), _ptr(d), _ptr(ws),
                                       ws.numel(), _stream(torch))
    _check("gptq_build_equilibrated", code)
    return a, d


def ladder(w):
    import torch

    lib = load()
    rows, n = _matrix(w)
    tab = torch.empty(rows, 32, dtype=torch.float32, device=w.device)
    lost = torch.empty(rows, 2, dtype=torch.float32, device=w.device)
    _check("gptq_ladder", lib.gptq_ladder(_ptr(w), rows, n, _ptr(tab), _ptr(lost), _stream(torch)))
    return tab, lost


def _outs(torch, rows, n, dev, out=None):
    gpr = n // 32
    if out is not None:
        _check_outs(out, ("nibbles", "rungs", "scales"), (rows * n // 2, rows * gpr, rows * gpr),
                    (torch.uint8, torch.uint8, torch.float32), dev)
        return out
    nib = torch.empty(rows * n // 2, dtype=torch.uint8, device=dev)
    rungs = torch.empty(rows * gpr, dtype=torch.uint8, device=dev)
    scales = torch.empty(rows * gpr, dtype=torch.float32, device=dev)
    return nib, rungs, scales


def _sweep_inputs(w, u, hw, tab, lost=None):
    """rows, n after checking W [rows, n], U n*n, hw n, tab rows*32, lost rows*2."""
    rows, n = _matrix(w)
    dev = w.device
    _need(u, "u", numel=n * n, device=dev)
    _need(hw, "hw", numel=n, device=dev)
    _need(tab, "tab", numel=rows * 32, device=dev)
    if lost is not None:
        _need(lost, "lost", numel=rows * 2, device=dev)
    return rows, n


def q4tp_sweep(w, u, hw, tab, lost, ws=None, out=None, stream=None):
    """Sweep W (consumed in place).  Returns (nibbles, rungs, scales)."""
    import torch

    lib = load()
    rows, n = _sweep_inputs(w, u, hw, tab, lost)
    nib, rungs, scales = _outs(torch, rows, n, w.device, out)
    if ws is None:
        ws = workspace(lib.gptq_sweep_workspace_bytes(rows, n), w.device)
    _ws(ws, w.device)
    code = lib.gptq_q4tp_sweep(_ptr(w), rows, n, _ptr(u), _ptr(hw), _ptr(tab), _ptr(lost),
                               _ptr(nib), _ptr(rungs), _ptr(scales), _ptr(ws), ws.numel(),
                               _stream(torch, stream))
    _check("gptq_q4tp_sweep", code)
    return nib, rungs, scales


def q4tp_sweep_noalloc(w, u, hw, tab, lost, out=None, stream=None):
    """gptq_q4tp_sweep_noalloc: the sweep with the library's own static
    scratch instead of a workspace (for callers that cannot allocate device
    memory).  Returns (nibbles, rungs, scales); W is consumed in place."""
    import torch

    lib = load()
    rows, n = _sweep_inputs(w, u, hw, tab, lost)
    nib, rungs, scales = _outs(torch, rows, n, w.device, out)
    code = lib.gptq_q4tp_sweep_noalloc(_ptr(w), rows, n, _ptr(u), _ptr(hw), _ptr(tab), _ptr(lost),
                                       _ptr(nib), _ptr(rungs), _ptr(scales), _stream(torch, stream))
    _check("gptq_q4tp_sweep_noalloc", code)
    return nib, rungs, scales


def _group_inputs(tile, ublk, hw, tab, lost=None):
    """rows after checking tile [rows, 32], ublk 32*32, hw 32, tab rows*32, lost rows*2."""
    rows, c = _matrix(tile, "tile")
    if c != 32:
        raise ValueError(f"tile must be [rows, 32], got shape {tuple(tile.shape)}")
    dev = tile.device
    _need(ublk, "ublk", numel=32 * 32, device=dev)
    _need(hw, "hw", numel=32, device=dev)
    _need(tab, "tab", numel=rows * 32, device=dev)
    if lost is not None:
        _need(lost, "lost", numel=rows * 2, device=dev)
    return rows


def q4tp_group(tile, ublk, hw, tab, lost):
    """The group rule on given tiles: (nibbles [rows,16], rungs, scales, E)."""
    import torch

    lib = load()
    rows = _group_inputs(tile, ublk, hw, tab, lost)
    dev = tile.device
    nib = torch.empty(rows, 16, dtype=torch.uint8, device=dev)
    rungs = torch.empty(rows, dtype=torch.uint8, device=dev)
    scales = torch.empty(rows, dtype=torch.float32, device=dev)
    e = torch.empty(rows, 32, dtype=torch.float32, device=dev)
    code = lib.gptq_q4tp_group(_ptr(tile), rows, _ptr(ublk), _ptr(hw), _ptr(tab), _ptr(lost),
                               _ptr(nib), _ptr(rungs), _ptr(scales), _ptr(e), _stream(torch))
    _check("gptq_q4tp_group", code)
    return nib, rungs, scales, e


def quantize_group(h_packed, n, w, lam=0.01, ws=None, want_u=True, stream=None, out=None, want_aux=True):
    """Fold + ladder + sweep.  Returns dict(nibbles, rungs, scales, tab, lost,
    u, d, hdiag, lam); with want_aux=False, tab, lost, d and hdiag stay in the
    workspace (None here), so that repeated calls on the same buffers pass the
    library the same arguments (its graph replay keys on them)."""
    import torch

    lib = load()
    rows, _ = _matrix(w, n=n)
    dev = w.device
    _packed(h_packed, n, dev)
    nib, rungs, scales = _outs(torch, rows, n, dev, out)
    tab = torch.empty(rows, 32, dtype=torch.float32, device=dev) if want_aux else None
    lost = torch.empty(rows, 2, dtype=torch.float32, device=dev) if want_aux else None
    u = torch.empty(n, n, dtype=torch.float32, device=dev) if want_u else None
    d = torch.empty(n, dtype=torch.float32, device=dev) if want_aux else None
    hd = torch.empty(n, dtype=torch.float32, device=dev) if want_aux else None
    if ws is None:
        ws = workspace(lib.gptq_group_workspace_bytes(rows, n), dev)
    _ws(ws, dev)
    lam_used = ctypes.c_double(0.0)
    code = lib.gptq_quantize_group(_ptr(h_packed), n, float(lam), _ptr(w), rows, _ptr(nib),
                                   _ptr(rungs), _ptr(scales), _ptr(tab), _ptr(lost), _ptr(u),
                                   _ptr(d), _ptr(hd), ctypes.byref(lam_used), _ptr(ws), ws.numel(),
                                   _stream(torch, stream))
    _check("gptq_quantize_group", code)
    return dict(nibbles=nib, rungs=rungs, scales=scales, tab=tab, lost=lost, u=u, d=d, hdiag=hd,
                lam=lam_used.value)


def test_set_wait(wait_ns: int = 0, no_loads: bool = False):
    """gptq_test_set_wait: the device-wait limit in ns (0 = the default 2 s)
    and the test hook that makes the GEMM producers issue no loads."""
    _check("gptq_test_set_wait", load().gptq_test_set_wait(int(wait_ns), 1 if no_loads else 0))


def launch_count() -> int:
    return int(load().gptq_launch_count())


def profile_start(max_launches: int = 100000, kinds=None):
    """Record events for the launches that follow; `kinds`: names to record
    (default all)."""
    lib = load()
    mask = 0xFFFFFFFF
    if kinds is not None:
        names = [lib.gptq_kernel_kind_name(k).decode() for k in range(lib.gptq_kernel_kinds())]
        mask = 0
        for name in kinds:
            mask |= 1 << names.index(name)
    lib.gptq_profile_select(mask)
    _check("gptq_profile_start", lib.gptq_profile_start(int(max_launches)))


def profile_stop():
    """{kind name: (total ms, launches)} for the launches since profile_start."""
    lib = load()
    nk = lib.gptq_kernel_kinds()
    ms = (ctypes.c_double * nk)()
    cnt = (ctypes.c_longlong * nk)()
    r = lib.gptq_profile_stop(ms, cnt, nk)
    if r == -1:
        raise GptqError("gptq_profile_stop", 5)
    out = {lib.gptq_kernel_kind_name(k).decode(): (ms[k], cnt[k]) for k in range(nk)}
    if r == -2:
        out["_truncated"] = (0.0, 1)
    return out


def gram_add(h_packed, x, ws=None, stream=None):
    """H_packed += X^T X in place (X [T, n] f32); returns h_packed."""
    import torch

    lib = load()
    t, n = _matrix(x, "x")
    _packed(h_packed, n, x.device)
    if ws is None:
        ws = workspace(lib.gptq_gram_workspace_bytes(n), x.device)
    _ws(ws, x.device)
    code = lib.gptq_gram_add(_ptr(h_packed), n, _ptr(x), t, _ptr(ws), ws.numel(), _stream(torch, stream))
    _check("gptq_gram_add", code)
    return h_packed


def act_order_perm(hdiag):
    import torch

    lib = load()
    _need(hdiag, "hdiag")
    n = hdiag.numel()
    perm = torch.empty(n, dtype=torch.int32, device=hdiag.device)
    _check("gptq_act_order_perm", lib.gptq_act_order_perm(_ptr(hdiag), n, _ptr(perm), _stream(torch)))
    return perm


def fold_permuted(h_packed, n, perm, lam=0.01):
    """U, D, hdiag (permuted order), lambda_used of H[perm][perm]."""
    import torch

    lib = load()
    _packed(h_packed, n)
    dev = h_packed.device
    _need(perm, "perm", dtype=torch.int32, numel=n, device=dev)
    u = torch.empty(n, n, dtype=torch.float32, device=dev)
    d = torch.empty(n, dtype=torch.float32, device=dev)
    hd = torch.empty(n, dtype=torch.float32, device=dev)
    ws = workspace(lib.gptq_fold_workspace_bytes(n), dev)
    lam_used = ctypes.c_double(0.0)
    code = lib.gptq_fold_permuted(_ptr(h_packed), n, float(lam), _ptr(perm), _ptr(u), _ptr(d), _ptr(hd),
                                  ctypes.byref(lam_used), _ptr(ws), ws.numel(), _stream(torch))
    _check("gptq_fold_permuted", code)
    return u, d, hd, lam_used.value


def static_rungs(w, tab, lost):
    import torch

    lib = load()
    rows, n = _matrix(w)
    _need(tab, "tab", numel=rows * 32, device=w.device)
    _need(lost, "lost", numel=rows * 2, device=w.device)
    rungs = torch.empty(rows * (n // 32), dtype=torch.uint8, device=w.device)
    scales = torch.empty(rows * (n // 32), dtype=torch.float32, device=w.device)
    code = lib.gptq_static_rungs(_ptr(w), rows, n, _ptr(tab), _ptr(lost), _ptr(rungs), _ptr(scales),
                                 _stream(torch))
    _check("gptq_static_rungs", code)
    return rungs, scales


def q4tp_sweep_act_order(w, u, perm, tab, rungs):
    import torch

    lib = load()
    rows, n = _matrix(w)
    dev = w.device
    _need(u, "u", numel=n * n, device=dev)
    _need(perm, "perm", dtype=torch.int32, numel=n, device=dev)
    _need(tab, "tab", numel=rows * 32, device=dev)
    _need(rungs, "rungs", dtype=torch.uint8, numel=rows * (n // 32), device=dev)
    nib = torch.empty(rows * n // 2, dtype=torch.uint8, device=w.device)
    ws = workspace(lib.gptq_sweep_act_order_workspace_bytes(rows, n), w.device)
    code = lib.gptq_q4tp_sweep_act_order(_ptr(w), rows, n, _ptr(u), _ptr(perm), _ptr(tab), _ptr(rungs),
                                         _ptr(nib), _ptr(ws), ws.numel(), _stream(torch))
    _check("gptq_q4tp_sweep_act_order", code)
    return nib


def quantize_group_act_order(h_packed, n, w, lam=0.01, ws=None, want_u=True, stream=None):
    import torch

    lib = load()
    rows, _ = _matrix(w, n=n)
    dev = w.device
    _packed(h_packed, n, dev)
    nib, rungs, scales = _outs(torch, rows, n, dev)
    perm = torch.empty(n, dtype=torch.int32, device=dev)
    u = torch.empty(n, n, dtype=torch.float32, device=dev) if want_u else None
    if ws is None:
        ws = workspace(lib.gptq_group_act_order_workspace_bytes(rows, n), dev)
    _ws(ws, dev)
    lam_used = ctypes.c_double(0.0)
    code = lib.gptq_quantize_group_act_order(_ptr(h_packed), n, float(lam), _ptr(w), rows, _ptr(nib),
                                             _ptr(rungs), _ptr(scales), _ptr(perm), _ptr(u),
                                             ctypes.byref(lam_used), _ptr(ws), ws.numel(),
                                             _stream(torch, stream))
    _check("gptq_quantize_group_act_order", code)
    return dict(nibbles=nib, rungs=rungs, scales=scales, perm=perm, u=u, lam=lam_used.value)


# ------------------------------------------------------------------ q2tp


def q2tp_place(w, hw, want_gscale=False):
    """Placed q2tp ladder of the (dead-zeroed) W: (tab [rows, 32], lost
    [rows, 2], gscale [rows, n/32] or None)."""
    import torch

    lib = load()
    rows, n = _matrix(w)
    _need(hw, "hw", numel=n, device=w.device)
    tab = torch.empty(rows, 32, dtype=torch.float32, device=w.device)
    lost = torch.empty(rows, 2, dtype=torch.float32, device=w.device)
    gs = torch.empty(rows, n // 32, dtype=torch.float32, device=w.device) if want_gscale else None
    _check("gptq_q2tp_place", lib.gptq_q2tp_place(_ptr(w), rows, n, _ptr(hw), _ptr(tab), _ptr(lost),
                                                  _ptr(gs), _stream(torch)))
    return tab, lost, gs


def q2tp_group(tile, ublk, hw, tab):
    """The q2tp group rule on given tiles: (codes [rows, 8] u8, rungs, scales, E)."""
    import torch

    lib = load()
    rows = _group_inputs(tile, ublk, hw, tab)
    dev = tile.device
    codes = torch.empty(rows, 8, dtype=torch.uint8, device=dev)
    rungs = torch.empty(rows, dtype=torch.uint8, device=dev)
    scales = torch.empty(rows, dtype=torch.float32, device=dev)
    e = torch.empty(rows, 32, dtype=torch.float32, device=dev)
    code = lib.gptq_q2tp_group(_ptr(tile), rows, _ptr(ublk), _ptr(hw), _ptr(tab), _ptr(codes),
                               _ptr(rungs), _ptr(scales), _ptr(e), _stream(torch))
    _check("gptq_q2tp_group", code)
    return codes, rungs, scales, e


def _outs_q2(torch, rows, n, dev, out=None):
    gpr = n // 32
    if out is not None:
        _check_outs(out, ("codes", "rungs", "scales"), (rows * n // 4, rows * gpr, rows * gpr),
                    (torch.uint8, torch.uint8, torch.float32), dev)
        return out
    codes = torch.empty(rows * n // 4, dtype=torch.uint8, device=dev)
    rungs = torch.empty(rows * gpr, dtype=torch.uint8, device=dev)
    scales = torch.empty(rows * gpr, dtype=torch.float32, device=dev)
    return codes, rungs, scales


def q2tp_sweep(w, u, hw, tab, ws=None, out=None, stream=None):
    """q2tp sweep of W (consumed in place).  Returns (codes, rungs, scales)."""
    import torch

    lib = load()
    rows, n = _sweep_inputs(w, u, hw, tab)
    codes, rungs, scales = _outs_q2(torch, rows, n, w.device, out)
    if ws is None:
        ws = workspace(lib.gptq_sweep_workspace_bytes(rows, n), w.device)
    _ws(ws, w.device)
    code = lib.gptq_q2tp_sweep(_ptr(w), rows, n, _ptr(u), _ptr(hw), _ptr(tab), _ptr(codes),
                               _ptr(rungs), _ptr(scales), _ptr(ws), ws.numel(), _stream(torch, stream))
    _check("gptq_q2tp_sweep", code)
    return codes, rungs, scales


def quantize_group_q2tp(h_packed, n, w, lam=0.01, ws=None, want_u=True, stream=None, out=None,
                        want_aux=True):
    """Fold + placed ladder + q2tp sweep.  Returns dict(codes, rungs, scales,
    tab, lost, u, d, hdiag, lam); want_aux as for quantize_group."""
    import torch

    lib = load()
    rows, _ = _matrix(w, n=n)
    dev = w.device
    _packed(h_packed, n, dev)
    codes, rungs, scales = _outs_q2(torch, rows, n, dev, out)
    tab = torch.empty(rows, 32, dtype=torch.float32, device=dev) if want_aux else None
    lost = torch.empty(rows, 2, dtype=torch.float32, device=dev) if want_aux else None
    u = torch.empty(n, n, dtype=torch.float32, device=dev) if want_u else None
    d = torch.empty(n, dtype=torch.float32, device=dev) if want_aux else None
    hd = torch.empty(n, dtype=torch.float32, device=dev) if want_aux else None
    if ws is None:
        ws = workspace(lib.gptq_group_workspace_bytes(rows, n), dev)
    _ws(ws, dev)
    lam_used = ctypes.c_double(0.0)
    code = lib.gptq_quantize_group_q2tp(_ptr(h_packed), n, float(lam), _ptr(w), rows, _ptr(codes),
                                        _ptr(rungs), _ptr(scales), _ptr(tab), _ptr(lost), _ptr(u),
                                        _ptr(d), _ptr(hd), ctypes.byref(lam_used), _ptr(ws),
                                        ws.numel(), _stream(torch, stream))
    _check("gptq_quantize_group_q2tp", code)
    return dict(codes=codes, rungs=rungs, scales=scales, tab=tab, lost=lost, u=u, d=d, hdiag=hd,
                lam=lam_used.value)


def debias(bits, w, h_packed, codes, rungs, tab, lost, scales, ws=None, want_num_den=False, stream=None):
    """Output debias (in place on tab, lost, scales).  Returns num_den [rows, 2]
    f64 or None."""
    import torch

    lib = load()
    rows, n = _matrix(w)
    dev = w.device
    _packed(h_packed, n, dev)
    if int(bits) in (2, 4):
        gpr = n // 32
        _need(codes, "codes", dtype=torch.uint8, numel=rows * n * int(bits) // 8, device=dev)
        _need(rungs, "rungs", dtype=torch.uint8, numel=rows * gpr, device=dev)
        _need(tab, "tab", numel=rows * 32, device=dev)
        _need(lost, "lost", numel=rows * 2, device=dev)
        _need(scales, "scales", numel=rows * gpr, device=dev)
    nd = torch.empty(rows, 2, dtype=torch.float64, device=w.device) if want_num_den else None
    if ws is None:
        ws = workspace(lib.gptq_debias_workspace_bytes(rows, n), w.device)
    _ws(ws, dev)
    code = lib.gptq_debias(int(bits), _ptr(w), rows, n, _ptr(h_packed), _ptr(codes), _ptr(rungs), _ptr(tab),
                           _ptr(lost), _ptr(scales), _ptr(nd), _ptr(ws), ws.numel(), _stream(torch, stream))
    _check("gptq_debias", code)
    return nd


# ------------------------------------------------------------------ serving
#
# These calls are short, so the host's part of them counts: each wrapper first
# looks at its arguments in one expression of cheap attributes, and only where
# that does not hold goes through the checks that name the argument.  What the
# library gets of an argument is taken whether or not the expression holds,
# since the long checks let through some calls that it does not know.

ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}
_serve = {}  # torch, its dtypes and the raw-stream call, once the first wrapper ran
_serve_words = {}  # device index -> the status word its serving calls set (tensor, address)
_serve_lock = threading.Lock()
_attention_ws = {}  # device index and shape of a kv4_attention call -> its workspace bytes


def _serving():
    import torch

    load()  # first: another thread's call goes ahead as soon as _serve holds anything
    _serve.update(torch=torch, empty=torch.empty, f32=torch.float32, u8=torch.uint8, i32=torch.int32, i64=torch.int64,
                  dtypes={torch.bfloat16: 0, torch.float16: 1},
                  raw=getattr(torch._C, "_cuda_getCurrentRawStream", None),
                  current=getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device))
    return _serve


def _raw_stream(sv, stream, index):
    """The call's stream as an integer: the given one, or the device's current one."""
    if stream is not None:
        at = getattr(stream, "device", None)
        if at is not None and at.index != index:
            raise ValueError(f"the stream is on {at}, the call's data on cuda:{index}")
        return stream.cuda_stream
    raw = sv["raw"]
    return raw(index) if raw is not None else sv["torch"].cuda.current_stream(index).cuda_stream


def _empty(sv, stream):
    """torch.empty for what a call on the given `stream` writes: memory of that
    stream, so that neither an earlier use of it nor its next one overlaps the
    call."""

    def empty(*size, **kw):
        with sv["torch"].cuda.stream(stream):
            return sv["empty"](*size, **kw)

    return empty


def _serve_word(index):
    with _serve_lock:  # one word a device, whoever is first: calls in flight keep its address
        w = _serve_words.get(index)
        if w is None:
            import torch

            t = torch.zeros(4, dtype=torch.int32, device=torch.device("cuda", index))
            torch.cuda.current_stream(index).synchronize()  # before a call on any stream may set it
            w = _serve_words[index] = (t, t.data_ptr())
    return w[1]


def serve_check(device=None):
    """Raises GptqError(TIMEOUT) if a bounded device wait of a serving call on
    `device` (default: the current one) ran out since the last check.  Waits
    for the device and reads one word back."""
    import torch

    device = torch.device("cuda") if device is None else torch.device(device)
    index = torch.cuda.current_device() if device.index is None else device.index
    w = _serve_words.get(index)
    if w is not None:
        torch.cuda.synchronize(index)
        if int(w[0][0]) != 0:
            w[0].zero_()
            raise GptqError("serving call", 6)


def _here(t, name):
    """Raise ValueError unless ``t`` is on the current device.  The library
    launches there, and the default stream has one handle on every device, so
    nothing else would notice."""
    _ptr(t)
    at, current = t.get_device(), _serve["current"]()
    if at != current:
        raise ValueError(f"{name} is on cuda:{at}, the current device is cuda:{current}")


def _no_gradient(**tensors):
    """Raise ValueError if one of them would need the operator's gradient."""
    import torch

    if torch.is_grad_enabled():
        for name, t in tensors.items():
            if t is not None and t.requires_grad:
                raise ValueError(f"{name} requires a gradient, and the call has none: make it under torch.no_grad()")


def _dtype16(t, name):
    import torch

    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a torch tensor")
    if t.dtype not in (torch.bfloat16, torch.float16):
        raise ValueError(f"{name} must be torch.bfloat16 or torch.float16, got {t.dtype}")


def _strided(t, name, shape, like):
    """Raise ValueError unless ``t`` has ``shape``, the dtype and device of
    ``like``, dense last dimension and other strides of a multiple of 8
    elements (16 bytes)."""
    import torch

    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a torch tensor")
    if t.dtype != like.dtype:
        raise ValueError(f"{name} must be {like.dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.device != like.device:
        raise ValueError(f"{name} is on {t.device}, the call's data on {like.device}")
    st = t.stride()
    if t.numel() == 0:
        return
    if st[-1] != 1 and shape[-1] > 1:
        raise ValueError(f"{name} must be contiguous in its last dimension")
    if any(s % 8 and n > 1 for s, n in zip(st[:-1], shape[:-1])):
        raise ValueError(f"{name} must have strides of a multiple of 8 elements, got {st}")


def _rows_of(t, name, tokens, rows, like):
    """Raise ValueError unless ``t`` is a [tokens, rows] matrix of like's dtype
    whose rows are dense and do not overlap."""
    import torch

    if not isinstance(t, torch.Tensor) or t.dtype != like.dtype:
        raise ValueError(f"{name} must be a {like.dtype} tensor")
    if t.shape != (tokens, rows):
        raise ValueError(f"{name} must have shape {(tokens, rows)}, got {tuple(t.shape)}")
    if t.device != like.device:
        raise ValueError(f"{name} is on {t.device}, the call's data on {like.device}")
    st = t.stride()
    if (rows > 1 and st[1] != 1) or (tokens > 1 and st[0] < rows):
        raise ValueError(f"{name} must have dense rows that do not overlap, got strides {st}")


def _refuse_linear(x, nibbles, rungs, tab, bias, act, residual, out, last=True):
    import torch

    _dtype16(x, "x")
    if x.dim() != 2:
        raise ValueError(f"x must be 2-D [tokens, n], got shape {tuple(x.shape)}")
    tokens, n = x.shape
    if n <= 0 or n % 32:
        raise ValueError(f"x must have a multiple of 32 columns, got {n}")
    dev = x.device
    _strided(x, "x", x.shape, x)
    if tokens > 1 and x.stride(0) < n:
        raise ValueError(f"x must have rows that do not overlap, got strides {x.stride()}")
    _need(tab, "tab", device=dev)
    if tab.dim() != 2 or tab.shape[1] != 32:
        raise ValueError(f"tab must be [rows, 32], got shape {tuple(tab.shape)}")
    rows = tab.shape[0]
    _need(nibbles, "nibbles", dtype=torch.uint8, numel=rows * n // 2, device=dev)
    _need(rungs, "rungs", dtype=torch.uint8, numel=rows * (n // 32), device=dev)
    if bias is not None:
        _need(bias, "bias", dtype=x.dtype, numel=rows, device=dev)
    if act not in ACTIVATIONS:
        raise ValueError(f"act must be one of {', '.join(ACTIVATIONS)}, got {act!r}")
    if residual is not None:
        _rows_of(residual, "residual", tokens, rows, x)
    if out is not None:
        _rows_of(out, "out", tokens, rows, x)
    _no_gradient(x=x, bias=bias, residual=residual)
    if last:
        _here(x, "x")


def q4tp_linear(x, nibbles, rungs, tab, bias=None, act="none", residual=None, out=None, stream=None):
    """act(x W^T + bias) + residual with W [rows, n] in q4tp form (nibbles,
    rungs, tab as quantize_group returns them).  x [tokens, n] bf16 or f16
    (rows may be strided, not overlap), bias [rows], residual [tokens, rows] and
    the result [tokens, rows] of x's dtype.  act: a key of ACTIVATIONS.  `out` may
    be the residual itself, and overlaps no other input."""
    sv = _serve or _serving()
    try:
        xt, xs, u8 = x.dtype, x.shape, sv["u8"]
        dt, dev = sv["dtypes"][xt], x.get_device()
        tokens, n = xs
        rows = tab.shape[0]
        code = ACTIVATIONS[act]
        st = x.stride()
        ldx = st[0] if tokens > 1 else n
        fine = (dev >= 0 and dev == sv["current"]() and n > 0 and n % 32 == 0 and st[1] == 1 and ldx % 8 == 0
                and ldx >= n and not x.requires_grad
                and tab.dtype is sv["f32"] and tab.shape == (rows, 32) and tab.is_contiguous()
                and tab.get_device() == dev
                and nibbles.dtype is u8 and nibbles.numel() == rows * n // 2 and nibbles.is_contiguous()
                and nibbles.get_device() == dev
                and rungs.dtype is u8 and rungs.numel() == rows * n // 32 and rungs.is_contiguous()
                and rungs.get_device() == dev)
        bp = rp = None
        ldr = 0
        if bias is not None:
            fine = (fine and bias.dtype is xt and bias.numel() == rows and bias.is_contiguous()
                    and bias.get_device() == dev and not bias.requires_grad)
            bp = bias.data_ptr()
        if residual is not None:
            st = residual.stride()
            ldr = st[0] if tokens > 1 else rows
            fine = (fine and residual.dtype is xt and residual.shape == (tokens, rows) and (rows == 1 or st[1] == 1)
                    and ldr >= rows and residual.get_device() == dev and not residual.requires_grad)
            rp = residual.data_ptr()
        ldy = rows
        if out is not None:
            st = out.stride()
            ldy = st[0] if tokens > 1 else rows
            fine = (fine and out.dtype is xt and out.shape == (tokens, rows) and (rows == 1 or st[1] == 1)
                    and ldy >= rows and out.get_device() == dev)
    except (AttributeError, KeyError, TypeError, ValueError, IndexError):
        fine = False
    if not fine:
        _refuse_linear(x, nibbles, rungs, tab, bias, act, residual, out)
    if out is None:
        out = (sv["empty"] if stream is None else _empty(sv, stream))((tokens, rows), dtype=xt, device=x.device)
    code = _lib.gptq_q4tp_linear(dt, x.data_ptr(), ldx, tokens, nibbles.data_ptr(), rungs.data_ptr(), tab.data_ptr(),
                                 rows, n, bp, code, rp, ldr, out.data_ptr(), ldy,
                                 (_serve_words.get(dev) or (0, _serve_word(dev)))[1], _raw_stream(sv, stream, dev))
    if code:
        raise GptqError("gptq_q4tp_linear", code)
    return out


def _refuse_gated(x, nibbles, rungs, tab, bias, act, out, ws):
    _refuse_linear(x, nibbles, rungs, tab, bias, act, None, None, last=False)
    if tab.shape[0] == 0 or tab.shape[0] % 2:
        raise ValueError(f"tab must have the gate's rows and as many of the up projection, got {tab.shape[0]}")
    if out is not None:
        _rows_of(out, "out", x.shape[0], tab.shape[0] // 2, x)
    if ws is not None:
        _ws(ws, x.device)
    _here(x, "x")


def q4tp_gated(x, nibbles, rungs, tab, bias=None, act="silu", out=None, ws=None, stream=None):
    """act(x Wg^T + bg) * (x Wu^T + bu), the first half of a gated feed-forward
    block, in one launch (bf16 above 8 tokens: two, of which the first brings x to
    f16).  W [2 * inner, n] in q4tp form holds the gate's rows and
    then the up projection's, as quantize_group returns them for the two matrices
    one above the other; bias [2 * inner].  x [tokens, n] and the result [tokens,
    inner] as in q4tp_linear.  `out` overlaps no input."""
    sv = _serve or _serving()
    try:
        xt, xs, u8 = x.dtype, x.shape, sv["u8"]
        dt, dev = sv["dtypes"][xt], x.get_device()
        tokens, n = xs
        rows = tab.shape[0]
        inner = rows // 2
        code = ACTIVATIONS[act]
        st = x.stride()
        ldx = st[0] if tokens > 1 else n
        fine = (dev >= 0 and dev == sv["current"]() and n > 0 and n % 32 == 0 and st[1] == 1 and ldx % 8 == 0
                and ldx >= n and not x.requires_grad
                and tab.dtype is sv["f32"] and tab.shape == (rows, 32) and tab.is_contiguous()
                and tab.get_device() == dev and rows > 0 and rows % 2 == 0
                and nibbles.dtype is u8 and nibbles.numel() == rows * n // 2 and nibbles.is_contiguous()
                and nibbles.get_device() == dev
                and rungs.dtype is u8 and rungs.numel() == rows * n // 32 and rungs.is_contiguous()
                and rungs.get_device() == dev)
        bp = None
        if bias is not None:
            fine = (fine and bias.dtype is xt and bias.numel() == rows and bias.is_contiguous()
                    and bias.get_device() == dev and not bias.requires_grad)
            bp = bias.data_ptr()
        ldy = inner
        if out is not None:
            st = out.stride()
            ldy = st[0] if tokens > 1 else inner
            fine = (fine and out.dtype is xt and out.shape == (tokens, inner) and (inner == 1 or st[1] == 1)
                    and ldy >= inner and out.get_device() == dev)
        if ws is not None:
            fine = fine and ws.dtype is u8 and ws.is_contiguous() and ws.get_device() == dev
    except (AttributeError, KeyError, TypeError, ValueError, IndexError):
        fine = False
    if not fine:
        _refuse_gated(x, nibbles, rungs, tab, bias, act, out, ws)
    if out is None:
        out = (sv["empty"] if stream is None else _empty(sv, stream))((tokens, inner), dtype=xt, device=x.device)
    wp = wn = 0
    if ws is None and dt == 0 and tokens > 8:
        wn = _lib.gptq_q4tp_gated_workspace_bytes(dt, tokens, n)
        ws = (sv["empty"] if stream is None else _empty(sv, stream))(wn, dtype=u8, device=x.device)
    if ws is not None:
        wp, wn = ws.data_ptr(), ws.numel()
    status = _lib.gptq_q4tp_gated(dt, x.data_ptr(), ldx, tokens, nibbles.data_ptr(), rungs.data_ptr(), tab.data_ptr(),
                                  inner, n, bp, code, out.data_ptr(), ldy, wp, wn,
                                  (_serve_words.get(dev) or (0, _serve_word(dev)))[1], _raw_stream(sv, stream, dev))
    if status:
        raise GptqError("gptq_q4tp_gated", status)
    return out


def _cache(cache, dim, page_size):
    """pages, heads of a cache pool after checking it against dim and page_size."""
    import torch

    _need(cache, "cache", dtype=torch.uint8)
    if dim not in (64, 128, 256):
        raise ValueError(f"dim must be 64, 128 or 256, got {dim}")
    if page_size <= 0 or page_size > 4096 or page_size % 16:
        raise ValueError(f"page_size must be a multiple of 16 up to 4096, got {page_size}")
    if cache.dim() != 3 or cache.shape[2] != page_size * dim * 5 // 4:
        raise ValueError(f"cache must be [pages, heads, {page_size * dim * 5 // 4}] for dim {dim} and pages of "
                         f"{page_size} tokens, got shape {tuple(cache.shape)}")
    return cache.shape[0], cache.shape[1]


def kv4_cache(pages, heads, dim, page_size, device="cuda"):
    """An empty 4-bit key/value pool: u8 [pages, heads, page_size * dim * 5 / 4]."""
    import torch

    cache = torch.zeros(pages, heads, page_size * dim * 5 // 4, dtype=torch.uint8, device=device)
    _cache(cache, dim, page_size)
    return cache


def _refuse_write(cache, k, v, slots, page_size, last=True):
    import torch

    _dtype16(k, "k")
    if k.dim() != 3:
        raise ValueError(f"k must be 3-D [tokens, heads, dim], got shape {tuple(k.shape)}")
    tokens, heads, dim = k.shape
    pages, ch = _cache(cache, dim, page_size)
    if heads != ch:
        raise ValueError(f"k has {heads} heads, the cache {ch}")
    if cache.device != k.device:
        raise ValueError(f"cache is on {cache.device}, the call's data on {k.device}")
    _strided(k, "k", k.shape, k)
    _strided(v, "v", k.shape, k)
    _need(slots, "slots", dtype=torch.int64, numel=tokens, device=k.device)
    if last:
        _here(k, "k")


def kv4_write(cache, k, v, slots, page_size, stream=None):
    """Quantise k, v [tokens, heads, dim] (bf16 or f16, strided views allowed)
    into the cache at slots [tokens] i64 (page * page_size + place; negative:
    left out).  The slots of a call have to differ: one given twice ends as a mix
    of its tokens.  Returns the cache."""
    sv = _serve or _serving()
    try:
        kt, shape, dev = k.dtype, k.shape, k.get_device()
        dt = sv["dtypes"][kt]
        tokens, heads, dim = shape
        pages = cache.shape[0]
        kts, khs, k1 = k.stride()
        vts, vhs, v1 = v.stride()
        fine = (dev >= 0 and dev == sv["current"]() and dim in (64, 128, 256) and tokens > 1 and heads > 1
                and v.dtype is kt and v.shape == shape
                and k1 == 1 and v1 == 1 and (kts | khs | vts | vhs) % 8 == 0 and v.get_device() == dev
                and 0 < page_size <= 4096 and page_size % 16 == 0 and cache.dtype is sv["u8"]
                and cache.shape == (pages, heads, page_size * dim * 5 // 4) and cache.is_contiguous()
                and cache.get_device() == dev and slots.dtype is sv["i64"] and slots.numel() == tokens
                and slots.is_contiguous() and slots.get_device() == dev)
    except (AttributeError, KeyError, TypeError, ValueError, IndexError):
        fine = False
    if not fine:
        _refuse_write(cache, k, v, slots, page_size)
        # A dimension of one element may carry any stride (the library wants a multiple of 8).
        kts, vts = (kts, vts) if tokens > 1 else (0, 0)
        khs, vhs = (khs, vhs) if heads > 1 else (0, 0)
    code = _lib.gptq_kv4_write(dt, cache.data_ptr(), pages, heads, dim, page_size, k.data_ptr(), v.data_ptr(), kts,
                               khs, vts, vhs, slots.data_ptr(), tokens, _raw_stream(sv, stream, dev))
    if code:
        raise GptqError("gptq_kv4_write", code)
    return cache


def rotary_frequencies(rot, base=10000.0, scaling="none", factor=1.0, length=8192, low=1.0, high=4.0):
    """Radians a position of the rot / 2 pairs, base ** (-2 i / rot), as floats.
    scaling, for contexts `factor` times as long as those trained on: "linear"
    divides every frequency by factor; "base" raises the base to base * factor **
    (rot / (rot - 2)), which divides the last frequency by factor and leaves the first; "ramp"
    divides those that make less than `low` turns in `length` positions, leaves
    those that make more than `high`, and goes from one to the other between."""
    if rot <= 0 or rot % 2:
        raise ValueError(f"rot must be a positive even number, got {rot}")
    if not (base > 0 and factor > 0):
        raise ValueError(f"base and factor must be positive, got {base} and {factor}")
    if scaling not in ("none", "linear", "base", "ramp"):
        raise ValueError(f"scaling must be one of none, linear, base, ramp, got {scaling!r}")
    if scaling == "base":
        if rot < 4:
            raise ValueError(f"scaling by the base needs rot of 4 and more, got {rot}")
        base = base * factor ** (rot / (rot - 2))
    f = [base ** (-2 * i / rot) for i in range(rot // 2)]
    if scaling == "linear":
        f = [v / factor for v in f]
    elif scaling == "ramp":
        if not (high > low and length > 0):
            raise ValueError(f"ramp needs high above low and a positive length, got {high}, {low} and {length}")
        w = [min(max((length * v / (2 * math.pi) - low) / (high - low), 0.0), 1.0) for v in f]
        f = [v * (a + (1 - a) / factor) for v, a in zip(f, w)]
    return f


def rotary_turns(frequencies, device="cuda"):
    """The form of frequencies (radians a position) that the rotary calls take:
    i64, 2^64ths of a turn a position, modulo one turn."""
    import torch

    f = [float(v) for v in frequencies]
    if not f or not all(math.isfinite(v) for v in f):
        raise ValueError("frequencies must be finite numbers, at least one")
    t = [(round(v / (2 * math.pi) * 2 ** 64) + 2 ** 63) % 2 ** 64 - 2 ** 63 for v in f]
    return torch.tensor(t, dtype=torch.int64, device=device)


ROTARY_LAYOUTS = {"half": 0, "interleaved": 1}


def _refuse_turns(positions, turns, layout, gain, tokens, dim, device):
    import torch

    _need(positions, "positions", dtype=torch.int64, numel=tokens, device=device)
    _need(turns, "turns", dtype=torch.int64, device=device)
    rot = 2 * turns.numel()
    if rot == 0 or rot > dim or rot % 16:
        raise ValueError(f"turns must have a multiple of 8 elements up to {dim // 2}, got {turns.numel()}")
    if layout not in ROTARY_LAYOUTS:
        raise ValueError(f"layout must be one of {', '.join(ROTARY_LAYOUTS)}, got {layout!r}")
    if not math.isfinite(gain):
        raise ValueError(f"gain must be finite, got {gain}")


def _heads_out(out, name, x):
    """Raise ValueError unless `out` can take what `x` [tokens, heads, dim] becomes."""
    _strided(out, name, x.shape, x)
    tokens, heads, dim = x.shape
    ts, hs, _ = out.stride()
    # Rows that do not overlap: heads inside a token's stride, or tokens inside a head's.
    if out.numel() and ((heads > 1 and hs < dim) or (tokens > 1 and ts < dim) or (
            tokens > 1 and heads > 1 and ts < (heads - 1) * hs + dim and hs < (tokens - 1) * ts + dim)):
        raise ValueError(f"{name} must have rows that do not overlap, got strides {out.stride()}")
    if out.data_ptr() == x.data_ptr() and out.numel() and any(
            a != b and n > 1 for a, b, n in zip(out.stride(), x.stride(), x.shape)):
        raise ValueError(f"{name} is the input with other strides: {out.stride()}, {x.stride()}")


def _refuse_rotary(x, positions, turns, layout, gain, out):
    _dtype16(x, "x")
    if x.dim() != 3:
        raise ValueError(f"x must be 3-D [tokens, heads, dim], got shape {tuple(x.shape)}")
    tokens, heads, dim = x.shape
    if heads == 0 or dim == 0 or dim % 16 or dim > 1024:
        raise ValueError(f"x must have heads of a multiple of 16 channels, at most 1024, got shape {tuple(x.shape)}")
    _strided(x, "x", x.shape, x)
    _refuse_turns(positions, turns, layout, gain, tokens, dim, x.device)
    if out is not None:
        _heads_out(out, "out", x)
    _no_gradient(x=x)
    _here(x, "x")


def rotary(x, positions, turns, layout="half", gain=1.0, out=None, stream=None):
    """x [tokens, heads, dim] (bf16 or f16, strided views allowed) turned to
    its positions [tokens] i64: pair i of a head's first 2 * len(turns) channels
    by positions * turns[i] (see rotary_turns), times gain; the other channels
    stay.  layout "half": pair i is channels (i, i + len(turns)); "interleaved":
    (2 i, 2 i + 1).  `out` may be x itself, else overlaps no input."""
    sv = _serve or _serving()
    try:
        xt, dev, i64 = x.dtype, x.get_device(), sv["i64"]
        dt = sv["dtypes"][xt]
        tokens, heads, dim = x.shape
        ts, hs, x1 = x.stride()
        # A dimension of one element may carry any stride (the library wants a multiple of 8).
        ts, hs = ts if tokens > 1 else 0, hs if heads > 1 else 0
        rot = 2 * turns.numel()
        code = ROTARY_LAYOUTS[layout]
        fine = (dev >= 0 and dev == sv["current"]() and x1 == 1 and heads > 0 and 0 < dim <= 1024
                and dim % 16 == 0 and (ts | hs) % 8 == 0 and not x.requires_grad
                and positions.dtype is i64 and positions.numel() == tokens and positions.is_contiguous()
                and positions.get_device() == dev and turns.dtype is i64 and turns.is_contiguous()
                and turns.get_device() == dev and 0 < rot <= dim and rot % 16 == 0
                and (out is None or (out is x and (hs >= dim or heads == 1)
                                     and (ts >= (heads - 1) * hs + dim or tokens <= 1)))
                and -3e38 < gain < 3e38)
    except (AttributeError, KeyError, TypeError, ValueError, IndexError):
        fine = False
    if not fine:
        _refuse_rotary(x, positions, turns, layout, gain, out)
    if out is x:
        ots, ohs = ts, hs
    elif out is None:
        out = (sv["empty"] if stream is None else _empty(sv, stream))((tokens, heads, dim), dtype=xt, device=x.device)
        ots, ohs = heads * dim, dim
    else:
        ots, ohs, _ = out.stride()
        ots, ohs = ots if tokens > 1 else 0, ohs if heads > 1 else 0
    status = _lib.gptq_rotary(dt, x.data_ptr(), ts, hs, tokens, heads, dim, rot, code, positions.data_ptr(),
                              turns.data_ptr(), gain, out.data_ptr(), ots, ohs, _raw_stream(sv, stream, dev))
    if status:
        raise GptqError("gptq_rotary", status)
    return out


def _refuse_write_rotary(cache, q, k, v, slots, page_size, positions, turns, layout, gain, out):
    _refuse_write(cache, k, v, slots, page_size, last=False)
    tokens, _, dim = k.shape
    _dtype16(q, "q")
    if q.dim() != 3 or q.shape[0] != tokens or q.shape[2] != dim or q.shape[1] == 0:
        raise ValueError(f"q must be [{tokens}, heads, {dim}], got shape {tuple(q.shape)}")
    _strided(q, "q", q.shape, k)
    _refuse_turns(positions, turns, layout, gain, tokens, dim, k.device)
    if out is not None:
        _heads_out(out, "out", q)
    _no_gradient(q=q, k=k, v=v)
    _here(k, "k")


def kv4_write_rotary(cache, q, k, v, slots, page_size, positions, turns, layout="half", gain=1.0, out=None,
                     stream=None):
    """What rotary does to q and k and kv4_write with the turned k and v, in one
    call and with the same bits.  q [tokens, query heads, dim], k, v [tokens,
    heads, dim] (strided views allowed), slots (each different, or outside the
    pool), positions [tokens] i64.  Returns the turned q; `out` may be q itself,
    else overlaps no input."""
    sv = _serve or _serving()
    try:
        kt, shape, dev, i64 = k.dtype, k.shape, k.get_device(), sv["i64"]
        dt = sv["dtypes"][kt]
        tokens, heads, dim = shape
        hq = q.shape[1]
        pages = cache.shape[0]
        qts, qhs, q1 = q.stride()
        kts, khs, k1 = k.stride()
        vts, vhs, v1 = v.stride()
        # (As in rotary: what one element does not use.)
        if tokens <= 1:
            qts = kts = vts = 0
        if heads == 1:
            khs = vhs = 0
        if hq == 1:
            qhs = 0
        rot = 2 * turns.numel()
        code = ROTARY_LAYOUTS[layout]
        fine = (dev >= 0 and dev == sv["current"]() and dim in (64, 128, 256) and heads > 0 and hq > 0
                and q.dtype is kt and q.shape == (tokens, hq, dim) and v.dtype is kt and v.shape == shape
                and k1 == 1 and v1 == 1 and q1 == 1 and (kts | khs | vts | vhs | qts | qhs) % 8 == 0
                and v.get_device() == dev and q.get_device() == dev
                and not (q.requires_grad or k.requires_grad or v.requires_grad)
                and 0 < page_size <= 4096 and page_size % 16 == 0 and cache.dtype is sv["u8"]
                and cache.shape == (pages, heads, page_size * dim * 5 // 4) and cache.is_contiguous()
                and cache.get_device() == dev
                and slots.dtype is i64 and slots.numel() == tokens and slots.is_contiguous() and slots.get_device() == dev
                and positions.dtype is i64 and positions.numel() == tokens and positions.is_contiguous()
                and positions.get_device() == dev and turns.dtype is i64 and turns.is_contiguous()
                and turns.get_device() == dev and 0 < rot <= dim and rot % 16 == 0
                and (out is None or (out is q and (qhs >= dim or hq == 1)
                                     and (qts >= (hq - 1) * qhs + dim or tokens <= 1)))
                and -3e38 < gain < 3e38)
    except (AttributeError, KeyError, TypeError, ValueError, IndexError):
        fine = False
    if not fine:
        _refuse_write_rotary(cache, q, k, v, slots, page_size, positions, turns, layout, gain, out)
    if out is q:
        ots, ohs = qts, qhs
    elif out is None:
        out = (sv["empty"] if stream is None else _empty(sv, stream))((tokens, hq, dim), dtype=kt, device=k.device)
        ots, ohs = hq * dim, dim
    else:
        ots, ohs, _ = out.stride()
        ots, ohs = ots if tokens > 1 else 0, ohs if hq > 1 else 0
    status = _lib.gptq_kv4_write_rotary(dt, cache.data_ptr(), pages, heads, dim, page_size, q.data_ptr(), qts, qhs, hq,
                                        k.data_ptr(), v.data_ptr(), kts, khs, vts, vhs, slots.data_ptr(), tokens, rot,
                                        code, positions.data_ptr(), turns.data_ptr(), gain, out.data_ptr(), ots, ohs,
                                        _raw_stream(sv, stream, dev))
    if status:
        raise GptqError("gptq_kv4_write_rotary", status)
    return out


def _refuse_read(cache, slots, dim, page_size, dtype):
    import torch

    _cache(cache, dim, page_size)
    _need(slots, "slots", dtype=torch.int64, device=cache.device)
    if dtype not in (torch.bfloat16, torch.float16):
        raise ValueError(f"dtype must be torch.bfloat16 or torch.float16, got {dtype}")
    _here(cache, "cache")


def kv4_read(cache, slots, dim, page_size, dtype, stream=None):
    """The values k, v [tokens, heads, dim] that the cache holds at slots
    [tokens] i64, in the dtype it was written in (zeros outside the pool)."""
    sv = _serve or _serving()
    try:
        dt, dev = sv["dtypes"][dtype], cache.get_device()
        pages, heads, size = cache.shape
        tokens = slots.numel()
        fine = (dev >= 0 and dev == sv["current"]() and dim in (64, 128, 256) and 0 < page_size <= 4096
                and page_size % 16 == 0
                and cache.dtype is sv["u8"] and size == page_size * dim * 5 // 4 and cache.is_contiguous()
                and slots.dtype is sv["i64"] and slots.is_contiguous() and slots.get_device() == dev)
    except (AttributeError, KeyError, TypeError, ValueError, IndexError):
        fine = False
    if not fine:
        _refuse_read(cache, slots, dim, page_size, dtype)
    empty = sv["empty"] if stream is None else _empty(sv, stream)
    k = empty((tokens, heads, dim), dtype=dtype, device=cache.device)
    v = empty((tokens, heads, dim), dtype=dtype, device=cache.device)
    code = _lib.gptq_kv4_read(dt, cache.data_ptr(), pages, heads, dim, page_size, slots.data_ptr(), tokens,
                              k.data_ptr(), v.data_ptr(), _raw_stream(sv, stream, dev))
    if code:
        raise GptqError("gptq_kv4_read", code)
    return k, v


def _refuse_attention(q, cache, table, kv_lens, page_size, q_starts, max_q, out, ws, lse, last=True):
    import torch

    _dtype16(q, "q")
    if q.dim() != 3:
        raise ValueError(f"q must be 3-D [tokens, heads, dim], got shape {tuple(q.shape)}")
    tq, hq, dim = q.shape
    dev = q.device
    pages, heads = _cache(cache, dim, page_size)
    if heads <= 0 or hq % heads or hq == 0:
        raise ValueError(f"q has {hq} heads, not a multiple of the cache's {heads}")
    if cache.device != dev:
        raise ValueError(f"cache is on {cache.device}, the call's data on {dev}")
    _strided(q, "q", q.shape, q)
    _need(table, "table", dtype=torch.int32, device=dev)
    if table.dim() != 2 or table.shape[1] == 0:
        raise ValueError(f"table must be 2-D [seqs, pages], got shape {tuple(table.shape)}")
    seqs = table.shape[0]
    _need(kv_lens, "kv_lens", dtype=torch.int32, numel=seqs, device=dev)
    if q_starts is not None:
        _need(q_starts, "q_starts", dtype=torch.int32, numel=seqs + 1, device=dev)
    elif tq != seqs or max_q != 1:
        raise ValueError(f"without q_starts there is one query a sequence: q has {tq} tokens for {seqs} sequences")
    if max_q <= 0:
        raise ValueError(f"max_q must be positive, got {max_q}")
    if out is not None:
        _need(out, "out", dtype=q.dtype, numel=q.numel(), device=dev)
    if lse is not None:
        _need(lse, "lse", numel=tq * hq, device=dev)
    if ws is not None:
        _ws(ws, dev)
    _no_gradient(q=q)
    if last:
        _here(q, "q")


def kv4_attention(q, cache, table, kv_lens, page_size, q_starts=None, max_q=1, scale=None, out=None, ws=None,
                  stream=None, lse=None):
    """Causal attention of q [tokens, query heads, dim] (bf16 or f16) over the
    4-bit cache: softmax(scale q k^T) v per sequence and head, scale default
    1 / sqrt(dim).  table [seqs, pages per sequence] i32, kv_lens [seqs] i32
    (the queries' own keys included).  The queries of sequence b are its last
    tokens, rows q_starts[b] .. q_starts[b + 1] - 1 of q (i32 [seqs + 1], the
    first max_q of each); without q_starts, one a sequence.  Outputs of rows
    that are no sequence's are zero.  `lse` (f32 [tokens, query heads]) receives
    the logarithm of each row's sum of exponentials, -inf where it sees nothing.
    `out` and `lse` overlap no input."""
    sv = _serve or _serving()
    try:
        qt, dev, i32 = q.dtype, q.get_device(), sv["i32"]
        dt = sv["dtypes"][qt]
        tq, hq, dim = q.shape
        pages, heads, size = cache.shape
        seqs, per = table.shape
        qts, qhs, q1 = q.stride()
        fine = (dev >= 0 and dev == sv["current"]() and dim in (64, 128, 256) and tq > 0 and hq > 1
                and hq % heads == 0 and q1 == 1 and not q.requires_grad
                and (qts | qhs) % 8 == 0 and 0 < page_size <= 4096 and page_size % 16 == 0 and max_q > 0
                and cache.dtype is sv["u8"] and size == page_size * dim * 5 // 4 and cache.is_contiguous()
                and cache.get_device() == dev and table.dtype is i32 and per > 0 and table.is_contiguous()
                and table.get_device() == dev and kv_lens.dtype is i32 and kv_lens.numel() == seqs
                and kv_lens.is_contiguous() and kv_lens.get_device() == dev)
        sp = None
        if q_starts is None:
            fine = fine and tq == seqs and max_q == 1
        else:
            fine = (fine and q_starts.dtype is i32 and q_starts.numel() == seqs + 1 and q_starts.is_contiguous()
                    and q_starts.get_device() == dev)
            sp = q_starts.data_ptr()
        if fine and out is not None:
            fine = (out.dtype is qt and out.numel() == tq * hq * dim and out.is_contiguous()
                    and out.get_device() == dev)
        if fine and lse is not None:
            fine = (lse.dtype is sv["f32"] and lse.numel() == tq * hq and lse.is_contiguous()
                    and lse.get_device() == dev)
        if fine and ws is not None:
            fine = ws.dtype is sv["u8"] and ws.is_contiguous() and ws.get_device() == dev
    except (AttributeError, KeyError, TypeError, ValueError, IndexError):
        fine = False
    if not fine:
        _refuse_attention(q, cache, table, kv_lens, page_size, q_starts, max_q, out, ws, lse)
        qts, qhs = qts if tq > 1 else 0, qhs if hq > 1 else 0
    if out is None:
        out = (sv["empty"] if stream is None else _empty(sv, stream))((tq, hq, dim), dtype=qt, device=q.device)
    wp = wn = 0
    if ws is None:
        shape = (dev, dim, heads, hq, max_q, seqs, sp is None, per * page_size)
        wn = _attention_ws.get(shape)
        if wn is None:
            wn = _lib.gptq_kv4_attention_call_bytes(dim, heads, hq // heads, max_q, seqs, sp is None, per * page_size)
            if len(_attention_ws) < 4096:
                _attention_ws[shape] = wn
        if wn:
            ws = (sv["empty"] if stream is None else _empty(sv, stream))(wn, dtype=sv["u8"], device=q.device)
    if ws is not None:
        wp, wn = ws.data_ptr(), ws.numel()
    scale = dim ** -0.5 if scale is None else float(scale)
    word = (_serve_words.get(dev) or (0, _serve_word(dev)))[1]
    if lse is None:
        code = _lib.gptq_kv4_attention(dt, q.data_ptr(), qts, qhs, tq, cache.data_ptr(), pages, heads, hq // heads, dim,
                                       page_size, table.data_ptr(), per, kv_lens.data_ptr(), sp, seqs, int(max_q),
                                       scale, out.data_ptr(), wp, wn, word, _raw_stream(sv, stream, dev))
    else:
        code = _lib.gptq_kv4_attention_lse(dt, q.data_ptr(), qts, qhs, tq, cache.data_ptr(), pages, heads, hq // heads,
                                           dim, page_size, table.data_ptr(), per, kv_lens.data_ptr(), sp, seqs,
                                           int(max_q), scale, out.data_ptr(), lse.data_ptr(), wp, wn, word,
                                           _raw_stream(sv, stream, dev))
    if code:
        raise GptqError("gptq_kv4_attention", code)
    return out


def kv4_weights(table, page_size, heads):
    """Running totals for kv4_attention_weights, zeros: f32 [seqs, heads, places
    of a row of `table`]."""
    import torch

    return torch.zeros(table.shape[0], heads, table.shape[1] * page_size, dtype=torch.float32, device=table.device)


def _refuse_weights(weights, q, lse, cache, table, kv_lens, page_size, q_starts, max_q, ws):
    _refuse_attention(q, cache, table, kv_lens, page_size, q_starts, max_q, None, ws, lse, last=False)
    _need(lse, "lse", numel=q.shape[0] * q.shape[1], device=q.device)
    shape = (table.shape[0], cache.shape[1], table.shape[1] * page_size)
    _need(weights, "weights", device=q.device)
    if weights.shape != shape:
        raise ValueError(f"weights must be {shape}, got shape {tuple(weights.shape)}")
    _no_gradient(weights=weights)
    _here(q, "q")


def kv4_attention_weights(weights, q, lse, cache, table, kv_lens, page_size, q_starts=None, max_q=1, scale=None,
                          ws=None, stream=None):
    """Adds to `weights` (f32 [seqs, heads, places of a row of table], see
    kv4_weights) what the queries of a kv4_attention call looked at: for each cached
    token and key head the sum of exp(scale q k - lse) over the queries that see
    it and the query heads of the key head.  `lse` is what that call gave, the
    other arguments are its own.  Returns weights."""
    sv = _serve or _serving()
    try:
        qt, dev, i32 = q.dtype, q.get_device(), sv["i32"]
        dt = sv["dtypes"][qt]
        tq, hq, dim = q.shape
        pages, heads, size = cache.shape
        seqs, per = table.shape
        qts, qhs, q1 = q.stride()
        fine = (dev >= 0 and dev == sv["current"]() and dim in (64, 128, 256) and tq > 0 and hq > 1
                and hq % heads == 0 and q1 == 1 and not q.requires_grad
                and (qts | qhs) % 8 == 0 and 0 < page_size <= 4096 and page_size % 16 == 0 and max_q > 0
                and cache.dtype is sv["u8"] and size == page_size * dim * 5 // 4 and cache.is_contiguous()
                and cache.get_device() == dev and table.dtype is i32 and per > 0 and table.is_contiguous()
                and table.get_device() == dev and kv_lens.dtype is i32 and kv_lens.numel() == seqs
                and kv_lens.is_contiguous() and kv_lens.get_device() == dev
                and lse.dtype is sv["f32"] and lse.numel() == tq * hq and lse.is_contiguous() and lse.get_device() == dev
                and weights.dtype is sv["f32"] and weights.shape == (seqs, heads, per * page_size)
                and weights.is_contiguous() and weights.get_device() == dev and not weights.requires_grad)
        sp = None
        if q_starts is None:
            fine = fine and tq == seqs and max_q == 1
        else:
            fine = (fine and q_starts.dtype is i32 and q_starts.numel() == seqs + 1 and q_starts.is_contiguous()
                    and q_starts.get_device() == dev)
            sp = q_starts.data_ptr()
        if ws is not None:
            fine = fine and ws.dtype is sv["u8"] and ws.is_contiguous() and ws.get_device() == dev
    except (AttributeError, KeyError, TypeError, ValueError, IndexError):
        fine = False
    if not fine:
        _refuse_weights(weights, q, lse, cache, table, kv_lens, page_size, q_starts, max_q, ws)
        qts, qhs = qts if tq > 1 else 0, qhs if hq > 1 else 0
    wp = wn = 0
    if ws is None and max_q * hq > 64 * heads:  # (fewer rows never need one)
        wn = _lib.gptq_kv4_attention_weights_workspace_bytes(dim, heads, hq // heads, max_q, seqs, per * page_size)
        if wn:
            ws = (sv["empty"] if stream is None else _empty(sv, stream))(wn, dtype=sv["u8"], device=q.device)
    if ws is not None:
        wp, wn = ws.data_ptr(), ws.numel()
    code = _lib.gptq_kv4_attention_weights(dt, q.data_ptr(), qts, qhs, tq, lse.data_ptr(), cache.data_ptr(), pages, heads,
                                           hq // heads, dim, page_size, table.data_ptr(), per, kv_lens.data_ptr(), sp,
                                           seqs, int(max_q), dim ** -0.5 if scale is None else float(scale),
                                           weights.data_ptr(), wp, wn,
                                           (_serve_words.get(dev) or (0, _serve_word(dev)))[1],
                                           _raw_stream(sv, stream, dev))
    if code:
        raise GptqError("gptq_kv4_attention_weights", code)
    return weights


def _refuse_evict(cache, table, kv_lens, weights, keep, page_size, recent, out_table):
    import torch

    _need(cache, "cache", dtype=torch.uint8)
    dev = cache.device
    if cache.dim() != 3 or page_size <= 0 or cache.shape[2] * 4 % (page_size * 5):
        raise ValueError(f"cache must be a pool of pages of {page_size} tokens, got shape {tuple(cache.shape)}")
    _cache(cache, cache.shape[2] * 4 // (page_size * 5), page_size)
    _need(table, "table", dtype=torch.int32, device=dev)
    if table.dim() != 2 or table.shape[1] == 0:
        raise ValueError(f"table must be 2-D [seqs, pages], got shape {tuple(table.shape)}")
    seqs, per = table.shape
    _need(kv_lens, "kv_lens", dtype=torch.int32, numel=seqs, device=dev)
    _need(weights, "weights", device=dev)
    if weights.shape != (seqs, cache.shape[1], per * page_size):
        raise ValueError(f"weights must be {(seqs, cache.shape[1], per * page_size)}, got shape {tuple(weights.shape)}")
    if out_table is not None:
        _need(out_table, "out_table", dtype=torch.int32, device=dev)
        if out_table.dim() != 2 or out_table.shape[0] != seqs or out_table.shape[1] == 0:
            raise ValueError(f"out_table must be [{seqs}, pages], got shape {tuple(out_table.shape)}")
        if seqs and out_table.data_ptr() == table.data_ptr():
            raise ValueError("out_table is table: leave it out to keep the tokens in their sequence's pages")
        per = out_table.shape[1]
    if keep <= 0 or keep > per * page_size:
        raise ValueError(f"keep must be 1 to {per * page_size}, the places of a sequence, got {keep}")
    if recent < 0:
        raise ValueError(f"recent must not be negative, got {recent}")
    _no_gradient(weights=weights)
    _here(cache, "cache")


def kv4_evict(cache, table, kv_lens, weights, keep, page_size, recent=0, out_table=None, stream=None):
    """Cuts every sequence of the cache to `keep` tokens a key head: its last
    `recent` ones and the heaviest of the others by `weights` (kv4_attention_weights;
    equal ones: the earlier), each head its own, in order, from place 0 on.  They
    move within their sequence's pages or, with `out_table` [seqs, pages] i32, into
    those of it, which are in no row of `table`.  Pages that take tokens belong to one
    sequence.  Returns (kept i32 [seqs, heads, keep]: the earlier place of each, -1
    past the end; the new kv_lens; the new weights, zeros past the end)."""
    sv = _serve or _serving()
    try:
        dev, i32 = cache.get_device(), sv["i32"]
        pages, heads, size = cache.shape
        seqs, per = table.shape
        dim = size * 4 // (page_size * 5)
        to, op, ostride = per, None, 0
        fine = (dev >= 0 and dev == sv["current"]() and dim in (64, 128, 256) and 0 < page_size <= 4096
                and page_size % 16 == 0 and cache.dtype is sv["u8"] and size == page_size * dim * 5 // 4
                and cache.is_contiguous() and table.dtype is i32 and per > 0 and table.is_contiguous()
                and table.get_device() == dev and kv_lens.dtype is i32 and kv_lens.numel() == seqs
                and kv_lens.is_contiguous() and kv_lens.get_device() == dev and weights.dtype is sv["f32"]
                and weights.shape == (seqs, heads, per * page_size) and weights.is_contiguous()
                and weights.get_device() == dev and not weights.requires_grad and recent >= 0)
        if out_table is not None:
            fine = (fine and out_table.dtype is i32 and out_table.shape[0] == seqs and out_table.dim() == 2
                    and out_table.is_contiguous() and out_table.get_device() == dev)
            to = ostride = out_table.shape[1]
            op = out_table.data_ptr()
            fine = fine and op != table.data_ptr()
        fine = fine and 0 < keep <= to * page_size
    except (AttributeError, KeyError, TypeError, ValueError, IndexError, ZeroDivisionError):
        fine = False
    if not fine:
        _refuse_evict(cache, table, kv_lens, weights, keep, page_size, recent, out_table)
    empty = sv["empty"] if stream is None else _empty(sv, stream)
    kept = empty((seqs, heads, keep), dtype=i32, device=cache.device)
    lens = empty((seqs,), dtype=i32, device=cache.device)
    out = empty((seqs, heads, to * page_size), dtype=sv["f32"], device=cache.device)
    code = _lib.gptq_kv4_evict(cache.data_ptr(), pages, heads, dim, page_size, table.data_ptr(), per, op, ostride,
                               kv_lens.data_ptr(), seqs, weights.data_ptr(), int(keep), min(int(recent), 2 ** 31 - 1),
                               kept.data_ptr(), lens.data_ptr(), out.data_ptr(), _raw_stream(sv, stream, dev))
    if code:
        raise GptqError("gptq_kv4_evict", code)
    return kept, lens, out
