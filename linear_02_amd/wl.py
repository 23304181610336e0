"""Python binding of libwl (the C ABI in include/wl.h).

Argument marshalling only: every function here checks tensor dtypes, shapes
and devices, passes raw device pointers and the current HIP stream to the
library, and returns the output tensor. All arithmetic runs in the library's
HIP kernels; there is no fallback of any kind. If libwl.so is missing the
import fails loudly (build it with ``python -m linear_02_amd.build``).

A theta is a dict with device tensors ``W0`` ([d_out][d_in]), ``s`` (fp32
[d_out] or None), ``U`` ([d_out][r]), ``V`` ([d_in][r]) and the ints ``d_in``,
``d_out``, ``r``, as drawn by ``linear_02_amd.inputs.theta`` and moved with
:func:`theta_to`. W0, U, V, x and the outputs are all bf16 or all fp32 (the
dtype of W0 picks the variant).
"""
from __future__ import annotations

import contextlib
import ctypes
import os

import torch

LIBRARY = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libwl.so")

OP_LINEAR, OP_QKV, OP_MLP = 0, 1, 2
ABI_VERSION = 6
# The first SYNC_BYTES of a projection workspace are the library's sync area:
# cleared by wl_workspace_init (new_workspace does it) before first use, then
# written only by the library's calls.
SYNC_BYTES = 9764864
# Bytes of the static workspace wl_linear_static uses on each device.
STATIC_SCRATCH_BYTES = 33554432
_FALLBACK_WORD = 511   # int64 word of the sync area counting decode workgroups that stopped waiting
STATUS = {0: "ok", 1: "invalid argument", 2: "unsupported", 3: "HIP error", 4: "workspace too small"}
WL_OK, WL_ERR_INVALID_ARG, WL_ERR_UNSUPPORTED, WL_ERR_HIP, WL_ERR_WORKSPACE = 0, 1, 2, 3, 4


class WlError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS.get(status, status)}: {message}")
        self.status = status


DTYPE_BF16, DTYPE_F32 = 0, 1
_CODES = {torch.bfloat16: DTYPE_BF16, torch.float32: DTYPE_F32}


class Theta(ctypes.Structure):
    _fields_ = [("W0", ctypes.c_void_p), ("s", ctypes.c_void_p), ("U", ctypes.c_void_p),
                ("V", ctypes.c_void_p), ("d_in", ctypes.c_int32), ("d_out", ctypes.c_int32),
                ("r", ctypes.c_int32), ("dtype", ctypes.c_int32)]


class Call(ctypes.Structure):
    _fields_ = [("op", ctypes.c_int32), ("th", ctypes.POINTER(Theta) * 3), ("x", ctypes.c_void_p),
                ("y", ctypes.c_void_p), ("T", ctypes.c_int32)]


STEP_GROUP_SHARED_W0 = 1

# The operations between the projections: norms, rotary positions, cache, attention.
OP_NORM, OP_ROPE, OP_CACHE_WRITE, OP_CACHE_READ, OP_ATTENTION = 3, 4, 5, 6, 7
# Those around a batch of a serving step: its plan, the latent cache, verification.
OP_BATCH_PLAN, OP_LATENT_WRITE, OP_LATENT_READ, OP_LATENT_ATTENTION, OP_VERIFY_DRAFTS = 16, 17, 18, 19, 20
LATENT_FORMS = {"auto": 0, "absorbed": 1, "expanded": 2}
VERIFY_LOGITS, VERIFY_PROBABILITIES = 0, 1
VERIFY_ROWS = 1024   # most rows of a sequence in wl_verify_drafts
ROPE_HALF, ROPE_INTERLEAVED = 0, 1
ROPE_SCALINGS = {"plain": 0, "linear": 1, "base": 2, "parts": 3}
MASKS = {"causal": 0, "tree": 1, "full": 2}
CACHE_FORMATS = {torch.bfloat16: 0, torch.float32: 1, torch.int8: 2, torch.float8_e4m3fn: 3}


def _struct(name: str, pointers: str, ints: str, floats: str = "") -> type:
    """A ctypes struct of pointers, then int32 fields, then fp32 ones."""
    fields = [(f, t) for names, t in ((pointers, ctypes.c_void_p), (ints, ctypes.c_int32), (floats, ctypes.c_float))
              for f in names.split()]
    return type(name, (ctypes.Structure,), {"_fields_": fields})


NormArgs = _struct("NormArgs", "x y post pre gate x_out n_out", "T d gate_ld dtype", "eps offset res_scale branch_scale")
Rotary = _struct("Rotary", "freq pos", "rot style", "scale")
RopeArgs = _struct("RopeArgs", "q k q_weight k_weight q_out k_out rotary",
                   "T n_q n_k d ldq ldk ldq_out ldk_out dtype", "eps offset")
CacheStruct = _struct("CacheStruct", "k v k_scale v_scale table", "n_pages page n_kv d n_seq max_pages format")
CacheWriteArgs = _struct("CacheWriteArgs", "cache k v q q_weight k_weight q_out seq slot rotary",
                         "T n_q ldk ldv ldq ldq_out dtype", "eps offset")
CacheReadArgs = _struct("CacheReadArgs", "cache seq slot k_out v_out", "T ldk ldv dtype")
AttentionArgs = _struct("AttentionArgs", "cache q o q_start kv_len tree q_pos",
                        "T n_q ldq ldo max_q max_kv mask window tree_words dtype", "scale")
BatchPlanArgs = _struct("BatchPlanArgs", "table held free_pages n_free past n_new q_start kv_len seq slot",
                        "T n_seq max_pages n_pages page")
LatentCacheStruct = _struct("LatentCacheStruct", "rows scale table", "n_pages page latent rot n_seq max_pages format")
LatentWriteArgs = _struct("LatentWriteArgs", "cache c norm q q_out seq slot rotary", "T n_q nope ldc ldq ldq_out dtype",
                          "eps offset")
LatentReadArgs = _struct("LatentReadArgs", "cache seq slot out", "T ld dtype")
LatentAttentionArgs = _struct("LatentAttentionArgs", "cache q w o q_start kv_len tree q_pos",
                              "T n_q nope value ldq ldo max_q max_kv mask window tree_words dtype form", "scale")
VerifyArgs = _struct("VerifyArgs", "target draft token q_start parent u temperature out path n_out len",
                     "T n_seq vocab ld_target ld_draft max_q kind dtype")


class StepOp(ctypes.Structure):
    _fields_ = [("op", ctypes.c_int32), ("args", ctypes.c_void_p)]


def _load(path: str = LIBRARY) -> ctypes.CDLL:
    if not os.path.exists(path):
        raise ImportError(f"{path} is not built; run `python -m linear_02_amd.build`")
    lib = ctypes.CDLL(path)
    P = ctypes.POINTER(Theta)
    vp, i32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
    lib.wl_workspace_bytes.argtypes = [i32, ctypes.POINTER(P), i32, i32]
    lib.wl_workspace_bytes.restype = sz
    lib.wl_linear.argtypes = [P, vp, vp, i32, vp, sz, vp]
    lib.wl_linear_static.argtypes = [P, vp, vp, i32, vp]
    lib.wl_qkv_fused.argtypes = [P, P, P, vp, vp, i32, vp, sz, vp]
    lib.wl_mlp_fused.argtypes = [P, P, P, vp, vp, i32, vp, sz, vp]
    lib.wl_materialize_weff.argtypes = [P, vp, vp]
    lib.wl_materialize_weff_batch.argtypes = [ctypes.POINTER(P), ctypes.POINTER(vp), i32, vp]
    lib.wl_materialize_weff_batch.restype = ctypes.c_int
    for name in ("wl_linear", "wl_linear_static", "wl_qkv_fused", "wl_mlp_fused", "wl_materialize_weff"):
        getattr(lib, name).restype = ctypes.c_int
    lib.wl_set_regime.argtypes = [i32]
    lib.wl_set_regime.restype = i32
    lib.wl_set_spin_limit.argtypes = [i32]
    lib.wl_set_spin_limit.restype = i32
    lib.wl_status_str.argtypes = [ctypes.c_int]
    lib.wl_status_str.restype = ctypes.c_char_p
    lib.wl_last_error.argtypes = []
    lib.wl_last_error.restype = ctypes.c_char_p
    lib.wl_abi_version.argtypes = []
    lib.wl_abi_version.restype = i32
    lib.wl_bundle_size.argtypes = [ctypes.POINTER(P), i32, ctypes.POINTER(sz), ctypes.POINTER(sz)]
    lib.wl_bundle_size.restype = ctypes.c_int
    lib.wl_rel_frob_workspace_bytes.argtypes = [ctypes.c_int64]
    lib.wl_rel_frob_workspace_bytes.restype = sz
    lib.wl_relative_frobenius_error.argtypes = [vp, vp, ctypes.c_int64, vp, vp, sz, vp]
    lib.wl_relative_frobenius_error.restype = ctypes.c_int
    lib.wl_step_workspace_bytes.argtypes = [ctypes.POINTER(Call), i32]
    lib.wl_step_workspace_bytes.restype = sz
    lib.wl_step_create.argtypes = [ctypes.POINTER(Call), i32, i32, vp, sz, ctypes.POINTER(vp)]
    lib.wl_step_create.restype = ctypes.c_int
    lib.wl_step_launch.argtypes = [vp, vp]
    lib.wl_step_launch.restype = ctypes.c_int
    lib.wl_step_destroy.argtypes = [vp]
    lib.wl_step_destroy.restype = ctypes.c_int
    for name, args in (("wl_norm_residual", NormArgs), ("wl_rope", RopeArgs), ("wl_cache_write", CacheWriteArgs),
                       ("wl_cache_read", CacheReadArgs), ("wl_latent_write", LatentWriteArgs),
                       ("wl_latent_read", LatentReadArgs)):
        getattr(lib, name).argtypes = [ctypes.POINTER(args), vp]
        getattr(lib, name).restype = ctypes.c_int
    for name, args in (("wl_batch_plan", BatchPlanArgs), ("wl_latent_attention", LatentAttentionArgs),
                       ("wl_verify_drafts", VerifyArgs)):
        getattr(lib, name + "_workspace_bytes").argtypes = [ctypes.POINTER(args)]
        getattr(lib, name + "_workspace_bytes").restype = sz
        getattr(lib, name).argtypes = [ctypes.POINTER(args), vp, sz, vp]
        getattr(lib, name).restype = ctypes.c_int
    lib.wl_rope_frequencies.argtypes = [i32, ctypes.c_double, i32] + [ctypes.c_double] * 4 + \
        [ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_float)]
    lib.wl_rope_frequencies.restype = ctypes.c_int
    lib.wl_attention_workspace_bytes.argtypes = [ctypes.POINTER(AttentionArgs)]
    lib.wl_attention_workspace_bytes.restype = sz
    lib.wl_attention.argtypes = [ctypes.POINTER(AttentionArgs), vp, sz, vp]
    lib.wl_attention.restype = ctypes.c_int
    lib.wl_step_ops_workspace_bytes.argtypes = [ctypes.POINTER(StepOp), i32]
    lib.wl_step_ops_workspace_bytes.restype = sz
    lib.wl_step_create_ops.argtypes = [ctypes.POINTER(StepOp), i32, vp, sz, ctypes.POINTER(vp)]
    lib.wl_step_create_ops.restype = ctypes.c_int
    # Of the HIP runtime that the library is linked to.
    lib.hipStreamGetCaptureInfo.argtypes = [vp, ctypes.POINTER(ctypes.c_int), ctypes.POINTER(ctypes.c_ulonglong)]
    lib.hipStreamGetCaptureInfo.restype = ctypes.c_int
    lib.wl_workspace_init.argtypes = [vp, sz, vp]
    lib.wl_workspace_init.restype = ctypes.c_int
    lib.wl_sync_bytes.argtypes = []
    lib.wl_sync_bytes.restype = sz
    if lib.wl_abi_version() != ABI_VERSION or lib.wl_sync_bytes() != SYNC_BYTES:
        raise ImportError(f"{path}: ABI version {lib.wl_abi_version()} / sync area {lib.wl_sync_bytes()} bytes, "
                          f"this binding expects {ABI_VERSION} / {SYNC_BYTES}; rebuild the library")
    return lib


lib = _load()


def _check(status: int) -> None:
    if status != 0:
        raise WlError(status, lib.wl_last_error().decode())


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


# The handle of a device's current stream, without building a Stream object.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)


def _index(device: torch.device) -> int:
    return device.index if device.index is not None else torch.cuda.current_device()


def _stream(device: torch.device):
    return ctypes.c_void_p(_raw_stream(_index(device)))


def _on(device: torch.device):
    """Context in which a device is the current one."""
    if device.index is None or device.index == torch.cuda.current_device():
        return contextlib.nullcontext()
    return torch.cuda.device(device)


def _capture(stream: int) -> int | None:
    """Id of the graph capture that a stream is part of, None if it is in none."""
    if not stream:
        return None   # the default stream cannot be captured
    status, ident = ctypes.c_int(0), ctypes.c_ulonglong(0)
    lib.hipStreamGetCaptureInfo(stream, ctypes.byref(status), ctypes.byref(ident))
    return ident.value if status.value == 1 else None


def theta_to(th: dict, device) -> dict:
    """Copy a theta's tensors to ``device`` (contiguous); ints are kept."""
    out = dict(th)
    for key in ("W0", "s", "U", "V"):
        if th.get(key) is not None:
            out[key] = th[key].to(device).contiguous()
    return out


def make_theta(th: dict) -> Theta:
    """The C struct of a theta dict (device tensors). The dict keeps them alive."""
    W0, s, U, V = th["W0"], th.get("s"), th.get("U"), th.get("V")
    d_in, d_out, r = int(th["d_in"]), int(th["d_out"]), int(th["r"])
    if W0.dtype not in _CODES or not W0.is_contiguous() or tuple(W0.shape) != (d_out, d_in):
        raise ValueError("W0 must be a contiguous bf16 or fp32 [d_out][d_in] tensor")
    if s is not None and (s.dtype != torch.float32 or not s.is_contiguous() or s.numel() != d_out):
        raise ValueError("s must be a contiguous fp32 [d_out] tensor or None")
    if r > 0:
        for name, t, rows in (("U", U, d_out), ("V", V, d_in)):
            if t is None or t.dtype != W0.dtype or not t.is_contiguous() or tuple(t.shape) != (rows, r):
                raise ValueError(f"{name} must be a contiguous [{rows}][{r}] tensor of W0's dtype")
    return Theta(_ptr(W0), _ptr(s), _ptr(U) if r > 0 else None, _ptr(V) if r > 0 else None, d_in, d_out, r,
                 _CODES[W0.dtype])


def workspace_bytes(op: int, thetas: list, T: int) -> int:
    structs = [make_theta(t) for t in thetas]
    arr = (ctypes.POINTER(Theta) * len(structs))(*[ctypes.pointer(s) for s in structs])
    return int(lib.wl_workspace_bytes(op, arr, len(structs), T))


def workspace_init(ws: torch.Tensor) -> None:
    """Clear the sync area of a projection workspace (wl_workspace_init, on the
    current stream)."""
    _check(lib.wl_workspace_init(_ptr(ws), ws.numel() * ws.element_size(), _stream(ws.device)))


def new_workspace(nbytes: int, device) -> torch.Tensor:
    """A projection workspace of at least nbytes (and at least the sync area),
    prepared by wl_workspace_init."""
    ws = _bytes(max(int(nbytes), SYNC_BYTES), torch.device(device))
    workspace_init(ws)
    return ws


def _bytes(nbytes: int, device: torch.device) -> torch.Tensor:
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


class Workspace:
    """A device workspace per (device, stream) that grows on demand, prepared by
    wl_workspace_init when allocated.

    Calls on one stream run in order, so they can share one workspace. Calls that a
    graph capture records share one of that capture's own, allocated and prepared
    within it: under torch.cuda.graph its memory is the graph's, so that no later
    call can replace it, and no replay finds it prepared by another graph alone or in
    use by one. Pass ``ws`` to a call to leave the preparing out of the graph, and in a
    capture that is not torch's, whose graph owns no memory."""

    def __init__(self):
        self._bufs: dict = {}
        self._captured: dict = {}   # the capture that a stream was last in, its workspace

    def get(self, device: torch.device, nbytes: int) -> torch.Tensor | None:
        if nbytes == 0:
            return None
        stream = _raw_stream(_index(device))
        key, capture = (device.index, stream), _capture(stream)
        if capture is None:
            buf = self._bufs.get(key)
        else:
            of, buf = self._captured.pop(key, (None, None))
            buf = buf if of == capture else None
        if buf is None or buf.numel() < nbytes:
            buf = new_workspace(max(nbytes, 1 << 20), device)
        if capture is None:
            self._bufs[key] = buf
        else:
            self._captured[key] = capture, buf
        return buf

    def scratch(self, device: torch.device, nbytes: int) -> torch.Tensor | None:
        """get() for a call that leaves the sync area alone: in a capture, memory of the
        graph's for this call, with nothing to prepare."""
        if nbytes and _capture(_raw_stream(_index(device))) is not None:
            return _bytes(nbytes, device)
        return self.get(device, nbytes)


WORKSPACE = Workspace()


def _io(x: torch.Tensor, d_in: int, dtype: torch.dtype) -> int:
    if x.dtype != dtype or not x.is_contiguous() or x.dim() != 2 or x.shape[1] != d_in:
        raise ValueError(f"x must be a contiguous {dtype} [T][{d_in}] tensor")
    if not x.is_cuda:
        raise ValueError("x must be a device tensor")
    return x.shape[0]


def wl_linear(th: dict, x: torch.Tensor, y: torch.Tensor | None = None, ws: torch.Tensor | None = None):
    """y = s (.) (W0 x) + U (V^T x), [T][d_out] of W0's dtype."""
    T = _io(x, int(th["d_in"]), th["W0"].dtype)
    st = make_theta(th)
    if y is None:
        y = torch.empty(T, int(th["d_out"]), dtype=th["W0"].dtype, device=x.device)
    need = workspace_bytes(OP_LINEAR, [th], T)
    ws = ws if ws is not None else WORKSPACE.get(x.device, need)
    _check(lib.wl_linear(ctypes.byref(st), _ptr(x), _ptr(y), T, _ptr(ws),
                         0 if ws is None else ws.numel() * ws.element_size(), _stream(x.device)))
    return y


def wl_linear_static(th: dict, x: torch.Tensor, y: torch.Tensor | None = None):
    """wl_linear with the library's static workspace (no workspace argument;
    the C call allocates no device memory). y is allocated here when not given."""
    T = _io(x, int(th["d_in"]), th["W0"].dtype)
    st = make_theta(th)
    if y is None:
        y = torch.empty(T, int(th["d_out"]), dtype=th["W0"].dtype, device=x.device)
    _check(lib.wl_linear_static(ctypes.byref(st), _ptr(x), _ptr(y), T, _stream(x.device)))
    return y


def wl_qkv_fused(q: dict, k: dict, v: dict, x: torch.Tensor, y: torch.Tensor | None = None,
                 ws: torch.Tensor | None = None):
    """Q | K | V side by side, [T][dq + dk + dv] of the thetas' dtype."""
    T = _io(x, int(q["d_in"]), q["W0"].dtype)
    sq, sk, sv = make_theta(q), make_theta(k), make_theta(v)
    width = int(q["d_out"]) + int(k["d_out"]) + int(v["d_out"])
    if y is None:
        y = torch.empty(T, width, dtype=q["W0"].dtype, device=x.device)
    need = workspace_bytes(OP_QKV, [q, k, v], T)
    ws = ws if ws is not None else WORKSPACE.get(x.device, need)
    _check(lib.wl_qkv_fused(ctypes.byref(sq), ctypes.byref(sk), ctypes.byref(sv), _ptr(x), _ptr(y), T,
                            _ptr(ws), 0 if ws is None else ws.numel() * ws.element_size(), _stream(x.device)))
    return y


def wl_mlp_fused(gate: dict, up: dict, down: dict, x: torch.Tensor, y: torch.Tensor | None = None,
                 ws: torch.Tensor | None = None):
    """down(round(gelu_tanh(gate x) * up x)), [T][down.d_out] of the thetas' dtype."""
    T = _io(x, int(gate["d_in"]), gate["W0"].dtype)
    sg, su, sd = make_theta(gate), make_theta(up), make_theta(down)
    if y is None:
        y = torch.empty(T, int(down["d_out"]), dtype=gate["W0"].dtype, device=x.device)
    need = workspace_bytes(OP_MLP, [gate, up, down], T)
    ws = ws if ws is not None else WORKSPACE.get(x.device, need)
    _check(lib.wl_mlp_fused(ctypes.byref(sg), ctypes.byref(su), ctypes.byref(sd), _ptr(x), _ptr(y), T,
                            _ptr(ws), 0 if ws is None else ws.numel() * ws.element_size(), _stream(x.device)))
    return y


def wl_materialize_weff(th: dict, W_eff: torch.Tensor | None = None):
    """W_eff = round(s (.) W0 + U V^T), [d_out][d_in] of W0's dtype."""
    st = make_theta(th)
    dev = th["W0"].device
    if W_eff is None:
        W_eff = torch.empty(int(th["d_out"]), int(th["d_in"]), dtype=th["W0"].dtype, device=dev)
    _check(lib.wl_materialize_weff(ctypes.byref(st), _ptr(W_eff), _stream(dev)))
    return W_eff


def wl_materialize_weff_batch(thetas: list, W_effs: list | None = None) -> list:
    """wl_materialize_weff for every theta in one launch per eight; returns the
    W_eff tensors (allocated when W_effs is None)."""
    if not thetas:
        return []
    dev = thetas[0]["W0"].device
    if W_effs is None:
        W_effs = [torch.empty(int(t["d_out"]), int(t["d_in"]), dtype=t["W0"].dtype, device=dev) for t in thetas]
    structs = [make_theta(t) for t in thetas]
    arr = (ctypes.POINTER(Theta) * len(structs))(*[ctypes.pointer(st) for st in structs])
    outs = (ctypes.c_void_p * len(W_effs))(*[_ptr(w) for w in W_effs])
    _check(lib.wl_materialize_weff_batch(arr, outs, len(structs), _stream(dev)))
    return W_effs


def bundle_size(thetas: list) -> tuple:
    """(bundle bytes, dense bytes) of a set of thetas: each distinct W0 counted once,
    s, U and V per theta, against the dense weights (of the thetas' dtype) they stand for."""
    structs = [make_theta(t) for t in thetas]
    arr = (ctypes.POINTER(Theta) * len(structs))(*[ctypes.pointer(st) for st in structs])
    b, d = ctypes.c_size_t(0), ctypes.c_size_t(0)
    _check(lib.wl_bundle_size(arr, len(structs), ctypes.byref(b), ctypes.byref(d)))
    return int(b.value), int(d.value)


def relative_frobenius_error(W: torch.Tensor, R: torch.Tensor) -> float:
    """||W - R||_F / ||W||_F of two bf16 device tensors of equal size (waits for the
    result)."""
    for name, t in (("W", W), ("R", R)):
        if t.dtype != torch.bfloat16 or not t.is_contiguous() or not t.is_cuda:
            raise ValueError(f"{name} must be a contiguous bf16 device tensor")
    if W.numel() != R.numel():
        raise ValueError("W and R must have the same number of elements")
    n = W.numel()
    out = torch.empty(1, dtype=torch.float64, device=W.device)
    ws = torch.empty(max(int(lib.wl_rel_frob_workspace_bytes(n)), 256), dtype=torch.uint8, device=W.device)
    _check(lib.wl_relative_frobenius_error(_ptr(W), _ptr(R), n, _ptr(out), _ptr(ws),
                                            ws.numel(), _stream(W.device)))
    return float(out.item())


REGIME_AUTO, REGIME_GEMV, REGIME_MFMA, REGIME_GEMV_TWO_LAUNCH, REGIME_SKINNY, REGIME_GEMV_MLP_SPLIT = 0, 1, 2, 3, 4, 5


def set_regime(regime: int) -> int:
    """0 auto, 1 decode kernels (the MLP in one launch where it applies), 2
    matrix-core GEMM, 3 decode GEMV always after a separate V^T x launch, 4
    few-token split path, 5 as 1 with the MLP as two launches, 6 as 2 with
    V^T x always in a launch of its own and the rank term in the GEMM epilogue;
    returns the previous setting (wl_testing.h)."""
    prev = int(lib.wl_set_regime(regime))
    if prev < 0:
        raise ValueError(f"regime {regime} is not one of 0 to 6")
    return prev


def set_spin_limit(polls: int) -> int:
    """Times a decode workgroup reads each group of in-launch V^T x words before
    it computes V^T x itself (0: at once); returns the previous setting."""
    prev = int(lib.wl_set_spin_limit(polls))
    if prev < 0:
        raise ValueError(f"spin limit {polls} is negative")
    return prev


def fallback_count(ws: torch.Tensor) -> int:
    """Decode workgroups, over all calls on workspace ``ws`` so far, whose wait
    for the in-launch V^T x ran out (a counter in the sync area); waits for the
    device."""
    w = _FALLBACK_WORD * 8
    return int(ws[w:w + 8].view(torch.int64).item())


def abi_version() -> int:
    return int(lib.wl_abi_version())


def _one_device(device: torch.device | None, other: torch.device, i: int) -> torch.device:
    if device is not None and other != device:
        raise ValueError(f"call {i} is on {other}, those before it on {device}")
    return other


class Step:
    """A decode step: a fixed list of calls that the library records once into a
    HIP graph (wl_step_create) and launches with one call.

    calls: (op, thetas, x, y) tuples, op one of OP_LINEAR (one theta), OP_QKV
    (Q, K, V), OP_MLP (gate, up, down); tensors of one device, which must stay alive
    while the step exists (the step keeps references). group_shared_w0 launches
    calls that share their first theta's W0 back to back (independent calls
    only)."""

    def __init__(self, calls, ws: torch.Tensor | None = None, group_shared_w0: bool = False):
        n = len(calls)
        arr = (Call * n)()
        self._keep = []
        device = None
        for i, (op, thetas, x, y) in enumerate(calls):
            if len(thetas) != (1 if op == OP_LINEAR else 3):
                raise ValueError(f"call {i}: {len(thetas)} thetas for op {op}")
            T = _io(x, int(thetas[0]["d_in"]), thetas[0]["W0"].dtype)
            structs = [make_theta(t) for t in thetas]
            self._keep += [structs, [dict(t) for t in thetas], x, y]   # the thetas are the caller's to reuse
            arr[i].op = op
            for j, st in enumerate(structs):
                arr[i].th[j] = ctypes.pointer(st)
            arr[i].x, arr[i].y, arr[i].T = _ptr(x), _ptr(y), T
            device = _one_device(device, x.device, i)
        need = int(lib.wl_step_workspace_bytes(arr, n))
        if need == 0:
            raise ValueError("invalid calls for a step")
        self._create(lambda *a: lib.wl_step_create(arr, n, STEP_GROUP_SHARED_W0 if group_shared_w0 else 0, *a), need, ws, device)

    def _create(self, make, need: int, ws: torch.Tensor | None, device: torch.device) -> None:
        """make(workspace, its bytes, handle) on the calls' device."""
        h = ctypes.c_void_p()
        with _on(device):
            self.ws = ws if ws is not None else new_workspace(need, device)
            self.device = device
            _check(make(_ptr(self.ws), self.ws.numel() * self.ws.element_size(), ctypes.byref(h)))
        self.handle = h

    def launch(self) -> None:
        with _on(self.device):
            _check(lib.wl_step_launch(self.handle, _stream(self.device)))

    def close(self) -> None:
        if getattr(self, "handle", None) is not None and self.handle.value:
            with _on(self.device):
                torch.cuda.current_stream(self.device).synchronize()
                lib.wl_step_destroy(self.handle)
        self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# ---- the operations between the projections ------------------------------------
#
# Each has a ``..._call`` that checks its tensors, allocates the outputs that are
# not given and returns an OpCall, and a function that makes the call and
# launches it on the current stream. An OpCall can be launched again (new values
# in the same tensors) or recorded with others in a LayerStep.


# Workspace bytes of the operations that take a workspace.
_WORKSPACE_BYTES = {OP_ATTENTION: lib.wl_attention_workspace_bytes, OP_BATCH_PLAN: lib.wl_batch_plan_workspace_bytes,
                    OP_LATENT_ATTENTION: lib.wl_latent_attention_workspace_bytes,
                    OP_VERIFY_DRAFTS: lib.wl_verify_drafts_workspace_bytes}


class OpCall:
    """A checked call of one operation: ``out`` are its outputs, ``launch`` runs it
    on the current stream of its device. Keeps its tensors alive."""

    __slots__ = ("op", "args", "out", "device", "fn", "ws", "keep")

    def __init__(self, op, fn, args, out, device, keep, ws=None):
        self.op, self.fn, self.args, self.out, self.device, self.keep, self.ws = op, fn, args, out, device, keep, ws

    def launch(self):
        if self.device.index != torch.cuda.current_device():
            with torch.cuda.device(self.device):
                return self._launch()
        return self._launch()

    def _launch(self):
        stream = _raw_stream(self.device.index)
        need_of = _WORKSPACE_BYTES.get(self.op)
        if need_of is None:
            status = self.fn(self.args, stream)
        else:
            need = need_of(self.args)
            ws = self.ws if self.ws is not None else WORKSPACE.scratch(self.device, need)
            status = self.fn(self.args, _ptr(ws), 0 if ws is None else ws.numel() * ws.element_size(), stream)
        if status:
            _check(status)
        return self.out


def _tensor(t, name: str, like: torch.Tensor, dtype=None) -> None:
    if t.get_device() != like.get_device() or not t.is_cuda:
        raise ValueError(f"{name} must be on the device of the call's first tensor ({like.device})")
    if t.dtype is not (dtype or like.dtype):
        raise ValueError(f"{name} must be {dtype or like.dtype}")


def _matrix(t, name: str, like: torch.Tensor, T: int, width: int) -> int:
    """Row stride of a [T][width] tensor whose rows are contiguous."""
    if t is not like:
        _tensor(t, name, like)
    if t.shape != (T, width):
        raise ValueError(f"{name} must be [{T}][{width}]")
    ld, one = t.stride()
    if one != 1 and width > 1:
        raise ValueError(f"{name} must have contiguous rows")
    return ld if T > 1 else width


def _vector(t, name: str, like: torch.Tensor, n: int, dtype=None):
    if t is None:
        return None
    if t.dtype is not (dtype or like.dtype) or t.get_device() != like.get_device():
        _tensor(t, name, like, dtype)
    if t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous with {n} elements")
    return t.data_ptr()


def _first(t, name: str) -> torch.Tensor:
    if t.dtype not in _CODES or not t.is_cuda or t.dim() != 2:
        raise ValueError(f"{name} must be a bf16 or fp32 device matrix")
    return t


def norm_call(x, y=None, post=None, pre=None, gate=None, eps: float = 1e-6, offset: float = 0.0,
              res_scale: float = 1.0, branch_scale: float = 1.0, x_out=None, n_out=None, want_x: bool = True,
              want_n: bool = True) -> OpCall:
    """wl_norm_residual as an OpCall; out = (x_out, n_out). want_x / want_n False
    leave that output out (None)."""
    T, d = _first(x, "x").shape
    for name, t in (("x", x), ("y", y), ("x_out", x_out), ("n_out", n_out)):
        if t is not None and _matrix(t, name, x, T, d) != d:
            raise ValueError(f"{name} must be contiguous")
    gate_ld = 0
    if gate is not None:
        if gate.dim() == 1:
            _vector(gate, "gate", x, d)
        else:
            gate_ld = _matrix(gate, "gate", x, T, d)
    if want_x and x_out is None:
        x_out = torch.empty_like(x)
    if want_n and n_out is None:
        n_out = torch.empty_like(x)
    args = NormArgs(x.data_ptr(), _ptr(y), _vector(post, "post", x, d), _vector(pre, "pre", x, d), _ptr(gate),
                    _ptr(x_out), _ptr(n_out), T, d, gate_ld, _CODES[x.dtype], eps, offset, res_scale, branch_scale)
    return OpCall(OP_NORM, lib.wl_norm_residual, args, (x_out, n_out), x.device, (x, y, post, pre, gate))


def wl_norm_residual(x, **kw):
    """(x', n): p = rms(y) (post + offset), x' = res_scale x + branch_scale gate p,
    n = rms(x') (pre + offset); see norm_call for the arguments."""
    return norm_call(x, **kw).launch()


def rope_frequencies(rot: int, base: float = 10000.0, scaling: str = "plain", factor: float = 1.0,
                     original: float = 4096.0, slow: float = 1.0, fast: float = 32.0, device="cuda"):
    """(freq, scale) of Rope for ``rot`` rotated elements (wl_rope_frequencies):
    scaling "plain", "linear", "base" or "parts"."""
    if scaling not in ROPE_SCALINGS:
        raise ValueError(f"scaling {scaling!r} is not one of {sorted(ROPE_SCALINGS)}")
    buf, scale = (ctypes.c_double * max(int(rot) // 2, 1))(), ctypes.c_float()
    _check(lib.wl_rope_frequencies(int(rot), base, ROPE_SCALINGS[scaling], factor, original, slow, fast, buf,
                                   ctypes.byref(scale)))
    return torch.tensor(list(buf), dtype=torch.float64, device=device), float(scale.value)


class Rope:
    """How heads are rotated: fp64 radians per position of every pair, the pairs'
    style, a factor on cos and sin."""

    __slots__ = ("freq", "interleaved", "scale")

    def __init__(self, freq: torch.Tensor, interleaved: bool = False, scale: float = 1.0):
        self.freq, self.interleaved, self.scale = freq, interleaved, scale

    def struct(self, pos, T: int, like: torch.Tensor):
        f = _vector(self.freq, "freq", like, self.freq.numel(), torch.float64)
        rot = Rotary(f, _vector(pos, "pos", like, T, torch.int32), 2 * self.freq.numel(),
                     ROPE_INTERLEAVED if self.interleaved else ROPE_HALF, self.scale)
        rot.freq_tensor = self.freq
        return rot


def _at(struct) -> int | None:
    return None if struct is None else ctypes.addressof(struct)


def _heads(t, name: str, d: int) -> int:
    if d < 1 or t.dim() != 2 or t.shape[1] % d:
        raise ValueError(f"{name} must be a matrix of whole heads of {d}")
    return t.shape[1] // d


def rope_call(q, k, pos, rope: Rope | None, d: int, q_norm=None, k_norm=None, eps: float = 1e-6,
              offset: float = 0.0, q_out=None, k_out=None) -> OpCall:
    """wl_rope as an OpCall; out = (q_out, k_out). q or k may be None; both may be
    column ranges of one wider matrix (Q/K/V side by side), and their own outputs."""
    first = _first(q if q is not None else k, "q" if q is not None else "k")
    T = first.shape[0]
    n, ld, ldo, outs = [0, 0], [0, 0], [0, 0], [q_out, k_out]
    for i, (t, name) in enumerate(((q, "q"), (k, "k"))):
        if t is None:
            continue
        n[i] = _heads(t, name, d)
        ld[i] = _matrix(t, name, first, T, n[i] * d)
        if outs[i] is None:
            outs[i] = t.new_empty((T, n[i] * d))
        ldo[i] = _matrix(outs[i], name + "_out", first, T, n[i] * d)
    rot = None if rope is None else rope.struct(pos, T, first)
    args = RopeArgs(_ptr(q), _ptr(k), _vector(q_norm, "q_norm", first, d), _vector(k_norm, "k_norm", first, d),
                    _ptr(outs[0]), _ptr(outs[1]), _at(rot), T, n[0], n[1], d, ld[0], ld[1], ldo[0], ldo[1],
                    _CODES[first.dtype], eps, offset)
    return OpCall(OP_ROPE, lib.wl_rope, args, tuple(outs), first.device, (q, k, pos, rot, q_norm, k_norm))


def wl_rope(q, k, pos, rope, d, **kw):
    """(q, k) rotated by their positions, each head normalised first where q_norm /
    k_norm are given; see rope_call."""
    return rope_call(q, k, pos, rope, d, **kw).launch()


class Cache:
    """A paged cache of keys and values: k, v [n_pages][n_kv][page][d] (bf16, fp32,
    int8 or float8_e4m3fn), table int32 [n_seq][max_pages] of page numbers, and
    fp32 [n_pages][n_kv][page] scales for the one-byte types."""

    __slots__ = ("k", "v", "table", "k_scale", "v_scale", "struct")

    def __init__(self, k, v, table, k_scale=None, v_scale=None):
        if k.dtype not in CACHE_FORMATS or k.dim() != 4 or not k.is_contiguous() or not k.is_cuda:
            raise ValueError("k must be a contiguous [n_pages][n_kv][page][d] device tensor of a cache type")
        _tensor(v, "v", k)
        if v.shape != k.shape or not v.is_contiguous():
            raise ValueError("v must be contiguous and shaped as k")
        _tensor(table, "table", k, torch.int32)
        if table.dim() != 2 or not table.is_contiguous():
            raise ValueError("table must be a contiguous [n_seq][max_pages] tensor")
        n_pages, n_kv, page, d = k.shape
        scales = [None, None]
        if k.dtype.itemsize == 1:
            for i, (t, name) in enumerate(((k_scale, "k_scale"), (v_scale, "v_scale"))):
                if t is None or t.shape != k.shape[:3]:
                    raise ValueError(f"{name} must be [n_pages][n_kv][page]")
                scales[i] = _vector(t, name, k, t.numel(), torch.float32)
        self.k, self.v, self.table, self.k_scale, self.v_scale = k, v, table, k_scale, v_scale
        self.struct = CacheStruct(k.data_ptr(), v.data_ptr(), scales[0], scales[1], table.data_ptr(), n_pages, page,
                                  n_kv, d, table.shape[0], table.shape[1], CACHE_FORMATS[k.dtype])
        self.struct.tensors = k, v, table, k_scale, v_scale   # what it points into, for calls that hold it


def new_cache(n_pages: int, n_kv: int, page: int, d: int, table: torch.Tensor, dtype=torch.bfloat16) -> Cache:
    """A Cache of uninitialised pages on the table's device."""
    shape = (n_pages, n_kv, page, d)
    k, v = (torch.empty(shape, dtype=dtype, device=table.device) for _ in range(2))
    scales = [torch.empty(shape[:3], dtype=torch.float32, device=table.device) if dtype.itemsize == 1 else None
              for _ in range(2)]
    return Cache(k, v, table, *scales)


def cache_write_call(cache: Cache, k, v, seq, slot, q=None, rope: Rope | None = None, pos=None, q_norm=None,
                     k_norm=None, eps: float = 1e-6, offset: float = 0.0, q_out=None) -> OpCall:
    """wl_cache_write as an OpCall; out = q_out (None without q). pos None: the slots
    are the positions."""
    c = cache.struct
    T = _first(k, "k").shape[0]
    width = c.n_kv * c.d
    _tensor(cache.k, "the cache", k, cache.k.dtype)
    n_q = ldq = ldo = 0
    if q is not None:
        n_q = _heads(q, "q", c.d)
        ldq = _matrix(q, "q", k, T, n_q * c.d)
        if q_out is None:
            q_out = q.new_empty((T, n_q * c.d))
        ldo = _matrix(q_out, "q_out", k, T, n_q * c.d)
    rot = None if rope is None else rope.struct(pos, T, k)
    args = CacheWriteArgs(_at(c), k.data_ptr(), v.data_ptr(), _ptr(q), _vector(q_norm, "q_norm", k, c.d),
                          _vector(k_norm, "k_norm", k, c.d), _ptr(q_out), _vector(seq, "seq", k, T, torch.int32),
                          _vector(slot, "slot", k, T, torch.int32), _at(rot), T, n_q, _matrix(k, "k", k, T, width),
                          _matrix(v, "v", k, T, width), ldq, ldo, _CODES[k.dtype], eps, offset)
    return OpCall(OP_CACHE_WRITE, lib.wl_cache_write, args, q_out, k.device,
                  (c, k, v, seq, slot, q, rot, pos, q_norm, k_norm))


def wl_cache_write(cache, k, v, seq, slot, **kw):
    """Writes the tokens' K and V into the cache, K (and q beside it) normalised and
    rotated on the way; returns the rotated q, or None. See cache_write_call."""
    return cache_write_call(cache, k, v, seq, slot, **kw).launch()


def cache_read_call(cache: Cache, seq, slot, dtype: torch.dtype | None = None, k_out=None, v_out=None) -> OpCall:
    """wl_cache_read as an OpCall; out = (k, v), [T][n_kv * d] of dtype (None: fp32
    for an fp32 cache, else bf16). Rows of tokens without a place in the cache keep
    what the outputs held (new ones are uninitialised)."""
    c, T = cache.struct, seq.numel()
    if dtype is None:
        dtype = torch.float32 if cache.k.dtype == torch.float32 else torch.bfloat16
    outs = [t if t is not None else cache.k.new_empty((T, c.n_kv * c.d), dtype=dtype) for t in (k_out, v_out)]
    first = _first(outs[0], "k_out")
    _tensor(first, "k_out", cache.k, dtype)
    args = CacheReadArgs(_at(c), _vector(seq, "seq", first, T, torch.int32), _vector(slot, "slot", first, T, torch.int32),
                         outs[0].data_ptr(), outs[1].data_ptr(), T, _matrix(outs[0], "k_out", first, T, c.n_kv * c.d),
                         _matrix(outs[1], "v_out", first, T, c.n_kv * c.d), _CODES[dtype])
    return OpCall(OP_CACHE_READ, lib.wl_cache_read, args, tuple(outs), first.device, (c, seq, slot))


def wl_cache_read(cache, seq, slot, **kw):
    """(k, v) of the tokens at (seq, slot), read back from the cache."""
    return cache_read_call(cache, seq, slot, **kw).launch()


def attention_call(q, cache: Cache, q_start, kv_len, max_q: int, max_kv: int, scale: float, mask: str | None = None,
                   window: int = 0, tree=None, q_pos=None, o=None, ws: torch.Tensor | None = None) -> OpCall:
    """wl_attention as an OpCall; out = o. mask: "causal" (the default), "full", or
    "tree" (the default where ``tree``, int32 [T][words], is given)."""
    c = cache.struct
    T = _first(q, "q").shape[0]
    n_q = _heads(q, "q", c.d)
    _tensor(cache.k, "the cache", q, cache.k.dtype)
    if o is None:
        o = q.new_empty((T, n_q * c.d))
    mask = mask or ("causal" if tree is None else "tree")
    if mask not in MASKS:
        raise ValueError(f"mask {mask!r} is not one of {sorted(MASKS)}")
    if (tree is None) == (mask == "tree"):
        raise ValueError("tree goes with mask='tree'")
    words = 0
    if tree is not None:
        if tree.dim() != 2 or tree.shape[0] != T:
            raise ValueError(f"tree must be [{T}][words]")
        words = tree.shape[1]
    elif q_pos is not None:
        raise ValueError("q_pos goes with mask='tree'")
    n_seq = c.n_seq
    args = AttentionArgs(_at(c), q.data_ptr(), o.data_ptr(), _vector(q_start, "q_start", q, n_seq + 1, torch.int32),
                         _vector(kv_len, "kv_len", q, n_seq, torch.int32),
                         _vector(tree, "tree", q, T * words, torch.int32), _vector(q_pos, "q_pos", q, T, torch.int32),
                         T, n_q, _matrix(q, "q", q, T, n_q * c.d), _matrix(o, "o", q, T, n_q * c.d), max_q, max_kv,
                         MASKS[mask], window, words, _CODES[q.dtype], scale)
    return OpCall(OP_ATTENTION, lib.wl_attention, args, o, q.device, (q, c, q_start, kv_len, tree, q_pos), ws)


def wl_attention(q, cache, q_start, kv_len, max_q, max_kv, scale, **kw):
    """softmax(scale q k) v of the tokens over the cache; see attention_call."""
    return attention_call(q, cache, q_start, kv_len, max_q, max_kv, scale, **kw).launch()


# ---- around a batch of a serving step ---------------------------------------------


class Pages:
    """The pages of a cache's sequences, as wl_batch_plan keeps them on the device:
    table int32 [n_seq][max_pages], held int32 [n_seq] pages of every row of it, free
    int32 [n_pages] (a stack, -1 above its top) and its height n_free int32 [1], of
    pages of ``page`` tokens. ``table`` is the cache's own."""

    __slots__ = ("table", "held", "free", "n_free", "page")

    def __init__(self, table, held, free, n_free, page: int):
        if table.dtype != torch.int32 or table.dim() != 2 or not table.is_contiguous() or not table.is_cuda:
            raise ValueError("table must be a contiguous int32 [n_seq][max_pages] device tensor")
        _vector(held, "held", table, table.shape[0])
        _vector(free, "free", table, free.numel())
        _vector(n_free, "n_free", table, 1)
        self.table, self.held, self.free, self.n_free, self.page = table, held, free, n_free, page


def new_pages(n_seq: int, max_pages: int, n_pages: int, page: int, device="cuda") -> Pages:
    """Pages of n_seq empty sequences, all of 0 .. n_pages - 1 free (the lowest first)."""
    i32 = dict(dtype=torch.int32, device=device)
    return Pages(torch.full((n_seq, max_pages), -1, **i32), torch.zeros(n_seq, **i32),
                 torch.arange(n_pages - 1, -1, -1, **i32), torch.full((1,), n_pages, **i32), page)


def batch_plan_call(pages: Pages, past, n_new, T: int, q_start=None, kv_len=None, seq=None, slot=None,
                    ws: torch.Tensor | None = None) -> OpCall:
    """wl_batch_plan as an OpCall; out = (q_start, kv_len, seq, slot) of a batch of T rows."""
    t = pages.table
    n_seq, max_pages = t.shape
    q_start = t.new_empty(n_seq + 1) if q_start is None else q_start
    kv_len = t.new_empty(n_seq) if kv_len is None else kv_len
    seq = t.new_empty(T) if seq is None else seq
    slot = t.new_empty(T) if slot is None else slot
    args = BatchPlanArgs(t.data_ptr(), pages.held.data_ptr(), pages.free.data_ptr(), pages.n_free.data_ptr(),
                         _vector(past, "past", t, n_seq), _vector(n_new, "n_new", t, n_seq),
                         _vector(q_start, "q_start", t, n_seq + 1), _vector(kv_len, "kv_len", t, n_seq),
                         _vector(seq, "seq", t, T), _vector(slot, "slot", t, T), T, n_seq, max_pages,
                         pages.free.numel(), pages.page)
    return OpCall(OP_BATCH_PLAN, lib.wl_batch_plan, args, (q_start, kv_len, seq, slot), t.device,
                  (t, pages.held, pages.free, pages.n_free, past, n_new), ws)


def wl_batch_plan(pages, past, n_new, T, **kw):
    """(q_start, kv_len, seq, slot) of the next batch: n_new tokens behind past keys of
    every sequence, in T rows; pages are given and taken back. See batch_plan_call."""
    return batch_plan_call(pages, past, n_new, T, **kw).launch()


class LatentCache:
    """A paged cache of latent vectors: rows [n_pages][page][latent + rot] (bf16 or
    fp32), or uint8 [n_pages][page][latent + 2 rot] (e4m3 codes, then the key in bf16)
    with fp32 scale [n_pages][page]; table int32 [n_seq][max_pages] of page numbers."""

    __slots__ = ("rows", "table", "scale", "latent", "rot", "struct")

    def __init__(self, rows, table, latent: int, rot: int, scale=None):
        codes = rows.dtype == torch.uint8
        if not (codes or rows.dtype in _CODES) or rows.dim() != 3 or not rows.is_contiguous() or not rows.is_cuda:
            raise ValueError("rows must be a contiguous [n_pages][page][width] device tensor of bf16, fp32 or uint8")
        if rows.shape[2] != latent + (2 * rot if codes else rot):
            raise ValueError(f"rows must be {latent + (2 * rot if codes else rot)} wide")
        _tensor(table, "table", rows, torch.int32)
        if table.dim() != 2 or not table.is_contiguous():
            raise ValueError("table must be a contiguous [n_seq][max_pages] tensor")
        if codes and (scale is None or scale.shape != rows.shape[:2]):
            raise ValueError("scale must be [n_pages][page]")
        self.rows, self.table, self.scale, self.latent, self.rot = rows, table, scale, latent, rot
        self.struct = LatentCacheStruct(
            rows.data_ptr(), _vector(scale, "scale", rows, scale.numel(), torch.float32) if codes else None,
            table.data_ptr(), rows.shape[0], rows.shape[1], latent, rot, table.shape[0], table.shape[1],
            CACHE_FORMATS[torch.float8_e4m3fn] if codes else CACHE_FORMATS[rows.dtype])
        self.struct.tensors = rows, table, scale   # what it points into, for calls that hold it

    @property
    def dtype(self) -> torch.dtype:
        """Of the tensors that go with it."""
        return torch.float32 if self.rows.dtype == torch.float32 else torch.bfloat16


def new_latent_cache(n_pages: int, page: int, latent: int, rot: int, table: torch.Tensor,
                     dtype=torch.bfloat16) -> LatentCache:
    """A LatentCache of uninitialised pages on the table's device; dtype bf16, fp32 or
    float8_e4m3fn."""
    if dtype not in (torch.bfloat16, torch.float32, torch.float8_e4m3fn):
        raise ValueError("dtype must be bf16, fp32 or float8_e4m3fn")
    codes = dtype == torch.float8_e4m3fn
    rows = torch.empty(n_pages, page, latent + (2 * rot if codes else rot), dtype=torch.uint8 if codes else dtype,
                       device=table.device)
    scale = torch.empty(n_pages, page, dtype=torch.float32, device=table.device) if codes else None
    return LatentCache(rows, table, latent, rot, scale)


def latent_write_call(cache: LatentCache, c, seq, slot, q=None, n_q: int = 0, rope: Rope | None = None, pos=None,
                      norm=None, eps: float = 1e-6, offset: float = 0.0, q_out=None) -> OpCall:
    """wl_latent_write as an OpCall; out = q_out (None without q). c: [T][latent + rot];
    q: [T] rows of n_q heads, of which the last rot elements are rotated. pos None: the
    slots are the positions."""
    s = cache.struct
    T = _first(c, "c").shape[0]
    _tensor(cache.rows, "the cache", c, cache.rows.dtype)
    nope = ldq = ldo = 0
    if q is not None:
        if n_q < 1 or q.dim() != 2 or q.shape[1] % n_q or q.shape[1] // n_q < s.rot:
            raise ValueError(f"q must be a matrix of n_q heads of at least {s.rot}")
        nope = q.shape[1] // n_q - s.rot
        ldq = _matrix(q, "q", c, T, q.shape[1])
        if q_out is None:
            q_out = q.new_empty(q.shape)
        ldo = _matrix(q_out, "q_out", c, T, q.shape[1])
    elif n_q:
        raise ValueError("n_q goes with q")
    rot = None if rope is None else rope.struct(pos, T, c)
    args = LatentWriteArgs(_at(s), c.data_ptr(), _vector(norm, "norm", c, s.latent), _ptr(q), _ptr(q_out),
                           _vector(seq, "seq", c, T, torch.int32), _vector(slot, "slot", c, T, torch.int32), _at(rot), T,
                           n_q, nope, _matrix(c, "c", c, T, s.latent + s.rot), ldq, ldo, _CODES[c.dtype], eps, offset)
    return OpCall(OP_LATENT_WRITE, lib.wl_latent_write, args, q_out, c.device, (s, c, norm, q, seq, slot, rot, pos))


def wl_latent_write(cache, c, seq, slot, **kw):
    """Writes the tokens' latents (normalised by ``norm``) and keys (rotated) into the
    cache, q rotated beside them; returns the rotated q, or None. See latent_write_call."""
    return latent_write_call(cache, c, seq, slot, **kw).launch()


def latent_read_call(cache: LatentCache, seq, slot, out=None) -> OpCall:
    """wl_latent_read as an OpCall; out = [T][latent + rot] of cache.dtype. Rows of
    tokens without a place in the cache keep what it held (a new one is uninitialised)."""
    s, T = cache.struct, seq.numel()
    out = cache.rows.new_empty((T, s.latent + s.rot), dtype=cache.dtype) if out is None else _first(out, "out")
    _tensor(out, "out", cache.rows, cache.dtype)
    args = LatentReadArgs(_at(s), _vector(seq, "seq", out, T, torch.int32), _vector(slot, "slot", out, T, torch.int32),
                          out.data_ptr(), T, _matrix(out, "out", out, T, s.latent + s.rot), _CODES[out.dtype])
    return OpCall(OP_LATENT_READ, lib.wl_latent_read, args, out, out.device, (s, seq, slot))


def wl_latent_read(cache, seq, slot, **kw):
    """The rows of the tokens at (seq, slot), read back from the cache."""
    return latent_read_call(cache, seq, slot, **kw).launch()


def latent_attention_call(q, cache: LatentCache, w, q_start, kv_len, max_q: int, max_kv: int, scale: float,
                          mask: str | None = None, window: int = 0, tree=None, q_pos=None, form: str = "auto", o=None,
                          ws: torch.Tensor | None = None) -> OpCall:
    """wl_latent_attention as an OpCall; out = o. q: [T] rows of heads of nope + rot; w:
    [n_q][nope + value][latent], or None, where q's heads are latent + rot wide and o's
    latent. mask, window, tree, q_pos as in attention_call; form "auto", "absorbed" or
    "expanded"."""
    s = cache.struct
    T = _first(q, "q").shape[0]
    _tensor(cache.rows, "the cache", q, cache.rows.dtype)
    if w is None:
        n_q, nope, value = _heads(q, "q", s.latent + s.rot), s.latent, s.latent
    else:
        _tensor(w, "w", q)
        if w.dim() != 3 or not w.is_contiguous() or w.shape[2] != s.latent:
            raise ValueError(f"w must be a contiguous [n_q][nope + value][{s.latent}] tensor")
        n_q = w.shape[0]
        if n_q < 1 or q.shape[1] % n_q:
            raise ValueError(f"q must be a matrix of {n_q} heads")
        nope = q.shape[1] // n_q - s.rot
        value = w.shape[1] - nope
        if nope < 1 or value < 1:
            raise ValueError(f"q's heads of {q.shape[1] // n_q} do not go with w's {w.shape[1]} rows a head")
    if o is None:
        o = q.new_empty((T, n_q * value))
    mask = mask or ("causal" if tree is None else "tree")
    if mask not in MASKS:
        raise ValueError(f"mask {mask!r} is not one of {sorted(MASKS)}")
    if form not in LATENT_FORMS:
        raise ValueError(f"form {form!r} is not one of {sorted(LATENT_FORMS)}")
    if (tree is None) == (mask == "tree"):
        raise ValueError("tree goes with mask='tree'")
    words = 0
    if tree is not None:
        if tree.dim() != 2 or tree.shape[0] != T:
            raise ValueError(f"tree must be [{T}][words]")
        words = tree.shape[1]
    elif q_pos is not None:
        raise ValueError("q_pos goes with mask='tree'")
    n_seq = s.n_seq
    args = LatentAttentionArgs(
        _at(s), q.data_ptr(), _ptr(w), o.data_ptr(), _vector(q_start, "q_start", q, n_seq + 1, torch.int32),
        _vector(kv_len, "kv_len", q, n_seq, torch.int32), _vector(tree, "tree", q, T * words, torch.int32),
        _vector(q_pos, "q_pos", q, T, torch.int32), T, n_q, nope, value, _matrix(q, "q", q, T, n_q * (nope + s.rot)),
        _matrix(o, "o", q, T, n_q * value), max_q, max_kv, MASKS[mask], window, words, _CODES[q.dtype],
        LATENT_FORMS[form], scale)
    return OpCall(OP_LATENT_ATTENTION, lib.wl_latent_attention, args, o, q.device,
                  (q, s, w, q_start, kv_len, tree, q_pos), ws)


def wl_latent_attention(q, cache, w, q_start, kv_len, max_q, max_kv, scale, **kw):
    """softmax(scale q k) v of the tokens over the latent cache, every head's keys and
    values formed from its rows by w; see latent_attention_call."""
    return latent_attention_call(q, cache, w, q_start, kv_len, max_q, max_kv, scale, **kw).launch()


def verify_drafts_call(target, token, q_start, u, draft=None, parent=None, temperature=None, probabilities: bool = False,
                       max_q: int = VERIFY_ROWS, length=None, out=None, n_out=None, path=None,
                       ws: torch.Tensor | None = None) -> OpCall:
    """wl_verify_drafts as an OpCall; out = (out, n_out, path). target, draft: [T][vocab]
    logits, or probabilities; token int32 [T]; q_start int32 [n_seq + 1]; u fp32 [T][2];
    parent int32 [T] for trees; temperature fp32 [n_seq] (0: greedy); length int32
    [n_seq]: n_out is added to it."""
    T, vocab = _first(target, "target").shape
    n_seq = q_start.numel() - 1
    lds = [0, 0]
    for i, (t, name) in enumerate(((target, "target"), (draft, "draft"))):
        if t is not None:
            lds[i] = _matrix(t, name, target, T, vocab)
    out = token.new_empty(T) if out is None else out
    n_out = token.new_empty(n_seq) if n_out is None else n_out
    path = token.new_empty(T) if path is None else path
    i32, f32 = torch.int32, torch.float32
    args = VerifyArgs(target.data_ptr(), _ptr(draft), _vector(token, "token", target, T, i32),
                      _vector(q_start, "q_start", target, n_seq + 1, i32), _vector(parent, "parent", target, T, i32),
                      _vector(u, "u", target, 2 * T, f32), _vector(temperature, "temperature", target, n_seq, f32),
                      _vector(out, "out", target, T, i32), _vector(path, "path", target, T, i32),
                      _vector(n_out, "n_out", target, n_seq, i32), _vector(length, "length", target, n_seq, i32), T, n_seq,
                      vocab, lds[0], lds[1], max_q, VERIFY_PROBABILITIES if probabilities else VERIFY_LOGITS,
                      _CODES[target.dtype])
    return OpCall(OP_VERIFY_DRAFTS, lib.wl_verify_drafts, args, (out, n_out, path), target.device,
                  (target, draft, token, q_start, parent, u, temperature, length), ws)


def wl_verify_drafts(target, token, q_start, u, **kw):
    """(out, n_out, path): of every sequence the drafted tokens that stay and the one
    behind them, how many, and their rows; see verify_drafts_call."""
    return verify_drafts_call(target, token, q_start, u, **kw).launch()


class LayerStep(Step):
    """A step of whole layers: projection calls as in Step, (op, thetas, x, y), mixed
    with OpCalls, recorded into one HIP graph (wl_step_create_ops) and launched
    with one call. Values in the calls' tensors are read at each launch."""

    def __init__(self, calls, ws: torch.Tensor | None = None):
        n = len(calls)
        ops = (StepOp * n)()
        # What the graph's addresses point into: the list, the calls and the thetas are the
        # caller's to reuse.
        self._keep = []
        device = None
        for i, call in enumerate(calls):
            if isinstance(call, OpCall):
                ops[i].op, ops[i].args = call.op, ctypes.addressof(call.args)
                device = _one_device(device, call.device, i)
                self._keep.append((call.args, call.out, call.keep))
                continue
            op, thetas, x, y = call
            self._keep += [x, y, [dict(t) for t in thetas]]
            if len(thetas) != (1 if op == OP_LINEAR else 3):
                raise ValueError(f"call {i}: {len(thetas)} thetas for op {op}")
            c = Call()
            structs = [make_theta(t) for t in thetas]
            c.op, c.x, c.y, c.T = op, _ptr(x), _ptr(y), _io(x, int(thetas[0]["d_in"]), thetas[0]["W0"].dtype)
            for j, st in enumerate(structs):
                c.th[j] = ctypes.pointer(st)
            self._keep += [structs, c]
            ops[i].op, ops[i].args = op, ctypes.addressof(c)
            device = _one_device(device, x.device, i)
        need = int(lib.wl_step_ops_workspace_bytes(ops, n))
        if need == 0:
            raise ValueError("invalid calls for a step")
        self._create(lambda *a: lib.wl_step_create_ops(ops, n, *a), need, ws, device)
