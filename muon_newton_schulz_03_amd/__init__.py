"""Python binding of libmuon.so, the MI355X (gfx950) Muon optimizer-step library.

Argument marshalling only: every step of the computation runs in the HIP
kernels behind the C ABI declared in include/muon.h. The functions here carry
the C names; torch tensors supply device pointers, shapes and the current
stream. There is no CPU fallback: if the library is missing, every call
raises.
"""
import ctypes
import functools
import json
import operator
import os
import struct

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libmuon.so")

MUON_OK = 0
STATUS_NAMES = {
    0: "MUON_OK", 1: "MUON_ERR_INVALID_ARG", 2: "MUON_ERR_SHAPE", 3: "MUON_ERR_DTYPE",
    4: "MUON_ERR_ALIGN", 5: "MUON_ERR_ALIAS", 6: "MUON_ERR_WORKSPACE", 7: "MUON_ERR_HIP",
}
MUON_ERR_INVALID_ARG = 1
MUON_ERR_SHAPE = 2
MUON_ERR_DTYPE = 3
MUON_ERR_ALIGN = 4
MUON_ERR_ALIAS = 5
MUON_ERR_WORKSPACE = 6
MUON_ERR_HIP = 7
MUON_F32 = 0
MUON_BF16 = 1

MUON_NS_FULL = 0x000
MUON_NS_BLOCKWISE = 0x001
MUON_NS_DISTRIBUTED = 0x002
MUON_PACK_RR = 0x000
MUON_PACK_COST = 0x010
MUON_PLACE_RR = 0
MUON_PLACE_LPT = 1
MUON_AA_PLAIN = 0x000
MUON_AA_SPLIT = 0x100

DEFAULT_COEFFS = (3.4445, -4.7750, 2.0315)
DEFAULT_MODE = MUON_NS_FULL | MUON_PACK_COST | MUON_AA_PLAIN

EXPORTED = (
    "muon_ns_batched", "muon_step", "muon_set_stream", "muon_workspace_size",
    "muon_workspace_min_size", "muon_set_workspace", "muon_set_step_options",
    "muon_last_error", "muon_plan_info", "muon_set_phase_timing", "muon_phase_times",
    "muon_place", "muon_adamw_step", "muon_step_noalloc", "muon_get_workspace", "muon_exchange_workspace",
    "muon_layernorm_forward", "muon_layernorm_backward", "muon_layernorm_workspace_size",
    "muon_ckpt_save", "muon_ckpt_load", "muon_ckpt_weight_grad", "muon_ckpt_weight_grad_workspace_size",
    "muon_route_forward", "muon_route_backward", "muon_route_workspace_size",
    "muon_gated_forward", "muon_gated_backward", "muon_expert_forward", "muon_expert_backward",
    "muon_gated_workspace_size", "muon_expert_workspace_size",
    "muon_combine_forward", "muon_combine_backward", "muon_combine_workspace_size",
    "muon_dropout_forward", "muon_dropout_backward",
)
MUON_ACT_SILU = 0
MUON_ACT_GELU = 1
MUON_CKPT_GROUP = 128  # columns that share one scale byte of a checkpoint
MUON_NOALLOC_SCRATCH_BYTES = 256 << 20
PHASES = ("prep", "norm", "gram", "aa", "bx", "finish", "adamw", "reduce")


class MuonError(RuntimeError):
    def __init__(self, status, msg):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {msg}")
        self.status = status


class muon_mat(ctypes.Structure):
    _fields_ = [
        ("data", ctypes.c_void_p),
        ("rows", ctypes.c_int64),
        ("cols", ctypes.c_int64),
        ("ld", ctypes.c_int64),
        ("dtype", ctypes.c_int32),
        ("col_blocks", ctypes.c_int32),
    ]


class muon_ckpt(ctypes.Structure):
    _fields_ = [
        ("codes", ctypes.c_void_p),
        ("scales", ctypes.c_void_p),
        ("rows", ctypes.c_int64),
        ("cols", ctypes.c_int64),
        ("ld_codes", ctypes.c_int64),
        ("ld_scales", ctypes.c_int64),
    ]


_lib = None


def load_library(path=LIB_PATH):
    """Load libmuon.so (built by build.py). Raises if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is not built; run python -m muon_newton_schulz_03_amd.build")
    lib = ctypes.CDLL(path)
    mat_p = ctypes.POINTER(muon_mat)
    f3 = ctypes.POINTER(ctypes.c_float)
    sz = ctypes.POINTER(ctypes.c_size_t)
    sigs = {
        "muon_ns_batched": ([mat_p, ctypes.c_int32, ctypes.c_int32, f3, ctypes.c_uint32], ctypes.c_int),
        "muon_step": ([mat_p, mat_p, mat_p, ctypes.c_int32, ctypes.c_float, ctypes.c_float, ctypes.c_int32],
                      ctypes.c_int),
        "muon_step_noalloc": ([mat_p, mat_p, mat_p, ctypes.c_int32, ctypes.c_float, ctypes.c_float,
                               ctypes.c_int32], ctypes.c_int),
        "muon_set_stream": ([ctypes.c_void_p], ctypes.c_int),
        "muon_workspace_size": ([mat_p, ctypes.c_int32, ctypes.c_uint32, sz], ctypes.c_int),
        "muon_workspace_min_size": ([mat_p, ctypes.c_int32, ctypes.c_uint32, sz], ctypes.c_int),
        "muon_set_workspace": ([ctypes.c_void_p, ctypes.c_size_t], ctypes.c_int),
        "muon_set_step_options": ([ctypes.c_int32, f3, ctypes.c_float, ctypes.c_uint32], ctypes.c_int),
        "muon_last_error": ([], ctypes.c_char_p),
        "muon_plan_info": ([mat_p, ctypes.c_int32, ctypes.c_int32, ctypes.c_uint32, ctypes.c_size_t,
                            ctypes.c_char_p, ctypes.c_size_t, sz], ctypes.c_int),
        "muon_set_phase_timing": ([ctypes.c_int32], ctypes.c_int),
        "muon_phase_times": ([ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_int64)], ctypes.c_int),
        "muon_adamw_step": ([mat_p, mat_p, mat_p, mat_p, ctypes.c_int32, ctypes.c_float, ctypes.c_float,
                             ctypes.c_float, ctypes.c_float, ctypes.c_float, ctypes.c_int32], ctypes.c_int),
        "muon_place": ([ctypes.POINTER(ctypes.c_double), ctypes.c_int32, ctypes.c_int32, ctypes.c_uint32,
                        ctypes.POINTER(ctypes.c_int32), ctypes.POINTER(ctypes.c_double),
                        ctypes.POINTER(ctypes.c_double)], ctypes.c_int),
        "muon_get_workspace": ([ctypes.POINTER(ctypes.c_void_p), sz], ctypes.c_int),
        "muon_exchange_workspace": ([ctypes.c_void_p, ctypes.c_size_t, ctypes.POINTER(ctypes.c_void_p), sz], ctypes.c_int),
    }
    # the training operators take packed descriptors (bytes) where the header has struct pointers
    p, i32, i64, f = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float
    for name, args in {
        "muon_layernorm_forward": [p, p, p, p, p, p, f, p],
        "muon_layernorm_backward": [p] * 8,
        "muon_layernorm_workspace_size": [i64, i64, sz],
        "muon_ckpt_save": [p, p],
        "muon_ckpt_load": [p, p],
        "muon_ckpt_weight_grad": [p, p, p, i64, i32, p, p, i32],
        "muon_ckpt_weight_grad_workspace_size": [i32, i64, i64, i64, i64, sz],
        "muon_route_forward": [p, i32, i32, f, p, p, p, p, p, p],
        "muon_route_workspace_size": [i64, i64, i32, sz],
        "muon_route_backward": [p, i32, i32, f, p, p, p, p, p],
        "muon_gated_forward": [p, p, i64, p, i64, i32, p, p, i32, i32, p, p, p],
        "muon_gated_backward": [p, p, p, p, i64, p, i64, i32, p, p, i32, p, p, p],
        "muon_expert_forward": [p, p, i64, i32, i64, p, p, i32, i32, p],
        "muon_expert_backward": [p, p, i64, i32, i64, p, p, i32, i32, p],
        "muon_gated_workspace_size": [i32, i64, i64, i64, i64, i32, sz],
        "muon_expert_workspace_size": [i32, i64, i64, i64, i64, i32, sz],
        "muon_combine_forward": [p, i32, p, p, p, f, p, p],
        "muon_combine_backward": [p, p, i32, p, p, p, f, p, p, p],
        "muon_combine_workspace_size": [i64, i32, sz],
        "muon_dropout_forward": [p, p, f, p, p],
        "muon_dropout_backward": [p, f, p, p],
    }.items():
        sigs[name] = (args, ctypes.c_int)
    for name, (args, res) in sigs.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    _lib = lib
    return lib


def lib():
    return load_library()


def muon_last_error():
    return lib().muon_last_error().decode()


def _check(status):
    if status != MUON_OK:
        raise MuonError(status, muon_last_error())


# ---------------------------------------------------------------------------
# descriptors
# ---------------------------------------------------------------------------

def _dtype_code(t):
    import torch
    if t.dtype == torch.float32:
        return MUON_F32
    if t.dtype == torch.bfloat16:
        return MUON_BF16
    raise TypeError(f"unsupported dtype {t.dtype}")


def mat_of(t, col_blocks=1):
    """Descriptor of a 2-D row-major device tensor (unit column stride)."""
    if t.dim() != 2:
        raise ValueError("expected a 2-D tensor")
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError("expected unit column stride")
    ld = t.stride(0) if t.shape[0] > 1 else t.shape[1]
    ld = max(ld, t.shape[1])
    return muon_mat(ctypes.c_void_p(t.data_ptr()), t.shape[0], t.shape[1], ld, _dtype_code(t), col_blocks)


def mats(descs):
    """Pack a list of muon_mat (or raw tuples) into a C array."""
    arr = (muon_mat * max(len(descs), 1))()
    for i, d in enumerate(descs):
        arr[i] = d
    return arr


def _coeffs(c):
    if c is None:
        return None
    return (ctypes.c_float * 3)(*[float(x) for x in c])


# ---------------------------------------------------------------------------
# C entry points (same names, raw descriptors)
# ---------------------------------------------------------------------------

def muon_set_stream(stream=None):
    """stream: a torch.cuda.Stream, a raw hipStream_t integer, or None for
    torch's current stream."""
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    _check(lib().muon_set_stream(ctypes.c_void_p(handle)))


def muon_set_workspace(ptr, nbytes):
    _check(lib().muon_set_workspace(ctypes.c_void_p(ptr), ctypes.c_size_t(nbytes)))


def muon_workspace_size(descs, mode=DEFAULT_MODE):
    out = ctypes.c_size_t()
    _check(lib().muon_workspace_size(mats(descs), len(descs), mode, ctypes.byref(out)))
    return out.value


def muon_workspace_min_size(descs, mode=DEFAULT_MODE):
    out = ctypes.c_size_t()
    _check(lib().muon_workspace_min_size(mats(descs), len(descs), mode, ctypes.byref(out)))
    return out.value


def muon_set_step_options(iters=5, coeffs=DEFAULT_COEFFS, eps=1e-7, mode=DEFAULT_MODE):
    _check(lib().muon_set_step_options(iters, _coeffs(coeffs), eps, mode))


def muon_plan_info(descs, iters=5, mode=DEFAULT_MODE, workspace_bytes=0):
    need = ctypes.c_size_t()
    arr = mats(descs)
    _check(lib().muon_plan_info(arr, len(descs), iters, mode, workspace_bytes, None, 0, ctypes.byref(need)))
    buf = ctypes.create_string_buffer(need.value)
    _check(lib().muon_plan_info(arr, len(descs), iters, mode, workspace_bytes, buf, need.value,
                                ctypes.byref(need)))
    return json.loads(buf.value.decode())


def muon_set_phase_timing(enable=True):
    _check(lib().muon_set_phase_timing(1 if enable else 0))


def muon_phase_times():
    """{kind: (milliseconds, launches)} since the last query (see muon.h)."""
    ms = (ctypes.c_double * len(PHASES))()
    n = (ctypes.c_int64 * len(PHASES))()
    _check(lib().muon_phase_times(ms, n))
    return {k: (ms[i], n[i]) for i, k in enumerate(PHASES)}


def muon_place(costs, ranks, policy="lpt"):
    """Place matrices with the given costs on `ranks` ranks (see muon.h).
    Returns (owner list, per-rank load list, max/mean imbalance)."""
    n = len(costs)
    c = (ctypes.c_double * max(n, 1))(*[float(x) for x in costs])
    owner = (ctypes.c_int32 * max(n, 1))()
    load = (ctypes.c_double * ranks)()
    imb = ctypes.c_double()
    pol = {"rr": MUON_PLACE_RR, "lpt": MUON_PLACE_LPT}[policy] if isinstance(policy, str) else policy
    _check(lib().muon_place(c, n, ranks, pol, owner, load, ctypes.byref(imb)))
    return list(owner[:n]), list(load), imb.value


# ---------------------------------------------------------------------------
# tensor-level wrappers
# ---------------------------------------------------------------------------

class Workspace:
    """A caller-owned workspace (a torch uint8 buffer) set for this thread."""

    def __init__(self, nbytes, device="cuda"):
        import torch
        self.nbytes = int(nbytes)
        self.buf = torch.empty(max(self.nbytes, 256), dtype=torch.uint8, device=device)
        muon_set_workspace(self.buf.data_ptr(), self.nbytes)


_ws = None


def ensure_workspace(descs, mode=DEFAULT_MODE, max_bytes=None):
    """Make sure this thread has a workspace large enough for the call:
    everything in flight when it fits under max_bytes, else at least one
    matrix."""
    global _ws
    full = muon_workspace_size(descs, mode)
    want = full
    if max_bytes is not None and full > max_bytes:
        want = max(muon_workspace_min_size(descs, mode), int(max_bytes))
    if _ws is None or _ws.nbytes < want:
        _ws = None
        _ws = Workspace(want)
    else:
        muon_set_workspace(_ws.buf.data_ptr(), _ws.nbytes)
    return _ws


def muon_ns_batched(tensors, iters=5, coeffs=DEFAULT_COEFFS, mode=DEFAULT_MODE, col_blocks=None,
                    workspace=None, max_workspace_bytes=None):
    """Orthogonalize each 2-D device tensor in place (see muon.h)."""
    cb = col_blocks if col_blocks is not None else [1] * len(tensors)
    if isinstance(cb, int):
        cb = [cb] * len(tensors)
    descs = [mat_of(t, c) for t, c in zip(tensors, cb)]
    muon_set_stream(None)
    if workspace is None:
        if descs:
            ensure_workspace(descs, mode, max_workspace_bytes)
    else:
        muon_set_workspace(workspace.data_ptr(), workspace.numel() * workspace.element_size())
    _check(lib().muon_ns_batched(mats(descs), len(descs), iters, _coeffs(coeffs), mode))


def muon_step(params, grads, moms, lr=0.02, beta=0.95, nesterov=False, iters=5, coeffs=DEFAULT_COEFFS,
              eps=1e-7, mode=DEFAULT_MODE, col_blocks=None, workspace=None, max_workspace_bytes=None):
    """One Muon step over lists of 2-D device tensors; params and moms are
    updated in place (see muon.h)."""
    cb = col_blocks if col_blocks is not None else [1] * len(params)
    if isinstance(cb, int):
        cb = [cb] * len(params)
    W = [mat_of(t, c) for t, c in zip(params, cb)]
    G = [mat_of(t) for t in grads]
    M = [mat_of(t) for t in moms]
    muon_set_stream(None)
    muon_set_step_options(iters, coeffs, eps, mode)
    if workspace is None:
        if W:
            ensure_workspace(W, mode, max_workspace_bytes)
    else:
        muon_set_workspace(workspace.data_ptr(), workspace.numel() * workspace.element_size())
    _check(lib().muon_step(mats(W), mats(G), mats(M), len(W), lr, beta, 1 if nesterov else 0))


def muon_step_noalloc(params, grads, moms, lr=0.02, beta=0.95, nesterov=False, iters=5,
                      coeffs=DEFAULT_COEFFS, eps=1e-7, mode=DEFAULT_MODE, col_blocks=None):
    """muon_step with the library's device scratch instead of a workspace
    (see muon.h): no device memory is allocated by the library or here."""
    cb = col_blocks if col_blocks is not None else [1] * len(params)
    if isinstance(cb, int):
        cb = [cb] * len(params)
    W = [mat_of(t, c) for t, c in zip(params, cb)]
    G = [mat_of(t) for t in grads]
    M = [mat_of(t) for t in moms]
    muon_set_stream(None)
    muon_set_step_options(iters, coeffs, eps, mode)
    _check(lib().muon_step_noalloc(mats(W), mats(G), mats(M), len(W), lr, beta, 1 if nesterov else 0))


def muon_adamw_step(params, grads, exp_avg, exp_avg_sq, lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8,
                    weight_decay=0.0, step=1):
    """One AdamW step over lists of 2-D device tensors (see muon.h): params
    (bf16 or float32) and the float32 moments are updated in place."""
    W = [mat_of(t) for t in params]
    G = [mat_of(t) for t in grads]
    Mo = [mat_of(t) for t in exp_avg]
    V = [mat_of(t) for t in exp_avg_sq]
    muon_set_stream(None)
    _check(lib().muon_adamw_step(mats(W), mats(G), mats(Mo), mats(V), len(W), lr, beta1, beta2, eps,
                                 weight_decay, step))


# ---------------------------------------------------------------------------
# training operators
# ---------------------------------------------------------------------------

_MAT = struct.Struct("=Qqqqii").pack   # muon_mat: data, rows, cols, ld, dtype, col_blocks
_CKPT = struct.Struct("=QQqqqq").pack  # muon_ckpt
_torch = _codes = _ckpt_dtypes = None


def _load_torch():
    """torch and the dtypes of operands, looked up by the first call; the dtypes of a checkpoint."""
    global _torch, _codes, _ckpt_dtypes
    import torch
    _torch, _codes = torch, {torch.float32: MUON_F32, torch.bfloat16: MUON_BF16}
    _ckpt_dtypes = (torch.float8_e4m3fn, torch.uint8)
    return _ckpt_dtypes


# The smallest calls take about as long here as on the GPU, so these helpers ask
# a tensor for each fact once.

def _on_gpu(name, t, device):
    """The device of a tensor that a kernel will touch, which has to be the others'."""
    d = t.get_device()
    if d != device or d < 0:
        if not t.is_cuda:
            raise ValueError(f"{name}: expected a GPU tensor")
        if device is not None:
            raise ValueError(f"{name}: on another device than the other tensors")
    return d


def _mat(name, t, device):
    """Packed muon_mat of a 2-D tensor with unit column stride (NULL for None)."""
    if t is None:
        return None
    if t.get_device() != device:
        _on_gpu(name, t, device)
    strides = t.stride()
    if len(strides) != 2:
        raise ValueError(f"{name}: expected a 2-D tensor")
    ld, unit = strides
    rows, cols = t.shape
    if cols > 1 and unit != 1:
        raise ValueError(f"{name}: expected unit column stride")
    if rows <= 1 or ld < cols:
        if rows > 1:
            raise ValueError(f"{name}: rows overlap")
        ld = cols
    code = _codes.get(t.dtype)
    if code is None:
        raise TypeError(f"{name}: unsupported dtype {t.dtype}")
    return _MAT(t.data_ptr(), rows, cols, ld, code, 1)


def _vec(name, t, dtype, shape, device):
    """Address of a contiguous tensor of the given dtype and shape (None for None)."""
    if t is None:
        return None
    if t.get_device() != device:
        _on_gpu(name, t, device)
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous tensor")
    return t.data_ptr()


class Checkpoint:
    """An activation checkpoint in 8 bits (see muon_ckpt in muon.h): `codes`,
    rows x cols float8_e4m3fn, and `scales`, rows x ceil(cols / 128) uint8,
    both with unit column stride. The two tensors stay the checkpoint's own; if
    their memory is exchanged (`codes.data = ...`), later calls use the new."""

    __slots__ = ("_codes", "_scales", "_key", "_packed")

    def __init__(self, codes, scales):
        self._codes, self._scales = codes, scales
        self._pack()

    def _pack(self):
        codes, scales = self._codes, self._scales
        if (codes.dtype, scales.dtype) != (_ckpt_dtypes or _load_torch()):
            raise TypeError("a checkpoint holds float8_e4m3fn codes and uint8 scales")
        strides_c, strides_s = codes.stride(), scales.stride()
        if len(strides_c) != 2 or len(strides_s) != 2:
            raise ValueError("a checkpoint's codes and scales are 2-D")
        rows, cols = codes.shape
        groups = -(-cols // MUON_CKPT_GROUP)
        if scales.shape != (rows, groups):
            raise ValueError(f"scales: expected shape {(rows, groups)}, got {tuple(scales.shape)}")
        ld_c, unit_c = strides_c
        ld_s, unit_s = strides_s
        if (cols > 1 and unit_c != 1) or (groups > 1 and unit_s != 1):
            raise ValueError("a checkpoint's codes and scales have unit column stride")
        if rows <= 1:
            ld_c, ld_s = cols, groups
        if ld_c < cols or ld_s < groups:
            raise ValueError("a checkpoint's rows overlap")
        device = codes.get_device()
        if device < 0 or scales.get_device() != device:
            _on_gpu("scales", scales, _on_gpu("codes", codes, None))
        at_c, at_s = codes.data_ptr(), scales.data_ptr()
        self._key = (at_c, at_s, rows * cols, rows * groups)
        self._packed = _CKPT(at_c, at_s, rows, cols, ld_c, ld_s)

    def _desc(self, device):
        """Packed muon_ckpt of the tensors as they are now, on a call's device."""
        codes, scales = self._codes, self._scales
        if self._key != (codes.data_ptr(), scales.data_ptr(), codes.numel(), scales.numel()):
            for t in (codes, scales):
                if t.numel() and not t.untyped_storage().nbytes():
                    raise ValueError("the checkpoint's memory has been freed")
            self._pack()
        if codes.get_device() != device:
            _on_gpu("ckpt", codes, device)
        return self._packed

    codes = property(operator.attrgetter("_codes"))
    scales = property(operator.attrgetter("_scales"))

    @classmethod
    def empty(cls, rows, cols, device="cuda"):
        """Room for the checkpoint of a rows x cols matrix (rows on 16-byte boundaries)."""
        import torch
        codes = torch.empty((rows, -(-cols // 16) * 16), dtype=torch.float8_e4m3fn, device=device)[:, :cols]
        return cls(codes, torch.empty((rows, -(-cols // MUON_CKPT_GROUP)), dtype=torch.uint8, device=device))

    @property
    def shape(self):
        return self._codes.shape


def _enter(t):
    """The device index of a call's first tensor; its current stream becomes the call's."""
    if _codes is None:
        _load_torch()
    device = _on_gpu("argument", t, None)
    # torch.cuda.current_device and the raw handle of torch.cuda.current_stream, without what they wrap around them
    if device != _torch._C._cuda_getDevice():
        raise ValueError("the tensors are not on the current device")
    _check((_lib or lib()).muon_set_stream(_torch._C._cuda_getCurrentRawStream(device)))
    return device


def _with_scratch(nbytes, workspace, device, fn, *args):
    """Calls fn with a workspace of nbytes: the caller's (a uint8 tensor), or a
    temporary one from torch's allocator, whose memory is reused in stream order
    only. What the thread had set before is set again afterwards."""
    if not nbytes:
        return _check(fn(*args))
    if workspace is None:
        workspace = _torch.empty(nbytes, dtype=_torch.uint8, device="cuda")
    else:
        _on_gpu("workspace", workspace, device)
        if not workspace.is_contiguous():
            raise ValueError("workspace: expected a contiguous tensor")
    old, old_bytes = ctypes.c_void_p(), ctypes.c_size_t()
    _check(_lib.muon_exchange_workspace(workspace.data_ptr(), workspace.nbytes, old, old_bytes))
    try:
        _check(fn(*args))
    finally:
        _lib.muon_exchange_workspace(old, old_bytes, None, None)


def _size(fn, *args):
    out = ctypes.c_size_t()
    _check(fn(*args, ctypes.byref(out)))
    return out.value


# the sizes depend on these numbers alone
@functools.lru_cache(256)
def muon_layernorm_workspace_size(rows, cols):
    return _size(lib().muon_layernorm_workspace_size, rows, cols)


@functools.lru_cache(256)
def muon_ckpt_weight_grad_workspace_size(dtype, slots, n, k, groups=1):
    return _size(lib().muon_ckpt_weight_grad_workspace_size, dtype, slots, n, k, groups)


@functools.lru_cache(256)
def muon_route_workspace_size(tokens, experts, topk):
    return _size(lib().muon_route_workspace_size, tokens, experts, topk)


def muon_layernorm_forward(x, y, mean=None, rstd=None, weight=None, bias=None, eps=1e-5, ckpt=None):
    """y = layer norm of x's rows (see muon.h). mean, rstd: float32 vectors
    that the backward pass reads; weight, bias: 1 x cols; ckpt: a Checkpoint
    that receives y in 8 bits in the same pass."""
    d = _enter(x)
    f32, rows = _torch.float32, x.shape[:1]
    _check(_lib.muon_layernorm_forward(
        _mat("x", x, d), _mat("y", y, d), _vec("mean", mean, f32, rows, d), _vec("rstd", rstd, f32, rows, d),
        _mat("weight", weight, d), _mat("bias", bias, d), eps, None if ckpt is None else ckpt._desc(d)))


def muon_layernorm_backward(dy, x, mean, rstd, dx, weight=None, dweight=None, dbias=None, workspace=None):
    """dx, and where given dweight and dbias (1 x cols), of the layer norm (see
    muon.h). workspace: a uint8 tensor of muon_layernorm_workspace_size bytes
    (default: a temporary one)."""
    d = _enter(dy)
    f32, rows = _torch.float32, dy.shape[:1]
    args = (_mat("dy", dy, d), _mat("x", x, d), _vec("mean", mean, f32, rows, d), _vec("rstd", rstd, f32, rows, d),
            _mat("dx", dx, d), _mat("weight", weight, d), _mat("dweight", dweight, d), _mat("dbias", dbias, d))
    need = muon_layernorm_workspace_size(*dy.shape) if dweight is not None or dbias is not None else 0
    _with_scratch(need, workspace, d, _lib.muon_layernorm_backward, *args)


def muon_ckpt_save(x, ckpt):
    """Save the matrix x as an 8-bit checkpoint (see muon.h)."""
    d = _enter(x)
    _check(_lib.muon_ckpt_save(_mat("x", x, d), ckpt._desc(d)))


def muon_ckpt_load(ckpt, out):
    """Load a checkpoint's values into the matrix out (see muon.h)."""
    d = _enter(out)
    _check(_lib.muon_ckpt_load(ckpt._desc(d), _mat("out", out, d)))


def muon_ckpt_weight_grad(dy, ckpt, grads, offsets=None, rows=None, rows_per_token=1, workspace=None):
    """Weight gradients of a group of layers from their input's checkpoint (see
    muon.h): grads[g] = sum over the slots of group g of dy[s]^T x[token(s)].
    dy: slots x n; grads: groups x n x k (its matrices are what muon_step
    takes); offsets (groups + 1) and rows (slots): int32, as
    muon_route_forward writes them with rows_per_token = topk."""
    d = _enter(dy)
    if grads.dim() != 3:
        raise ValueError("grads: expected a 3-D tensor (groups x n x k)")
    _on_gpu("grads", grads, d)
    groups, n, k = grads.shape
    stride, ld, unit = grads.stride()
    if (k > 1 and unit != 1) or (n > 1 and ld < k):
        raise ValueError("grads: expected unit column stride")
    if n <= 1:
        ld = k
    dy_mat = _mat("dy", dy, d)
    if grads.dtype != dy.dtype:
        raise TypeError("dy and grads differ in dtype")
    code = _codes[dy.dtype]
    if groups > 1 and offsets is None:
        raise ValueError("offsets: needed with more than one group")
    args = (dy_mat, ckpt._desc(d), _MAT(grads.data_ptr(), n, k, ld, code, 1), stride, groups,
            _vec("offsets", offsets, _torch.int32, (groups + 1,), d), _vec("rows", rows, _torch.int32, dy.shape[:1], d),
            rows_per_token)
    _with_scratch(muon_ckpt_weight_grad_workspace_size(code, dy.shape[0], n, k, groups), workspace, d,
                  _lib.muon_ckpt_weight_grad, *args)


def muon_route_forward(logits, indices, weights, counts, offsets, rows, loss, alpha=1e-2, renormalize=True,
                       workspace=None):
    """Route tokens to their topk experts (see muon.h). logits: tokens x
    experts; indices (int32) and weights (float32): tokens x topk, which sets
    topk; counts and offsets: experts + 1, rows: tokens * topk, all int32;
    loss: one float32. All outputs are overwritten."""
    d = _enter(logits)
    m = _mat("logits", logits, d)
    tokens, experts = logits.shape
    if indices.dim() != 2:
        raise ValueError("indices: expected a 2-D tensor (tokens x topk)")
    topk = indices.shape[1]
    i32, pair, table = _torch.int32, (tokens, topk), (experts + 1,)
    args = (m, topk, int(renormalize), alpha, _vec("indices", indices, i32, pair, d),
            _vec("weights", weights, _torch.float32, pair, d), _vec("counts", counts, i32, table, d),
            _vec("offsets", offsets, i32, table, d), _vec("rows", rows, i32, (tokens * topk,), d),
            _vec("loss", loss, _torch.float32, (1,), d))
    _with_scratch(muon_route_workspace_size(tokens, experts, topk), workspace, d, _lib.muon_route_forward, *args)


def muon_route_backward(logits, indices, counts, dlogits, dweights=None, dloss=None, alpha=1e-2, renormalize=True):
    """Gradient of loss * dloss + (weights * dweights).sum() with respect to
    the logits (see muon.h)."""
    d = _enter(logits)
    if indices.dim() != 2:
        raise ValueError("indices: expected a 2-D tensor (tokens x topk)")
    pair = (logits.shape[0], indices.shape[1])
    f32 = _torch.float32
    _check(_lib.muon_route_backward(
        _mat("logits", logits, d), pair[1], int(renormalize), alpha, _vec("indices", indices, _torch.int32, pair, d),
        _vec("counts", counts, _torch.int32, (logits.shape[1] + 1,), d), _vec("dweights", dweights, f32, pair, d),
        _vec("dloss", dloss, f32, (1,), d), _mat("dlogits", dlogits, d)))


# ---------------------------------------------------------------------------
# feed-forward operators
# ---------------------------------------------------------------------------

_ACTIVATIONS = {"silu": MUON_ACT_SILU, "gelu": MUON_ACT_GELU}


def _activation(name):
    code = _ACTIVATIONS.get(name)
    if code is None:
        raise ValueError(f"activation: expected one of {sorted(_ACTIVATIONS)}, got {name!r}")
    return code


def _stack(name, t, device):
    """(packed muon_mat of the first matrix, stride, groups) of a 3-D tensor groups x rows x cols, or of one 2-D matrix."""
    if t.get_device() != device:
        _on_gpu(name, t, device)
    if t.dim() == 2:
        return _mat(name, t, device), 0, 1
    if t.dim() != 3:
        raise ValueError(f"{name}: expected a 3-D tensor (groups x rows x cols) or a matrix")
    groups, rows, cols = t.shape
    stride, ld, unit = t.stride()
    if (cols > 1 and unit != 1) or (rows > 1 and ld < cols):
        raise ValueError(f"{name}: expected unit column stride")
    code = _codes.get(t.dtype)
    if code is None:
        raise TypeError(f"{name}: unsupported dtype {t.dtype}")
    return _MAT(t.data_ptr(), rows, cols, ld if rows > 1 else cols, code, 1), stride, groups


def _slots(offsets, rows, groups, slots, device):
    """Addresses of the slot lists of a call."""
    if groups > 1 and offsets is None:
        raise ValueError("offsets: needed with more than one group")
    return (_vec("offsets", offsets, _torch.int32, (groups + 1,), device),
            _vec("rows", rows, _torch.int32, (slots,), device))


@functools.lru_cache(256)
def muon_gated_workspace_size(dtype, slots, n, k, groups=1, backward=0):
    return _size(lib().muon_gated_workspace_size, dtype, slots, n, k, groups, backward)


@functools.lru_cache(256)
def muon_expert_workspace_size(dtype, slots, n, k, groups=1, backward=0):
    return _size(lib().muon_expert_workspace_size, dtype, slots, n, k, groups, backward)


def muon_gated_forward(x, wgate, wup, h, gate=None, up=None, offsets=None, rows=None, rows_per_token=1,
                       activation="silu", workspace=None):
    """h = act(x wgate^T) * (x wup^T), one kernel (see muon.h). x: tokens x k;
    wgate, wup: groups x n x k (or n x k: one group); h, and where given gate
    and up (what the backward pass reads): slots x n; offsets (groups + 1) and
    rows (slots): int32, as muon_route_forward writes them with rows_per_token
    = topk. Rows of the outputs behind the last group are left as they were.
    workspace: a uint8 tensor of muon_gated_workspace_size bytes (default: a
    temporary one)."""
    d = _enter(x)
    g, g_stride, groups = _stack("wgate", wgate, d)
    u, u_stride, groups_u = _stack("wup", wup, d)
    if groups != groups_u:
        raise ValueError("wgate and wup differ in their number of groups")
    h_mat = _mat("h", h, d)
    args = (_mat("x", x, d), g, g_stride, u, u_stride, groups, *_slots(offsets, rows, groups, h.shape[0], d), rows_per_token,
            _activation(activation), h_mat, _mat("gate", gate, d), _mat("up", up, d))
    need = muon_gated_workspace_size(_codes[x.dtype], h.shape[0], wgate.shape[-2], wgate.shape[-1], groups)
    _with_scratch(need, workspace, d, _lib.muon_gated_forward, *args)


def muon_gated_backward(dh, gate, up, wgate, wup, dgate, dup, dx=None, offsets=None, rows=None, activation="silu",
                        workspace=None):
    """dgate, dup (slots x n) and, where given, dx of the gated block (see
    muon.h): dx[rows[s]] = dgate[s] wgate + dup[s] wup (without rows: dx[s]).
    wgate and wup may be None without dx. workspace: a uint8 tensor of
    muon_gated_workspace_size bytes (default: a temporary one)."""
    d = _enter(dh)
    g = u = None
    g_stride = u_stride = 0
    groups = 1 if offsets is None else offsets.shape[0] - 1
    if wgate is not None or wup is not None or dx is not None:
        if wgate is None or wup is None:
            raise ValueError("wgate and wup: both are needed for dx")
        g, g_stride, groups = _stack("wgate", wgate, d)
        u, u_stride, groups_u = _stack("wup", wup, d)
        if groups != groups_u:
            raise ValueError("wgate and wup differ in their number of groups")
    dh_mat = _mat("dh", dh, d)
    args = (dh_mat, _mat("gate", gate, d), _mat("up", up, d), g, g_stride, u, u_stride, groups,
            *_slots(offsets, rows, groups, dh.shape[0], d), _activation(activation), _mat("dgate", dgate, d),
            _mat("dup", dup, d), _mat("dx", dx, d))
    need = 0 if dx is None else muon_gated_workspace_size(_codes[dh.dtype], dh.shape[0], wgate.shape[-2], wgate.shape[-1], groups, 1)
    _with_scratch(need, workspace, d, _lib.muon_gated_backward, *args)


def _expert(fn, back, x, w, y, offsets, rows, gather, scatter, workspace):
    if gather and scatter and rows is None:
        raise ValueError("rows: needed with gather and scatter, whose slots they count")
    d = _enter(x)
    w_mat, stride, groups = _stack("w", w, d)
    x_mat, y_mat = _mat("x", x, d), _mat("y", y, d)
    slots = x.shape[0] if not gather else y.shape[0] if not scatter else rows.shape[0]
    args = (x_mat, w_mat, stride, groups, slots, *_slots(offsets, rows, groups, slots, d), int(gather), int(scatter), y_mat)
    _with_scratch(muon_expert_workspace_size(_codes[x.dtype], slots, w.shape[-2], w.shape[-1], groups, back), workspace, d, fn, *args)


def muon_expert_forward(x, w, y, offsets=None, rows=None, gather=0, scatter=False, workspace=None):
    """y[p(s)] = x[q(s)] w_g^T over the slots of each group g (see muon.h). w:
    groups x n x k (or n x k: one group). gather: 0 (row s of x) or the rows
    per token (row rows[s] // gather); scatter: whether slot s writes row
    rows[s] of y instead of row s. workspace: a uint8 tensor of
    muon_expert_workspace_size bytes (default: a temporary one)."""
    _expert((_lib or lib()).muon_expert_forward, 0, x, w, y, offsets, rows, gather, scatter, workspace)


def muon_expert_backward(dy, w, dx, offsets=None, rows=None, gather=0, scatter=False, workspace=None):
    """dx[p(s)] = dy[q(s)] w_g (see muon.h); the arguments are those of
    muon_expert_forward."""
    _expert((_lib or lib()).muon_expert_backward, 1, dy, w, dx, offsets, rows, gather, scatter, workspace)


@functools.lru_cache(256)
def muon_combine_workspace_size(tokens, topk):
    return _size(lib().muon_combine_workspace_size, tokens, topk)


def _topk(x, y, weights, indices):
    """Rows of x for each row of y."""
    for t in (weights, indices):
        if t is not None:
            if t.dim() != 2:
                raise ValueError("weights and indices: expected 2-D tensors (tokens x topk)")
            return t.shape[1]
    tokens = y.shape[0]
    return x.shape[0] // tokens if tokens else 1


def muon_combine_forward(x, y, weights=None, indices=None, residual=None, p=0.0, key=None):
    """y[t] = residual[t] + drop(sum over j of weights[t, j] x[t topk + j])
    (see muon.h). x: (tokens topk) x cols; weights (float32), indices (int32):
    tokens x topk; topk is theirs, or the rows of x for each row of y. key: the
    generator's seed and offset, two int64 on the GPU, needed for p > 0."""
    d = _enter(x)
    x_mat, y_mat = _mat("x", x, d), _mat("y", y, d)
    topk = _topk(x, y, weights, indices)
    pair = (y.shape[0], topk)
    _check(_lib.muon_combine_forward(
        x_mat, topk, _vec("weights", weights, _torch.float32, pair, d), _vec("indices", indices, _torch.int32, pair, d),
        _mat("residual", residual, d), p, _vec("key", key, _torch.int64, (2,), d), y_mat))


def muon_combine_backward(dy, x, dx, dweights=None, weights=None, indices=None, rows=None, p=0.0, key=None,
                          workspace=None):
    """dx and, where given, dweights (tokens x topk float32) of
    muon_combine_forward (see muon.h), with the same weights, indices, p and
    key. rows (tokens topk int32, as muon_route_forward writes them): dx is
    written in their order instead of x's. x may be None without dweights.
    workspace: a uint8 tensor of muon_combine_workspace_size bytes, with rows
    (default: a temporary one)."""
    d = _enter(dy)
    dy_mat, dx_mat = _mat("dy", dy, d), _mat("dx", dx, d)
    topk = _topk(dx, dy, weights, indices)
    f32, i32, pair = _torch.float32, _torch.int32, (dy.shape[0], topk)
    args = (dy_mat, _mat("x", x, d), topk, _vec("weights", weights, f32, pair, d), _vec("indices", indices, i32, pair, d),
            _vec("rows", rows, i32, (pair[0] * topk,), d), p, _vec("key", key, _torch.int64, (2,), d), dx_mat,
            _vec("dweights", dweights, f32, pair, d))
    _with_scratch(muon_combine_workspace_size(*pair) if rows is not None else 0, workspace, d, _lib.muon_combine_backward, *args)


def muon_dropout_forward(x, y, p, key=None, residual=None):
    """y = residual + drop(x) (see muon.h); key as for muon_combine_forward."""
    d = _enter(x)
    _check(_lib.muon_dropout_forward(_mat("x", x, d), _mat("residual", residual, d), p,
                                     _vec("key", key, _torch.int64, (2,), d), _mat("y", y, d)))


def muon_dropout_backward(dy, dx, p, key=None):
    """dx = drop(dy), with p and key of the forward pass (see muon.h)."""
    d = _enter(dy)
    _check(_lib.muon_dropout_backward(_mat("dy", dy, d), p, _vec("key", key, _torch.int64, (2,), d), _mat("dx", dx, d)))
