"""MI355X (gfx950) MuonH optimizer step: Python binding of libmuonh.so.

The binding only marshals arguments: it groups matrices by shape, builds the
device arrays of device pointers the C ABI takes (include/muonh.h), allocates
the workspace with torch and passes torch's current HIP stream. Every step of
the optimizer runs in the library's HIP kernels. There is no fallback: if the
library is missing, the first call into it raises ImportError.

MuonH (digest page "Puro-2B trains for $6.9K, attention sinks hit 99%,
LoopArena tops at 24.69%", section "The load-bearing tricks aren't in the
abstract"; model card "Puro", section "Training"): momentum, Newton-Schulz
orthogonalization, then projection of every weight matrix back onto the
sphere of its initial Frobenius norm, with no weight decay.

MuonH(shapes, precision=..., grad_dtype=..., mom_dtype=...) runs the step
(step, step_timed) and, on the same plan, the Muon baseline with decoupled
weight decay (step_muon_wd); AdamW(numels) updates the parameters outside
the matrix group. Gradients and momenta may be float32 or bfloat16 tensors
(grad_dtype / mom_dtype); weights are float32.

fp8_quantize and fp8_matmul run the linear layers beside the step in e4m3
with a scale per block of 128 (model card "Puro", section "Training"; the
report page, part 6/7, section 4.3 "Cost Estimation": blockwise FP8), and
step(..., fp8=set) leaves the updated weights quantized for them.
"""
from __future__ import annotations

import ctypes
import functools
import re
from collections import OrderedDict
from pathlib import Path
from typing import Dict, List, Optional, Sequence, Tuple

_PKG = Path(__file__).resolve().parent
LIB_PATH = _PKG / "libmuonh.so"
HEADER_PATH = _PKG.parent / "include" / "muonh.h"

MUONH_OK = 0
MUONH_EINVAL = -1
MUONH_ESHAPE = -2
MUONH_EWORKSPACE = -3
MUONH_EHIP = -4
MUONH_ENOMEM = -5
MUONH_EALIAS = -6
MUONH_NS_FP32 = 1
MUONH_NS_SPLIT_BF16 = 2
MUONH_GRAD_BF16 = 4
MUONH_MOM_BF16 = 8
MUONH_NONFINITE_MOMENTUM = 1
MUONH_NONFINITE_UPDATE = 2
MUONH_FP8_ROWS = 0
MUONH_FP8_TILES = 1
MUONH_DT_FP32 = 0
MUONH_DT_BF16 = 1
MUONH_FP8_FAST = 256
MUONH_MAX_FP8_DIM = 1 << 24
# Bytes of muonh_step_noalloc's fixed per-GPU workspace (include/muonh.h).
MUONH_NOALLOC_WORKSPACE_BYTES = 128 << 20

# Newton-Schulz operand precision -> plan flag
PRECISIONS = {"bf16": 0, "split_bf16": MUONH_NS_SPLIT_BF16, "fp32": MUONH_NS_FP32}
# Storage dtype of the gradient / momentum -> whether it takes the bf16 flag
STATE_DTYPES = ("fp32", "bf16")

# Tensors per grouped AdamW launch (the library splits larger lists).
ADAMW_MAX_TENSORS_PER_LAUNCH = 128

NS_COEFFS = (3.4445, -4.7750, 2.0315)


class MuonHError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"muonh error {status}: {message}")
        self.status = status


class MuonHAliasError(MuonHError, ValueError):
    """MUONH_EALIAS: two of the W, G, M tensors overlap in memory."""

    def __init__(self, message: str):
        super().__init__(MUONH_EALIAS, message)


# Device pointer arrays kept per pointer tuple (a least-recently-used cache):
# a training loop that cycles through a few gradient buffers uploads each
# array once.
PTR_CACHE_ENTRIES = 64


class Fp8Desc(ctypes.Structure):
    """muonh_fp8_matrix."""
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("rows", ctypes.c_int64),
                ("cols", ctypes.c_int64), ("block", ctypes.c_int32)]


class Fp4Desc(ctypes.Structure):
    """muonh_fp4_matrix."""
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("rows", ctypes.c_int64),
                ("cols", ctypes.c_int64)]


class GroupDesc(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int32), ("cols", ctypes.c_int32), ("count", ctypes.c_int32)]


def _load_library() -> ctypes.CDLL:
    if not LIB_PATH.exists():
        raise ImportError(
            f"{LIB_PATH} is not built; run `python -m orthogonalized_updates_amd.build` "
            "(the MuonH step has no non-HIP implementation)")
    lib = ctypes.CDLL(str(LIB_PATH))
    vp, i32, i64, sz, f32 = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t,
                             ctypes.c_float)
    sig = {
        "muonh_abi_version": (i32, []),
        "muonh_plan_create": (ctypes.c_int, [ctypes.POINTER(vp), ctypes.POINTER(GroupDesc), i32,
                                             ctypes.c_uint32]),
        "muonh_plan_destroy": (None, [vp]),
        "muonh_plan_num_matrices": (i64, [vp]),
        "muonh_plan_num_params": (i64, [vp]),
        "muonh_workspace_bytes": (sz, [vp]),
        "muonh_init": (ctypes.c_int, [vp, vp, vp, vp, sz, vp]),
        "muonh_step": (ctypes.c_int, [vp, vp, vp, vp, vp, f32, f32, i32, vp, sz, vp]),
        "muonh_step_noalloc": (ctypes.c_int, [vp, vp, vp, vp, vp, f32, f32, i32, vp]),
        "muonh_step_timed": (ctypes.c_int, [vp, vp, vp, vp, vp, f32, f32, i32, vp, sz, vp,
                                            ctypes.POINTER(vp), i32]),
        "muonh_step_muon_wd": (ctypes.c_int, [vp, vp, vp, vp, f32, f32, f32, i32, vp, sz, vp]),
        "muonh_step_muon_wd_timed": (ctypes.c_int, [vp, vp, vp, vp, f32, f32, f32, i32, vp, sz,
                                                    vp, ctypes.POINTER(vp), i32]),
        "muonh_read_update": (ctypes.c_int, [vp, i64, vp, vp, sz, vp]),
        "muonh_adamw_step": (ctypes.c_int, [i32, vp, vp, vp, vp, vp, f32, f32, f32, f32, f32,
                                            i32, vp]),
        "muonh_step_status": (ctypes.c_int, [vp, vp, sz, vp, ctypes.POINTER(ctypes.c_uint32)]),
        "muonh_check_disjoint": (ctypes.c_int, [vp, vp, vp, vp]),
        "muonh_fp8_ld": (i64, [i64]),
        "muonh_fp8_scale_ld": (i64, [i64]),
        "muonh_fp8_scale_rows": (i64, [i64, i32]),
        "muonh_fp8_quantize": (ctypes.c_int, [vp, i32, i64, i64, i64, i32, vp, vp, vp, vp, vp]),
        "muonh_fp8_weights": (ctypes.c_int, [vp, vp, vp, vp, vp, vp, vp]),
        "muonh_fp8_matmul_workspace_bytes": (sz, [i64, i64, i64, i32]),
        "muonh_fp8_matmul": (ctypes.c_int, [ctypes.POINTER(Fp8Desc), ctypes.POINTER(Fp8Desc), vp,
                                            i32, i64, i32, vp, sz, vp]),
        "muonh_fp4_ld": (i64, [i64]),
        "muonh_fp4_scale_ld": (i64, [i64]),
        "muonh_fp4_quantize": (ctypes.c_int, [vp, i32, i64, i64, i64, vp, vp, vp, vp, vp]),
        "muonh_fp4_dequantize": (ctypes.c_int, [ctypes.POINTER(Fp4Desc), vp, i32, i64, vp]),
        "muonh_fp4_matmul_workspace_bytes": (sz, [i64, i64, i64]),
        "muonh_fp4_matmul": (ctypes.c_int, [ctypes.POINTER(Fp4Desc), ctypes.POINTER(Fp4Desc), vp, i32, i64, i32,
                                            vp, sz, vp]),
        "muonh_rms_norm": (ctypes.c_int, [vp, i32, i64, i64, i64, vp, i32, i64, vp, i64, vp, f32, vp, vp,
                                          i32, i64, vp, vp, vp, vp, vp]),
        "muonh_rms_norm_backward_workspace_bytes": (sz, [i64, i64]),
        "muonh_rms_norm_backward": (ctypes.c_int, [vp, i32, i64, vp, i32, i64, i64, i64, vp, vp, vp, i64,
                                                   vp, i64, vp, i32, vp, sz, vp]),
        "muonh_embedding": (ctypes.c_int, [vp, i32, i64, i64, vp, i32, i64, i64, i64, f32, vp, i32, i64, vp]),
        "muonh_embedding_backward_workspace_bytes": (sz, [i64, i64]),
        "muonh_embedding_backward": (ctypes.c_int, [vp, i32, i64, i64, vp, i32, i64, f32, vp, i64, i64, i64,
                                                    i32, vp, sz, vp]),
        "muonh_status_string": (ctypes.c_char_p, [ctypes.c_int]),
        "muonh_last_error": (ctypes.c_char_p, []),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


_LIB: Optional[ctypes.CDLL] = None


def get_lib() -> ctypes.CDLL:
    """The loaded libmuonh.so (loaded on first use; ImportError if not built)."""
    global _LIB
    if _LIB is None:
        _LIB = _load_library()
    return _LIB


def __getattr__(name):
    if name == "lib":
        return get_lib()
    raise AttributeError(name)


def check(status: int) -> None:
    if status != MUONH_OK:
        lib = get_lib()
        raise MuonHError(status, lib.muonh_last_error().decode(errors="replace")
                         or lib.muonh_status_string(status).decode())


def _precision(precision: str, ns_fp32: bool) -> str:
    if ns_fp32:
        if precision not in ("bf16", "fp32"):
            raise ValueError("ns_fp32=True conflicts with precision=%r" % (precision,))
        precision = "fp32"
    if precision not in PRECISIONS:
        raise ValueError("precision must be one of %s, got %r" % (sorted(PRECISIONS), precision))
    return precision


class Plan:
    """Owns a muonh_plan for shape groups [(rows, cols, count), ...].

    precision: Newton-Schulz operand precision, "bf16" (default),
    "split_bf16" (hi + lo bf16 pairs, three bf16 products each) or "fp32";
    ns_fp32=True is the same as precision="fp32". grad_dtype / mom_dtype:
    storage of G and M, "fp32" (default) or "bf16".
    """

    def __init__(self, groups: Sequence[Tuple[int, int, int]], ns_fp32: bool = False,
                 precision: str = "bf16", grad_dtype: str = "fp32", mom_dtype: str = "fp32"):
        precision = _precision(precision, ns_fp32)
        for name, v in (("grad_dtype", grad_dtype), ("mom_dtype", mom_dtype)):
            if v not in STATE_DTYPES:
                raise ValueError(f"{name} must be one of {STATE_DTYPES}, got {v!r}")
        flags = (PRECISIONS[precision] | (MUONH_GRAD_BF16 if grad_dtype == "bf16" else 0)
                 | (MUONH_MOM_BF16 if mom_dtype == "bf16" else 0))
        arr = (GroupDesc * len(groups))(*[GroupDesc(int(r), int(c), int(n)) for r, c, n in groups])
        handle = ctypes.c_void_p()
        check(get_lib().muonh_plan_create(ctypes.byref(handle), arr, len(groups), flags))
        self.handle = handle
        self.groups = [tuple(int(v) for v in g) for g in groups]
        self.precision = precision
        self.ns_fp32 = precision == "fp32"
        self.grad_dtype = grad_dtype
        self.mom_dtype = mom_dtype

    @property
    def num_matrices(self) -> int:
        return int(get_lib().muonh_plan_num_matrices(self.handle))

    @property
    def num_params(self) -> int:
        return int(get_lib().muonh_plan_num_params(self.handle))

    @property
    def workspace_bytes(self) -> int:
        return int(get_lib().muonh_workspace_bytes(self.handle))

    def __del__(self):
        h = getattr(self, "handle", None)
        if h is not None and h.value and _LIB is not None:
            _LIB.muonh_plan_destroy(h)
            self.handle = None


class _PtrArrays:
    """Device arrays of device pointers, one per pointer tuple, kept in a
    least-recently-used cache of PTR_CACHE_ENTRIES. A new array is copied
    from pinned host memory without blocking (the copy is ordered on the
    current stream before the launch that reads it; torch keeps the pinned
    buffer until the copy is done), so changing pointers never waits for
    the GPU. Each use records the current stream on the array, so that an
    array evicted while a launch on another stream still reads it is not
    reused before that launch completes."""

    def __init__(self, torch, device):
        self.torch = torch
        self.device = device
        self.cache: "OrderedDict" = OrderedDict()

    def get(self, ptrs: Tuple[int, ...]) -> int:
        torch = self.torch
        arr = self.cache.get(ptrs)
        if arr is None:
            host = torch.tensor(ptrs, dtype=torch.int64).pin_memory()
            arr = host.to(self.device, non_blocking=True)
            self.cache[ptrs] = arr
            if len(self.cache) > PTR_CACHE_ENTRIES:
                self.cache.popitem(last=False)
        else:
            self.cache.move_to_end(ptrs)
        arr.record_stream(torch.cuda.current_stream(self.device))
        return int(arr.data_ptr())


class MuonH:
    """MuonH over a list of fp32 weight matrices on one GPU.

    shapes: (rows, cols) of each matrix, in the caller's order. Matrices are
    grouped by shape internally; every method takes and returns lists in the
    caller's order. grad_dtype / mom_dtype ("fp32" or "bf16"): the torch
    dtype the gradients / momenta must have (float32 or bfloat16).
    """

    def __init__(self, shapes: Sequence[Tuple[int, int]], *, ns_fp32: bool = False,
                 precision: str = "bf16", grad_dtype: str = "fp32", mom_dtype: str = "fp32",
                 device=None):
        import torch
        get_lib()
        self.torch = torch
        self.shapes = [(int(r), int(c)) for r, c in shapes]
        if not self.shapes:
            raise ValueError("MuonH needs at least one matrix")
        dev = torch.device(device if device is not None else "cuda")
        if dev.type != "cuda":
            raise ValueError("MuonH runs on a ROCm GPU device only")
        if dev.index is None:
            dev = torch.device("cuda", torch.cuda.current_device())
        self.device = dev
        buckets: Dict[Tuple[int, int], List[int]] = {}
        for i, s in enumerate(self.shapes):
            buckets.setdefault(s, []).append(i)
        self.plan_order: List[int] = [i for idx in buckets.values() for i in idx]
        self.plan_index = {caller: p for p, caller in enumerate(self.plan_order)}
        self.plan = Plan([(r, c, len(idx)) for (r, c), idx in buckets.items()], ns_fp32=ns_fp32,
                         precision=precision, grad_dtype=grad_dtype, mom_dtype=mom_dtype)
        tdt = {"fp32": torch.float32, "bf16": torch.bfloat16}
        self._dtypes = {"weights": torch.float32, "grads": tdt[grad_dtype],
                        "moms": tdt[mom_dtype]}
        nbytes = max(self.plan.workspace_bytes, 256)
        self.workspace = torch.empty(nbytes, dtype=torch.uint8, device=self.device)
        if self.workspace.data_ptr() % 256:
            raise MuonHError(MUONH_EWORKSPACE, "torch returned a workspace that is not 256-aligned")
        self.R = torch.zeros(len(self.shapes), dtype=torch.float32, device=self.device)
        self._ptrs = _PtrArrays(torch, self.device)
        self._disjoint_ok: "OrderedDict" = OrderedDict()  # (W, G, M) pointer tuples checked

    # -- marshalling ------------------------------------------------------
    def _check(self, tensors, name: str):
        torch = self.torch
        if len(tensors) != len(self.shapes):
            raise ValueError(f"{name}: expected {len(self.shapes)} tensors, got {len(tensors)}")
        dt = self._dtypes[name]
        for i, t in enumerate(tensors):
            if not isinstance(t, torch.Tensor) or t.dtype != dt:
                raise TypeError(f"{name}[{i}] must be a {dt} torch tensor")
            if t.device != self.device:
                raise ValueError(f"{name}[{i}] is on {t.device}, expected {self.device}")
            if tuple(t.shape) != self.shapes[i] or not t.is_contiguous():
                raise ValueError(f"{name}[{i}] must be a contiguous {self.shapes[i]} tensor")

    def _check_state(self, weights, grads, moms):
        """Types and shapes of W, G and M, and that no two of their tensors
        overlap in memory (the step updates W and M in place and reads G).
        The library checks the byte ranges on the host
        (muonh_check_disjoint), once per combination of pointers; an overlap
        raises MuonHAliasError (a ValueError) naming the caller's tensors."""
        self._check(weights, "weights")
        self._check(grads, "grads")
        self._check(moms, "moms")
        ptrs = [tuple(int(ts[c].data_ptr()) for c in self.plan_order)
                for ts in (weights, grads, moms)]
        key = tuple(ptrs)
        if key in self._disjoint_ok:
            self._disjoint_ok.move_to_end(key)
            return
        arrs = [(ctypes.c_void_p * len(p))(*p) for p in ptrs]
        st = get_lib().muonh_check_disjoint(self.plan.handle, *arrs)
        if st == MUONH_EALIAS:
            raise MuonHAliasError(self._caller_names(get_lib().muonh_last_error().decode()))
        check(st)
        self._disjoint_ok[key] = True
        if len(self._disjoint_ok) > PTR_CACHE_ENTRIES:
            self._disjoint_ok.popitem(last=False)

    def _caller_names(self, msg: str) -> str:
        """The library names matrices by plan index ("G[3] overlaps W[3]");
        translate to the caller's lists and indices."""
        names = {"W": "weights", "G": "grads", "M": "moms"}

        def repl(m):
            return f"{names[m.group(1)]}[{self.plan_order[int(m.group(2))]}]"
        return re.sub(r"\b([WGM])\[(\d+)\]", repl, msg) + "; W, G and M must be disjoint"

    def _ptr_array(self, name: str, tensors) -> int:
        return self._ptrs.get(tuple(int(tensors[c].data_ptr()) for c in self.plan_order))

    def _stream(self) -> int:
        return int(self.torch.cuda.current_stream(self.device).cuda_stream)

    # -- API ----------------------------------------------------------------
    def init(self, weights) -> "object":
        """R[i] = ||W0[i]||_F (device float32, caller order)."""
        self._check(weights, "weights")
        r_plan = self.torch.empty_like(self.R)
        check(get_lib().muonh_init(self.plan.handle, self._ptr_array("W", weights), r_plan.data_ptr(),
                             self.workspace.data_ptr(), self.workspace.numel(), self._stream()))
        inv = self.torch.tensor(self.plan_order, dtype=self.torch.int64, device=self.device)
        self.R = self.torch.empty_like(r_plan).index_copy_(0, inv, r_plan)
        self._R_plan = r_plan
        return self.R

    def set_radius(self, radius) -> None:
        """Restore R (caller order), e.g. from a checkpoint."""
        r = radius.to(device=self.device, dtype=self.torch.float32).contiguous()
        if r.numel() != len(self.shapes):
            raise ValueError("radius must have one entry per matrix")
        self.R = r
        inv = self.torch.tensor(self.plan_order, dtype=self.torch.int64, device=self.device)
        self._R_plan = r.index_select(0, inv)

    def step(self, weights, grads, moms, lr: float, beta: float = 0.95, ns_iters: int = 5,
             fp8: "Optional[Fp8Weights]" = None) -> None:
        """One MuonH step: moms and weights are updated in place. With `fp8`
        (a set from fp8_weights()), the updated weights are then quantized
        into it, as quantize_weights() does."""
        self._check_state(weights, grads, moms)
        if not hasattr(self, "_R_plan"):
            raise RuntimeError("call init() (or set_radius()) before step()")
        if fp8 is not None:
            self._check_fp8(fp8, weights, grads, moms)
        check(get_lib().muonh_step(self.plan.handle, self._ptr_array("W", weights),
                             self._ptr_array("G", grads), self._ptr_array("M", moms),
                             self._R_plan.data_ptr(), float(lr), float(beta), int(ns_iters),
                             self.workspace.data_ptr(), self.workspace.numel(), self._stream()))
        if fp8 is not None:
            self._quantize(weights, fp8)

    def step_noalloc(self, weights, grads, moms, lr: float, beta: float = 0.95,
                     ns_iters: int = 5) -> None:
        """step() without this object's workspace (muonh_step_noalloc): the
        library's fixed per-GPU array of MUONH_NOALLOC_WORKSPACE_BYTES serves
        instead, for plans that fit it. read_update() and status() do not
        see such a step. The pointer arrays are still device tensors of this
        object (uploaded once per pointer combination)."""
        self._check_state(weights, grads, moms)
        if not hasattr(self, "_R_plan"):
            raise RuntimeError("call init() (or set_radius()) before step_noalloc()")
        check(get_lib().muonh_step_noalloc(self.plan.handle, self._ptr_array("W", weights),
                                           self._ptr_array("G", grads),
                                           self._ptr_array("M", moms), self._R_plan.data_ptr(),
                                           float(lr), float(beta), int(ns_iters),
                                           self._stream()))

    def step_timed(self, weights, grads, moms, lr: float, beta: float, ns_iters: int,
                   events) -> None:
        """step() plus hipEventRecord of `events` (torch.cuda.Event list of
        length 3*ns_iters+3, already recorded once) at the phase boundaries."""
        self._check_state(weights, grads, moms)
        if not hasattr(self, "_R_plan"):
            raise RuntimeError("call init() (or set_radius()) before step_timed()")
        arr = (ctypes.c_void_p * len(events))(*[int(e.cuda_event) for e in events])
        check(get_lib().muonh_step_timed(self.plan.handle, self._ptr_array("W", weights),
                                   self._ptr_array("G", grads), self._ptr_array("M", moms),
                                   self._R_plan.data_ptr(), float(lr), float(beta), int(ns_iters),
                                   self.workspace.data_ptr(), self.workspace.numel(),
                                   self._stream(), arr, len(events)))

    def step_muon_wd(self, weights, grads, moms, lr: float, beta: float = 0.95,
                     weight_decay: float = 0.1, ns_iters: int = 5, events=None,
                     fp8: "Optional[Fp8Weights]" = None) -> None:
        """The baseline MuonH is measured against: Muon with decoupled weight
        decay, W <- (1 - lr*wd) W - lr O (no projection, no radius). With
        `events` (as for step_timed), records the phase boundaries; `fp8` as
        for step() (after the last event)."""
        self._check_state(weights, grads, moms)
        if fp8 is not None:
            self._check_fp8(fp8, weights, grads, moms)
        args = [self.plan.handle, self._ptr_array("W", weights), self._ptr_array("G", grads),
                self._ptr_array("M", moms), float(lr), float(beta), float(weight_decay),
                int(ns_iters), self.workspace.data_ptr(), self.workspace.numel(), self._stream()]
        if events is None:
            check(get_lib().muonh_step_muon_wd(*args))
        else:
            arr = (ctypes.c_void_p * len(events))(*[int(e.cuda_event) for e in events])
            check(get_lib().muonh_step_muon_wd_timed(*args, arr, len(events)))
        if fp8 is not None:
            self._quantize(weights, fp8)

    # -- 8-bit weights ------------------------------------------------------
    def fp8_weights(self, transposed: bool = True) -> "Fp8Weights":
        """Storage for this optimizer's weights in e4m3 with 128 x 128 scales:
        .weights[i] is matrix i as the forward product reads it,
        .transposed[i] its transpose (for the data gradient). Contents are
        undefined until a quantize_weights() or a step(..., fp8=set)."""
        return Fp8Weights(self.shapes, self.device, transposed, self.plan_order)

    def quantize_weights(self, weights, out: "Fp8Weights") -> "Fp8Weights":
        """Quantize the weights into `out` (a set from fp8_weights()), in
        grouped launches (muonh_fp8_weights)."""
        self._check(weights, "weights")
        self._check_fp8(out, weights)
        self._quantize(weights, out)
        return out

    def _check_fp8(self, out, *lists) -> None:
        if not isinstance(out, Fp8Weights):
            raise TypeError("expected an Fp8Weights set (see fp8_weights())")
        if out.shapes != self.shapes or out.device != self.device or out.order != self.plan_order:
            raise ValueError("the Fp8Weights set has other shapes or another device")
        lo, hi = out.span
        if not lo <= out.arrays[0] < hi:
            raise ValueError("the Fp8Weights set's memory was moved, or it is a copy: its pointers are another's")
        for ts in lists:
            for t in ts:
                p = t.data_ptr()
                if p < hi and lo < p + t.numel() * t.element_size():
                    raise MuonHAliasError("a tensor of the call overlaps the Fp8Weights set")

    def _quantize(self, weights, out) -> None:
        # the launch reads the set's pointer arrays and writes its matrices,
        # perhaps on another stream than the one they were made on
        out.memory.record_stream(self.torch.cuda.current_stream(self.device))
        _on_device(self.torch, self.device, get_lib().muonh_fp8_weights, self.plan.handle,
                   self._ptr_array("W", weights), *out.arrays)
        _written(out.memory)

    def read_update(self, index: int):
        """The update O of matrix `index` from the last step (fp32, rows x cols)."""
        r, c = self.shapes[index]
        out = self.torch.empty((r, c), dtype=self.torch.float32, device=self.device)
        check(get_lib().muonh_read_update(self.plan.handle, self.plan_index[index], out.data_ptr(),
                                    self.workspace.data_ptr(), self.workspace.numel(),
                                    self._stream()))
        return out

    def status(self) -> int:
        """Non-finite bits of the last step (MUONH_NONFINITE_MOMENTUM: a
        momentum norm was NaN or infinite; MUONH_NONFINITE_UPDATE: a trial
        update norm was). Waits for the current stream."""
        flags = ctypes.c_uint32(0)
        check(get_lib().muonh_step_status(self.plan.handle, self.workspace.data_ptr(),
                                          self.workspace.numel(), self._stream(),
                                          ctypes.byref(flags)))
        return int(flags.value)


__all__ = ["MuonH", "Plan", "MuonHError", "GroupDesc", "get_lib", "check", "LIB_PATH", "HEADER_PATH",
           "NS_COEFFS", "MUONH_OK", "MUONH_EINVAL", "MUONH_ESHAPE", "MUONH_EWORKSPACE",
           "MUONH_EHIP", "MUONH_ENOMEM", "MUONH_EALIAS", "MuonHAliasError", "MUONH_NS_FP32", "MUONH_NS_SPLIT_BF16", "MUONH_GRAD_BF16",
           "MUONH_MOM_BF16", "MUONH_NONFINITE_MOMENTUM", "MUONH_NONFINITE_UPDATE",
           "MUONH_NOALLOC_WORKSPACE_BYTES", "AdamW",
           "PTR_CACHE_ENTRIES", "Fp8Matrix", "Fp8Weights", "fp8_quantize", "fp8_matmul",
           "MUONH_FP8_ROWS", "MUONH_FP8_TILES", "MUONH_FP8_FAST", "MUONH_DT_FP32", "MUONH_DT_BF16",
           "MUONH_MAX_FP8_DIM", "rms_norm", "rms_norm_fp8", "rms_norm_backward",
           "embedding", "embedding_backward", "Fp4Matrix", "fp4_quantize", "fp4_matmul"]


class AdamW:
    """AdamW over a list of fp32 tensors on one GPU: the parameters outside
    the MuonH group (model card page "Puro", section "Training": AdamW with
    weight decay 0.1). Any shapes; tensors are treated as flat arrays and
    updated in place by the library's grouped HIP launch (muonh_adamw_step).
    """

    def __init__(self, numels: Sequence[int], *, device=None):
        import torch
        get_lib()
        self.torch = torch
        self.numels = [int(n) for n in numels]
        if any(n < 0 for n in self.numels):
            raise ValueError("numels must be >= 0")
        dev = torch.device(device if device is not None else "cuda")
        if dev.type != "cuda":
            raise ValueError("AdamW runs on a ROCm GPU device only")
        if dev.index is None:
            dev = torch.device("cuda", torch.cuda.current_device())
        self.device = dev
        self._sizes = (ctypes.c_int64 * max(len(self.numels), 1))(*self.numels)
        self._ptrs = _PtrArrays(torch, self.device)

    def _check(self, tensors, name: str):
        torch = self.torch
        if len(tensors) != len(self.numels):
            raise ValueError(f"{name}: expected {len(self.numels)} tensors, got {len(tensors)}")
        for i, t in enumerate(tensors):
            if not isinstance(t, torch.Tensor) or t.dtype != torch.float32:
                raise TypeError(f"{name}[{i}] must be a float32 torch tensor")
            if t.device != self.device:
                raise ValueError(f"{name}[{i}] is on {t.device}, expected {self.device}")
            if t.numel() != self.numels[i] or not t.is_contiguous():
                raise ValueError(f"{name}[{i}] must be contiguous with {self.numels[i]} elements")

    def _ptr_array(self, name: str, tensors) -> int:
        return self._ptrs.get(tuple(int(t.data_ptr()) for t in tensors))

    def step(self, params, grads, exp_avg, exp_avg_sq, lr: float, beta1: float = 0.9,
             beta2: float = 0.95, eps: float = 1e-8, weight_decay: float = 0.1,
             step: int = 1) -> None:
        """One AdamW step (1-based `step`); params, exp_avg, exp_avg_sq in place."""
        for ts, nm in ((params, "params"), (grads, "grads"), (exp_avg, "exp_avg"),
                       (exp_avg_sq, "exp_avg_sq")):
            self._check(ts, nm)
        if not self.numels:
            return
        stream = int(self.torch.cuda.current_stream(self.device).cuda_stream)
        check(get_lib().muonh_adamw_step(
            len(self.numels), ctypes.cast(self._sizes, ctypes.c_void_p),
            self._ptr_array("P", params), self._ptr_array("G", grads),
            self._ptr_array("M", exp_avg), self._ptr_array("V", exp_avg_sq),
            float(lr), float(beta1), float(beta2), float(eps), float(weight_decay), int(step),
            stream))


# -- block-scaled 8-bit matrices ---------------------------------------------
# Entries per scale along a row, and per tile edge (include/muonh.h).
FP8_BLOCK = 128
FP8_BLOCKS = {"rows": MUONH_FP8_ROWS, "tiles": MUONH_FP8_TILES}
FP8_FORMS = ("plain", "transposed", "both")


def _up(v: int, m: int) -> int:
    return -(-v // m) * m


@functools.lru_cache(maxsize=1024)
def _fp8_layout(rows: int, cols: int, block: str):
    """(codes shape, scales shape) of a rows x cols matrix."""
    if block not in FP8_BLOCKS:
        raise ValueError(f"block must be one of {sorted(FP8_BLOCKS)}, got {block!r}")
    if not (0 <= rows <= MUONH_MAX_FP8_DIM and 0 <= cols <= MUONH_MAX_FP8_DIM):
        raise ValueError(f"shape {(rows, cols)} out of [0, {MUONH_MAX_FP8_DIM}]")
    srows = rows if block == "rows" else -(-rows // FP8_BLOCK)
    return (rows, _up(cols, FP8_BLOCK)), (srows, _up(-(-cols // FP8_BLOCK), 4))


def _check_part(name: str, t, dtype, shape) -> None:
    if getattr(t, "dtype", None) != dtype:
        raise TypeError(f"{name} must be a {dtype} torch tensor")
    if t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {shape} tensor")


class _BlockMatrix:
    """Codes and scales in their layout, whose addresses `desc` holds: read-only attributes."""
    __slots__ = ("codes", "scales", "shape", "device", "desc")

    def __setattr__(self, name, value):
        kind = type(self).__name__
        raise AttributeError(f"{kind}.{name} is read-only; make another {kind}")

    __delattr__ = functools.partialmethod(__setattr__, value=None)


class Fp8Matrix(_BlockMatrix):
    """A rows x cols matrix held as e4m3 codes with a power-of-two scale per
    block (muonh_fp8_matrix): per 128 columns of a row (block="rows") or per
    128 x 128 entries ("tiles").

    codes: torch.float8_e4m3fn, rows x (cols rounded up to 128), zeros past
    cols; scales: torch.float8_e8m0fnu, (rows, or rows/128 rounded up) x
    (cols/128 rounded up, then to a multiple of 4); the byte 255 is NaN. Both
    contiguous, on one GPU. shape: (rows, cols). The attributes are read-only, since `desc` holds
    the tensors' addresses: write into codes and scales, or make another
    Fp8Matrix. A matrix whose tensors were moved or resized in place is
    refused by the calls that take it.
    """
    __slots__ = ("block",)

    def _set(self, codes, scales, shape, block) -> None:
        put = object.__setattr__
        put(self, "codes", codes)
        put(self, "scales", scales)
        put(self, "shape", shape)
        put(self, "block", block)
        put(self, "device", codes.device)
        put(self, "desc", Fp8Desc(codes.data_ptr(), scales.data_ptr(), shape[0], shape[1], FP8_BLOCKS[block]))

    def __reduce__(self):  # copies and pickles take the addresses of their own tensors
        return Fp8Matrix, (self.codes, self.scales, self.shape, self.block)

    def __init__(self, codes, scales, shape: Tuple[int, int], block: str = "rows"):
        import torch
        rows, cols = int(shape[0]), int(shape[1])
        c, e = _fp8_layout(rows, cols, block)
        _check_part("codes", codes, torch.float8_e4m3fn, c)
        _check_part("scales", scales, torch.float8_e8m0fnu, e)
        if codes.device != scales.device or codes.device.type != "cuda":
            raise ValueError("codes and scales must be on one ROCm GPU")
        self._set(codes, scales, (rows, cols), block)

    @classmethod
    def empty(cls, rows: int, cols: int, block: str = "rows", device=None) -> "Fp8Matrix":
        """Storage with undefined contents."""
        import torch
        c, s = _fp8_layout(rows, cols, block)
        dev = device if isinstance(device, torch.device) else torch.device("cuda" if device is None else device)
        if dev.type != "cuda":
            raise ValueError("codes and scales must be on one ROCm GPU")
        # made in its layout, so without __init__'s checks
        m = cls.__new__(cls)
        m._set(torch.empty(c, dtype=torch.float8_e4m3fn, device=dev),
               torch.empty(s, dtype=torch.float8_e8m0fnu, device=dev), (rows, cols), block)
        return m

    def dequantize(self):
        """The values it stands for, fp32 (torch operations; for inspection)."""
        rows, cols = self.shape
        s = self.scales[:, :-(-cols // FP8_BLOCK)].float()
        if self.block == "tiles":
            s = s.repeat_interleave(FP8_BLOCK, 0)[:rows]
        return self.codes[:, :cols].float() * s.repeat_interleave(FP8_BLOCK, 1)[:, :cols]


def _held(name: str, m: _BlockMatrix):
    """m's descriptor, if its tensors are where they were."""
    d = m.desc
    if m.codes.data_ptr() != (d.codes or 0) or m.scales.data_ptr() != (d.scales or 0):
        raise ValueError(f"{name}'s codes or scales were moved since the {type(m).__name__} was made")
    return d


class Fp8Weights:
    """The weights of a MuonH optimizer in 8 bits (MuonH.fp8_weights): lists
    of Fp8Matrix with block "tiles" in the caller's order, `weights` and
    `transposed` (empty without transposed forms). They and the device arrays
    of pointers to their parts (`order`: matrices in plan order) share one
    allocation, which any of the matrices keeps alive, and every call that
    writes the set records its stream on it. A captured graph that does must
    not outlive all of them, nor the optimizer."""

    def __init__(self, shapes, device, transposed: bool, order: Sequence[int]):
        import torch
        self.shapes = list(shapes)
        self.device = device
        self.order = list(order)
        self.weights: List[Fp8Matrix] = []
        self.transposed: List[Fp8Matrix] = []
        places, total = [], 0
        for r, c in self.shapes:
            for shape, to in ((r, c), self.weights), ((c, r), self.transposed):
                if to is self.transposed and not transposed:
                    continue
                at = []
                for h, w in _fp8_layout(*shape, "tiles"):
                    at.append((total, h, w))
                    total = _up(total + h * w, 256)
                places.append((shape, to, at))
        parts = ("codes", "scales")
        sets = 2 if transposed else 1
        nptrs = len(parts) * sets * len(self.order)
        self.memory = torch.empty(total + 8 * nptrs, dtype=torch.uint8, device=device)
        self.storage = self.memory[:total]  # codes and scales; the pointers follow
        for shape, to, at in places:
            held = [self.storage[o:o + h * w].view(dt).view(h, w)
                    for (o, h, w), dt in zip(at, (torch.float8_e4m3fn, torch.float8_e8m0fnu))]
            to.append(Fp8Matrix(*held, shape, "tiles"))
        ptrs = [getattr(ms[i], part).data_ptr() for ms in (self.weights, self.transposed)[:sets] for part in parts
                for i in self.order]
        self.memory[total:].view(torch.int64).copy_(torch.tensor(ptrs, dtype=torch.int64))
        # codes, scales, codes_t, scales_t of muonh_fp8_weights
        at = int(self.memory.data_ptr()) + total
        self.arrays = [at + 8 * len(self.order) * i if i < len(parts) * sets else None for i in range(4)]

    @property
    def span(self) -> Tuple[int, int]:
        p = int(self.memory.data_ptr())
        return p, p + self.memory.numel()


def _fp8_dt(torch, dtype) -> int:
    if dtype == torch.float32:
        return MUONH_DT_FP32
    if dtype == torch.bfloat16:
        return MUONH_DT_BF16
    raise TypeError(f"expected torch.float32 or torch.bfloat16, got {dtype}")


def _row_pitch(t, name: str) -> int:
    """Elements between the rows of a 2-d tensor whose rows are contiguous."""
    rows, cols = t.shape
    ld, step = t.stride()
    if cols > 1 and step != 1:
        raise ValueError(f"{name}'s rows must be contiguous (stride 1 along columns)")
    if rows <= 1:
        return max(cols, 1)
    if ld < cols:
        raise ValueError(f"{name}'s rows overlap")
    return ld


def _on_device(torch, dev, fn, *args) -> None:
    """fn(*args, stream) with dev current, on its current stream. The raw
    stream handle and the comparison cost well under a microsecond; a device
    guard and a Stream object on every call took about a third of a small
    call's host time."""
    if torch.cuda.current_device() == dev.index:
        check(fn(*args, torch._C._cuda_getCurrentRawStream(dev.index)))
    else:
        with torch.cuda.device(dev):
            check(fn(*args, torch._C._cuda_getCurrentRawStream(dev.index)))


@functools.lru_cache(maxsize=None)
def _increment_version():
    from torch.autograd.graph import increment_version
    return increment_version


def _written(*tensors) -> None:
    """Tells autograd that the library wrote into the tensors, so that a
    backward pass that saved one of them before refuses to use it."""
    _increment_version()(tensors)


def fp8_quantize(x, block: str = "rows", forms: str = "plain",
                 out: Optional[Fp8Matrix] = None, out_t: Optional[Fp8Matrix] = None):
    """Quantize x (a 2-d fp32 or bf16 tensor on the GPU whose rows are
    contiguous, any row stride) to block-scaled e4m3 (muonh_fp8_quantize).

    forms: "plain" (x itself), "transposed" (its transpose: with block "rows",
    grouped along x's rows) or "both", in one pass. Returns (q, q_t), None in
    the place of a form that was not asked for. out / out_t: matrices to
    write into instead of new ones. Runs on the current stream of x's device.
    Autograd does not see it: the results carry no gradient to x, and a
    backward pass is the caller's (fp8_matmul).
    """
    import torch
    if not isinstance(x, torch.Tensor):
        raise TypeError("x must be a torch tensor")
    dt = _fp8_dt(torch, x.dtype)
    dev = x.device
    if x.dim() != 2 or dev.type != "cuda":
        raise ValueError("x must be a 2-d tensor on a ROCm GPU")
    if forms not in FP8_FORMS:
        raise ValueError(f"forms must be one of {FP8_FORMS}, got {forms!r}")
    rows, cols = x.shape
    ld = _row_pitch(x, "x")
    q = _form("out", out, forms != "transposed", rows, cols, block, dev)
    qt = _form("out_t", out_t, forms != "plain", cols, rows, block, dev)
    d, t = _NO_FORM if q is None else q.desc, _NO_FORM if qt is None else qt.desc
    _on_device(torch, dev, get_lib().muonh_fp8_quantize, x.data_ptr(), dt, rows, cols, ld,
               FP8_BLOCKS[block], d.codes, d.scales, t.codes, t.scales)
    for o in (out, out_t):
        if o is not None:
            _written(o.codes, o.scales)
    return q, qt


_NO_FORM = Fp8Desc(None, None, 0, 0, 0)


def _form(name: str, o, wanted: bool, rows: int, cols: int, block: str, dev):
    """The output for one form of fp8_quantize: `o` checked, a new one, or None."""
    if not wanted:
        if o is not None:
            raise ValueError(f"{name} given for a form that was not asked for")
        return None
    if o is None:
        return Fp8Matrix.empty(rows, cols, block, dev)
    if not isinstance(o, Fp8Matrix):
        raise TypeError(f"{name} must be an Fp8Matrix")
    if o.shape != (rows, cols) or o.block != block or o.device != dev:
        raise ValueError(f"{name} must be a {(rows, cols)} Fp8Matrix of block {block!r} on {dev}")
    _held(name, o)
    return o


def fp8_matmul(a: Fp8Matrix, b: Fp8Matrix, out=None, out_dtype=None, accumulate: bool = False,
               fast: bool = False):
    """out[i][j] = sum_k a[i][k] * b[j][k] (muonh_fp8_matmul), plus out's old
    values with accumulate=True.

    out: a 2-d fp32 or bf16 tensor (a rows x b rows) whose rows are
    contiguous; otherwise a new one of out_dtype (default bfloat16). The
    products of a linear layer Y = X W^T: matmul(X, W); dX = matmul(dY, W_t);
    G += matmul(dY_t, X_t) into the gradient the optimizer step reads. Runs on
    the current stream of the operands' device.

    Sums are fp32; entries of 2^128 and more count as infinite and those below
    2^-130 to within 2^-134. fast=True, for bf16 results, takes 8-bit matrix
    instructions instead, up to twice as fast, whose sums hold fewer bits: a
    result is off by up to 15 * 2^-13 * sum_k |a[i][k] * b[j][k]|.

    Autograd does not see the product: its result carries no gradient, and
    the caller runs the two others in the backward pass of a
    torch.autograd.Function, say. Only the version of a given `out` moves on.
    """
    import torch
    for name, m in (("a", a), ("b", b)):
        if not isinstance(m, Fp8Matrix):
            raise TypeError(f"{name} must be an Fp8Matrix")
    da, db = _held("a", a), _held("b", b)
    dev = a.device
    if dev != b.device:
        raise ValueError(f"a is on {dev}, b on {b.device}")
    if a.shape[1] != b.shape[1]:
        raise ValueError(f"a has {a.shape[1]} columns, b {b.shape[1]}")
    m, n = shape = (a.shape[0], b.shape[0])
    if out is None:
        if accumulate:
            raise ValueError("accumulate=True needs out")
        out_dtype = torch.bfloat16 if out_dtype is None else out_dtype
        dt = _fp8_dt(torch, out_dtype)
        out, given = torch.empty(shape, device=dev, dtype=out_dtype), False
    else:
        given = True
        if not isinstance(out, torch.Tensor):
            raise TypeError("out must be a torch tensor")
        dt = _fp8_dt(torch, out.dtype)
        if out_dtype is not None and out_dtype != out.dtype:
            raise ValueError(f"out is {out.dtype}, out_dtype {out_dtype}")
        if tuple(out.shape) != shape or out.device != dev:
            raise ValueError(f"out must be a {shape} tensor on {dev}")
    if fast:
        if dt != MUONH_DT_BF16:
            raise ValueError("fast=True gives bfloat16 results only")
        dt |= MUONH_FP8_FAST
    ld = _row_pitch(out, "out")
    lib = get_lib()
    nbytes = lib.muonh_fp8_matmul_workspace_bytes(m, n, a.shape[1], dt)
    # from torch's allocator on the current stream: calls on other streams and
    # captured graphs get memory of their own
    ws = torch.empty(nbytes, dtype=torch.uint8, device=dev) if nbytes else None
    _on_device(torch, dev, lib.muonh_fp8_matmul, da, db, out.data_ptr(), dt, ld,
               1 if accumulate else 0, None if ws is None else ws.data_ptr(), nbytes)
    if given:
        _written(out)
    return out


# -- microscaled 4-bit matrices ------------------------------------------------
FP4_GROUP = 32  # entries per scale along a row (include/muonh.h)


@functools.lru_cache(maxsize=1024)
def _fp4_layout(rows: int, cols: int):
    """(codes shape, scales shape) of a rows x cols matrix, in bytes."""
    if not (0 <= rows <= MUONH_MAX_FP8_DIM and 0 <= cols <= MUONH_MAX_FP8_DIM):
        raise ValueError(f"shape {(rows, cols)} out of [0, {MUONH_MAX_FP8_DIM}]")
    return (rows, _up(cols, 256) // 2), (rows, _up(cols, 256) // FP4_GROUP)


class Fp4Matrix(_BlockMatrix):
    """A rows x cols matrix held as e2m1 codes with a power-of-two scale per 32
    columns of a row (muonh_fp4_matrix).

    codes: torch.float4_e2m1fn_x2 (two codes to a byte, the first in the low half),
    rows x (cols rounded up to 256, over 2), zeros past cols; scales:
    torch.float8_e8m0fnu, rows x (cols rounded up to 256, over 32); the byte 255 is
    NaN. Both contiguous, on one GPU. shape: (rows, cols). Read-only attributes, and
    moved tensors, as for Fp8Matrix.
    """
    __slots__ = ()

    def _set(self, codes, scales, shape) -> None:
        put = object.__setattr__
        put(self, "codes", codes)
        put(self, "scales", scales)
        put(self, "shape", shape)
        put(self, "device", codes.device)
        put(self, "desc", Fp4Desc(codes.data_ptr(), scales.data_ptr(), shape[0], shape[1]))

    def __reduce__(self):  # copies and pickles take the addresses of their own tensors
        return Fp4Matrix, (self.codes, self.scales, self.shape)

    def __init__(self, codes, scales, shape: Tuple[int, int]):
        import torch
        rows, cols = int(shape[0]), int(shape[1])
        c, e = _fp4_layout(rows, cols)
        _check_part("codes", codes, torch.float4_e2m1fn_x2, c)
        _check_part("scales", scales, torch.float8_e8m0fnu, e)
        if codes.device != scales.device or codes.device.type != "cuda":
            raise ValueError("codes and scales must be on one ROCm GPU")
        self._set(codes, scales, (rows, cols))

    @classmethod
    def empty(cls, rows: int, cols: int, device=None) -> "Fp4Matrix":
        """Storage with undefined contents."""
        import torch
        c, s = _fp4_layout(rows, cols)
        dev = device if isinstance(device, torch.device) else torch.device("cuda" if device is None else device)
        if dev.type != "cuda":
            raise ValueError("codes and scales must be on one ROCm GPU")
        # made in its layout, so without __init__'s checks
        m = cls.__new__(cls)
        m._set(torch.empty(c, dtype=torch.float4_e2m1fn_x2, device=dev),
               torch.empty(s, dtype=torch.float8_e8m0fnu, device=dev), (rows, cols))
        return m

    def dequantize(self, dtype=None):
        """The values it stands for (muonh_fp4_dequantize), fp32 by default or bf16:
        both hold them exactly."""
        import torch
        dtype = torch.float32 if dtype is None else dtype
        dt = _fp8_dt(torch, dtype)
        d = _held("the matrix", self)
        out = torch.empty(self.shape, dtype=dtype, device=self.device)
        _on_device(torch, self.device, get_lib().muonh_fp4_dequantize, d, out.data_ptr(), dt, max(self.shape[1], 1))
        return out


_NO_FORM4 = Fp4Desc(None, None, 0, 0)


def _form4(name: str, o, wanted: bool, rows: int, cols: int, dev):
    """The output for one form of fp4_quantize: `o` checked, a new one, or None."""
    if not wanted:
        if o is not None:
            raise ValueError(f"{name} given for a form that was not asked for")
        return None
    if o is None:
        return Fp4Matrix.empty(rows, cols, dev)
    if not isinstance(o, Fp4Matrix):
        raise TypeError(f"{name} must be an Fp4Matrix")
    if o.shape != (rows, cols) or o.device != dev:
        raise ValueError(f"{name} must be a {(rows, cols)} Fp4Matrix on {dev}")
    _held(name, o)
    return o


def fp4_quantize(x, forms: str = "plain", out: Optional[Fp4Matrix] = None, out_t: Optional[Fp4Matrix] = None):
    """Quantize x (a 2-d fp32 or bf16 tensor on the GPU whose rows are
    contiguous, any row stride) to microscaled 4-bit floats (muonh_fp4_quantize).

    forms: "plain" (x itself, grouped along its columns), "transposed" (its
    transpose, grouped along x's rows) or "both", in one pass. Returns (q, q_t), None in the
    place of a form that was not asked for; out / out_t: matrices to write into.
    Runs on the current stream of x's device, outside autograd, as fp8_quantize.
    """
    import torch
    dt, ld = _rows("x", x, getattr(x, "device", None))
    dev = x.device
    if forms not in FP8_FORMS:
        raise ValueError(f"forms must be one of {FP8_FORMS}, got {forms!r}")
    rows, cols = x.shape
    q = _form4("out", out, forms != "transposed", rows, cols, dev)
    qt = _form4("out_t", out_t, forms != "plain", cols, rows, dev)
    d, t = _NO_FORM4 if q is None else q.desc, _NO_FORM4 if qt is None else qt.desc
    _on_device(torch, dev, get_lib().muonh_fp4_quantize, x.data_ptr(), dt, rows, cols, ld, d.codes, d.scales, t.codes,
               t.scales)
    for o in (out, out_t):
        if o is not None:
            _written(o.codes, o.scales)
    return q, qt


def fp4_matmul(a: Fp4Matrix, b: Fp4Matrix, out=None, out_dtype=None, accumulate: bool = False):
    """out[i][j] = sum_k a[i][k] * b[j][k] (muonh_fp4_matmul), plus out's old
    values with accumulate=True.

    out: a 2-d fp32 or bf16 tensor (a rows x b rows) whose rows are contiguous;
    otherwise a new one of out_dtype (default bfloat16). Products and the sums of a group of 32
    are exact, other sums fp32. The products of a linear layer as for fp8_matmul; here
    a weight's transposed form is a quantization of its own (forms="both"), since groups
    lie along k. Runs on the current stream of the operands' device, outside autograd.
    """
    import torch
    for name, m in (("a", a), ("b", b)):
        if not isinstance(m, Fp4Matrix):
            raise TypeError(f"{name} must be an Fp4Matrix")
    da, db = _held("a", a), _held("b", b)
    dev = a.device
    if dev != b.device:
        raise ValueError(f"a is on {dev}, b on {b.device}")
    if a.shape[1] != b.shape[1]:
        raise ValueError(f"a has {a.shape[1]} columns, b {b.shape[1]}")
    m, n = shape = (a.shape[0], b.shape[0])
    given = out is not None
    if not given:
        if accumulate:
            raise ValueError("accumulate=True needs out")
        out_dtype = torch.bfloat16 if out_dtype is None else out_dtype
        dt, ld = _fp8_dt(torch, out_dtype), max(n, 1)
        out = torch.empty(shape, device=dev, dtype=out_dtype)
    else:
        dt, ld = _rows("out", out, dev, shape, out_dtype)
    lib = get_lib()
    nbytes = lib.muonh_fp4_matmul_workspace_bytes(m, n, a.shape[1])
    # from torch's allocator on the current stream, as fp8_matmul's
    ws = torch.empty(nbytes, dtype=torch.uint8, device=dev) if nbytes else None
    _on_device(torch, dev, lib.muonh_fp4_matmul, da, db, out.data_ptr(), dt, ld, 1 if accumulate else 0,
               None if ws is None else ws.data_ptr(), nbytes)
    if given:
        _written(out)
    return out


# -- RMS norm ------------------------------------------------------------------
@functools.lru_cache(maxsize=None)
def _dt_codes():
    import torch
    return {torch.float32: MUONH_DT_FP32, torch.bfloat16: MUONH_DT_BF16}


def _rows(name: str, t, dev, shape=None, dtype=None):
    """(dtype code, row pitch) of a 2-d fp32 or bf16 tensor whose rows are
    contiguous."""
    try:
        dt, (rows, cols), (ld, step) = _dt_codes()[t.dtype], t.shape, t.stride()
    except (AttributeError, KeyError, TypeError, ValueError):
        _refuse_rows(name, t)
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != dev or dev.type != "cuda":
        raise ValueError(f"{name} must be a 2-d tensor on {dev if dev.type == 'cuda' else 'a ROCm GPU'}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if step == 1 and ld >= cols and rows > 1:
        return dt, ld
    return dt, _row_pitch(t, name)


def _refuse_rows(name: str, t) -> None:
    """Says why t is no 2-d fp32 or bf16 tensor."""
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    _fp8_dt(torch, t.dtype)
    raise ValueError(f"{name} must be a 2-d tensor")


def _floats(name: str, t, dev, n: int) -> None:
    """A contiguous fp32 vector of n entries."""
    import torch
    if not isinstance(t, torch.Tensor) or t.dtype != torch.float32:
        raise TypeError(f"{name} must be a float32 torch tensor")
    if t.shape != (n,) or not t.is_contiguous() or t.device != dev:
        raise ValueError(f"{name} must be a contiguous vector of {n} entries on {dev}")


def _norm_inputs(x, weight, residual, residual_out):
    """Checks what both forms of the norm take: (x's dtype code and pitch, h's
    dtype code, residual's pitch, h or None, its pitch, rstd)."""
    import torch
    dt, ld = _rows("x", x, getattr(x, "device", None))
    dev, shape = x.device, x.shape
    _floats("weight", weight, dev, shape[1])
    rstd = torch.empty(shape[0], dtype=torch.float32, device=dev)
    if residual is None:
        if residual_out is not None:
            raise ValueError("residual_out without residual")
        return dt, ld, dt, 0, None, 0, rstd
    hdt, rld = _rows("residual", residual, dev, shape)
    if residual_out is None:
        h = torch.empty(shape, dtype=residual.dtype, device=dev)
        return dt, ld, hdt, rld, h, max(shape[1], 1), rstd
    _, hld = _rows("residual_out", residual_out, dev, shape, residual.dtype)
    return dt, ld, hdt, rld, residual_out, hld, rstd


def rms_norm(x, weight, residual=None, eps: float = 1e-6, out=None, out_dtype=None, residual_out=None):
    """h = x + residual; y = h / sqrt(mean(h^2) + eps) * weight along each row
    (muonh_rms_norm). Returns (y, h, rstd): h is x itself without a residual,
    rstd (rows, fp32) and h are what rms_norm_backward takes.

    x, residual: 2-d fp32 or bf16 tensors whose rows are contiguous, any row
    stride, each of its own type (heads that lie in wider rows of tokens have no one
    stride: copy them out first); h has the residual's, and y is the norm of h as
    stored. weight: fp32 vector. residual_out: a tensor for h, which may be
    `residual` or `x` itself. out: a tensor for y; otherwise a new one of out_dtype
    (default: h's type). Runs on the current stream of x's device, outside
    autograd: rms_norm_backward is the gradient.
    """
    import torch
    dt, ld, hdt, rld, h, hld, rstd = _norm_inputs(x, weight, residual, residual_out)
    dev, shape = x.device, tuple(x.shape)
    if out is None:
        ydt = hdt if out_dtype is None else _fp8_dt(torch, out_dtype)
        y = torch.empty(shape, dtype=(x if h is None else h).dtype if out_dtype is None else out_dtype, device=dev)
        yld = shape[1]
    else:
        y = out
        ydt, yld = _rows("out", y, dev, shape, out_dtype)
    _on_device(torch, dev, get_lib().muonh_rms_norm, x.data_ptr(), dt, shape[0], shape[1], ld,
               None if h is None else residual.data_ptr(), hdt, rld, None if h is None else h.data_ptr(), hld,
               weight.data_ptr(), float(eps), rstd.data_ptr(), y.data_ptr(), ydt, yld, None, None, None, None)
    for o in (out, residual_out):
        if o is not None:
            _written(o)
    return y, x if h is None else h, rstd


def rms_norm_fp8(x, weight, residual=None, eps: float = 1e-6, forms: str = "plain",
                 out: Optional[Fp8Matrix] = None, out_t: Optional[Fp8Matrix] = None, residual_out=None):
    """rms_norm with y quantized to block-scaled e4m3 as fp8_quantize(...,
    block="rows") does, from its unrounded values. Returns (q, q_t, h, rstd);
    forms, out and out_t as for fp8_quantize, the rest as for rms_norm."""
    import torch
    if forms not in FP8_FORMS:
        raise ValueError(f"forms must be one of {FP8_FORMS}, got {forms!r}")
    dt, ld, hdt, rld, h, hld, rstd = _norm_inputs(x, weight, residual, residual_out)
    dev = x.device
    rows, cols = x.shape
    q = _form("out", out, forms != "transposed", rows, cols, "rows", dev)
    qt = _form("out_t", out_t, forms != "plain", cols, rows, "rows", dev)
    d, t = _NO_FORM if q is None else q.desc, _NO_FORM if qt is None else qt.desc
    _on_device(torch, dev, get_lib().muonh_rms_norm, x.data_ptr(), dt, rows, cols, ld,
               None if h is None else residual.data_ptr(), hdt, rld, None if h is None else h.data_ptr(), hld,
               weight.data_ptr(), float(eps), rstd.data_ptr(), None, 0, 0, d.codes, d.scales, t.codes, t.scales)
    for o in (out, out_t):
        if o is not None:
            _written(o.codes, o.scales)
    if residual_out is not None:
        _written(residual_out)
    return q, qt, x if h is None else h, rstd


def rms_norm_backward(dy, h, weight, rstd, dresidual=None, out=None, dweight=None, accumulate: bool = False):
    """The gradient of rms_norm (muonh_rms_norm_backward): (dh, dweight). dh, of
    h's type, is the gradient of x and of residual alike; dresidual, the gradient that
    reaches h past the norm, is added to it.

    dy: gradient of y, fp32 or bf16; h, rstd: from the forward call; dresidual: of
    h's type. out: a tensor for dh, which may be `dresidual` or `dy` itself. dweight: an fp32
    vector to write into (new otherwise), with accumulate=True to add to.
    Deterministic. Runs on the current stream of h's device.
    """
    import torch
    hdt, hld = _rows("h", h, getattr(h, "device", None))
    dev = h.device
    rows, cols = shape = tuple(h.shape)
    ddt, dld = _rows("dy", dy, dev, shape)
    _floats("weight", weight, dev, cols)
    _floats("rstd", rstd, dev, rows)
    rld = 0
    if dresidual is not None:
        _, rld = _rows("dresidual", dresidual, dev, shape, h.dtype)
    if out is None:
        dh, old = torch.empty(shape, dtype=h.dtype, device=dev), max(cols, 1)
    else:
        dh = out
        _, old = _rows("out", dh, dev, shape, h.dtype)
    if dweight is None:
        if accumulate:
            raise ValueError("accumulate=True needs dweight")
        dw = torch.empty(cols, dtype=torch.float32, device=dev)
    else:
        _floats("dweight", dweight, dev, cols)
        dw = dweight
    lib = get_lib()
    nbytes = lib.muonh_rms_norm_backward_workspace_bytes(rows, cols)
    # from torch's allocator on the current stream, as fp8_matmul's
    ws = torch.empty(nbytes, dtype=torch.uint8, device=dev) if nbytes else None
    _on_device(torch, dev, lib.muonh_rms_norm_backward, dy.data_ptr(), ddt, dld, h.data_ptr(), hdt, rows, cols, hld,
               weight.data_ptr(), rstd.data_ptr(), None if dresidual is None else dresidual.data_ptr(), rld,
               dh.data_ptr(), old, dw.data_ptr(), 1 if accumulate else 0, None if ws is None else ws.data_ptr(), nbytes)
    for o in (out, dweight):
        if o is not None:
            _written(o)
    return dh, dw


# -- embedding -------------------------------------------------------------------
def _ids(ids, dev, first) -> int:
    """Bytes per id of a contiguous int32 or int64 tensor; first: a whole number that an id can be."""
    import torch
    if not isinstance(ids, torch.Tensor) or ids.dtype not in (torch.int32, torch.int64):
        raise TypeError("ids must be an int32 or int64 torch tensor")
    if ids.device != dev or not ids.is_contiguous():
        raise ValueError(f"ids must be contiguous and on {dev}")
    # ctypes would take it modulo 2^64; the call refuses what is below zero
    if not -(1 << 63) <= first < 1 << 63 or first != int(first):
        raise ValueError(f"first must be a whole number of 64 bits, got {first}")
    return ids.element_size()


def _by_token(name: str, t, ids, cols: int):
    """A tensor of shape ids.shape + (cols,) as one row per token."""
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.shape != (*ids.shape, cols):
        raise ValueError(f"{name} must have shape {(*ids.shape, cols)}, got {tuple(t.shape)}")
    if t.dim() == 2:
        return t
    try:
        return t.view(ids.numel(), cols)
    except RuntimeError:
        raise ValueError(f"{name}'s tokens must lie at one distance from each other") from None


def embedding(ids, table, scale: float = 1.0, out=None, out_dtype=None, first: int = 0):
    """out[...] = scale * table[ids[...] - first] (muonh_embedding); an id that is
    no row of the table (padding, or a row of another part of it) gives zeros. first >= 0: the
    id of the table's first row.

    ids: a contiguous int32 or int64 tensor of any shape; table: a 2-d fp32 or
    bf16 tensor whose rows are contiguous; out: a tensor of shape ids.shape +
    (columns,), otherwise a new one of out_dtype (default: the table's type). Runs on the
    current stream of the table's device, outside autograd: embedding_backward is
    the gradient.
    """
    import torch
    dt, ld = _rows("table", table, getattr(table, "device", None))
    dev = table.device
    nbytes = _ids(ids, dev, first)
    rows, cols = table.shape
    if out is None:
        odt = dt if out_dtype is None else _fp8_dt(torch, out_dtype)
        y = flat = torch.empty((*ids.shape, cols), dtype=table.dtype if out_dtype is None else out_dtype, device=dev)
        old = max(cols, 1)
    else:
        y, flat = out, _by_token("out", out, ids, cols)
        odt, old = _rows("out", flat, dev, None, out_dtype)
    _on_device(torch, dev, get_lib().muonh_embedding, ids.data_ptr(), nbytes, ids.numel(), int(first), table.data_ptr(),
               dt, rows, cols, ld, float(scale), flat.data_ptr(), odt, old)
    if out is not None:
        _written(out)
    return y


def embedding_backward(ids, dy, out, scale: float = 1.0, accumulate: bool = False, first: int = 0):
    """out[v] = scale * (sum of dy over the tokens with ids - first = v), zeros
    where there is none, or added to out's old values with accumulate=True
    (muonh_embedding_backward). Returns out.

    ids: as for embedding; dy: fp32 or bf16, shape ids.shape + (columns,); out: the
    table's gradient, 2-d fp32 with contiguous rows (AdamW.step reads it). Deterministic. Runs on the
    current stream of out's device.
    """
    import torch
    _, ld = _rows("out", out, getattr(out, "device", None), None, torch.float32)
    dev = out.device
    nbytes = _ids(ids, dev, first)
    rows, cols = out.shape
    flat = _by_token("dy", dy, ids, cols)
    ddt, dld = _rows("dy", flat, dev)
    lib = get_lib()
    n = ids.numel()
    size = lib.muonh_embedding_backward_workspace_bytes(n, cols)
    # from torch's allocator on the current stream, as fp8_matmul's
    ws = torch.empty(size, dtype=torch.uint8, device=dev) if size else None
    _on_device(torch, dev, lib.muonh_embedding_backward, ids.data_ptr(), nbytes, n, int(first), flat.data_ptr(), ddt, dld,
               float(scale), out.data_ptr(), rows, cols, ld, 1 if accumulate else 0, None if ws is None else ws.data_ptr(),
               size)
    _written(out)
    return out
