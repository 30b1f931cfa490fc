"""Python binding of the B200 e-means library (libemeans.so, C ABI in include/emeans.h).

Argument marshalling only: every step of the method runs in the library's CUDA
kernels. Functions keep the ABI's names; `Model` wraps a handle for convenience
and takes torch tensors (or raw pointers) for X and the outputs.

Importing fails loudly if libemeans.so has not been built (python
mini_ema_means_b200/build.py); there is no fallback path.
"""

from __future__ import annotations

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libemeans.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: build it with `python mini_ema_means_b200/build.py`")

lib = ctypes.CDLL(LIB_PATH)

# ---- status codes and options (mirrors include/emeans.h) ----
EM_OK = 0
EM_E_INVAL = -1
EM_E_NOMEM = -2
EM_E_CUDA = -3
EM_E_BOUNDS = -4
EM_E_TIMEOUT = -5
EM_E_NONFINITE = -6
EM_E_STATE = -7
EM_E_NODEVICE = -8
EM_E_COMM = -9

EM_OPT_BATCH_SIZE = 1
EM_OPT_ALPHA0 = 2
EM_OPT_UNUSED_THRESHOLD = 3
EM_OPT_REVIVAL = 4
EM_OPT_FINALIZE = 5
EM_OPT_LAW = 6
EM_OPT_INPUT_DTYPE = 7
EM_OPT_CHECK_FINITE = 8
EM_OPT_WAIT_LIMIT_MS = 9
EM_OPT_AUTO_REVIVE = 10
EM_OPT_CAPTURE_LABELS = 11
EM_OPT_GRAPHS = 12
EM_OPT_ASSIGN_KERNEL = 13
EM_OPT_PROFILE = 14
EM_OPT_EXACT_TIES = 15
EM_OPT_SPHERICAL = 16
EM_OPT_PREFETCH = 17
EM_OPT_SEARCH_FORMAT = 18
EM_OPT_PDL = 19

EM_DTYPE_F32 = 0
EM_DTYPE_BF16 = 1
EM_DTYPE_F16 = 2
EM_DTYPE_BLOCK8 = 3

EM_PHASE_PREPARE = 0
EM_PHASE_GATHER = 1
EM_PHASE_ASSIGN = 2
EM_PHASE_UPDATE = 3
EM_PHASE_REVIVE = 4
EM_PHASE_FINALIZE = 5
EM_NPHASES = 6
PHASE_NAMES = ("prepare", "gather", "assign", "update", "revive", "finalize")

EM_NOALLOC_MAX_ROWS = 524288
EM_NOALLOC_MAX_K = 65536
EM_NOALLOC_MAX_KD = 4194304

EM_REVIVE_NONE = 0
EM_REVIVE_SPLIT = 1
EM_REVIVE_RESAMPLE = 2

REVIVAL_MODES = {"none": EM_REVIVE_NONE, "split": EM_REVIVE_SPLIT, "resample": EM_REVIVE_RESAMPLE}


class em_recipe_t(ctypes.Structure):
    _fields_ = [
        ("n", ctypes.c_int64), ("k", ctypes.c_int64), ("d", ctypes.c_int64),
        ("epochs", ctypes.c_double), ("batch_raw", ctypes.c_double),
        ("batch_size", ctypes.c_int64), ("alpha0", ctypes.c_double),
        ("passes", ctypes.c_int64), ("rows_last_pass", ctypes.c_int64),
        ("steps_full_pass", ctypes.c_int64), ("steps_last_pass", ctypes.c_int64),
        ("total_steps", ctypes.c_int64),
    ]

    def as_dict(self):
        return {name: getattr(self, name) for name, _ in self._fields_}


class em_stats_t(ctypes.Structure):
    _fields_ = [
        ("steps_done", ctypes.c_int64), ("passes_done", ctypes.c_int64),
        ("rows_assigned", ctypes.c_int64), ("n_splits", ctypes.c_int64),
        ("last_dead", ctypes.c_int64), ("imbalance", ctypes.c_double),
        ("last_alpha", ctypes.c_double),
    ]

    def as_dict(self):
        return {name: getattr(self, name) for name, _ in self._fields_}


class em_profile_t(ctypes.Structure):
    _fields_ = [
        ("ms", ctypes.c_double * EM_NPHASES), ("spans", ctypes.c_int64 * EM_NPHASES),
        ("launches", ctypes.c_int64), ("assign_flops", ctypes.c_double),
        ("update_bytes", ctypes.c_double), ("gather_bytes", ctypes.c_double),
    ]

    def as_dict(self):
        return {
            "ms": dict(zip(PHASE_NAMES, list(self.ms))),
            "spans": dict(zip(PHASE_NAMES, list(self.spans))),
            "launches": self.launches, "assign_flops": self.assign_flops,
            "update_bytes": self.update_bytes, "gather_bytes": self.gather_bytes,
        }


class em_block8_t(ctypes.Structure):
    _fields_ = [
        ("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("claims", ctypes.c_void_p),
        ("status", ctypes.c_void_p), ("rows", ctypes.c_int64), ("d", ctypes.c_int64),
    ]


_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_B8 = ctypes.POINTER(em_block8_t)
_SIGS = {
    "em_last_error": (ctypes.c_char_p, []),
    "em_device_count": (ctypes.c_int, []),
    "em_last_error_code": (ctypes.c_int, []),
    "em_fail_allocation": (_I64, [_I64]),
    "em_compute_recipe": (ctypes.c_int, [_I64, _I64, ctypes.c_double, ctypes.c_int, _I64, ctypes.c_double,
                                         ctypes.POINTER(em_recipe_t)]),
    "em_permutation": (ctypes.c_int, [_I64, ctypes.c_uint64, ctypes.c_int, _I64, _P, _I64, _P]),
    "em_dp_schedule": (ctypes.c_int, [_I64, _I64, ctypes.c_double, ctypes.c_int, _I64, ctypes.c_double, _I64, _I64,
                                      _I64, _P, _P, _P, _P]),
    "em_search_schedule": (ctypes.c_int, [_I64, _I64, ctypes.c_int, ctypes.POINTER(ctypes.c_int),
                                          ctypes.POINTER(ctypes.c_int)]),
    "em_create": (_P, [_I64, _I64, ctypes.c_uint64]),
    "em_destroy": (None, [_P]),
    "em_set_option": (ctypes.c_int, [_P, ctypes.c_int, ctypes.c_double]),
    "em_get_option": (ctypes.c_int, [_P, ctypes.c_int, ctypes.POINTER(ctypes.c_double)]),
    "em_set_stream": (ctypes.c_int, [_P, _P]),
    "em_train": (ctypes.c_int, [_P, _P, _I64, ctypes.c_double]),
    "em_begin": (ctypes.c_int, [_P, _P, _I64, ctypes.c_double]),
    "em_step": (ctypes.c_int, [_P, _I64, ctypes.POINTER(_I64)]),
    "em_finalize": (ctypes.c_int, [_P]),
    "em_revive": (ctypes.c_int, [_P]),
    "em_lloyd": (ctypes.c_int, [_P, _P, _I64, _I64]),
    "em_assign": (ctypes.c_int, [_P, _P, _I64, _P, _P]),
    "em_mse": (ctypes.c_int, [_P, _P, _I64, ctypes.POINTER(ctypes.c_double)]),
    "em_centroids": (ctypes.c_int, [_P, _P]),
    "em_labels": (ctypes.c_int, [_P, _P]),
    "em_recipe": (ctypes.c_int, [_P, ctypes.POINTER(em_recipe_t)]),
    "em_stats": (ctypes.c_int, [_P, ctypes.POINTER(em_stats_t)]),
    "em_obj": (ctypes.c_int, [_P, _P, _I64, ctypes.POINTER(_I64)]),
    "em_get_state": (ctypes.c_int, [_P, _P, _P, _P, ctypes.POINTER(_I64)]),
    "em_set_state": (ctypes.c_int, [_P, _P, _P, _P, _I64]),
    "em_last_batch": (ctypes.c_int, [_P, _P, _P, _P, ctypes.POINTER(_I64)]),
    "em_profile": (ctypes.c_int, [_P, ctypes.POINTER(em_profile_t), ctypes.c_int]),
    "em_assign_noalloc": (ctypes.c_int, [_P, _I64, _I64, _P, _I64, _P, _P, _P]),
    "em_sync": (ctypes.c_int, [_P]),
    "em_selftest": (ctypes.c_int, [_P, ctypes.c_int, ctypes.c_double]),
    "em_fp8_converter": (ctypes.c_int, [_P, _P, ctypes.POINTER(ctypes.c_float)]),
    "em_block8_layout": (ctypes.c_int, [_I64, _I64] + [ctypes.POINTER(_I64)] * 3),
    "em_block8_write": (ctypes.c_int, [_B8, _P, ctypes.c_int, _I64, _I64, _I64, _I64, _P, _P]),
    "em_block8_read": (ctypes.c_int, [_B8, _I64, _P, _I64, _P, ctypes.c_int, _I64, _P]),
    "em_block8_matmul": (ctypes.c_int, [_B8, _I64, _B8, _I64, _P, ctypes.c_int, _I64, _P]),
    "em_block8_check": (ctypes.c_int, [_B8, _P]),
    "em_dp_unique_id": (ctypes.c_int, [_P]),
    "em_dp_init": (ctypes.c_int, [_P, ctypes.c_int, ctypes.c_int, _P]),
    "em_dp_world": (ctypes.c_int, [_P, ctypes.POINTER(ctypes.c_int), ctypes.POINTER(ctypes.c_int)]),
}

EM_NCCL_ID_BYTES = 128


def dp_unique_id() -> bytes:
    """A fresh communicator id for em_dp_init (rank 0 makes it, the others receive it)."""
    buf = ctypes.create_string_buffer(EM_NCCL_ID_BYTES)
    check(em_dp_unique_id(ctypes.cast(buf, ctypes.c_void_p)), "em_dp_unique_id")
    return buf.raw

for _name, (_res, _args) in _SIGS.items():
    _fn = getattr(lib, _name)
    _fn.restype = _res
    _fn.argtypes = _args
    globals()[_name] = _fn

ABI_FUNCTIONS = tuple(_SIGS)


class EmeansError(RuntimeError):
    def __init__(self, code: int, where: str):
        msg = em_last_error().decode(errors="replace")
        super().__init__(f"{where} failed with status {code}: {msg}")
        self.code = code


def check(rc: int, where: str = "call") -> None:
    if rc != EM_OK:
        raise EmeansError(rc, where)


def _ptr(x):
    """Address of a tensor / ndarray / raw int (0 for None); of a Block8's C struct."""
    if x is None:
        return None
    if isinstance(x, Block8):
        return ctypes.addressof(x.view)
    if isinstance(x, int):
        return x
    if hasattr(x, "data_ptr"):
        return x.data_ptr()
    if hasattr(x, "ctypes"):
        return x.ctypes.data
    raise TypeError(f"cannot take the address of {type(x)}")


def compute_recipe(n, k, epochs, law=0, batch_size=0, alpha0=0.0) -> dict:
    r = em_recipe_t()
    check(em_compute_recipe(n, k, float(epochs), int(law), int(batch_size), float(alpha0), ctypes.byref(r)),
          "em_compute_recipe")
    return r.as_dict()


def search_schedule(rows, k, sms):
    """(split, m_full) of the nearest-centroid search for `rows` rows and k
    centroids on `sms` SMs (host code)."""
    split, m_full = ctypes.c_int(), ctypes.c_int()
    check(em_search_schedule(int(rows), int(k), int(sms), ctypes.byref(split), ctypes.byref(m_full)),
          "em_search_schedule")
    return split.value, m_full.value


def permutation(n, seed, stream, which, idx):
    """pi(idx) of the library's keyed bijection (host code; idx: int64 ndarray)."""
    import numpy as np

    idx = np.ascontiguousarray(idx, dtype=np.int64)
    out = np.empty_like(idx)
    check(em_permutation(n, seed, stream, which, idx.ctypes.data, len(idx), out.ctypes.data), "em_permutation")
    return out


def fail_allocation(nth: int) -> int:
    """Makes the library's nth device allocation from now on fail as a failed
    cudaMalloc does (nth <= 0: off); returns the allocations attempted since the
    previous call (host code)."""
    return int(em_fail_allocation(int(nth)))


def dp_schedule(n_local, k, epochs, world, rank, count, law=0, batch_size=0, alpha0=0.0):
    """The rows rank `rank` of `world` takes at each of the first `count` steps of a
    data-parallel run (host code): arrays pass, first, rows, key (int64)."""
    import numpy as np

    out = [np.empty(count, dtype=np.int64) for _ in range(4)]
    check(em_dp_schedule(n_local, k, epochs, law, batch_size, alpha0, world, rank, count,
                         *(o.ctypes.data for o in out)), "em_dp_schedule")
    return tuple(out)


def block8_layout(rows, d):
    """(pitch, code bytes, scale bytes) of a rows x d block8 matrix (host code)."""
    out = [_I64() for _ in range(3)]
    check(em_block8_layout(int(rows), int(d), *(ctypes.byref(o) for o in out)), "em_block8_layout")
    return tuple(o.value for o in out)


class Block8:
    """A rows x d matrix held as E4M3 codes with a power-of-two scale per block of 128
    values of a row (em_block8_t in include/emeans.h says what is held and where).

    The memory is torch tensors: `codes` (rows x pitch, uint8), `scales` (uint8, in the
    order of the header), `claims` and `status` (scratch). `codes` and `scales` may be
    given, filled or not; otherwise they are made, on the current stream, and stand for
    zeros. The calls run on `stream` (a torch.cuda.Stream; by default the current stream
    of the matrix's device; one given by its handle alone is not recorded with the
    memory it uses) and do not wait for it. They are no part of autograd: write takes
    the values of X as if detached, and what the calls write counts as modified in place
    (`out`, `codes`, `scales`), so that a backward pass which saved it refuses. An `out`
    that requires gradients is refused, but under torch.no_grad(). A Block8 is also an X
    for Model.train, begin, lloyd, assign and mse, which wait for the current stream of its
    device first and read it into a bf16 copy, which train, begin and lloyd leave with the
    model and assign and mse free at their end."""

    def __init__(self, rows, d, device=None, codes=None, scales=None):
        import torch

        pitch, code_bytes, scale_bytes = block8_layout(rows, d)
        given = codes if codes is not None else scales
        if device is None:
            device = given.device if given is not None else torch.device("cuda", torch.cuda.current_device())
        self.device = torch.device(device)
        if self.device.type == "cuda" and self.device.index is None:
            self.device = torch.device("cuda", torch.cuda.current_device())
        self.rows, self.d, self.pitch = int(rows), int(d), pitch
        for name, t, n in (("codes", codes, code_bytes), ("scales", scales, scale_bytes)):
            if t is not None and (t.dtype != torch.uint8 or t.numel() != n or not t.is_contiguous()
                                  or t.device != self.device):
                raise ValueError(f"{name} must be {n} contiguous uint8 values on {self.device}")
        self.codes = (torch.zeros(self.rows, pitch, dtype=torch.uint8, device=self.device) if codes is None
                      else codes.view(self.rows, pitch))
        self.scales = (torch.full((scale_bytes,), 127, dtype=torch.uint8, device=self.device) if scales is None
                       else scales.view(-1))
        self.claims = torch.empty(self.rows, dtype=torch.int32, device=self.device)
        self.status = torch.zeros(1, dtype=torch.int32, device=self.device)
        self.view = em_block8_t(self.codes.data_ptr(), self.scales.data_ptr(), self.claims.data_ptr(),
                                self.status.data_ptr(), self.rows, self.d)
        self._ref = ctypes.byref(self.view)
        self._index = -1 if self.device.index is None else self.device.index
        self._types = {torch.float32: EM_DTYPE_F32, torch.bfloat16: EM_DTYPE_BF16, torch.float16: EM_DTYPE_F16}
        self._int64 = torch.int64
        self._held = (self.codes, self.scales)
        # marks tensors as modified in place (the public function wraps this one, for 0.1 us)
        self._modified = getattr(torch._C, "_increment_version", None) or torch.autograd.graph.increment_version
        self._grad_mode = torch.is_grad_enabled
        # the current stream's handle alone (torch.cuda.current_stream makes an object of
        # it, 2 us of a call of 7)
        self._current = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
            lambda index: torch.cuda.current_stream(index).cuda_stream)

    @property
    def shape(self):
        return (self.rows, self.d)

    def _stream(self, stream, *used):
        """The handle to launch on. A given torch stream is recorded with the memory used,
        so that the caching allocator keeps it until that stream is done."""
        if stream is None:
            return self._current(self._index)
        if isinstance(stream, int):
            return stream
        for t in (self.codes, self.scales, self.claims, self.status, *used):
            if t is not None:
                t.record_stream(stream)
        return stream.cuda_stream

    def _here(self, t, name):
        if t.get_device() != self._index or (self._index < 0 and t.device != self.device):
            raise ValueError(f"{name} is on {t.device}, the matrix on {self.device}")

    def _matrix(self, t, cols, name):
        """Rows, type code and element strides of a 2-D tensor of `cols` columns on this device."""
        dtype = self._types.get(t.dtype)
        if dtype is None:
            raise TypeError(f"{name} must be float32, bfloat16 or float16, not {t.dtype}")
        shape = t.shape
        if len(shape) != 2 or shape[1] != cols:
            raise ValueError(f"{name} must be 2-D with {cols} columns, not {tuple(shape)}")
        if t.get_device() != self._index or self._index < 0:
            self._here(t, name)
        rs, cs = t.stride()
        # a dimension of one element has no stride of its own
        if cols == 1:
            cs = 1
        if shape[0] == 1 and cs != 1:
            rs = 1
        return shape[0], dtype, rs, cs

    def _slots(self, slots, n, first):
        if slots is None:
            return None
        if slots.dtype != self._int64 or slots.dim() != 1 or not slots.is_contiguous():
            raise ValueError("slots must be a contiguous 1-D int64 tensor")
        if len(slots) != n:
            raise ValueError(f"{len(slots)} slots for {n} rows")
        if slots.get_device() != self._index or self._index < 0:
            self._here(slots, "slots")
        if first:
            raise ValueError("first must be 0 with slots")
        return slots.data_ptr() if n else None

    def write(self, X, first=0, slots=None, stream=None):
        """Quantises X (n x d; row- or column-contiguous) into rows first, first + 1, ...,
        or into rows slots[i] (-1: not written; the last of equal slots stays)."""
        n, dtype, rs, cs = self._matrix(X, self.d, "X")
        rc = em_block8_write(self._ref, X.data_ptr(), dtype, n, rs, cs, first, self._slots(slots, n, first),
                             self._stream(stream, X, slots))
        if rc:
            check(rc, "em_block8_write")
        self._modified(self._held)

    def read(self, out, first=0, slots=None, stream=None):
        """Reads out.shape[0] rows from `first` on, or rows slots[i] (-1: zeros), into out."""
        n, dtype, rs, cs = self._matrix(out, self.d, "out")
        if out.requires_grad and self._grad_mode():
            raise ValueError("out requires gradients, which this call has none of")
        if cs != 1 and n:
            raise ValueError("the rows of out must be contiguous")
        rc = em_block8_read(self._ref, first, self._slots(slots, n, first), n, out.data_ptr(), dtype,
                            rs if n > 1 else self.d, self._stream(stream, out, slots))
        if rc:
            check(rc, "em_block8_read")
        self._modified((out,))
        return out

    def matmul(self, other, out, stream=None):
        """out[i, j] = row i of this matrix . row j of `other`, for out's shape."""
        nb = out.shape[-1]
        na, dtype, rs, cs = self._matrix(out, nb, "out")
        if out.requires_grad and self._grad_mode():
            raise ValueError("out requires gradients, which this call has none of")
        if other.device != self.device:
            raise ValueError(f"the other matrix is on {other.device}, this one on {self.device}")
        if cs != 1 and na and nb:
            raise ValueError("the rows of out must be contiguous")
        rc = em_block8_matmul(self._ref, na, other._ref, nb, out.data_ptr(), dtype, rs if na > 1 else nb,
                              self._stream(stream, out, other.codes, other.scales))
        if rc:
            check(rc, "em_block8_matmul")
        self._modified((out,))
        return out

    def check(self, stream=None):
        """Waits for the stream; raises EmeansError for a device-side error (a slot
        outside the matrix) since the last check."""
        check(em_block8_check(self._ref, self._stream(stream)), "em_block8_check")


def exchange_dp_id(group=None):
    """(world, rank, id): rank 0 of a torch.distributed group makes a communicator id
    and broadcasts it to the group's other ranks."""
    import torch.distributed as dist

    world, rank = dist.get_world_size(group), dist.get_rank(group)
    obj = [dp_unique_id() if rank == 0 else None]
    src = 0 if group is None else dist.get_global_rank(group, 0)
    dist.broadcast_object_list(obj, src=src, group=group)
    return world, rank, obj[0]


class Model:
    """One e-means model (handle owner). X and outputs are torch tensors or pointers; X
    may be a Block8."""

    def __init__(self, d: int, k: int, seed: int = 1234, **options):
        h = em_create(int(d), int(k), int(seed))
        if not h:
            raise EmeansError(em_last_error_code() or EM_E_INVAL, "em_create")
        self.h = h
        self.d, self.k, self.seed = int(d), int(k), int(seed)
        self._raw_dtype = None
        for name, value in options.items():
            self.set_option(name, value)

    _OPTS = {
        "batch_size": EM_OPT_BATCH_SIZE, "alpha0": EM_OPT_ALPHA0, "unused_threshold": EM_OPT_UNUSED_THRESHOLD,
        "revival": EM_OPT_REVIVAL, "finalize": EM_OPT_FINALIZE, "law": EM_OPT_LAW,
        "input_dtype": EM_OPT_INPUT_DTYPE, "check_finite": EM_OPT_CHECK_FINITE,
        "wait_limit_ms": EM_OPT_WAIT_LIMIT_MS, "auto_revive": EM_OPT_AUTO_REVIVE,
        "capture_labels": EM_OPT_CAPTURE_LABELS, "graphs": EM_OPT_GRAPHS, "assign_kernel": EM_OPT_ASSIGN_KERNEL,
        "profile": EM_OPT_PROFILE, "exact_ties": EM_OPT_EXACT_TIES, "spherical": EM_OPT_SPHERICAL,
        "prefetch": EM_OPT_PREFETCH, "search_format": EM_OPT_SEARCH_FORMAT, "pdl": EM_OPT_PDL,
    }

    def set_option(self, name, value):
        if name == "revival" and isinstance(value, str):
            value = REVIVAL_MODES[value]
        if name == "search_format" and isinstance(value, str):
            value = {"bf16": 0, "fp8": 1, "e4m3": 1}[value]
        if name == "law" and isinstance(value, str):
            value = {"throughput": 0, "quality": 1, "auto": 2}[value]
        if name == "input_dtype" and not isinstance(value, (int, float)):
            value = 1 if "bfloat16" in str(value) or str(value) == "bf16" else 3 if str(value) == "block8" else 0
        if name == "input_dtype":
            self._raw_dtype = None
        check(em_set_option(self.h, self._OPTS[name], float(value)), f"em_set_option({name})")

    def get_option(self, name) -> float:
        v = ctypes.c_double()
        check(em_get_option(self.h, self._OPTS[name], ctypes.byref(v)), "em_get_option")
        return v.value

    def _dtype_of(self, X):
        was = int(self.get_option("input_dtype"))
        if isinstance(X, Block8):
            import torch

            raw = was if was != EM_DTYPE_BLOCK8 else self._raw_dtype  # what a raw pointer points to
            self.set_option("input_dtype", EM_DTYPE_BLOCK8)
            self._raw_dtype = raw
            torch.cuda.current_stream(X.device).synchronize()  # (the model reads on a stream of its own)
        elif hasattr(X, "dtype"):
            name = str(X.dtype)
            if "bfloat16" not in name and "float32" not in name:
                raise TypeError(f"X must be float32, bfloat16 or a Block8, not {X.dtype}")
            self.set_option("input_dtype", 1 if "bfloat16" in name else 0)
        elif was == EM_DTYPE_BLOCK8 and self._raw_dtype is not None:
            self.set_option("input_dtype", self._raw_dtype)

    def set_stream(self, stream):
        check(em_set_stream(self.h, stream), "em_set_stream")

    def dp_init(self, group=None):
        """Data-parallel training over the ranks of a torch.distributed group (one
        process per GPU): rank 0 makes the communicator id and the group broadcasts
        it; the library then runs its own NCCL communicator."""
        world, rank, uid = exchange_dp_id(group)
        self.dp_init_id(world, rank, uid)

    def dp_init_id(self, world, rank, uid: bytes):
        """em_dp_init with an id already shared by the caller (every rank calls it)."""
        buf = ctypes.create_string_buffer(bytes(uid), EM_NCCL_ID_BYTES)
        check(em_dp_init(self.h, int(world), int(rank), ctypes.cast(buf, ctypes.c_void_p)), "em_dp_init")

    def fp8_converter(self):
        """(shift, scale) of the fitted FP8 converter: shift as a float32 ndarray of d."""
        import numpy as np

        shift = np.empty(self.d, dtype=np.float32)
        sc = ctypes.c_float()
        check(em_fp8_converter(self.h, shift.ctypes.data, ctypes.byref(sc)), "em_fp8_converter")
        return shift, float(sc.value)

    def selftest(self, which, wait_ms=200.0) -> int:
        """Status of em_selftest (EM_E_TIMEOUT for which=0 and 3, EM_E_BOUNDS for which=1)."""
        return int(em_selftest(self.h, int(which), float(wait_ms)))

    def dp_world(self):
        w, r = ctypes.c_int(), ctypes.c_int()
        check(em_dp_world(self.h, ctypes.byref(w), ctypes.byref(r)), "em_dp_world")
        return w.value, r.value

    def train(self, X, n=None, epochs=5.0):
        self._dtype_of(X)
        check(em_train(self.h, _ptr(X), int(n if n is not None else X.shape[0]), float(epochs)), "em_train")

    def begin(self, X, n=None, epochs=5.0):
        self._dtype_of(X)
        check(em_begin(self.h, _ptr(X), int(n if n is not None else X.shape[0]), float(epochs)), "em_begin")
        return self.recipe()

    def step(self, nsteps=1) -> int:
        done = _I64()
        check(em_step(self.h, int(nsteps), ctypes.byref(done)), "em_step")
        return done.value

    def finalize(self):
        check(em_finalize(self.h), "em_finalize")

    def revive(self):
        check(em_revive(self.h), "em_revive")

    def lloyd(self, X, iters, n=None):
        self._dtype_of(X)
        check(em_lloyd(self.h, _ptr(X), int(n if n is not None else X.shape[0]), int(iters)), "em_lloyd")

    def assign(self, X, labels=None, dists=None, n=None):
        self._dtype_of(X)
        check(em_assign(self.h, _ptr(X), int(n if n is not None else X.shape[0]), _ptr(labels), _ptr(dists)),
              "em_assign")

    def mse(self, X, n=None) -> float:
        self._dtype_of(X)
        out = ctypes.c_double()
        check(em_mse(self.h, _ptr(X), int(n if n is not None else X.shape[0]), ctypes.byref(out)), "em_mse")
        return out.value

    def centroids(self, out):
        check(em_centroids(self.h, _ptr(out)), "em_centroids")
        return out

    def labels(self, out):
        check(em_labels(self.h, _ptr(out)), "em_labels")
        return out

    def recipe(self) -> dict:
        r = em_recipe_t()
        check(em_recipe(self.h, ctypes.byref(r)), "em_recipe")
        return r.as_dict()

    def stats(self) -> dict:
        s = em_stats_t()
        check(em_stats(self.h, ctypes.byref(s)), "em_stats")
        return s.as_dict()

    def obj(self):
        import numpy as np

        cnt = _I64()
        check(em_obj(self.h, None, 0, ctypes.byref(cnt)), "em_obj")
        out = np.zeros(max(cnt.value, 1))
        check(em_obj(self.h, out.ctypes.data, cnt.value, ctypes.byref(cnt)), "em_obj")
        return out[:cnt.value]

    def get_state(self, N=None, S=None, c=None) -> int:
        step = _I64()
        check(em_get_state(self.h, _ptr(N), _ptr(S), _ptr(c), ctypes.byref(step)), "em_get_state")
        return step.value

    def set_state(self, N=None, S=None, c=None, step=0):
        check(em_set_state(self.h, _ptr(N), _ptr(S), _ptr(c), int(step)), "em_set_state")

    def last_batch(self, ids=None, labels=None, dists=None) -> int:
        rows = _I64()
        check(em_last_batch(self.h, _ptr(ids), _ptr(labels), _ptr(dists), ctypes.byref(rows)), "em_last_batch")
        return rows.value

    def profile(self, reset=False) -> dict:
        p = em_profile_t()
        check(em_profile(self.h, ctypes.byref(p), int(reset)), "em_profile")
        return p.as_dict()

    def sync(self):
        check(em_sync(self.h), "em_sync")

    def close(self):
        if getattr(self, "h", None):
            em_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
