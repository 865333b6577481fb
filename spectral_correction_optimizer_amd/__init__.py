"""Spectral-correction AdamW on AMD MI355X: Python binding of libscopt.

Argument marshalling only: every step of the optimizer runs in the HIP
kernels of ``libscopt.so`` (C ABI in ``include/scopt.h``).  PyTorch supplies
device memory and the current HIP stream.  There is no CPU fallback: if the
library has not been built, importing the binding works but constructing an
optimizer raises ``ScoptError``.

The method (papernotes.org notes on "Communication-Efficient LLM Adaptation
over Decentralized GPU Meshes", "Key design 2" and "Key design 3"): per weight
matrix, an anchor-momentum EMA, a thin SVD of it, the Tikhonov response
d_i = s_i / (s_i + tau_p), the two-sided projection and reconstruction
G_filt = U diag(d) (U^T G V) diag(d) V^T, the combination
G_proj = alpha G + (1 - alpha) G_filt, then AdamW.
"""
from __future__ import annotations

import collections
import ctypes
import functools
import os

import torch  # loaded first: libscopt then binds to torch's HIP runtime

__all__ = ["SpectralAdamW", "ScoptError", "library_path", "load_library", "EXPORTED_SYMBOLS",
           "mask_keep_count", "mask_seed", "mask_indices", "mask_pack", "mask_unpack",
           "ActCheckpoint", "RmsNorm", "CrossEntropy", "embed", "embed_grad", "act_pack", "act_unpack",
           "rmsnorm", "rmsnorm_grad", "act_wgrad", "xent"]

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "libscopt.so")
_lib = None

EXPORTED_SYMBOLS = (
    "sc_default_hparams", "sc_opt_create", "sc_opt_destroy", "sc_anchor_update", "sc_refresh",
    "sc_anchor_update_async", "sc_refresh_wait", "sc_refresh_pending", "sc_step", "sc_step_noalloc", "sc_set_lr", "sc_set_tau", "sc_set_state", "sc_get_state", "sc_set_step",
    "sc_get_step", "sc_set_factors", "sc_get_factors", "sc_keep_proj", "sc_get_filtered",
    "sc_set_solve_waves", "sc_set_fused_gram", "sc_set_v_rounds", "sc_set_sweep_stop", "sc_set_quad",
    "sc_get_stats", "sc_get_sweep_counts", "sc_profile", "sc_get_kernel_times", "sc_last_error",
    "sc_mask_keep_count", "sc_mask_seed", "sc_mask_indices", "sc_mask_pack", "sc_mask_unpack",
    "sc_embed", "sc_embed_grad_workspace", "sc_embed_grad", "sc_act_pack", "sc_act_unpack", "sc_rmsnorm",
    "sc_rmsnorm_grad_workspace", "sc_rmsnorm_grad", "sc_act_wgrad_workspace", "sc_act_wgrad",
    "sc_xent_workspace", "sc_xent",
)

SC_F32, SC_BF16 = 0, 1
STATE_KINDS = {"m_anc": 0, "adam_m": 1, "adam_v": 2}


class ScoptError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"libscopt error {code}: {msg}")
        self.code = code


class HParams(ctypes.Structure):
    _fields_ = [("tau_p", ctypes.c_float), ("alpha", ctypes.c_float), ("beta_anc", ctypes.c_float),
                ("lr", ctypes.c_float), ("beta1", ctypes.c_float), ("beta2", ctypes.c_float),
                ("eps", ctypes.c_float), ("weight_decay", ctypes.c_float),
                ("max_sweeps", ctypes.c_int), ("jacobi_tol", ctypes.c_float),
                ("sync_check", ctypes.c_int), ("warm_start", ctypes.c_int),
                ("precondition", ctypes.c_int)]


class KernelTime(ctypes.Structure):
    _fields_ = [("name", ctypes.c_char * 32), ("launches", ctypes.c_int64),
                ("total_ms", ctypes.c_double), ("flops", ctypes.c_double),
                ("bytes", ctypes.c_double)]


class Stats(ctypes.Structure):
    _fields_ = [("n_mats", ctypes.c_int), ("step", ctypes.c_int64), ("refreshes", ctypes.c_int),
                ("sweeps_max", ctypes.c_int), ("not_converged", ctypes.c_int),
                ("nonfinite_grad", ctypes.c_int), ("nonfinite_anchor", ctypes.c_int),
                ("factor_sweeps_max", ctypes.c_int), ("factor_rejected", ctypes.c_int)]


def library_path() -> str:
    return _LIB_PATH


def load_library():
    """Load libscopt.so (raises ScoptError if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise ScoptError(-100, f"{_LIB_PATH} is missing; build it with __graft_entry__.build()")
    lib = ctypes.CDLL(_LIB_PATH)
    vp, i64p = ctypes.c_void_p, ctypes.POINTER(ctypes.c_int64)
    sig = {
        "sc_default_hparams": (None, [ctypes.POINTER(HParams)]),
        "sc_opt_create": (ctypes.c_int, [ctypes.POINTER(vp), ctypes.c_int, i64p, i64p, ctypes.c_int,
                                         ctypes.c_int, ctypes.POINTER(HParams), ctypes.c_int]),
        "sc_opt_destroy": (ctypes.c_int, [vp]),
        "sc_anchor_update": (ctypes.c_int, [vp, ctypes.POINTER(vp), vp]),
        "sc_refresh": (ctypes.c_int, [vp, vp]),
        "sc_anchor_update_async": (ctypes.c_int, [vp, ctypes.POINTER(vp), vp]),
        "sc_refresh_wait": (ctypes.c_int, [vp, vp]),
        "sc_refresh_pending": (ctypes.c_int, [vp, ctypes.POINTER(ctypes.c_int)]),
        "sc_step": (ctypes.c_int, [vp, ctypes.POINTER(vp), ctypes.POINTER(vp), vp]),
        "sc_step_noalloc": (ctypes.c_int, [vp, ctypes.POINTER(vp), ctypes.POINTER(vp), vp]),
        "sc_set_lr": (ctypes.c_int, [vp, ctypes.c_float]),
        "sc_set_tau": (ctypes.c_int, [vp, ctypes.c_float]),
        "sc_set_state": (ctypes.c_int, [vp, ctypes.c_int, ctypes.c_int, vp, vp]),
        "sc_get_state": (ctypes.c_int, [vp, ctypes.c_int, ctypes.c_int, vp, vp]),
        "sc_set_step": (ctypes.c_int, [vp, ctypes.c_int64]),
        "sc_get_step": (ctypes.c_int, [vp, i64p]),
        "sc_set_factors": (ctypes.c_int, [vp, ctypes.c_int, vp, vp, vp, vp]),
        "sc_get_factors": (ctypes.c_int, [vp, ctypes.c_int, vp, vp, vp, vp]),
        "sc_keep_proj": (ctypes.c_int, [vp, ctypes.c_int]),
        "sc_set_solve_waves": (ctypes.c_int, [vp, ctypes.c_int, ctypes.c_int]),
        "sc_set_fused_gram": (ctypes.c_int, [vp, ctypes.c_int]),
        "sc_set_v_rounds": (ctypes.c_int, [vp, ctypes.c_int]),
        "sc_set_sweep_stop": (ctypes.c_int, [vp, ctypes.c_float]),
        "sc_set_quad": (ctypes.c_int, [vp, ctypes.c_int]),
        "sc_get_filtered": (ctypes.c_int, [vp, ctypes.c_int, vp, vp, vp]),
        "sc_get_stats": (ctypes.c_int, [vp, ctypes.POINTER(Stats), ctypes.POINTER(ctypes.c_int)]),
        "sc_get_sweep_counts": (ctypes.c_int, [vp, ctypes.POINTER(ctypes.c_int),
                                               ctypes.POINTER(ctypes.c_int)]),
        "sc_profile": (ctypes.c_int, [vp, ctypes.c_int]),
        "sc_get_kernel_times": (ctypes.c_int, [vp, ctypes.POINTER(KernelTime), ctypes.c_int,
                                               ctypes.POINTER(ctypes.c_int)]),
        "sc_last_error": (ctypes.c_char_p, []),
        "sc_mask_keep_count": (ctypes.c_int, [ctypes.c_int, ctypes.c_float, ctypes.POINTER(ctypes.c_int)]),
        "sc_mask_seed": (ctypes.c_int, [ctypes.c_uint64, ctypes.c_uint64, ctypes.c_uint64,
                                        ctypes.POINTER(ctypes.c_uint64)]),
        "sc_mask_indices": (ctypes.c_int, [ctypes.c_uint64, ctypes.c_int64, ctypes.c_int, ctypes.c_int,
                                           vp, vp]),
        "sc_mask_pack": (ctypes.c_int, [ctypes.c_int, vp, vp, ctypes.c_int64, ctypes.c_int, ctypes.c_int,
                                        vp, vp]),
        "sc_mask_unpack": (ctypes.c_int, [ctypes.c_int, vp, vp, ctypes.c_int64, ctypes.c_int, ctypes.c_int,
                                          vp, vp]),
    }
    i64, i32, f32, dt = ctypes.c_int64, ctypes.c_int, ctypes.c_float, ctypes.c_int
    sig.update({
        "sc_embed": (i32, [dt, vp, vp, i64, i64, i32, f32, vp, vp]),
        "sc_embed_grad_workspace": (i32, [i64, i64, i32, i64p]),
        "sc_embed_grad": (i32, [dt, vp, vp, i64, i64, i32, f32, vp, vp, i64, vp]),
        "sc_act_pack": (i32, [dt, vp, i64, i32, vp, vp, vp]),
        "sc_act_unpack": (i32, [dt, vp, vp, i64, i32, vp, vp]),
        "sc_rmsnorm": (i32, [dt, vp, vp, vp, f32, i64, i32, vp, vp, vp, vp, vp, vp]),
        "sc_rmsnorm_grad_workspace": (i32, [i64, i32, i64p]),
        "sc_rmsnorm_grad": (i32, [dt, vp, vp, vp, vp, vp, vp, i64, i32, vp, vp, vp, i64, vp]),
        "sc_act_wgrad_workspace": (i32, [dt, i64, i64, i32, i64p]),
        "sc_act_wgrad": (i32, [dt, vp, vp, vp, vp, i64, i64, i32, vp, vp, i64, vp]),
        "sc_xent_workspace": (i32, [dt, i64, i64, i32, i64, i64p]),
        "sc_xent": (i32, [dt, vp, vp, vp, i64, i64, i32, i64, vp, vp, vp, vp, vp, i64, vp]),
    })
    for name, (res, args) in sig.items():
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args
    _lib = lib
    return lib


def _check(rc: int):
    if rc != 0:
        raise ScoptError(rc, load_library().sc_last_error().decode())


def default_hparams() -> dict:
    hp = HParams()
    load_library().sc_default_hparams(ctypes.byref(hp))
    return {name: getattr(hp, name) for name, _ in HParams._fields_}


_DT = {torch.float32: SC_F32, torch.bfloat16: SC_BF16}


class SpectralAdamW:
    """Spectral-correction AdamW over a fixed list of weight-matrix shapes.

    shapes: [(rows, cols), ...] of the row-major weights ([out, in]).
    w_dtype: torch.float32 or torch.bfloat16 (storage of W); g_dtype: type of
    G_mask and G_anc.  Keyword hyper-parameters: tau_p, alpha, beta_anc, lr,
    beta1, beta2, eps, weight_decay, max_sweeps, jacobi_tol, sync_check,
    warm_start, precondition.
    """

    def __init__(self, shapes, w_dtype=torch.float32, g_dtype=torch.float32, device=None, **hp):
        lib = load_library()
        self.shapes = [(int(r), int(c)) for r, c in shapes]
        self.n = len(self.shapes)
        if w_dtype not in _DT or g_dtype not in _DT:
            raise ValueError("dtypes must be torch.float32 or torch.bfloat16")
        self.w_dtype, self.g_dtype = w_dtype, g_dtype
        self.device = torch.device(device if device is not None else "cuda")
        if self.device.index is None:
            self.device = torch.device("cuda", torch.cuda.current_device())
        h = HParams()
        lib.sc_default_hparams(ctypes.byref(h))
        for k, v in hp.items():
            if not hasattr(h, k):
                raise TypeError(f"unknown hyper-parameter {k}")
            setattr(h, k, v)
        self.hp = {name: getattr(h, name) for name, _ in HParams._fields_}
        rows = (ctypes.c_int64 * self.n)(*[r for r, _ in self.shapes])
        cols = (ctypes.c_int64 * self.n)(*[c for _, c in self.shapes])
        handle = ctypes.c_void_p()
        _check(lib.sc_opt_create(ctypes.byref(handle), self.n, rows, cols, _DT[w_dtype],
                                 _DT[g_dtype], ctypes.byref(h), self.device.index))
        self._h = handle
        self._lib = lib

    # -- helpers -------------------------------------------------------------------------
    def _stream(self):
        return ctypes.c_void_p(torch.cuda.current_stream(self.device).cuda_stream)

    def _ptrs(self, tensors, dtype, what):
        if len(tensors) != self.n:
            raise ValueError(f"{what}: expected {self.n} tensors, got {len(tensors)}")
        arr = (ctypes.c_void_p * self.n)()
        for i, (t, shp) in enumerate(zip(tensors, self.shapes)):
            if t.device != self.device or t.dtype != dtype or tuple(t.shape) != shp or \
                    not t.is_contiguous():
                raise ValueError(f"{what}[{i}] must be a contiguous {dtype} tensor of shape {shp} "
                                 f"on {self.device}, got {t.dtype} {tuple(t.shape)} on {t.device}")
            arr[i] = t.data_ptr()
        return arr

    def _f32(self, idx, t, shape, what):
        if t.device != self.device or t.dtype != torch.float32 or tuple(t.shape) != tuple(shape) \
                or not t.is_contiguous():
            raise ValueError(f"{what} must be a contiguous float32 tensor of shape {tuple(shape)}")
        return ctypes.c_void_p(t.data_ptr())

    # -- the method ----------------------------------------------------------------------
    def anchor_update(self, G_anc):
        """EMA of the anchor momentum with G_anc, then SVD refresh."""
        _check(self._lib.sc_anchor_update(self._h, self._ptrs(G_anc, self.g_dtype, "G_anc"),
                                          self._stream()))

    def refresh(self):
        _check(self._lib.sc_refresh(self._h, self._stream()))

    def anchor_update_async(self, G_anc):
        """EMA with G_anc and SVD refresh beside the following steps, which use the
        previous factors until refresh_wait().  G_anc must stay valid and
        unchanged until then."""
        _check(self._lib.sc_anchor_update_async(self._h, self._ptrs(G_anc, self.g_dtype, "G_anc"),
                                                self._stream()))

    def refresh_wait(self):
        """Complete a pending asynchronous refresh: the current stream waits for it
        and later steps use its factors."""
        _check(self._lib.sc_refresh_wait(self._h, self._stream()))

    def refresh_pending(self) -> bool:
        p = ctypes.c_int()
        _check(self._lib.sc_refresh_pending(self._h, ctypes.byref(p)))
        return bool(p.value)

    def step(self, W, G_mask):
        """One spectral-corrected AdamW step; W is updated in place."""
        _check(self._lib.sc_step(self._h, self._ptrs(W, self.w_dtype, "W"),
                                 self._ptrs(G_mask, self.g_dtype, "G_mask"), self._stream()))

    def step_noalloc(self, W, G_mask):
        """The same step through the allocation-free entry point (intermediates in
        the library's per-GPU scratch array)."""
        _check(self._lib.sc_step_noalloc(self._h, self._ptrs(W, self.w_dtype, "W"),
                                         self._ptrs(G_mask, self.g_dtype, "G_mask"), self._stream()))

    def set_lr(self, lr: float):
        _check(self._lib.sc_set_lr(self._h, float(lr)))

    def set_tau(self, tau_p: float):
        _check(self._lib.sc_set_tau(self._h, float(tau_p)))

    def set_state(self, idx: int, kind: str, src: torch.Tensor):
        _check(self._lib.sc_set_state(self._h, idx, STATE_KINDS[kind],
                                      self._f32(idx, src, self.shapes[idx], kind), self._stream()))

    def get_state(self, idx: int, kind: str) -> torch.Tensor:
        out = torch.empty(self.shapes[idx], dtype=torch.float32, device=self.device)
        _check(self._lib.sc_get_state(self._h, idx, STATE_KINDS[kind],
                                      ctypes.c_void_p(out.data_ptr()), self._stream()))
        return out

    @property
    def step_count(self) -> int:
        t = ctypes.c_int64()
        _check(self._lib.sc_get_step(self._h, ctypes.byref(t)))
        return t.value

    @step_count.setter
    def step_count(self, t: int):
        _check(self._lib.sc_set_step(self._h, int(t)))

    def set_factors(self, idx: int, U: torch.Tensor, s: torch.Tensor, V: torch.Tensor):
        m, n = self.shapes[idx]
        r = min(m, n)
        _check(self._lib.sc_set_factors(self._h, idx, self._f32(idx, U, (m, r), "U"),
                                        self._f32(idx, s, (r,), "s"), self._f32(idx, V, (n, r), "V"),
                                        self._stream()))

    def get_factors(self, idx: int):
        m, n = self.shapes[idx]
        r = min(m, n)
        U = torch.empty((m, r), dtype=torch.float32, device=self.device)
        s = torch.empty((r,), dtype=torch.float32, device=self.device)
        V = torch.empty((n, r), dtype=torch.float32, device=self.device)
        _check(self._lib.sc_get_factors(self._h, idx, ctypes.c_void_p(U.data_ptr()),
                                        ctypes.c_void_p(s.data_ptr()), ctypes.c_void_p(V.data_ptr()),
                                        self._stream()))
        return U, s, V

    def set_solve_waves(self, waves: int = 0, copies: int = 0):
        """Jacobi pair-solve variant: `waves` (1, 2, 4, 8) wavefronts per pair and
        `copies` (1, 2) LDS copies of its Gram; 0 picks by each launch's pair
        count.  All variants give identical results."""
        _check(self._lib.sc_set_solve_waves(self._h, int(waves), int(copies)))

    def set_fused_gram(self, enable: bool = True):
        """Fused rotation apply + next-round pair Gram (default on)."""
        _check(self._lib.sc_set_fused_gram(self._h, 1 if enable else 0))

    def set_v_rounds(self, rounds: int = 2):
        """V-row rotations of the fused sweeps: 2 rounds per pass (default) or 1;
        bit-identical results."""
        _check(self._lib.sc_set_v_rounds(self._h, int(rounds)))

    def set_sweep_stop(self, stop: float = 1e-4):
        """Sweep-stop rule of the Jacobi sweeps (0 = off); a certificate checks
        the result."""
        _check(self._lib.sc_set_sweep_stop(self._h, float(stop)))

    def set_quad(self, mode: int = 1):
        """Quad passes of the Jacobi sweeps (three pair rounds per pass over groups
        of four column blocks): 0 off, 1 (default) where a list's block counts
        allow and its groups fill the GPU, 2 wherever the block counts allow."""
        _check(self._lib.sc_set_quad(self._h, int(mode)))

    def keep_proj(self, enable: bool = True):
        _check(self._lib.sc_keep_proj(self._h, 1 if enable else 0))

    def get_filtered(self, idx: int, proj: bool = False):
        shp = self.shapes[idx]
        gf = torch.empty(shp, dtype=torch.float32, device=self.device)
        gp = torch.empty(shp, dtype=torch.float32, device=self.device) if proj else None
        _check(self._lib.sc_get_filtered(self._h, idx, ctypes.c_void_p(gf.data_ptr()),
                                         ctypes.c_void_p(gp.data_ptr() if gp is not None else None),
                                         self._stream()))
        return (gf, gp) if proj else gf

    def stats(self):
        st = Stats()
        per = (ctypes.c_int * self.n)()
        _check(self._lib.sc_get_stats(self._h, ctypes.byref(st), per))
        d = {name: getattr(st, name) for name, _ in Stats._fields_}
        d["sweeps"] = list(per)
        fac = (ctypes.c_int * self.n)()
        _check(self._lib.sc_get_sweep_counts(self._h, None, fac))
        d["factor_sweeps"] = list(fac)
        return d

    def profile(self, enable: bool = True, serial: bool = False):
        """Enable / disable per-kernel event timing (resets the totals).  serial:
        every kernel alone on the current stream (slower pass); otherwise the
        production schedule, each launch timed on its own stream."""
        _check(self._lib.sc_profile(self._h, (2 if serial else 1) if enable else 0))

    def kernel_times(self):
        """{family: dict(launches, total_ms, flops, bytes)} accumulated since profile(True)."""
        arr = (KernelTime * 64)()
        cnt = ctypes.c_int()
        _check(self._lib.sc_get_kernel_times(self._h, arr, 64, ctypes.byref(cnt)))
        out = {}
        for i in range(min(cnt.value, 64)):
            k = arr[i]
            out[k.name.decode()] = dict(launches=k.launches, total_ms=k.total_ms, flops=k.flops,
                                        bytes=k.bytes)
        return out

    def close(self):
        if getattr(self, "_h", None):
            self._lib.sc_opt_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# ---- in-graph activation mask ("Key design 1"): stateless calls --------------------

def mask_keep_count(H: int, p: float) -> int:
    """Kept dimensions per token at mask rate p: floor((1 - p) H + 1/2)."""
    k = ctypes.c_int()
    _check(load_library().sc_mask_keep_count(int(H), float(p), ctypes.byref(k)))
    return k.value


def mask_seed(layer: int, step: int, batch: int) -> int:
    """The mask seed of (layer, step, batch)."""
    s = ctypes.c_uint64()
    _check(load_library().sc_mask_seed(int(layer), int(step), int(batch), ctypes.byref(s)))
    return s.value


def _cur_stream(dev):
    return ctypes.c_void_p(torch.cuda.current_stream(dev).cuda_stream)


def mask_indices(seed: int, T: int, H: int, K: int, device=None) -> "torch.Tensor":
    """Kept dimensions of each of T tokens: int32 [T, K] on the device, ascending."""
    dev = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
    idx = torch.empty((T, K), dtype=torch.int32, device=dev)
    _check(load_library().sc_mask_indices(int(seed), int(T), int(H), int(K),
                                          ctypes.c_void_p(idx.data_ptr()), _cur_stream(dev)))
    return idx


def _mask_dt(t):
    if t.dtype == torch.float32:
        return SC_F32
    if t.dtype == torch.bfloat16:
        return SC_BF16
    raise ValueError(f"mask tensors must be float32 or bfloat16, got {t.dtype}")


def mask_pack(x: "torch.Tensor", idx: "torch.Tensor") -> "torch.Tensor":
    """Kept values of each token (x: [T, H] contiguous; idx: int32 [T, K])."""
    T, H = x.shape
    K = idx.shape[1]
    if not (x.is_contiguous() and idx.is_contiguous() and idx.dtype == torch.int32 and idx.shape[0] == T
            and idx.device == x.device):
        raise ValueError("mask_pack: contiguous x [T, H] and int32 idx [T, K] on one device")
    out = torch.empty((T, K), dtype=x.dtype, device=x.device)
    _check(load_library().sc_mask_pack(_mask_dt(x), ctypes.c_void_p(x.data_ptr()),
                                       ctypes.c_void_p(idx.data_ptr()), T, H, K,
                                       ctypes.c_void_p(out.data_ptr()), _cur_stream(x.device)))
    return out


def mask_unpack(packed: "torch.Tensor", idx: "torch.Tensor", H: int) -> "torch.Tensor":
    """Dense [T, H] rows with the packed values at idx and zeros elsewhere."""
    T, K = packed.shape
    if not (packed.is_contiguous() and idx.is_contiguous() and idx.dtype == torch.int32
            and tuple(idx.shape) == (T, K) and idx.device == packed.device):
        raise ValueError("mask_unpack: contiguous packed [T, K] and int32 idx [T, K] on one device")
    out = torch.empty((T, H), dtype=packed.dtype, device=packed.device)
    _check(load_library().sc_mask_unpack(_mask_dt(packed), ctypes.c_void_p(packed.data_ptr()),
                                         ctypes.c_void_p(idx.data_ptr()), T, int(H), K,
                                         ctypes.c_void_p(out.data_ptr()), _cur_stream(packed.device)))
    return out


# ---- training-step operators: stateless calls --------------------------------------
# Tensors are contiguous and on one device; work is queued on its current stream.  These are plain
# functions, not autograd ones: tensors that require gradients are taken as values, and the
# results carry no graph.  The gradients are calls of their own (embed_grad, rmsnorm_grad, act_wgrad, xent).

ActCheckpoint = collections.namedtuple("ActCheckpoint", "q e")
ActCheckpoint.__doc__ = """An 8-bit checkpoint of a matrix [T, H]: int8 q [T, H] and uint8 e [T, ceil(H / 32)];
32 elements along a row stand for q * 2^(e - 133).  e = 255 marks a block that held a NaN or
an infinity; it reads as NaN."""

RmsNorm = collections.namedtuple("RmsNorm", "h y rstd kept")
RmsNorm.__doc__ = """Of rmsnorm: the residual sum h, the output y, 1 / rms (float32 [T]) and the
checkpoint of the normalised rows (None where none was kept)."""

CrossEntropy = collections.namedtuple("CrossEntropy", "loss mean dh dW")
CrossEntropy.__doc__ = """Of xent: float32 losses [T], their mean over the counted tokens (0-dim), and the mean's
gradients."""


def _train_check(who, dtype, dev, *named):
    """named: (name, tensor, dtype, shape)."""
    if dtype not in _DT:
        raise ValueError(f"{who}: tensors must be float32 or bfloat16, got {dtype}")
    if dev.type != "cuda":
        raise ValueError(f"{who}: tensors must be on a GPU, got {dev}")
    for name, t, dt, shape in named:
        if t.dtype is not dt or t.shape != shape or t.device != dev or not t.is_contiguous():
            raise ValueError(f"{who}: {name} must be a contiguous {dt} tensor of shape {tuple(shape)} on {dev}, "
                             f"got {t.dtype} {tuple(t.shape)} on {t.device}"
                             f"{'' if t.is_contiguous() else ' (not contiguous)'}")


def _matrix(who, name, t):
    if t.dim() != 2:
        raise ValueError(f"{who}: {name} must be a matrix, got shape {tuple(t.shape)}")
    return t.shape


def _at16(t):
    """t, or a copy where a view starts off 16 bytes (the products fetch 16 bytes at a time)."""
    return t if t.data_ptr() % 16 == 0 else t.clone()


def _run(dev, fn, *args):
    """Call with the device current and its stream last (the raw handle: a Stream object costs a
    small call 2 us of its 10)."""
    if dev.index == torch.cuda.current_device():
        rc = fn(*args, torch._C._cuda_getCurrentRawStream(dev.index))
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, torch._C._cuda_getCurrentRawStream(dev.index))
    if rc:
        _check(rc)


@functools.lru_cache(maxsize=1024)
def _workspace_bytes(query, *sizes):
    n = ctypes.c_int64()
    _check(getattr(load_library(), query)(*sizes, ctypes.byref(n)))
    return n.value


def _workspace(dev, query, *sizes):
    n = _workspace_bytes(query, *sizes)
    return torch.empty(n, dtype=torch.uint8, device=dev), n


def _ptr(t):
    return None if t is None else t.data_ptr()


def embed(table: "torch.Tensor", ids: "torch.Tensor", scale: float = 1.0) -> "torch.Tensor":
    """scale * table[ids] (table [V, H], ids int64 of any shape); rows of zeros where an id is
    outside [0, V)."""
    V, H = _matrix("embed", "table", table)
    _train_check("embed", table.dtype, table.device, ("table", table, table.dtype, (V, H)),
                 ("ids", ids, torch.int64, ids.shape))
    out = torch.empty((*ids.shape, H), dtype=table.dtype, device=table.device)
    _run(table.device, load_library().sc_embed, _DT[table.dtype], table.data_ptr(), ids.data_ptr(), ids.numel(), V, H,
         float(scale), out.data_ptr())
    return out


def embed_grad(dy: "torch.Tensor", ids: "torch.Tensor", V: int, scale: float = 1.0) -> "torch.Tensor":
    """Gradient [V, H] of the table of embed: scale * the sum of dy [..., H] over each id's
    tokens, in float32, in an order that the ids fix."""
    if dy.dim() < 1 or tuple(dy.shape[:-1]) != tuple(ids.shape):
        raise ValueError(f"embed_grad: dy {tuple(dy.shape)} must be ids {tuple(ids.shape)} and the hidden size")
    H = dy.shape[-1]
    _train_check("embed_grad", dy.dtype, dy.device, ("dy", dy, dy.dtype, dy.shape), ("ids", ids, torch.int64, ids.shape))
    lib, T, V = load_library(), ids.numel(), int(V)
    ws, n = _workspace(dy.device, "sc_embed_grad_workspace", T, V, H)
    dW = torch.empty((V, H), dtype=dy.dtype, device=dy.device)
    _run(dy.device, lib.sc_embed_grad, _DT[dy.dtype], dy.data_ptr(), ids.data_ptr(), T, V, H, float(scale),
         dW.data_ptr(), ws.data_ptr(), n)
    return dW


def act_pack(x: "torch.Tensor") -> ActCheckpoint:
    """The 8-bit checkpoint of x [T, H]."""
    T, H = _matrix("act_pack", "x", x)
    _train_check("act_pack", x.dtype, x.device, ("x", x, x.dtype, (T, H)))
    q = torch.empty((T, H), dtype=torch.int8, device=x.device)
    e = torch.empty((T, -(-H // 32)), dtype=torch.uint8, device=x.device)
    _run(x.device, load_library().sc_act_pack, _DT[x.dtype], x.data_ptr(), T, H, q.data_ptr(), e.data_ptr())
    return ActCheckpoint(q, e)


def _check_kept(who, kept, T, H, dtype, dev):
    _train_check(who, dtype, dev, ("q", kept.q, torch.int8, (T, H)), ("e", kept.e, torch.uint8, (T, -(-H // 32))))


def act_unpack(kept: ActCheckpoint, dtype: "torch.dtype" = torch.bfloat16) -> "torch.Tensor":
    """The values of a checkpoint (exact in either dtype)."""
    T, H = _matrix("act_unpack", "q", kept.q)
    _check_kept("act_unpack", kept, T, H, dtype, kept.q.device)
    x = torch.empty((T, H), dtype=dtype, device=kept.q.device)
    _run(x.device, load_library().sc_act_unpack, _DT[dtype], kept.q.data_ptr(), kept.e.data_ptr(), T, H, x.data_ptr())
    return x


def rmsnorm(x: "torch.Tensor", gain: "torch.Tensor", residual: "torch.Tensor" = None, eps: float = 1e-5,
            keep: bool = True) -> RmsNorm:
    """h = x + residual (x without one), rstd = 1 / sqrt(mean(h^2) + eps), y = h * rstd * gain
    for rows of x [T, H], and with keep the 8-bit checkpoint of h * rstd for the backward pass."""
    T, H = _matrix("rmsnorm", "x", x)
    named = [("x", x, x.dtype, (T, H)), ("gain", gain, x.dtype, (H,))]
    if residual is not None:
        named.append(("residual", residual, x.dtype, (T, H)))
    dev = x.device
    _train_check("rmsnorm", x.dtype, dev, *named)
    h = x if residual is None else torch.empty_like(x)
    y = torch.empty_like(x)
    rstd = torch.empty(T, dtype=torch.float32, device=dev)
    kept = None
    if keep:
        kept = ActCheckpoint(torch.empty((T, H), dtype=torch.int8, device=dev),
                             torch.empty((T, -(-H // 32)), dtype=torch.uint8, device=dev))
    _run(dev, load_library().sc_rmsnorm, _DT[x.dtype], x.data_ptr(), _ptr(residual), gain.data_ptr(), float(eps), T, H,
         None if residual is None else h.data_ptr(), y.data_ptr(), rstd.data_ptr(),
         kept.q.data_ptr() if keep else None, kept.e.data_ptr() if keep else None)
    return RmsNorm(h, y, rstd, kept)


def rmsnorm_grad(dy: "torch.Tensor", gain: "torch.Tensor", rstd: "torch.Tensor", kept: ActCheckpoint,
                 dh: "torch.Tensor" = None):
    """(dx, dgain) of rmsnorm from its checkpoint: dx [T, H] is the gradient of x and of the
    residual, with dh, the gradient that reaches h past the norm, added; dgain float32 [H]."""
    T, H = _matrix("rmsnorm_grad", "dy", dy)
    named = [("dy", dy, dy.dtype, (T, H)), ("gain", gain, dy.dtype, (H,)), ("rstd", rstd, torch.float32, (T,))]
    if dh is not None:
        named.append(("dh", dh, dy.dtype, (T, H)))
    dev = dy.device
    _train_check("rmsnorm_grad", dy.dtype, dev, *named)
    _check_kept("rmsnorm_grad", kept, T, H, dy.dtype, dev)
    lib = load_library()
    ws, n = _workspace(dev, "sc_rmsnorm_grad_workspace", T, H)
    dx = torch.empty_like(dy)
    dgain = torch.empty(H, dtype=torch.float32, device=dev)
    _run(dev, lib.sc_rmsnorm_grad, _DT[dy.dtype], dy.data_ptr(), gain.data_ptr(), rstd.data_ptr(), kept.q.data_ptr(),
         kept.e.data_ptr(), _ptr(dh), T, H, dx.data_ptr(), dgain.data_ptr(), ws.data_ptr(), n)
    return dx, dgain


def act_wgrad(dy: "torch.Tensor", kept: ActCheckpoint, gain: "torch.Tensor" = None) -> "torch.Tensor":
    """Weight gradient [N, H] of a projection whose input is n * gain, with n read from its
    checkpoint: (dy^T n) * gain for dy [T, N]."""
    T, N = _matrix("act_wgrad", "dy", dy)
    H = _matrix("act_wgrad", "q", kept.q)[1]
    dev = dy.device
    named = [("dy", dy, dy.dtype, (T, N))]
    if gain is not None:
        named.append(("gain", gain, dy.dtype, (H,)))
    _train_check("act_wgrad", dy.dtype, dev, *named)
    _check_kept("act_wgrad", kept, T, H, dy.dtype, dev)
    lib = load_library()
    dy = _at16(dy)
    ws, n = _workspace(dev, "sc_act_wgrad_workspace", _DT[dy.dtype], T, N, H)
    dW = torch.empty((N, H), dtype=dy.dtype, device=dev)
    _run(dev, lib.sc_act_wgrad, _DT[dy.dtype], dy.data_ptr(), kept.q.data_ptr(), kept.e.data_ptr(), _ptr(gain), T, N,
         H, dW.data_ptr(), ws.data_ptr(), n)
    return dW


def xent(h: "torch.Tensor", W: "torch.Tensor", targets: "torch.Tensor", limit: int = 0) -> CrossEntropy:
    """Softmax cross entropy of the logits h W^T (h [T, H], W [V, H]) against int64 targets [T], with the
    gradients of the mean over the counted tokens.  A target outside [0, V) is not counted: its loss
    is 0.  limit: bytes for a vocabulary piece's intermediate values (0: 4 GiB).  Where the whole
    vocabulary's fit (2 bytes for each of T x V entries, 10 in float32) they are kept between the
    passes; otherwise there is no matrix of logits, and each piece's are computed again, about a
    quarter slower."""
    T, H = _matrix("xent", "h", h)
    V = _matrix("xent", "W", W)[0]
    dev = h.device
    _train_check("xent", h.dtype, dev, ("h", h, h.dtype, (T, H)), ("W", W, h.dtype, (V, H)),
                 ("targets", targets, torch.int64, (T,)))
    lib = load_library()
    h, W = _at16(h), _at16(W)
    ws, n = _workspace(dev, "sc_xent_workspace", _DT[h.dtype], T, V, H, int(limit))
    loss = torch.empty(T, dtype=torch.float32, device=dev)
    mean = torch.empty((), dtype=torch.float32, device=dev)
    dh, dW = torch.empty_like(h), torch.empty_like(W)
    _run(dev, lib.sc_xent, _DT[h.dtype], h.data_ptr(), W.data_ptr(), targets.data_ptr(), T, V, H, int(limit),
         loss.data_ptr(), mean.data_ptr(), dh.data_ptr(), dW.data_ptr(), ws.data_ptr(), n)
    return CrossEntropy(loss, mean, dh, dW)
