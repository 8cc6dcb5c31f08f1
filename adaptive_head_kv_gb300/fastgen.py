"""Python binding of libfastgen.so: argument marshalling only.

Every function has the name and argument order of the C entry point in
include/fastgen.h.  Tensor arguments are torch tensors (their data_ptr() is
passed) or raw integer addresses; `stream` defaults to torch's current CUDA
stream.  A negative status raises FastGenError.  There is no fallback: if the
shared library is missing, every call raises.  The rotation and the paged
calls (at the end) take tensors only and check their types and sizes.
"""
from __future__ import annotations

import ctypes
import os

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libfastgen.so")

FG_OK, FG_EINVAL, FG_EDTYPE, FG_EWORKSPACE, FG_ECAPACITY, FG_ECUDA, FG_EDEVICE = 0, -1, -2, -3, -4, -5, -6
FG_BF16, FG_FP32 = 0, 1
FG_POLICY_S, FG_POLICY_SP, FG_POLICY_SPF, FG_POLICY_SPFL, FG_POLICY_FULL = range(5)
POLICY_NAMES = ("special", "special+punct", "special+punct+frequent",
                "special+punct+frequent+local", "full")
FG_KEEP_DROP, FG_KEEP_STATIC, FG_KEEP_WINDOW = 0, 1, 2
FG_ROPE_INTERLEAVED, FG_ROPE_HALF = 0, 1
FG_PAGE_ROWS, FG_BLOCK_ROWS = 64, 16

# kernels launched by one call of each entry point (counted in the bench)
LAUNCHES = {"profile": 4, "profile_attn": 5, "profile_with_policy": 5, "plan": 3, "compact": 1,
            "decode": 2, "decode_acc": 3, "refresh": 1, "refresh_init": 1, "rope": 1, "paged_plan": 5,
            "paged_schedule": 2, "compact_q8": 1, "append_q8": 2, "decode_q8": 2}

EXPORTS = (
    "fastgen_status_string", "fastgen_version", "fastgen_profile_workspace_bytes",
    "fastgen_profile", "fastgen_plan_bytes", "fastgen_compact_plan", "fastgen_compact",
    "fastgen_decode_workspace_bytes", "fastgen_decode_attn", "fastgen_read_error",
    "fastgen_decode_attn_noalloc", "fastgen_profile_with_policy", "fastgen_profile_attn",
    "fastgen_plan_compact", "fastgen_refresh_state_bytes", "fastgen_refresh_init",
    "fastgen_decode_attn_refresh", "fastgen_profile_stall_test", "fastgen_rope_table",
    "fastgen_rope", "fastgen_paged_table_len", "fastgen_paged_sched_bytes", "fastgen_paged_plan",
    "fastgen_paged_schedule", "fastgen_compact_q8", "fastgen_append_q8_workspace_bytes",
    "fastgen_append_q8", "fastgen_decode_q8_workspace_bytes", "fastgen_decode_attn_q8",
)

# size of the library-held scratch array used by fastgen_decode_attn_noalloc
NOALLOC_SCRATCH_BYTES = 8 * 1024 * 1024


class Params(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("L", ctypes.c_int32), ("H", ctypes.c_int32),
                ("n", ctypes.c_int32), ("d", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("T", ctypes.c_float), ("r_l", ctypes.c_float), ("r_f", ctypes.c_float),
                ("scale", ctypes.c_float), ("Hkv", ctypes.c_int32)]


class HeadDesc(ctypes.Structure):
    _fields_ = [("off", ctypes.c_int64), ("n_static", ctypes.c_int32),
                ("static_cap", ctypes.c_int32), ("win_off", ctypes.c_int64),
                ("w", ctypes.c_int32), ("policy", ctypes.c_int32),
                ("work_off", ctypes.c_int32), ("n_work", ctypes.c_int32)]


class PlanInfo(ctypes.Structure):
    _fields_ = [("pool_rows", ctypes.c_int64), ("n_work", ctypes.c_int32),
                ("rows_per_work", ctypes.c_int32)]


class RopeStruct(ctypes.Structure):
    _fields_ = [("turns", ctypes.c_void_p), ("rot_dim", ctypes.c_int32),
                ("style", ctypes.c_int32)]


class PagedDesc(ctypes.Structure):
    _fields_ = [("policy", ctypes.c_int32), ("w", ctypes.c_int32),
                ("first_page", ctypes.c_int32), ("max_pages", ctypes.c_int32),
                ("ring_page", ctypes.c_int32), ("ring_pages", ctypes.c_int32)]


class PagedCacheStruct(ctypes.Structure):
    _fields_ = [("k_pages", ctypes.c_void_p), ("v_pages", ctypes.c_void_p),
                ("exps", ctypes.c_void_p), ("pos", ctypes.c_void_p),
                ("page_table", ctypes.c_void_p), ("caches", ctypes.c_void_p),
                ("rows", ctypes.c_void_p), ("rows_out", ctypes.c_void_p),
                ("next_page", ctypes.c_void_p), ("sched", ctypes.c_void_p),
                ("sched_bytes", ctypes.c_int64), ("n_pages", ctypes.c_int32),
                ("table_len", ctypes.c_int32), ("n_work", ctypes.c_int32),
                ("n_ctas", ctypes.c_int32)]


class PagedInfo(ctypes.Structure):
    _fields_ = [("pages", ctypes.c_int32), ("max_pages", ctypes.c_int32),
                ("table_used", ctypes.c_int32)]


class FastGenError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} ({status})")


_lib = None
_P = ctypes.c_void_p
_I32, _I64, _SZ = ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
_PP, _CP, _RP = (ctypes.POINTER(x) for x in (Params, PagedCacheStruct, RopeStruct))
_SIGS = {
    "fastgen_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "fastgen_version": (_I32, []),
    "fastgen_profile_workspace_bytes": (_SZ, [ctypes.POINTER(Params)]),
    "fastgen_profile": (ctypes.c_int, [ctypes.POINTER(Params), _P, _P, _P, _P, _I32, _P, _I32,
                                       _P, _P, _P, _P, _P, _P, _P, _SZ, _P, _P]),
    "fastgen_profile_with_policy": (ctypes.c_int, [ctypes.POINTER(Params), _P, _P, _P, _P, _I32,
                                                   _P, _I32, _P, _P, _P, _P, _P, _SZ, _P, _P]),
    "fastgen_profile_attn": (ctypes.c_int, [ctypes.POINTER(Params), _P, _P, _P, _P, _P, _I32, _P,
                                            _I32, _P, _P, _P, _P, _P, _P, _P, _P, _SZ, _P, _P]),
    "fastgen_plan_bytes": (_SZ, [ctypes.POINTER(Params), _I32]),
    "fastgen_compact_plan": (ctypes.c_int, [ctypes.POINTER(Params), _P, _P, _I32, _P, _SZ,
                                            ctypes.POINTER(PlanInfo), _P]),
    "fastgen_compact": (ctypes.c_int, [ctypes.POINTER(Params), _P, _P, _P, _P,
                                       ctypes.POINTER(PlanInfo), _P, _P, _P, _I64, _P]),
    "fastgen_plan_compact": (ctypes.c_int, [ctypes.POINTER(Params), _P, _P, ctypes.c_int32, _P,
                                            _SZ, _P, _P, _P, _P, _P, _I64,
                                            ctypes.POINTER(PlanInfo), _P]),
    "fastgen_decode_workspace_bytes": (_SZ, [ctypes.POINTER(Params), ctypes.POINTER(PlanInfo)]),
    "fastgen_decode_attn": (ctypes.c_int, [ctypes.POINTER(Params), _P, ctypes.POINTER(PlanInfo),
                                           _P, _P, _P, _P, _P, _P, _P, _P, _I32, _P, _I32, _I32,
                                           _P, _P, _SZ, _P, _P]),
    "fastgen_read_error": (ctypes.c_int, [_P, _P]),
    "fastgen_profile_stall_test": (ctypes.c_int, [ctypes.POINTER(Params), _P, _P, _P, _P, _I32,
                                                  _P, _I32, _P, _P, _P, _P, _P, _P, _P, _SZ, _P,
                                                  _I32, _P]),
    "fastgen_refresh_state_bytes": (_SZ, [ctypes.POINTER(Params), ctypes.POINTER(PlanInfo)]),
    "fastgen_refresh_init": (ctypes.c_int, [ctypes.POINTER(Params), _P, ctypes.POINTER(PlanInfo),
                                            _P, _P, _P, _P, _I32, _P, _I32, _P, _SZ, _P]),
    "fastgen_decode_attn_refresh": (ctypes.c_int, [ctypes.POINTER(Params), _P,
                                                   ctypes.POINTER(PlanInfo), _P, _P, _P, _P, _P,
                                                   _P, _P, _P, _I32, _P, _I32, _I32, _I32, _P, _P,
                                                   _SZ, _P, _SZ, _P, _P]),
    "fastgen_decode_attn_noalloc": (ctypes.c_int, [ctypes.POINTER(Params), _P,
                                                   ctypes.POINTER(PlanInfo), _P, _P, _P, _P, _P,
                                                   _P, _P, _P, _I32, _P, _I32, _I32, _P, _P, _P]),
    "fastgen_rope_table": (ctypes.c_int, [_P, _I32, _P]),
    "fastgen_rope": (ctypes.c_int, [_PP, _P, _P, _P, _RP, _P, _P, _P]),
    "fastgen_paged_table_len": (_I32, [_PP, _I32]),
    "fastgen_paged_sched_bytes": (_SZ, [_PP, _I32]),
    "fastgen_paged_plan": (ctypes.c_int, [_PP, _P, _P, _I32, _CP, ctypes.POINTER(PagedInfo), _P]),
    "fastgen_paged_schedule": (ctypes.c_int, [_PP, _CP, _P]),
    "fastgen_compact_q8": (ctypes.c_int, [_PP, _P, _P, _P, _CP, _P, _P]),
    "fastgen_append_q8_workspace_bytes": (_SZ, [_PP, _I32]),
    "fastgen_append_q8": (ctypes.c_int, [_PP, _CP, _P, _P, _P, _I32, _P, _P, _I32, _P, _I32, _P,
                                         _RP, _P, _SZ, _P, _P]),
    "fastgen_decode_q8_workspace_bytes": (_SZ, [_PP, _CP]),
    "fastgen_decode_attn_q8": (ctypes.c_int, [_PP, _CP, _P, _P, _P, _P, _P, _I32, _P, _I32, _P,
                                              _RP, _P, _P, _SZ, _P, _P]),
}


def lib() -> ctypes.CDLL:
    """The loaded library; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise FileNotFoundError(
                f"{LIB_PATH} is missing: build it with adaptive_head_kv_gb300.build.build()")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def _ptr(x) -> int | None:
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _count(x) -> int:
    return 0 if x is None else int(x.numel())


def _stream(stream) -> int | None:
    if stream is None:
        import torch

        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(status: int, where: str) -> None:
    if status != FG_OK:
        raise FastGenError(status, where)


def status_string(status: int) -> str:
    return lib().fastgen_status_string(status).decode()


def fastgen_status_string(status: int) -> str:
    return status_string(status)


def fastgen_version() -> int:
    return lib().fastgen_version()


def fastgen_profile_workspace_bytes(params: Params) -> int:
    return lib().fastgen_profile_workspace_bytes(ctypes.byref(params))


def fastgen_profile(params, Q, K, token_ids, special_ids, punct_ids, policy, mass, cost, colsum,
                    keep, kept, workspace, dev_err, stream=None) -> None:
    ws_bytes = workspace.numel() * workspace.element_size() if hasattr(workspace, "numel") else 0
    _check(lib().fastgen_profile(ctypes.byref(params), _ptr(Q), _ptr(K), _ptr(token_ids),
                                 _ptr(special_ids), _count(special_ids), _ptr(punct_ids),
                                 _count(punct_ids), _ptr(policy), _ptr(mass), _ptr(cost),
                                 _ptr(colsum), _ptr(keep), _ptr(kept), _ptr(workspace), ws_bytes,
                                 _ptr(dev_err), _stream(stream)), "fastgen_profile")


def fastgen_profile_with_policy(params, Q, K, token_ids, special_ids, punct_ids, policy, colsum,
                                keep, kept, workspace, dev_err, stream=None) -> None:
    ws_bytes = workspace.numel() * workspace.element_size() if hasattr(workspace, "numel") else 0
    _check(lib().fastgen_profile_with_policy(
        ctypes.byref(params), _ptr(Q), _ptr(K), _ptr(token_ids), _ptr(special_ids),
        _count(special_ids), _ptr(punct_ids), _count(punct_ids), _ptr(policy), _ptr(colsum),
        _ptr(keep), _ptr(kept), _ptr(workspace), ws_bytes, _ptr(dev_err), _stream(stream)),
        "fastgen_profile_with_policy")


def fastgen_profile_attn(params, Q, K, V, token_ids, special_ids, punct_ids, policy, mass, cost,
                         colsum, keep, kept, out, workspace, dev_err, stream=None) -> None:
    ws_bytes = workspace.numel() * workspace.element_size() if hasattr(workspace, "numel") else 0
    _check(lib().fastgen_profile_attn(
        ctypes.byref(params), _ptr(Q), _ptr(K), _ptr(V), _ptr(token_ids), _ptr(special_ids),
        _count(special_ids), _ptr(punct_ids), _count(punct_ids), _ptr(policy), _ptr(mass),
        _ptr(cost), _ptr(colsum), _ptr(keep), _ptr(kept), _ptr(out), _ptr(workspace), ws_bytes,
        _ptr(dev_err), _stream(stream)), "fastgen_profile_attn")


def fastgen_plan_bytes(params: Params, max_new_tokens: int) -> int:
    return lib().fastgen_plan_bytes(ctypes.byref(params), max_new_tokens)


def fastgen_compact_plan(params, policy, keep, max_new_tokens, plan, stream=None) -> PlanInfo:
    info = PlanInfo()
    _check(lib().fastgen_compact_plan(ctypes.byref(params), _ptr(policy), _ptr(keep),
                                      max_new_tokens, _ptr(plan), plan.numel() * plan.element_size(),
                                      ctypes.byref(info), _stream(stream)), "fastgen_compact_plan")
    return info


def fastgen_compact(params, K, V, keep, plan, info, K_pool, V_pool, pos_pool, stream=None) -> None:
    _check(lib().fastgen_compact(ctypes.byref(params), _ptr(K), _ptr(V), _ptr(keep), _ptr(plan),
                                 ctypes.byref(info), _ptr(K_pool), _ptr(V_pool), _ptr(pos_pool),
                                 int(pos_pool.numel()), _stream(stream)), "fastgen_compact")


def fastgen_plan_compact(params, policy, keep, max_new_tokens, plan, K, V, K_pool, V_pool,
                         pos_pool, stream=None):
    """Plan and gather in one call.  Returns (done, info): done is False when
    the pools are smaller than info.pool_rows (nothing was gathered)."""
    info = PlanInfo()
    st = lib().fastgen_plan_compact(
        ctypes.byref(params), _ptr(policy), _ptr(keep), max_new_tokens, _ptr(plan),
        plan.numel() * plan.element_size(), _ptr(K), _ptr(V), _ptr(K_pool), _ptr(V_pool),
        _ptr(pos_pool), int(pos_pool.numel()), ctypes.byref(info), _stream(stream))
    if st == FG_EWORKSPACE and info.pool_rows > pos_pool.numel():
        return False, info
    _check(st, "fastgen_plan_compact")
    return True, info


def fastgen_decode_workspace_bytes(params: Params, info: PlanInfo) -> int:
    return lib().fastgen_decode_workspace_bytes(ctypes.byref(params), ctypes.byref(info))


def fastgen_decode_attn(params, plan, info, K_pool, V_pool, pos_pool, q, k_new, v_new, new_ids,
                        special_ids, punct_ids, pos, out, workspace, dev_err, stream=None) -> None:
    _check(lib().fastgen_decode_attn(ctypes.byref(params), _ptr(plan), ctypes.byref(info),
                                     _ptr(K_pool), _ptr(V_pool), _ptr(pos_pool), _ptr(q),
                                     _ptr(k_new), _ptr(v_new), _ptr(new_ids), _ptr(special_ids),
                                     _count(special_ids), _ptr(punct_ids), _count(punct_ids),
                                     int(pos), _ptr(out), _ptr(workspace),
                                     workspace.numel() * workspace.element_size(), _ptr(dev_err),
                                     _stream(stream)), "fastgen_decode_attn")


def fastgen_read_error(dev_err, stream=None) -> int:
    return lib().fastgen_read_error(_ptr(dev_err), _stream(stream))


def fastgen_decode_attn_noalloc(params, plan, info, K_pool, V_pool, pos_pool, q, k_new, v_new,
                                new_ids, special_ids, punct_ids, pos, out, dev_err,
                                stream=None) -> None:
    """fastgen_decode_attn without a workspace: for callers that cannot
    allocate device memory while decoding (the scratch is a fixed array held
    by the library; calls must not overlap on the GPU)."""
    _check(lib().fastgen_decode_attn_noalloc(
        ctypes.byref(params), _ptr(plan), ctypes.byref(info), _ptr(K_pool), _ptr(V_pool),
        _ptr(pos_pool), _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(new_ids), _ptr(special_ids),
        _count(special_ids), _ptr(punct_ids), _count(punct_ids), int(pos), _ptr(out),
        _ptr(dev_err), _stream(stream)), "fastgen_decode_attn_noalloc")


def _nbytes(t) -> int:
    return t.numel() * t.element_size()


def fastgen_refresh_state_bytes(params: Params, info: PlanInfo) -> int:
    return lib().fastgen_refresh_state_bytes(ctypes.byref(params), ctypes.byref(info))


def fastgen_refresh_init(params, plan, info, pos_pool, colsum, token_ids, special_ids, punct_ids,
                         state, stream=None) -> None:
    _check(lib().fastgen_refresh_init(
        ctypes.byref(params), _ptr(plan), ctypes.byref(info), _ptr(pos_pool), _ptr(colsum),
        _ptr(token_ids), _ptr(special_ids), _count(special_ids), _ptr(punct_ids),
        _count(punct_ids), _ptr(state), _nbytes(state), _stream(stream)), "fastgen_refresh_init")


def fastgen_decode_attn_refresh(params, plan, info, K_pool, V_pool, pos_pool, q, k_new, v_new,
                                new_ids, special_ids, punct_ids, pos, period, out, state,
                                workspace, dev_err, stream=None) -> None:
    _check(lib().fastgen_decode_attn_refresh(
        ctypes.byref(params), _ptr(plan), ctypes.byref(info), _ptr(K_pool), _ptr(V_pool),
        _ptr(pos_pool), _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(new_ids), _ptr(special_ids),
        _count(special_ids), _ptr(punct_ids), _count(punct_ids), int(pos), int(period),
        _ptr(out), _ptr(state), _nbytes(state), _ptr(workspace), _nbytes(workspace),
        _ptr(dev_err), _stream(stream)), "fastgen_decode_attn_refresh")


def fastgen_profile_stall_test(params, Q, K, token_ids, special_ids, punct_ids, policy, mass,
                               cost, colsum, keep, kept, workspace, dev_err, stall_pass,
                               stream=None) -> None:
    """fastgen_profile with one tensor-core pass's producer held back, so
    that pass's bounded waits run out (a test of the error path)."""
    _check(lib().fastgen_profile_stall_test(
        ctypes.byref(params), _ptr(Q), _ptr(K), _ptr(token_ids), _ptr(special_ids),
        _count(special_ids), _ptr(punct_ids), _count(punct_ids), _ptr(policy), _ptr(mass),
        _ptr(cost), _ptr(colsum), _ptr(keep), _ptr(kept), _ptr(workspace), _nbytes(workspace),
        _ptr(dev_err), int(stall_pass), _stream(stream)), "fastgen_profile_stall_test")


# ---------------------------------------------------------------------------
# Position rotation and paged 8-bit caches.  These calls take torch tensors
# and check their types, sizes and device before the library sees them; they
# run on the tensors' device, on its current stream unless one is given.


_T = None  # torch, once one of these calls needs it


def _torch():
    global _T
    if _T is None:
        import torch

        _T = torch
    return _T


def _refuse(where: str, what: str) -> None:
    raise FastGenError(FG_EINVAL, f"{where}: {what}")


def _heads(p: Params) -> tuple[int, int]:
    """Query and key/value head instances of the batch."""
    layers = p.B * p.L
    return layers * p.H, layers * (p.Hkv or p.H)


def _is(x, where: str, name: str, dtype, count: int, dev: int) -> int:
    """The address of tensor x, which must be contiguous, of that type, on
    device `dev` (-1: the CPU), with `count` elements."""
    if (x.dtype is not dtype or x.numel() != count or x.get_device() != dev
            or not x.is_contiguous()):
        _refuse(where, f"{name} must be contiguous, {count} elements of {dtype} on device {dev}; "
                       f"got {tuple(x.shape)} of {x.dtype} on {x.device}")
    return x.data_ptr()


def _id_set(x, where: str, name: str, dev: int):
    if x is None:
        return None, 0
    n = x.numel()
    return _is(x, where, name, _T.int32, n, dev), n


def _elem(p: Params):
    torch = _T or _torch()
    return torch.bfloat16 if p.dtype == FG_BF16 else torch.float32


class _Sizes:
    """What the checks of a call need of its parameters."""

    def __init__(self, p: Params):
        self.B, self.d, self.n, self.dt = p.B, p.d, p.n, _elem(p)
        self.G, self.Gkv = _heads(p)
        self.queries, self.rows = self.G * p.d, self.Gkv * p.d  # values of one row each


def _run(where: str, dev: int, stream, fn, *args) -> None:
    """Calls fn(*args, stream) with device `dev` current."""
    torch = _T or _torch()
    if dev < 0:
        _refuse(where, "tensors must be on a GPU")
    here = torch._C._cuda_getDevice()
    if stream is None:
        stream = torch._C._cuda_getCurrentRawStream(dev)
    elif not isinstance(stream, int):
        stream = stream.cuda_stream
    if dev == here:
        st = fn(*args, stream)
    else:
        with torch.cuda.device(dev):
            st = fn(*args, stream)
    if st != FG_OK:
        raise FastGenError(st, where)


class Rope:
    """A position rotation: turns [rot_dim / 2] int64 on the device (64-bit
    fractions of a turn per position, see fastgen_rope_table) and the pairing
    (FG_ROPE_INTERLEAVED or FG_ROPE_HALF)."""

    def __init__(self, turns, style: int = FG_ROPE_INTERLEAVED):
        torch = _torch()
        if turns.dtype != torch.int64 or not turns.is_contiguous():
            _refuse("Rope", "turns must be a contiguous int64 tensor")
        self.turns, self.dev = turns, turns.get_device()
        self.c = RopeStruct(turns.data_ptr(), 2 * turns.numel(), style)

    @classmethod
    def make(cls, rot_dim: int, base: float = 10000.0, style: int = FG_ROPE_INTERLEAVED,
             device="cuda", inv_freq=None):
        """inv_freq (radians per position, default base^(-2i/rot_dim))."""
        if inv_freq is None:
            inv_freq = [float(base) ** (-2.0 * i / rot_dim) for i in range(rot_dim // 2)]
        return cls(fastgen_rope_table(inv_freq).to(device), style)


def _rope(rope, where: str, dev: int):
    if rope is None:
        return None
    if rope.dev != dev:
        _refuse(where, f"rope must be on device {dev}")
    return rope.c


def fastgen_rope_table(inv_freq):
    """int64 CPU tensor of the turns per position of each frequency."""
    torch = _torch()
    f = torch.as_tensor(inv_freq, dtype=torch.float64).contiguous().cpu()
    out = torch.empty(f.numel(), dtype=torch.int64)
    _check(lib().fastgen_rope_table(f.data_ptr(), f.numel(), out.data_ptr()), "fastgen_rope_table")
    return out


def fastgen_rope(params, Q, K, pos, rope, Q_out, K_out, stream=None) -> None:
    """Rotates Q [G, n, d] and K [Gkv, n, d] at pos [B, n] (None: 0 .. n-1)."""
    w, p = "fastgen_rope", params
    G, Gkv = _heads(p)
    dt, size = _elem(p), p.n * p.d
    if rope is None or (Q is None and K is None):
        _refuse(w, "no rotation, or nothing to rotate")
    dev = (K if Q is None else Q).get_device()
    _run(w, dev, stream, lib().fastgen_rope, p,
         None if Q is None else _is(Q, w, "Q", dt, G * size, dev),
         None if K is None else _is(K, w, "K", dt, Gkv * size, dev),
         None if pos is None else _is(pos, w, "pos", _T.int32, p.B * p.n, dev),
         _rope(rope, w, dev),
         None if Q_out is None else _is(Q_out, w, "Q_out", dt, G * size, dev),
         None if K_out is None else _is(K_out, w, "K_out", dt, Gkv * size, dev))


def fastgen_paged_table_len(params, max_new_tokens: int) -> int:
    return lib().fastgen_paged_table_len(params, max_new_tokens)


def fastgen_paged_sched_bytes(params, table_len: int) -> int:
    return lib().fastgen_paged_sched_bytes(params, table_len)


class PagedCache:
    """The buffers of one batch of paged 8-bit caches (fg_paged_cache):
    k_pages, v_pages [n_pages, 64, d] float8_e4m3fn, exps [n_pages, 4, 2] int8, pos
    [n_pages, 64] int32, page_table int32, caches [Gkv, 6] int32, rows [Gkv]
    int32, next_page [1] int32, rows_out [Gkv] int32 (default: rows, in
    place).  The page buffers may be None until set_pages.  Holds the decode
    work list, which schedule or fastgen_paged_plan fills."""

    def __init__(self, params, k_pages, v_pages, exps, pos, page_table, caches, rows, next_page,
                 rows_out=None):
        torch, w = _torch(), "PagedCache"
        self.key, self.sizes = bytes(params), _Sizes(params)
        Gkv = self.sizes.Gkv
        dev, i32 = page_table.get_device(), torch.int32
        self.dev, self.d = dev, params.d
        c = self.c = PagedCacheStruct()
        c.table_len = page_table.numel()
        c.page_table = _is(page_table, w, "page_table", i32, page_table.numel(), dev)
        c.caches = _is(caches, w, "caches", i32, Gkv * 6, dev)
        c.rows = _is(rows, w, "rows", i32, Gkv, dev)
        c.next_page = _is(next_page, w, "next_page", i32, 1, dev)
        c.rows_out = c.rows if rows_out is None else _is(rows_out, w, "rows_out", i32, Gkv, dev)
        need = fastgen_paged_sched_bytes(params, c.table_len)
        if need == 0:
            _refuse(w, "parameters or table length")
        self.sched = torch.empty(need, dtype=torch.uint8, device=page_table.device)
        c.sched, c.sched_bytes = self.sched.data_ptr(), need
        self.page_table, self.caches, self.rows, self.next_page = page_table, caches, rows, next_page
        self.rows_out = rows if rows_out is None else rows_out
        self.k_pages = self.v_pages = self.exps = self.pos = None
        if k_pages is not None:
            self.set_pages(k_pages, v_pages, exps, pos)

    def set_pages(self, k_pages, v_pages, exps, pos) -> None:
        torch, w, c = _torch(), "PagedCache", self.c
        pages, row = exps.numel() // 8, FG_PAGE_ROWS * self.d
        codes = torch.uint8 if k_pages.dtype is torch.uint8 else torch.float8_e4m3fn
        c.k_pages = _is(k_pages, w, "k_pages", codes, pages * row, self.dev)
        c.v_pages = _is(v_pages, w, "v_pages", codes, pages * row, self.dev)
        c.exps = _is(exps, w, "exps", torch.int8, pages * 8, self.dev)
        c.pos = _is(pos, w, "pos", torch.int32, pages * FG_PAGE_ROWS, self.dev)
        c.n_pages = pages
        self.k_pages, self.v_pages, self.exps, self.pos = k_pages, v_pages, exps, pos

    def schedule(self, params, stream=None) -> None:
        fastgen_paged_schedule(params, self, stream)


def _of_cache(p: Params, cache, w: str):
    """The sizes of a call on `cache`, which must have been made for the same
    sequences, heads and head dim (other parameters may differ)."""
    if bytes(p) == cache.key:
        return cache.sizes
    z = _Sizes(p)
    if z.Gkv != cache.sizes.Gkv or z.B != cache.sizes.B or z.d != cache.d:
        _refuse(w, "the cache was made for other parameters")
    return z


def fastgen_paged_plan(params, policy, keep, max_new_tokens, cache, stream=None) -> PagedInfo:
    w, torch = "fastgen_paged_plan", _torch()
    z, dev, info = _of_cache(params, cache, w), cache.dev, PagedInfo()
    _run(w, dev, stream, lib().fastgen_paged_plan, params,
         _is(policy, w, "policy", torch.int8, z.G, dev),
         _is(keep, w, "keep", torch.uint8, z.G * z.n, dev), max_new_tokens, cache.c, info)
    return info


def fastgen_paged_schedule(params, cache, stream=None) -> None:
    w = "fastgen_paged_schedule"
    _of_cache(params, cache, w)
    _run(w, cache.dev, stream, lib().fastgen_paged_schedule, params, cache.c)


def fastgen_compact_q8(params, K, V, keep, cache, dev_err, stream=None) -> None:
    w, torch = "fastgen_compact_q8", _torch()
    z, dev = _of_cache(params, cache, w), cache.dev
    _run(w, dev, stream, lib().fastgen_compact_q8, params, _is(K, w, "K", z.dt, z.rows * z.n, dev),
         _is(V, w, "V", z.dt, z.rows * z.n, dev), _is(keep, w, "keep", torch.uint8, z.G * z.n, dev),
         cache.c, _is(dev_err, w, "dev_err", torch.int32, 1, dev))


def fastgen_append_q8_workspace_bytes(params, m: int) -> int:
    return lib().fastgen_append_q8_workspace_bytes(params, m)


def fastgen_append_q8(params, cache, k_new, v_new, new_ids, n_new, special_ids, punct_ids, pos,
                      rope, workspace, dev_err, stream=None) -> None:
    """Appends m tokens: k_new, v_new [Gkv, m, d], new_ids [B, m], n_new [B] or
    None (m each), pos [B] the first new position of each sequence (< 0: idle)."""
    w, torch = "fastgen_append_q8", _torch()
    z, dev, i32 = _of_cache(params, cache, w), cache.dev, torch.int32
    m, ws = new_ids.numel() // z.B, workspace.numel()
    special, n_special = _id_set(special_ids, w, "special_ids", dev)
    punct, n_punct = _id_set(punct_ids, w, "punct_ids", dev)
    _run(w, dev, stream, lib().fastgen_append_q8, params, cache.c,
         _is(k_new, w, "k_new", z.dt, z.rows * m, dev),
         _is(v_new, w, "v_new", z.dt, z.rows * m, dev),
         _is(new_ids, w, "new_ids", i32, z.B * m, dev), m,
         None if n_new is None else _is(n_new, w, "n_new", i32, z.B, dev), special, n_special,
         punct, n_punct, _is(pos, w, "pos", i32, z.B, dev), _rope(rope, w, dev),
         _is(workspace, w, "workspace", torch.uint8, ws, dev), ws,
         _is(dev_err, w, "dev_err", i32, 1, dev))


def fastgen_decode_q8_workspace_bytes(params, cache) -> int:
    return lib().fastgen_decode_q8_workspace_bytes(params, cache.c)


def fastgen_decode_attn_q8(params, cache, q, k_new, v_new, new_ids, special_ids, punct_ids, pos,
                           rope, out, workspace, dev_err, stream=None) -> None:
    """One generation step: q, out [G, d], k_new, v_new [Gkv, d] (None: nothing is
    appended), new_ids [B], pos [B] int32 on the device (< 0: idle)."""
    w, torch = "fastgen_decode_attn_q8", _torch()
    z, dev, i32, ws = _of_cache(params, cache, w), cache.dev, torch.int32, workspace.numel()
    special, n_special = _id_set(special_ids, w, "special_ids", dev)
    punct, n_punct = _id_set(punct_ids, w, "punct_ids", dev)
    _run(w, dev, stream, lib().fastgen_decode_attn_q8, params, cache.c,
         _is(q, w, "q", z.dt, z.queries, dev),
         None if k_new is None else _is(k_new, w, "k_new", z.dt, z.rows, dev),
         None if v_new is None else _is(v_new, w, "v_new", z.dt, z.rows, dev),
         None if new_ids is None else _is(new_ids, w, "new_ids", i32, z.B, dev), special,
         n_special, punct, n_punct, _is(pos, w, "pos", i32, z.B, dev), _rope(rope, w, dev),
         _is(out, w, "out", z.dt, z.queries, dev),
         _is(workspace, w, "workspace", torch.uint8, ws, dev), ws,
         _is(dev_err, w, "dev_err", i32, 1, dev))
