"""ctypes binding of librs_hip.so: the C-ABI calls under the same names.

Argument marshalling only (torch tensors -> device pointers and sizes, spec
lists -> C structs, the current HIP stream); every step of the layout
transform runs in the library. torch is imported before the library is
opened so that the library binds to the HIP runtime torch already loaded.
If the library is missing, load() raises: there is no fallback.
"""
from __future__ import annotations

import ctypes
import json
import os
from typing import List, NamedTuple, Optional, Sequence

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "librs_hip.so")

RS_OK, RS_EINVAL, RS_EPLAN, RS_EALIGN, RS_EDTYPE, RS_ENOMEM, RS_EHIP, RS_ERANGE = 0, -1, -2, -3, -4, -5, -6, -7
STATUS_NAMES = {0: "RS_OK", -1: "RS_EINVAL", -2: "RS_EPLAN", -3: "RS_EALIGN", -4: "RS_EDTYPE",
                -5: "RS_ENOMEM", -6: "RS_EHIP", -7: "RS_ERANGE"}
KINDS = {"ELEM": 0, "ROWS": 1, "TILE": 2, "FLAT": 3, "WHOLE": 4, "TILEMAJOR": 5}
ORDER_KINDS = {0: "default", 1: "by_block_size", 2: "by_shape"}
RS_F32, RS_BF16, RS_E4M3, RS_I8, RS_U8 = 0, 1, 2, 3, 4
CODE_FORMATS = {"e4m3": RS_E4M3, "i8": RS_I8, "u8": RS_U8}
EXPORTS = ("rs_plan_build", "rs_plan_load", "rs_plan_load_with", "rs_plan_info", "rs_plan_free", "rs_unpack_gathered",
           "rs_pack_scatter", "rs_block_quant", "rs_block_dequant", "rs_unpack_dequant", "rs_adam8_step",
           "rs_last_error", "rs_block_quant_noalloc", "rs_orthogonalize", "rs_muon_step", "rs_muon_workspace",
           "rs_embed_rows", "rs_embed_grad", "rs_embed_workspace")


class RsError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {message}")
        self.status = status


class AdamHParamsC(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_float), ("beta1", ctypes.c_float), ("beta2", ctypes.c_float),
                ("eps", ctypes.c_float), ("weight_decay", ctypes.c_float), ("reserved", ctypes.c_int32),
                ("step", ctypes.c_int64)]


class MuonHParamsC(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_float), ("momentum", ctypes.c_float), ("weight_decay", ctypes.c_float),
                ("eps", ctypes.c_float), ("steps", ctypes.c_int32), ("nesterov", ctypes.c_int32),
                ("scale_mode", ctypes.c_int32)]


class PlanOptionsC(ctypes.Structure):
    _fields_ = [("muon_parts", ctypes.c_int32), ("reserved", ctypes.c_int32 * 7)]


class TensorSpecC(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("cols", ctypes.c_int64), ("kind", ctypes.c_int32),
                ("reserved", ctypes.c_int32), ("p0", ctypes.c_int64), ("p1", ctypes.c_int64)]


_lib = None


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Open the HIP library (once). Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with structure_aware_grouped_amd.build "
                           "(there is no CPU fallback)")
    lib = ctypes.CDLL(path)
    P, I64, I32, F = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float
    PI64 = ctypes.POINTER(ctypes.c_int64)
    PI32 = ctypes.POINTER(ctypes.c_int32)
    lib.rs_plan_build.argtypes = [ctypes.POINTER(TensorSpecC), I64, I64, I64, I32, PI64, PI64, PI64, PI32]
    lib.rs_plan_load.argtypes = [ctypes.POINTER(TensorSpecC), I64, I64, I64, PI64, I64, I32,
                                 ctypes.POINTER(P)]
    lib.rs_plan_load_with.argtypes = [ctypes.POINTER(TensorSpecC), I64, I64, I64, PI64, I64, I32,
                                      ctypes.POINTER(PlanOptionsC), ctypes.POINTER(P)]
    lib.rs_plan_info.argtypes = [P, PI64, PI64, PI64]
    lib.rs_plan_free.argtypes = [P]
    lib.rs_plan_free.restype = None
    lib.rs_unpack_gathered.argtypes = [P, P, I32, ctypes.POINTER(P), P]
    lib.rs_pack_scatter.argtypes = [P, ctypes.POINTER(P), I32, P, P, I32, I32, F, P]
    lib.rs_block_quant.argtypes = [P, P, I32, P, I32, P, P]
    lib.rs_block_dequant.argtypes = [P, P, I32, P, P, P]
    lib.rs_unpack_dequant.argtypes = [P, P, I32, P, ctypes.POINTER(P), I32, P]
    lib.rs_adam8_step.argtypes = [P, P, P, P, P, P, P, ctypes.POINTER(AdamHParamsC), P]
    lib.rs_block_quant_noalloc.argtypes = [ctypes.POINTER(TensorSpecC), I64, I64, I64, PI64, I64, P, I32, P, I32,
                                           P, I64, P]
    PF = ctypes.POINTER(ctypes.c_float)
    lib.rs_orthogonalize.argtypes = [P, P, I32, P, PF, I32, F, P, I64, P]
    lib.rs_muon_step.argtypes = [P, P, P, I32, P, ctypes.POINTER(MuonHParamsC), PF, P, I64, P]
    lib.rs_muon_workspace.argtypes = [P, PI64]
    lib.rs_embed_rows.argtypes = [P, I64, P, I32, P, I32, I64, F, P, I32, P]
    lib.rs_embed_grad.argtypes = [P, I64, P, I32, I64, P, I32, P, P, I32, I32, F, P, I64, P]
    lib.rs_embed_workspace.argtypes = [P, I64, I64, PI64]
    lib.rs_last_error.argtypes = []
    lib.rs_last_error.restype = ctypes.c_char_p
    for name in EXPORTS:
        if name not in ("rs_plan_free", "rs_last_error"):
            getattr(lib, name).restype = ctypes.c_int
    _lib = lib
    return lib


def _check(status: int):
    if status != RS_OK:
        raise RsError(status, load().rs_last_error().decode())


def specs_array(specs) -> ctypes.Array:
    arr = (TensorSpecC * len(specs))()
    for i, s in enumerate(specs):
        arr[i].rows, arr[i].cols = int(s.rows), int(s.cols)
        arr[i].kind = KINDS[s.kind] if isinstance(s.kind, str) else int(s.kind)
        arr[i].reserved = 0
        arr[i].p0, arr[i].p1 = int(getattr(s, "p0", 0)), int(getattr(s, "p1", 0))
    return arr


def _i64(values) -> ctypes.Array:
    return (ctypes.c_int64 * len(values))(*[int(v) for v in values])


def _ptrs(tensors) -> ctypes.Array:
    return (ctypes.c_void_p * len(tensors))(*[t.data_ptr() for t in tensors])


def _stream(device) -> ctypes.c_void_p:
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _copy_code(t: torch.Tensor) -> int:
    """Unpack copies bits: only the element size matters (4, 2 or 1 bytes)."""
    code = {4: RS_F32, 2: RS_BF16, 1: RS_U8}.get(t.element_size())
    if code is None:
        raise TypeError(f"unsupported element size {t.element_size()}")
    return code


# ---------------------------------------------------------------- planner

def rs_plan_build(specs, V: int, align: int = 16, policy: str = "best"):
    """(S, starts, order, order_name) from the host planner. policy: "best" (the three orders),
    or one order: "default", "by_block_size", "by_shape"."""
    lib = load()
    n = len(specs)
    S = ctypes.c_int64()
    starts = (ctypes.c_int64 * n)()
    order = (ctypes.c_int64 * n)()
    kind = ctypes.c_int32()
    pol = {"best": 0, "default": 1, "by_block_size": 2, "by_shape": 3}[policy]
    _check(lib.rs_plan_build(specs_array(specs), n, int(V), int(align), pol, ctypes.byref(S),
                             starts, order, ctypes.byref(kind)))
    return S.value, list(starts), list(order), ORDER_KINDS[kind.value]


# ---------------------------------------------------------------- plans as data

PLAN_FORMAT = "rs-plan/1"


class PlanSpec(NamedTuple):
    """One tensor of a plan read back from JSON (the fields rs_plan_load reads)."""
    name: str
    rows: int
    cols: int
    kind: str
    p0: int = 0
    p1: int = 0

    @property
    def numel(self) -> int:
        return self.rows * self.cols


def plan_to_json(specs, V: int, S: int, starts: Sequence[int], R_mat: Optional[int] = None) -> str:
    """A plan as JSON. A plan is pure data: the tensors (shape and atomic block),
    V, S, the starts and the materialised ranks. rs_plan_load validates it again
    and rebuilds the same device work lists from it, so a saved plan resumes a
    group without planning again."""
    kinds = {v: k for k, v in KINDS.items()}
    out = []
    for i, sp in enumerate(specs):
        kind = sp.kind if isinstance(sp.kind, str) else kinds[int(sp.kind)]
        out.append({"name": str(getattr(sp, "name", f"t{i}")), "rows": int(sp.rows), "cols": int(sp.cols),
                    "kind": kind, "p0": int(getattr(sp, "p0", 0)), "p1": int(getattr(sp, "p1", 0))})
    return json.dumps({"format": PLAN_FORMAT, "V": int(V), "S": int(S), "R_mat": int(V if R_mat is None else R_mat),
                       "starts": [int(x) for x in starts], "tensors": out})


def plan_from_json(text: str):
    """(specs, V, S, starts, R_mat) from plan_to_json's output; checks the format
    and the field types only (validation is rs_plan_load's)."""
    d = json.loads(text)
    if d.get("format") != PLAN_FORMAT:
        raise ValueError(f"not an {PLAN_FORMAT} plan: format {d.get('format')!r}")
    specs = []
    for t in d["tensors"]:
        if t["kind"] not in KINDS:
            raise ValueError(f"unknown block kind {t['kind']!r}")
        specs.append(PlanSpec(str(t["name"]), int(t["rows"]), int(t["cols"]), t["kind"], int(t["p0"]), int(t["p1"])))
    starts = [int(x) for x in d["starts"]]
    if len(starts) != len(specs):
        raise ValueError(f"{len(starts)} starts for {len(specs)} tensors")
    return specs, int(d["V"]), int(d["S"]), starts, int(d["R_mat"])


class Plan:
    """A loaded plan (device work lists); freed with close() or when collected."""

    def __init__(self, handle, specs, V, S, starts, R_mat, device):
        self._h = handle
        self.specs, self.V, self.S, self.starts = list(specs), V, S, list(starts)
        self.R_mat, self.device = R_mat, device
        r, q, pad = ctypes.c_int64(), ctypes.c_int64(), ctypes.c_int64()
        _check(load().rs_plan_info(handle, ctypes.byref(r), ctypes.byref(q), ctypes.byref(pad)))
        self.R_used, self.n_qblocks, self.padding = r.value, q.value, pad.value
        self.numels = [int(s.rows) * int(s.cols) for s in specs]

    def to_json(self) -> str:
        return plan_to_json(self.specs, self.V, self.S, self.starts, self.R_mat)

    @property
    def handle(self):
        if self._h is None:
            raise RuntimeError("plan already freed")
        return self._h

    def close(self):
        if self._h is not None:
            load().rs_plan_free(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def rs_plan_load(specs, V: int, S: int, starts: Sequence[int], R_mat: Optional[int] = None,
                 device: int = 0, muon_parts: int = 1) -> Plan:
    """Validate a plan and build its work lists on `device`. muon_parts: fp16 parts of the operands
    of rs_orthogonalize and rs_muon_step; 2 brings their results as near as fp32 products', at
    1.4 to 2.9 times the time and up to 1.7 times the workspace (an option of the loaded plan: a
    plan's JSON does not hold it)."""
    lib = load()
    n = len(specs)
    if R_mat is None:
        R_mat = V
    h = ctypes.c_void_p()
    options = PlanOptionsC(muon_parts=int(muon_parts))
    _check(lib.rs_plan_load_with(specs_array(specs), n, int(V), int(S), _i64(starts), int(R_mat),
                                 int(device), ctypes.byref(options), ctypes.byref(h)))
    return Plan(h, specs, int(V), int(S), starts, int(R_mat), int(device))


# ---------------------------------------------------------------- transforms

def _count_check(plan: Plan, items, what: str):
    """The C calls read exactly one pointer per tensor of the plan."""
    if len(items) != len(plan.numels):
        raise ValueError(f"{what}: {len(items)} entries for a plan of {len(plan.numels)} tensors")


def _scales_check(plan: Plan, scales: torch.Tensor):
    """The kernels read n_qblocks fp32 scales: a tensor of another dtype with that many
    entries would be read past its end."""
    if scales.dtype != torch.float32 or scales.numel() < plan.n_qblocks:
        raise ValueError("scales: fp32 with n_qblocks entries")


def _dev_check(plan: Plan, *tensors):
    for t in tensors:
        if t is None:
            continue
        if t.device.type != "cuda" or t.device.index != plan.device:
            raise ValueError(f"tensor on {t.device}, plan on cuda:{plan.device}")
        if not t.is_contiguous():
            raise ValueError("tensors must be contiguous")


def rs_unpack_gathered(plan: Plan, gathered: torch.Tensor, dsts: List[torch.Tensor]):
    """dst_i <- gathered[s_i : s_i + n_i] for every tensor (same dtype)."""
    _count_check(plan, dsts, "dsts")
    _dev_check(plan, gathered, *dsts)
    if gathered.numel() < plan.R_mat * plan.S:
        raise ValueError("gathered buffer shorter than R_mat * S")
    for d, n in zip(dsts, plan.numels):
        if d.numel() != n or d.dtype != gathered.dtype:
            raise ValueError("destination size or dtype does not match its tensor")
    _check(load().rs_unpack_gathered(plan.handle, gathered.data_ptr(), _copy_code(gathered),
                                     _ptrs(dsts), _stream(plan.device)))


def rs_pack_scatter(plan: Plan, srcs: List[torch.Tensor], packed: torch.Tensor,
                    prev: Optional[torch.Tensor] = None, scale: Optional[float] = None):
    """packed <- [prev +] src * sigma on tensors, +0.0 on padding; sigma = fl32(1/V) unless given.
    packed is fp32, or bf16 (each fp32 result rounded once to nearest even); prev is fp32."""
    _count_check(plan, srcs, "srcs")
    if srcs[0].dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("sources are fp32 or bf16")
    _dev_check(plan, packed, prev, *srcs)
    if packed.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("packed is fp32 or bf16")
    if prev is not None and prev.dtype != torch.float32:
        raise ValueError("prev is fp32")
    if packed.numel() < plan.R_mat * plan.S or (prev is not None and prev.numel() < plan.R_mat * plan.S):
        raise ValueError("packed / prev shorter than R_mat * S")
    dt = srcs[0].dtype
    for s, n in zip(srcs, plan.numels):
        if s.numel() != n or s.dtype != dt:
            raise ValueError("source size or dtype does not match its tensor")
    mode, val = (0, 0.0) if scale is None else (1, float(scale))
    _check(load().rs_pack_scatter(plan.handle, _ptrs(srcs), RS_F32 if dt == torch.float32 else RS_BF16,
                                  prev.data_ptr() if prev is not None else None, packed.data_ptr(),
                                  RS_F32 if packed.dtype == torch.float32 else RS_BF16,
                                  mode, ctypes.c_float(val), _stream(plan.device)))


def rs_block_quant(plan: Plan, src: torch.Tensor, q: torch.Tensor, fmt: str, scales: torch.Tensor):
    """Per-block absmax codes (fmt "e4m3" | "i8" | "u8") of the flat buffer, plus fp32 scales."""
    _scales_check(plan, scales)
    _dev_check(plan, src, q, scales)
    if src.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("src is fp32 or bf16")
    if src.numel() < plan.R_mat * plan.S or q.numel() * q.element_size() < plan.R_mat * plan.S:
        raise ValueError("src / q shorter than R_mat * S")
    _check(load().rs_block_quant(plan.handle, src.data_ptr(),
                                 RS_F32 if src.dtype == torch.float32 else RS_BF16, q.data_ptr(),
                                 CODE_FORMATS[fmt], scales.data_ptr(), _stream(plan.device)))


def rs_block_dequant(plan: Plan, q: torch.Tensor, fmt: str, scales: torch.Tensor, out: torch.Tensor):
    """out <- code value * block scale inside blocks, +0.0 elsewhere."""
    _scales_check(plan, scales)
    _dev_check(plan, q, scales, out)
    if out.dtype != torch.float32 or out.numel() < plan.R_mat * plan.S:
        raise ValueError("out: fp32 with R_mat * S entries")
    if q.numel() * q.element_size() < plan.R_mat * plan.S or scales.numel() < plan.n_qblocks:
        raise ValueError("q / scales too short")
    _check(load().rs_block_dequant(plan.handle, q.data_ptr(), CODE_FORMATS[fmt], scales.data_ptr(),
                                   out.data_ptr(), _stream(plan.device)))


def rs_unpack_dequant(plan: Plan, q: torch.Tensor, fmt: str, scales: torch.Tensor,
                      dsts: List[Optional[torch.Tensor]]):
    """dst_i <- fl32(code value * block scale) (rounded to bf16 for bf16 tensors) for every
    quantised tensor; entries for other tensors may be None."""
    _scales_check(plan, scales)
    _count_check(plan, dsts, "dsts")
    _dev_check(plan, q, scales, *[d for d in dsts if d is not None])
    if q.numel() * q.element_size() < plan.R_mat * plan.S or scales.numel() < plan.n_qblocks:
        raise ValueError("q / scales too short")
    dt = None
    for d, n, sp in zip(dsts, plan.numels, plan.specs):
        if d is None:
            continue
        if d.numel() != n or d.dtype not in (torch.float32, torch.bfloat16):
            raise ValueError("destination size or dtype does not match its tensor")
        if dt is not None and d.dtype != dt:
            raise ValueError("destinations share one dtype")
        dt = d.dtype
    ptrs = (ctypes.c_void_p * len(dsts))(*[d.data_ptr() if d is not None else None for d in dsts])
    _check(load().rs_unpack_dequant(plan.handle, q.data_ptr(), CODE_FORMATS[fmt], scales.data_ptr(), ptrs,
                                    RS_BF16 if dt == torch.bfloat16 else RS_F32, _stream(plan.device)))


def rs_adam8_step(plan: Plan, param: torch.Tensor, grad: torch.Tensor, q_m: torch.Tensor,
                  s_m: torch.Tensor, q_v: torch.Tensor, s_v: torch.Tensor, lr: float, beta1: float,
                  beta2: float, eps: float, weight_decay: float, step: int):
    """One AdamW step on every quantisation block, in place: param (fp32 flat), int8 m codes and
    scales, uint8 v codes and scales; grad is the packed fp32 gradient."""
    _dev_check(plan, param, grad, q_m, s_m, q_v, s_v)
    total = plan.R_mat * plan.S
    for t, dt in ((param, torch.float32), (grad, torch.float32), (s_m, torch.float32), (s_v, torch.float32)):
        if t.dtype != dt:
            raise ValueError("param, grad and scales are fp32")
    if param.numel() < total or grad.numel() < total or q_m.numel() < total or q_v.numel() < total:
        raise ValueError("buffers shorter than R_mat * S")
    if s_m.numel() < plan.n_qblocks or s_v.numel() < plan.n_qblocks:
        raise ValueError("scales shorter than n_qblocks")
    hp = AdamHParamsC(lr, beta1, beta2, eps, weight_decay, 0, int(step))
    _check(load().rs_adam8_step(plan.handle, param.data_ptr(), grad.data_ptr(), q_m.data_ptr(), s_m.data_ptr(),
                                q_v.data_ptr(), s_v.data_ptr(), ctypes.byref(hp), _stream(plan.device)))


# ---------------------------------------------------------------- embeddings

def _table(plan: Plan, tensor: int, ids: torch.Tensor, rows: torch.Tensor, what: str):
    """(tokens) of an embedding call: ids are int32 or int64, `rows` holds one row per id."""
    if not 0 <= int(tensor) < len(plan.specs):
        raise ValueError(f"no tensor {tensor} in a plan of {len(plan.specs)}")
    if ids.dtype not in (torch.int32, torch.int64):
        raise ValueError("ids: int32 or int64")
    if rows.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError(f"{what}: fp32 or bf16")
    if rows.numel() != ids.numel() * int(plan.specs[tensor].cols):
        raise ValueError(f"{what}: one row of {plan.specs[tensor].cols} columns per id")
    return ids.numel()


def _code(t: torch.Tensor) -> int:
    return RS_F32 if t.dtype == torch.float32 else RS_BF16


def _embed_bytes(plan: Plan, tensor: int, n_ids: int) -> int:
    n = ctypes.c_int64()
    _check(load().rs_embed_workspace(plan.handle, int(tensor), int(n_ids), ctypes.byref(n)))
    return n.value


def rs_embed_workspace(plan: Plan, tensor: int, n_ids: int) -> torch.Tensor:
    """Workspace for rs_embed_grad with up to n_ids tokens (uint8, on the plan's device). Calls
    that may overlap need a workspace each."""
    return torch.empty(max(_embed_bytes(plan, tensor, n_ids), 1), dtype=torch.uint8, device=f"cuda:{plan.device}")


def rs_embed_rows(plan: Plan, tensor: int, gathered: torch.Tensor, ids: torch.Tensor, out: torch.Tensor,
                  scale: float = 1.0):
    """out[t] <- scale * row ids[t] of tensor number `tensor` of the gathered flat buffer (fp32 or
    bf16); ids outside [0, rows) give rows of +0.0."""
    n = _table(plan, tensor, ids, out, "out")
    _dev_check(plan, gathered, ids, out)
    _flat_check(plan, gathered, (torch.float32, torch.bfloat16), "gathered")
    _apart_check(gathered=gathered, out=out, ids=ids)
    _check(load().rs_embed_rows(plan.handle, int(tensor), gathered.data_ptr(), _code(gathered), ids.data_ptr(),
                                ids.element_size(), n, float(scale), out.data_ptr(), _code(out),
                                _stream(plan.device)))


def rs_embed_grad(plan: Plan, tensor: int, ids: torch.Tensor, dy: torch.Tensor, packed: torch.Tensor,
                  work: torch.Tensor, prev: Optional[torch.Tensor] = None, scale: float = 1.0, inv_v: bool = False):
    """Tensor number `tensor`'s interval of packed <- [prev +] sigma * the sum of dy's rows by id,
    sigma = scale, or scale / V with inv_v. prev=packed (fp32) adds in place to the named rows."""
    n = _table(plan, tensor, ids, dy, "dy")
    _dev_check(plan, ids, dy, packed, work, prev)
    _flat_check(plan, packed, (torch.float32, torch.bfloat16), "packed")
    if work.dtype != torch.uint8:      # its size is checked by the call itself
        raise ValueError("work: uint8")
    apart = {"ids": ids, "dy": dy, "packed": packed, "work": work}
    if prev is not None:
        _flat_check(plan, prev, (torch.float32,), "prev")
        if prev.data_ptr() != packed.data_ptr() or packed.dtype != torch.float32:
            apart["prev"] = prev
    _apart_check(**apart)
    _check(load().rs_embed_grad(plan.handle, int(tensor), ids.data_ptr(), ids.element_size(), n, dy.data_ptr(),
                                _code(dy), prev.data_ptr() if prev is not None else None, packed.data_ptr(),
                                _code(packed), 0 if inv_v else 1, float(scale), work.data_ptr(), work.numel(),
                                _stream(plan.device)))


# ---------------------------------------------------------------- whole matrices

# a, b, c of the quintic of the published Muon optimiser: singular values in (0, 1] go to
# about [0.7, 1.2] in five steps
MUON_COEFFS = (3.4445, -4.7750, 2.0315)
UPDATE_SCALES = {"none": 0, "spectral": 1, "rms": 2}


def _coeffs(coeffs, steps: int) -> ctypes.Array:
    """3 * steps floats: one (a, b, c) for every step, or a sequence of one per step."""
    rows = list(coeffs)
    if rows and not hasattr(rows[0], "__len__"):
        rows = [rows] * int(steps)
    if len(rows) != int(steps) or any(len(r) != 3 for r in rows):
        raise ValueError("coeffs: (a, b, c), or one (a, b, c) per step")
    flat = [float(v) for r in rows for v in r]
    return (ctypes.c_float * max(len(flat), 1))(*flat)


def _flat_check(plan: Plan, t: torch.Tensor, dtypes, what: str):
    if t.dtype not in dtypes:
        raise ValueError(f"{what}: dtype {t.dtype}, expected one of {[str(d) for d in dtypes]}")
    if t.numel() < plan.R_mat * plan.S:
        raise ValueError(f"{what} shorter than R_mat * S")


def _apart_check(**tensors: torch.Tensor):
    """The named buffers share no byte: the kernels read some while they write others."""
    spans = []
    for name, t in tensors.items():
        size = t.nbytes
        if size:
            at = t.data_ptr()
            spans.append((at, at + size, name))
    spans.sort()
    for k in range(1, len(spans)):
        if spans[k][0] < spans[k - 1][1]:
            raise ValueError(f"{spans[k - 1][2]} and {spans[k][2]} overlap")


def _work_check(work: torch.Tensor, need: int):
    if work.dtype != torch.uint8 or work.numel() < need:
        raise ValueError(f"work: uint8 with at least {need} entries")


def _muon_bytes(plan: Plan) -> int:
    n = ctypes.c_int64()
    _check(load().rs_muon_workspace(plan.handle, ctypes.byref(n)))
    return n.value


def rs_muon_workspace(plan: Plan) -> torch.Tensor:
    """Workspace for rs_orthogonalize and rs_muon_step on this plan (uint8, on the plan's
    device). Calls that may overlap need a workspace each."""
    return torch.empty(max(_muon_bytes(plan), 1), dtype=torch.uint8, device=f"cuda:{plan.device}")


def rs_orthogonalize(plan: Plan, src: torch.Tensor, out: torch.Tensor, work: torch.Tensor,
                     coeffs=MUON_COEFFS, steps: int = 5, eps: float = 1e-7):
    """out <- the Newton-Schulz orthogonalisation of every WHOLE matrix of the flat buffer src
    (fp32 or bf16), in bf16; the rest of out is left as it is."""
    _dev_check(plan, src, out, work)
    _flat_check(plan, src, (torch.float32, torch.bfloat16), "src")
    _flat_check(plan, out, (torch.bfloat16,), "out")
    _work_check(work, _muon_bytes(plan))
    _apart_check(src=src, out=out, work=work)
    _check(load().rs_orthogonalize(plan.handle, src.data_ptr(), RS_F32 if src.dtype == torch.float32 else RS_BF16,
                                   out.data_ptr(), _coeffs(coeffs, steps), int(steps), float(eps), work.data_ptr(),
                                   work.numel(), _stream(plan.device)))


def rs_muon_step(plan: Plan, param: torch.Tensor, grad: torch.Tensor, momentum: torch.Tensor, work: torch.Tensor,
                 lr: float, momentum_decay: float = 0.95, weight_decay: float = 0.0, nesterov: bool = True,
                 update_scale: str = "rms", coeffs=MUON_COEFFS, steps: int = 5, eps: float = 1e-7):
    """One Muon step on every WHOLE matrix, in place: param and momentum (fp32 flat) with the
    packed gradient (fp32 or bf16). update_scale: "none", "spectral" (sqrt(max(1, rows/cols)))
    or "rms" (0.2 sqrt(max(rows, cols)))."""
    _dev_check(plan, param, grad, momentum, work)
    _flat_check(plan, param, (torch.float32,), "param")
    _flat_check(plan, momentum, (torch.float32,), "momentum")
    _flat_check(plan, grad, (torch.float32, torch.bfloat16), "grad")
    _work_check(work, _muon_bytes(plan))
    _apart_check(param=param, grad=grad, momentum=momentum, work=work)
    if update_scale not in UPDATE_SCALES:
        raise ValueError(f"update_scale: one of {sorted(UPDATE_SCALES)}")
    hp = MuonHParamsC(lr, momentum_decay, weight_decay, eps, int(steps), int(bool(nesterov)),
                      UPDATE_SCALES[update_scale])
    _check(load().rs_muon_step(plan.handle, param.data_ptr(), grad.data_ptr(),
                               RS_F32 if grad.dtype == torch.float32 else RS_BF16, momentum.data_ptr(),
                               ctypes.byref(hp), _coeffs(coeffs, steps), work.data_ptr(), work.numel(),
                               _stream(plan.device)))


def rs_block_quant_noalloc(specs, V: int, S: int, starts: Sequence[int], R_mat: int, src: torch.Tensor,
                           q: torch.Tensor, fmt: str, scales: torch.Tensor):
    """rs_block_quant without a loaded plan and without any allocation on the device: the
    plan is passed as data and its work list goes into the library's static device memory
    (calls that overlap on one GPU race; calls in order on one stream do not)."""
    if src.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("src is fp32 or bf16")
    if scales.dtype != torch.float32:
        raise ValueError("scales: fp32")
    for t in (src, q, scales):
        if t.device.type != "cuda" or not t.is_contiguous():
            raise ValueError("src, q and scales are contiguous device tensors")
    if src.numel() < R_mat * S or q.numel() * q.element_size() < R_mat * S:
        raise ValueError("src / q shorter than R_mat * S")
    _check(load().rs_block_quant_noalloc(specs_array(specs), len(specs), int(V), int(S), _i64(starts), int(R_mat),
                                         src.data_ptr(), RS_F32 if src.dtype == torch.float32 else RS_BF16,
                                         q.data_ptr(), CODE_FORMATS[fmt], scales.data_ptr(), scales.numel(),
                                         _stream(src.device)))
