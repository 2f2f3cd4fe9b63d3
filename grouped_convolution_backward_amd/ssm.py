"""The short causal convolution and the selective scan of libwgrad.so (C ABI:
include/wgrad_ssm.h), for MI355X (gfx950).

Plans are made from a problem dict and used any number of times, from several
threads and streams; outputs, states and workspaces are the caller's:

    conv = CausalConvPlan({"dtype": "bf16", "N": 4, "L": 2048, "C": 4096, "W": 4, "activation": "silu"})
    conv.run(x, w, y, bias=b)                                      # whole sequences
    conv.run_backward(x, w, dy, dx, dw, dbias=db, bias=b, ws=conv.new_workspace())
    conv.run_step(x1, w, state, y1, bias=b, slots=slots)           # one token per row

    scan = ScanPlan({"dtype": "bf16", "N": 4, "L": 2048, "C": 4096, "S": 16, "G": 1, "softplus": True})
    scan.run(x, delta, A, B, C, y, D=D, z=z, delta_bias=bias, saved=saved, ws=ws)
    scan.run_backward(x, delta, A, B, C, dy, saved, dx=..., ddelta=..., dA=..., dB=..., dC=..., ws=ws)
    scan.run_step(x1, delta1, A, B1, C1, state, y1, D=D, z=z1, delta_bias=bias, slots=slots)

Problem keys: dtype ("bf16", "fp16", "fp32"), N sequences, L rows per sequence
(packed: at most), C channels; packed (False) with T rows in all, whose runs
take seq_start, an int32 GPU tensor of N + 1; W and activation ("none",
"silu") of a convolution; S states, G groups (1) and softplus (True) of a
scan. Activations are [N, L, C] or [T, C] (B and C: [..., G, S] or, for one
group, [..., S]); rows may have a stride, as the halves of a wider matrix do,
elements of a row are adjacent. Neighbouring axes may be merged or split, and
axes of 1 added. A tensor that does not fit is a ValueError, what the library
refuses a WgradError.
"""

from __future__ import annotations

import ctypes
import struct

ACTIVATIONS = {"none": 0, "silu": 1}
_vp, _i32, _i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64


class wgrad_rows(ctypes.Structure):
    _fields_ = [("ptr", _vp), ("stride", _i64)]


class wgrad_cconv_problem(ctypes.Structure):
    _fields_ = [("dtype", _i32), ("activation", _i32), ("W", _i32), ("packed", _i32),
                ("N", _i64), ("L", _i64), ("T", _i64), ("C", _i64)]


class wgrad_cconv_args(ctypes.Structure):
    _fields_ = [("x", wgrad_rows), ("y", wgrad_rows), ("dy", wgrad_rows), ("dx", wgrad_rows),
                ("w", _vp), ("bias", _vp), ("init_state", _vp), ("final_state", _vp), ("seq_start", _vp),
                ("dw", _vp), ("dbias", _vp), ("dfinal_state", _vp), ("dinit_state", _vp), ("state", _vp), ("slots", _vp),
                ("rows", _i64), ("num_slots", _i64), ("ws", _vp), ("ws_bytes", ctypes.c_size_t)]


class wgrad_scan_problem(ctypes.Structure):
    _fields_ = [("dtype", _i32), ("softplus", _i32), ("packed", _i32), ("reserved", _i32),
                ("N", _i64), ("L", _i64), ("T", _i64), ("C", _i64), ("G", _i64), ("S", _i64)]


class wgrad_scan_args(ctypes.Structure):
    _fields_ = [(k, wgrad_rows) for k in ("x", "delta", "B", "C", "z", "y")] + [
        ("A", _vp), ("D", _vp), ("delta_bias", _vp), ("init_state", _vp), ("final_state", _vp), ("seq_start", _vp),
        ("saved", _vp)] + [(k, wgrad_rows) for k in ("dy", "dx", "ddelta", "dB", "dC", "dz")] + [
        ("dA", _vp), ("dD", _vp), ("ddelta_bias", _vp), ("dfinal_state", _vp), ("dinit_state", _vp), ("state", _vp),
        ("slots", _vp), ("rows", _i64), ("num_slots", _i64), ("ws", _vp), ("ws_bytes", ctypes.c_size_t)]


def _layout(cls):
    """The 8-byte words of an argument block by name ("x" of a wgrad_rows is its pointer and "x.stride" the next word), and
    their packer: a call's block is built in one go from its operands, which takes a fraction of the time of setting the
    fields of a ctypes structure one by one."""
    at = {}
    for name, t in cls._fields_:
        off = getattr(cls, name).offset
        at[name] = off // 8
        if t is wgrad_rows:
            at[name + ".stride"] = off // 8 + 1
    return at, struct.Struct(f"={ctypes.sizeof(cls) // 8}q")


class wgrad_scan_plan_info(ctypes.Structure):
    _fields_ = [("lanes", _i32), ("states_per_lane", _i32), ("segments", _i32), ("segments_backward", _i32),
                ("segment_rows", _i64), ("segment_rows_backward", _i64), ("chunk_rows", _i64),
                ("workspace_bytes", _i64), ("workspace_bytes_backward", _i64), ("saved_bytes", _i64)]


class wgrad_scan_overrides(ctypes.Structure):
    _fields_ = [("segments", _i32), ("segments_backward", _i32)]


# every symbol include/wgrad_ssm.h declares
SSM_EXPORTS = ("wgrad_cconv_plan", "wgrad_cconv_plan_destroy", "wgrad_cconv_workspace_bytes", "wgrad_cconv_run",
               "wgrad_cconv_backward_run", "wgrad_cconv_step_run", "wgrad_scan_plan", "wgrad_scan_plan_destroy",
               "wgrad_scan_plan_query", "wgrad_scan_workspace_bytes", "wgrad_scan_saved_bytes", "wgrad_scan_run",
               "wgrad_scan_backward_run", "wgrad_scan_step_run")


def declare(lib):
    """Argument and result types of the entry points."""
    P = ctypes.POINTER
    for op, prob, args in (("cconv", wgrad_cconv_problem, wgrad_cconv_args), ("scan", wgrad_scan_problem, wgrad_scan_args)):
        create, destroy = getattr(lib, f"wgrad_{op}_plan"), getattr(lib, f"wgrad_{op}_plan_destroy")
        create.argtypes = [P(prob), ctypes.c_int, P(_vp)]
        if op == "scan":
            create.argtypes = [P(prob), P(wgrad_scan_overrides), ctypes.c_int, P(_vp)]
        create.restype = ctypes.c_int
        destroy.argtypes, destroy.restype = [_vp], None
        for what in ("run", "backward_run", "step_run"):
            f = getattr(lib, f"wgrad_{op}_{what}")
            f.argtypes, f.restype = [_vp, _vp, _vp], ctypes.c_int   # the block: bytes or a pointer to a structure
    lib.wgrad_cconv_workspace_bytes.argtypes, lib.wgrad_cconv_workspace_bytes.restype = [_vp], ctypes.c_size_t
    lib.wgrad_scan_workspace_bytes.argtypes = [_vp, ctypes.c_int]
    lib.wgrad_scan_workspace_bytes.restype = ctypes.c_size_t
    lib.wgrad_scan_saved_bytes.argtypes, lib.wgrad_scan_saved_bytes.restype = [_vp], ctypes.c_size_t
    lib.wgrad_scan_plan_query.argtypes, lib.wgrad_scan_plan_query.restype = [_vp, P(wgrad_scan_plan_info)], ctypes.c_int


def _same_order(shape, want):
    """Whether a tensor of `shape` holds the elements of one of shape `want` in the same order: its axes, or some of them
    merged, or split, wherever axes of 1 stand. Then the ends of the one's axes are among the ends of the other's."""
    def ends(dims):
        n, at = 1, set()
        for v in dims:
            n *= v
            at.add(n)
        return n, at - {1}
    (n, a), (m, b) = ends(shape), ends(want)
    return n == m and (n == 0 or a <= b or b <= a)


class _Form:
    """The shape that an operand has to have, and the shapes that have been found to hold it."""

    __slots__ = ("shape", "rows", "width", "known")

    def __init__(self, *shape, rows=None):
        self.shape, self.known = shape, set()
        self.rows = rows
        if rows is not None:                                # a row operand: `rows` rows of `width` elements
            self.width = 1
            for v in shape:
                self.width *= v
            self.width = self.width // rows if rows else 0


def _gcb():
    import grouped_convolution_backward_amd as gcb
    return gcb


def _torch_dtype(name):
    import torch
    return {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}[name]


class _SsmPlan:
    """What both plans share: the handle, the checks of tensors, the call."""

    _op = ""

    def __init__(self, problem, hip_device):
        import torch
        gcb = _gcb()
        self._lib = gcb.load_library()
        self.problem = dict(problem)
        if hip_device is None:
            hip_device = torch.cuda.current_device()
        self._torch = torch
        self._check_rc = gcb._check
        p = self._struct = self._problem(gcb, problem)
        self.handle = _vp()
        self._check_rc(self._create(p, int(hip_device)))
        self.dtype = _torch_dtype(problem["dtype"])
        self.rows = int(p.T) if p.packed else int(p.N * p.L)
        self._run = getattr(self._lib, f"wgrad_{self._op}_run")
        self._backward_run = getattr(self._lib, f"wgrad_{self._op}_backward_run")
        self._step_run = getattr(self._lib, f"wgrad_{self._op}_step_run")
        # the current stream's handle without a Stream object around it, where this torch offers that
        self._raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
            lambda dev: torch.cuda.current_stream(dev).cuda_stream)
        # the current device's number, likewise without the check that the GPU is initialised: operands are on it
        self._current = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
        self._strides = {}          # row stride by (shape, strides, row width) of strided operands
        self._step_forms = {}       # forms of a step's operands by (rows, states)

    def close(self):
        if getattr(self, "handle", None) is not None and self.handle.value:
            getattr(self._lib, f"wgrad_{self._op}_plan_destroy")(self.handle)
            self.handle = _vp()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    # -- operands, as words of the argument block w
    def _block(self, x):
        """An empty block and the device that every operand has to be on: x's, which has to be the current one."""
        dev = x.get_device()
        if dev < 0 or dev != self._current():
            raise ValueError(f"x: need a tensor on the current GPU (got one on {x.device})")
        return [0] * self._words, dev

    def _look(self, name, t, form, dtype, dev):
        """t is not known to fit `form`: a ValueError, or its shape is known from now on."""
        if t.dtype is not dtype or t.get_device() != dev or not _same_order(t.shape, form.shape):
            raise ValueError(f"{name}: need a {dtype} tensor of shape {form.shape} on cuda:{dev}, the current device (got "
                             f"{t.dtype}, {tuple(t.shape)} on {t.device})")
        if len(form.known) >= 16:
            form.known.clear()
        form.known.add(t.shape)

    def _rows_of(self, w, dev, name, t, form):
        """A row operand: rows of adjacent elements at one distance."""
        if t.dtype is not self.dtype or t.shape not in form.known or t.get_device() != dev:
            self._look(name, t, form, self.dtype, dev)
        i = self._at[name]
        w[i] = t.data_ptr()
        width = form.width
        if t.is_contiguous() or form.rows == 0:
            w[i + 1] = width
            return
        key = (t.shape, t.stride(), width)
        step = self._strides.get(key)
        if step is None:
            step = self._row_stride(name, *key)
            if len(self._strides) >= 64:
                self._strides.clear()
            self._strides[key] = step
        w[i + 1] = step

    @staticmethod
    def _row_stride(name, shape, stride, width):
        need, k = 1, len(shape) - 1
        while k >= 0 and need < width:                   # the row's own axes
            if shape[k] != 1 and stride[k] != need:
                raise ValueError(f"{name}: the elements of a row must be adjacent (strides {tuple(stride)})")
            need *= shape[k]
            k -= 1
        if need != width:
            raise ValueError(f"{name}: rows must have {width} elements (shape {tuple(shape)})")
        step, span = 0, 1
        for i in range(k, -1, -1):                       # the axes over rows, innermost first
            if shape[i] == 1:
                continue
            if span == 1:
                step = stride[i]
            elif stride[i] != step * span:
                raise ValueError(f"{name}: rows must lie at one distance (shape {tuple(shape)}, strides {tuple(stride)})")
            span *= shape[i]
        return step if span > 1 else width

    def _dense(self, w, dev, name, t, form, dtype):
        """A contiguous operand; None is a null pointer."""
        if t is None:
            return
        if t.dtype is not dtype or t.shape not in form.known or t.get_device() != dev:
            self._look(name, t, form, dtype, dev)
        if not t.is_contiguous():
            raise ValueError(f"{name}: need a contiguous tensor (strides {tuple(t.stride())} of shape {tuple(t.shape)})")
        w[self._at[name]] = t.data_ptr()

    def _vector(self, w, dev, name, t, numel, dtype):
        """A contiguous operand of one axis; None is a null pointer."""
        if t is None:
            return
        if t.dtype is not dtype or t.get_device() != dev or t.numel() != numel or not t.is_contiguous():
            raise ValueError(f"{name}: need a contiguous {dtype} tensor on cuda:{dev}, the current device, with {numel} elements "
                             f"(got {t.dtype}, {tuple(t.shape)} on {t.device})")
        w[self._at[name]] = t.data_ptr()

    def _lead(self):
        """The axes over rows of whole sequences."""
        p = self._struct
        return (int(p.T),) if p.packed else (int(p.N), int(p.L))

    def _new_step(self, rows, pool, *forms):
        """The forms of a step's operands, kept by its rows and states."""
        if len(self._step_forms) >= 64:
            self._step_forms.clear()
        self._step_forms[rows, pool] = forms
        return forms

    def _seq(self, w, dev, seq_start):
        p = self._struct
        if bool(p.packed) != (seq_start is not None):
            raise ValueError("seq_start belongs to packed problems, and only to them")
        self._vector(w, dev, "seq_start", seq_start, p.N + 1, self._torch.int32)

    def _buffer(self, w, dev, name, t, need):
        if t is None or t.get_device() != dev or not t.is_contiguous() or t.numel() * t.element_size() < need:
            raise ValueError(f"{name}: a contiguous buffer of {need} bytes on the current device required")
        w[self._at[name]] = t.data_ptr()
        return t.numel() * t.element_size()

    def _workspace(self, w, dev, ws, need):
        if need:
            w[self._at["ws_bytes"]] = self._buffer(w, dev, "ws", ws, need)

    def _slots(self, w, dev, slots, rows, pool):
        w[self._at["rows"]], w[self._at["num_slots"]] = rows, pool
        self._vector(w, dev, "slots", slots, rows, self._torch.int32)

    def _call(self, f, w, dev, stream):
        if stream is None:
            sp = self._raw_stream(dev)
        else:
            sp = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
        rc = f(self.handle, self._pack(*w), sp or None)
        if rc:
            self._check_rc(rc)

    def _bytes(self, n, device):
        return self._torch.empty(max(n, 16), dtype=self._torch.uint8, device=device or "cuda")


class CausalConvPlan(_SsmPlan):
    """Causal depthwise convolution: y[r] = act(bias + sum_k w[:, k] x[r - (W-1) + k])."""

    _op = "cconv"
    _at, _packer = _layout(wgrad_cconv_args)
    _words, _pack = _packer.size // 8, _packer.pack

    def __init__(self, problem: dict, hip_device: int | None = None):
        super().__init__(problem, hip_device)
        p = self._struct
        C, W = self._C, self._W = int(p.C), int(p.W)
        self._row_form, self._taps = _Form(*self._lead(), C, rows=self.rows), _Form(C, W)
        self._states = _Form(int(p.N), W - 1, C)
        self.workspace_bytes = int(self._lib.wgrad_cconv_workspace_bytes(self.handle))

    @staticmethod
    def _problem(gcb, d):
        act = d.get("activation", "none")
        if act not in ACTIVATIONS:
            raise ValueError(f"activation must be one of {tuple(ACTIVATIONS)}")
        return wgrad_cconv_problem(gcb.DTYPES[d["dtype"]], ACTIVATIONS[act], int(d["W"]), int(bool(d.get("packed"))),
                                   int(d["N"]), int(d["L"]), int(d.get("T", 0)), int(d["C"]))

    def _create(self, p, dev):
        return self._lib.wgrad_cconv_plan(ctypes.byref(p), dev, ctypes.byref(self.handle))

    def new_workspace(self, device=None):
        """Workspace of run_backward."""
        return self._bytes(self.workspace_bytes, device)

    def run(self, x, w, y, bias=None, init_state=None, final_state=None, seq_start=None, stream=None):
        (a, dev), C, t, rows = self._block(x), self._C, self.dtype, self._row_form
        self._rows_of(a, dev, "x", x, rows)
        self._rows_of(a, dev, "y", y, rows)
        self._dense(a, dev, "w", w, self._taps, t)
        self._vector(a, dev, "bias", bias, C, t)
        self._dense(a, dev, "init_state", init_state, self._states, t)
        self._dense(a, dev, "final_state", final_state, self._states, t)
        self._seq(a, dev, seq_start)
        self._call(self._run, a, dev, stream)

    def run_backward(self, x, w, dy, dx, dw, dbias=None, bias=None, init_state=None, dinit_state=None, dfinal_state=None,
                     seq_start=None, ws=None, stream=None):
        (a, dev), C, t, f32, rows = self._block(x), self._C, self.dtype, self._torch.float32, self._row_form
        self._rows_of(a, dev, "x", x, rows)
        self._rows_of(a, dev, "dy", dy, rows)
        self._rows_of(a, dev, "dx", dx, rows)
        self._dense(a, dev, "w", w, self._taps, t)
        self._dense(a, dev, "dw", dw, self._taps, f32)
        self._vector(a, dev, "dbias", dbias, C, f32)
        self._vector(a, dev, "bias", bias, C, t)
        for name, s in (("init_state", init_state), ("dinit_state", dinit_state), ("dfinal_state", dfinal_state)):
            self._dense(a, dev, name, s, self._states, t)
        self._seq(a, dev, seq_start)
        self._workspace(a, dev, ws, self.workspace_bytes)
        self._call(self._backward_run, a, dev, stream)

    def run_step(self, x, w, state, y, bias=None, slots=None, stream=None):
        """x, y [rows, C]; state [num_slots, W-1, C], updated in place; slots int32 [rows] or None (row i uses state i)."""
        (a, dev), C, t = self._block(x), self._C, self.dtype
        rows, pool = x.numel() // C, state.shape[0]
        row_form, states = self._step_forms.get((rows, pool)) or self._new_step(
            rows, pool, _Form(rows, C, rows=rows), _Form(pool, self._W - 1, C))
        self._rows_of(a, dev, "x", x, row_form)
        self._rows_of(a, dev, "y", y, row_form)
        self._dense(a, dev, "w", w, self._taps, t)
        self._vector(a, dev, "bias", bias, C, t)
        self._dense(a, dev, "state", state, states, t)
        self._slots(a, dev, slots, rows, pool)
        self._call(self._step_run, a, dev, stream)


class ScanPlan(_SsmPlan):
    """Selective scan: h = exp(d A) h + d x B, y = (C h + D x) silu(z), d = softplus(delta + delta_bias)."""

    _op = "scan"
    _at, _packer = _layout(wgrad_scan_args)
    _words, _pack = _packer.size // 8, _packer.pack

    def __init__(self, problem: dict, segments: int = 0, segments_backward: int = 0, hip_device: int | None = None):
        self._overrides = wgrad_scan_overrides(int(segments), int(segments_backward))
        super().__init__(problem, hip_device)
        p = self._struct
        self._C, self._G, self._S = int(p.C), int(p.G), int(p.S)
        self._row_forms = self._forms(self.rows, *self._lead())
        self._rates, self._states = _Form(self._C, self._S), _Form(int(p.N), self._C, self._S)
        self.info = wgrad_scan_plan_query(self)
        self.workspace_bytes = self.info["workspace_bytes"]
        self.workspace_bytes_backward = self.info["workspace_bytes_backward"]
        self.saved_bytes = self.info["saved_bytes"]

    @staticmethod
    def _problem(gcb, d):
        return wgrad_scan_problem(gcb.DTYPES[d["dtype"]], int(bool(d.get("softplus", True))), int(bool(d.get("packed"))), 0,
                                  int(d["N"]), int(d["L"]), int(d.get("T", 0)), int(d["C"]), int(d.get("G", 1)), int(d["S"]))

    def _create(self, p, dev):
        return self._lib.wgrad_scan_plan(ctypes.byref(p), ctypes.byref(self._overrides), dev, ctypes.byref(self.handle))

    def new_workspace(self, device=None):
        """Workspace that run and run_backward may share on one stream."""
        return self._bytes(max(self.workspace_bytes, self.workspace_bytes_backward), device)

    def new_saved(self, device=None):
        """Buffer for the states that run leaves for run_backward."""
        return self._bytes(self.saved_bytes, device)

    def _forms(self, rows, *lead):
        """The forms of rows of channels, and of B and C."""
        return _Form(*lead, self._C, rows=rows), _Form(*lead, self._G, self._S, rows=rows)

    def _inputs(self, forms, x, delta, A, B, C, D, z, delta_bias):
        (a, dev), n, f32, (rows, bc) = self._block(x), self._C, self._torch.float32, forms
        self._rows_of(a, dev, "x", x, rows)
        self._rows_of(a, dev, "delta", delta, rows)
        self._rows_of(a, dev, "B", B, bc)
        self._rows_of(a, dev, "C", C, bc)
        if z is not None:
            self._rows_of(a, dev, "z", z, rows)
        self._dense(a, dev, "A", A, self._rates, f32)
        self._vector(a, dev, "D", D, n, f32)
        self._vector(a, dev, "delta_bias", delta_bias, n, f32)
        return a, dev

    def run(self, x, delta, A, B, C, y, D=None, z=None, delta_bias=None, init_state=None, final_state=None, saved=None,
            seq_start=None, ws=None, stream=None):
        a, dev = self._inputs(self._row_forms, x, delta, A, B, C, D, z, delta_bias)
        self._rows_of(a, dev, "y", y, self._row_forms[0])
        states, f32 = self._states, self._torch.float32
        self._dense(a, dev, "init_state", init_state, states, f32)
        self._dense(a, dev, "final_state", final_state, states, f32)
        self._seq(a, dev, seq_start)
        if saved is not None:
            self._buffer(a, dev, "saved", saved, self.saved_bytes)
        self._workspace(a, dev, ws, self.workspace_bytes)
        self._call(self._run, a, dev, stream)

    def run_backward(self, x, delta, A, B, C, dy, saved, dx, ddelta, dA, dB, dC, D=None, z=None, delta_bias=None, dD=None,
                     dz=None, ddelta_bias=None, dinit_state=None, dfinal_state=None, seq_start=None, ws=None, stream=None):
        """The gradients from the same inputs as run's and the states that it left in saved."""
        (rows, bc), n, f32 = self._row_forms, self._C, self._torch.float32
        a, dev = self._inputs(self._row_forms, x, delta, A, B, C, D, z, delta_bias)
        self._rows_of(a, dev, "dy", dy, rows)
        self._rows_of(a, dev, "dx", dx, rows)
        self._rows_of(a, dev, "ddelta", ddelta, rows)
        if (z is None) != (dz is None):
            raise ValueError("dz belongs to z, and only to it")
        if dz is not None:
            self._rows_of(a, dev, "dz", dz, rows)
        self._rows_of(a, dev, "dB", dB, bc)
        self._rows_of(a, dev, "dC", dC, bc)
        self._dense(a, dev, "dA", dA, self._rates, f32)
        self._vector(a, dev, "dD", dD, n, f32)
        self._vector(a, dev, "ddelta_bias", ddelta_bias, n, f32)
        self._dense(a, dev, "dinit_state", dinit_state, self._states, f32)
        self._dense(a, dev, "dfinal_state", dfinal_state, self._states, f32)
        self._seq(a, dev, seq_start)
        self._buffer(a, dev, "saved", saved, self.saved_bytes)
        self._workspace(a, dev, ws, self.workspace_bytes_backward)
        self._call(self._backward_run, a, dev, stream)

    def run_step(self, x, delta, A, B, C, state, y, D=None, z=None, delta_bias=None, slots=None, stream=None):
        """x, delta, z, y [rows, C]; state [num_slots, C, S] fp32, updated in place; slots int32 [rows] or None."""
        rows, pool = x.numel() // self._C, state.shape[0]
        forms, states = self._step_forms.get((rows, pool)) or self._new_step(
            rows, pool, self._forms(rows, rows), _Form(pool, self._C, self._S))
        a, dev = self._inputs(forms, x, delta, A, B, C, D, z, delta_bias)
        self._rows_of(a, dev, "y", y, forms[0])
        self._dense(a, dev, "state", state, states, self._torch.float32)
        self._slots(a, dev, slots, rows, pool)
        self._call(self._step_run, a, dev, stream)


# ---------------------------------------------------------------- ABI-named wrappers


def wgrad_cconv_plan(problem: dict, hip_device: int | None = None) -> CausalConvPlan:
    """Create a plan. hip_device as in wgrad_plan (-1 = host only)."""
    return CausalConvPlan(problem, hip_device)


def wgrad_cconv_plan_destroy(plan: CausalConvPlan) -> None:
    plan.close()


def wgrad_cconv_workspace_bytes(plan: CausalConvPlan) -> int:
    return plan.workspace_bytes


def wgrad_cconv_run(plan: CausalConvPlan, *args, **kw) -> None:
    plan.run(*args, **kw)


def wgrad_cconv_backward_run(plan: CausalConvPlan, *args, **kw) -> None:
    plan.run_backward(*args, **kw)


def wgrad_cconv_step_run(plan: CausalConvPlan, *args, **kw) -> None:
    plan.run_step(*args, **kw)


def wgrad_scan_plan(problem: dict, segments: int = 0, segments_backward: int = 0, hip_device: int | None = None) -> ScanPlan:
    """Create a plan; segments are overrides for tests and benchmarks."""
    return ScanPlan(problem, segments, segments_backward, hip_device)


def wgrad_scan_plan_destroy(plan: ScanPlan) -> None:
    plan.close()


def wgrad_scan_plan_query(plan: ScanPlan) -> dict:
    info = wgrad_scan_plan_info()
    gcb = _gcb()
    gcb._check(gcb.load_library().wgrad_scan_plan_query(plan.handle, ctypes.byref(info)))
    return {name: getattr(info, name) for name, _ in info._fields_}


def wgrad_scan_workspace_bytes(plan: ScanPlan, backward: bool = False) -> int:
    return plan.workspace_bytes_backward if backward else plan.workspace_bytes


def wgrad_scan_saved_bytes(plan: ScanPlan) -> int:
    return plan.saved_bytes


def wgrad_scan_run(plan: ScanPlan, *args, **kw) -> None:
    plan.run(*args, **kw)


def wgrad_scan_backward_run(plan: ScanPlan, *args, **kw) -> None:
    plan.run_backward(*args, **kw)


def wgrad_scan_step_run(plan: ScanPlan, *args, **kw) -> None:
    plan.run_step(*args, **kw)


def _on_stream(x, stream, call):
    """call() with `stream` (as the plans take it) as the current one, so that what it allocates belongs to the stream that
    the kernels run on; its result may then be used on the caller's current stream too."""
    import torch
    if stream is None:
        return call()
    handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    here = torch.cuda.current_stream(x.device)
    there = torch.cuda.ExternalStream(handle, x.device) if handle else torch.cuda.default_stream(x.device)
    with torch.cuda.stream(there):
        y = call()
    y.record_stream(here)
    return y


def causal_conv(problem: dict, x, w, bias=None, stream=None, **kw):
    """Convenience: plan, allocate y with torch, run. On another stream than the current one the caller orders that stream
    after its inputs, and the use of y after it."""
    import torch

    def call():
        y = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        CausalConvPlan(problem).run(x, w, y, bias=bias, **kw)
        return y
    return _on_stream(x, stream, call)


def selective_scan(problem: dict, x, delta, A, B, C, stream=None, **kw):
    """Convenience: plan, allocate y (and the workspace) with torch, run. Streams as with causal_conv."""
    import torch

    def call():
        plan = ScanPlan(problem)
        y = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        plan.run(x, delta, A, B, C, y, ws=plan.new_workspace(x.device) if plan.workspace_bytes else None, **kw)
        return y
    return _on_stream(x, stream, call)
