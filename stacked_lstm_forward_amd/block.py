"""The block operators (``include/block/lstm_block.h``): layer norm of a residual
sum and the gated linear recurrence, each with its gradients, and the clipping of
all gradients of a network by their common norm.

Binding (argument marshalling only) under the C names,

    lstm_norm_validate(desc, train), lstm_glr_validate(desc, train) -> status
    lstm_norm_bwd_workspace_size(desc), lstm_glr_reserve_size(desc), lstm_glr_workspace_size(desc) -> int
    lstm_norm_fwd(desc, x, r, w, b, lengths, s, y, mean, rstd, stream=None) -> status
    lstm_norm_bwd(desc, s, w, lengths, mean, rstd, dy, ds, dx, dw, db, ws, stream=None) -> status
    lstm_glr_fwd(desc, f, u, o, c0, lengths, y, cT, reserve, ws, stream=None) -> status
    lstm_glr_bwd(desc, f, u, o, c0, lengths, reserve, dy, dcT, df, du, dout_o, dc0, ws, stream=None) -> status
    lstm_glr_last_error(desc, train, ws, stream=None) -> status
    lstm_clip_table_size(tensors, n) -> int
    lstm_clip_table(tensors, n, table, stream=None) -> status
    lstm_clip(tensors, n, table, max_norm, eps, out, stream=None) -> status

and on top of it problems that own outputs and workspaces, made once per shape:

    p = prepare_norm(x, w, b, residual=r, train=True)
    p.forward();  p.backward(dy, ds)                          # p.y, p.s, p.dx, p.dw, p.db
    p = prepare_glr(f, u, o, c0=c0, train=True)
    p.forward();  p.backward(dy, dcT)                         # p.y, p.cT, p.df, p.du, p.do, p.dc0
    p = prepare_clip(gradients, max_norm=1.0);  p.run()       # p.norm, p.coef, the gradients

Problems read their tensors as those of ``decoder.py`` do: whatever they hold at
the call, and what replaces one (``p.x = t``) is checked like the first.  The tensors
themselves keep their shape, strides and type; those of a clipping problem may be
given other memory (``t.data = ..``) and are looked at before every call.
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass

from . import LSTM_BF16, LSTM_F32, LSTM_OK, _ptr, _stream, check, load_library
from .decoder import _dtype, _like, _on, _Problem, _ref, _workspace
from .held import Held

EXPORTED = ("lstm_norm_validate", "lstm_norm_bwd_workspace_size", "lstm_norm_fwd", "lstm_norm_bwd",
            "lstm_glr_validate", "lstm_glr_reserve_size", "lstm_glr_workspace_size", "lstm_glr_fwd", "lstm_glr_bwd",
            "lstm_glr_last_error", "lstm_clip_table_size", "lstm_clip_table", "lstm_clip")
LSTM_GLR_LINEAR, LSTM_GLR_TANH = 0, 1


class SeqStride(ctypes.Structure):
    _fields_ = [("b", ctypes.c_int64), ("t", ctypes.c_int64)]


class NormDesc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "T", "N", "dtype", "grad_dtype")] + [("eps", ctypes.c_float)] + [
        (n, SeqStride) for n in ("x", "r", "s", "y", "dy", "ds", "dx")]


class GlrDesc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "T", "H", "dtype", "grad_dtype", "cand")] + [
        (n, SeqStride) for n in ("f", "u", "o", "y", "dy", "df", "du", "dout_o")] + [("wait_timeout_us", ctypes.c_int64)]


class ClipTensor(ctypes.Structure):
    _fields_ = [("src", ctypes.c_void_p), ("dst", ctypes.c_void_p), ("count", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("reserved", ctypes.c_int32)]


_ready = None


def _lib() -> ctypes.CDLL:
    global _ready
    if _ready is not None:
        return _ready
    lib = load_library()
    vp, i32, sz, f64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t, ctypes.c_double
    pn, pg, pc = ctypes.POINTER(NormDesc), ctypes.POINTER(GlrDesc), ctypes.POINTER(ClipTensor)
    for name, restype, args in (("lstm_norm_validate", i32, [pn, ctypes.c_int]),
                                ("lstm_norm_bwd_workspace_size", sz, [pn]), ("lstm_norm_fwd", i32, [pn] + [vp] * 10),
                                ("lstm_norm_bwd", i32, [pn] + [vp] * 12),
                                ("lstm_glr_validate", i32, [pg, ctypes.c_int]), ("lstm_glr_reserve_size", sz, [pg]), ("lstm_glr_workspace_size", sz, [pg]),
                                ("lstm_glr_fwd", i32, [pg] + [vp] * 10), ("lstm_glr_bwd", i32, [pg] + [vp] * 14),
                                ("lstm_glr_last_error", i32, [pg, ctypes.c_int, vp, vp]),
                                ("lstm_clip_table_size", sz, [pc, i32]), ("lstm_clip_table", i32, [pc, i32, vp, vp]),
                                ("lstm_clip", i32, [pc, i32, vp, f64, f64, vp, vp])):
        f = getattr(lib, name)
        f.argtypes, f.restype = args, restype
    _ready = lib
    return lib


def lstm_norm_validate(desc, train=False) -> int:
    return int(_lib().lstm_norm_validate(_ref(desc), int(train)))


def lstm_norm_bwd_workspace_size(desc) -> int:
    return int(_lib().lstm_norm_bwd_workspace_size(_ref(desc)))


def lstm_norm_fwd(desc, x, r, w, b, lengths, s, y, mean, rstd, stream=None) -> int:
    return int(_lib().lstm_norm_fwd(_ref(desc), _ptr(x), _ptr(r), _ptr(w), _ptr(b), _ptr(lengths), _ptr(s), _ptr(y),
                                    _ptr(mean), _ptr(rstd), _stream(stream)))


def lstm_norm_bwd(desc, s, w, lengths, mean, rstd, dy, ds, dx, dw, db, ws, stream=None) -> int:
    return int(_lib().lstm_norm_bwd(_ref(desc), _ptr(s), _ptr(w), _ptr(lengths), _ptr(mean), _ptr(rstd), _ptr(dy),
                                    _ptr(ds), _ptr(dx), _ptr(dw), _ptr(db), _ptr(ws), _stream(stream)))


def lstm_glr_validate(desc, train=False) -> int:
    return int(_lib().lstm_glr_validate(_ref(desc), int(train)))


def lstm_glr_reserve_size(desc) -> int:
    return int(_lib().lstm_glr_reserve_size(_ref(desc)))


def lstm_glr_workspace_size(desc) -> int:
    return int(_lib().lstm_glr_workspace_size(_ref(desc)))


def lstm_glr_fwd(desc, f, u, o, c0, lengths, y, cT, reserve, ws, stream=None) -> int:
    return int(_lib().lstm_glr_fwd(_ref(desc), _ptr(f), _ptr(u), _ptr(o), _ptr(c0), _ptr(lengths), _ptr(y), _ptr(cT),
                                   _ptr(reserve), _ptr(ws), _stream(stream)))


def lstm_glr_bwd(desc, f, u, o, c0, lengths, reserve, dy, dcT, df, du, dout_o, dc0, ws, stream=None) -> int:
    return int(_lib().lstm_glr_bwd(_ref(desc), _ptr(f), _ptr(u), _ptr(o), _ptr(c0), _ptr(lengths), _ptr(reserve),
                                   _ptr(dy), _ptr(dcT), _ptr(df), _ptr(du), _ptr(dout_o), _ptr(dc0), _ptr(ws),
                                   _stream(stream)))


def lstm_glr_last_error(desc, train, ws, stream=None) -> int:
    return int(_lib().lstm_glr_last_error(_ref(desc), int(train), _ptr(ws), _stream(stream)))


def lstm_clip_table_size(tensors, n) -> int:
    return int(_lib().lstm_clip_table_size(tensors, n))


def lstm_clip_table(tensors, n, table, stream=None) -> int:
    return int(_lib().lstm_clip_table(tensors, n, _ptr(table), _stream(stream)))


def lstm_clip(tensors, n, table, max_norm, eps, out, stream=None) -> int:
    return int(_lib().lstm_clip(tensors, n, _ptr(table), max_norm, eps, _ptr(out), _stream(stream)))


# ---- checks of tensors (host only) --------------------------------------------


def _seq(t, what: str) -> SeqStride:
    """Strides of a [B, T, width] tensor whose steps are contiguous."""
    if t.shape[2] > 1 and t.stride(2) != 1:
        raise ValueError(f"{what}: the values of a step must be contiguous (stride {t.stride(2)})")
    return SeqStride(*(0 if n == 1 else st for n, st in zip(t.shape[:2], t.stride()[:2])))


def _apart(t, s: SeqStride, what: str) -> None:
    """An output's steps lie apart: the inner stride holds a step, the outer one all that is inside."""
    B, T, W = t.shape
    (n, inner), (_, outer) = sorted(((B, s.b), (T, s.t)), key=lambda x: x[1] if x[0] > 1 else 0)
    if B * T > 1 and (outer < W or (n > 1 and (inner < W or outer < inner * (n - 1) + W))):
        raise ValueError(f"{what}: steps that overlap (strides {tuple(t.stride())})")


def _sequence(t, what: str) -> None:
    if t.dim() != 3 or t.numel() == 0:
        raise ValueError(f"{what}: [batch, length, width], none of them 0, not {tuple(t.shape)}")


def _made(t, dtype):
    """A new tensor like t, dense, the dimensions in the order of t's strides."""
    import torch
    first = (0, 1) if t.stride(0) >= t.stride(1) else (1, 0)
    x = torch.empty([t.shape[first[0]], t.shape[first[1]], t.shape[2]], dtype=dtype, device=t.device)
    return x if first == (0, 1) else x.transpose(0, 1)


def _grad_dtype(grad_dtype, dtype):
    import torch
    g = torch.float32 if grad_dtype is None else grad_dtype
    if g not in (torch.float32, dtype):
        raise TypeError(f"grad_dtype: float32 or the tensors' {dtype}, not {g}")
    return g


class _SeqProblem(_Problem):
    """Problems of sequences: strides go into the description with the tensor that has them.  Of each
    class: _seqs {attribute: field of the description}, _outputs among them, _flat {attribute: (shape, dtype)},
    _optional those that may be None."""

    def _place(self, name, t) -> None:
        s = _seq(t, name)
        if name in self._outputs:
            _apart(t, s, name)
        setattr(self.desc, self._seqs[name], s)

    def _place_all(self) -> None:
        for name in self._seqs:
            if getattr(self, name) is not None:
                self._place(name, getattr(self, name))

    def _checked(self, name, t):
        held = self.__dict__[name]
        if name in self._seqs:
            if held is None or t is None:
                raise ValueError(f"{name}: the problem was made {'without' if held is None else 'with'} it")
            _like(t, name, held.shape, held.dtype, held.device, dense=False)
            self._place(name, t)
        elif name in self._flat:
            if t is None:
                if name not in self._optional:
                    raise ValueError(f"{name}: the problem was made with it")
                return None
            shape, dtype = self._flat[name]
            _like(t, name, shape, dtype, self.device)
        elif name in ("ws", "reserve"):
            self._workspace_like(t, name)
        return t

    def _gradients(self, made, what: str) -> None:
        if made is None:
            raise RuntimeError(f"backward: {what}(..., train=True)")
        if not self.gpu:
            self._runs_on(self.device)

    def _upstream(self, name: str, t, like, dtype) -> None:
        """Checks a gradient from above, a tensor like `like`, and puts its strides into the description."""
        if t.dtype is not dtype or t.shape != like.shape or t.device != self.device:
            _like(t, name, like.shape, dtype, self.device, dense=False)
        strides = t.stride()
        if self._above.get(name) != strides:
            setattr(self.desc, name, _seq(t, name))
            self._above[name] = strides


def _at(t):
    return None if t is None else t.data_ptr()


# ---- layer norm ---------------------------------------------------------------


@dataclass
class NormProblem(_SeqProblem):
    desc: NormDesc
    x: object
    r: object
    w: object
    b: object
    lengths: object
    s: object
    y: object
    mean: object
    rstd: object
    dx: object = None
    dw: object = None
    db: object = None
    ws: object = None

    _seqs = {n: n for n in ("x", "r", "s", "y", "dx")}
    _outputs = ("s", "y", "dx")
    _optional = ("lengths", "w", "b", "mean", "rstd", "dw", "db")

    def __post_init__(self):
        import torch
        self.gpu, self.device = self.x.is_cuda, self.x.device  # (for good: what replaces a tensor is there too)
        self._above = {}
        B, T, N = self.x.shape
        f32 = torch.float32
        self._flat = {"lengths": ((B,), torch.int32), "w": ((N,), self.x.dtype), "b": ((N,), self.x.dtype),
                      "mean": ((B, T), f32), "rstd": ((B, T), f32), "dw": ((N,), f32), "db": ((N,), f32)}

    def _place(self, name, t) -> None:
        super()._place(name, t)
        if name == "x" and self.r is None:  # what is normalised is x itself
            self.desc.s = self.desc.x

    def forward(self, stream=None) -> None:
        """y [B, T, N], with a residual s = x + r, and of each step mean and rstd [B, T]."""
        if not self.gpu:
            self._runs_on(self.device)
        st = _lib().lstm_norm_fwd(self.desc, self.x.data_ptr(), _at(self.r), _at(self.w), _at(self.b),
                                  _at(self.lengths), _at(self.s), self.y.data_ptr(), _at(self.mean), _at(self.rstd),
                                  _on(stream, self.x))
        if st != LSTM_OK:
            check(st, "lstm_norm_fwd")

    def backward(self, dy, ds=None, stream=None) -> None:
        """dx (of x and of the residual alike), dw, db from dy, a tensor like y in the gradients' type, and ds,
        what reaches s past the norm, after a forward() of the same inputs."""
        self._gradients(self.dx, "prepare_norm")
        self._upstream("dy", dy, self.x, self.dx.dtype)
        if ds is not None:
            self._upstream("ds", ds, self.x, self.dx.dtype)
        st = _lib().lstm_norm_bwd(self.desc, (self.x if self.s is None else self.s).data_ptr(), _at(self.w),
                                  _at(self.lengths), _at(self.mean), _at(self.rstd), dy.data_ptr(), _at(ds),
                                  self.dx.data_ptr(), _at(self.dw), _at(self.db), self.ws.data_ptr(),
                                  _on(stream, self.x))
        if st != LSTM_OK:
            check(st, "lstm_norm_bwd")


def prepare_norm(x, w=None, b=None, *, residual=None, lengths=None, eps: float = 1e-5, train: bool = False,
                 grad_dtype=None) -> NormProblem:
    """Outputs and workspace for the layer norm of x [B, T, N] (+ residual, a tensor like it) with weight w
    and bias b [N] of its type, each of which may be None.

    The values of a step are contiguous, the other strides free: a stack's [T][B][H] outputs enter as
    ``y.transpose(0, 1)``.  lengths [B] int32 leaves later steps out.  Outputs and gradients have x's
    layout; the type of dy, ds and dx is fp32 or x's (grad_dtype), dw and db are fp32.
    """
    import torch
    _sequence(x, "x")
    B, T, N = x.shape
    dt = _dtype(x, "x")
    for t, what in ((w, "w"), (b, "b")):
        if t is not None:
            _like(t, what, (N,), x.dtype, x.device)
    if residual is not None:
        _like(residual, "residual", x.shape, x.dtype, x.device, dense=False)
    if lengths is not None:
        _like(lengths, "lengths", (B,), torch.int32, x.device)
    g = _grad_dtype(grad_dtype, x.dtype)
    desc = NormDesc(B, T, N, dt, LSTM_F32 if g == torch.float32 else LSTM_BF16, eps)
    y, s = _made(x, x.dtype), _made(x, x.dtype) if residual is not None else None

    def small(*shape):
        return torch.empty(shape, dtype=torch.float32, device=x.device)

    mean, rstd = (small(B, T), small(B, T)) if train else (None, None)
    p = NormProblem(desc, x, residual, w, b, lengths, s, y, mean, rstd)
    if train:
        p.__dict__.update(dx=_made(x, g), dw=None if w is None else small(N), db=None if b is None else small(N))
    p._place_all()
    check(lstm_norm_validate(desc, train), "lstm_norm_validate")
    if train:
        p.__dict__["ws"] = _workspace(lstm_norm_bwd_workspace_size(desc), x.device)
    return p


# ---- gated linear recurrence --------------------------------------------------


@dataclass
class GlrProblem(_SeqProblem):
    desc: GlrDesc
    f: object
    u: object
    o: object
    c0: object
    lengths: object
    y: object
    cT: object
    ws: object
    reserve: object = None
    df: object = None
    du: object = None
    do: object = None
    dc0: object = None

    _seqs = {"f": "f", "u": "u", "o": "o", "y": "y", "df": "df", "du": "du", "do": "dout_o"}
    _outputs = ("y", "df", "du", "do")
    _optional = ("lengths", "c0", "cT", "dc0")

    def __post_init__(self):
        import torch
        self.gpu, self.device = self.f.is_cuda, self.f.device
        self._above = {}
        B, _, H = self.f.shape
        self._flat = {"lengths": ((B,), torch.int32),
                      **{n: ((B, H), torch.float32) for n in ("c0", "cT", "dc0")}}

    def forward(self, stream=None) -> None:
        """y [B, T, H] and the states after the last steps, cT [B, H]."""
        if not self.gpu:
            self._runs_on(self.device)
        st = _lib().lstm_glr_fwd(self.desc, self.f.data_ptr(), self.u.data_ptr(), _at(self.o), _at(self.c0),
                                 _at(self.lengths), self.y.data_ptr(), _at(self.cT), _at(self.reserve),
                                 self.ws.data_ptr(), _on(stream, self.f))
        if st != LSTM_OK:
            check(st, "lstm_glr_fwd")

    def backward(self, dy, dcT=None, stream=None) -> None:
        """df, du, do (with an output gate) and dc0 from dy, a tensor like y in the gradients' type, and dcT
        [B, H] fp32, after a forward() of the same inputs."""
        import torch
        self._gradients(self.df, "prepare_glr")
        self._upstream("dy", dy, self.f, self.df.dtype)
        if dcT is not None and (dcT.dtype is not torch.float32 or dcT.shape != self._flat["cT"][0] or
                                dcT.device != self.device or not dcT.is_contiguous()):
            _like(dcT, "dcT", self._flat["cT"][0], torch.float32, self.device)
        st = _lib().lstm_glr_bwd(self.desc, self.f.data_ptr(), self.u.data_ptr(), _at(self.o), _at(self.c0),
                                 _at(self.lengths), self.reserve.data_ptr(), dy.data_ptr(), _at(dcT),
                                 self.df.data_ptr(), self.du.data_ptr(), _at(self.do), _at(self.dc0),
                                 self.ws.data_ptr(), _on(stream, self.f))
        if st != LSTM_OK:
            check(st, "lstm_glr_bwd")

    def last_error(self, train=False, stream=None) -> int:
        """The status that the last forward() (train: backward()), if it was the last call, left on the device:
        LSTM_OK, or LSTM_ERR_BARRIER_TIMEOUT where a wait passed desc.wait_timeout_us.  Waits for the stream."""
        if not self.gpu:
            self._runs_on(self.device)
        return lstm_glr_last_error(self.desc, train, self.ws, _on(stream, self.f))

    def advance(self) -> None:
        """Makes the states after this call the next call's first ones (serving: the next step or stretch of
        the same sentences).  The buffers are swapped, not copied; without a c0, the first advance() adds one."""
        import torch
        own = self.__dict__
        if self.cT is None:
            raise ValueError("cT: the problem has none to go on from")
        if self.c0 is None:
            own["c0"] = torch.empty_like(self.cT)
        own["c0"], own["cT"] = self.cT, self.c0


def prepare_glr(f, u, o=None, *, c0=None, lengths=None, tanh: bool = False, train: bool = False,
                grad_dtype=None) -> GlrProblem:
    """Outputs and workspace for the gated linear recurrence over f, u and (output gate) o [B, T, H]: what comes
    before their sigmoids, and before u's tanh if there is one.

    The values of a step are contiguous, the other strides free, so the parts of one projection [.., 3H] enter
    in place, and df, du, do may be set to parts of one tensor as well.  c0 [B, H] fp32; lengths [B] int32
    leaves later steps out.  Outputs and gradients have the layout of the tensor they belong to; the type of dy,
    df, du and do is fp32 or f's (grad_dtype), dc0 is fp32.
    """
    import torch
    _sequence(f, "f")
    B, T, H = f.shape
    dt = _dtype(f, "f")
    for t, what in ((u, "u"), (o, "o")):
        if t is not None:
            _like(t, what, f.shape, f.dtype, f.device, dense=False)
    if c0 is not None:
        _like(c0, "c0", (B, H), torch.float32, f.device)
    if lengths is not None:
        _like(lengths, "lengths", (B,), torch.int32, f.device)
    g = _grad_dtype(grad_dtype, f.dtype)
    desc = GlrDesc(B, T, H, dt, LSTM_F32 if g == torch.float32 else LSTM_BF16, LSTM_GLR_TANH if tanh else LSTM_GLR_LINEAR)

    def state():
        return torch.empty((B, H), dtype=torch.float32, device=f.device)

    p = GlrProblem(desc, f, u, o, c0, lengths, _made(f, f.dtype), state(), None)
    if train:
        p.__dict__.update(df=_made(f, g), du=_made(u, g), do=None if o is None else _made(o, g),
                          dc0=None if c0 is None else state())
    p._place_all()
    check(lstm_glr_validate(desc, train), "lstm_glr_validate")
    p.__dict__["ws"] = _workspace(lstm_glr_workspace_size(desc), f.device)
    if train:
        p.__dict__["reserve"] = _workspace(lstm_glr_reserve_size(desc), f.device)
    return p


# ---- clipping -----------------------------------------------------------------


class ClipProblem:
    """Made by prepare_clip.  norm and coef are 0-dimensional tensors on the device.  Calls of one problem follow
    each other: they share its table and sums."""

    def __init__(self, tensors, out, max_norm: float, eps: float):
        import torch
        self.tensors, self.out = tuple(tensors), tuple(out)
        self.max_norm, self.eps = max_norm, eps
        self._all = self.tensors + self.out
        n = len(self.tensors)
        if n == 0 or len(self.out) != n:
            raise ValueError(f"{n} tensors and {len(self.out)} outputs: one tensor at least, and an output for each")
        self.device = self.tensors[0].device
        self._list = (ClipTensor * n)()
        for i, (t, x) in enumerate(zip(self.tensors, self.out)):
            if not t.is_contiguous():
                raise ValueError(f"tensor {i}: must be contiguous")
            if t.device != self.device:
                raise ValueError(f"tensor {i}: on {t.device}, expected {self.device}")
            _like(x, f"output {i}", t.shape, t.dtype, self.device)
            self._list[i].count, self._list[i].dtype = t.numel(), _dtype(t, f"tensor {i}")
        self._held = Held(self._all)
        self._point()
        size = lstm_clip_table_size(self._list, n)
        if size == 0:
            raise ValueError("unsupported tensors: lstm_clip_table_size returned 0")
        self._table = _workspace(size, self.device)
        self._written = None  # the stream that the table was written on
        self._captured = False  # a graph may write it again, for the addresses of its capture
        self._result = torch.empty(2, dtype=torch.float32, device=self.device)
        self.norm, self.coef = self._result[0], self._result[1]

    def _point(self) -> None:
        n, at = len(self.tensors), [t.data_ptr() for t in self._all]
        # an output may be its own tensor, and nothing else that is read or written
        spans = []
        for i, (t, src, dst) in enumerate(zip(self.tensors, at[:n], at[n:])):
            size = t.numel() * t.element_size()
            spans += [(dst, dst + size, True)] + ([] if dst == src else [(src, src + size, False)])
        end = written = 0
        for lo, hi, out in sorted(x for x in spans if x[0] < x[1]):
            if lo < written or (out and lo < end):
                raise ValueError("outputs that overlap each other or other tensors")
            end = max(end, hi)
            written = max(written, hi) if out else written
        for e, src, dst in zip(self._list, at[:n], at[n:]):
            e.src, e.dst = src, dst

    def _moved(self) -> bool:
        """Whether a tensor was given other memory since the last call, which the entries then point to.  Another
        size, type, device or order of its values is refused, at the same address too."""
        if self._held.same():
            return False
        n = len(self.tensors)
        for i, t in enumerate(self._all):
            e = self._list[i % n]
            if (t.numel() != e.count or t.device != self.device or not t.is_contiguous() or
                    _dtype(t, f"tensor {i % n}") != e.dtype):
                raise ValueError(f"{'tensor' if i < n else 'output'} {i % n}: no longer what the problem was made for")
        self._point()
        self._held.read()
        return True

    def run(self, stream=None) -> None:
        """norm, coef, and every output = coef * its tensor.  Calls on the current stream write the table once; one on
        an explicit stream, which may be capturing, or captured, and every call after it write it again: a launch for
        each 64 tensors and one more (301 tensors: 110 us for 95)."""
        import torch
        if self._moved():
            self._written = None
        if self.device.type != "cuda":
            raise ValueError(f"the problem's tensors are on {self.device}: the kernels run on a GPU")
        s = _on(stream, self._result)
        lib, n, table = _lib(), len(self.tensors), self._table.data_ptr()
        # the table is written once for the current stream; a captured call, and one on a stream that may be
        # captured, writes its own, and so does every call after it
        if stream is not None or torch.cuda.is_current_stream_capturing():
            self._captured = True
        once = not self._captured
        if not once or self._written != s:
            check(lib.lstm_clip_table(self._list, n, table, s), "lstm_clip_table")
            self._written = s if once else None
        st = lib.lstm_clip(self._list, n, table, self.max_norm, self.eps, self._result.data_ptr(), s)
        if st != LSTM_OK:
            check(st, "lstm_clip")


def prepare_clip(tensors, max_norm: float, *, out=None, eps: float = 1e-6) -> ClipProblem:
    """The table for clipping contiguous tensors (fp32 or bf16, any shapes) by their common norm: in place, or
    into out, a list of tensors like them.  max_norm = inf only takes the norm (and copies into out)."""
    tensors = list(tensors)
    if not max_norm >= 0 or not 0 <= eps < float("inf"):
        raise ValueError(f"max_norm {max_norm} and eps {eps}: must be at least 0, eps finite")
    return ClipProblem(tensors, tensors if out is None else out, max_norm, eps)
