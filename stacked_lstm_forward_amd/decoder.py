"""The decoder operators (``include/decoder/lstm_dec.h``): attention over an
encoder's outputs with its gradients, and the step of beam search.

Binding (argument marshalling only) under the C names,

    lstm_attn_validate(desc, train) -> status
    lstm_attn_workspace_size(desc), lstm_attn_bwd_workspace_size(desc) -> int
    lstm_attn_fwd(desc, q, k, v, kv_len, key_mask, o, lse, ws, stream=None) -> status
    lstm_attn_bwd(desc, q, k, v, kv_len, key_mask, o, lse, dout, dq, dk, dv, ws, stream=None) -> status
    lstm_beam_workspace_size(desc) -> int
    lstm_beam_step(desc, logits, scores, finished, lengths, tokens, parents, scores_out, finished_out,
                   lengths_out, h, c, h_out, c_out, ws, stream=None) -> status

and on top of it problems that own outputs and workspaces, made once per shape:

    p = prepare_attn(q, k, v, kv_len=n, train=True);  p.forward();  p.backward(dout)   # p.o, p.lse, p.dq, p.dk, p.dv
    s = prepare_beam(logits, scores, finished, lengths, eos=2, states=(h, c));  s.step()

A problem reads the tensors that it was made with, whatever they hold at the
call (or those that its attributes were set to since: they are checked like the
first ones).  ``runner.py`` is its counterpart for the recurrent stacks.
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass
from typing import Optional

from . import LSTM_BF16, LSTM_F32, LSTM_OK, _ptr, _stream, check, load_library

EXPORTED = ("lstm_attn_validate", "lstm_attn_workspace_size", "lstm_attn_bwd_workspace_size", "lstm_attn_fwd",
            "lstm_attn_bwd", "lstm_beam_workspace_size", "lstm_beam_step")


class AttnStride(ctypes.Structure):
    _fields_ = [("b", ctypes.c_int64), ("t", ctypes.c_int64), ("h", ctypes.c_int64)]


class AttnDesc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "Tq", "S", "Hq", "Hkv", "D", "dtype")] + [
        ("scale", ctypes.c_float)] + [(n, AttnStride) for n in ("q", "k", "v", "o", "dout", "dq", "dk", "dv")] + [
        ("o_rest", ctypes.c_void_p)]


class BeamDesc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "K", "V", "dtype", "eos")] + [
        ("alpha", ctypes.c_float), ("L", ctypes.c_int32), ("H", ctypes.c_int32), ("logits_stride", ctypes.c_int64)]


_ready = None


def _lib() -> ctypes.CDLL:
    global _ready
    if _ready is not None:
        return _ready
    lib = load_library()
    vp, i32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
    pa, pb = ctypes.POINTER(AttnDesc), ctypes.POINTER(BeamDesc)
    for name, restype, args in (("lstm_attn_validate", i32, [pa, ctypes.c_int]),
                                ("lstm_attn_workspace_size", sz, [pa]), ("lstm_attn_bwd_workspace_size", sz, [pa]),
                                ("lstm_attn_fwd", i32, [pa] + [vp] * 9), ("lstm_attn_bwd", i32, [pa] + [vp] * 13),
                                ("lstm_beam_workspace_size", sz, [pb]), ("lstm_beam_step", i32, [pb] + [vp] * 15)):
        f = getattr(lib, name)
        f.argtypes, f.restype = args, restype
    _ready = lib
    return lib


def _ref(desc):
    return None if desc is None else ctypes.byref(desc)


def lstm_attn_validate(desc, train=False) -> int:
    return int(_lib().lstm_attn_validate(_ref(desc), int(train)))


def lstm_attn_workspace_size(desc) -> int:
    return int(_lib().lstm_attn_workspace_size(_ref(desc)))


def lstm_attn_bwd_workspace_size(desc) -> int:
    return int(_lib().lstm_attn_bwd_workspace_size(_ref(desc)))


def lstm_attn_fwd(desc, q, k, v, kv_len, key_mask, o, lse, ws, stream=None) -> int:
    return int(_lib().lstm_attn_fwd(_ref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(kv_len), _ptr(key_mask), _ptr(o),
                                    _ptr(lse), _ptr(ws), _stream(stream)))


def lstm_attn_bwd(desc, q, k, v, kv_len, key_mask, o, lse, dout, dq, dk, dv, ws, stream=None) -> int:
    return int(_lib().lstm_attn_bwd(_ref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(kv_len), _ptr(key_mask), _ptr(o),
                                    _ptr(lse), _ptr(dout), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(ws), _stream(stream)))


def lstm_beam_workspace_size(desc) -> int:
    return int(_lib().lstm_beam_workspace_size(_ref(desc)))


def lstm_beam_step(desc, logits, scores, finished, lengths, tokens, parents, scores_out, finished_out, lengths_out,
                   h, c, h_out, c_out, ws, stream=None) -> int:
    return int(_lib().lstm_beam_step(_ref(desc), _ptr(logits), _ptr(scores), _ptr(finished), _ptr(lengths),
                                     _ptr(tokens), _ptr(parents), _ptr(scores_out), _ptr(finished_out),
                                     _ptr(lengths_out), _ptr(h), _ptr(c), _ptr(h_out), _ptr(c_out), _ptr(ws),
                                     _stream(stream)))


def _on(stream, t) -> int:
    """The stream's handle; by default the current stream of t's device (a single token's launch is
    short beside building a torch.cuda.Stream object, so the handle is asked for directly).  That device
    has to be the current one: a default stream's handle is 0 on every device, and the launch would go
    to the current device with addresses of the other."""
    import torch
    index = t.device.index
    if torch._C._cuda_getDevice() != index:
        raise ValueError(f"the problem's tensors are on {t.device}, which is not the current device")
    return torch._C._cuda_getCurrentRawStream(index) if stream is None else _stream(stream)


# ---- checks of tensors (host only) --------------------------------------------


def _dtype(t, what: str) -> int:
    import torch
    ids = {torch.float32: LSTM_F32, torch.bfloat16: LSTM_BF16}
    if t.dtype not in ids:
        raise TypeError(f"{what}: float32 or bfloat16, not {t.dtype}")
    return ids[t.dtype]


def _like(t, what: str, shape, dtype, device, dense=True) -> None:
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{what}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{what}: {t.dtype}, expected {dtype}")
    if t.device != device:
        raise ValueError(f"{what}: on {t.device}, expected {device}")
    if dense and not t.is_contiguous():
        raise ValueError(f"{what}: must be contiguous")


def _bytes(t, what: str):
    """A uint8 or bool tensor as bytes."""
    import torch
    if t.dtype not in (torch.uint8, torch.bool):
        raise TypeError(f"{what}: uint8 or bool, not {t.dtype}")
    return t.view(torch.uint8) if t.dtype == torch.bool else t


def _rows(t, what: str) -> AttnStride:
    """Strides of a [B, T, heads, D] tensor whose heads are contiguous and aligned."""
    unit = 16 // t.element_size()
    s = [0 if n == 1 else st for n, st in zip(t.shape[:3], t.stride()[:3])]
    if t.shape[3] > 1 and t.stride(3) != 1:
        raise ValueError(f"{what}: the values of a head must be contiguous (stride {t.stride(3)})")
    if any(x % unit for x in s) or t.data_ptr() % 16:
        raise ValueError(f"{what}: strides {tuple(t.stride())} and address must be multiples of 16 bytes")
    return AttnStride(*s)


def _workspace(n: int, device):
    import torch
    raw = torch.empty(n + 256, dtype=torch.uint8, device=device)
    off = (-raw.data_ptr()) % 256
    return raw[off:off + n]


class _Problem:
    """The kernels read a problem's tensors by address, so what replaces one is checked first."""

    def _runs_on(self, device) -> None:
        if device.type != "cuda":
            raise ValueError(f"the problem's tensors are on {device}: the kernels run on a GPU")

    def __setattr__(self, name, value):
        if name in self.__dict__:
            value = self._checked(name, value)
        object.__setattr__(self, name, value)

    def _workspace_like(self, t, name: str) -> None:
        held = self.__dict__[name]
        if held is None:
            raise ValueError(f"{name}: the problem was made without it")
        if t.numel() * t.element_size() < held.numel() or t.data_ptr() % 256 or not t.is_contiguous():
            raise ValueError(f"{name}: {held.numel()} bytes, contiguous and aligned to 256")
        if t.device != held.device:
            raise ValueError(f"{name}: on {t.device}, expected {held.device}")


# ---- attention ----------------------------------------------------------------


@dataclass
class AttnProblem(_Problem):
    desc: AttnDesc
    q: object
    k: object
    v: object
    kv_len: object
    key_mask: object
    o: object
    lse: object
    ws: object
    dq: object = None
    dk: object = None
    dv: object = None
    bws: object = None
    o_rest: object = None

    def __post_init__(self):
        self.gpu = self.q.is_cuda  # (for good: what replaces a tensor is on its device)

    def _checked(self, name, t):
        import torch
        d, device = self.desc, self.q.device
        if name in ("q", "k", "v", "o", "dq", "dk", "dv"):
            held = self.__dict__[name]
            if held is None:
                raise ValueError(f"{name}: the problem was made without gradients")
            _like(t, name, held.shape, held.dtype, device, dense=False)
            setattr(d, name, _rows(t, name))
        elif name in ("kv_len", "key_mask", "lse") and t is not None:
            shape, dtype = {"kv_len": ((d.B,), torch.int32), "key_mask": ((d.B, d.S), torch.uint8),
                            "lse": ((d.B, d.Hq, d.Tq), torch.float32)}[name]
            t = _bytes(t, name) if name == "key_mask" else t
            _like(t, name, shape, dtype, device)
        elif name == "o_rest" and t is not None:
            _like(t, name, self.o.shape, torch.bfloat16, device)
            if t.dtype != self.o.dtype or t.data_ptr() % 16:
                raise ValueError("o_rest: of bf16 problems, aligned to 16 bytes")
        elif name in ("ws", "bws"):
            self._workspace_like(t, name)
        if name == "o_rest":
            d.o_rest = None if t is None else t.data_ptr()
        return t

    def forward(self, stream=None) -> None:
        """o [B, Tq, Hq, D] and lse [B, Hq, Tq]."""
        if not self.gpu:
            self._runs_on(self.q.device)
        n, m, e = self.kv_len, self.key_mask, self.lse
        st = _lib().lstm_attn_fwd(self.desc, self.q.data_ptr(), self.k.data_ptr(), self.v.data_ptr(),
                                  None if n is None else n.data_ptr(), None if m is None else m.data_ptr(),
                                  self.o.data_ptr(), None if e is None else e.data_ptr(), self.ws.data_ptr(),
                                  _on(stream, self.q))
        if st != LSTM_OK:
            check(st, "lstm_attn_fwd")

    def backward(self, dout, stream=None) -> None:
        """dq, dk, dv from dout, a tensor like o, after a forward() of the same inputs."""
        if self.bws is None:
            raise RuntimeError("backward: prepare_attn(..., train=True)")
        self._runs_on(self.q.device)
        _like(dout, "dout", self.o.shape, self.o.dtype, self.o.device, dense=False)
        self.desc.dout = _rows(dout, "dout")
        check(lstm_attn_bwd(self.desc, self.q, self.k, self.v, self.kv_len, self.key_mask, self.o, self.lse, dout,
                            self.dq, self.dk, self.dv, self.bws, _on(stream, self.q)), "lstm_attn_bwd")


def attn_desc(q, k, v, scale: Optional[float] = None) -> AttnDesc:
    """The description of q [B, Tq, Hq, D], k, v [B, S, Hkv, D] (o like q; gradients left out)."""
    for t, what in ((q, "q"), (k, "k"), (v, "v")):
        if t.dim() != 4:
            raise ValueError(f"{what}: [batch, length, heads, head size], not {tuple(t.shape)}")
    B, Tq, Hq, D = q.shape
    S, Hkv = k.shape[1:3]
    dt = _dtype(q, "q")
    _like(k, "k", (B, S, Hkv, D), q.dtype, q.device, dense=False)
    _like(v, "v", (B, S, Hkv, D), q.dtype, q.device, dense=False)
    if scale is not None and not ctypes.c_float(scale).value > 0:  # (0 would select the default)
        raise ValueError(f"scale: {scale}, must be positive in fp32")
    return AttnDesc(B, Tq, S, Hq, Hkv, D, dt, 0.0 if scale is None else scale, _rows(q, "q"), _rows(k, "k"),
                    _rows(v, "v"))


def prepare_attn(q, k, v, *, kv_len=None, key_mask=None, scale: Optional[float] = None,
                 train: bool = False) -> AttnProblem:
    """Outputs and workspaces for attention of q [B, Tq, Hq, D] over k, v [B, S, Hkv, D].

    The heads' values are contiguous, the other strides free (multiples of 16 bytes): a stack's
    [T][B][H] outputs enter as ``y.view(T, B, heads, D).transpose(0, 1)``.  kv_len [B] int32 and
    key_mask [B, S] (uint8 or bool, 0 leaves a key out) may each be given.  Outputs and gradients
    have the layout of the tensor they belong to.  With train, a bf16 problem also keeps what o's
    rounding leaves (o_rest), from which backward() takes <dout, o>.
    """
    import torch
    desc = attn_desc(q, k, v, scale)
    B, S = desc.B, desc.S
    if kv_len is not None:
        _like(kv_len, "kv_len", (B,), torch.int32, q.device)
    if key_mask is not None:
        key_mask = _bytes(key_mask, "key_mask")
        _like(key_mask, "key_mask", (B, S), torch.uint8, q.device)

    def like(t):
        # dense, the dimensions in the order of t's strides
        order = sorted(range(3), key=lambda i: -t.stride(i)) + [3]
        x = torch.empty([t.shape[i] for i in order], dtype=t.dtype, device=t.device)
        return x.permute([order.index(i) for i in range(4)])

    o = like(q)
    desc.o = _rows(o, "o")
    dq = dk = dv = None
    if train:
        dq, dk, dv = like(q), like(k), like(v)
        desc.dq, desc.dk, desc.dv = _rows(dq, "dq"), _rows(dk, "dk"), _rows(dv, "dv")
    check(lstm_attn_validate(desc, train), "lstm_attn_validate")
    lse = torch.empty((B, desc.Hq, desc.Tq), dtype=torch.float32, device=q.device)
    ws = _workspace(lstm_attn_workspace_size(desc), q.device)
    bws = _workspace(lstm_attn_bwd_workspace_size(desc), q.device) if train else None
    rest = torch.empty(q.shape, dtype=q.dtype, device=q.device) if train and q.dtype == torch.bfloat16 else None
    desc.o_rest = _ptr(rest)
    return AttnProblem(desc, q, k, v, kv_len, key_mask, o, lse, ws, dq, dk, dv, bws, rest)


# ---- beam search --------------------------------------------------------------


def _beam_rows(logits) -> int:
    """Elements from one beam's logits [B, K, V] to the next."""
    B, K, V = logits.shape
    row = logits.stride(1) if K > 1 else (logits.stride(0) if B > 1 else V)
    if (V > 1 and logits.stride(2) != 1) or row < V or (B > 1 and logits.stride(0) != K * row):
        raise ValueError(f"logits: rows of contiguous values at one stride, not strides {tuple(logits.stride())}")
    return row


@dataclass
class BeamProblem(_Problem):
    desc: BeamDesc
    logits: object
    scores: object
    finished: object
    lengths: object
    states: tuple
    tokens: object
    parents: object
    scores_out: object
    finished_out: object
    lengths_out: object
    states_out: tuple
    ws: object

    def _checked(self, name, t):
        import torch
        d, device = self.desc, self.logits.device
        small = {"scores": torch.float32, "lengths": torch.int32, "finished": torch.uint8, "tokens": torch.int32,
                 "parents": torch.int32}
        kind = name[:-4] if name.endswith("_out") else name
        if name == "logits":
            _like(t, name, (d.B, d.K, d.V), self.logits.dtype, device, dense=False)
            d.logits_stride = _beam_rows(t)
        elif kind in small:
            t = _bytes(t, name) if kind == "finished" else t
            _like(t, name, (d.B, d.K), small[kind], device)
        elif kind == "states":
            for x, what, dtype in zip(t, ("h", "c"), (self.logits.dtype, torch.float32), strict=True):
                if x is not None:
                    _like(x, f"{name} {what}", (d.L, d.B * d.K, d.H), dtype, device)
        elif name == "ws":
            self._workspace_like(t, name)
        return t

    def step(self, stream=None) -> None:
        """One selection: tokens, parents, scores_out, finished_out, lengths_out [B, K], states_out."""
        self._runs_on(self.logits.device)
        check(lstm_beam_step(self.desc, self.logits, self.scores, self.finished, self.lengths, self.tokens,
                             self.parents, self.scores_out, self.finished_out, self.lengths_out, self.states[0],
                             self.states[1], self.states_out[0], self.states_out[1], self.ws,
                             _on(stream, self.logits)),
              "lstm_beam_step")

    def advance(self) -> None:
        """Makes the step's outputs the next step's inputs.  The buffers are swapped, not copied: the next
        step() writes over the tensors that this one read, the ones the problem was made with among them."""
        own = self.__dict__
        for name in ("scores", "finished", "lengths", "states"):
            own[name], own[name + "_out"] = own[name + "_out"], own[name]


def prepare_beam(logits, scores, finished, lengths, *, eos: int, alpha: float = 0.0,
                 states=None) -> BeamProblem:
    """Outputs and workspace for beam search steps over logits [B, K, V].

    scores [B, K] fp32, finished [B, K] uint8 or bool, lengths [B, K] int32; states (h, c): h [L, B*K, H]
    of the logits' type, c like it in fp32, each may be None.
    """
    import torch
    if logits.dim() != 3:
        raise ValueError(f"logits: [batch, beams, vocabulary], not {tuple(logits.shape)}")
    B, K, V = logits.shape
    dt = _dtype(logits, "logits")
    dev = logits.device
    row = _beam_rows(logits)
    _like(scores, "scores", (B, K), torch.float32, dev)
    finished = _bytes(finished, "finished")
    _like(finished, "finished", (B, K), torch.uint8, dev)
    _like(lengths, "lengths", (B, K), torch.int32, dev)
    h, c = states if states is not None else (None, None)
    L = H = 0
    for t, what, d in ((h, "states h", logits.dtype), (c, "states c", torch.float32)):
        if t is None:
            continue
        if t.dim() != 3:
            raise ValueError(f"{what}: [layers, batch * beams, width], not {tuple(t.shape)}")
        if L == 0:
            L, H = t.shape[0], t.shape[2]
        _like(t, what, (L, B * K, H), d, dev)
    desc = BeamDesc(B, K, V, dt, eos, alpha, L, H, row)
    n = lstm_beam_workspace_size(desc)
    if n == 0:
        raise ValueError("unsupported problem: lstm_beam_workspace_size returned 0")

    def like(t):
        return None if t is None else torch.empty_like(t)

    return BeamProblem(desc, logits, scores, finished, lengths, (h, c),
                       torch.empty((B, K), dtype=torch.int32, device=dev),
                       torch.empty((B, K), dtype=torch.int32, device=dev), like(scores), like(finished),
                       like(lengths), (like(h), like(c)), _workspace(n, dev))
