"""What a tuple of tensors was when it was looked at: each one's address, number of elements, type and contiguity.

    held = Held(tensors)       # raises for what is not a tensor
    held.same()                # whether all of it still holds: 8 ns a tensor

A tensor's ``.data`` may be set, and ``resize_`` and ``set_`` change it in place, so an object that was checked once
need not be what it was, at the same address either.
"""
from __future__ import annotations

import ctypes
import os

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "lib", "liblstm_held.so")
_lib = None


def load_library() -> ctypes.PyDLL:
    """Load lib/liblstm_held.so (raises if it is not built, or built for another torch)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is not built; run `python -m stacked_lstm_forward_amd.build`")
    import torch
    lib = ctypes.PyDLL(LIB_PATH)
    lib.lstm_held_torch.restype = ctypes.c_char_p
    built = lib.lstm_held_torch().decode()
    if built != torch.__version__.split("+")[0]:
        raise RuntimeError(f"{LIB_PATH} is built for torch {built}, not {torch.__version__}: build it again")
    for name in ("lstm_held_read", "lstm_held_same"):
        f = getattr(lib, name)
        f.argtypes, f.restype = [ctypes.py_object, ctypes.c_void_p], ctypes.c_int
    _lib = lib
    return lib


class Held:
    def __init__(self, tensors):
        self._tensors = tuple(tensors)
        self._was = (ctypes.c_int64 * (3 * len(self._tensors)))()
        self._same = load_library().lstm_held_same
        self.read()

    def read(self) -> None:
        """Takes what the tensors are now."""
        if not load_library().lstm_held_read(self._tensors, self._was):
            raise TypeError("tensors whose memory can be read, and nothing else")

    def same(self) -> bool:
        return bool(self._same(self._tensors, self._was))
