"""Norm and rotation of the heads of queries and keys (include/spmm_dynamic.h, "heads").

What comes before the selection of key blocks and the attention over them: each head
normed (where there is a weight) and its pairs of elements turned by the token's
position, in one pass over queries and keys; the same with the new keys and values
written into a cache; and every gradient.

As in the rest of the binding, calls are asynchronous on ``stream`` (default: the
current one), on which their outputs and scratch are allocated, and never synchronise;
:class:`HeadRotation` itself copies its frequencies to the device when it is made.
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import _check, lib
from .dynamic import (_DTYPE, _INT, _UNKNOWN, _Rows, _dense, _elsewhere, _heads, _lent, _like,
                      _raw_stream, _tensor)

__all__ = ["HeadRotation"]


class _HeadsShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("B", "T", "Hq", "Hk", "D", "R")] + [
        ("dtype", ctypes.c_int32), ("weight_dtype", ctypes.c_int32),
        ("interleaved", ctypes.c_int32), ("eps", ctypes.c_float), ("magnitude", ctypes.c_float),
        ("turns", ctypes.c_void_p), ("positions", ctypes.c_void_p), ("p_sb", ctypes.c_int64),
        ("p_st", ctypes.c_int64), ("lengths", ctypes.c_void_p), ("wq", ctypes.c_void_p),
        ("wk", ctypes.c_void_p)]


def _declare():
    vp, i64, S, R = ctypes.c_void_p, ctypes.c_int64, ctypes.POINTER(_HeadsShape), _Rows
    sigs = {
        "spmm_heads_rotate": ([S, R, R, vp, vp, vp], ctypes.c_int),
        "spmm_heads_append": ([S, R, R, R, vp, R, R, i64, vp], ctypes.c_int),
        "spmm_heads_backward_workspace": ([S], i64),
        "spmm_heads_rotate_backward": ([S, R, R, R, R, vp, vp, vp, vp, vp, i64, vp], ctypes.c_int),
    }
    for name, (args, res) in sigs.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = res


_declare()
_BYTES = {torch.float32: 4, torch.bfloat16: 2, torch.float16: 2}
_NONE = _Rows(None, 0, 0, 0)
_Tensor = torch.Tensor


def _rows(t, name, dt, dev):
    """``_heads`` for a tensor of one type, on one device; the usual case at half the time."""
    if type(t) is _Tensor and t.dtype is dt and t.device == dev:
        strides = t.stride()
        if len(strides) == 4:
            sb, st, sh, sd = strides
            at = t.data_ptr()
            if sd == 1 and not ((sb | st | sh) * _BYTES[dt] | at) & 15:
                return _Rows(at, sb, st, sh)
    return _heads(t, name, (dt,), dev)


def _frequencies(R, base, scaling):
    """Radians per position of the R / 2 pairs, and the factor on sines and cosines."""
    how = dict(scaling or {"kind": "none"})
    kind, s = how.pop("kind", None), how.pop("factor", None)
    wants = {"none": (), "linear": (), "base": (),
             "parts": ("original_length", "fast", "slow", "magnitude"),
             "bands": ("original_length", "fast", "slow")}
    if kind not in wants:
        raise ValueError(f"scaling's kind must be one of {sorted(wants)}, got {kind!r}")
    if kind != "none" and not (s is not None and math.isfinite(s) and s > 0):
        raise ValueError(f"scaling {kind!r} needs a positive factor, got {s}")
    length = how.get("original_length")
    if "original_length" in wants[kind] and not (length is not None and 0 < length < math.inf):
        raise ValueError(f"scaling {kind!r} needs a positive original_length, got {length}")
    unknown = sorted(set(how) - set(wants[kind]))
    if unknown:
        raise ValueError(f"scaling {kind!r} does not know {', '.join(unknown)}")
    if kind == "base" and R > 2:
        base = base * s ** (R / (R - 2))
    f = [base ** (-2 * i / R) for i in range(R // 2)]
    if kind == "linear":
        return [x / s for x in f], 1.0
    if kind == "parts":
        # pairs that make more than `fast` turns in the original length stay, those that
        # make fewer than `slow` are slowed by s, in between in proportion to their number
        def pair(turns):
            return R * math.log(length / (math.tau * turns)) / (2 * math.log(base))

        fast, slow = how.get("fast", 32.0), how.get("slow", 1.0)
        if not math.inf > fast >= slow > 0:
            raise ValueError(f"scaling 'parts' needs fast >= slow > 0, got {fast} and {slow}")
        lo = max(0, math.floor(pair(fast)))
        hi = min(R - 1, math.ceil(pair(slow)))
        ramp = [min(1.0, max(0.0, (i - lo) / max(hi - lo, 1e-3))) for i in range(R // 2)]
        magnitude = how.get("magnitude")
        if magnitude is None:
            magnitude = 0.1 * math.log(s) + 1 if s > 1 else 1.0
        return [x * (1 - r) + x / s * r for x, r in zip(f, ramp)], float(magnitude)
    if kind == "bands":
        # the same by the number of turns itself
        fast, slow = how.get("fast", 4.0), how.get("slow", 1.0)
        if not fast > slow:
            raise ValueError(f"scaling 'bands' needs fast > slow, got {fast} and {slow}")
        keep = [min(1.0, max(0.0, (length * x / math.tau - slow) / (fast - slow))) for x in f]
        return [x * m + x / s * (1 - m) for x, m in zip(f, keep)], 1.0
    return f, 1.0


class HeadRotation:
    """The rotation of heads of ``dim`` elements by their token's position.

    The first ``rotary_dim`` elements (None: all) are turned in pairs, element i with
    i + rotary_dim / 2 (``layout`` "half") or 2 i with 2 i + 1 ("interleaved"), by
    position * frequency radians; the others stay. Frequencies are
    ``base ** (-2 i / rotary_dim)``, changed by ``scaling`` for long contexts:

    * ``{"kind": "linear", "factor": s}``: all divided by s;
    * ``{"kind": "base", "factor": s}``: base times s ** (R / (R - 2));
    * ``{"kind": "parts", "factor": s, "original_length": L}``: fast pairs stay, slow ones
      are divided by s, those between ``fast`` (32) and ``slow`` (1) turns in L in
      proportion to their number; sines and cosines times ``magnitude`` (0.1 ln s + 1);
    * ``{"kind": "bands", "factor": s, "original_length": L}``: the same by the number of
      turns in L, between ``slow`` (1) and ``fast`` (4);

    or given: ``frequencies``, rotary_dim / 2 numbers in radians per position, and
    ``magnitude``. Angles are formed in 64-bit integers: a far position costs no accuracy.

    Tensors are [B, T, heads, dim], float32, bfloat16 or float16, with adjacent elements
    in a row and rows at 16-byte boundaries; dim and rotary_dim multiples of 16, dim at
    most 256. Token t of sequence b is at ``positions`` (int32 [B, T] or [T]), or with
    ``lengths`` (int32 [B]; the tokens are each sequence's last, as in a selection) at
    lengths[b] - T + t, or at t. With ``q_weight`` / ``k_weight`` ([dim], float32 or the
    tensors' type) that tensor's heads are first normed: x * weight / sqrt(mean(x^2) + eps).
    """

    def __init__(self, dim: int, rotary_dim: int | None = None, layout: str = "half",
                 base: float = 10000.0, scaling: dict | None = None, frequencies=None,
                 magnitude: float | None = None, device="cuda"):
        R = dim if rotary_dim is None else rotary_dim
        if dim % 16 or not 16 <= dim <= 256:
            raise ValueError(f"the width of a head must be a multiple of 16 up to 256, got {dim}")
        if R % 16 or not 0 <= R <= dim:
            raise ValueError(f"rotary_dim must be a multiple of 16 up to {dim}, got {R}")
        if layout not in ("half", "interleaved"):
            raise ValueError(f"layout must be 'half' or 'interleaved', got {layout!r}")
        if frequencies is None:
            if not (math.isfinite(base) and base > 1):
                raise ValueError(f"base must be above 1, got {base}")
            f, m = _frequencies(R, float(base), scaling)
        else:
            if scaling is not None:
                raise ValueError("frequencies are given: scaling must be None")
            f, m = [float(x) for x in frequencies], 1.0
            if len(f) != R // 2 or not all(math.isfinite(x) for x in f):
                raise ValueError(f"frequencies must be {R // 2} finite numbers")
        self.dim, self.rotary_dim, self.layout = int(dim), int(R), layout
        self.frequencies = f
        self.magnitude = m if magnitude is None else float(magnitude)
        if not math.isfinite(self.magnitude):
            raise ValueError(f"magnitude must be finite, got {self.magnitude}")
        turns = [round(x / math.tau % 1.0 * 2 ** 64) % 2 ** 64 for x in f]
        turns = [x - 2 ** 64 if x >= 2 ** 63 else x for x in turns]
        device = torch.device(device)
        if device.type != "cuda":
            raise ValueError("device must be a CUDA device (there is no CPU path)")
        with torch.cuda.device(device):
            self.turns = torch.tensor(turns, dtype=torch.int64).to(device)
        self._tell(_raw_stream(self.turns.device.index))
        self._interleaved = 1 if layout == "interleaved" else 0
        self._weight_shape = (self.dim,)

    def _tell(self, stream):
        """Where the frequencies are, and the stream they were made on."""
        self.device = self.turns.device
        self._turns = self.turns.data_ptr() or None
        self._stream = stream

    def __setstate__(self, state):
        # (a copy, as a model's are made, or what a file held: its tensor is another)
        self.__dict__.update(state)
        self._tell(_UNKNOWN)

    def _on_stream(self):
        """The current stream, which the frequencies are now used on."""
        stream = _raw_stream(self.device.index)
        if stream != self._stream:
            _lent(self.device, self.turns)
            if self._stream == _UNKNOWN:
                self._stream = stream
        return stream

    def _weight(self, w, name, dtype):
        """A weight's address."""
        if type(w) is not _Tensor or not (w.dtype is dtype or w.dtype is torch.float32) or \
                w.shape != self._weight_shape or w.device != self.device or not w.is_contiguous():
            _dense(w, name, (dtype, torch.float32), self._weight_shape, self.device)
        at = w.data_ptr()
        if at & 15:
            raise ValueError(f"{name} must start at a 16-byte boundary")
        return at

    def _problem(self, q, k, positions, lengths, q_weight, k_weight, eps):
        """The call's shape, and the rows of q and k."""
        dev = self.device
        dtype = getattr(q, "dtype", None)
        rows = _rows(q, "q", dtype, dev) if dtype in _DTYPE else _heads(q, "q", _DTYPE, dev)
        B, T, Hq, D = q.shape
        Hk, krows = 0, _NONE
        if k is not None:
            krows = _rows(k, "k", dtype, dev)
            Bk, Tk, Hk, Dk = k.shape
            if Bk != B or Tk != T or Dk != D:
                raise ValueError(f"k must be [{B}, {T}, heads, {D}], got {list(k.shape)}")
        elif k_weight is not None:
            raise ValueError("k_weight is given without k")
        if D != self.dim:
            raise ValueError(f"the width of a head must be {self.dim}, got {D}")
        at = lat = wq = wk = None
        sb = st = 0
        if lengths is not None:
            if positions is not None:
                raise ValueError("give positions or lengths, not both")
            if type(lengths) is not _Tensor or lengths.dtype is not torch.int32 or \
                    lengths.shape != (B,) or lengths.device != dev or not lengths.is_contiguous():
                _dense(lengths, "lengths", _INT, (B,), dev)
            lat = lengths.data_ptr() or None
        elif positions is not None:
            if not isinstance(positions, _Tensor):
                raise TypeError("positions must be a torch.Tensor")
            n = positions.dim()
            _tensor(positions, "positions", _INT, 1 if n == 1 else 2, dev)
            if positions.shape != ((T,) if n == 1 else (B, T)):
                raise ValueError(f"positions must be [{B}, {T}] or [{T}], got "
                                 f"{list(positions.shape)}")
            strides = positions.stride()
            st = strides[-1]
            if n == 2:
                sb = strides[0]
            at = positions.data_ptr() or None
        dt = wt = _DTYPE[dtype]
        if q_weight is not None:
            wq = self._weight(q_weight, "q_weight", dtype)
            wt = _DTYPE[q_weight.dtype]
        if k_weight is not None:
            wk = self._weight(k_weight, "k_weight", dtype)
            if wq is not None and k_weight.dtype is not q_weight.dtype:
                raise TypeError("q_weight and k_weight must have one type, got "
                                f"{q_weight.dtype} and {k_weight.dtype}")
            wt = _DTYPE[k_weight.dtype]
        return _HeadsShape(B, T, Hq, Hk, D, self.rotary_dim, dt, wt, self._interleaved, eps,
                           self.magnitude, self._turns, at, sb, st, lat, wq, wk), rows, krows

    def rotate(self, q, k=None, positions=None, lengths=None, q_weight=None, k_weight=None,
               eps: float = 1e-6, stream=None):
        """(q', k'): queries and keys normed and turned, contiguous; k' is None without k."""
        ctx = _elsewhere(self.device, stream)
        if ctx is not None:
            with ctx:
                got = self.rotate(q, k, positions, lengths, q_weight, k_weight, eps)
                _lent(self.device, q, k, positions, lengths, q_weight, k_weight)
                return got
        s, rows, krows = self._problem(q, k, positions, lengths, q_weight, k_weight, eps)
        q2 = _like(q)
        k2 = None if k is None else _like(k)
        st = lib.spmm_heads_rotate(s, rows, krows, q2.data_ptr(),
                                   None if k2 is None else k2.data_ptr(), self._on_stream())
        if st:
            _check(st, "spmm_heads_rotate")
        return q2, k2

    def append(self, q, k, v, cache_k, cache_v, lengths, q_weight=None, k_weight=None,
               eps: float = 1e-6, stream=None):
        """q' as ``rotate`` gives it; the new keys, normed and turned, and the values as they are
        go to their positions in the caches [B, rows, Hk, dim] (any strides as the inputs').

        ``lengths``: each sequence's keys with the new ones, its last T. Keys at positions
        outside the cache (before the sequence's start, past its rows) are not written, and
        no other row is. The caches overlap neither each other nor q, k and v."""
        ctx = _elsewhere(self.device, stream)
        if ctx is not None:
            with ctx:
                got = self.append(q, k, v, cache_k, cache_v, lengths, q_weight, k_weight, eps)
                _lent(self.device, q, k, v, cache_k, cache_v, lengths, q_weight, k_weight)
                return got
        if k is None or lengths is None:
            raise ValueError("append needs k and lengths")
        s, rows, krows = self._problem(q, k, None, lengths, q_weight, k_weight, eps)
        dev, dt, shape = self.device, q.dtype, k.shape
        vrows = _rows(v, "v", dt, dev)
        if v.shape != shape:
            raise ValueError(f"v must be {list(shape)}, got {list(v.shape)}")
        ck, cv = _rows(cache_k, "cache_k", dt, dev), _rows(cache_v, "cache_v", dt, dev)
        want = cache_k.shape
        B, Tk, Hk, D = want
        if cache_v.shape != want or (B, Hk, D) != (shape[0], shape[2], shape[3]):
            raise ValueError(f"cache_k and cache_v must be [{s.B}, rows, {s.Hk}, {s.D}], got "
                             f"{list(want)} and {list(cache_v.shape)}")
        if ck.data == cv.data and cache_k.numel():
            raise ValueError("cache_k and cache_v are in one place")
        for c, name in ((cache_k, "cache_k"), (cache_v, "cache_v")):
            strides = c.stride()
            if 0 in strides and any(n > 1 and x == 0 for n, x in zip(want, strides)):
                raise ValueError(f"{name} has rows that share memory (strides {strides})")
        q2 = _like(q)
        st = lib.spmm_heads_append(s, rows, krows, vrows, q2.data_ptr(), ck, cv, Tk,
                                   self._on_stream())
        if st:
            _check(st, "spmm_heads_append")
        return q2

    def _input(self, x, grad, name):
        """The rows of the forward's input for its weight's gradient."""
        if x is None:
            raise ValueError(f"the gradient of {name}_weight needs {name}")
        rows = _rows(x, name, grad.dtype, self.device)
        if x.shape != grad.shape:
            raise ValueError(f"{name} must be {list(grad.shape)}, got {list(x.shape)}")
        return rows

    def rotate_backward(self, grad_q, grad_k, q=None, k=None, positions=None, lengths=None,
                        q_weight=None, k_weight=None, eps: float = 1e-6, stream=None):
        """(dq, dk, dq_weight, dk_weight) of ``rotate(q, k, ...)``, given the gradients of its
        results. q and k are needed where there is a weight; dk is None without grad_k, a
        weight's gradient None without the weight (and of its type)."""
        ctx = _elsewhere(self.device, stream)
        if ctx is not None:
            with ctx:
                grads = self.rotate_backward(grad_q, grad_k, q, k, positions, lengths, q_weight,
                                             k_weight, eps)
                _lent(self.device, grad_q, grad_k, q, k, positions, lengths, q_weight, k_weight)
                return grads
        s, gq, gk = self._problem(grad_q, grad_k, positions, lengths, q_weight, k_weight, eps)
        xq = xk = _NONE
        dk = dwq = dwk = work = None
        need = 0
        if q_weight is not None:
            xq = self._input(q, grad_q, "q")
            dwq = torch.empty_like(q_weight)
        if k_weight is not None:
            xk = self._input(k, grad_k, "k")
            dwk = torch.empty_like(k_weight)
        dq = _like(grad_q)
        if grad_k is not None:
            dk = _like(grad_k)
        if dwq is not None or dwk is not None:
            need = lib.spmm_heads_backward_workspace(s)
            work = torch.empty(need, dtype=torch.uint8, device=self.device)
        st = lib.spmm_heads_rotate_backward(
            s, gq, gk, xq, xk, dq.data_ptr(), None if dk is None else dk.data_ptr(),
            None if dwq is None else dwq.data_ptr(), None if dwk is None else dwk.data_ptr(),
            None if work is None else work.data_ptr(), need, self._on_stream())
        if st:
            _check(st, "spmm_heads_rotate_backward")
        return dq, dk, dwq, dwk
