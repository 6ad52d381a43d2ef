"""Products whose sparse matrix a model chooses anew in every call (include/spmm_dynamic.h).

* :class:`ExpertRoutes` -- the tokens x slots matrix of a router: tokens sorted
  by expert and gathered (``dispatch``), the experts' rows weighted and added
  back per token (``combine``), and every gradient.
* :func:`block_means`, :func:`select_blocks`, :class:`BlockSelection` -- the
  queries x key-blocks matrix of a cheap score, attention over the selected
  blocks (many queries, or single tokens over a cache) and its gradient.

Like the rest of the binding this marshals arguments only; the computation runs
in the CUDA library. Calls are asynchronous on ``stream`` (default: the current
one), on which their outputs and scratch are allocated, and never synchronise,
except the check of lists that a caller made (``BlockSelection(validate=True)``).
Ordering streams is the caller's: a call does not wait for the work that made its
inputs on another one. What a call on a given stream reads, and what routes and
selections hold, keeps its memory until that stream is done with it.
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import SpmmError, _check, lib

__all__ = ["ExpertRoutes", "BlockSelection", "block_means", "select_blocks",
           "dynamic_sync", "ROUTES_MAX_EXPERTS", "BLOCK_SIZES"]

ROUTES_MAX_EXPERTS = 2048
BLOCK_SIZES = (16, 32, 64, 128)

# A small call's time is mostly the host's: the current device and stream are
# read directly (0.15 us; building a torch.cuda.Stream object takes 3 us), and
# each check below costs one attribute access.
_current_device = torch._C._cuda_getDevice
_raw_stream = torch._C._cuda_getCurrentRawStream


class _Rows(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("sb", ctypes.c_int64), ("st", ctypes.c_int64),
                ("sh", ctypes.c_int64)]


class _Shape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("B", "Tq", "Tk", "Hq", "Hk", "D", "block", "n")] + [
        ("dtype", ctypes.c_int32), ("causal", ctypes.c_int32), ("scale", ctypes.c_float),
        ("lengths", ctypes.c_void_p)]


def _declare():
    vp, i64, i32, S = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.POINTER(_Shape)
    sigs = {
        "spmm_dynamic_sync": ([vp], i32),
        "spmm_dynamic_check_wait_timeout": ([i64, vp], i32),
        "spmm_routes_workspace": ([i64] * 3, i64),
        "spmm_routes_sort": ([vp, i64, i64, i64, vp, vp, vp, i64, vp], i32),
        "spmm_routes_dispatch": ([i32, vp, i64, vp, vp, i64, i64, i64, i64, vp, vp], i32),
        "spmm_routes_combine": ([i32, vp, vp, vp, vp, i64, i64, i64, i64, vp, vp], i32),
        "spmm_routes_combine_backward": ([i32, vp, i64, vp, vp, vp, vp, i64, i64, i64, i64, vp, vp,
                                          vp], i32),
        "spmm_blocks_means": ([S, _Rows, i64, vp, vp], i32),
        "spmm_blocks_select_workspace": ([S], i64),
        "spmm_blocks_select": ([S, _Rows, vp, vp, vp, i64, vp], i32),
        "spmm_blocks_select_kept": ([S, _Rows, vp, vp, vp, vp, i64, vp], i32),
        "spmm_blocks_check": ([S, vp, vp, vp], i32),
        "spmm_blocks_attend": ([S, _Rows, _Rows, _Rows, vp, vp, vp, vp], i32),
        "spmm_blocks_backward_workspace": ([S], i64),
        "spmm_blocks_backward": ([S, _Rows, _Rows, _Rows, vp, vp, vp, _Rows, vp, vp, vp, vp, i64,
                                  vp], i32),
    }
    for name, (args, res) in sigs.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = res


_declare()
_DTYPE = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
_INT, _FLOAT, _HALVES = (torch.int32,), (torch.float32,), (torch.bfloat16, torch.float16)


def _elsewhere(dev, stream):
    """A context in which `dev` and `stream` are current, or None if they are."""
    if stream is None:
        return None if _current_device() == dev.index else torch.cuda.device(dev)
    if stream.device != dev:
        raise ValueError(f"stream is on {stream.device}, expected {dev}")
    return torch.cuda.stream(stream)


def _lent(dev, *tensors):
    """The current stream uses them: their memory is not handed out before it is done."""
    stream = torch.cuda.current_stream(dev)
    for t in tensors:
        if t is not None:
            t.record_stream(stream)


def _tensor(t, name, dtypes, ndim, dev=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (there is no CPU path)")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dimensions, got {tuple(t.shape)}")
    if dev is not None and t.device != dev:
        raise ValueError(f"{name} is on {t.device}, expected {dev}")
    return t


def _dense(t, name, dtypes, shape, dev):
    _tensor(t, name, dtypes, len(shape), dev)
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def dynamic_sync(stream=None) -> None:
    """Wait for the stream; SpmmError (SPMM_ERR_TIMEOUT) if a bounded device-side wait of
    one of these calls on it, or of one in a captured graph, gave up since it was last asked."""
    if stream is not None and stream.device.index != _current_device():
        with torch.cuda.device(stream.device):
            return dynamic_sync(stream)
    handle = _raw_stream(_current_device()) if stream is None else stream.cuda_stream
    _check(lib.spmm_dynamic_sync(handle), "spmm_dynamic_sync")


def _scratch(like, need):
    return like.new_empty(need, dtype=torch.uint8) if need else None


# -------------------------------------------------------------------- routes
class ExpertRoutes:
    """The routes of T tokens to k of E experts each, sorted by expert.

    ``ids`` int32 [T, k], contiguous: the expert of each choice; a value outside
    [0, E) drops the pair. Afterwards

    * ``slots`` int32 [T, k]: the pair's row among the kept pairs in order of
      (expert, token, choice), -1 for a dropped pair;
    * ``offsets`` int32 [E + 1]: expert e's rows are [offsets[e], offsets[e + 1]).

    Row tensors are float32, bfloat16 or float16. ``x`` and ``grad`` are [T, H]
    with adjacent elements in a row and any row stride; tensors by slot are
    [T * k, H], contiguous, of which the rows from offsets[E] on belong to no
    pair: they are written as 0 and never read.
    """

    def __init__(self, ids, num_experts: int, stream=None):
        _tensor(ids, "ids", _INT, 2)
        if not ids.is_contiguous():
            raise ValueError("ids must be contiguous")
        E = int(num_experts)
        if not 0 <= E <= ROUTES_MAX_EXPERTS:
            raise ValueError(f"num_experts must be in [0, {ROUTES_MAX_EXPERTS}], got {E}")
        self.device = dev = ids.device
        self.num_experts = E
        self.T, self.k = ids.shape
        ctx = _elsewhere(dev, stream)
        if ctx is None:
            self._sort(ids)
        else:
            with ctx:
                self._sort(ids)
                _lent(dev, ids)

    def _sort(self, ids):
        T, k, E = self.T, self.k, self.num_experts
        self._stream = stream = _raw_stream(self.device.index)
        self.slots = torch.empty_like(ids)
        self.offsets = ids.new_empty(E + 1)
        need = lib.spmm_routes_workspace(T, k, E)
        work = _scratch(ids, need)
        # what every product's call begins its list of routes with
        self._routes = (self.slots.data_ptr(), self.offsets.data_ptr(), T, k, E)
        st = lib.spmm_routes_sort(ids.data_ptr(), T, k, E, *self._routes[:2],
                                  None if work is None else work.data_ptr(), need, stream)
        if st:
            _check(st, "spmm_routes_sort")

    def _on_stream(self):
        """The current stream, which the routes' own tensors are now used on."""
        stream = _raw_stream(self.device.index)
        if stream != self._stream:
            _lent(self.device, self.slots, self.offsets)
        return stream

    def _by_token(self, x, name):
        _tensor(x, name, _DTYPE, 2, self.device)
        T, H = x.shape
        if T != self.T:
            raise ValueError(f"{name} must be [{self.T}, H], got {list(x.shape)}")
        ld, step = x.stride()
        if step != 1 and H > 1:
            raise ValueError(f"{name} must have adjacent elements in a row")
        return H, ld

    def _by_slot(self, y, name, H=None):
        _tensor(y, name, _DTYPE, 2, self.device)
        P, width = y.shape
        if P != self.T * self.k or (H is not None and width != H):
            raise ValueError(f"{name} must be [{self.T * self.k}, {'H' if H is None else H}], "
                             f"got {list(y.shape)}")
        if not y.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        return width

    def _weights(self, w):
        if w is None:
            return None
        return _dense(w, "weights", _FLOAT, (self.T, self.k), self.device).data_ptr()

    def dispatch(self, x, stream=None):
        """xs [T * k, H]: token t's row at each of its slots."""
        ctx = _elsewhere(self.device, stream)
        if ctx is not None:
            with ctx:
                xs = self.dispatch(x)
                _lent(self.device, x)
                return xs
        H, ld = self._by_token(x, "x")
        xs = x.new_empty((self.T * self.k, H))
        st = lib.spmm_routes_dispatch(_DTYPE[x.dtype], x.data_ptr(), ld, *self._routes, H,
                                      xs.data_ptr(), self._on_stream())
        if st:
            _check(st, "spmm_routes_dispatch")
        return xs

    def combine(self, y, weights=None, stream=None):
        """out [T, H]: sum over j of weights[t, j] (float32; None: 1) times y at the slot of
        (t, j), summed in fp32 in the order of j."""
        ctx = _elsewhere(self.device, stream)
        if ctx is not None:
            with ctx:
                out = self.combine(y, weights)
                _lent(self.device, y, weights)
                return out
        H = self._by_slot(y, "y")
        w = self._weights(weights)
        out = y.new_empty((self.T, H))
        st = lib.spmm_routes_combine(_DTYPE[y.dtype], y.data_ptr(), w, *self._routes, H,
                                     out.data_ptr(), self._on_stream())
        if st:
            _check(st, "spmm_routes_combine")
        return out

    def dispatch_backward(self, grad, stream=None):
        """The gradient of ``dispatch`` with respect to x, given that of xs."""
        return self.combine(grad, None, stream)

    def combine_backward(self, grad, y, weights=None, stream=None):
        """(dy [T * k, H], dweights float32 [T, k]) of ``combine(y, weights)``, given the
        gradient [T, H] of its result; dweights is None without weights."""
        ctx = _elsewhere(self.device, stream)
        if ctx is not None:
            with ctx:
                grads = self.combine_backward(grad, y, weights)
                _lent(self.device, grad, y, weights)
                return grads
        H, ld = self._by_token(grad, "grad")
        self._by_slot(y, "y", H)
        if y.dtype != grad.dtype:
            raise TypeError(f"y must be {grad.dtype}, got {y.dtype}")
        w = self._weights(weights)
        dy = torch.empty_like(y)
        dw = None if w is None else torch.empty_like(weights)
        st = lib.spmm_routes_combine_backward(
            _DTYPE[y.dtype], grad.data_ptr(), ld, y.data_ptr(), w, *self._routes, H, dy.data_ptr(),
            None if dw is None else dw.data_ptr(), self._on_stream())
        if st:
            _check(st, "spmm_routes_combine_backward")
        return dy, dw


# -------------------------------------------------------------------- blocks
def _heads(t, name, dtypes, dev=None):
    """The rows of a [B, T, heads, D] tensor: adjacent elements at 16-byte boundaries."""
    _tensor(t, name, dtypes, 4, dev)
    sb, st, sh, sd = t.stride()
    at, e = t.data_ptr(), t.element_size()
    if ((sb | st | sh) * e | at) % 16 or (sd != 1 and t.shape[3] > 1):
        # the stride of a dimension of one means nothing, and may be any number
        sb, st, sh = (0 if n == 1 else x for n, x in zip(t.shape, (sb, st, sh)))
        if t.numel() and (((sb | st | sh) * e | at) % 16 or (sd != 1 and t.shape[3] > 1)):
            raise ValueError(f"{name} must have adjacent elements in a row and rows at 16-byte "
                             f"boundaries (strides {tuple(t.stride())})")
    return _Rows(at, sb, st, sh)


def _block_size(block):
    if block not in BLOCK_SIZES:
        raise ValueError(f"block must be one of {BLOCK_SIZES}, got {block}")
    return int(block)


def _lengths_ptr(lengths, B, dev):
    return None if lengths is None else _dense(lengths, "lengths", _INT, (B,), dev).data_ptr()


def block_means(k, block: int = 64, lengths=None, out=None, new_keys: int | None = None,
                stream=None):
    """float32 [B, ceil(Tk / block), Hk, D]: the mean of each block's valid keys (0 for none).

    ``k`` [B, Tk, Hk, D]; sequence b holds lengths[b] keys (int32 [B]; None: Tk). With
    ``new_keys`` and ``out`` (the means so far) only the blocks that hold one of each
    sequence's last new_keys keys are computed again, after those keys were appended."""
    rows = _heads(k, "k", _DTYPE)
    dev = k.device
    ctx = _elsewhere(dev, stream)
    if ctx is not None:
        with ctx:
            means = block_means(k, block, lengths, out, new_keys)
            _lent(dev, k, lengths, out)
            return means
    B, Tk, Hk, D = k.shape
    block = _block_size(block)
    if D % 8 or not 8 <= D <= 256:
        raise ValueError(f"the width of a key must be a multiple of 8 up to 256, got {D}")
    shape = (B, -(-Tk // block), Hk, D)
    if new_keys is not None and (out is None or new_keys < 0):
        raise ValueError("new_keys (>= 0) updates the means given as out")
    if out is None:
        out = k.new_empty(shape, dtype=torch.float32)
    else:
        _dense(out, "out", _FLOAT, shape, dev)
    s = _Shape(B, 1, Tk, Hk, Hk, D, block, 1, _DTYPE[k.dtype], 1, 1.0,
               _lengths_ptr(lengths, B, dev))
    st = lib.spmm_blocks_means(s, rows, -1 if new_keys is None else new_keys, out.data_ptr(),
                               _raw_stream(dev.index))
    if st:
        _check(st, "spmm_blocks_means")
    return out


def select_blocks(q, means, n: int, block: int, num_keys: int, lengths=None, causal: bool = True,
                  stream=None) -> "BlockSelection":
    """The blocks each query attends to: ``BlockSelection`` with lists of n entries.

    ``q`` [B, Tq, Hq, D], ``means`` from :func:`block_means` over ``num_keys`` keys. The
    score of a block is (the sum of the group's query rows) . (its mean key), in fp32.
    Query i is at position lengths[b] - Tq + i; causal lists hold the block of that
    position and the n - 1 best ones before it, others the n best of the sequence's
    blocks. Ties go to the lowest block."""
    rows = _heads(q, "q", _DTYPE)
    dev = q.device
    ctx = _elsewhere(dev, stream)
    if ctx is not None:
        with ctx:
            sel = select_blocks(q, means, n, block, num_keys, lengths, causal)
            _lent(dev, q, means, lengths)
            return sel
    B, Tq, Hq, D = q.shape
    block, n, Tk = _block_size(block), int(n), int(num_keys)
    _tensor(means, "means", _FLOAT, 4, dev)
    Hk = means.shape[2]
    if n < 1 or Tk < 0:
        raise ValueError(f"n must be at least 1 and num_keys at least 0, got {n} and {Tk}")
    if Hk < 1 or Hq % Hk:
        raise ValueError(f"{Hq} query heads do not divide into {Hk} groups")
    if D % 8 or not 8 <= D <= 256:
        raise ValueError(f"the width of a query must be a multiple of 8 up to 256, got {D}")
    _dense(means, "means", _FLOAT, (B, -(-Tk // block), Hk, D), dev)
    s = _Shape(B, Tq, Tk, Hq, Hk, D, block, n, _DTYPE[q.dtype], 1 if causal else 0, 1.0,
               _lengths_ptr(lengths, B, dev))
    sel = BlockSelection.__new__(BlockSelection)
    shape = (B, Tq, Hk, n)
    if lengths is None or not Tq:
        sel._set(q.new_empty(shape, dtype=torch.int32), shape, block, Tk, causal)
        if lengths is not None:
            sel._keep(lengths)
    else:
        # room for the call's copy of lengths behind the lists: a second allocation takes
        # longer than the views that are made of this one when they are asked for
        rows_ = B * Tq * Hk
        sel._set(q.new_empty(rows_ * n + B, dtype=torch.int32), shape, block, Tk, causal)
        sel._lengths = sel._lists + 4 * rows_ * n
    need = lib.spmm_blocks_select_workspace(s)
    work = _scratch(q, need)
    st = lib.spmm_blocks_select_kept(s, rows, means.data_ptr() or None, sel._lists, sel._lengths,
                                     None if work is None else work.data_ptr(), need,
                                     _raw_stream(dev.index))
    if st:
        _check(st, "spmm_blocks_select")
    return sel


class BlockSelection:
    """The key blocks that each query (per kv head) attends to, and the attention.

    ``blocks`` int32 [B, Tq, Hk, n]: strictly ascending block numbers, then -1.
    ``lengths`` int32 [B] (None: num_keys): the valid keys of each sequence, whose Tq
    queries are its last tokens. Causal, a query sees the keys up to its position.
    ``validate=True`` checks the lists (it synchronises).

    A selection has a copy of its lengths (a decode loop may add to its own in place);
    given ``blocks`` are not copied."""

    def __init__(self, blocks, block: int, num_keys: int, lengths=None, causal: bool = True,
                 validate: bool = True):
        _tensor(blocks, "blocks", _INT, 4)
        if not blocks.is_contiguous():
            raise ValueError("blocks must be contiguous")
        B, Tq, Hk, n = blocks.shape
        num_keys = int(num_keys)
        if Hk < 1 or n < 1 or num_keys < 0:
            raise ValueError(f"blocks must be [B, Tq, Hk >= 1, n >= 1], got {list(blocks.shape)}")
        _lengths_ptr(lengths, B, blocks.device)                 # its checks
        with torch.cuda.device(blocks.device):
            self._set(blocks, (B, Tq, Hk, n), _block_size(block), num_keys, causal)
            if lengths is not None:
                self._keep(lengths)
            if validate:
                bad = blocks.new_empty(1)
                s = _Shape(B, Tq, num_keys, Hk, Hk, 64, self.block, n, 1, int(self.causal), 1.0,
                           self._lengths)
                _check(lib.spmm_blocks_check(s, self._lists or None, bad.data_ptr(),
                                             _raw_stream(self.device.index)), "spmm_blocks_check")
                if int(bad.item()):
                    raise SpmmError(2, "a list of blocks is not strictly ascending block numbers "
                                       "followed by -1")

    def _set(self, lists, shape, block, num_keys, causal):
        """`lists`: the blocks, or one dimension of them with the lengths behind."""
        self.device, self._mem, self._lists = lists.device, lists, lists.data_ptr()
        self._shape, self.block, self.num_keys = shape, block, num_keys
        self.causal, self._lengths, self._kept = bool(causal), None, None
        self._stream = _raw_stream(self.device.index)

    def _on_stream(self):
        """The current stream, which the selection's own tensors are now used on."""
        stream = _raw_stream(self.device.index)
        if stream != self._stream:
            _lent(self.device, self._mem, self._kept)
        return stream

    def _keep(self, lengths):
        self._kept = lengths.clone()
        self._lengths = self._kept.data_ptr()

    @property
    def blocks(self):
        """int32 [B, Tq, Hk, n]"""
        if self._mem.dim() == 4:
            return self._mem
        B, Tq, Hk, n = self._shape
        return self._mem.as_strided(self._shape, (Tq * Hk * n, Hk * n, n, 1))

    @property
    def lengths(self):
        """int32 [B], or None"""
        if self._kept is None and self._lengths is not None:
            self._kept = self._mem[self._mem.numel() - self._shape[0]:]
        return self._kept

    def _problem(self, q, k, v, scale):
        """The call's shape, and the rows of q, k and v."""
        dev = self.device
        rows = (_heads(q, "q", _HALVES, dev), _heads(k, "k", (q.dtype,), dev),
                _heads(v, "v", (q.dtype,), dev))
        B, Tq, Hk, n = self._shape
        Bq, T, Hq, D = q.shape
        if Bq != B or T != Tq or Hq % Hk or Hq < 1:
            raise ValueError(f"q must be [{B}, {Tq}, a multiple of {Hk}, D], got {list(q.shape)}")
        if D != 64 and D != 128:
            raise ValueError(f"the width of a head must be 64 or 128, got {D}")
        want = (B, self.num_keys, Hk, D)
        if k.shape != want or v.shape != want:
            raise ValueError(f"k and v must be {list(want)}, got {list(k.shape)} and "
                             f"{list(v.shape)}")
        scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
        return _Shape(B, Tq, self.num_keys, Hq, Hk, D, self.block, n, _DTYPE[q.dtype],
                      1 if self.causal else 0, scale, self._lengths), rows

    def attend(self, q, k, v, scale: float | None = None, stream=None):
        """(out [B, Tq, Hq, D], lse float32 [B, Tq, Hq]): softmax attention over the seen keys of
        each query's blocks; lse is the natural logarithm of the sum of exp(scale q . k)
        (scale None: 1 / sqrt(D)). A query that sees no key gives 0 and -inf.

        q, k, v: bfloat16 or float16, D 64 or 128, k and v [B, num_keys, Hk, D]; any
        strides with adjacent elements in a row and rows at 16-byte boundaries."""
        ctx = _elsewhere(self.device, stream)
        if ctx is not None:
            with ctx:
                got = self.attend(q, k, v, scale)
                _lent(self.device, q, k, v)
                return got
        s, rows = self._problem(q, k, v, scale)
        out = q.new_empty(q.shape)
        lse = q.new_empty(q.shape[:3], dtype=torch.float32)
        st = lib.spmm_blocks_attend(s, *rows, self._lists, out.data_ptr(),
                                    lse.data_ptr(), self._on_stream())
        if st:
            _check(st, "spmm_blocks_attend")
        return out, lse

    def backward(self, grad, q, k, v, out, lse, scale: float | None = None, stream=None):
        """(dq, dk, dv) of ``attend(q, k, v, scale)`` = (out, lse), given the gradient of out.
        The selection is a constant; keys that nothing attends to get 0."""
        ctx = _elsewhere(self.device, stream)
        if ctx is not None:
            with ctx:
                grads = self.backward(grad, q, k, v, out, lse, scale)
                _lent(self.device, grad, q, k, v, out, lse)
                return grads
        s, rows = self._problem(q, k, v, scale)
        g = _heads(grad, "grad", (q.dtype,), self.device)
        if grad.shape != q.shape:
            raise ValueError(f"grad must be {list(q.shape)}, got {list(grad.shape)}")
        _dense(out, "out", (q.dtype,), q.shape, self.device)
        _dense(lse, "lse", _FLOAT, q.shape[:3], self.device)
        dq, dk, dv = q.new_empty(q.shape), k.new_empty(k.shape), v.new_empty(v.shape)
        need = lib.spmm_blocks_backward_workspace(s)
        work = _scratch(q, need)
        st = lib.spmm_blocks_backward(s, *rows, self._lists, out.data_ptr(),
                                      lse.data_ptr(), g, dq.data_ptr(), dk.data_ptr(),
                                      dv.data_ptr(), None if work is None else work.data_ptr(),
                                      need, self._on_stream())
        if st:
            _check(st, "spmm_blocks_backward")
        return dq, dk, dv
