"""Python binding of libslotkv: batched decode attention over slot KV on GB300.

Argument marshalling only.  Every step of the decode attention runs in the
library's CUDA kernels; PyTorch supplies device memory and streams.  There is
no CPU fallback: importing this package raises if ``libslotkv.so`` has not
been built (``__graft_entry__.build()`` or ``python -m
sequence_slot_kv_gb300.build``).

The functions mirror the C ABI in ``include/slotkv.h`` name for name
(``EXPORTS`` lists every symbol): the handle (``slot_kv_alloc``,
``slot_kv_free``, ``slot_kv_offset_bytes``, ``slot_kv_reset``), the step
(``decode_batch_attn``, its host-buffer form ``decode_batch_attn_host``,
``prefill_batch_attn`` and its host-buffer form ``prefill_batch_attn_host``
(with ``slot_kv_prefill_host_parts``), ``decode_batch_attn_paged`` and its
host-buffer form ``decode_batch_attn_paged_host``, the allocation-free
``decode_batch_attn_noalloc``), the step with a score rule (``Scores``:
``decode_batch_attn_scored``, ``decode_batch_attn_paged_scored``,
``prefill_batch_attn_scored``) and over shared prefixes
(``decode_batch_attn_shared``), index arrays from request lengths
(``slot_kv_token_map``, ``slot_kv_extend_tables``), multi-step support
(``slot_kv_advance_positions``), and control (``slot_kv_get_status``,
``slot_kv_set_split``, ``slot_kv_set_options``, ``slot_kv_call_shape``).
``SlotKV`` wraps a handle.
"""
import ctypes
import os

__all__ = [
    "SlotKV", "SlotKVError", "slot_kv_alloc", "slot_kv_free", "slot_kv_offset_bytes",
    "slot_kv_reset", "decode_batch_attn", "decode_batch_attn_host", "prefill_batch_attn",
    "prefill_batch_attn_host", "slot_kv_prefill_host_parts", "PREFILL_HOST_MAX_PARTS",
    "decode_batch_attn_paged", "decode_batch_attn_paged_host", "decode_batch_attn_noalloc",
    "Scores", "decode_batch_attn_scored", "decode_batch_attn_paged_scored",
    "prefill_batch_attn_scored", "decode_batch_attn_shared", "slot_kv_token_map",
    "slot_kv_extend_tables", "slot_kv_advance_positions",
    "slot_kv_get_status", "slot_kv_set_split", "HostCall", "LIB_PATH", "EXPORTS", "DEV_RANGE",
    "DEV_TIMEOUT", "OPT_VNORM", "OPT_NORM_PLUS_ONE", "OPT_TEST_STALL",
]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libslotkv.so")
DEV_RANGE = 1
DEV_TIMEOUT = 2
OPT_VNORM = 1
OPT_NORM_PLUS_ONE = 2
OPT_TEST_STALL = 0x80000000
PREFILL_HOST_MAX_PARTS = 8  # SLOTKV_PREFILL_HOST_MAX_PARTS
SIZE_MAX = ctypes.c_size_t(-1).value

_u32, _f32, _vp, _int = ctypes.c_uint32, ctypes.c_float, ctypes.c_void_p, ctypes.c_int


class _CScores(ctypes.Structure):
    """slotkv_scores"""
    _fields_ = [("cap", _f32), ("window", _u32), ("slopes", _vp), ("doc_start", _vp),
                ("prefix_end", _vp)]


_SCP = ctypes.POINTER(_CScores)
_DECODE_ARGS = [_vp, _u32, _u32, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                _f32, _f32, _vp]
EXPORTS = {
    "slot_kv_alloc": ([ctypes.POINTER(_vp), _u32, _u32, _u32, _u32, _vp, _vp, _u32, _u32],
                      _int),
    "slot_kv_free": ([_vp], _int),
    "slot_kv_offset_bytes": ([_vp, _u32, _u32], ctypes.c_size_t),
    "slot_kv_reset": ([_vp, _u32, _vp], _int),
    "slot_kv_k_ptr": ([_vp, ctypes.POINTER(_vp)], _int),
    "slot_kv_v_ptr": ([_vp, ctypes.POINTER(_vp)], _int),
    "slot_kv_geometry": ([_vp] + [ctypes.POINTER(_u32)] * 6, _int),
    "decode_batch_attn": (_DECODE_ARGS, _int),
    "decode_batch_attn_host": (_DECODE_ARGS, _int),
    "prefill_batch_attn": (_DECODE_ARGS, _int),
    "prefill_batch_attn_host": (_DECODE_ARGS, _int),
    "slot_kv_prefill_host_parts": ([_u32, _vp, ctypes.POINTER(_u32), _u32,
                                    ctypes.POINTER(_u32)], _int),
    "decode_batch_attn_paged": ([_vp, _u32, _u32, _vp, _vp, _vp, _vp, _vp, _u32, _vp, _vp, _vp,
                                 _vp, _vp, _f32, _f32, _vp], _int),
    "decode_batch_attn_paged_host": ([_vp, _u32, _u32, _vp, _vp, _vp, _vp, _vp, _u32, _vp, _vp,
                                      _vp, _vp, _vp, _f32, _f32, _vp], _int),
    "decode_batch_attn_scored": ([_vp, _u32, _u32] + [_vp] * 9 + [_SCP, _vp, _f32, _f32, _vp],
                                 _int),
    "decode_batch_attn_paged_scored": ([_vp, _u32, _u32] + [_vp] * 5 + [_u32] + [_vp] * 4 +
                                       [_SCP, _vp, _f32, _f32, _vp], _int),
    "prefill_batch_attn_scored": ([_vp, _u32, _u32] + [_vp] * 9 + [_SCP, _vp, _f32, _f32, _vp],
                                  _int),
    "decode_batch_attn_shared": ([_vp, _u32, _u32] + [_vp] * 12 +
                                 [_SCP, _vp, _f32, _f32, _vp], _int),
    "slot_kv_token_map": ([_vp, _u32, _vp, _vp, _vp, _u32, _vp, _vp, _vp, _vp], _int),
    "slot_kv_extend_tables": ([_vp, _u32, _vp, _vp, _vp, _u32, _vp, _u32, _vp, _vp, _vp], _int),
    "slot_kv_get_status": ([_vp, _vp, ctypes.POINTER(_u32)], _int),
    "slot_kv_set_split": ([_vp, _u32, _u32], _int),
    "slot_kv_call_shape": ([_vp, _u32, _u32, _u32, ctypes.POINTER(_u32), ctypes.POINTER(_u32),
                            ctypes.POINTER(_u32)], _int),
    "slot_kv_advance_positions": ([_vp, _u32, _u32, _vp], _int),
    "slot_kv_set_options": ([_vp, _u32], _int),
    "decode_batch_attn_noalloc": ([_vp, _vp, _u32, _u32, _u32, _u32, _u32, _u32, _vp, _vp, _vp,
                                   _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _f32, _f32, _vp],
                                  _int),
    "slot_kv_shard_range": ([_u32, _u32, _u32, ctypes.POINTER(_u32), ctypes.POINTER(_u32)],
                            _int),
    "slot_kv_shard_route": ([_u32, _u32, _u32, _vp, _vp, _vp, _vp], _int),
    "slot_kv_host_call_create": ([_vp, ctypes.POINTER(_vp), _u32, _u32, _vp, _vp, _vp, _vp, _vp,
                                  _u32, _vp, _vp, _vp, _vp, _vp, _f32, _f32], _int),
    "slot_kv_host_call_run": ([_vp, _vp], _int),
    "slot_kv_host_call_enqueue": ([_vp, _vp], _int),
    "slot_kv_host_call_free": ([_vp], _int),
    "slot_kv_last_error": ([], ctypes.c_char_p),
}


class SlotKVError(RuntimeError):
    def __init__(self, code, what):
        super().__init__(f"{what} failed with status {code}: {last_error()}")
        self.code = code


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is not built; run __graft_entry__.build() (no CPU fallback exists)")
    lib = ctypes.CDLL(LIB_PATH)
    for name, (args, res) in EXPORTS.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    return lib


_lib = _load()


def last_error():
    msg = _lib.slot_kv_last_error()
    return msg.decode() if msg else ""


def _check(code, what):
    if code != 0:
        raise SlotKVError(code, what)


def _ptr(t, dtype=None, what="tensor", cuda=True):
    """Address of a contiguous tensor that lives on the GPU (cuda=True) or in
    host memory (cuda=False); None stays NULL.  The library reads these
    addresses from its kernels or copies, so a tensor in the wrong place is
    refused here."""
    if t is None:
        return None
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{what} must be a torch.Tensor")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{what} must be {dtype}, got {t.dtype}")
    if cuda is not None and t.is_cuda != cuda:
        raise ValueError(f"{what} must be a {'CUDA' if cuda else 'CPU'} tensor")
    return t.data_ptr()


def _shape(t):
    return None if t is None else tuple(int(x) for x in t.shape)


def _check_step(q, k_new, v_new, positions, rows_idx, out, q_norm_w, k_norm_w, inv_freq,
                sinks, n_kv_head, head_dim, idx_name="slots"):
    """Shapes of one step's tensors against (B, n_head) taken from q and the
    slot geometry (n_kv_head, head_dim).  The library reads and writes these
    buffers by those sizes, so a mismatch is refused before any call."""
    if q is None or q.dim() != 3:
        raise ValueError("q must be [B][n_head][head_dim]")
    B, n_head, hd = _shape(q)
    if hd != head_dim:
        raise ValueError(f"q's head_dim {hd} != the slot buffers' {head_dim}")
    want = {
        "q": (q, (B, n_head, hd)), "k_new": (k_new, (B, n_kv_head, hd)),
        "v_new": (v_new, (B, n_kv_head, hd)), "positions": (positions, (B,)),
        "out": (out, (B, n_head, hd)), "q_norm_w": (q_norm_w, (hd,)),
        "k_norm_w": (k_norm_w, (hd,)), "inv_freq": (inv_freq, (hd // 2,)),
    }
    if idx_name == "slots":
        want["slots"] = (rows_idx, (B,))
    for name, (t, shape) in want.items():
        if t is None:
            raise ValueError(f"{name} is required")
        if _shape(t) != shape:
            raise ValueError(f"{name} has shape {_shape(t)}, expected {shape}")
    if sinks is not None and _shape(sinks) != (n_head,):
        raise ValueError(f"sinks has shape {_shape(sinks)}, expected ({n_head},)")
    return B, n_head


def _stream_ptr(stream):
    import torch
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


_call = None  # the compiled calls: None not looked for yet, False not built


def _compiled():
    """The module of the compiled calls (csrc/call.cpp), which check a call's
    tensors and make it in one go; False if it is not built.  A call it
    declines (returning None) goes through the checks here, for their message."""
    global _call
    if _call is None:
        import torch  # noqa: F401 -- its libraries first
        try:
            from . import _slotkv_call
            _call = _slotkv_call
        except ImportError:
            _call = False
    return _call


class _Unlike(Exception):
    """An argument is not what the fast path takes; the slow path says why."""


def _addr(t, dtype, dev, shape):
    """Address of a contiguous tensor of this type and shape on CUDA device
    ``dev``.  Where the compiled calls are not built these checks are part of
    every step, so those of a good argument are a handful of attribute reads
    (a scored decode's call takes the host 8.5 us so, 16 with _check_step and
    _ptr); anything else raises _Unlike and is looked at again by those for its
    message."""
    if (t.dtype is dtype and t.get_device() == dev and t.shape == shape and
            t.is_contiguous()):
        return t.data_ptr()
    raise _Unlike


def _step_addrs(kv, q, k_new, v_new, positions, rows_idx, out, q_norm_w, k_norm_w, inv_freq,
                sinks, idx_name="slots"):
    """(B, n_head, addresses of q, k_new, v_new, positions, the row index,
    q_norm_w, k_norm_w, inv_freq, sinks, out, current device) of one step on
    the current device."""
    import torch
    dev = torch.cuda.current_device() if torch.cuda.is_initialized() else 0
    f, u = torch.float32, torch.int32
    try:
        B, n_head, hd = q.shape
        row, kv_row = (B, n_head, hd), (B, kv.n_kv_head, hd)
        if hd != kv.head_dim:
            raise _Unlike
        idx_shape = (B,) if idx_name == "slots" else (B, rows_idx.shape[1])
        return (B, n_head, _addr(q, f, dev, row), _addr(k_new, f, dev, kv_row),
                _addr(v_new, f, dev, kv_row), _addr(positions, u, dev, (B,)),
                _addr(rows_idx, u, dev, idx_shape), _addr(q_norm_w, f, dev, (hd,)),
                _addr(k_norm_w, f, dev, (hd,)), _addr(inv_freq, f, dev, (hd // 2,)),
                None if sinks is None else _addr(sinks, f, dev, (n_head,)),
                _addr(out, f, dev, row), dev)
    except (_Unlike, AttributeError, TypeError, ValueError, IndexError):
        pass
    B, n_head = _check_step(q, k_new, v_new, positions, rows_idx, out, q_norm_w, k_norm_w,
                            inv_freq, sinks, kv.n_kv_head, kv.head_dim, idx_name)
    if idx_name != "slots" and (rows_idx is None or rows_idx.dim() != 2 or
                                int(rows_idx.shape[0]) != B):
        raise ValueError("block_tables must be [B][max_blocks]")
    for name, t, dt in (("q", q, f), ("k_new", k_new, f), ("v_new", v_new, f),
                        ("positions", positions, u), (idx_name, rows_idx, u),
                        ("q_norm_w", q_norm_w, f), ("k_norm_w", k_norm_w, f),
                        ("inv_freq", inv_freq, f), ("sinks", sinks, f), ("out", out, f)):
        _ptr(t, dt, name)
        _on_device(t, dev, name)
    raise ValueError("the step's tensors cannot be used")


def _on_device(t, dev, what):
    if t is not None and t.get_device() != dev:
        raise ValueError(f"{what} is on device {t.get_device()}, but device {dev} is current")


def _int_addr(t, dev, what):
    """Address of a contiguous int32 tensor on CUDA device ``dev`` (its shape
    has been checked)."""
    import torch
    if t.get_device() != dev or t.dtype is not torch.int32 or not t.is_contiguous():
        _ptr(t, torch.int32, what)
        _on_device(t, dev, what)
    return t.data_ptr()


def _stream_arg(stream):
    """A stream argument for the compiled calls: an address, or None for torch's."""
    return stream if stream is None or isinstance(stream, int) else stream.cuda_stream


def _done(rc, name):
    """Whether a compiled call was made (None: declined); raises for its status."""
    if rc:
        _check(rc, name)
    return rc is not None


def _raw_stream(stream, dev):
    if stream is None:
        import torch
        return torch._C._cuda_getCurrentRawStream(dev)
    return stream if isinstance(stream, int) else stream.cuda_stream


def _rule_array(i, doc):
    """An array of a Scores: what is assigned to it is what the next call uses."""
    def put(self, t):
        self._args = self._args[:i] + (t,) + self._args[i + 1:]
    return property(lambda self: self._args[i], put, doc=doc)


class Scores:
    """A score rule (slotkv_scores): tanh cap, window, per-head slopes of the
    distance bias (float32 [n_head]), the rows' document starts and, in a
    prefill, prefix ends (int32 [rows]); CUDA tensors, kept referenced.  The
    arrays may be replaced between calls, each of which checks them."""

    def __init__(self, cap=0.0, window=0, slopes=None, doc_start=None, prefix_end=None):
        import torch
        if not 0 <= int(window) < 2 ** 32:
            raise ValueError("window must be 0 .. 2^32 - 1")
        _ptr(slopes, torch.float32, "slopes")
        _ptr(doc_start, torch.int32, "doc_start")
        _ptr(prefix_end, torch.int32, "prefix_end")
        # as the compiled calls take it
        self._args = (float(cap), int(window), slopes, doc_start, prefix_end)

    cap = property(lambda self: self._args[0], doc="tanh cap, 0: none")
    window = property(lambda self: self._args[1], doc="keys t with p - t < window, 0: all")
    slopes = _rule_array(2, "distance slopes [n_head], or None")
    doc_start = _rule_array(3, "first key of each row's document [rows], or None")
    prefix_end = _rule_array(4, "end of each row's prefix [rows], or None (prefill)")


def _scores(sc, rows, n_head, dev):
    """The struct of a Scores, by reference, for a step of ``rows`` rows on
    device ``dev``; None stays NULL."""
    if sc is None:
        return None
    import torch
    ptrs = []
    for name, t, dtype, n in (("slopes", sc.slopes, torch.float32, n_head),
                              ("doc_start", sc.doc_start, torch.int32, rows),
                              ("prefix_end", sc.prefix_end, torch.int32, rows)):
        ptrs.append(_ptr(t, dtype, name))
        if t is not None and t.shape != (n,):
            raise ValueError(f"{name} has shape {_shape(t)}, expected {(n,)}")
        _on_device(t, dev, name)
    return ctypes.byref(_CScores(sc.cap, sc.window, *ptrs))


class SlotKV:
    """One attention layer's slot KV: ``[n_slots][slot_ctx][n_kv_head][head_dim]``
    f32 K and V, plus the split-K workspace for up to ``max_rows`` rows and
    ``max_n_head`` query heads.  ``k_buf``/``v_buf`` (torch CUDA tensors) are
    adopted in place when given; otherwise the library allocates them."""

    def __init__(self, n_slots, slot_ctx, n_kv_head, head_dim, max_rows, max_n_head,
                 k_buf=None, v_buf=None):
        import torch
        self._h = _vp()
        self.n_slots, self.slot_ctx = int(n_slots), int(slot_ctx)
        self.n_kv_head, self.head_dim = int(n_kv_head), int(head_dim)
        self.kv_dim = self.n_kv_head * self.head_dim
        self.max_rows, self.max_n_head = int(max_rows), int(max_n_head)
        self._keep = (k_buf, v_buf)
        kp = _ptr(k_buf, torch.float32, "k_buf")
        vp = _ptr(v_buf, torch.float32, "v_buf")
        _check(_lib.slot_kv_alloc(ctypes.byref(self._h), n_slots, slot_ctx, n_kv_head,
                                  head_dim, kp, vp, max_rows, max_n_head), "slot_kv_alloc")

    @property
    def handle(self):
        return self._h.value

    def free(self):
        if self._h.value:
            _check(_lib.slot_kv_free(self._h), "slot_kv_free")
            self._h = _vp()
        self._keep = (None, None)

    def __del__(self):
        try:
            self.free()
        except Exception:  # noqa: BLE001 -- interpreter shutdown
            pass

    def offset_bytes(self, slot, pos):
        v = _lib.slot_kv_offset_bytes(self._h, slot, pos)
        return None if v == SIZE_MAX else int(v)

    def reset(self, slot, stream=None):
        _check(_lib.slot_kv_reset(self._h, slot, _stream_ptr(stream)), "slot_kv_reset")

    def k_ptr(self):
        p = _vp()
        _check(_lib.slot_kv_k_ptr(self._h, ctypes.byref(p)), "slot_kv_k_ptr")
        return p.value

    def v_ptr(self):
        p = _vp()
        _check(_lib.slot_kv_v_ptr(self._h, ctypes.byref(p)), "slot_kv_v_ptr")
        return p.value

    def kv_tensors(self):
        """(K, V) as torch views of the slot buffers (adopted or owned)."""
        if self._keep[0] is not None:
            return self._keep
        # owned buffers: wrap the device addresses without copying
        n = self.n_slots * self.slot_ctx * self.kv_dim
        shape = (self.n_slots, self.slot_ctx, self.n_kv_head, self.head_dim)
        return tuple(_wrap_device(ptr, n).view(shape) for ptr in (self.k_ptr(), self.v_ptr()))

    def decode_batch_attn(self, q, k_new, v_new, positions, slots, q_norm_w, k_norm_w,
                          inv_freq, sinks, out, eps, scale, stream=None):
        import torch
        B, n_head = _check_step(q, k_new, v_new, positions, slots, out, q_norm_w, k_norm_w,
                                inv_freq, sinks, self.n_kv_head, self.head_dim)
        f, u = torch.float32, torch.int32
        _check(_lib.decode_batch_attn(
            self._h, B, n_head, _ptr(q, f, "q"), _ptr(k_new, f, "k_new"),
            _ptr(v_new, f, "v_new"), _ptr(positions, u, "positions"), _ptr(slots, u, "slots"),
            _ptr(q_norm_w, f, "q_norm_w"), _ptr(k_norm_w, f, "k_norm_w"),
            _ptr(inv_freq, f, "inv_freq"), _ptr(sinks, f, "sinks"), _ptr(out, f, "out"),
            eps, scale, _stream_ptr(stream)), "decode_batch_attn")
        return out

    def prefill_batch_attn(self, q, k_new, v_new, positions, slots, q_norm_w, k_norm_w,
                           inv_freq, sinks, out, eps, scale, stream=None):
        """Batched causal prefill: tokens (rows of q, k_new, v_new, positions,
        slots, out) are written into their slots and each attends keys
        0..pos of its slot, the call's other new rows included."""
        import torch
        n, n_head = _check_step(q, k_new, v_new, positions, slots, out, q_norm_w, k_norm_w,
                                inv_freq, sinks, self.n_kv_head, self.head_dim)
        f, u = torch.float32, torch.int32
        _check(_lib.prefill_batch_attn(
            self._h, n, n_head, _ptr(q, f, "q"), _ptr(k_new, f, "k_new"),
            _ptr(v_new, f, "v_new"), _ptr(positions, u, "positions"), _ptr(slots, u, "slots"),
            _ptr(q_norm_w, f, "q_norm_w"), _ptr(k_norm_w, f, "k_norm_w"),
            _ptr(inv_freq, f, "inv_freq"), _ptr(sinks, f, "sinks"), _ptr(out, f, "out"),
            eps, scale, _stream_ptr(stream)), "prefill_batch_attn")
        return out

    def prefill_batch_attn_host(self, q, k_new, v_new, positions, slots, q_norm_w, k_norm_w,
                                inv_freq, sinks, out, eps, scale, stream=None):
        """As prefill_batch_attn, with q/k_new/v_new/positions/slots/out in host
        memory (CPU tensors, ideally pinned); synchronous."""
        import torch
        n, n_head = _check_step(q, k_new, v_new, positions, slots, out, q_norm_w, k_norm_w,
                                inv_freq, sinks, self.n_kv_head, self.head_dim)
        f, u = torch.float32, torch.int32
        _check(_lib.prefill_batch_attn_host(
            self._h, n, n_head, _ptr(q, f, "q", cuda=False), _ptr(k_new, f, "k_new", cuda=False),
            _ptr(v_new, f, "v_new", cuda=False), _ptr(positions, u, "positions", cuda=False),
            _ptr(slots, u, "slots", cuda=False), _ptr(q_norm_w, f, "q_norm_w"),
            _ptr(k_norm_w, f, "k_norm_w"), _ptr(inv_freq, f, "inv_freq"), _ptr(sinks, f, "sinks"),
            _ptr(out, f, "out", cuda=False), eps, scale, _stream_ptr(stream)),
            "prefill_batch_attn_host")
        return out

    def decode_batch_attn_paged(self, q, k_new, v_new, positions, block_tables, q_norm_w,
                                k_norm_w, inv_freq, sinks, out, eps, scale, stream=None):
        """Decode over a paged pool (this handle's buffers as blocks of
        slot_ctx positions): block_tables is int32 [B][max_blocks], row b's
        key t in block block_tables[b][t // slot_ctx]."""
        import torch
        B, n_head = _check_step(q, k_new, v_new, positions, block_tables, out, q_norm_w,
                                k_norm_w, inv_freq, sinks, self.n_kv_head, self.head_dim,
                                idx_name="block_tables")
        f, u = torch.float32, torch.int32
        if block_tables.dim() != 2 or int(block_tables.shape[0]) != B:
            raise ValueError("block_tables must be [B][max_blocks]")
        _check(_lib.decode_batch_attn_paged(
            self._h, B, n_head, _ptr(q, f, "q"), _ptr(k_new, f, "k_new"),
            _ptr(v_new, f, "v_new"), _ptr(positions, u, "positions"),
            _ptr(block_tables, u, "block_tables"), int(block_tables.shape[1]),
            _ptr(q_norm_w, f, "q_norm_w"), _ptr(k_norm_w, f, "k_norm_w"),
            _ptr(inv_freq, f, "inv_freq"), _ptr(sinks, f, "sinks"), _ptr(out, f, "out"),
            eps, scale, _stream_ptr(stream)), "decode_batch_attn_paged")
        return out

    def decode_batch_attn_paged_host(self, q, k_new, v_new, positions, block_tables, q_norm_w,
                                     k_norm_w, inv_freq, sinks, out, eps, scale, stream=None):
        """As decode_batch_attn_paged, with q/k_new/v_new/positions/block_tables/out
        in host memory (CPU tensors, ideally pinned); synchronous."""
        import torch
        B, n_head = _check_step(q, k_new, v_new, positions, block_tables, out, q_norm_w,
                                k_norm_w, inv_freq, sinks, self.n_kv_head, self.head_dim,
                                idx_name="block_tables")
        f, u = torch.float32, torch.int32
        if block_tables.dim() != 2 or int(block_tables.shape[0]) != B:
            raise ValueError("block_tables must be [B][max_blocks]")
        _check(_lib.decode_batch_attn_paged_host(
            self._h, B, n_head, _ptr(q, f, "q", cuda=False),
            _ptr(k_new, f, "k_new", cuda=False), _ptr(v_new, f, "v_new", cuda=False),
            _ptr(positions, u, "positions", cuda=False),
            _ptr(block_tables, u, "block_tables", cuda=False), int(block_tables.shape[1]),
            _ptr(q_norm_w, f, "q_norm_w"), _ptr(k_norm_w, f, "k_norm_w"),
            _ptr(inv_freq, f, "inv_freq"), _ptr(sinks, f, "sinks"),
            _ptr(out, f, "out", cuda=False), eps, scale, _stream_ptr(stream)),
            "decode_batch_attn_paged_host")
        return out

    def decode_batch_attn_scored(self, q, k_new, v_new, positions, slots, q_norm_w, k_norm_w,
                                 inv_freq, sinks, scores, out, eps, scale, stream=None):
        """As decode_batch_attn, with a score rule (Scores, or None)."""
        return self._slot_step_scored("decode_batch_attn_scored", q, k_new, v_new, positions,
                                      slots, q_norm_w, k_norm_w, inv_freq, sinks, scores, out,
                                      eps, scale, stream)

    def prefill_batch_attn_scored(self, q, k_new, v_new, positions, slots, q_norm_w, k_norm_w,
                                  inv_freq, sinks, scores, out, eps, scale, stream=None):
        """As prefill_batch_attn, with a score rule (Scores, or None)."""
        return self._slot_step_scored("prefill_batch_attn_scored", q, k_new, v_new, positions,
                                      slots, q_norm_w, k_norm_w, inv_freq, sinks, scores, out,
                                      eps, scale, stream)

    def _slot_step_scored(self, name, q, k_new, v_new, positions, slots, q_norm_w, k_norm_w,
                          inv_freq, sinks, scores, out, eps, scale, stream):
        c = _compiled()
        if c and _done(getattr(c, name)(
                self._h.value, self.n_kv_head, self.head_dim, q, k_new, v_new, positions, slots,
                q_norm_w, k_norm_w, inv_freq, sinks, None if scores is None else scores._args, out,
                eps, scale, _stream_arg(stream)), name):
            return out
        (B, n_head, aq, ak, av, ap, ai, aqw, akw, af, asn, ao, dev) = _step_addrs(
            self, q, k_new, v_new, positions, slots, out, q_norm_w, k_norm_w, inv_freq, sinks)
        _check(getattr(_lib, name)(self._h, B, n_head, aq, ak, av, ap, ai, aqw, akw, af, asn,
                                   _scores(scores, B, n_head, dev), ao, eps, scale,
                                   _raw_stream(stream, dev)), name)
        return out

    def decode_batch_attn_paged_scored(self, q, k_new, v_new, positions, block_tables, q_norm_w,
                                       k_norm_w, inv_freq, sinks, scores, out, eps, scale,
                                       stream=None):
        """As decode_batch_attn_paged, with a score rule (Scores, or None)."""
        c, name = _compiled(), "decode_batch_attn_paged_scored"
        if c and _done(c.decode_batch_attn_paged_scored(
                self._h.value, self.n_kv_head, self.head_dim, q, k_new, v_new, positions,
                block_tables, q_norm_w, k_norm_w, inv_freq, sinks,
                None if scores is None else scores._args, out, eps, scale, _stream_arg(stream)),
                name):
            return out
        (B, n_head, aq, ak, av, ap, ai, aqw, akw, af, asn, ao, dev) = _step_addrs(
            self, q, k_new, v_new, positions, block_tables, out, q_norm_w, k_norm_w, inv_freq,
            sinks, "block_tables")
        _check(_lib.decode_batch_attn_paged_scored(
            self._h, B, n_head, aq, ak, av, ap, ai, int(block_tables.shape[1]), aqw, akw, af, asn,
            _scores(scores, B, n_head, dev), ao, eps, scale, _raw_stream(stream, dev)), name)
        return out

    def decode_batch_attn_shared(self, q, k_new, v_new, positions, slots, prefix, prefix_slots,
                                 prefix_lens, q_norm_w, k_norm_w, inv_freq, sinks, scores, out,
                                 eps, scale, stream=None):
        """The decode step for rows on shared prefixes: row b's positions
        0 .. prefix_lens[b] - 1 are in slot prefix_slots[b] of the SlotKV
        ``prefix``, the later ones in its own slot from position 0 on."""
        if not isinstance(prefix, SlotKV):
            raise TypeError("prefix must be a SlotKV")
        c, name = _compiled(), "decode_batch_attn_shared"
        if c and _done(c.decode_batch_attn_shared(
                self._h.value, self.n_kv_head, self.head_dim, q, k_new, v_new, positions, slots,
                prefix._h.value, prefix_slots, prefix_lens, q_norm_w, k_norm_w, inv_freq, sinks,
                None if scores is None else scores._args, out, eps, scale, _stream_arg(stream)),
                name):
            return out
        for what, t in (("prefix_slots", prefix_slots), ("prefix_lens", prefix_lens)):
            if t is None or t.dim() != 1 or t.shape != positions.shape:
                raise ValueError(f"{what} must be [B]")
        (B, n_head, aq, ak, av, ap, ai, aqw, akw, af, asn, ao, dev) = _step_addrs(
            self, q, k_new, v_new, positions, slots, out, q_norm_w, k_norm_w, inv_freq, sinks)
        _check(_lib.decode_batch_attn_shared(
            self._h, B, n_head, aq, ak, av, ap, ai, prefix._h,
            _int_addr(prefix_slots, dev, "prefix_slots"),
            _int_addr(prefix_lens, dev, "prefix_lens"), aqw, akw, af, asn,
            _scores(scores, B, n_head, dev), ao, eps, scale, _raw_stream(stream, dev)), name)
        return out

    def token_map(self, slots, past, fresh, starts, tok_slots, tok_positions, stream=None):
        """slot_kv_token_map: the slots and positions of a prefill's tokens from
        the requests' (slot, cached length, new length), int32 CUDA tensors."""
        c = _compiled()
        if c and _done(c.slot_kv_token_map(self._h.value, slots, past, fresh, starts, tok_slots,
                                           tok_positions, _stream_arg(stream)),
                       "slot_kv_token_map"):
            return starts, tok_slots, tok_positions
        import torch
        n, n_tok = slots.numel(), tok_slots.numel()
        if not (slots.shape == past.shape == fresh.shape == (n,) and starts.shape == (n + 1,) and
                tok_slots.shape == tok_positions.shape == (n_tok,)):
            for name, t, m in (("slots", slots, n), ("past", past, n), ("fresh", fresh, n),
                               ("starts", starts, n + 1), ("tok_slots", tok_slots, n_tok),
                               ("tok_positions", tok_positions, n_tok)):
                if t.shape != (m,):
                    raise ValueError(f"{name} has shape {_shape(t)}, expected {(m,)}")
        dev = torch.cuda.current_device() if torch.cuda.is_initialized() else 0
        _check(_lib.slot_kv_token_map(
            self._h, n, _int_addr(slots, dev, "slots"), _int_addr(past, dev, "past"),
            _int_addr(fresh, dev, "fresh"), n_tok, _int_addr(starts, dev, "starts"),
            _int_addr(tok_slots, dev, "tok_slots"),
            _int_addr(tok_positions, dev, "tok_positions"), _raw_stream(stream, dev)),
            "slot_kv_token_map")
        return starts, tok_slots, tok_positions

    def extend_tables(self, past, fresh, block_tables, free_blocks, head, head_out=None,
                      stream=None):
        """slot_kv_extend_tables: block_tables (int32 [requests][max_blocks], in
        place) extended from the free list; head_out None advances ``head``
        itself.  int32 CUDA tensors."""
        if head_out is None:
            head_out = head
        c = _compiled()
        if c and _done(c.slot_kv_extend_tables(self._h.value, past, fresh, block_tables,
                                               free_blocks, head, head_out, _stream_arg(stream)),
                       "slot_kv_extend_tables"):
            return block_tables, head_out
        import torch
        n = past.numel()
        if block_tables.dim() != 2 or block_tables.shape[0] != n:
            raise ValueError("block_tables must be [requests][max_blocks]")
        if free_blocks.dim() != 1:
            raise ValueError("free_blocks must be [n_free]")
        if not (past.shape == fresh.shape == (n,) and head.shape == head_out.shape == (1,)):
            for name, t, m in (("past", past, n), ("fresh", fresh, n), ("head", head, 1),
                               ("head_out", head_out, 1)):
                if t.shape != (m,):
                    raise ValueError(f"{name} has shape {_shape(t)}, expected {(m,)}")
        dev = torch.cuda.current_device() if torch.cuda.is_initialized() else 0
        n_free = free_blocks.shape[0]
        _check(_lib.slot_kv_extend_tables(
            self._h, n, _int_addr(past, dev, "past"), _int_addr(fresh, dev, "fresh"),
            _int_addr(block_tables, dev, "block_tables"), block_tables.shape[1],
            _int_addr(free_blocks, dev, "free_blocks"), n_free,
            _int_addr(head, dev, "head"), _int_addr(head_out, dev, "head_out"),
            _raw_stream(stream, dev)), "slot_kv_extend_tables")
        return block_tables, head_out

    def prepare_host_call(self, q, k_new, v_new, positions, slots, q_norm_w, k_norm_w,
                          inv_freq, sinks, out, eps, scale, block_tables=None):
        """A prepared host step (slot_kv_host_call_create): the arguments of
        decode_batch_attn_host -- or, with ``block_tables`` given in place of
        ``slots`` (pass slots=None), of decode_batch_attn_paged_host --
        checked once.  Calling the returned HostCall runs one step on the
        buffers' current contents, synchronously."""
        return HostCall(self, q, k_new, v_new, positions, slots, q_norm_w, k_norm_w, inv_freq,
                        sinks, out, eps, scale, block_tables)

    def decode_batch_attn_host(self, q, k_new, v_new, positions, slots, q_norm_w,
                               k_norm_w, inv_freq, sinks, out, eps, scale, stream=None):
        """As decode_batch_attn, with q/k_new/v_new/positions/slots/out in host
        memory (CPU tensors, ideally pinned); synchronous."""
        import torch
        B, n_head = _check_step(q, k_new, v_new, positions, slots, out, q_norm_w, k_norm_w,
                                inv_freq, sinks, self.n_kv_head, self.head_dim)
        f, u = torch.float32, torch.int32
        _check(_lib.decode_batch_attn_host(
            self._h, B, n_head, _ptr(q, f, "q", cuda=False),
            _ptr(k_new, f, "k_new", cuda=False), _ptr(v_new, f, "v_new", cuda=False),
            _ptr(positions, u, "positions", cuda=False), _ptr(slots, u, "slots", cuda=False),
            _ptr(q_norm_w, f, "q_norm_w"), _ptr(k_norm_w, f, "k_norm_w"),
            _ptr(inv_freq, f, "inv_freq"), _ptr(sinks, f, "sinks"),
            _ptr(out, f, "out", cuda=False), eps, scale, _stream_ptr(stream)),
            "decode_batch_attn_host")
        return out

    def get_status(self, stream=None):
        v = _u32()
        _check(_lib.slot_kv_get_status(self._h, _stream_ptr(stream), ctypes.byref(v)),
               "slot_kv_get_status")
        return int(v.value)

    def set_options(self, flags):
        """OPT_VNORM and/or OPT_NORM_PLUS_ONE (see slot_kv_set_options)."""
        _check(_lib.slot_kv_set_options(self._h, flags), "slot_kv_set_options")

    def call_shape(self, B, bt_stride=0, prefill=False):
        """(chunk_keys, ctas, kernels) of a call of B rows (slot_kv_call_shape)."""
        c, n, k = _u32(), _u32(), _u32()
        _check(_lib.slot_kv_call_shape(self._h, B, bt_stride, 1 if prefill else 0,
                                       ctypes.byref(c), ctypes.byref(n), ctypes.byref(k)),
               "slot_kv_call_shape")
        return c.value, n.value, k.value

    def set_split(self, min_chunk_keys, max_splits):
        _check(_lib.slot_kv_set_split(self._h, min_chunk_keys, max_splits), "slot_kv_set_split")


def _wrap_device(ptr, numel):
    """A float32 CUDA tensor aliasing ``numel`` floats at device address ``ptr``."""
    import torch

    class _Holder:
        pass

    h = _Holder()
    h.__cuda_array_interface__ = {
        "shape": (numel,), "typestr": "<f4", "data": (ptr, False), "version": 3,
        "strides": None,
    }
    return torch.as_tensor(h, device="cuda")


# ---- C-ABI names ---------------------------------------------------------
def slot_kv_alloc(n_slots, slot_ctx, n_kv_head, head_dim, max_rows, max_n_head,
                  k_buf=None, v_buf=None):
    return SlotKV(n_slots, slot_ctx, n_kv_head, head_dim, max_rows, max_n_head, k_buf, v_buf)


def slot_kv_free(h):
    h.free()


def slot_kv_offset_bytes(h, slot, pos):
    return h.offset_bytes(slot, pos)


def slot_kv_reset(h, slot, stream=None):
    h.reset(slot, stream)


def decode_batch_attn(h, q, k_new, v_new, positions, slots, q_norm_w, k_norm_w, inv_freq,
                      sinks, out, eps, scale, stream=None):
    return h.decode_batch_attn(q, k_new, v_new, positions, slots, q_norm_w, k_norm_w,
                               inv_freq, sinks, out, eps, scale, stream)


def prefill_batch_attn(h, q, k_new, v_new, positions, slots, q_norm_w, k_norm_w, inv_freq,
                       sinks, out, eps, scale, stream=None):
    return h.prefill_batch_attn(q, k_new, v_new, positions, slots, q_norm_w, k_norm_w,
                                inv_freq, sinks, out, eps, scale, stream)


def prefill_batch_attn_host(h, q, k_new, v_new, positions, slots, q_norm_w, k_norm_w,
                            inv_freq, sinks, out, eps, scale, stream=None):
    return h.prefill_batch_attn_host(q, k_new, v_new, positions, slots, q_norm_w, k_norm_w,
                                     inv_freq, sinks, out, eps, scale, stream)


def slot_kv_prefill_host_parts(slots):
    """Where prefill_batch_attn_host cuts a call with these slots (one per
    token, a host sequence of ints): the part boundaries [0, ..., n_tok].
    Host only."""
    import numpy as np
    sl = np.ascontiguousarray(np.asarray(slots).astype(np.uint32, copy=False))
    cuts = (_u32 * (PREFILL_HOST_MAX_PARTS + 1))()
    n = _u32()
    _check(_lib.slot_kv_prefill_host_parts(len(sl), sl.ctypes.data if len(sl) else None, cuts,
                                           len(cuts), ctypes.byref(n)),
           "slot_kv_prefill_host_parts")
    return [int(cuts[i]) for i in range(n.value + 1)]


def decode_batch_attn_paged(h, q, k_new, v_new, positions, block_tables, q_norm_w, k_norm_w,
                            inv_freq, sinks, out, eps, scale, stream=None):
    return h.decode_batch_attn_paged(q, k_new, v_new, positions, block_tables, q_norm_w,
                                     k_norm_w, inv_freq, sinks, out, eps, scale, stream)


def decode_batch_attn_scored(h, q, k_new, v_new, positions, slots, q_norm_w, k_norm_w, inv_freq,
                             sinks, scores, out, eps, scale, stream=None):
    return h.decode_batch_attn_scored(q, k_new, v_new, positions, slots, q_norm_w, k_norm_w,
                                      inv_freq, sinks, scores, out, eps, scale, stream)


def decode_batch_attn_paged_scored(h, q, k_new, v_new, positions, block_tables, q_norm_w,
                                   k_norm_w, inv_freq, sinks, scores, out, eps, scale,
                                   stream=None):
    return h.decode_batch_attn_paged_scored(q, k_new, v_new, positions, block_tables, q_norm_w,
                                            k_norm_w, inv_freq, sinks, scores, out, eps, scale,
                                            stream)


def prefill_batch_attn_scored(h, q, k_new, v_new, positions, slots, q_norm_w, k_norm_w, inv_freq,
                              sinks, scores, out, eps, scale, stream=None):
    return h.prefill_batch_attn_scored(q, k_new, v_new, positions, slots, q_norm_w, k_norm_w,
                                       inv_freq, sinks, scores, out, eps, scale, stream)


def decode_batch_attn_shared(h, q, k_new, v_new, positions, slots, prefix, prefix_slots,
                             prefix_lens, q_norm_w, k_norm_w, inv_freq, sinks, scores, out, eps,
                             scale, stream=None):
    return h.decode_batch_attn_shared(q, k_new, v_new, positions, slots, prefix, prefix_slots,
                                      prefix_lens, q_norm_w, k_norm_w, inv_freq, sinks, scores,
                                      out, eps, scale, stream)


def slot_kv_token_map(h, slots, past, fresh, starts, tok_slots, tok_positions, stream=None):
    return h.token_map(slots, past, fresh, starts, tok_slots, tok_positions, stream)


def slot_kv_extend_tables(h, past, fresh, block_tables, free_blocks, head, head_out=None,
                          stream=None):
    return h.extend_tables(past, fresh, block_tables, free_blocks, head, head_out, stream)


class HostCall:
    """A prepared host step on a SlotKV handle (slot_kv_host_call_create):
    the host tensors (q, k_new, v_new, positions, slots or block_tables, out;
    ideally pinned) and the device parameters are checked once and kept
    referenced; ``call(stream=None)`` runs one synchronous step on their
    current contents (slot_kv_host_call_run), the same step the host entry
    runs; ``call(stream, sync=False)`` only enqueues it
    (slot_kv_host_call_enqueue).  ``free()`` releases it (also on garbage
    collection)."""

    def __init__(self, kv, q, k_new, v_new, positions, slots, q_norm_w, k_norm_w, inv_freq,
                 sinks, out, eps, scale, block_tables=None):
        import torch
        paged = block_tables is not None
        idx = block_tables if paged else slots
        B, n_head = _check_step(q, k_new, v_new, positions, idx, out, q_norm_w, k_norm_w,
                                inv_freq, sinks, kv.n_kv_head, kv.head_dim,
                                idx_name="block_tables" if paged else "slots")
        if paged and (block_tables.dim() != 2 or int(block_tables.shape[0]) != B):
            raise ValueError("block_tables must be [B][max_blocks]")
        f, u = torch.float32, torch.int32
        self._c = _vp()
        self._kv = kv
        self._keep = (q, k_new, v_new, positions, idx, q_norm_w, k_norm_w, inv_freq, sinks, out)
        _check(_lib.slot_kv_host_call_create(
            kv._h, ctypes.byref(self._c), B, n_head, _ptr(q, f, "q", cuda=False),
            _ptr(k_new, f, "k_new", cuda=False), _ptr(v_new, f, "v_new", cuda=False),
            _ptr(positions, u, "positions", cuda=False),
            _ptr(idx, u, "block_tables" if paged else "slots", cuda=False),
            int(block_tables.shape[1]) if paged else 0,
            _ptr(q_norm_w, f, "q_norm_w"), _ptr(k_norm_w, f, "k_norm_w"),
            _ptr(inv_freq, f, "inv_freq"), _ptr(sinks, f, "sinks"),
            _ptr(out, f, "out", cuda=False), eps, scale), "slot_kv_host_call_create")
        self.out = out

    def __call__(self, stream=None, sync=True):
        """One step.  sync=False only enqueues it (slot_kv_host_call_enqueue):
        out is complete, and the host inputs may be refilled, once the stream
        has been synchronised."""
        if sync:
            _check(_lib.slot_kv_host_call_run(self._c, _stream_ptr(stream)),
                   "slot_kv_host_call_run")
        else:
            _check(_lib.slot_kv_host_call_enqueue(self._c, _stream_ptr(stream)),
                   "slot_kv_host_call_enqueue")
        return self.out

    def free(self):
        if self._c.value:
            _check(_lib.slot_kv_host_call_free(self._c), "slot_kv_host_call_free")
            self._c = _vp()
        self._keep = None

    def __del__(self):
        try:
            self.free()
        except Exception:  # noqa: BLE001 -- interpreter shutdown
            pass


def decode_batch_attn_host(h, q, k_new, v_new, positions, slots, q_norm_w, k_norm_w,
                           inv_freq, sinks, out, eps, scale, stream=None):
    return h.decode_batch_attn_host(q, k_new, v_new, positions, slots, q_norm_w, k_norm_w,
                                    inv_freq, sinks, out, eps, scale, stream)


def decode_batch_attn_paged_host(h, q, k_new, v_new, positions, block_tables, q_norm_w,
                                 k_norm_w, inv_freq, sinks, out, eps, scale, stream=None):
    return h.decode_batch_attn_paged_host(q, k_new, v_new, positions, block_tables, q_norm_w,
                                          k_norm_w, inv_freq, sinks, out, eps, scale, stream)


def slot_kv_get_status(h, stream=None):
    return h.get_status(stream)


def slot_kv_set_split(h, min_chunk_keys, max_splits):
    h.set_split(min_chunk_keys, max_splits)


def slot_kv_advance_positions(positions, delta=1, stream=None):
    """positions += delta on the device (int32 CUDA tensor), on ``stream``."""
    import torch
    _check(_lib.slot_kv_advance_positions(_ptr(positions, torch.int32, "positions"),
                                          int(positions.numel()), int(delta),
                                          _stream_ptr(stream)), "slot_kv_advance_positions")


def decode_batch_attn_noalloc(K, V, q, k_new, v_new, positions, slots, q_norm_w, k_norm_w,
                              inv_freq, sinks, out, eps, scale, dev_flags=None, stream=None):
    """The decode step for callers that cannot allocate device memory: no
    handle; the slot buffers K, V ([n_slots][slot_ctx][n_kv_head][head_dim]
    torch CUDA tensors) and every input and output come from the caller, and
    the library's split-K scratch is a fixed array inside it.  ``dev_flags``
    is an optional int32 CUDA tensor of one element that receives the device
    flags.  The first call on a device should come before any stream capture;
    calls that overlap on the GPU race on the shared scratch."""
    import torch
    if K.dim() != 4 or _shape(V) != _shape(K):
        raise ValueError("K and V must both be [n_slots][slot_ctx][n_kv_head][head_dim]")
    n_slots, slot_ctx, n_kv_head, head_dim = _shape(K)
    B, n_head = _check_step(q, k_new, v_new, positions, slots, out, q_norm_w, k_norm_w,
                            inv_freq, sinks, n_kv_head, head_dim)
    if dev_flags is not None and int(dev_flags.numel()) < 1:
        raise ValueError("dev_flags must hold one element")
    f, u = torch.float32, torch.int32
    _check(_lib.decode_batch_attn_noalloc(
        _ptr(K, f, "K"), _ptr(V, f, "V"), n_slots, slot_ctx, n_kv_head, head_dim, B, n_head,
        _ptr(q, f, "q"), _ptr(k_new, f, "k_new"), _ptr(v_new, f, "v_new"),
        _ptr(positions, u, "positions"), _ptr(slots, u, "slots"), _ptr(q_norm_w, f, "q_norm_w"),
        _ptr(k_norm_w, f, "k_norm_w"), _ptr(inv_freq, f, "inv_freq"), _ptr(sinks, f, "sinks"),
        _ptr(out, f, "out"), _ptr(dev_flags, u, "dev_flags"), eps, scale, _stream_ptr(stream)),
        "decode_batch_attn_noalloc")
    return out
