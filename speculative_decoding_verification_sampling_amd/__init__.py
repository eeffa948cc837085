"""Python binding of libspecv, the speculative-sampling verify step for MI355X.

Argument marshalling only: every step of the verify path runs in the HIP
kernels of ``libspecv.so``.  PyTorch supplies device memory (tensors) and
the stream (``torch.cuda.current_stream()``); no torch computation happens
on the path.  Build the library first with
``python -m speculative_decoding_verification_sampling_amd.build``; if it is
missing, importing works but every call raises.

    v = Verifier(max_batch=64, max_gamma=5, max_vocab=128256)
    params = make_row_params(64, temperature=0.7, device="cuda")
    out = v.verify_sample(target, draft, tokens, params, seed=1234)
    out["out_tokens"], out["num_emitted"], out["num_accepted"], out["row_flags"]
"""

import ctypes
import os

import numpy as np
import torch

__all__ = [
    "Verifier",
    "make_row_params",
    "load_library",
    "library_path",
    "SpecvError",
    "FLAG_TOKEN_OOR",
    "FLAG_NONFINITE_ROW",
    "FLAG_Q_ZERO",
    "FLAG_RESIDUAL_FALLBACK",
    "FLAG_CAND_OVERFLOW",
    "FLAG_TOPP_NEAR",
    "FLAG_UNSUPPORTED",
    "FLAG_INTERNAL",
    "EXPORTED_SYMBOLS",
    "read_ceiling",
    "verify_sample_noalloc",
    "debug_set_wait_limit",
    "TokenHistory",
    "make_penalties",
    "make_bias",
    "pack_token_mask",
    "MAX_RECORD_K",
]

_HERE = os.path.dirname(os.path.abspath(__file__))

FLAG_TOKEN_OOR = 1 << 0
FLAG_NONFINITE_ROW = 1 << 1
FLAG_Q_ZERO = 1 << 2
FLAG_RESIDUAL_FALLBACK = 1 << 3
FLAG_CAND_OVERFLOW = 1 << 4
FLAG_TOPP_NEAR = 1 << 5
FLAG_UNSUPPORTED = 1 << 6
FLAG_INTERNAL = 1 << 7

SPECV_F32 = 0
SPECV_BF16 = 1

EXPORTED_SYMBOLS = ("specv_create", "specv_verify_sample", "specv_verify_point_mass",
                    "specv_verify_sample_qstats", "specv_sample_draft", "specv_verify_greedy",
                    "specv_destroy", "specv_status_string", "specv_set_profiling",
                    "specv_get_profile", "specv_get_profile_samples", "specv_read_ceiling",
                    "specv_verify_sample_noalloc", "specv_debug_set_wait_limit",
                    "specv_adjust_logits", "specv_history_add", "specv_history_reset",
                    "specv_top_logits", "specv_distill_loss", "specv_distill_grad",
                    "specv_distill_loss_grad", "specv_distill_workspace")

MAX_RECORD_K = 256
TAILS = {"renorm": 0, "bucket": 1}


class SpecvError(RuntimeError):
    pass


class _Config(ctypes.Structure):
    _fields_ = [("device", ctypes.c_int), ("max_batch", ctypes.c_int),
                ("max_gamma", ctypes.c_int), ("max_vocab", ctypes.c_int),
                ("max_top_k", ctypes.c_int)]


class _Diag(ctypes.Structure):
    _fields_ = [("p_at_draft", ctypes.c_void_p), ("q_at_draft", ctypes.c_void_p),
                ("residual_sum", ctypes.c_void_p)]


class _Adjustments(ctypes.Structure):
    _fields_ = [("penalties", ctypes.c_void_p), ("counts", ctypes.c_void_p), ("seen", ctypes.c_void_p),
                ("n_slots", ctypes.c_int32), ("draft_tokens", ctypes.c_void_p),
                ("token_stride", ctypes.c_int64), ("bias_offsets", ctypes.c_void_p),
                ("bias_tokens", ctypes.c_void_p), ("bias_values", ctypes.c_void_p),
                ("n_bias", ctypes.c_int32), ("mask", ctypes.c_void_p),
                ("mask_stride_b", ctypes.c_int64), ("mask_stride_pos", ctypes.c_int64)]


class _Teacher(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_void_p), ("logits", ctypes.c_void_p), ("lse", ctypes.c_void_p),
                ("stride_b", ctypes.c_int64), ("K", ctypes.c_int32)]


_lib = None

# The current stream's handle without a Stream object around it (a tenth of
# the time), where torch offers it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def library_path():
    return os.environ.get("SPECV_LIBRARY", os.path.join(_HERE, "libspecv.so"))


def load_library():
    """Load libspecv.so (once).  Raises SpecvError if it is not built."""
    global _lib
    if _lib is not None:
        return _lib
    path = library_path()
    if not os.path.exists(path):
        raise SpecvError(f"libspecv.so not found at {path}; build it with "
                         "`python -m speculative_decoding_verification_sampling_amd.build`")
    lib = ctypes.CDLL(path)
    vp, i32, i64, u32, u64 = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64,
                              ctypes.c_uint32, ctypes.c_uint64)
    lib.specv_create.argtypes = [ctypes.POINTER(_Config), ctypes.POINTER(vp)]
    lib.specv_create.restype = ctypes.c_int
    lib.specv_destroy.argtypes = [vp]
    lib.specv_destroy.restype = ctypes.c_int
    lib.specv_status_string.argtypes = [ctypes.c_int]
    lib.specv_status_string.restype = ctypes.c_char_p
    lib.specv_verify_sample.argtypes = [
        vp, vp,
        vp, i64, i64,
        vp, i64, i64,
        ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int,
        vp, vp,
        u64, u32, i32,
        vp, vp, vp, vp,
        ctypes.POINTER(_Diag)]
    lib.specv_verify_sample.restype = ctypes.c_int
    lib.specv_verify_point_mass.argtypes = [
        vp, vp,
        vp, i64, i64,
        ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int,
        vp, vp,
        u64, u32, i32,
        vp, vp, vp, vp,
        ctypes.POINTER(_Diag)]
    lib.specv_verify_point_mass.restype = ctypes.c_int
    lib.specv_verify_sample_qstats.argtypes = [
        vp, vp,
        vp, i64, i64,
        vp, i64, i64,
        vp, i64,
        ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int,
        vp, vp,
        u64, u32, i32,
        vp, vp, vp, vp,
        ctypes.POINTER(_Diag)]
    lib.specv_verify_sample_qstats.restype = ctypes.c_int
    lib.specv_sample_draft.argtypes = [
        vp, vp,
        vp, i64, i64,
        ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int,
        vp, u64, u32,
        vp, vp, i64]
    lib.specv_sample_draft.restype = ctypes.c_int
    lib.specv_verify_greedy.argtypes = [
        vp, vp,
        vp, i64, i64,
        ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int,
        vp, vp, i32,
        vp, vp, vp, vp]
    lib.specv_verify_greedy.restype = ctypes.c_int
    lib.specv_set_profiling.argtypes = [vp, ctypes.c_int]
    lib.specv_set_profiling.restype = ctypes.c_int
    lib.specv_get_profile.argtypes = [vp, ctypes.c_int, ctypes.POINTER(ctypes.c_int),
                                      ctypes.POINTER(ctypes.c_double)]
    lib.specv_get_profile.restype = ctypes.c_int
    lib.specv_get_profile_samples.argtypes = [vp, ctypes.c_int, ctypes.POINTER(ctypes.c_float),
                                              ctypes.POINTER(ctypes.c_int)]
    lib.specv_get_profile_samples.restype = ctypes.c_int
    lib.specv_read_ceiling.argtypes = [vp, vp, i64, ctypes.c_int, vp]
    lib.specv_read_ceiling.restype = ctypes.c_int
    lib.specv_verify_sample_noalloc.argtypes = [ctypes.c_int] + lib.specv_verify_sample.argtypes[1:]
    lib.specv_verify_sample_noalloc.restype = ctypes.c_int
    c_int, f32 = ctypes.c_int, ctypes.c_float
    rows = [vp, i64, i64, c_int, c_int, c_int, c_int]              # pointer, strides, dtype, B, n, V
    teacher = [ctypes.POINTER(_Teacher), vp, f32, c_int]           # record, weights, temperature, tail
    lib.specv_adjust_logits.argtypes = [vp, vp, vp, i64, i64, vp, i64, i64, c_int, c_int, c_int, c_int, c_int,
                                        ctypes.POINTER(_Adjustments)]
    lib.specv_history_add.argtypes = [vp, vp, vp, vp, i64, vp, c_int, c_int, c_int, c_int, vp, vp, c_int]
    lib.specv_history_reset.argtypes = [vp, vp, vp, c_int, c_int, vp, vp, c_int]
    lib.specv_top_logits.argtypes = [vp, vp, *rows, c_int, f32, vp, vp, vp]
    lib.specv_distill_loss.argtypes = [vp, vp, *rows, *teacher, vp, vp, vp, vp, i64]
    lib.specv_distill_grad.argtypes = [vp, vp, *rows, *teacher, vp, vp, i64, i64]
    lib.specv_distill_loss_grad.argtypes = [vp, vp, *rows, *teacher, vp, vp, vp, i64, i64, vp, i64]
    lib.specv_distill_workspace.argtypes = [c_int] * 5
    lib.specv_distill_workspace.restype = i64
    for name in ("adjust_logits", "history_add", "history_reset", "top_logits", "distill_loss", "distill_grad",
                 "distill_loss_grad"):
        getattr(lib, "specv_" + name).restype = c_int
    _lib = lib
    return lib


def _check(status, what):
    if status != 0:
        msg = load_library().specv_status_string(status).decode()
        raise SpecvError(f"{what} failed: status {status} ({msg})")


def make_row_params(B, temperature=1.0, top_k=0, top_p=1.0, max_new_tokens=0, device="cuda"):
    """specv_row_params[B] as an int32 tensor [B, 4] on ``device``.

    Columns: temperature (float32 bits), top_k, top_p (float32 bits),
    max_new_tokens.  Each argument is a scalar or a length-B sequence.
    """
    rec = np.zeros(B, dtype=[("t", "<f4"), ("k", "<i4"), ("p", "<f4"), ("cap", "<i4")])
    rec["t"] = temperature
    rec["k"] = top_k
    rec["p"] = top_p
    rec["cap"] = max_new_tokens
    host = torch.from_numpy(rec.view(np.int32).reshape(B, 4).copy())
    return host.to(device)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


def _dtype_code(t):
    if t.dtype == torch.bfloat16:
        return SPECV_BF16
    if t.dtype == torch.float32:
        return SPECV_F32
    raise SpecvError(f"unsupported logits dtype {t.dtype} (float32 or bfloat16)")


def _rows(t, name, lead):
    if not t.is_cuda:
        raise SpecvError(f"{name} must be a device tensor")
    if t.dim() != 3 or (lead is not None and t.shape[0] != lead):
        raise SpecvError(f"{name} must be [B, positions, V], got {tuple(t.shape)}")
    if t.shape[2] > 1 and t.stride(2) != 1:
        raise SpecvError(f"{name} must be contiguous along the vocabulary")
    return t.stride(0), t.stride(1)


def verify_sample_noalloc(target, draft, tokens, row_params, seed, step=0, eos_id=-1, out=None,
                          diag=False):
    """specv_verify_sample_noalloc: Verifier.verify_sample without a handle,
    for callers that cannot allocate device memory (the library's static
    per-device scratch array; B <= 256, gamma <= 15, V <= 262144, no
    truncated rows).  Runs on the current torch device and stream.  The
    output tensors are allocated here unless ``out`` (and, with ``diag``,
    its diagnostics) are given."""
    B, g1, V = target.shape
    gamma = g1 - 1
    tsb, tsp = _rows(target, "target", None)
    dsb = dsp = 0
    if gamma > 0:
        dsb, dsp = _rows(draft, "draft", B)
        if draft.shape[1] != gamma or draft.shape[2] != V or draft.dtype != target.dtype:
            raise SpecvError("draft must be [B, gamma, V] with the target's dtype")
    for t, n in ((tokens, "tokens"), (row_params, "row_params")):
        if t.dtype != torch.int32 or not t.is_contiguous() or not t.is_cuda:
            raise SpecvError(f"{n} must be a contiguous int32 device tensor")
    if tokens.shape != (B, gamma) or row_params.shape != (B, 4):
        raise SpecvError("tokens must be [B, gamma] and row_params [B, 4]")
    dev = target.device
    if out is None:
        z = dict(dtype=torch.int32, device=dev)
        out = {"num_accepted": torch.empty(B, **z), "out_tokens": torch.empty(B, gamma + 1, **z),
               "num_emitted": torch.empty(B, **z), "row_flags": torch.empty(B, **z)}
    d = None
    if diag:
        for key, shape in (("p_at_draft", (B, gamma)), ("q_at_draft", (B, gamma)), ("residual_sum", (B,))):
            if key not in out:
                out[key] = torch.empty(*shape, dtype=torch.float32, device=dev)
        d = _Diag(out["p_at_draft"].data_ptr(), out["q_at_draft"].data_ptr(),
                  out["residual_sum"].data_ptr())
    st = load_library().specv_verify_sample_noalloc(
        dev.index if dev.index is not None else torch.cuda.current_device(),
        ctypes.c_void_p(torch.cuda.current_stream(dev).cuda_stream),
        _ptr(target), tsb, tsp, _ptr(draft if gamma > 0 else None), dsb, dsp,
        _dtype_code(target), B, gamma, V, _ptr(tokens), _ptr(row_params),
        int(seed) & 0xFFFFFFFFFFFFFFFF, int(step) & 0xFFFFFFFF, int(eos_id),
        _ptr(out["num_accepted"]), _ptr(out["out_tokens"]), _ptr(out["num_emitted"]),
        _ptr(out.get("row_flags")), ctypes.byref(d) if d is not None else None)
    _check(st, "specv_verify_sample_noalloc")
    return out


def read_ceiling(buf, grid, sink):
    """One streaming read of the device tensor ``buf`` (its bytes, a multiple
    of 16) by ``grid`` workgroups on the current stream (measurement aid);
    ``sink`` is an int32 device tensor of at least ``grid`` entries."""
    nbytes = buf.numel() * buf.element_size()
    if not buf.is_cuda or not buf.is_contiguous() or sink.numel() < grid or sink.dtype != torch.int32:
        raise SpecvError("read_ceiling needs a contiguous device buffer and an int32 sink of grid entries")
    st = load_library().specv_read_ceiling(ctypes.c_void_p(torch.cuda.current_stream().cuda_stream),
                                           _ptr(buf), nbytes, int(grid), _ptr(sink))
    _check(st, "specv_read_ceiling")


def debug_set_wait_limit(polls, device=None):
    """Failure-path tests only: the polls every bounded wait of the kernels
    makes before it gives up and flags its row INTERNAL (0 restores the
    default).  Process-wide for the device."""
    dev = torch.cuda.current_device() if device is None else int(device)
    fn = load_library().specv_debug_set_wait_limit
    fn.argtypes = [ctypes.c_int, ctypes.c_int32]
    fn.restype = ctypes.c_int
    _check(fn(dev, int(polls)), "specv_debug_set_wait_limit")


class TokenHistory:
    """Token histories of ``n_slots`` sequences for Verifier.adjust_logits:
    ``counts`` int32 [n_slots, vocab] (occurrences among the generated tokens)
    and ``seen`` int32 [n_slots, ceil(vocab / 32)] (bits: in the prompt or
    generated).  Empty at first; Verifier.history_add and history_reset keep
    them.  Existing tensors may be given instead."""

    def __init__(self, n_slots, vocab, device="cuda", counts=None, seen=None):
        self.n_slots, self.vocab = int(n_slots), int(vocab)
        self.words = (self.vocab + 31) // 32
        z = dict(dtype=torch.int32, device=device)
        self.counts = torch.zeros(self.n_slots, self.vocab, **z) if counts is None else counts
        self.seen = torch.zeros(self.n_slots, self.words, **z) if seen is None else seen
        for t, n, cols in ((self.counts, "counts", self.vocab), (self.seen, "seen", self.words)):
            if t.dtype != torch.int32 or not t.is_contiguous() or t.shape != (self.n_slots, cols):
                raise SpecvError(f"{n} must be a contiguous int32 [{self.n_slots}, {cols}] tensor")
        if self.counts.device != self.seen.device:
            raise SpecvError("counts and seen must be on one device")


def make_penalties(B, repetition=1.0, presence=0.0, frequency=0.0, slot=None, device="cuda"):
    """specv_penalties[B] as an int32 tensor [B, 4] on ``device``.  Columns:
    repetition, presence, frequency (float32 bits), slot.  Each argument is a
    scalar or a length-B sequence; ``slot`` defaults to the row's number, and
    -1 stands for an empty history.  repetition must be > 0."""
    rec = np.zeros(B, dtype=[("r", "<f4"), ("a", "<f4"), ("f", "<f4"), ("s", "<i4")])
    rec["r"] = repetition
    rec["a"] = presence
    rec["f"] = frequency
    rec["s"] = np.arange(B) if slot is None else slot
    if not (rec["r"] > 0).all():
        raise SpecvError("repetition must be > 0 (1: off)")
    return torch.from_numpy(rec.view(np.int32).reshape(B, 4).copy()).to(device)


def make_bias(rows, device="cuda"):
    """The (offsets, tokens, values) tensors of Verifier.adjust_logits from
    one {token: bias} dict (or list of (token, bias) pairs, or None) per batch
    row."""
    pairs = [list(r.items()) if isinstance(r, dict) else list(r or ()) for r in rows]
    offsets = np.zeros(len(pairs) + 1, np.int32)
    offsets[1:] = np.cumsum([len(p) for p in pairs])
    flat = [e for p in pairs for e in p]
    tokens = np.array([t for t, _ in flat], np.int32)
    values = np.array([x for _, x in flat], np.float32)
    return tuple(torch.from_numpy(x).to(device) for x in (offsets, tokens, values))


def pack_token_mask(allowed):
    """Truth values [..., V] (True: token allowed) as the bit words int32
    [..., ceil(V / 32)] of Verifier.adjust_logits, on the same device."""
    V = allowed.shape[-1]
    bits = torch.nn.functional.pad(allowed.to(torch.uint8), (0, -V % 32))
    bits = bits.view(*allowed.shape[:-1], -1, 8)
    weight = 1 << torch.arange(8, device=allowed.device, dtype=torch.uint8)
    return (bits * weight).sum(-1, dtype=torch.uint8).view(torch.int32)


class Verifier:
    """A libspecv handle: owns the device workspace for calls up to the given
    maxima.  Calls run on the current torch stream of the handle's device."""

    def __init__(self, max_batch, max_gamma, max_vocab, max_top_k=0, device=0):
        lib = load_library()
        self.device = int(device)
        cfg = _Config(self.device, int(max_batch), int(max_gamma), int(max_vocab), int(max_top_k))
        h = ctypes.c_void_p()
        _check(lib.specv_create(ctypes.byref(cfg), ctypes.byref(h)), "specv_create")
        self._h = h
        self.max_batch, self.max_gamma, self.max_vocab = max_batch, max_gamma, max_vocab
        self.max_top_k = max_top_k

    def close(self):
        if getattr(self, "_h", None) is not None and self._h.value:
            load_library().specv_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def set_profiling(self, enable=True):
        """Record HIP events around each kernel of later calls."""
        _check(load_library().specv_set_profiling(self._h, int(bool(enable))), "specv_set_profiling")

    def profile(self, reset=True):
        """(calls, summed kernel milliseconds) over profiled calls; waits for
        the recorded events."""
        n = ctypes.c_int()
        ms = ctypes.c_double()
        _check(load_library().specv_get_profile(self._h, int(bool(reset)), ctypes.byref(n),
                                                ctypes.byref(ms)),
               "specv_get_profile")
        return n.value, ms.value

    def profile_samples(self, max_samples=1 << 16):
        """Per-call kernel milliseconds recorded since the last reset (numpy
        float32); waits for the recorded events, does not reset."""
        buf = (ctypes.c_float * max_samples)()
        n = ctypes.c_int()
        _check(load_library().specv_get_profile_samples(self._h, max_samples, buf, ctypes.byref(n)),
               "specv_get_profile_samples")
        return np.frombuffer(buf, dtype=np.float32, count=n.value).copy()

    def _stream(self):
        if _raw_stream is not None:
            return ctypes.c_void_p(_raw_stream(self.device))
        return ctypes.c_void_p(torch.cuda.current_stream(self.device).cuda_stream)

    def _outputs(self, B, gamma, device, out):
        if out is not None:
            return out
        z = dict(dtype=torch.int32, device=device)
        return {"num_accepted": torch.empty(B, **z), "out_tokens": torch.empty(B, gamma + 1, **z),
                "num_emitted": torch.empty(B, **z), "row_flags": torch.empty(B, **z)}

    def verify_sample(self, target, draft, tokens, row_params, seed, step=0, eos_id=-1,
                      out=None, diag=False):
        """Stochastic verification.  target [B, gamma+1, V], draft [B, gamma, V]
        (same dtype), tokens int32 [B, gamma], row_params from make_row_params.
        Returns a dict of device tensors (plus p_at_draft, q_at_draft,
        residual_sum when ``diag``).  Asynchronous on the current stream."""
        return self._verify_two_model(target, draft, None, tokens, row_params, seed, step, eos_id,
                                      out, diag)

    def verify_sample_qstats(self, target, draft, draft_stats, tokens, row_params, seed, step=0,
                             eos_id=-1, out=None, diag=False):
        """Stochastic verification reusing the drafter's row statistics:
        draft_stats float32 [B, >= gamma, 4] records (max, sum, threshold,
        flags as int32 bits) per draft row, as ``sample_draft`` returns them.
        Otherwise as verify_sample."""
        return self._verify_two_model(target, draft, draft_stats, tokens, row_params, seed, step,
                                      eos_id, out, diag)

    def _verify_two_model(self, target, draft, draft_stats, tokens, row_params, seed, step, eos_id,
                          out, diag):
        B, g1, V = target.shape
        gamma = g1 - 1
        tsb, tsp = _rows(target, "target", None)
        dsb = dsp = 0
        if gamma > 0:
            dsb, dsp = _rows(draft, "draft", B)
            if draft.shape[1] != gamma or draft.shape[2] != V or draft.dtype != target.dtype:
                raise SpecvError("draft must be [B, gamma, V] with the target's dtype")
        for t, n in ((tokens, "tokens"), (row_params, "row_params")):
            if t.dtype != torch.int32 or not t.is_contiguous() or not t.is_cuda:
                raise SpecvError(f"{n} must be a contiguous int32 device tensor")
        if tokens.shape != (B, gamma) or row_params.shape != (B, 4):
            raise SpecvError("tokens must be [B, gamma] and row_params [B, 4]")
        o = self._outputs(B, gamma, target.device, out)
        d = None
        if diag:
            o["p_at_draft"] = torch.empty(B, gamma, dtype=torch.float32, device=target.device)
            o["q_at_draft"] = torch.empty(B, gamma, dtype=torch.float32, device=target.device)
            o["residual_sum"] = torch.empty(B, dtype=torch.float32, device=target.device)
            d = _Diag(o["p_at_draft"].data_ptr(), o["q_at_draft"].data_ptr(),
                      o["residual_sum"].data_ptr())
        common = (_dtype_code(target), B, gamma, V,
                  _ptr(tokens), _ptr(row_params),
                  int(seed) & 0xFFFFFFFFFFFFFFFF, int(step) & 0xFFFFFFFF, int(eos_id),
                  _ptr(o["num_accepted"]), _ptr(o["out_tokens"]), _ptr(o["num_emitted"]),
                  _ptr(o.get("row_flags")),
                  ctypes.byref(d) if d is not None else None)
        drows = (_ptr(target), tsb, tsp, _ptr(draft if gamma > 0 else None), dsb, dsp)
        if draft_stats is None:
            st = load_library().specv_verify_sample(self._h, self._stream(), *drows, *common)
            _check(st, "specv_verify_sample")
            return o
        if (draft_stats.dtype != torch.float32 or not draft_stats.is_cuda or draft_stats.dim() != 3
                or draft_stats.shape[0] != B or draft_stats.shape[1] < gamma
                or draft_stats.shape[2] != 4 or not draft_stats.is_contiguous()):
            raise SpecvError("draft_stats must be a contiguous float32 [B, >= gamma, 4] device tensor")
        st = load_library().specv_verify_sample_qstats(
            self._h, self._stream(), *drows, _ptr(draft_stats), draft_stats.shape[1], *common)
        _check(st, "specv_verify_sample_qstats")
        return o

    def sample_draft(self, draft, row_params, seed, step=0, pos0=0, width=None, out=None):
        """Draft-side sampler: d_i ~ q_i for positions pos0 .. pos0 + n - 1
        of the round, from draft logits [B, n, V] (float32 or bfloat16), with
        each row's statistics for verify_sample_qstats.  Returns
        {"tokens": int32 [B, width], "stats": float32 [B, width, 4],
        "flags": int32 [B, width]}: stats holds (max, sum, threshold, flags
        bits) records and "flags" is a view of their last field.  ``width``
        defaults to pos0 + n; pass ``out`` (such a dict) to fill columns of
        existing tensors, e.g. one position per call.  Asynchronous on the
        current stream."""
        B, n, V = draft.shape
        dsb, dsp = _rows(draft, "draft", None)
        if row_params.dtype != torch.int32 or not row_params.is_contiguous() or row_params.shape != (B, 4):
            raise SpecvError("row_params must be a contiguous int32 [B, 4] device tensor")
        if out is None:
            w = pos0 + n if width is None else int(width)
            st = torch.full((B, w, 4), float("nan"), dtype=torch.float32, device=draft.device)
            st.view(torch.int32)[..., 3] = 0
            out = {"tokens": torch.full((B, w), -1, dtype=torch.int32, device=draft.device),
                   "stats": st, "flags": st.view(torch.int32)[..., 3]}
        tok, sts = out["tokens"], out.get("stats")
        w = tok.shape[1]
        if tok.dtype != torch.int32 or not tok.is_contiguous() or tok.shape[0] != B:
            raise SpecvError("tokens output must be a contiguous int32 [B, width] tensor")
        if sts is not None and (sts.dtype != torch.float32 or not sts.is_contiguous()
                                or tuple(sts.shape) != (B, w, 4)):
            raise SpecvError("stats output must be a contiguous float32 [B, width, 4] tensor")
        st = load_library().specv_sample_draft(
            self._h, self._stream(), _ptr(draft), dsb, dsp, _dtype_code(draft), B, n, V, int(pos0),
            _ptr(row_params), int(seed) & 0xFFFFFFFFFFFFFFFF, int(step) & 0xFFFFFFFF,
            _ptr(tok), _ptr(sts), w)
        _check(st, "specv_sample_draft")
        return out

    def verify_point_mass(self, target, tokens, row_params, seed, step=0, eos_id=-1, out=None,
                          diag=False):
        """Stochastic verification against deterministic drafts (q_i is the
        point mass on d_i; no draft logits).  target [B, gamma+1, V], tokens
        int32 [B, gamma], row_params from make_row_params.  Returns a dict of
        device tensors as verify_sample."""
        B, g1, V = target.shape
        gamma = g1 - 1
        tsb, tsp = _rows(target, "target", None)
        for t, n in ((tokens, "tokens"), (row_params, "row_params")):
            if t.dtype != torch.int32 or not t.is_contiguous() or not t.is_cuda:
                raise SpecvError(f"{n} must be a contiguous int32 device tensor")
        if tokens.shape != (B, gamma) or row_params.shape != (B, 4):
            raise SpecvError("tokens must be [B, gamma] and row_params [B, 4]")
        o = self._outputs(B, gamma, target.device, out)
        d = None
        if diag:
            o["p_at_draft"] = torch.empty(B, gamma, dtype=torch.float32, device=target.device)
            o["q_at_draft"] = torch.empty(B, gamma, dtype=torch.float32, device=target.device)
            o["residual_sum"] = torch.empty(B, dtype=torch.float32, device=target.device)
            d = _Diag(o["p_at_draft"].data_ptr(), o["q_at_draft"].data_ptr(),
                      o["residual_sum"].data_ptr())
        st = load_library().specv_verify_point_mass(
            self._h, self._stream(),
            _ptr(target), tsb, tsp,
            _dtype_code(target), B, gamma, V,
            _ptr(tokens), _ptr(row_params),
            int(seed) & 0xFFFFFFFFFFFFFFFF, int(step) & 0xFFFFFFFF, int(eos_id),
            _ptr(o["num_accepted"]), _ptr(o["out_tokens"]), _ptr(o["num_emitted"]),
            _ptr(o.get("row_flags")),
            ctypes.byref(d) if d is not None else None)
        _check(st, "specv_verify_point_mass")
        return o

    def verify_greedy(self, target, tokens, max_new_tokens=None, eos_id=-1, out=None):
        """Greedy verification.  target [B, gamma+1, V], tokens int32 [B, gamma],
        max_new_tokens int32 [B] device tensor or None."""
        B, g1, V = target.shape
        gamma = g1 - 1
        tsb, tsp = _rows(target, "target", None)
        if tokens.dtype != torch.int32 or not tokens.is_contiguous() or tokens.shape != (B, gamma):
            raise SpecvError("tokens must be a contiguous int32 [B, gamma] device tensor")
        if max_new_tokens is not None and (max_new_tokens.dtype != torch.int32 or
                                           max_new_tokens.shape != (B,)):
            raise SpecvError("max_new_tokens must be an int32 [B] device tensor")
        o = self._outputs(B, gamma, target.device, out)
        st = load_library().specv_verify_greedy(
            self._h, self._stream(),
            _ptr(target), tsb, tsp,
            _dtype_code(target), B, gamma, V,
            _ptr(tokens), _ptr(max_new_tokens), int(eos_id),
            _ptr(o["num_accepted"]), _ptr(o["out_tokens"]), _ptr(o["num_emitted"]),
            _ptr(o.get("row_flags")))
        _check(st, "specv_verify_greedy")
        return o

    # ---- logits operators around a round

    def _on_device(self, t, name, dtype=None):
        if t.get_device() != self.device:
            raise SpecvError(f"{name} must be on the handle's device (cuda:{self.device})")
        if dtype is not None and t.dtype is not dtype:
            raise SpecvError(f"{name} must be {dtype}")

    def _dense(self, t, name, dtype, shape):
        if t.get_device() != self.device or t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
            raise SpecvError(f"{name} must be a contiguous {dtype} {list(shape)} tensor on cuda:{self.device}, got "
                             f"{t.dtype} {list(t.shape)} on {t.device}")
        return t.data_ptr()

    def _logits(self, t, name):
        """(address, strides of the first two dimensions, dtype code, B, n, V) of logits rows."""
        if t.get_device() != self.device:
            raise SpecvError(f"{name} must be on the handle's device (cuda:{self.device})")
        if t.dim() != 3:
            raise SpecvError(f"{name} must be [B, positions, V], got {tuple(t.shape)}")
        B, n, V = t.shape
        sb, sp, sv = t.stride()
        if sv != 1 and V > 1:
            raise SpecvError(f"{name} must be contiguous along the vocabulary")
        return t.data_ptr(), sb, sp, _dtype_code(t), B, n, V

    def _out_rows(self, t, name, like):
        if t.shape != like.shape or t.dtype is not like.dtype:
            raise SpecvError(f"{name} must be {like.dtype} {tuple(like.shape)}, got {t.dtype} {tuple(t.shape)}")
        return self._logits(t, name)[:3]

    def adjust_logits(self, logits, penalties=None, history=None, draft_tokens=None, pos0=0, bias=None,
                      mask=None, out=None):
        """Penalties, biases and grammar masks on logits [B, n, V] (float32 or
        bfloat16), the rows of positions pos0 .. pos0 + n - 1 of a round.

        penalties     from make_penalties, with ``history`` (a TokenHistory;
                      None: empty histories) and ``draft_tokens`` int32
                      [B, >= pos0 + n - 1], which count as generated at the
                      positions behind them (None: they do not)
        bias          (offsets, tokens, values) from make_bias
        mask          int32 bit words [B, n, ceil(V / 32)] from
                      pack_token_mask (rows may be broadcast); bit 0: -inf
        out           rows to write; ``logits`` itself: in place; None: new
                      rows

        Returns the written rows.  Asynchronous on the current stream."""
        ptr, isb, isp, code, B, n, V = self._logits(logits, "logits")
        if out is None:
            out = torch.empty(B, n, V, dtype=logits.dtype, device=logits.device)
        optr, osb, osp = self._out_rows(out, "out", logits)
        adj = _Adjustments()
        if penalties is not None:
            adj.penalties = self._dense(penalties, "penalties", torch.int32, (B, 4))
            if history is not None:
                if history.vocab != V:
                    raise SpecvError(f"history is of {history.vocab} tokens, the logits of {V}")
                self._on_device(history.counts, "history")
                adj.counts, adj.seen = history.counts.data_ptr(), history.seen.data_ptr()
                adj.n_slots = history.n_slots
            if draft_tokens is not None:
                if draft_tokens.dim() != 2 or draft_tokens.shape[1] < pos0 + n - 1:
                    raise SpecvError("draft_tokens must be a contiguous int32 [B, >= pos0 + n - 1] tensor")
                width = draft_tokens.shape[1]
                adj.draft_tokens = self._dense(draft_tokens, "draft_tokens", torch.int32, (B, width))
                adj.token_stride = width
        elif history is not None or draft_tokens is not None:
            raise SpecvError("history and draft_tokens need penalties")
        if bias is not None:
            offsets, tokens, values = bias
            n_bias = tokens.numel()
            adj.bias_offsets = self._dense(offsets, "bias offsets", torch.int32, (B + 1,))
            adj.bias_tokens = self._dense(tokens, "bias tokens", torch.int32, (n_bias,))
            adj.bias_values = self._dense(values, "bias values", torch.float32, (n_bias,))
            adj.n_bias = n_bias
        if mask is not None:
            self._on_device(mask, "mask", torch.int32)
            if mask.shape != (B, n, (V + 31) // 32) or (mask.shape[2] > 1 and mask.stride(2) != 1):
                raise SpecvError("mask must be int32 [B, n, ceil(V / 32)], contiguous along the words")
            adj.mask, adj.mask_stride_b, adj.mask_stride_pos = mask.data_ptr(), mask.stride(0), mask.stride(1)
        st = load_library().specv_adjust_logits(self._h, self._stream(), ptr, isb, isp, optr, osb, osp, code, B,
                                                n, V, int(pos0), ctypes.byref(adj))
        _check(st, "specv_adjust_logits")
        return out

    def _history_args(self, history, slots):
        self._on_device(history.counts, "history")
        return (self._dense(slots, "slots", torch.int32, (slots.numel(),)), history.counts.data_ptr(),
                history.seen.data_ptr(), history.n_slots)

    def history_add(self, history, slots, tokens, lengths=None, prompt=False):
        """Adds tokens int32 [B, n] to the histories of ``slots`` int32 [B],
        the first ``lengths`` int32 [B] of each row (None: all): as prompt
        tokens (seen, not counted) or as generated ones.  Entries outside the
        vocabulary are skipped, so a verify call's out_tokens can be given,
        with or without its num_emitted.  In place, on the current stream."""
        sptr, *h = self._history_args(history, slots)
        self._on_device(tokens, "tokens", torch.int32)
        B = slots.numel()
        if tokens.dim() != 2 or tokens.shape[0] != B or (tokens.shape[1] > 1 and tokens.stride(1) != 1):
            raise SpecvError("tokens must be int32 [B, n], contiguous along n")
        lptr = None if lengths is None else self._dense(lengths, "lengths", torch.int32, (B,))
        st = load_library().specv_history_add(
            self._h, self._stream(), sptr, tokens.data_ptr(), tokens.stride(0), lptr, B, tokens.shape[1],
            history.vocab, 1 if prompt else 0, *h)
        _check(st, "specv_history_add")

    def history_reset(self, history, slots):
        """Empties the histories of ``slots`` (int32 [n]), on the current
        stream."""
        sptr, *h = self._history_args(history, slots)
        st = load_library().specv_history_reset(self._h, self._stream(), sptr, slots.numel(), history.vocab, *h)
        _check(st, "specv_history_reset")

    def top_logits(self, logits, k, temperature=1.0):
        """The teacher's record of logits [B, n, V]: {"tokens": int32
        [B, n, k], "logits": float32 [B, n, k], "lse": float32 [B, n, 2]}, the
        k <= 256 largest logits by value (equal ones by token) and the
        log-sum-exps of logits / temperature over the row and over the tokens
        outside the record.  Asynchronous on the current stream."""
        rows = self._logits(logits, "logits")
        B, n = rows[4:6]
        k, dev = int(k), logits.device
        tokens = torch.empty((B, n, max(k, 0)), dtype=torch.int32, device=dev)
        values = torch.empty((B, n, max(k, 0)), dtype=torch.float32, device=dev)
        lse = torch.empty((B, n, 2), dtype=torch.float32, device=dev)
        st = load_library().specv_top_logits(self._h, self._stream(), *rows, k, temperature, tokens.data_ptr(),
                                             values.data_ptr(), lse.data_ptr())
        _check(st, "specv_top_logits")
        return {"tokens": tokens, "logits": values, "lse": lse}

    def _distill_args(self, student, record, weights, temperature, tail):
        rows = self._logits(student, "student")
        B, n = rows[4:6]
        if tail not in TAILS:
            raise SpecvError(f"tail must be one of {sorted(TAILS)}")
        tok, lse = record["tokens"], record.get("lse")
        if tok.dim() != 3 or tok.shape[0] != B or tok.shape[1] < n:
            raise SpecvError("the record's tokens must be int32 [B, >= n, K]")
        _, m, K = tok.shape
        if lse is None and tail == "bucket":
            raise SpecvError("tail='bucket' needs the record's lse")
        rec = _Teacher(self._dense(tok, "record tokens", torch.int32, (B, m, K)),
                       self._dense(record["logits"], "record logits", torch.float32, (B, m, K)),
                       None if lse is None else self._dense(lse, "record lse", torch.float32, (B, m, 2)), m, K)
        wptr = None if weights is None else self._dense(weights, "weights", torch.float32, (B, n))
        return (*rows, ctypes.byref(rec), wptr, temperature, TAILS[tail])

    def _distill_work(self, student, args, record):
        """(address, bytes, tensor) of a call's own workspace, from torch's
        allocator on the current stream; none where the library asks for none."""
        n = load_library().specv_distill_workspace(*args[3:7], record["tokens"].shape[2])
        if n == 0:
            return None, 0, None
        t = torch.empty(n, dtype=torch.uint8, device=student.device)
        return t.data_ptr(), n, t

    def distill_loss(self, student, record, weights=None, temperature=1.0, tail="bucket"):
        """Distillation loss of student logits [B, n, V] against a record of
        top_logits (of n positions or more: those behind the n-th, such as the
        bonus row, are left out), taken at ``temperature``.  ``weights``
        float32 [B, n] scale the rows' losses (None: 1).  tail: "bucket" (the
        tokens outside the record as one more outcome) or "renorm" (the
        teacher renormalised over the record).  Returns {"loss": float32
        [B, n], "lse": float32 [B, n, 2] (for distill_grad), "flags": int32
        [B, n]}.  Asynchronous on the current stream."""
        args = self._distill_args(student, record, weights, temperature, tail)
        B, n = args[4:6]
        loss = torch.empty((B, n), dtype=torch.float32, device=student.device)
        lse = torch.empty((B, n, 2), dtype=torch.float32, device=student.device)
        flags = torch.empty((B, n), dtype=torch.int32, device=student.device)
        work = self._distill_work(student, args, record)
        st = load_library().specv_distill_loss(self._h, self._stream(), *args, loss.data_ptr(), lse.data_ptr(),
                                               flags.data_ptr(), *work[:2])
        _check(st, "specv_distill_loss")
        return {"loss": loss, "lse": lse, "flags": flags}

    def _grad_rows(self, student, grad):
        if grad is None:
            grad = torch.empty(student.shape, dtype=student.dtype, device=student.device)
        return (grad, *self._out_rows(grad, "grad", student))

    def distill_grad(self, student, record, lse, weights=None, temperature=1.0, tail="bucket", grad=None):
        """Gradient of distill_loss's weighted losses with respect to the
        student's logits (in their dtype), from its ``lse``; ``grad`` may be
        given, also as ``student`` itself.  A gradient that reaches the losses
        goes into ``weights``.  Returns grad."""
        args = self._distill_args(student, record, weights, temperature, tail)
        lptr = self._dense(lse, "lse", torch.float32, (*args[4:6], 2))
        grad, gptr, gsb, gsp = self._grad_rows(student, grad)
        st = load_library().specv_distill_grad(self._h, self._stream(), *args, lptr, gptr, gsb, gsp)
        _check(st, "specv_distill_grad")
        return grad

    def distill_loss_grad(self, student, record, weights=None, temperature=1.0, tail="bucket", grad=None):
        """distill_loss and distill_grad in one call that reads the student's
        rows once, for weights known beforehand.  Returns {"loss", "grad",
        "flags"}; ``student.backward(out["grad"])`` takes the gradient on into
        the student's model."""
        args = self._distill_args(student, record, weights, temperature, tail)
        B, n = args[4:6]
        grad, gptr, gsb, gsp = self._grad_rows(student, grad)
        loss = torch.empty((B, n), dtype=torch.float32, device=student.device)
        flags = torch.empty((B, n), dtype=torch.int32, device=student.device)
        work = self._distill_work(student, args, record)
        st = load_library().specv_distill_loss_grad(self._h, self._stream(), *args, loss.data_ptr(),
                                                    flags.data_ptr(), gptr, gsb, gsp, *work[:2])
        _check(st, "specv_distill_loss_grad")
        return {"loss": loss, "grad": grad, "flags": flags}
