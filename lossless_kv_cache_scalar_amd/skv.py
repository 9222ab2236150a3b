"""Python binding of libskv (include/skv.h): argument marshalling only.

Every step of the coding path runs in the library's HIP kernels; this module
turns torch tensors into device pointers and the current torch stream into a
hipStream_t.  There is no fallback: if the library is not built, importing the
entry points raises.
"""
from __future__ import annotations

import contextlib
import ctypes as C
import os

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "_lib", "libskv.so")

OK, ERR_ARG, ERR_UNSUPPORTED, ERR_HIP, ERR_CAPACITY, ERR_CORRUPT, ERR_TABLE, ERR_SCRATCH, ERR_PAGES = range(9)
STATIC_SCRATCH_BYTES = 16 << 20  # SKV_STATIC_SCRATCH_BYTES
SYM_BF16, SYM_E4M3 = 0, 1
MU_BF16, MU_F32 = 0, 1
SIGMA_CHANNEL, SIGMA_OCTAVE = 0, 1
PHAT_STATIC, PHAT_ADAPTIVE = 0, 1
OCTAVES = 8
OCT_STRIDE = 1 + OCTAVES

# every function skv.h declares, in declaration order
EXPORTS = ["skv_status_string", "skv_num_chunks", "skv_encode_bound", "skv_workspace_size",
           "skv_calib_state_size", "skv_calib_reset", "skv_calib_accumulate", "skv_calib_finalize",
           "skv_calibrate", "skv_encode", "skv_decode", "skv_decode_static", "skv_pages_pool_size",
           "skv_pages_workspace_size", "skv_pages_reset", "skv_pages_extend", "skv_pages_fork", "skv_pages_truncate",
           "skv_pages_compact", "skv_pages_store", "skv_pages_gather", "skv_pages_scatter", "skv_attend_workspace_size",
           "skv_attend", "skv_timing_start", "skv_timing_stop", "skv_timed_kernel_name"]


class SkvShape(C.Structure):
    _fields_ = [("layers", C.c_int64), ("kv_heads", C.c_int64), ("tokens", C.c_int64),
                ("head_dim", C.c_int64), ("sym_fmt", C.c_int32), ("mu_fmt", C.c_int32),
                ("sigma_mode", C.c_int32), ("phat_mode", C.c_int32)]


class SkvPagesShape(C.Structure):
    _fields_ = [("layers", C.c_int64), ("kv_heads", C.c_int64), ("head_dim", C.c_int64), ("page_tokens", C.c_int64),
                ("n_pages", C.c_int64), ("max_seqs", C.c_int64), ("max_pages", C.c_int64), ("sym_fmt", C.c_int32),
                ("reserved", C.c_int32)]


class SkvPages(C.Structure):
    _fields_ = [("pool", C.c_void_p), ("table", C.c_void_p), ("lens", C.c_void_p), ("refs", C.c_void_p)]


# the current stream's address without a Stream object, where torch offers it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


class SkvError(RuntimeError):
    pass


_lib = None


def load():
    """Load libskv.so; raise if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise SkvError(f"libskv is not built ({LIB_PATH} missing); run python -m lossless_kv_cache_scalar_amd.build")
    L = C.CDLL(LIB_PATH)
    vp, i64, sz, i32p = C.c_void_p, C.c_int64, C.c_size_t, C.c_void_p
    sp = C.POINTER(SkvShape)
    L.skv_status_string.restype = C.c_char_p
    L.skv_status_string.argtypes = [C.c_int]
    for name in ("skv_num_chunks",):
        getattr(L, name).argtypes = [sp, C.POINTER(C.c_int64)]
    for name in ("skv_encode_bound", "skv_workspace_size", "skv_calib_state_size"):
        getattr(L, name).argtypes = [sp, C.POINTER(C.c_size_t)]
    L.skv_calib_reset.argtypes = [vp, sp, vp]
    L.skv_calib_accumulate.argtypes = [vp, sp, vp, vp, vp]
    L.skv_calib_finalize.argtypes = [vp, sp, vp, vp, vp]
    L.skv_calibrate.argtypes = [sp, i64, vp, vp, vp, vp, vp, vp]
    L.skv_encode.argtypes = [sp, vp, vp, vp, vp, vp, sz, vp, vp, sz, i32p, vp]
    L.skv_decode.argtypes = [sp, vp, sz, vp, vp, vp, vp, vp, vp, sz, i32p, vp]
    L.skv_decode_static.argtypes = [sp, vp, sz, vp, vp, vp, vp, vp, i32p, vp]
    pp, pg = C.POINTER(SkvPagesShape), C.POINTER(SkvPages)
    for name in ("skv_pages_pool_size", "skv_pages_workspace_size"):
        getattr(L, name).argtypes = [pp, C.POINTER(C.c_size_t)]
    L.skv_pages_reset.argtypes = [pp, pg, vp]
    L.skv_pages_extend.argtypes = [pp, pg, vp, vp, i64, vp, sz, i32p, vp]
    L.skv_pages_fork.argtypes = [pp, pg, vp, vp, vp, i64, vp, sz, i32p, vp]
    L.skv_pages_truncate.argtypes = [pp, pg, vp, vp, i64, vp, sz, i32p, vp]
    L.skv_pages_compact.argtypes = [pp, pg, vp, vp, sz, i32p, vp]
    L.skv_pages_store.argtypes = [pp, pg, i64, vp, i64, vp, i64, vp, vp, vp, vp, i64, i32p, vp]
    for name in ("skv_pages_gather", "skv_pages_scatter"):
        getattr(L, name).argtypes = [pp, pg, i64, i64, i64, vp, i32p, vp]
    L.skv_attend_workspace_size.argtypes = [pp, i64, C.POINTER(C.c_size_t)]
    L.skv_attend.argtypes = [pp, pg, i64, vp, i64, i64, C.c_float, vp, vp, vp, i64, vp, vp, vp, sz, i32p, vp]
    L.skv_timing_start.argtypes = [C.c_int32]
    L.skv_timing_stop.argtypes = [C.POINTER(C.c_int32), C.POINTER(C.c_float), C.c_int32, C.POINTER(C.c_int32)]
    L.skv_timed_kernel_name.argtypes = [C.c_int32]
    for name in EXPORTS[1:]:
        getattr(L, name).restype = C.c_int
    L.skv_timed_kernel_name.restype = C.c_char_p
    _lib = L
    return L


def shape(layers, kv_heads, tokens, head_dim, sym_fmt=SYM_BF16, mu_fmt=MU_BF16, sigma_mode=SIGMA_CHANNEL,
          phat_mode=PHAT_STATIC) -> SkvShape:
    return SkvShape(int(layers), int(kv_heads), int(tokens), int(head_dim), int(sym_fmt), int(mu_fmt),
                    int(sigma_mode), int(phat_mode))


def sigma_floats(sh: SkvShape) -> int:
    """Length of the sigma array for a shape: one per channel, or OCT_STRIDE per channel in octave mode."""
    nch = sh.layers * 2 * sh.kv_heads * sh.head_dim
    return nch * (OCT_STRIDE if sh.sigma_mode == SIGMA_OCTAVE else 1)


def status_string(code: int) -> str:
    return load().skv_status_string(int(code)).decode()


def _check(rc: int, what: str):
    if rc != OK:
        raise SkvError(f"{what}: {status_string(rc)} ({rc})")


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _fits(t, nbytes: int, what: str):
    """A tensor argument must be contiguous and hold at least nbytes (the
    library reads and writes whole arrays through raw pointers); integer
    addresses pass unchecked, as in C."""
    if isinstance(t, torch.Tensor):
        if not t.is_contiguous():
            raise SkvError(f"{what}: not contiguous")
        have = t.numel() * t.element_size()
        if have < nbytes:
            raise SkvError(f"{what}: {have} bytes, the shape needs {nbytes}")


def _offsets(sh: SkvShape, offsets):
    """offsets holds n_chunks + 1 entries (an invalid shape is left to the
    library, which returns its status code)."""
    n = C.c_int64(0)
    if load().skv_num_chunks(C.byref(sh), C.byref(n)) == OK:
        _fits(offsets, 8 * (n.value + 1), "offsets")


def _state(sh: SkvShape, state):
    n = C.c_size_t(0)
    if load().skv_calib_state_size(C.byref(sh), C.byref(n)) == OK:
        _fits(state, n.value, "state")


def _n_scalars(sh: SkvShape) -> int:
    return sh.layers * 2 * sh.kv_heads * sh.tokens * sh.head_dim


def _model_args(sh: SkvShape, mu, sigma, hist):
    n = _n_scalars(sh)
    _fits(mu, n * (2 if sh.mu_fmt == MU_BF16 else 4), "mu")
    _fits(sigma, 4 * sigma_floats(sh), "sigma")
    _fits(hist, 8 * (65536 if sh.sym_fmt == SYM_BF16 else 256), "hist")


def _symbols(sh: SkvShape, x, what: str):
    _fits(x, _n_scalars(sh) * (2 if sh.sym_fmt == SYM_BF16 else 1), what)


def _stream(stream):
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def num_chunks(sh: SkvShape) -> int:
    n = C.c_int64(0)
    _check(load().skv_num_chunks(C.byref(sh), C.byref(n)), "skv_num_chunks")
    return n.value


def _size(fn, sh):
    n = C.c_size_t(0)
    _check(getattr(load(), fn)(C.byref(sh), C.byref(n)), fn)
    return n.value


def encode_bound(sh: SkvShape) -> int:
    return _size("skv_encode_bound", sh)


def workspace_size(sh: SkvShape) -> int:
    return _size("skv_workspace_size", sh)


def calib_state_size(sh: SkvShape) -> int:
    return _size("skv_calib_state_size", sh)


# ---- raw entry points: same names and arguments as skv.h ----
def calib_reset(state, sh: SkvShape, stream=None) -> int:
    _state(sh, state)
    return load().skv_calib_reset(_ptr(state), C.byref(sh), _stream(stream))


def calib_accumulate(state, seq_shape: SkvShape, x, mu, stream=None) -> int:
    _state(seq_shape, state)
    _symbols(seq_shape, x, "x")
    _fits(mu, _n_scalars(seq_shape) * (2 if seq_shape.mu_fmt == MU_BF16 else 4), "mu")
    return load().skv_calib_accumulate(_ptr(state), C.byref(seq_shape), _ptr(x), _ptr(mu), _stream(stream))


def calib_finalize(state, sh: SkvShape, sigma, hist, stream=None) -> int:
    _state(sh, state)
    _fits(sigma, 4 * sigma_floats(sh), "sigma")
    _fits(hist, 8 * (65536 if sh.sym_fmt == SYM_BF16 else 256), "hist")
    return load().skv_calib_finalize(_ptr(state), C.byref(sh), _ptr(sigma), _ptr(hist), _stream(stream))


def calibrate(seq_shape: SkvShape, n_seq: int, x, mu, sigma, hist, state, stream=None) -> int:
    n = _n_scalars(seq_shape) * max(int(n_seq), 0)
    _fits(x, n * (2 if seq_shape.sym_fmt == SYM_BF16 else 1), "x")
    _fits(mu, n * (2 if seq_shape.mu_fmt == MU_BF16 else 4), "mu")
    _fits(sigma, 4 * sigma_floats(seq_shape), "sigma")
    _fits(hist, 8 * (65536 if seq_shape.sym_fmt == SYM_BF16 else 256), "hist")
    _state(seq_shape, state)
    return load().skv_calibrate(C.byref(seq_shape), int(n_seq), _ptr(x), _ptr(mu), _ptr(sigma), _ptr(hist),
                                _ptr(state), _stream(stream))


def encode(sh: SkvShape, x, mu, sigma, hist, bits, bits_cap: int, offsets, workspace, workspace_bytes: int,
           status, stream=None) -> int:
    _symbols(sh, x, "x")
    _model_args(sh, mu, sigma, hist)
    _fits(bits, int(bits_cap), "bits")
    _offsets(sh, offsets)
    _fits(workspace, int(workspace_bytes), "workspace")
    _fits(status, 4, "status")
    return load().skv_encode(C.byref(sh), _ptr(x), _ptr(mu), _ptr(sigma), _ptr(hist), _ptr(bits), int(bits_cap),
                             _ptr(offsets), _ptr(workspace), int(workspace_bytes), _ptr(status), _stream(stream))


def decode(sh: SkvShape, bits, bits_bytes: int, offsets, mu, sigma, hist, x_out, workspace, workspace_bytes: int,
           status, stream=None) -> int:
    _fits(bits, int(bits_bytes), "bits")
    _offsets(sh, offsets)
    _model_args(sh, mu, sigma, hist)
    _symbols(sh, x_out, "x_out")
    _fits(workspace, int(workspace_bytes), "workspace")
    _fits(status, 4, "status")
    return load().skv_decode(C.byref(sh), _ptr(bits), int(bits_bytes), _ptr(offsets), _ptr(mu), _ptr(sigma), _ptr(hist), _ptr(x_out),
                             _ptr(workspace), int(workspace_bytes), _ptr(status), _stream(stream))


def decode_static(sh: SkvShape, bits, bits_bytes: int, offsets, mu, sigma, hist, x_out, status, stream=None) -> int:
    _fits(bits, int(bits_bytes), "bits")
    _offsets(sh, offsets)
    _model_args(sh, mu, sigma, hist)
    _symbols(sh, x_out, "x_out")
    _fits(status, 4, "status")
    return load().skv_decode_static(C.byref(sh), _ptr(bits), int(bits_bytes), _ptr(offsets), _ptr(mu), _ptr(sigma),
                                    _ptr(hist), _ptr(x_out), _ptr(status), _stream(stream))


# ---- buffers sized for a shape (torch allocates, the library fills) ----
class Buffers:
    """Device buffers for one cache shape: workspace, stream, offsets, status."""

    def __init__(self, sh: SkvShape, device="cuda"):
        self.shape = sh
        self.n_chunks = num_chunks(sh)
        self.bound = encode_bound(sh)
        self.ws_bytes = workspace_size(sh)
        self.workspace = torch.empty(self.ws_bytes, dtype=torch.uint8, device=device)
        self.bits = torch.empty((self.bound + 15) // 16 * 16, dtype=torch.uint8, device=device)
        self.offsets = torch.empty(self.n_chunks + 1, dtype=torch.int64, device=device)
        self.status = torch.zeros(1, dtype=torch.int32, device=device)

    def encode(self, x, mu, sigma, hist, stream=None, status=None) -> None:
        """skv_encode into this object's stream; the status word is self.status unless given."""
        _check(encode(self.shape, x, mu, sigma, hist, self.bits, self.bits.numel(), self.offsets, self.workspace,
                      self.ws_bytes, self.status if status is None else status, stream), "skv_encode")

    def decode(self, mu, sigma, hist, x_out, bits=None, offsets=None, stream=None, status=None) -> None:
        """skv_decode of this object's stream (or the given one); the status word is self.status unless given."""
        bits = self.bits if bits is None else bits
        offsets = self.offsets if offsets is None else offsets
        _check(decode(self.shape, bits, bits.numel(), offsets, mu, sigma, hist, x_out, self.workspace,
                      self.ws_bytes, self.status if status is None else status, stream), "skv_decode")

    def stream_bytes(self) -> int:
        return int(self.offsets[-1].item())


def timing_start(capacity: int) -> None:
    """Start recording per-kernel HIP-event timings of the library's launches."""
    _check(load().skv_timing_start(int(capacity)), "skv_timing_start")


def timing_stop(capacity: int = 1 << 16):
    """Stop recording; [(kernel name, ms), ...] in launch order."""
    L = load()
    ids = (C.c_int32 * capacity)()
    ms = (C.c_float * capacity)()
    n = C.c_int32(0)
    _check(L.skv_timing_stop(ids, ms, int(capacity), C.byref(n)), "skv_timing_stop")
    return [(L.skv_timed_kernel_name(ids[i]).decode(), float(ms[i])) for i in range(min(n.value, capacity))]


def calibrate_sequences(seq_shape: SkvShape, seqs, device="cuda", stream=None):
    """sigma and hist from an iterable of (x, mu) device tensors, each of seq_shape."""
    nsym = 65536 if seq_shape.sym_fmt == SYM_BF16 else 256
    state = torch.empty(calib_state_size(seq_shape), dtype=torch.uint8, device=device)
    sigma = torch.empty(sigma_floats(seq_shape), dtype=torch.float32, device=device)
    hist = torch.empty(nsym, dtype=torch.int64, device=device)
    _check(calib_reset(state, seq_shape, stream), "skv_calib_reset")
    for x, mu in seqs:
        _check(calib_accumulate(state, seq_shape, x, mu, stream), "skv_calib_accumulate")
    _check(calib_finalize(state, seq_shape, sigma, hist, stream), "skv_calib_finalize")
    return sigma, hist


# ---- paged cache ----
def pages_shape(layers, kv_heads, head_dim, page_tokens, n_pages, max_seqs, max_pages, sym_fmt=SYM_BF16) -> SkvPagesShape:
    return SkvPagesShape(int(layers), int(kv_heads), int(head_dim), int(page_tokens), int(n_pages), int(max_seqs),
                         int(max_pages), int(sym_fmt), 0)


def pages_pool_size(sh: SkvPagesShape) -> int:
    return _size("skv_pages_pool_size", sh)


def pages_workspace_size(sh: SkvPagesShape) -> int:
    return _size("skv_pages_workspace_size", sh)


def attend_workspace_size(sh: SkvPagesShape, q_heads: int) -> int:
    n = C.c_size_t(0)
    _check(load().skv_attend_workspace_size(C.byref(sh), int(q_heads), C.byref(n)), "skv_attend_workspace_size")
    return n.value


class Pages:
    """A paged KV cache and the calls on it (skv.h, "paged cache").

    The arrays may be given (contiguous, of the shape's sizes) or are made here
    and emptied.  `q_heads` is the number of query heads `attend` will be called
    with (0: no attend).  Every call enqueues on `stream` or the current one and
    returns at once; errors that the device finds stay in `status` until
    `check()` reads and clears them.  Lists are int32 tensors on the cache's
    device, which has to be the current one.  The object's calls share its
    workspaces: on several streams they have to be ordered.  Tensors may be
    dropped after a call on the current stream, as after torch's own operations, or
    on a torch.cuda.Stream; those of a call on an address or an ExternalStream are
    to be kept until it has run, as in C.
    """

    def __init__(self, sh: SkvPagesShape, pool=None, table=None, lens=None, refs=None, q_heads: int = 0, device="cuda"):
        pool_bytes, ws = pages_pool_size(sh), pages_workspace_size(sh)
        att = attend_workspace_size(sh, q_heads) if q_heads else 0
        made = (pool, table, lens, refs)
        if any(t is None for t in made) and not all(t is None for t in made):
            raise SkvError("pool, table, lens and refs are given together, or none of them")
        new = pool is None
        if new:
            dt = torch.int16 if sh.sym_fmt == SYM_BF16 else torch.uint8
            pool = torch.empty(sh.layers, sh.n_pages, 2, sh.kv_heads, sh.page_tokens, sh.head_dim, dtype=dt, device=device)
            table = torch.empty(sh.max_seqs, sh.max_pages, dtype=torch.int32, device=device)
            lens = torch.empty(sh.max_seqs, dtype=torch.int32, device=device)
            refs = torch.empty(sh.n_pages, dtype=torch.int32, device=device)
        self.shape, self.q_heads, self._head_dim = sh, int(q_heads), sh.head_dim
        self._streams = set()  # on which the arrays were used by name
        self.pool, self.table, self.lens, self.refs = pool, table, lens, refs
        # a larger array has other rows than the library takes it to have
        self._esz = esz = 2 if sh.sym_fmt == SYM_BF16 else 1
        self._token_symbols = sh.layers * 2 * sh.kv_heads * sh.head_dim
        if pool.element_size() != esz or pool.numel() * esz != pool_bytes or not pool.is_contiguous():
            raise SkvError(f"pool: contiguous, {pool_bytes // esz} elements of {esz} bytes wanted")
        for t, want, what in ((table, (sh.max_seqs, sh.max_pages), "table"), (lens, (sh.max_seqs,), "lens"), (refs, (sh.n_pages,), "refs")):
            if t.dtype is not torch.int32 or t.shape != want or not t.is_contiguous():
                raise SkvError(f"{what}: contiguous int32 {list(want)} wanted")
        self.device, self._index = pool.device, pool.get_device() if pool.is_cuda else None
        for t, what in ((pool, "pool"), (table, "table"), (lens, "lens"), (refs, "refs")):
            self._here(t, what)
        self.ws_bytes, self.attend_bytes = ws, att
        self.workspace = torch.empty(ws, dtype=torch.uint8, device=self.device)
        self.attend_workspace = torch.empty(att, dtype=torch.uint8, device=self.device)
        self.status = torch.zeros(1, dtype=torch.int32, device=self.device)
        self._pages = SkvPages(pool.data_ptr(), table.data_ptr(), lens.data_ptr(), refs.data_ptr())
        self._sh, self._pg, self._lib = C.byref(sh), C.byref(self._pages), load()
        self._ws, self._aws, self._st = (t.data_ptr() for t in (self.workspace, self.attend_workspace, self.status))
        if new:
            self.reset()
        torch.cuda.current_stream(self.device).synchronize()  # the arrays are ready for calls on any stream

    def _here(self, t, what: str):
        if t.get_device() != self._index:  # -1: on the host
            raise SkvError(f"{what}: on {t.device}, not on the cache's GPU")

    def _call(self, stream, *given):
        """The stream of a call on the tensors `given`, once the cache's device is seen to be the current one."""
        if torch.cuda.current_device() != self._index:
            raise SkvError(f"the cache is on {self.device}, the current device is cuda:{torch.cuda.current_device()}")
        if stream is None and _raw_stream is not None:  # a tenth of the time of the Stream object
            return _raw_stream(self._index)
        self._keep(stream, *given)
        return _stream(stream)

    def _keep(self, stream, *given):
        """The tensors' memory, and the cache's own, goes to no other tensor before the stream has done with it.  An
        external stream may be gone by the time that a tensor is freed, and is not named to the allocator."""
        if isinstance(stream, torch.cuda.Stream) and not isinstance(stream, torch.cuda.ExternalStream):
            if _raw_stream is not None and stream.cuda_stream == _raw_stream(self._index):
                return  # the current one
            if stream.cuda_stream not in self._streams:
                self._streams.add(stream.cuda_stream)
                given += (self.pool, self.table, self.lens, self.refs, self.workspace, self.attend_workspace, self.status)
            for t in given:
                if t is not None:
                    t.record_stream(stream)

    def _made_on(self, stream):
        """What a call makes itself is made on the call's stream."""
        if stream is None:
            return contextlib.nullcontext()
        if not hasattr(stream, "cuda_stream"):  # an address; 0 is the default stream, which ExternalStream does not take
            address = int(stream)
            stream = torch.cuda.ExternalStream(address, self.device) if address else torch.cuda.default_stream(self.device)
        return torch.cuda.stream(stream)

    def _list(self, t, n, what: str):
        if not isinstance(t, torch.Tensor) or t.dtype is not torch.int32:
            raise SkvError(f"{what}: an int32 tensor is wanted")
        have = t.numel()
        if n is not None and have != n:
            raise SkvError(f"{what}: {have} entries, {n} wanted")
        if not t.is_contiguous():
            raise SkvError(f"{what}: not contiguous")
        if t.get_device() != self._index:
            self._here(t, what)
        return have

    def _rows(self, t, n, heads, what: str):
        """A bf16 [n][heads][head_dim] argument whose rows may lie apart; its row stride in elements."""
        d = self._head_dim
        if t.dtype is not torch.bfloat16 or t.shape != (n, heads, d):
            raise SkvError(f"{what}: {t.dtype} {list(t.shape)}, bfloat16 {[n, heads, d]} wanted")
        rows, one, unit = t.stride()
        if unit != 1 or (heads > 1 and one != d):
            raise SkvError(f"{what}: heads and channels are not contiguous")
        if t.get_device() != self._index:
            self._here(t, what)
        return rows if n > 1 else heads * d

    def _scales(self, t, what: str):
        if t is None:
            return None
        if t.dtype is not torch.float32 or t.shape != (self.shape.kv_heads,) or not t.is_contiguous():
            raise SkvError(f"{what}: {t.dtype} {list(t.shape)}, contiguous float32 {[self.shape.kv_heads]} wanted")
        self._here(t, what)
        return t.data_ptr()

    def reset(self, stream=None) -> None:
        """skv_pages_reset: no sequences, every page free."""
        _check(self._lib.skv_pages_reset(self._sh, self._pg, self._call(stream)), "skv_pages_reset")

    def check(self, stream=None) -> None:
        """Wait for the stream, then raise the first error that the device found since the last check."""
        with self._made_on(stream):
            code = int(self.status.item())
            if code != OK:
                self.status.zero_()
        if code != OK:
            raise SkvError(f"paged cache: {status_string(code)} ({code})")

    def extend(self, seqs, n_new, stream=None) -> None:
        """skv_pages_extend: room for n_new[i] more tokens of sequence seqs[i]."""
        n = self._list(seqs, None, "seqs")
        self._list(n_new, n, "n_new")
        _check(self._lib.skv_pages_extend(self._sh, self._pg, seqs.data_ptr(), n_new.data_ptr(), n, self._ws,
                                       self.ws_bytes, self._st, self._call(stream, seqs, n_new)), "skv_pages_extend")

    def fork(self, src, dst, n_tokens=None, stream=None) -> None:
        """skv_pages_fork: row dst[i] shares the pages of row src[i] (of its first n_tokens[i] tokens)."""
        n = self._list(src, None, "src")
        self._list(dst, n, "dst")
        if n_tokens is not None:
            self._list(n_tokens, n, "n_tokens")
        _check(self._lib.skv_pages_fork(self._sh, self._pg, src.data_ptr(), dst.data_ptr(), _ptr(n_tokens), n,
                                     self._ws, self.ws_bytes, self._st,
                                     self._call(stream, src, dst, n_tokens)), "skv_pages_fork")

    def truncate(self, seqs, keep=None, stream=None) -> None:
        """skv_pages_truncate: keep keep[i] tokens of sequence seqs[i]; free the rows without keep."""
        n = self._list(seqs, None, "seqs")
        if keep is not None:
            self._list(keep, n, "keep")
        _check(self._lib.skv_pages_truncate(self._sh, self._pg, seqs.data_ptr(), _ptr(keep), n, self._ws,
                                         self.ws_bytes, self._st, self._call(stream, seqs, keep)), "skv_pages_truncate")

    def compact(self, n_live=None, stream=None):
        """skv_pages_compact; the number of pages in use, an int32 tensor of one."""
        if n_live is None:
            with self._made_on(stream):
                n_live = torch.empty(1, dtype=torch.int32, device=self.device)
        self._list(n_live, 1, "n_live")
        _check(self._lib.skv_pages_compact(self._sh, self._pg, n_live.data_ptr(), self._ws, self.ws_bytes,
                                        self._st, self._call(stream, n_live)), "skv_pages_compact")
        return n_live

    def store(self, layer: int, k, v, seqs, pos, k_scale=None, v_scale=None, stream=None) -> None:
        """skv_pages_store: keys and values [n][kv_heads][head_dim] to positions pos of sequences seqs."""
        n = self._list(seqs, None, "seqs")
        self._list(pos, n, "pos")
        ks = self._rows(k, n, self.shape.kv_heads, "k")
        vs = self._rows(v, n, self.shape.kv_heads, "v")
        _check(self._lib.skv_pages_store(self._sh, self._pg, int(layer), k.data_ptr(), ks, v.data_ptr(), vs,
                                      self._scales(k_scale, "k_scale"), self._scales(v_scale, "v_scale"), seqs.data_ptr(),
                                      pos.data_ptr(), n, self._st, self._call(stream, k, v, seqs, pos, k_scale, v_scale)), "skv_pages_store")

    def coder_shape(self, tokens: int, mu_fmt=MU_BF16, sigma_mode=SIGMA_CHANNEL, phat_mode=PHAT_STATIC) -> SkvShape:
        """The coder's shape of `tokens` tokens of one sequence."""
        return shape(self.shape.layers, self.shape.kv_heads, tokens, self.shape.head_dim, self.shape.sym_fmt, mu_fmt,
                     sigma_mode, phat_mode)

    def _tokens(self, tokens: int, x, stream) -> bool:
        """Checks x, an array of `tokens` tokens in the coder's layout; False where the call is not made.

        An array whose rows hold more tokens may be meant with those apart, or packed at its start as the coder would
        read it: it is refused in the status, as a sequence that holds fewer tokens is."""
        esz, n = self._esz, self._token_symbols * max(tokens, 0)
        _fits(x, n * esz, "x")
        self._here(x, "x")
        size, flat = x.element_size(), x.dim() == 1  # flat: packed at its start, whatever lies behind; bytes too
        if size != esz and not (flat and x.dtype is torch.uint8):
            raise SkvError(f"x: elements of {size} bytes, the symbols have {esz}")
        if flat or x.numel() == n:
            return True
        rows, d = (self.shape.layers, 2, self.shape.kv_heads), self._head_dim
        if x.dim() != 5 or x.shape[:3] != rows or x.shape[4] != d:
            raise SkvError(f"x: {list(x.shape)}, {[*rows, tokens, d]} wanted")
        self._call(stream)
        with self._made_on(stream):
            self.status.masked_fill_(self.status == OK, ERR_ARG)
        return False

    def gather(self, seq: int, first: int, tokens: int, x=None, stream=None):
        """skv_pages_gather: tokens [first, first + tokens) of a sequence in the coder's layout, as encode() takes them.

        x, where it is given, is [layers][2][kv_heads][tokens][head_dim] symbols, or a flat buffer that begins with
        them.  One whose rows hold more tokens is left as it is, and check() reports an invalid argument."""
        sh, tokens = self.shape, int(tokens)
        if x is None:
            with self._made_on(stream):
                x = torch.empty(sh.layers, 2, sh.kv_heads, tokens, sh.head_dim, device=self.device,
                                dtype=torch.int16 if sh.sym_fmt == SYM_BF16 else torch.uint8)
        elif not self._tokens(tokens, x, stream):
            return x
        _check(self._lib.skv_pages_gather(self._sh, self._pg, int(seq), int(first), tokens, x.data_ptr(),
                                       self._st, self._call(stream, x)), "skv_pages_gather")
        return x

    def scatter(self, seq: int, first: int, tokens: int, x, stream=None) -> None:
        """skv_pages_scatter: the way back, from decode()'s output into the sequence's pages; x as gather() takes it."""
        tokens = int(tokens)
        if self._tokens(tokens, x, stream):
            _check(self._lib.skv_pages_scatter(self._sh, self._pg, int(seq), int(first), tokens, x.data_ptr(),
                                            self._st, self._call(stream, x)), "skv_pages_scatter")

    def attend(self, layer: int, q, seqs, scale=None, k_scale=None, v_scale=None, out=None, lse=None, stream=None):
        """skv_attend: attention of q [n][q_heads][head_dim], one token of each sequence in seqs, over the cached
        tokens; scale is 1 / sqrt(head_dim) unless given.  Without `out`, padded rows come back as zeros."""
        n = self._list(seqs, None, "seqs")
        if not self.q_heads:
            raise SkvError("attend: the cache was made without q_heads")
        qs = self._rows(q, n, self.q_heads, "q")
        if out is None:
            with self._made_on(stream):
                out = torch.zeros(n, self.q_heads, self.shape.head_dim, dtype=torch.bfloat16, device=self.device)
        elif self._rows(out, n, self.q_heads, "out") != self.q_heads * self.shape.head_dim:
            raise SkvError("out: not contiguous")
        if lse is not None:
            if lse.dtype is not torch.float32 or lse.shape != (n, self.q_heads) or not lse.is_contiguous():
                raise SkvError(f"lse: {lse.dtype} {list(lse.shape)}, contiguous float32 {[n, self.q_heads]} wanted")
            if lse.get_device() != self._index:
                self._here(lse, "lse")
        if scale is None:
            scale = self.shape.head_dim ** -0.5
        _check(self._lib.skv_attend(self._sh, self._pg, int(layer), q.data_ptr(), qs, self.q_heads, float(scale),
                                 self._scales(k_scale, "k_scale"), self._scales(v_scale, "v_scale"), seqs.data_ptr(), n,
                                 out.data_ptr(), _ptr(lse), self._aws, self.attend_bytes,
                                 self._st, self._call(stream, q, k_scale, v_scale, seqs, out, lse)), "skv_attend")
        return out

