"""ctypes binding of libspecverify with the same entry-point names as the C ABI.

Argument marshalling only: every step runs in the library's CUDA kernels.
Tensors are torch CUDA tensors (torch provides device memory and streams):

* ``wq``      int32 [N, K*bits/32]  (uint32 words reinterpreted)
* ``scales``  float16 [N, K/64],  ``biases`` float16 [N, K/64]
* activations bfloat16, logits / probabilities float32, tokens int32

Each call raises ``SVError`` when the library returns a non-OK status.  There
is no fallback: if the shared library is missing or the tensors are not on a
CUDA device the call fails.
"""

import ctypes
import os
import re

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libspecverify.so")
HEADER = os.path.join(os.path.dirname(HERE), "include", "specverify.h")

SV_OK, SV_EINVAL, SV_EUNSUPPORTED, SV_ECUDA, SV_ETIMEOUT = range(5)

_c_void_p, _c_int, _c_size_t, _c_float, _c_u64 = (ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t,
                                                  ctypes.c_float, ctypes.c_uint64)
_c_uint_p = ctypes.POINTER(ctypes.c_uint)
_c_i32_p = ctypes.POINTER(ctypes.c_int32)

class QWeight(ctypes.Structure):
    _fields_ = [("wq", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("biases", ctypes.c_void_p),
                ("N", ctypes.c_int), ("K", ctypes.c_int), ("packed", ctypes.c_void_p)]


class Layer(ctypes.Structure):
    _fields_ = [("qkv", QWeight), ("o", QWeight), ("gate_up", QWeight), ("down", QWeight)]


class Model(ctypes.Structure):
    _fields_ = [("n_layers", ctypes.c_int), ("hidden", ctypes.c_int), ("q_dim", ctypes.c_int),
                ("inter", ctypes.c_int), ("vocab", ctypes.c_int), ("bits", ctypes.c_int),
                ("rms_eps", ctypes.c_float), ("layers", ctypes.POINTER(Layer)), ("lm_head", QWeight)]


_c_model_p = ctypes.POINTER(Model)


class KVCacheView(ctypes.Structure):
    """sv_kv_cache."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scales", ctypes.c_void_p),
                ("k_biases", ctypes.c_void_p), ("v_scales", ctypes.c_void_p), ("v_biases", ctypes.c_void_p),
                ("n_pages", ctypes.c_int), ("page_size", ctypes.c_int), ("n_kv_heads", ctypes.c_int),
                ("head_dim", ctypes.c_int), ("bits", ctypes.c_int)]


_c_kv_p = ctypes.POINTER(KVCacheView)


class KVCache:
    """One layer's paged cache: its tensors (kept alive here) and the sv_kv_cache over them."""

    def __init__(self, view, tensors):
        self.view, self.tensors, self.ref = view, tensors, ctypes.byref(view)
        self.k, self.v = tensors[0], tensors[1]
        self.device, self.index = self.k.device, self.k.get_device()
        self.head_dim, self.width = view.head_dim, view.n_kv_heads * view.head_dim


class KVLayers:
    """The caches of several layers as one host array of sv_kv_cache."""

    def __init__(self, caches):
        self.caches = list(caches)
        if not self.caches or any(c.device != self.caches[0].device for c in self.caches):
            raise SVError(SV_EINVAL, "the layers' caches must be on one device, and at least one")
        self.array = (KVCacheView * len(self.caches))(*[c.view for c in self.caches])
        self.device, self.index = self.caches[0].device, self.caches[0].index


class PrefixGroups:
    """Groups of a batch's requests and the pages that each shares, as host arrays."""

    def __init__(self, offsets, pages):
        self.offsets, self.pages, self.n = offsets, pages, len(pages)


class KVPagesView(ctypes.Structure):
    """sv_kv_pages."""
    _fields_ = [("refs", ctypes.c_void_p), ("block_table", ctypes.c_void_p), ("held", ctypes.c_void_p),
                ("n_pages", ctypes.c_int), ("page_size", ctypes.c_int), ("slots", ctypes.c_int), ("table_pages", ctypes.c_int)]


_c_pages_p = ctypes.POINTER(KVPagesView)


class KVPages:
    """Who has which page: the state's tensors (kept alive here) and the sv_kv_pages over them."""

    def __init__(self, view, refs, block_table, held):
        self.view, self.ref = view, ctypes.byref(view)
        self.refs, self.block_table, self.held = refs, block_table, held
        self.device, self.index, self.slots = refs.device, refs.get_device(), view.slots


SV_CAP_MAX = 31


class CapState(ctypes.Structure):
    """sv_cap_controller (host memory)."""
    _fields_ = [("max_cap", ctypes.c_int), ("verify_us", ctypes.c_double * (SV_CAP_MAX + 1)),
                ("draft_us", ctypes.c_double * (SV_CAP_MAX + 1)), ("overhead_us", ctypes.c_double),
                ("alpha", ctypes.c_double), ("probe_every", ctypes.c_int), ("probe_cap", ctypes.c_int),
                ("S", ctypes.c_double), ("F", ctypes.c_double), ("parked", ctypes.c_int),
                ("since_probe", ctypes.c_int)]


_c_cap_p = ctypes.POINTER(CapState)
_c_f64_p = ctypes.POINTER(ctypes.c_double)
_c_int_p = ctypes.POINTER(ctypes.c_int)

_SIGNATURES = {
    "sv_status_string": (ctypes.c_char_p, [_c_int]),
    "sv_last_error": (ctypes.c_char_p, []),
    "sv_version": (_c_int, []),
    "sv_device_error": (_c_int, [_c_uint_p]),
    "sv_selftest_bounded_wait": (_c_int, [ctypes.c_uint, _c_void_p]),
    "sv_qmm_workspace_bytes": (_c_size_t, [_c_int, _c_int, _c_int, _c_int]),
    "sv_qmm_verify": (_c_int, [_c_void_p, _c_void_p, _c_void_p, _c_int, _c_int, _c_int, _c_int, _c_void_p, _c_int,
                               _c_int, _c_void_p, _c_int, _c_void_p, _c_int, _c_void_p, _c_size_t, _c_void_p]),
    "sv_qmm_noalloc_scratch_bytes": (_c_size_t, []),
    "sv_qmm_verify_noalloc": (_c_int, [_c_void_p, _c_void_p, _c_void_p, _c_int, _c_int, _c_int, _c_int, _c_void_p,
                                       _c_int, _c_int, _c_void_p, _c_int, _c_void_p, _c_int, _c_void_p]),
    "sv_qmm_prepare": (_c_int, [_c_void_p, _c_int, _c_int, _c_int, _c_int, _c_int, _c_void_p, _c_int, _c_void_p,
                                _c_float, _c_void_p, _c_size_t, _c_void_p]),
    "sv_qmm_run": (_c_int, [_c_void_p, _c_void_p, _c_void_p, _c_int, _c_int, _c_int, _c_int, _c_int, _c_void_p,
                            _c_int, _c_void_p, _c_int, _c_void_p, _c_size_t, _c_void_p]),
    "sv_lm_head_workspace_bytes": (_c_size_t, [_c_int, _c_int, _c_int, _c_int]),
    "sv_lm_head_run": (_c_int, [_c_void_p, _c_void_p, _c_void_p, _c_int, _c_int, _c_int, _c_int, _c_int, _c_float,
                                _c_void_p, _c_int, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_size_t,
                                _c_void_p]),
    "sv_round_workspace_bytes": (_c_size_t, [_c_model_p, _c_int]),
    "sv_qmm_pack_bytes": (_c_size_t, [_c_int, _c_int, _c_int]),
    "sv_qmm_pack": (_c_int, [_c_void_p, _c_void_p, _c_void_p, _c_int, _c_int, _c_int, _c_int, _c_void_p, _c_size_t,
                             _c_void_p]),
    "sv_round_plan_bytes": (_c_size_t, [_c_model_p]),
    "sv_round_plan_init": (_c_int, [_c_model_p, _c_void_p, _c_size_t]),
    "sv_verify_round": (_c_int, [_c_model_p, _c_void_p, _c_int, _c_i32_p, _c_void_p, _c_int, _c_float, _c_void_p, _c_int,
                                 _c_void_p, _c_void_p, _c_void_p, _c_int, _c_void_p, _c_void_p, _c_void_p,
                                 _c_size_t, _c_void_p, _c_void_p, _c_void_p, _c_void_p]),
    "sv_lm_head_verify": (_c_int, [_c_void_p, _c_void_p, _c_void_p, _c_int, _c_int, _c_int, _c_int, _c_void_p,
                                   _c_int, _c_int, _c_float, _c_void_p, _c_int, _c_void_p, _c_void_p, _c_void_p,
                                   _c_void_p, _c_size_t, _c_void_p]),
    "sv_accept_workspace_bytes": (_c_size_t, [_c_int, _c_int]),
    "sv_spec_accept": (_c_int, [_c_void_p, _c_int, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_int, _c_void_p,
                                _c_int, _c_int, _c_float, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_size_t,
                                _c_void_p]),
    "sv_spec_accept_batched": (_c_int, [_c_int, _c_i32_p, _c_void_p, _c_int, _c_void_p, _c_void_p, _c_void_p,
                                        _c_void_p, _c_int, _c_void_p, _c_int, _c_float, _c_void_p, _c_void_p,
                                        _c_void_p, _c_void_p, _c_size_t, _c_void_p]),
    "sv_philox_uniforms": (_c_int, [_c_u64, _c_u64, _c_u64, _c_int, _c_void_p, _c_void_p]),
    "sv_rmsnorm": (_c_int, [_c_void_p, _c_int, _c_int, _c_int, _c_void_p, _c_float, _c_void_p, _c_int, _c_void_p]),
    "sv_residual_add": (_c_int, [_c_void_p, _c_int, _c_void_p, _c_int, _c_int, _c_int, _c_void_p]),
    "sv_swiglu": (_c_int, [_c_void_p, _c_int, _c_void_p, _c_int, _c_int, _c_int, _c_void_p, _c_int, _c_void_p]),
    "sv_spec_accept_truncated": (_c_int, [_c_int, _c_i32_p, _c_void_p, _c_int, _c_void_p, _c_void_p, _c_void_p,
                                          _c_void_p, _c_int, _c_void_p, _c_int, _c_float, _c_void_p, _c_int,
                                          _c_float, _c_void_p, _c_void_p, _c_void_p, _c_size_t, _c_void_p]),
    "sv_truncate_probs": (_c_int, [_c_void_p, _c_int, _c_void_p, _c_int, _c_int, _c_int, _c_int, _c_float,
                                   _c_void_p]),
    "sv_logprobs": (_c_int, [_c_void_p, _c_int, _c_int, _c_int, _c_float, _c_void_p, _c_int, _c_void_p, _c_void_p,
                             _c_void_p, _c_void_p]),
    "sv_gather_qmm_workspace_bytes": (_c_size_t, [_c_int, _c_int, _c_int, _c_int, _c_int, _c_int]),
    "sv_gather_qmm": (_c_int, [_c_void_p, _c_void_p, _c_void_p, _c_int, _c_int, _c_int, _c_int, _c_int, _c_void_p,
                               _c_int, _c_int, _c_void_p, _c_void_p, _c_int, _c_void_p, _c_int, _c_void_p,
                               _c_size_t, _c_void_p]),
    "sv_qk_norm_rope": (_c_int, [_c_void_p, _c_int, _c_void_p, _c_int, _c_int, _c_int, _c_int, _c_int, _c_int,
                                 _c_void_p, _c_void_p, _c_float, _c_void_p, _c_void_p, _c_int, _c_int, _c_void_p,
                                 _c_int, _c_void_p, _c_int, _c_void_p]),
    "sv_kv_append": (_c_int, [_c_kv_p, _c_int, _c_i32_p, _c_void_p, _c_void_p, _c_int, _c_void_p, _c_int, _c_void_p,
                              _c_int, _c_void_p]),
    "sv_kv_read": (_c_int, [_c_kv_p, _c_int, _c_i32_p, _c_void_p, _c_void_p, _c_int, _c_void_p, _c_int, _c_void_p,
                            _c_int, _c_void_p]),
    "sv_tree_attention_workspace_bytes": (_c_size_t, [_c_kv_p, _c_int, _c_i32_p, _c_int]),
    "sv_tree_attention": (_c_int, [_c_kv_p, _c_int, _c_i32_p, _c_void_p, _c_void_p, _c_int, _c_void_p, _c_int, _c_int,
                                   _c_float, _c_void_p, _c_void_p, _c_int, _c_void_p, _c_size_t, _c_void_p]),
    "sv_kv_commit": (_c_int, [_c_kv_p, _c_int, _c_int, _c_void_p, _c_void_p, _c_int, _c_void_p, _c_int, _c_void_p,
                              _c_void_p]),
    "sv_tree_attention_shared_workspace_bytes": (_c_size_t, [_c_kv_p, _c_int, _c_i32_p, _c_i32_p, _c_int, _c_i32_p, _c_int]),
    "sv_tree_attention_shared": (_c_int, [_c_kv_p, _c_int, _c_i32_p, _c_i32_p, _c_int, _c_i32_p, _c_void_p, _c_void_p, _c_int,
                                          _c_void_p, _c_int, _c_int, _c_float, _c_void_p, _c_void_p, _c_int, _c_void_p,
                                          _c_size_t, _c_void_p]),
    "sv_tree_accept_workspace_bytes": (_c_size_t, [_c_int]),
    "sv_tree_accept": (_c_int, [_c_int, _c_i32_p, _c_void_p, _c_int, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p,
                                _c_void_p, _c_int, _c_int, _c_int, _c_float, _c_void_p, _c_int, _c_float, _c_void_p, _c_void_p,
                                _c_void_p, _c_int, _c_void_p, _c_size_t, _c_void_p]),
    "sv_kv_fork": (_c_int, [_c_pages_p, _c_int, _c_void_p, _c_void_p, _c_void_p, _c_void_p]),
    "sv_kv_reserve_workspace_bytes": (_c_size_t, [_c_pages_p]),
    "sv_kv_reserve": (_c_int, [_c_pages_p, _c_kv_p, _c_int, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_size_t,
                               _c_void_p]),
    "sv_kv_compact": (_c_int, [_c_pages_p, _c_kv_p, _c_int, _c_void_p, _c_void_p, _c_void_p]),
    "sv_kv_copy_pages": (_c_int, [_c_kv_p, _c_kv_p, _c_int, _c_int, _c_void_p, _c_void_p, _c_void_p]),
    "sv_expected_committed": (ctypes.c_double, [ctypes.c_double, _c_int]),
    "sv_best_cap": (_c_int, [ctypes.c_double, _c_int, _c_f64_p, _c_f64_p, ctypes.c_double, _c_int_p, _c_f64_p]),
    "sv_verify_knee": (_c_int, [_c_f64_p, _c_int, ctypes.c_double, _c_int_p]),
    "sv_cap_init": (_c_int, [_c_cap_p, _c_int, _c_f64_p, _c_f64_p, ctypes.c_double, ctypes.c_double, _c_int, _c_int,
                             ctypes.c_double]),
    "sv_cap_next": (_c_int, [_c_cap_p, _c_int_p]),
    "sv_cap_update": (_c_int, [_c_cap_p, _c_int, _c_int]),
    "sv_cap_acceptance": (ctypes.c_double, [_c_cap_p]),
}


def _f64_array(values):
    arr = (ctypes.c_double * len(values))(*[float(v) for v in values])
    return ctypes.cast(arr, _c_f64_p), arr


class CapController:
    """sv_cap_controller: per-round draft cap from measured costs (host only)."""

    def __init__(self, lib, max_cap, verify_us, draft_us, overhead_us, alpha, probe_every, probe_cap, p0):
        self.lib, self.state = lib, CapState()
        v, self._v = _f64_array(verify_us)
        d, self._d = _f64_array(draft_us)
        _check(lib, lib.sv_cap_init(ctypes.byref(self.state), max_cap, v, d, overhead_us, alpha, probe_every,
                                    probe_cap, p0))

    def next_cap(self):
        c = ctypes.c_int()
        _check(self.lib, self.lib.sv_cap_next(ctypes.byref(self.state), ctypes.byref(c)))
        return c.value

    def update(self, cap, accepted):
        _check(self.lib, self.lib.sv_cap_update(ctypes.byref(self.state), cap, accepted))

    def p(self):
        return self.lib.sv_cap_acceptance(ctypes.byref(self.state))

    @property
    def parked(self):
        return bool(self.state.parked)


def best_cap(lib, p, verify_us, draft_us, overhead_us):
    """(cap, rate) from sv_best_cap; max_cap = len(verify_us) - 1."""
    v, _v = _f64_array(verify_us)
    d, _d = _f64_array(draft_us)
    c, r = ctypes.c_int(), ctypes.c_double()
    _check(lib, lib.sv_best_cap(p, len(verify_us) - 1, v, d, overhead_us, ctypes.byref(c), ctypes.byref(r)))
    return c.value, r.value


def verify_knee(lib, verify_us, tol):
    v, _v = _f64_array(verify_us)
    w = ctypes.c_int()
    _check(lib, lib.sv_verify_knee(v, len(verify_us), tol, ctypes.byref(w)))
    return w.value


def _check(lib, status):
    if status != SV_OK:
        raise SVError(status, lib.sv_last_error().decode())


class SVError(RuntimeError):
    def __init__(self, status, detail):
        super().__init__("%s (status %d): %s" % (_STATUS_NAMES.get(status, "?"), status, detail))
        self.status = status


_STATUS_NAMES = {0: "SV_OK", 1: "SV_EINVAL", 2: "SV_EUNSUPPORTED", 3: "SV_ECUDA", 4: "SV_ETIMEOUT"}


def header_functions():
    """Names of the functions declared in include/specverify.h."""
    text = open(HEADER).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"^[A-Za-z_][\w\s\*]*?\b(sv_\w+)\s*\(", text, flags=re.M)))


def load_library(path=LIB_PATH):
    """dlopen the library and attach the argument types (no device work)."""
    if not os.path.exists(path):
        raise RuntimeError("libspecverify.so is not built (run __graft_entry__.build())")
    lib = ctypes.CDLL(path)
    for name, (res, args) in _SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


# Checks of the attention-side calls.  They run on every call of a latency-bound step, so each asks a tensor for as little
# as it can: dtypes by identity, devices by index.

def _refuse(what, t):
    raise SVError(SV_EINVAL, "%s, got %s %s with strides %s on %s" % (what, t.dtype, tuple(t.shape), t.stride(), t.device))


_INT_MAX = 2 ** 31 - 1      # sizes and strides are C ints


def _matrix(name, t, dtype, dev, rows, width):
    """Row stride of a [>= rows, >= width] matrix on device `dev` with adjacent elements; anything else is refused."""
    shape, strides = t.shape, t.stride()
    if t.dtype is not dtype or t.get_device() != dev or len(shape) != 2 or shape[0] < rows or shape[1] < width \
            or (strides[1] != 1 and width > 1):
        _refuse("%s must be a %s [%d, %d] matrix on cuda:%d with unit inner stride" % (name, dtype, rows, width, dev), t)
    stride = strides[0] if shape[0] > 1 else min(max(strides[0], width), _INT_MAX)
    if stride > _INT_MAX:
        _refuse("the row stride of %s must be below 2^31" % name, t)
    return stride


def _vector(name, t, dtype, dev, n):
    """Data pointer of a contiguous tensor of at least n elements on device `dev`; anything else is refused."""
    if t.dtype is not dtype or t.get_device() != dev or t.numel() < n or not t.is_contiguous():
        _refuse("%s must be a contiguous %s tensor of %d elements on cuda:%d" % (name, dtype, n, dev), t)
    return t.data_ptr()


def _empty(shape, dtype, device, stream):
    """An uninitialized tensor from the pool of the stream that writes it: memory just freed on another stream may still
    be in use there."""
    import torch
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _table(t, dtype, dev, B):
    """(data pointer, width) of a block table."""
    shape = t.shape
    if t.dtype is not dtype or t.get_device() != dev or len(shape) != 2 or shape[0] < B or shape[1] > _INT_MAX or not t.is_contiguous():
        _refuse("block_table must be a contiguous %s [%d, pages] tensor on cuda:%d" % (dtype, B, dev), t)
    return t.data_ptr(), shape[1]


class Library:
    """The loaded library plus tensor-level helpers named after the C calls."""

    def __init__(self, path=LIB_PATH):
        self.lib = load_library(path)
        self._torch = None

    # -------------------------------------------------------------- plumbing
    def check(self, status):
        if status != SV_OK:
            raise SVError(status, self.lib.sv_last_error().decode())

    def device_error(self):
        bits = ctypes.c_uint(0)
        st = self.lib.sv_device_error(ctypes.byref(bits))
        if st not in (SV_OK, SV_ETIMEOUT):
            self.check(st)
        return bits.value

    @staticmethod
    def workspace(nbytes, device="cuda"):
        """A zero-filled, 256-byte aligned device buffer (torch allocates it)."""
        import torch
        return torch.zeros(max(int(nbytes), 256), dtype=torch.uint8, device=device)

    # ------------------------------------------------------------------ qmm
    def qmm_workspace_bytes(self, M, N, K, bits):
        return self.lib.sv_qmm_workspace_bytes(M, N, K, bits)

    def qmm_verify(self, wq, scales, biases, K, bits, x, y=None, residual=None, workspace=None, stream=None):
        import torch
        M, N = x.shape[0], wq.shape[0]
        if y is None:
            y = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
        if workspace is None:
            workspace = self.workspace(self.qmm_workspace_bytes(M, N, K, bits), x.device)
        self.check(self.lib.sv_qmm_verify(
            _ptr(wq), _ptr(scales), _ptr(biases), N, K, bits, 64, _ptr(x), x.stride(0), M, _ptr(y), y.stride(0),
            _ptr(residual), residual.stride(0) if residual is not None else 0, _ptr(workspace),
            workspace.numel() * workspace.element_size(), _stream(stream)))
        return y

    def qmm_verify_noalloc(self, wq, scales, biases, K, bits, x, y=None, residual=None, stream=None):
        """sv_qmm_verify without a workspace (scratch in the library's own device array)."""
        import torch
        M, N = x.shape[0], wq.shape[0]
        if y is None:
            y = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
        self.check(self.lib.sv_qmm_verify_noalloc(
            _ptr(wq), _ptr(scales), _ptr(biases), N, K, bits, 64, _ptr(x), x.stride(0), M, _ptr(y), y.stride(0),
            _ptr(residual), residual.stride(0) if residual is not None else 0, _stream(stream)))
        return y

    def qmm_prepare(self, x, K, bits, mode=0, x2=None, rms_weight=None, eps=1e-6, workspace=None, stream=None):
        M = x.shape[0]
        self.check(self.lib.sv_qmm_prepare(
            _ptr(x), x.stride(0), M, K, bits, mode, _ptr(x2), x2.stride(0) if x2 is not None else 0,
            _ptr(rms_weight), eps, _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream)))

    def qmm_run(self, wq, scales, biases, K, bits, M, y=None, residual=None, workspace=None, stream=None):
        import torch
        N = wq.shape[0]
        if y is None:
            y = torch.empty((M, N), dtype=torch.bfloat16, device=wq.device)
        self.check(self.lib.sv_qmm_run(
            _ptr(wq), _ptr(scales), _ptr(biases), N, K, bits, 64, M, _ptr(y), y.stride(0), _ptr(residual),
            residual.stride(0) if residual is not None else 0, _ptr(workspace),
            workspace.numel() * workspace.element_size(), _stream(stream)))
        return y

    # -------------------------------------------------------------- lm_head
    def lm_head_workspace_bytes(self, M, V, K, bits):
        return self.lib.sv_lm_head_workspace_bytes(M, V, K, bits)

    def lm_head_verify(self, wq, scales, biases, K, bits, x, temperature, logits=None, stats=True, workspace=None,
                       stream=None):
        import torch
        M, V = x.shape[0], wq.shape[0]
        dev = x.device
        if logits is None:
            logits = torch.empty((M, V), dtype=torch.float32, device=dev)
        row_max = row_sumexp = row_argmax = None
        if stats:
            row_max = torch.empty(M, dtype=torch.float32, device=dev)
            row_sumexp = torch.zeros(M, dtype=torch.float32, device=dev)
            row_argmax = torch.empty(M, dtype=torch.int32, device=dev)
        if workspace is None:
            workspace = self.workspace(self.lm_head_workspace_bytes(M, V, K, bits), dev)
        self.check(self.lib.sv_lm_head_verify(
            _ptr(wq), _ptr(scales), _ptr(biases), V, K, bits, 64, _ptr(x), x.stride(0), M, float(temperature),
            _ptr(logits), logits.stride(0), _ptr(row_max), _ptr(row_sumexp), _ptr(row_argmax), _ptr(workspace),
            workspace.numel() * workspace.element_size(), _stream(stream)))
        return logits, row_max, row_sumexp, row_argmax

    def lm_head_run(self, wq, scales, biases, K, bits, M, temperature, logits=None, stats=None, workspace=None,
                    stream=None):
        import torch
        V = wq.shape[0]
        if logits is None:
            logits = torch.empty((M, V), dtype=torch.float32, device=wq.device)
        rmax, rsum, rarg = stats if stats is not None else (None, None, None)
        self.check(self.lib.sv_lm_head_run(
            _ptr(wq), _ptr(scales), _ptr(biases), V, K, bits, 64, M, float(temperature), _ptr(logits),
            logits.stride(0), _ptr(rmax), _ptr(rsum), _ptr(rarg), _ptr(workspace),
            workspace.numel() * workspace.element_size(), _stream(stream)))
        return logits

    # ---------------------------------------------------------------- round
    def make_model(self, layers, lm_head, hidden, q_dim, inter, vocab, bits, rms_eps=1e-6):
        """A ctypes sv_model over device weight dicts {'wq','scales','biases'}, with its round plan
        (``model.plan``, a device tensor built by sv_round_plan_init).

        ``layers``: list of dicts with keys qkv, o, gate_up, down."""
        def qw(w):
            packed = w.get("packed")
            return QWeight(w["wq"].data_ptr(), w["scales"].data_ptr(), w["biases"].data_ptr(), w["wq"].shape[0],
                           w["K"], packed.data_ptr() if packed is not None else None)
        arr = (Layer * len(layers))(*[Layer(qw(l["qkv"]), qw(l["o"]), qw(l["gate_up"]), qw(l["down"]))
                                      for l in layers])
        m = Model(len(layers), hidden, q_dim, inter, vocab, bits, rms_eps, arr, qw(lm_head))
        # the struct holds raw device pointers: keep the tensors (and the array) alive with it
        m._keep = (arr, layers, lm_head)
        nbytes = self.lib.sv_round_plan_bytes(ctypes.byref(m))
        if nbytes == 0:
            raise SVError(SV_EINVAL, "sv_round_plan_bytes: model rejected")
        m.plan = self.workspace(nbytes, device=lm_head["wq"].device)
        self.check(self.lib.sv_round_plan_init(ctypes.byref(m), _ptr(m.plan), nbytes))
        return m

    def pack(self, w, stream=None):
        """Unit-packed copy of a device weight dict (sv_qmm_pack); returns a uint8 device tensor."""
        import torch
        N, K, bits = w["wq"].shape[0], w["K"], w["bits"]
        nbytes = self.lib.sv_qmm_pack_bytes(N, K, bits)
        if nbytes == 0:
            raise SVError(SV_EUNSUPPORTED, "sv_qmm_pack_bytes: unsupported shape")
        out = torch.empty(nbytes, dtype=torch.uint8, device=w["wq"].device)
        self.check(self.lib.sv_qmm_pack(_ptr(w["wq"]), _ptr(w["scales"]), _ptr(w["biases"]), N, K, bits, 64, _ptr(out),
                                        nbytes, _stream(stream)))
        return out

    def round_workspace_bytes(self, model, rows):
        return self.lib.sv_round_workspace_bytes(ctypes.byref(model), rows)

    def verify_round(self, model, row_offsets, hidden, temperature, logits, out_len, out_tokens, workspace,
                     q=None, draft=None, u=None, stream=None, events=None, accept_wait=None):
        """events: optional (start, stop) torch.cuda.Event pair recorded around the matmul launch;
        accept_wait: optional torch.cuda.Event the accept step waits for (q, draft and u copied in
        on another stream while the projections run)."""
        B = len(row_offsets) - 1
        offs = (ctypes.c_int32 * (B + 1))(*[int(v) for v in row_offsets])
        ev0 = ev1 = None
        if events is not None:
            ev0, ev1 = (ctypes.c_void_p(e.cuda_event) for e in events)
        self.check(self.lib.sv_verify_round(
            ctypes.byref(model), _ptr(model.plan), B, offs, _ptr(hidden), hidden.stride(0), float(temperature), _ptr(q),
            q.stride(0) if q is not None else 0, _ptr(draft), _ptr(u), _ptr(logits), logits.stride(0),
            _ptr(out_len), _ptr(out_tokens), _ptr(workspace), workspace.numel() * workspace.element_size(),
            _stream(stream), ev0, ev1, ctypes.c_void_p(accept_wait.cuda_event) if accept_wait is not None else None))

    # --------------------------------------------------------------- accept
    def accept_workspace_bytes(self, B, rows):
        return self.lib.sv_accept_workspace_bytes(B, rows)

    def spec_accept(self, logits, draft, temperature, q=None, u=None, stats=None, workspace=None, stream=None):
        """stats: (row_max, row_sumexp, row_argmax) from lm_head_verify, or None."""
        import torch
        m = logits.shape[0] - 1
        V = logits.shape[1]
        dev = logits.device
        out_len = torch.zeros(1, dtype=torch.int32, device=dev)
        out_tokens = torch.full((m + 1,), -1, dtype=torch.int32, device=dev)
        if workspace is None:
            workspace = self.workspace(self.accept_workspace_bytes(1, m + 1), dev)
        rmax, rsum, rarg = stats if stats is not None else (None, None, None)
        self.check(self.lib.sv_spec_accept(
            _ptr(logits), logits.stride(0), _ptr(rmax), _ptr(rsum), _ptr(rarg), _ptr(q),
            q.stride(0) if q is not None else 0, _ptr(draft), m, V, float(temperature), _ptr(u), _ptr(out_len),
            _ptr(out_tokens), _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream)))
        return out_len, out_tokens

    def spec_accept_batched(self, row_offsets, logits, drafts, temperature, q=None, u=None, stats=None,
                            workspace=None, stream=None):
        import torch
        B = len(row_offsets) - 1
        rows = int(row_offsets[-1])
        V = logits.shape[1]
        dev = logits.device
        offs = (ctypes.c_int32 * (B + 1))(*[int(v) for v in row_offsets])
        out_len = torch.zeros(B, dtype=torch.int32, device=dev)
        out_tokens = torch.full((rows,), -1, dtype=torch.int32, device=dev)
        if workspace is None:
            workspace = self.workspace(self.accept_workspace_bytes(B, rows), dev)
        rmax, rsum, rarg = stats if stats is not None else (None, None, None)
        self.check(self.lib.sv_spec_accept_batched(
            B, offs, _ptr(logits), logits.stride(0), _ptr(rmax), _ptr(rsum), _ptr(rarg), _ptr(q),
            q.stride(0) if q is not None else 0, _ptr(drafts), V, float(temperature), _ptr(u), _ptr(out_len),
            _ptr(out_tokens), _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream)))
        return out_len, out_tokens

    def spec_accept_truncated(self, row_offsets, logits, drafts, temperature, top_k, top_p, q=None, u=None,
                              stats=None, workspace=None, stream=None):
        import torch
        B = len(row_offsets) - 1
        rows = int(row_offsets[-1])
        V = logits.shape[1]
        dev = logits.device
        offs = (ctypes.c_int32 * (B + 1))(*[int(v) for v in row_offsets])
        out_len = torch.zeros(B, dtype=torch.int32, device=dev)
        out_tokens = torch.full((rows,), -1, dtype=torch.int32, device=dev)
        if workspace is None:
            workspace = self.workspace(self.accept_workspace_bytes(B, rows), dev)
        rmax, rsum, rarg = stats if stats is not None else (None, None, None)
        self.check(self.lib.sv_spec_accept_truncated(
            B, offs, _ptr(logits), logits.stride(0), _ptr(rmax), _ptr(rsum), _ptr(rarg), _ptr(q),
            q.stride(0) if q is not None else 0, _ptr(drafts), V, float(temperature), _ptr(u), int(top_k),
            float(top_p), _ptr(out_len), _ptr(out_tokens), _ptr(workspace),
            workspace.numel() * workspace.element_size(), _stream(stream)))
        return out_len, out_tokens

    def tree_accept_workspace_bytes(self, rows):
        return self.lib.sv_tree_accept_workspace_bytes(rows)

    def tree_accept(self, row_offsets, logits, parent, tokens, temperature, q=None, u=None, distinct=False, top_k=0, top_p=1.0,
                    stats=None, out=None, max_path=None, workspace=None, stream=None):
        """(out_len [B], out_tokens [rows], path [B, max_path]).  Row i > 0 of a request drafts tokens[i] below its row parent[i];
        q [rows, V]: the distributions that each node's children were drawn from (None: drafts without one), distinct: without
        replacement; stats: (row_max, row_sumexp, row_argmax) of the head, or None; out: the three outputs to write to
        (entries behind a request's results are left as they are; fresh outputs hold -1 there)."""
        import torch
        f32, i32 = torch.float32, torch.int32
        offs, B, rows = self._rows_of(row_offsets)
        dev, V = logits.get_device(), logits.shape[-1]
        handle = self._launch_stream(stream, dev)
        ldl, ldq = _matrix("logits", logits, f32, dev, rows, V), 0
        if q is not None:
            ldq = _matrix("q", q, f32, dev, rows, V)
        if out is None:
            max_path = max([1] + [offs[b + 1] - offs[b] for b in range(B)]) if max_path is None else max_path
            out = [_empty(shape, i32, logits.device, stream) for shape in ((B,), (rows,), (B, max_path))]
            for t in out:
                if stream is None:
                    t.fill_(-1)
                else:
                    with torch.cuda.stream(stream):
                        t.fill_(-1)
        out_len, out_tokens, path = out
        if path.dim() != 2 or path.shape[0] < B or (max_path is not None and path.shape[1] != max_path):
            _refuse("path must be an int32 [%d, max_path] tensor" % B, path)
        ptrs = [None if t is None else _vector(name, t, dtype, dev, rows) for name, t, dtype in (
            ("row_max", None if stats is None else stats[0], f32), ("row_sumexp", None if stats is None else stats[1], f32),
            ("row_argmax", None if stats is None else stats[2], i32), ("parent", parent, i32), ("tokens", tokens, i32))]
        up = None if u is None else _vector("u", u, f32, dev, rows)
        outs = [_vector("out_len", out_len, i32, dev, B), _vector("out_tokens", out_tokens, i32, dev, rows),
                _vector("path", path, i32, dev, 0)]
        ws, size = (None, 0) if workspace is None else self._workspace(workspace, None, logits.device, dev, stream)
        status = self.lib.sv_tree_accept(B, offs, logits.data_ptr(), ldl, *ptrs, None if q is None else q.data_ptr(), ldq,
                                         bool(distinct), V, float(temperature), up, max(-1, min(int(top_k), _INT_MAX)), float(top_p), *outs,
                                         path.shape[1], None if ws is None else ws.data_ptr(), size, handle)
        if status:
            self.check(status)
        return out_len, out_tokens, path

    def truncate_probs(self, probs, top_k, top_p, out=None, stream=None):
        import torch
        if out is None:
            out = torch.empty_like(probs)
        self.check(self.lib.sv_truncate_probs(_ptr(probs), probs.stride(0), _ptr(out), out.stride(0), probs.shape[0],
                                              probs.shape[1], int(top_k), float(top_p), _stream(stream)))
        return out

    def logprobs(self, logits, temperature, chosen=None, top_n=0, stream=None):
        """(chosen_logprob [rows] or None, top_ids [rows, top_n], top_logprobs [rows, top_n])."""
        import torch
        rows, V = logits.shape
        dev = logits.device
        clp = torch.empty(rows, dtype=torch.float32, device=dev) if chosen is not None else None
        ids = torch.empty((rows, top_n), dtype=torch.int32, device=dev)
        tlp = torch.empty((rows, top_n), dtype=torch.float32, device=dev)
        self.check(self.lib.sv_logprobs(_ptr(logits), logits.stride(0), rows, V, float(temperature), _ptr(chosen),
                                        int(top_n), _ptr(clp), _ptr(ids) if top_n else None,
                                        _ptr(tlp) if top_n else None, _stream(stream)))
        return clp, ids, tlp

    # --------------------------------------------------------------- gather
    def gather_qmm(self, wq, scales, biases, E, K, bits, x, pair_rows, pair_experts, y=None, workspace=None,
                   stream=None):
        """Stacked expert weights [E*N, ...]; pair_rows / pair_experts int32 device tensors [P]."""
        import torch
        N = wq.shape[0] // E
        M, P = x.shape[0], pair_rows.shape[0]
        if y is None:
            y = torch.empty((P, N), dtype=torch.bfloat16, device=x.device)
        if workspace is None:
            nbytes = self.lib.sv_gather_qmm_workspace_bytes(P, M, N, K, E, bits)
            if nbytes == 0:
                raise SVError(SV_EINVAL, "sv_gather_qmm_workspace_bytes: unsupported sizes")
            workspace = self.workspace(nbytes, x.device)
        self.check(self.lib.sv_gather_qmm(_ptr(wq), _ptr(scales), _ptr(biases), E, N, K, bits, 64, _ptr(x),
                                          x.stride(0), M, _ptr(pair_rows), _ptr(pair_experts), P, _ptr(y), y.stride(0),
                                          _ptr(workspace), workspace.numel() * workspace.element_size(),
                                          _stream(stream)))
        return y

    # --------------------------------------------------------------- philox
    def philox_uniforms(self, seed, subsequence, offset, n, out=None, stream=None):
        import torch
        if out is None:
            out = torch.empty(n, dtype=torch.float32, device="cuda")
        self.check(self.lib.sv_philox_uniforms(seed, subsequence, offset, n, _ptr(out), _stream(stream)))
        return out

    # ----------------------------------------------------------------- glue
    def rmsnorm(self, x, weight=None, eps=1e-6, y=None, stream=None):
        import torch
        if y is None:
            y = torch.empty_like(x)
        self.check(self.lib.sv_rmsnorm(_ptr(x), x.stride(0), x.shape[0], x.shape[1], _ptr(weight), eps, _ptr(y),
                                       y.stride(0), _stream(stream)))
        return y

    # ------------------------------------------------------------ attention
    @staticmethod
    def row_offsets(offsets):
        """Host row offsets [B + 1] as the C calls take them (lists are accepted too, at some cost a call)."""
        if isinstance(offsets, ctypes.Array) and offsets._type_ is ctypes.c_int32:
            return offsets
        values = [int(v) for v in offsets]
        if any(abs(v) > _INT_MAX for v in values):                      # ctypes would take them modulo 2^32
            raise SVError(SV_EINVAL, "row_offsets must be below 2^31")
        return (ctypes.c_int32 * len(values))(*values)

    def _rows_of(self, row_offsets):
        """(row_offsets as the C calls take them, B, rows).  A call without rows ends in the binding, so its offsets are checked here."""
        offs = self.row_offsets(row_offsets)
        B = len(offs) - 1
        rows = offs[B] if B >= 0 else -1
        if rows < 0 or (rows == 0 and any(offs)):
            raise SVError(SV_EINVAL, "row_offsets must be [B + 1] numbers that start at 0 and do not decrease")
        return offs, B, rows

    @staticmethod
    def kv_cache(k, v, k_scales=None, k_biases=None, v_scales=None, v_biases=None):
        """A KVCache over device tensors: k, v bf16 [pages, heads, page, dim], or int32 words
        [pages, heads, page, dim * bits / 32] with fp16 scales and biases [pages, heads, page, dim / 64]."""
        import torch
        side = [t for t in (k_scales, k_biases, v_scales, v_biases) if t is not None]
        if k.dim() != 4 or k.shape != v.shape or k.device.type != "cuda" or len(side) not in (0, 4):
            raise SVError(SV_EINVAL, "k and v must be equal 4-d CUDA tensors, scales and biases all given or none")
        pages, heads, page, last = k.shape
        dim, bits = (side[0].shape[-1] * 64, 0) if side else (last, 16)
        if side:
            bits = last * 32 // dim if dim else 0
            if any(tuple(t.shape) != (pages, heads, page, dim // 64) for t in side) or last * 32 != dim * bits:
                raise SVError(SV_EINVAL, "scales and biases must be [pages, heads, page, dim / 64]")
        for t, want in [(t, torch.int32 if side else torch.bfloat16) for t in (k, v)] + [(t, torch.float16) for t in side]:
            if t.dtype is not want or t.device != k.device or not t.is_contiguous():
                _refuse("cache tensors must be contiguous, on one device, and %s" % want, t)
        ptrs = [t.data_ptr() for t in side] or [None] * 4
        return KVCache(KVCacheView(k.data_ptr(), v.data_ptr(), *ptrs, pages, page, heads, dim, bits), [k, v] + side)

    def kv_cache_alloc(self, n_pages, page_size, n_kv_heads, head_dim, bits, device="cuda"):
        """A zero-filled cache (torch allocates it)."""
        import torch
        shape = (n_pages, n_kv_heads, page_size)
        zeros = lambda last, dtype: torch.zeros(shape + (last,), dtype=dtype, device=device)  # noqa: E731
        if bits == 16:
            return self.kv_cache(zeros(head_dim, torch.bfloat16), zeros(head_dim, torch.bfloat16))
        return self.kv_cache(zeros(head_dim * bits // 32, torch.int32), zeros(head_dim * bits // 32, torch.int32),
                             *[zeros(head_dim // 64, torch.float16) for _ in range(4)])

    @staticmethod
    def kv_layers(caches):
        return KVLayers(caches)

    def _launch_stream(self, stream, dev):
        """Raw handle of the stream to launch on; the tensors' device must be the current one."""
        if self._torch is None:
            import torch
            self._torch = torch
        if dev < 0 or self._torch._C._cuda_getDevice() != dev:
            raise SVError(SV_EINVAL, "tensors on cuda:%d (-1: the host), which is not the current device" % dev)
        return self._torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream

    def qk_norm_rope(self, q, k, head_dim, positions=None, inv_freq=None, q_weight=None, k_weight=None, eps=1e-6,
                     norm=True, interleaved=False, q_out=None, k_out=None, stream=None):
        """(q_out, k_out).  q [rows, q_heads * head_dim], k [rows, kv_heads * head_dim] or None; the
        rotary width is 2 * len(inv_freq) (no rotation without it); q_out = q works in place."""
        import torch
        bf16, dev = torch.bfloat16, q.get_device()
        handle = self._launch_stream(stream, dev)
        (rows, qw), kw = q.shape, 0
        if q_out is None:
            q_out = _empty((rows, qw), bf16, q.device, stream)
        ldq, ldqo, ldk, ldko = _matrix("q", q, bf16, dev, rows, qw), _matrix("q_out", q_out, bf16, dev, rows, qw), 0, 0
        kp = kop = qwp = kwp = pos = inv = None
        if k is not None:
            kw = k.shape[-1]
            if k_out is None:
                k_out = _empty((rows, kw), bf16, q.device, stream)
            ldk, ldko = _matrix("k", k, bf16, dev, rows, kw), _matrix("k_out", k_out, bf16, dev, rows, kw)
            kp, kop = k.data_ptr(), k_out.data_ptr()
        if head_dim < 1 or qw % head_dim or kw % head_dim:
            raise SVError(SV_EINVAL, "q and k widths must be multiples of head_dim")
        if q_weight is not None:
            qwp = _vector("q_weight", q_weight, bf16, dev, head_dim)
        if k_weight is not None:
            kwp = _vector("k_weight", k_weight, bf16, dev, head_dim)
        rot = 0
        if inv_freq is not None:
            rot = 2 * inv_freq.numel()
            inv = _vector("inv_freq", inv_freq, torch.float32, dev, rot // 2)
            if rot and positions is None:
                raise SVError(SV_EINVAL, "a rotation needs positions")
            if rot:
                pos = _vector("positions", positions, torch.int32, dev, rows)
        if rows:
            status = self.lib.sv_qk_norm_rope(q.data_ptr(), ldq, kp, ldk, rows, qw // head_dim, kw // head_dim, head_dim, norm,
                                              qwp, kwp, eps, pos, inv if rot else None, rot, interleaved, q_out.data_ptr(), ldqo,
                                              kop, ldko, handle)
            if status:
                self.check(status)
        return q_out, k_out

    def _kv_rows(self, call, cache, row_offsets, first, block_table, k, v, stream):
        import torch
        i32, bf16, dev, width = torch.int32, torch.bfloat16, cache.index, cache.width
        offs, B, rows = self._rows_of(row_offsets)
        lens, (table, pages) = _vector("the lengths", first, i32, dev, B), _table(block_table, i32, dev, B)
        ldk, ldv = _matrix("k", k, bf16, dev, rows, width), _matrix("v", v, bf16, dev, rows, width)
        handle = self._launch_stream(stream, dev)
        if rows or B < 1:
            status = call(cache.ref, B, offs, lens, table, pages, k.data_ptr(), ldk, v.data_ptr(), ldv, handle)
            if status:
                self.check(status)

    def kv_append(self, cache, row_offsets, kv_len, block_table, k, v, stream=None):
        """Rows of k and v [rows, kv_heads * head_dim] into the cache at kv_len[b], kv_len[b] + 1, ..."""
        self._kv_rows(self.lib.sv_kv_append, cache, row_offsets, kv_len, block_table, k, v, stream)

    def kv_read(self, cache, row_offsets, first, block_table, k=None, v=None, stream=None):
        """(k, v) bf16 [rows, kv_heads * head_dim]: row i of request b from position first[b] + i."""
        if k is None or v is None:
            import torch
            row_offsets, _, rows = self._rows_of(row_offsets)
            shape = (rows, cache.width)
            k = _empty(shape, torch.bfloat16, cache.device, stream) if k is None else k
            v = _empty(shape, torch.bfloat16, cache.device, stream) if v is None else v
        self._kv_rows(self.lib.sv_kv_read, cache, row_offsets, first, block_table, k, v, stream)
        return k, v

    def tree_attention_workspace_bytes(self, cache, row_offsets, n_q_heads):
        offs = self.row_offsets(row_offsets)
        return self.lib.sv_tree_attention_workspace_bytes(cache.ref, len(offs) - 1, offs, n_q_heads)

    def tree_attention(self, cache, row_offsets, kv_len, block_table, q, n_q_heads, scale=None, tree_mask=None, out=None,
                       workspace=None, stream=None):
        """out bf16 [rows, q_heads * head_dim]; tree_mask int64 [rows] (bit j: the row sees the request's
        drafted row j), None for a chain; scale defaults to head_dim ** -0.5."""
        import torch
        i32, bf16, dev, dim = torch.int32, torch.bfloat16, cache.index, cache.head_dim
        (offs, B, rows), width = self._rows_of(row_offsets), n_q_heads * dim
        lens, (table, pages) = _vector("kv_len", kv_len, i32, dev, B), _table(block_table, i32, dev, B)
        mask = None if tree_mask is None else _vector("tree_mask", tree_mask, torch.int64, dev, rows)
        if out is None:
            out = _empty((q.shape[0], width), bf16, cache.device, stream)
        ldq, ldo = _matrix("q", q, bf16, dev, rows, width), _matrix("out", out, bf16, dev, rows, width)
        handle = self._launch_stream(stream, dev)
        if workspace is None:
            workspace = _empty(max(256, self.tree_attention_workspace_bytes(cache, offs, n_q_heads)), torch.uint8, cache.device,
                               stream)           # freed into the same pool: the call may outlive the tensor
        elif workspace.get_device() != dev or not workspace.is_contiguous():
            _refuse("the workspace must be contiguous and on cuda:%d" % dev, workspace)
        if rows or B < 1:
            status = self.lib.sv_tree_attention(cache.ref, B, offs, lens, table, pages, q.data_ptr(), ldq, n_q_heads,
                                                dim ** -0.5 if scale is None else scale, mask, out.data_ptr(), ldo,
                                                workspace.data_ptr(), workspace.numel() * workspace.element_size(), handle)
            if status:
                self.check(status)
        return out

    @staticmethod
    def prefix_groups(offsets, pages):
        """Group g is requests offsets[g] .. offsets[g + 1] - 1, whose first pages[g] table entries name the same pages."""
        ints = [int(v) for v in offsets], [int(v) for v in pages]
        if len(ints[0]) != len(ints[1]) + 1 or any(abs(v) > _INT_MAX for v in ints[0] + ints[1]):
            raise SVError(SV_EINVAL, "groups need [G + 1] offsets and [G] page counts below 2^31")
        return PrefixGroups(*[(ctypes.c_int32 * len(v))(*v) for v in ints])

    def tree_attention_shared_workspace_bytes(self, cache, groups, row_offsets, n_q_heads):
        offs = self.row_offsets(row_offsets)
        return self.lib.sv_tree_attention_shared_workspace_bytes(cache.ref, groups.n, groups.offsets, groups.pages, len(offs) - 1, offs,
                                                                 n_q_heads)

    def tree_attention_shared(self, cache, groups, row_offsets, kv_len, block_table, q, n_q_heads, scale=None, tree_mask=None, out=None,
                              workspace=None, stream=None):
        """tree_attention of a batch whose requests share prefixes; groups: prefix_groups()."""
        import torch
        i32, bf16, dev, dim = torch.int32, torch.bfloat16, cache.index, cache.head_dim
        (offs, B, rows), width = self._rows_of(row_offsets), n_q_heads * dim
        lens, (table, pages) = _vector("kv_len", kv_len, i32, dev, B), _table(block_table, i32, dev, B)
        mask = None if tree_mask is None else _vector("tree_mask", tree_mask, torch.int64, dev, rows)
        if out is None:
            out = _empty((q.shape[0], width), bf16, cache.device, stream)
        ldq, ldo = _matrix("q", q, bf16, dev, rows, width), _matrix("out", out, bf16, dev, rows, width)
        handle = self._launch_stream(stream, dev)
        workspace, size = self._workspace(workspace, lambda: self.tree_attention_shared_workspace_bytes(cache, groups, offs, n_q_heads),
                                          cache.device, dev, stream)
        if rows or B < 1:
            status = self.lib.sv_tree_attention_shared(cache.ref, groups.n, groups.offsets, groups.pages, B, offs, lens, table, pages,
                                                       q.data_ptr(), ldq, n_q_heads, dim ** -0.5 if scale is None else scale, mask,
                                                       out.data_ptr(), ldo, workspace.data_ptr(), size, handle)
            if status:
                self.check(status)
        return out

    def kv_commit(self, caches, kv_len, block_table, path, path_len, stream=None):
        """Move the drafted rows path[b, :path_len[b]] (int32) to the front of request b's drafted region, in
        every cache of `caches` (a list of KVCache, or kv_layers() of one)."""
        import torch
        layers = caches if isinstance(caches, KVLayers) else KVLayers(caches)
        i32, dev, B = torch.int32, layers.index, kv_len.numel()
        lens, (table, pages) = _vector("kv_len", kv_len, i32, dev, B), _table(block_table, i32, dev, B)
        if path.dim() != 2 or path.shape[0] < B:
            _refuse("path must be an int32 [%d, n] tensor" % B, path)
        status = self.lib.sv_kv_commit(layers.array, len(layers.array), B, lens, table, pages,
                                       _vector("path", path, i32, dev, 0), path.shape[1],
                                       _vector("path_len", path_len, i32, dev, B), self._launch_stream(stream, dev))
        if status:
            self.check(status)

    # ------------------------------------------------------------ cache pages
    @staticmethod
    def kv_pages(refs, block_table, held, page_size):
        """A KVPages over int32 device tensors: refs [pages], block_table [slots, n], held [slots]."""
        import torch
        if refs.device.type != "cuda" or block_table.dim() != 2 or refs.dim() != 1 or held.dim() != 1 or held.numel() != block_table.shape[0]:
            raise SVError(SV_EINVAL, "refs must be a CUDA vector, block_table [slots, n] and held [slots]")
        for t in (refs, block_table, held):
            if t.dtype is not torch.int32 or t.device != refs.device or not t.is_contiguous():
                _refuse("refs, block_table and held must be contiguous int32 tensors on one device", t)
        sizes = (refs.numel(), int(page_size), *block_table.shape)
        if any(abs(n) > _INT_MAX for n in sizes):
            raise SVError(SV_EINVAL, "sizes must be below 2^31")
        view = KVPagesView(refs.data_ptr(), block_table.data_ptr(), held.data_ptr(), *sizes)
        return KVPages(view, refs, block_table, held)

    def kv_pages_alloc(self, n_pages, page_size, slots, table_pages, device="cuda"):
        """A fresh state: every page free, every slot empty."""
        import torch
        zeros = lambda *shape: torch.zeros(shape, dtype=torch.int32, device=device)  # noqa: E731
        return self.kv_pages(zeros(n_pages), zeros(slots, table_pages), zeros(slots), page_size)

    def kv_fork(self, pages, parent, child, tokens, stream=None):
        """Slot child[f] gets the pages of slot parent[f]'s first tokens[f] tokens, shared (int32 device tensors)."""
        import torch
        i32, dev, n = torch.int32, pages.index, parent.numel()
        if child.numel() != n or tokens.numel() != n:
            raise SVError(SV_EINVAL, "parent, child and tokens must have one length")
        ptrs = [_vector(name, t, i32, dev, n) for name, t in (("parent", parent), ("child", child), ("tokens", tokens))]
        self.check(self.lib.sv_kv_fork(pages.ref, n, *ptrs, self._launch_stream(stream, dev)))

    def kv_reserve_workspace_bytes(self, pages):
        return self.lib.sv_kv_reserve_workspace_bytes(pages.ref)

    def _page_layers(self, caches, dev):
        """(array, number) of the layers' caches; none for bookkeeping alone."""
        if caches is None:
            return None, 0, None
        layers = caches if isinstance(caches, KVLayers) else KVLayers(caches)
        if layers.index != dev:
            raise SVError(SV_EINVAL, "the caches must be on cuda:%d" % dev)
        return layers.array, len(layers.array), layers

    def kv_reserve(self, pages, caches, keep, need, counts=None, copies=None, workspace=None, stream=None):
        """(counts, copies).  Slot s keeps keep[s] tokens and gets room for need[s] (need < 0: left alone), what it will
        write being its alone; caches: every layer's (a list of KVCache, kv_layers() of one, or None).  counts [3]: pages
        missing (0: done), copies, fresh pages; copies [slots, 3]: (from, to, places)."""
        import torch
        i32, dev, slots = torch.int32, pages.index, pages.slots
        array, n, _layers = self._page_layers(caches, dev)
        handle = self._launch_stream(stream, dev)
        counts = _empty((3,), i32, pages.device, stream) if counts is None else counts
        copies = _empty((slots, 3), i32, pages.device, stream) if copies is None else copies
        ptrs = [_vector(name, t, i32, dev, size) for name, t, size in (("keep", keep, slots), ("need", need, slots),
                                                                       ("counts", counts, 3), ("copies", copies, 3 * slots))]
        workspace, size = self._workspace(workspace, lambda: self.kv_reserve_workspace_bytes(pages), pages.device, dev, stream)
        self.check(self.lib.sv_kv_reserve(pages.ref, array, n, *ptrs, workspace.data_ptr(), size, handle))
        return counts, copies

    def kv_compact(self, pages, caches, counts=None, moves=None, stream=None):
        """(counts, moves).  The pages in use move to the front; counts [2]: pages in use, pages moved; moves [n_pages, 2]."""
        import torch
        i32, dev, n_pages = torch.int32, pages.index, pages.view.n_pages
        array, n, _layers = self._page_layers(caches, dev)
        handle = self._launch_stream(stream, dev)
        counts = _empty((2,), i32, pages.device, stream) if counts is None else counts
        moves = _empty((n_pages, 2), i32, pages.device, stream) if moves is None else moves
        self.check(self.lib.sv_kv_compact(pages.ref, array, n, _vector("counts", counts, i32, dev, 2),
                                          _vector("moves", moves, i32, dev, 2 * n_pages), handle))
        return counts, moves

    def kv_copy_pages(self, caches, src, dst, to=None, stream=None):
        """Page src[i] of each cache to page dst[i] of the same layer's cache in `to` (the same caches by default)."""
        import torch
        array, n, layers = self._page_layers(caches, src.get_device())
        array_to, n_to, _to = (array, n, layers) if to is None else self._page_layers(to, src.get_device())
        if n_to != n or dst.numel() != src.numel():
            raise SVError(SV_EINVAL, "as many caches to copy to as from, and as many destinations as sources")
        dev = layers.index if layers is not None else src.get_device()
        ptrs = [_vector(name, t, torch.int32, dev, t.numel()) for name, t in (("src", src), ("dst", dst))]
        self.check(self.lib.sv_kv_copy_pages(array, array_to, n, src.numel(), *ptrs, self._launch_stream(stream, dev)))

    def _workspace(self, workspace, nbytes, device, dev, stream):
        """(the caller's workspace, checked, or a fresh one; its bytes)."""
        import torch
        if workspace is None:                     # freed into the pool of the stream that uses it: the call may outlive the tensor
            workspace = _empty(max(256, nbytes()), torch.uint8, device, stream)
        elif workspace.get_device() != dev or not workspace.is_contiguous():
            _refuse("the workspace must be contiguous and on cuda:%d" % dev, workspace)
        return workspace, workspace.numel() * workspace.element_size()

    def residual_add(self, h, t, stream=None):
        self.check(self.lib.sv_residual_add(_ptr(h), h.stride(0), _ptr(t), t.stride(0), h.shape[0], h.shape[1],
                                            _stream(stream)))
        return h

    def swiglu(self, g, u, s=None, stream=None):
        import torch
        if s is None:
            s = torch.empty_like(g)
        self.check(self.lib.sv_swiglu(_ptr(g), g.stride(0), _ptr(u), u.stride(0), g.shape[0], g.shape[1], _ptr(s),
                                      s.stride(0), _stream(stream)))
        return s


_LIB = None


def load():
    """The process-wide Library; builds nothing and falls back to nothing."""
    global _LIB
    if _LIB is None:
        _LIB = Library()
    return _LIB
