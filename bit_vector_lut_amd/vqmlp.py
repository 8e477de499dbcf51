"""ctypes binding of libvqmlp.so (include/vqmlp.h).

Argument marshalling only: every step of the forward runs in the HIP kernels of the library.
PyTorch supplies device memory and the current HIP stream.  A missing library raises at import
of the first call; there is no CPU fallback.
"""
from __future__ import annotations

import ctypes as C
import os

import numpy as np

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libvqmlp.so")

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_WORKSPACE, ERR_HIP = 0, 1, 2, 3, 4
PATH_AUTO, PATH_FUSED, PATH_TILED = 0, 1, 2


class VqmlpError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__("vqmlp status %d: %s" % (status, msg))
        self.status = status


class _Desc(C.Structure):
    _fields_ = [("H", C.c_int), ("I", C.c_int), ("had_block_h", C.c_int),
                ("had_block_i", C.c_int), ("t_max", C.c_int),
                ("gate", C.c_void_p), ("up", C.c_void_p), ("down", C.c_void_p),
                ("s_in", C.c_void_p), ("sign_h", C.c_void_p), ("sign_i", C.c_void_p)]


class _NormDesc(C.Structure):
    _fields_ = [("dtype", C.c_int), ("res_dtype", C.c_int), ("kind", C.c_int), ("T", C.c_int),
                ("H", C.c_int), ("eps", C.c_float), ("res_scale", C.c_float),
                ("w_offset", C.c_float),
                ("y", C.c_void_p), ("ld_y", C.c_int64), ("res", C.c_void_p), ("ld_res", C.c_int64),
                ("gate", C.c_void_p), ("ld_gate", C.c_int64),
                ("post_w", C.c_void_p), ("post_b", C.c_void_p), ("pre_w", C.c_void_p),
                ("pre_b", C.c_void_p), ("res_out", C.c_void_p), ("ld_res_out", C.c_int64),
                ("x", C.c_void_p), ("ld_x", C.c_int64)]


class _PagesDesc(C.Structure):
    _fields_ = [("R", C.c_int), ("max_tokens", C.c_int), ("page_size", C.c_int),
                ("n_pages", C.c_int), ("n_free", C.c_int), ("table_width", C.c_int),
                ("ld_table", C.c_int64), ("ctx_len", C.c_void_p), ("q_len", C.c_void_p),
                ("free_pages", C.c_void_p), ("free_head", C.c_void_p), ("table", C.c_void_p),
                ("seq_len", C.c_void_p), ("cu_q", C.c_void_p), ("slot", C.c_void_p),
                ("position", C.c_void_p), ("status", C.c_void_p), ("free_head_out", C.c_void_p)]


class _AttnDesc(C.Structure):
    _fields_ = [("dtype", C.c_int), ("T", C.c_int), ("R", C.c_int), ("heads", C.c_int),
                ("kv_heads", C.c_int), ("D", C.c_int), ("page_size", C.c_int),
                ("n_pages", C.c_int), ("window", C.c_int), ("max_kv", C.c_int),
                ("scale", C.c_float), ("table_width", C.c_int), ("ld_table", C.c_int64),
                ("ld_q", C.c_int64), ("ld_y", C.c_int64), ("q", C.c_void_p), ("y", C.c_void_p),
                ("lse", C.c_void_p), ("k_cache", C.c_void_p), ("v_cache", C.c_void_p),
                ("table", C.c_void_p), ("cu_q", C.c_void_p), ("kv_len", C.c_void_p)]


class _LinearDesc(C.Structure):
    _fields_ = [("dtype", C.c_int), ("T", C.c_int), ("R", C.c_int), ("k_heads", C.c_int),
                ("v_heads", C.c_int), ("Dk", C.c_int), ("Dv", C.c_int), ("n_states", C.c_int),
                ("max_q", C.c_int), ("scale", C.c_float), ("ld_q", C.c_int64),
                ("ld_k", C.c_int64), ("ld_v", C.c_int64), ("ld_y", C.c_int64),
                ("ld_g", C.c_int64), ("q", C.c_void_p), ("k", C.c_void_p), ("v", C.c_void_p),
                ("g", C.c_void_p), ("y", C.c_void_p), ("state_in", C.c_void_p),
                ("state_out", C.c_void_p), ("cu_q", C.c_void_p), ("ctx_len", C.c_void_p),
                ("state_index", C.c_void_p)]


_lib = None


def lib():
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError("libvqmlp.so is not built (run __graft_entry__.build() or "
                              "python bit_vector_lut_amd/build.py)")
        L = C.CDLL(LIB_PATH)
        P, I, S = C.c_void_p, C.c_int, C.c_size_t
        L.vqmlp_abi_version.restype = I
        L.vqmlp_last_error.restype = C.c_char_p
        sigs = {
            "vqmlp_packed_bytes": [I, I, C.POINTER(S)],
            "vqmlp_pack": [I, I, P, P, P, P, S],
            "vqmlp_unpack": [I, I, P, S, P, P, P],
            "vqmlp_dequant": [I, I, P, P, P],
            "vqmlp_create": [C.POINTER(_Desc), C.POINTER(P)],
            "vqmlp_create_vq2": [C.POINTER(_Desc), C.POINTER(P)],
            "vqmlp_destroy": [P],
            "vqmlp_workspace_bytes": [P, I, C.POINTER(S)],
            "vqmlp_forward": [P, I, P, P, P, S, P],
            "vqmlp_forward_path": [P, I, P, P, P, S, I, P],
            "vqmlp_workspace_errors": [P, S, I, C.POINTER(C.c_uint32), P],
            "vqmlp_stream_read": [P, S, P, P],
            "vqmlp_forward_noalloc": [P, I, P, P, P],
            "vqmlp_rotate": [I, I, I, P, P, P, P, P],
            "vqmlp_lut_packed_bytes": [I, I, I, C.POINTER(S)],
            "vqmlp_lut_pack": [I, I, I, P, P, P, P, S],
            "vqmlp_lut_unpack": [I, I, I, P, S, P, P, P],
            "vqmlp_lut_workspace_bytes": [I, I, I, I, C.POINTER(S)],
            "vqmlp_lut_forward": [I, I, I, I, P, P, P, I, P, P, I, P, P, P, S, P],
            "vqmlp_lut_create": [I, I, I, P, P, P, I, P, P, I, C.POINTER(P)],
            "vqmlp_lut_destroy": [P],
            "vqmlp_lut_plan_forward": [P, I, P, P, P, S, P],
            "vqmlp_lut_plan_argmax": [P, I, P, P, P, P, S, P],
            "vqmlp_vq2_packed_bytes": [I, I, C.POINTER(S)],
            "vqmlp_vq2_pack": [I, I, P, P, P, P, S],
            "vqmlp_vq2_unpack": [I, I, P, S, P, P, P],
            "vqmlp_vq2_create": [I, I, P, C.POINTER(P)],
            "vqmlp_vq2_destroy": [P],
            "vqmlp_vq2_plan_forward": [P, I, P, P, P],
            "vqmlp_block_norm": [P, P],
            "vqmlp_page_plan": [P, P],
            "vqmlp_paged_store": [I, I, I, I, I, I, P, C.c_int64, P, C.c_int64, P, P, P, P],
            "vqmlp_paged_attn_workspace": [P, C.POINTER(S)],
            "vqmlp_paged_attn": [P, P, S, P],
            "vqmlp_linear_attn_workspace": [P, C.POINTER(S)],
            "vqmlp_linear_attn": [P, P, S, P],
        }
        for name, args in sigs.items():
            f = getattr(L, name)
            f.argtypes = args
            f.restype = I
        _lib = L
    return _lib


def _check(status: int):
    if status != OK:
        raise VqmlpError(status, lib().vqmlp_last_error().decode())


def _np_ptr(a):
    return None if a is None else a.ctypes.data_as(C.c_void_p)


def _u16(a):
    a = np.ascontiguousarray(a)
    return a.view(np.uint16) if a.dtype == np.float16 else a.astype(np.uint16, copy=False)


def _dptr(t):
    return None if t is None else C.c_void_p(t.data_ptr())


def _stream(stream=None):
    import torch

    s = stream if stream is not None else torch.cuda.current_stream()
    return C.c_void_p(s.cuda_stream)


# ------------------------------------------------------------------ host-side packing


def packed_bytes(N: int, K: int) -> int:
    n = C.c_size_t()
    _check(lib().vqmlp_packed_bytes(N, K, C.byref(n)))
    return n.value


def pack(codes, cb, sc) -> np.ndarray:
    """Pack one VQ3 matrix (codes [N/2,K] uint8, cb [N/8,64,2] f16, sc [N] f16) -> uint8."""
    codes = np.ascontiguousarray(codes, np.uint8)
    cb, sc = _u16(cb), _u16(sc)
    N, K = sc.shape[0], codes.shape[1]
    out = np.empty(packed_bytes(N, K), np.uint8)
    _check(lib().vqmlp_pack(N, K, _np_ptr(codes), _np_ptr(cb), _np_ptr(sc), _np_ptr(out),
                            out.size))
    return out


def unpack(N: int, K: int, packed):
    packed = np.ascontiguousarray(packed, np.uint8)
    codes = np.empty((N // 2, K), np.uint8)
    cb = np.empty((N // 8, 64, 2), np.uint16)
    sc = np.empty(N, np.uint16)
    _check(lib().vqmlp_unpack(N, K, _np_ptr(packed), packed.size, _np_ptr(codes), _np_ptr(cb),
                              _np_ptr(sc)))
    return codes, cb.view(np.float16), sc.view(np.float16)


def lut_packed_bytes(bits: int, N: int, K: int) -> int:
    n = C.c_size_t()
    _check(lib().vqmlp_lut_packed_bytes(bits, N, K, C.byref(n)))
    return n.value


def lut_pack(bits: int, codes, lut, sc) -> np.ndarray:
    codes = np.ascontiguousarray(codes, np.uint8)
    lut, sc = _u16(lut), _u16(sc)
    N, K = codes.shape
    out = np.empty(lut_packed_bytes(bits, N, K), np.uint8)
    _check(lib().vqmlp_lut_pack(bits, N, K, _np_ptr(codes), _np_ptr(lut), _np_ptr(sc),
                                _np_ptr(out), out.size))
    return out


def lut_unpack(bits: int, N: int, K: int, packed):
    packed = np.ascontiguousarray(packed, np.uint8)
    codes = np.empty((N, K), np.uint8)
    lut = np.empty((N // 8, 1 << bits), np.uint16)
    sc = np.empty(N, np.uint16)
    _check(lib().vqmlp_lut_unpack(bits, N, K, _np_ptr(packed), packed.size, _np_ptr(codes),
                                  _np_ptr(lut), _np_ptr(sc)))
    return codes, lut.view(np.float16), sc.view(np.float16)


# ------------------------------------------------------------------ device side (torch)


def vq2_packed_bytes(N: int, K: int) -> int:
    n = C.c_size_t()
    _check(lib().vqmlp_vq2_packed_bytes(N, K, C.byref(n)))
    return n.value


def vq2_pack(codes, cb, sc) -> np.ndarray:
    """2x16 matrix: codes uint8 [N/2, K] (0..15), cb [N/8, 16, 2] and sc [N] binary16."""
    codes = np.ascontiguousarray(codes, np.uint8)
    cb, sc = _u16(cb), _u16(sc)
    N, K = sc.shape[0], codes.shape[1]
    out = np.empty(vq2_packed_bytes(N, K), np.uint8)
    _check(lib().vqmlp_vq2_pack(N, K, _np_ptr(codes), _np_ptr(cb), _np_ptr(sc), _np_ptr(out),
                                out.size))
    return out


def vq2_unpack(N: int, K: int, packed):
    packed = np.ascontiguousarray(packed, np.uint8)
    codes = np.empty((N // 2, K), np.uint8)
    cb = np.empty((N // 8, 16, 2), np.uint16)
    sc = np.empty(N, np.uint16)
    _check(lib().vqmlp_vq2_unpack(N, K, _np_ptr(packed), packed.size, _np_ptr(codes),
                                  _np_ptr(cb), _np_ptr(sc)))
    return codes, cb, sc


def to_device(a, device="cuda"):
    """numpy -> torch device tensor (float16 kept as its bits in int16)."""
    import torch

    a = np.ascontiguousarray(a)
    if a.dtype == np.float16:
        a = a.view(np.int16)
    return torch.from_numpy(a).to(device)


def workspace_errors(workspace, clear: bool = True, stream=None) -> int:
    """Error bits of the fused kernel's bounded waits in a forward workspace (0 = none); waits
    for the stream and, with clear, zeroes the word."""
    bits = C.c_uint32()
    _check(lib().vqmlp_workspace_errors(_dptr(workspace), workspace.numel(), int(clear),
                                        C.byref(bits), _stream(stream)))
    return bits.value


def stream_read(buf, sink, stream=None):
    """Measurement hook: one streaming read of the device tensor buf (bytes a multiple of 16)."""
    _check(lib().vqmlp_stream_read(_dptr(buf), buf.numel() * buf.element_size(), _dptr(sink),
                                   _stream(stream)))


def dequant(N: int, K: int, packed_dev, stream=None):
    import torch

    w = torch.empty((N, K), dtype=torch.float32, device=packed_dev.device)
    _check(lib().vqmlp_dequant(N, K, _dptr(packed_dev), _dptr(w), _stream(stream)))
    return w


def rotate(x_dev, b: int, s_dev=None, sign_dev=None, stream=None):
    """FP32 rotation test hook; x_dev int16 (binary16 bits) or float16 [T, n]."""
    import torch

    T, n = x_dev.shape
    out = torch.empty((T, n), dtype=torch.float32, device=x_dev.device)
    _check(lib().vqmlp_rotate(T, n, b, _dptr(x_dev), _dptr(s_dev), _dptr(sign_dev), _dptr(out),
                              _stream(stream)))
    return out


class MLP:
    """Device-resident packed weights of one MLP layer plus its plan."""

    def __init__(self, H, I, gate, up, down, s, sign_h=None, sign_i=None, had_block_h=0,
                 had_block_i=0, t_max=512, vq2=False):
        """vq2: the three matrices are packed 2x16 buffers (vq2_pack), else three-bit (pack)."""
        self.H, self.I, self.t_max = H, I, t_max
        self._keep = (gate, up, down, s, sign_h, sign_i)  # the plan does not own these
        d = _Desc(H, I, had_block_h, had_block_i, t_max, gate.data_ptr(), up.data_ptr(),
                  down.data_ptr(), s.data_ptr(),
                  sign_h.data_ptr() if sign_h is not None else None,
                  sign_i.data_ptr() if sign_i is not None else None)
        self._plan = C.c_void_p()
        create = lib().vqmlp_create_vq2 if vq2 else lib().vqmlp_create
        _check(create(C.byref(d), C.byref(self._plan)))
        self.device = gate.device

    @classmethod
    def from_layer(cls, layer, device="cuda", t_max=None):
        """Pack a ``synth.MLPLayer`` on the host and upload it."""
        packs = [to_device(pack(*m.as_u16()), device) for m in (layer.gate, layer.up, layer.down)]
        return cls(layer.H, layer.I, *packs, to_device(layer.s, device),
                   to_device(layer.sign_h, device), to_device(layer.sign_i, device),
                   layer.had_block_h, layer.had_block_i,
                   t_max if t_max is not None else max(layer.T, 8))

    @classmethod
    def from_vq2_layer(cls, layer, device="cuda", t_max=None):
        """Pack a ``synth.vq2_mlp_layer`` (2x16 matrices) on the host and upload it."""
        packs = [to_device(vq2_pack(*m.as_u16()), device) for m in (layer.gate, layer.up, layer.down)]
        return cls(layer.H, layer.I, *packs, to_device(layer.s, device),
                   to_device(layer.sign_h, device), to_device(layer.sign_i, device),
                   layer.had_block_h, layer.had_block_i,
                   t_max if t_max is not None else max(layer.T, 8), vq2=True)

    def workspace_bytes(self, T: int) -> int:
        n = C.c_size_t()
        _check(lib().vqmlp_workspace_bytes(self._plan, T, C.byref(n)))
        return n.value

    def workspace(self, T=None):
        import torch

        return torch.zeros(self.workspace_bytes(self.t_max if T is None else T),
                           dtype=torch.uint8, device=self.device)

    def forward(self, x, y=None, workspace=None, path=PATH_AUTO, stream=None):
        """x: [T, H] int16 (binary16 bits) or float16 device tensor -> y (same dtype)."""
        import torch

        T = x.shape[0]
        if y is None:
            y = torch.empty_like(x)
        if workspace is None:
            workspace = self.workspace(T)
        _check(lib().vqmlp_forward_path(self._plan, T, _dptr(x), _dptr(y), _dptr(workspace),
                                        workspace.numel(), path, _stream(stream)))
        return y

    def forward_noalloc(self, x, y=None, stream=None):
        """The forward with the library's fixed per-GPU scratch array as its workspace."""
        import torch

        if y is None:
            y = torch.empty_like(x)
        _check(lib().vqmlp_forward_noalloc(self._plan, x.shape[0], _dptr(x), _dptr(y),
                                           _stream(stream)))
        return y

    def __del__(self):
        if getattr(self, "_plan", None) and _lib is not None:
            _lib.vqmlp_destroy(self._plan)
            self._plan = None


class LUTProjection:
    """Device-resident scalar-LUT projection (2- or 4-bit codes, group-8 tables, optional
    rank-r factors) with its input scale, sign and Hadamard block."""

    def __init__(self, bits, N, K, packed, U=None, V=None, s=None, sign=None, had_block=1024):
        self.bits, self.N, self.K = bits, N, K
        self.r = 0 if U is None else U.shape[1]
        self.had_block = had_block
        self.packed, self.U, self.V, self.s, self.sign = packed, U, V, s, sign
        self.device = packed.device
        self._plan = C.c_void_p()
        _check(lib().vqmlp_lut_create(bits, N, K, _dptr(packed), _dptr(U), _dptr(V), self.r,
                                      _dptr(s), _dptr(sign), had_block, C.byref(self._plan)))

    @classmethod
    def from_proj(cls, proj, device="cuda"):
        """Pack a ``synth.LUTProjection`` on the host and upload it."""
        packed = to_device(lut_pack(proj.bits, proj.codes, proj.lut, proj.sc), device)
        up = lambda a: None if a is None else to_device(a, device)  # noqa: E731
        return cls(proj.bits, proj.N, proj.K, packed, up(proj.U), up(proj.V), up(proj.s),
                   up(proj.sign), proj.had_block)

    def workspace_bytes(self, T: int) -> int:
        n = C.c_size_t()
        _check(lib().vqmlp_lut_workspace_bytes(self.N, self.K, T, self.r, C.byref(n)))
        return n.value

    def workspace(self, T: int):
        import torch

        return torch.zeros(self.workspace_bytes(T), dtype=torch.uint8, device=self.device)

    def forward(self, x, y=None, workspace=None, stream=None):
        """x: [T, K] int16 (binary16 bits) or float16 device tensor -> y [T, N] (same dtype)."""
        import torch

        T = x.shape[0]
        if y is None:
            y = torch.empty((T, self.N), dtype=x.dtype, device=x.device)
        if workspace is None:
            workspace = self.workspace(T)
        _check(lib().vqmlp_lut_plan_forward(self._plan, T, _dptr(x), _dptr(y), _dptr(workspace),
                                            workspace.numel(), _stream(stream)))
        return y

    def argmax(self, x, workspace=None, stream=None):
        """Greedy argmax head: x [T, K] float16 device tensor (T <= 8) -> (index int32 [T],
        value float32 [T]): per token the lowest row of the largest logit, and that logit."""
        import torch

        T = x.shape[0]
        index = torch.empty(T, dtype=torch.int32, device=x.device)
        value = torch.empty(T, dtype=torch.float32, device=x.device)
        if workspace is None:
            workspace = self.workspace(T)
        _check(lib().vqmlp_lut_plan_argmax(self._plan, T, _dptr(x), _dptr(index), _dptr(value),
                                           _dptr(workspace), workspace.numel(), _stream(stream)))
        return index, value

    def forward_stateless(self, x, y=None, workspace=None, stream=None):
        """The same through vqmlp_lut_forward (validates the packed buffer on every call)."""
        import torch

        T = x.shape[0]
        if y is None:
            y = torch.empty((T, self.N), dtype=x.dtype, device=x.device)
        if workspace is None:
            workspace = self.workspace(T)
        _check(lib().vqmlp_lut_forward(self.bits, self.N, self.K, T, _dptr(self.packed),
                                       _dptr(self.U), _dptr(self.V), self.r, _dptr(self.s),
                                       _dptr(self.sign), self.had_block, _dptr(x), _dptr(y),
                                       _dptr(workspace), workspace.numel(), _stream(stream)))
        return y

    def __del__(self):
        if getattr(self, "_plan", None) and _lib is not None:
            _lib.vqmlp_lut_destroy(self._plan)
            self._plan = None


class VQ2Projection:
    """Device-resident 2x16 vector-LUT projection for T <= 8 tokens (x used as given)."""

    def __init__(self, N, K, packed):
        self.N, self.K, self.packed = N, K, packed
        self._plan = C.c_void_p()
        _check(lib().vqmlp_vq2_create(N, K, _dptr(packed), C.byref(self._plan)))

    @classmethod
    def from_matrix(cls, m, device="cuda"):
        """Pack a ``synth.VQ2Matrix`` on the host and upload it."""
        return cls(m.N, m.K, to_device(vq2_pack(m.codes, m.cb, m.sc), device))

    def forward(self, x, y=None, stream=None):
        """x: [T, K] binary16 device tensor (T <= 8) -> y [T, N] (same dtype)."""
        import torch

        if y is None:
            y = torch.empty((x.shape[0], self.N), dtype=x.dtype, device=x.device)
        _check(lib().vqmlp_vq2_plan_forward(self._plan, x.shape[0], _dptr(x), _dptr(y),
                                            _stream(stream)))
        return y

    def __del__(self):
        if getattr(self, "_plan", None) and _lib is not None:
            _lib.vqmlp_vq2_destroy(self._plan)
            self._plan = None



# ------------------------------------------------------------------ around the MLP
# Operators of a serving step over requests packed one after another (include/vqmlp.h, "around the
# MLP").  Each class keeps what stays from call to call; a call checks its tensors, allocates what
# the caller did not pass on the call's stream, and enqueues.


# A call of these costs the host less than the launch that it makes, where it can: a step has dozens of
# them.  Checks take the usual case first, and descriptions start as copies of what does not change.


class _OnStream:
    """The stream of a call and the context in which its temporaries are allocated: memory comes
    from that stream's pool, so it cannot be handed to another stream while the call runs."""

    __slots__ = ("raw", "stream", "device")

    def __init__(self, stream, device):
        import torch

        if device.type != "cuda":
            _bad("tensors are on %s, not on a GPU" % device)
        self.device, self.stream = device, stream
        self.raw = torch._C._cuda_getCurrentRawStream(device.index) if stream is None else stream.cuda_stream

    def empty(self, shape, dtype):
        import torch

        if self.stream is None:
            return torch.empty(shape, dtype=dtype, device=self.device)
        with torch.cuda.stream(self.stream):
            return torch.empty(shape, dtype=dtype, device=self.device)

    def like(self, t):
        """A new tensor of t's shape and type, dense whatever t's token stride."""
        import torch

        if self.stream is None:
            return torch.empty_like(t, memory_format=torch.contiguous_format)
        with torch.cuda.stream(self.stream):
            return torch.empty_like(t, memory_format=torch.contiguous_format)

    def call(self, f, *args):
        """f(*args, stream) with the tensors' device current."""
        import torch

        if torch._C._cuda_getDevice() == self.device.index:
            status = f(*args, self.raw)
        else:
            with torch.cuda.device(self.device):
                status = f(*args, self.raw)
        if status != OK:
            _check(status)


def _bad(msg):
    raise VqmlpError(ERR_INVALID_ARG, msg)


def _fits(value, what):
    """value: sizes or-ed together.  ctypes cuts an integer to 32 bits without a word."""
    if value >> 31:
        _bad("%s: a size is negative or beyond 2^31 - 1" % what)


_DTYPES = None


def _dtype(t, name):
    """vqmlp_dtype of a tensor (int16 holds binary16 bits)."""
    global _DTYPES
    if _DTYPES is None:
        import torch

        _DTYPES = {torch.float16: 0, torch.int16: 0, torch.bfloat16: 1, torch.float32: 2}
    d = _DTYPES.get(t.dtype)
    if d is None:
        _bad("%s: unsupported type %s" % (name, t.dtype))
    return d


def _need(t, name, device, dtype=None, shape=None, contiguous=True):
    """A tensor on device, of a torch type and shape (None entries are free)."""
    if t.device != device:
        _bad("%s is on %s, not on %s" % (name, t.device, device))
    if dtype is not None and t.dtype != dtype:
        _bad("%s is %s, not %s" % (name, t.dtype, dtype))
    if shape is not None and t.shape != shape and (t.dim() != len(shape) or any(
            s is not None and s != n for s, n in zip(shape, t.shape))):
        _bad("%s has shape %s, wanted %s" % (name, tuple(t.shape), tuple(shape)))
    if contiguous and not t.is_contiguous():
        _bad("%s is not contiguous" % name)
    return t.data_ptr()


def _rows(t, name, device, shape):
    """Pointer and token stride of [T, heads, D] (or [T, H]) whose rows are dense."""
    if t.device != device or t.shape != shape:
        _need(t, name, device, None, shape, contiguous=False)
    inner = shape[1] if len(shape) == 2 else shape[1] * shape[2]
    if t.is_contiguous():
        return t.data_ptr(), inner
    at = 1
    for n, st in zip(reversed(t.shape[1:]), reversed(t.stride()[1:])):
        if n != 1 and st != at:
            _bad("%s: a token's elements do not lie one after another" % name)
        at *= n
    return t.data_ptr(), t.stride(0) if t.shape[0] > 1 else inner


def _work(on, workspace, nbytes):
    """Pointer and size of a call's workspace: the caller's, or a new one on the call's stream (held
    by the third value until the call has been enqueued)."""
    import torch

    if workspace is None:
        if not nbytes:
            return None, 0, None
        workspace = on.empty((nbytes,), torch.uint8)
    elif workspace.device != on.device or not workspace.is_contiguous():
        _bad("workspace: not contiguous, or not on %s" % on.device)
    return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace


def _fixed(name):
    """An attribute set once: the library was given its pointer or size."""
    return property(lambda self: getattr(self, "_" + name))


class BlockNorm:
    """r = residual + residual_scale * gate * N_post(y); x = N_pre(r): the norms, the gate and the
    residual sum between two blocks in one pass.  Weights [H] of y's type (None: that norm, or its
    bias, is left out); kind "rms" or "layer"; weight_offset is added to both weights."""

    KINDS = {"rms": 0, "layer": 1}

    def __init__(self, pre_weight=None, pre_bias=None, *, post_weight=None, post_bias=None,
                 kind="rms", eps=1e-6, residual_scale=1.0, weight_offset=0.0):
        if kind not in self.KINDS:
            _bad("unknown norm kind %r" % (kind,))
        ws = {"pre_w": pre_weight, "pre_b": pre_bias, "post_w": post_weight, "post_b": post_bias}
        if (pre_bias is not None and pre_weight is None) or (post_bias is not None and post_weight is None):
            _bad("a bias needs its weight")
        self._keep = [w for w in ws.values() if w is not None]
        self.has_pre, self.has_post = pre_weight is not None, post_weight is not None
        self._desc = _NormDesc(kind=self.KINDS[kind], eps=eps, res_scale=residual_scale,
                               w_offset=weight_offset)
        for name, w in ws.items():
            if w is not None:
                setattr(self._desc, name, _need(w, name, self._keep[0].device, self._keep[0].dtype,
                                                (self._keep[0].shape[0],)))

    def forward(self, y, residual=None, gate=None, residual_out=None, out=None, stream=None):
        """y [T, H] (None: only the norm of residual), residual [T, H] of y's type or float32, gate
        [T, H] or [H] -> (r of residual's type, x of y's type; None without pre_weight).
        residual_out may be residual and out may be y."""
        base = y if y is not None else residual
        if base is None:
            _bad("neither y nor residual")
        dev, shape = base.device, base.shape
        if len(shape) != 2:
            _bad("y and residual are [T, H]")
        T, H = shape
        x_dtype = y.dtype if y is not None else self._keep[0].dtype if self._keep else residual.dtype
        if self._keep:
            w = self._keep[0]
            if w.shape[0] != H or w.device != dev or _dtype(w, "weight") != _DTYPES.get(x_dtype):
                _bad("the weights do not fit y (H, type or device)")
        if y is None and self.has_post:
            _bad("post_weight without y")
        _fits(T | H, "block norm")
        d = _NormDesc.from_buffer_copy(self._desc)
        d.T, d.H = T, H
        on = _OnStream(stream, dev)
        if y is not None:
            kind = _dtype(y, "y")
            d.y, d.ld_y = _rows(y, "y", dev, shape)
        else:
            kind = _DTYPES[x_dtype] if self._keep else _dtype(residual, "residual")
        d.dtype = res_kind = kind
        if residual is not None:
            res_kind = _dtype(residual, "residual")
            d.res, d.ld_res = _rows(residual, "residual", dev, shape)
        elif residual_out is not None:
            res_kind = _dtype(residual_out, "residual_out")
        d.res_dtype = res_kind
        if gate is not None:
            if _dtype(gate, "gate") != kind:
                _bad("gate and y differ in type")
            if gate.dim() == 1:
                d.gate, d.ld_gate = _need(gate, "gate", dev, None, (H,)), 0
            else:
                d.gate, d.ld_gate = _rows(gate, "gate", dev, shape)
        if residual_out is None:
            residual_out = on.like(residual if residual is not None else y)
            d.res_out, d.ld_res_out = residual_out.data_ptr(), H
        else:
            if _dtype(residual_out, "residual_out") != res_kind:
                _bad("residual_out and residual differ in type")
            d.res_out, d.ld_res_out = _rows(residual_out, "residual_out", dev, shape)
        if self.has_pre:
            if out is None:
                out = on.like(y) if y is not None else on.empty(shape, x_dtype)
                d.x, d.ld_x = out.data_ptr(), H
            else:
                if _dtype(out, "out") != kind:
                    _bad("out and y differ in type")
                d.x, d.ld_x = _rows(out, "out", dev, shape)
        elif out is not None:
            _bad("out without pre_weight")
        on.call(lib().vqmlp_block_norm, C.byref(d))
        return residual_out, out


class PagePlan:
    """One step's plan on the device (all int32): seq_len [R], cu_q [R + 1], slot and position
    [max_tokens] (-1 behind the last token), status [4] = error bits, tokens, pages taken, 0."""

    __slots__ = ("seq_len", "cu_q", "slot", "position", "status")

    def __init__(self, *parts):
        self.seq_len, self.cu_q, self.slot, self.position, self.status = parts


class PagePlanner:
    """Block tables and slot maps from request lengths, made on the device.  table [R, width] int32
    is kept up to date in place; free_pages [n] int32 is the free list, taken from free_head (int32
    [1] on the device, None: 0) on.  See include/vqmlp.h for the error bits."""

    R, device, max_tokens = _fixed("R"), _fixed("device"), _fixed("max_tokens")
    table, free_pages, free_head = _fixed("table"), _fixed("free_pages"), _fixed("free_head")
    page_size, n_pages = _fixed("page_size"), _fixed("n_pages")

    def __init__(self, table, free_pages, page_size, n_pages, max_tokens, free_head=None):
        import torch

        dev = table.device
        _need(table, "table", dev, torch.int32, (None, None), contiguous=False)
        _fits(table.shape[0] | table.shape[1] | page_size | n_pages | max_tokens | free_pages.numel(), "page plan")
        if table.shape[1] > 1 and table.stride(1) != 1:
            _bad("table: a row's entries do not lie one after another")
        self._R, self._device, self._max_tokens = table.shape[0], dev, max_tokens
        self._table, self._free_pages, self._free_head = table, free_pages, free_head
        self._page_size, self._n_pages = page_size, n_pages
        self._sizes = [self._R, self._R + 1, max_tokens, max_tokens, 4]  # of a plan's parts
        self._total = sum(self._sizes)
        self._desc = _PagesDesc(R=self._R, max_tokens=max_tokens, page_size=page_size, n_pages=n_pages,
                                n_free=free_pages.numel(), table_width=table.shape[1],
                                ld_table=table.stride(0) if self._R > 1 else table.shape[1],
                                free_pages=_need(free_pages, "free_pages", dev, torch.int32, (None,)),
                                table=table.data_ptr())
        if free_head is not None:
            self._desc.free_head = _need(free_head, "free_head", dev, torch.int32, (1,))

    def empty_plan(self, stream=None):
        return self._empty_plan(_OnStream(stream, self._device))

    def _empty_plan(self, on):
        import torch

        buf = on.empty((self._total,), torch.int32)
        return PagePlan(*torch.split_with_sizes(buf, self._sizes))

    def forward(self, ctx_len, q_len, plan=None, free_head_out=None, stream=None):
        """ctx_len, q_len [R] int32 on the device -> PagePlan (plan: buffers to reuse)."""
        import torch

        i, dev = torch.int32, self._device
        d = _PagesDesc.from_buffer_copy(self._desc)
        d.ctx_len = _need(ctx_len, "ctx_len", dev, i, (self._R,))
        d.q_len = _need(q_len, "q_len", dev, i, (self._R,))
        on = _OnStream(stream, dev)
        if plan is None:
            plan = self._empty_plan(on)
            at = d.seq_len = plan.seq_len.data_ptr()
            d.cu_q = at = at + 4 * self._R
            d.slot = at = at + 4 * (self._R + 1)
            d.position = at = at + 4 * self._max_tokens
            d.status = at + 4 * self._max_tokens
        else:
            d.seq_len = _need(plan.seq_len, "seq_len", dev, i, (self._R,))
            d.cu_q = _need(plan.cu_q, "cu_q", dev, i, (self._R + 1,))
            d.slot = _need(plan.slot, "slot", dev, i, (self._max_tokens,))
            d.position = _need(plan.position, "position", dev, i, (self._max_tokens,))
            d.status = _need(plan.status, "status", dev, i, (4,))
        if free_head_out is not None:
            d.free_head_out = _need(free_head_out, "free_head_out", dev, i, (1,))
        on.call(lib().vqmlp_page_plan, C.byref(d))
        return plan


class PagedCache:
    """A paged key/value cache: k [pages, kv_heads, page_size, D], v [pages, kv_heads, D, page_size]
    (float16, int16 as binary16 bits, or bfloat16)."""

    k, v, device, dtype = _fixed("k"), _fixed("v"), _fixed("device"), _fixed("dtype")
    n_pages, kv_heads, page_size, D = _fixed("n_pages"), _fixed("kv_heads"), _fixed("page_size"), _fixed("D")

    def __init__(self, k, v):
        _need(k, "k", k.device, None, (None,) * 4)
        n, h, p, D = k.shape
        _fits(n | h | p | D, "paged cache")
        _need(v, "v", k.device, k.dtype, (n, h, D, p))
        self._k, self._v, self._device = k, v, k.device
        self._n_pages, self._kv_heads, self._page_size, self._D = n, h, p, D
        self._dtype = _dtype(k, "k")
        self._kp, self._vp = k.data_ptr(), v.data_ptr()
        self._work = {}  # workspace bytes of a description's sizes

    @classmethod
    def empty(cls, n_pages, kv_heads, page_size, D, dtype, device="cuda"):
        import torch

        return cls(torch.empty((n_pages, kv_heads, page_size, D), dtype=dtype, device=device),
                   torch.empty((n_pages, kv_heads, D, page_size), dtype=dtype, device=device))

    def store(self, k, v, slot, stream=None):
        """k, v [T, kv_heads, D] into slot[t] (int32 [T]; a slot outside the cache is skipped)."""
        import torch

        T, dev = k.shape[0], self._device
        _fits(T, "store")
        shape = (T, self._kv_heads, self._D)
        if _dtype(k, "k") != self._dtype or _dtype(v, "v") != self._dtype:
            _bad("k, v and the cache differ in type")
        kp, ld_k = _rows(k, "k", dev, shape)
        vp, ld_v = _rows(v, "v", dev, shape)
        sp = _need(slot, "slot", dev, torch.int32, (None,))
        if slot.shape[0] < T:
            _bad("slot has %d entries for %d tokens" % (slot.shape[0], T))
        _OnStream(stream, dev).call(lib().vqmlp_paged_store, self._dtype, T, self._kv_heads, self._D,
                                    self._page_size, self._n_pages, kp, ld_k, vp, ld_v, sp, self._kp,
                                    self._vp)

    def _attn_desc(self, T, R, heads, table_width, window, max_kv, scale):
        if max_kv is None:
            max_kv = table_width * self._page_size
        _fits(T | R | heads | table_width | window | max_kv, "attention")
        return _AttnDesc(self._dtype, T, R, heads, self._kv_heads, self._D, self._page_size, self._n_pages,
                         window, max_kv, self._D ** -0.5 if scale is None else scale, table_width)

    def _work_bytes(self, d):
        key = (d.T, d.R, d.heads, d.max_kv, d.table_width, d.window)
        n = self._work.get(key)
        if n is None:
            import torch

            n = C.c_size_t()
            with torch.cuda.device(self._device):
                _check(lib().vqmlp_paged_attn_workspace(C.byref(d), C.byref(n)))
            if len(self._work) >= 4096:
                self._work.clear()
            n = self._work[key] = n.value
        return n

    def workspace_bytes(self, T, R, heads, table_width, max_kv=None):
        return self._work_bytes(self._attn_desc(T, R, heads, table_width, 0, max_kv, None))

    def attention(self, q, table, cu_q, kv_len, *, scale=None, window=0, max_kv=None, y=None,
                  lse=None, with_lse=False, workspace=None, stream=None):
        """q [T, heads, D] against the cached positions of each request: table [R, width], cu_q
        [R + 1], kv_len [R] int32 on the device (kv_len counts the new tokens, stored before).
        scale: 1 / sqrt(D) if None.  max_kv: the longest kv_len expected (None: what the table
        holds).  Returns y, or (y, lse float32 [T, heads]) with with_lse or lse."""
        import torch

        dev, i = self._device, torch.int32
        if q.dim() != 3:
            _bad("q is [T, heads, D]")
        if _dtype(q, "q") != self._dtype:
            _bad("q and the cache differ in type")
        T, heads, R = q.shape[0], q.shape[1], kv_len.shape[0]
        _need(table, "table", dev, i, (R, None), contiguous=False)
        if table.shape[1] > 1 and table.stride(1) != 1:
            _bad("table: a row's entries do not lie one after another")
        d = self._attn_desc(T, R, heads, table.shape[1], window, max_kv, scale)
        on = _OnStream(stream, dev)
        d.q, d.ld_q = _rows(q, "q", dev, (T, heads, self._D))
        if y is None:
            y = on.like(q)
            d.y, d.ld_y = y.data_ptr(), heads * self._D
        else:
            if _dtype(y, "y") != self._dtype:
                _bad("y and the cache differ in type")
            d.y, d.ld_y = _rows(y, "y", dev, (T, heads, self._D))
        if lse is None and with_lse:
            lse = on.empty((T, heads), torch.float32)
        if lse is not None:
            d.lse = _need(lse, "lse", dev, torch.float32, (T, heads))
        d.k_cache, d.v_cache = self._kp, self._vp
        d.table, d.ld_table = table.data_ptr(), table.stride(0) if R > 1 else table.shape[1]
        d.cu_q = _need(cu_q, "cu_q", dev, i, (R + 1,))
        d.kv_len = _need(kv_len, "kv_len", dev, i, (R,))
        work, nbytes, _hold = _work(on, workspace, self._work_bytes(d))
        on.call(lib().vqmlp_paged_attn, C.byref(d), work, nbytes)
        return y if lse is None else (y, lse)


class LinearAttention:
    """S_t = exp(g_t) S_{t-1} + k_t v_t^T, y_t = scale * S_t^T q_t per value head (which shares key
    head h // (v_heads // k_heads)).  scale: 1 / sqrt(Dk) if None."""

    def __init__(self, k_heads, v_heads, Dk, Dv, scale=None):
        self.k_heads, self.v_heads, self.Dk, self.Dv = k_heads, v_heads, Dk, Dv
        self.scale = Dk ** -0.5 if scale is None else scale
        self._work = {}  # workspace bytes of (device, T, R, max_q)

    def state(self, n, device="cuda"):
        """Zero states for n requests."""
        import torch

        return torch.zeros((n, self.v_heads, self.Dk, self.Dv), dtype=torch.float32, device=device)

    def _desc(self, dtype, T, R, n_states, max_q):
        _fits(T | R | n_states | max_q, "linear attention")
        return _LinearDesc(dtype, T, R, self.k_heads, self.v_heads, self.Dk, self.Dv, n_states, max_q,
                           self.scale)

    def workspace_bytes(self, T, R, max_q):
        n = C.c_size_t()
        _check(lib().vqmlp_linear_attn_workspace(C.byref(self._desc(0, T, R, 0, max_q)), C.byref(n)))
        return n.value

    def _work_bytes(self, d, device):
        key = (device.index, d.T, d.R, d.max_q)
        n = self._work.get(key)
        if n is None:
            import torch

            with torch.cuda.device(device):
                n = self.workspace_bytes(d.T, d.R, d.max_q)
            if len(self._work) >= 4096:
                self._work.clear()
            self._work[key] = n
        return n

    def forward(self, q, k, v, g, state, cu_q, *, ctx_len=None, state_index=None, state_out=None,
                max_q=None, y=None, workspace=None, stream=None):
        """q, k [T, k_heads, Dk], v [T, v_heads, Dv], g float32 [T, v_heads], state float32 [slots,
        v_heads, Dk, Dv], cu_q int32 [R + 1]; ctx_len int32 [R]: a request with 0 starts from zero;
        state_index int32 [R]: its slot (None: r).  max_q: the most new tokens of one request that
        are expected (None: T).  state_out may be state; slots that no request uses are left as
        they are (a new state_out starts as a copy of state where there are such slots).  Returns
        (y [T, v_heads, Dv], state_out)."""
        import torch

        dev, i, f = q.device, torch.int32, torch.float32
        T, R = q.shape[0], cu_q.shape[0] - 1
        dt = _dtype(q, "q")
        if _dtype(k, "k") != dt or _dtype(v, "v") != dt:
            _bad("q, k and v differ in type")
        on = _OnStream(stream, dev)
        d = self._desc(dt, T, R, state.shape[0], T if max_q is None else max_q)
        d.q, d.ld_q = _rows(q, "q", dev, (T, self.k_heads, self.Dk))
        d.k, d.ld_k = _rows(k, "k", dev, (T, self.k_heads, self.Dk))
        d.v, d.ld_v = _rows(v, "v", dev, (T, self.v_heads, self.Dv))
        if g.dtype != f:
            _bad("g is %s, not %s" % (g.dtype, f))
        d.g, d.ld_g = _rows(g, "g", dev, (T, self.v_heads))
        if y is None:
            y = on.like(v) if v.dtype == q.dtype else on.empty(v.shape, q.dtype)
            d.y, d.ld_y = y.data_ptr(), self.v_heads * self.Dv
        else:
            if _dtype(y, "y") != dt:
                _bad("y and q differ in type")
            d.y, d.ld_y = _rows(y, "y", dev, (T, self.v_heads, self.Dv))
        shape = (state.shape[0], self.v_heads, self.Dk, self.Dv)
        d.state_in = _need(state, "state", dev, f, shape)
        if state_out is None:
            state_out = on.like(state)
            if state_index is not None or shape[0] > R:
                if stream is None:
                    state_out.copy_(state)
                else:
                    with torch.cuda.stream(stream):
                        state_out.copy_(state)
            d.state_out = state_out.data_ptr()
        else:
            d.state_out = _need(state_out, "state_out", dev, f, shape)
        d.cu_q = _need(cu_q, "cu_q", dev, i, (R + 1,))
        if ctx_len is not None:
            d.ctx_len = _need(ctx_len, "ctx_len", dev, i, (R,))
        if state_index is not None:
            d.state_index = _need(state_index, "state_index", dev, i, (R,))
        work, nbytes, _hold = _work(on, workspace, self._work_bytes(d, dev))
        on.call(lib().vqmlp_linear_attn, C.byref(d), work, nbytes)
        return y, state_out
