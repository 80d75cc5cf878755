"""ctypes view of the C ABI in include/vscan.h (libvscan.so, built in-tree).

Argument marshalling only: no arithmetic of the scan happens in Python. Loading
fails loudly when the library has not been built; there is no fallback path.
"""
import ctypes
import os
import struct

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libvscan.so")

OK = 0
STATUS = {
    0: "VSCAN_OK",
    -1: "VSCAN_ERR_INVALID_ARGUMENT",
    -2: "VSCAN_ERR_SHAPE",
    -3: "VSCAN_ERR_ALIGNMENT",
    -4: "VSCAN_ERR_UNSUPPORTED",
    -5: "VSCAN_ERR_CUDA",
    -6: "VSCAN_ERR_WORKSPACE",
    -7: "VSCAN_ERR_VALUE",
    -8: "VSCAN_ERR_DEVICE_TIMEOUT",
}
ROUTES = {"bidir": 0, "cross4": 1, "atrous2": 2, "pool_w": 3, "pool_h": 4}
F32, BF16 = 0, 1
ABI_VERSION = 5
FLAG_ZOH = 1
FLAG_CHECK_VALUES = 2


class VscanArgs(ctypes.Structure):
    """Mirror of struct vscan_args (include/vscan.h)."""

    _fields_ = [
        ("batch", ctypes.c_int32),
        ("channels", ctypes.c_int32),
        ("d_state", ctypes.c_int32),
        ("dtype", ctypes.c_int32),
        ("u", ctypes.c_void_p),
        ("delta", ctypes.c_void_p),
        ("B", ctypes.c_void_p),
        ("C", ctypes.c_void_p),
        ("z", ctypes.c_void_p),
        ("y", ctypes.c_void_p),
        ("A", ctypes.c_void_p),
        ("Dskip", ctypes.c_void_p),
        ("delta_bias", ctypes.c_void_p),
        ("per_dir_inputs", ctypes.c_int32),
        ("per_dir_params", ctypes.c_int32),
        ("delta_softplus", ctypes.c_int32),
        ("merge_scale", ctypes.c_float),
        ("workspace", ctypes.c_void_p),
        ("workspace_bytes", ctypes.c_uint64),
        ("seq_chunks", ctypes.c_int32),
        ("flags", ctypes.c_int32),
        ("conv_w", ctypes.c_void_p),
        ("conv_b", ctypes.c_void_p),
        ("token_pos", ctypes.c_void_p),
        ("n_tokens", ctypes.c_int32),
        ("reserved2", ctypes.c_int32),
        ("status", ctypes.c_void_p),
        ("tok_stride", ctypes.c_int64),
        ("batch_stride", ctypes.c_int64),
        ("bc_tok_stride", ctypes.c_int64),
        ("bc_batch_stride", ctypes.c_int64),
    ]


class VscanGrads(ctypes.Structure):
    """Mirror of struct vscan_grads (include/vscan.h)."""

    _fields_ = [(name, ctypes.c_void_p) for name in
                ("du", "ddelta", "dB", "dC", "dA", "dDskip", "dbias", "dz", "workspace")] + [
        ("workspace_bytes", ctypes.c_uint64)]


class VscanDeltaArgs(ctypes.Structure):
    """Mirror of struct vscan_delta_args (include/vscan.h)."""

    _fields_ = (
        [(name, ctypes.c_int32) for name in
         ("batch", "tokens", "heads_k", "heads_v", "dim_k", "dim_v", "dtype", "direction")]
        + [(name, ctypes.c_void_p) for name in
           ("q", "k", "v", "a", "b", "y", "A", "bias", "initial_state", "final_state", "seq_offsets")]
        + [("scale", ctypes.c_float), ("beta_scale", ctypes.c_float)]
        + [(f"{name}_{axis}_stride", ctypes.c_int64) for name in "qkvaby" for axis in ("tok", "batch")]
        + [("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_uint64), ("status", ctypes.c_void_p)]
    )


class VscanDeltaGrads(ctypes.Structure):
    """Mirror of struct vscan_delta_grads (include/vscan.h)."""

    _fields_ = [(name, ctypes.c_void_p) for name in
                ("dq", "dk", "dv", "da", "db", "dA", "dbias", "d_initial_state", "d_final_state", "workspace")] + [
        ("workspace_bytes", ctypes.c_uint64)]


class VscanQkNormArgs(ctypes.Structure):
    """Mirror of struct vscan_qknorm_args (include/vscan.h)."""

    _fields_ = (
        [(name, ctypes.c_int32) for name in
         ("batch", "tokens", "heads_q", "heads_k", "dim", "pairs", "axes", "dtype", "norm")]
        + [("eps", ctypes.c_float)]
        + [(name, ctypes.c_void_p) for name in ("q", "k", "yq", "yk", "wq", "wk", "inv_freq", "positions")]
        + [("pos_per_image", ctypes.c_int32), ("reserved", ctypes.c_int32)]
        + [(f"{name}_{axis}_stride", ctypes.c_int64) for name in ("q", "k", "yq", "yk") for axis in ("tok", "batch")]
    )


class VscanQkNormGrads(ctypes.Structure):
    """Mirror of struct vscan_qknorm_grads (include/vscan.h)."""

    _fields_ = [(name, ctypes.c_void_p) for name in ("dyq", "dyk", "dq", "dk", "dwq", "dwk", "workspace")] + [
        ("workspace_bytes", ctypes.c_uint64)]


class VscanError(RuntimeError):
    def __init__(self, status, message):
        self.status = status
        super().__init__(f"{STATUS.get(status, status)}: {message}")


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build it with `python -c 'import __graft_entry__ as g; g.build()'` "
            "(or python vision_selective_state_b200/build.py). There is no CPU fallback.")
    lib = ctypes.CDLL(LIB_PATH)
    i32, p, u64 = ctypes.c_int32, ctypes.c_void_p, ctypes.c_uint64
    pa = ctypes.POINTER(VscanArgs)
    pd = ctypes.POINTER(VscanDeltaArgs)
    pn = ctypes.POINTER(VscanQkNormArgs)
    sigs = {
        "vscan_create_route": ([ctypes.POINTER(p), i32, i32, i32, i32], i32),
        "vscan_destroy": ([p], i32),
        "vscan_route_info": ([p] + [ctypes.POINTER(i32)] * 5, i32),
        "vscan_route_indices": ([p, p, p], i32),
        "vscan_workspace_size": ([p, pa, ctypes.POINTER(u64)], i32),
        "vscan_forward": ([p, pa, p], i32),
        "vscan_plan_info": ([p, pa, ctypes.POINTER(i32)], i32),
        "vscan_plan_kernel": ([p, pa, ctypes.POINTER(ctypes.c_char_p)], i32),
        "vscan_forward_pooled_noalloc": ([p, pa, p], i32),
        "vscan_host_buffer_size": ([p, pa, ctypes.POINTER(u64)], i32),
        "vscan_forward_host": ([p, pa, p, u64, p], i32),
        "vscan_backward_workspace_size": ([p, pa, ctypes.POINTER(u64)], i32),
        "vscan_backward_plan_kernel": ([p, pa, ctypes.POINTER(ctypes.c_char_p)], i32),
        "vscan_backward": ([p, pa, p, ctypes.POINTER(VscanGrads), p], i32),
        "vscan_delta_workspace_size": ([p, pd, ctypes.POINTER(u64)], i32),
        "vscan_delta_forward": ([p, pd, p], i32),
        "vscan_delta_backward_workspace_size": ([p, pd, ctypes.POINTER(u64)], i32),
        "vscan_delta_backward": ([p, pd, p, ctypes.POINTER(VscanDeltaGrads), p], i32),
        "vscan_delta_step": ([pd, p], i32),
        "vscan_qknorm_forward": ([pn, p], i32),
        "vscan_qknorm_backward_workspace_size": ([pn, ctypes.POINTER(u64)], i32),
        "vscan_qknorm_backward": ([pn, ctypes.POINTER(VscanQkNormGrads), p], i32),
        "vscan_last_error": ([], ctypes.c_char_p),
        "vscan_status_string": ([i32], ctypes.c_char_p),
        "vscan_status_from_device_word": ([i32], i32),
        "vscan_abi_version": ([], i32),
    }
    for name, (argtypes, restype) in sigs.items():
        fn = getattr(lib, name)
        fn.argtypes = argtypes
        fn.restype = restype
    if lib.vscan_abi_version() != ABI_VERSION:
        raise ImportError(f"libvscan.so ABI {lib.vscan_abi_version()} != binding ABI {ABI_VERSION}")
    return lib


lib = _load()


class Call:
    """A library function whose argument struct is passed as the bytes of a struct.Struct: filling
    a ctypes structure field by field costs more than the smallest kernels take. `fields` is the
    struct's format, which has to have the ctypes mirror's size."""

    def __init__(self, name, fields, mirror, argtypes):
        self.pack = struct.Struct(fields).pack
        if struct.calcsize(fields) != ctypes.sizeof(mirror):
            raise ImportError(f"{name}: {fields} is not the layout of {mirror.__name__}")
        self.fn = ctypes.CDLL(LIB_PATH)[name]  # a function object of its own, with its own argument types
        self.fn.argtypes, self.fn.restype = argtypes, ctypes.c_int32


DELTA_FIELDS = "@8i11Q2f12q3Q"
QKNORM_FIELDS = "@9if8Q2i8q"
delta_workspace_size = Call("vscan_delta_workspace_size", DELTA_FIELDS, VscanDeltaArgs,
                            [ctypes.c_void_p, ctypes.c_char_p, ctypes.c_void_p])
delta_forward = Call("vscan_delta_forward", DELTA_FIELDS, VscanDeltaArgs, [ctypes.c_void_p, ctypes.c_char_p, ctypes.c_void_p])
delta_backward_workspace_size = Call("vscan_delta_backward_workspace_size", DELTA_FIELDS, VscanDeltaArgs,
                                     [ctypes.c_void_p, ctypes.c_char_p, ctypes.c_void_p])
delta_backward = Call("vscan_delta_backward", DELTA_FIELDS, VscanDeltaArgs,
                      [ctypes.c_void_p, ctypes.c_char_p, ctypes.c_void_p, ctypes.POINTER(VscanDeltaGrads), ctypes.c_void_p])
delta_step = Call("vscan_delta_step", DELTA_FIELDS, VscanDeltaArgs, [ctypes.c_char_p, ctypes.c_void_p])
qknorm_forward = Call("vscan_qknorm_forward", QKNORM_FIELDS, VscanQkNormArgs, [ctypes.c_char_p, ctypes.c_void_p])
qknorm_backward_workspace_size = Call("vscan_qknorm_backward_workspace_size", QKNORM_FIELDS, VscanQkNormArgs,
                                      [ctypes.c_char_p, ctypes.c_void_p])
qknorm_backward = Call("vscan_qknorm_backward", QKNORM_FIELDS, VscanQkNormArgs,
                       [ctypes.c_char_p, ctypes.POINTER(VscanQkNormGrads), ctypes.c_void_p])


def check(status):
    if status != OK:
        raise VscanError(status, lib.vscan_last_error().decode())
    return status
