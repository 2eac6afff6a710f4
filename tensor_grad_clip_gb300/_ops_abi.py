"""ctypes declarations of include/soma_ops.h, one Python name per C name."""
from __future__ import annotations

import ctypes

from . import _abi

SOMA_ACT_NONE = 0
SOMA_ACT_RELU = 1
SOMA_ACT_GELU = 2
SOMA_ACT_GELU_TANH = 3
SOMA_ACT_SILU = 4
SOMA_INDEX_I32 = 0
SOMA_INDEX_I64 = 1
SOMA_DISTILL_MAX_TOP = 1024

_S = _abi.soma_status_t
_I32 = ctypes.c_int32
_I64 = ctypes.c_int64
_I64P = ctypes.POINTER(ctypes.c_int64)
_D = ctypes.c_double
_P = ctypes.c_void_p

# name -> (restype, argtypes); every function the header declares.
SIGNATURES = {
    "soma_ops_last_error": (ctypes.c_char_p, []),
    "soma_layer_norm_forward": (_S, [_I32, _P, _I64, _P, _P, _P, _I64, _P, _P, _I64, _I64, _I32, _I32, _D, _P]),
    "soma_layer_norm_backward_workspace": (_S, [_I32, _I64, _I64, _I64P]),
    "soma_layer_norm_backward": (_S, [_I32, _P, _I64, _P, _I64, _P, _P, _P, _P, _I64, _P, _P, _P, _I64, _I64, _I64,
                                      _I32, _I32, _P]),
    "soma_linear_forward_workspace": (_S, [_I32, _P, _I64, _P, _I64, _I64, _I64, _I64, _I32, _I64P]),
    "soma_linear_forward": (_S, [_I32, _P, _I64, _P, _I64, _P, _P, _I64, _P, _I64, _P, _I64, _P, _I64, _I64, _I64,
                                 _I64, _I32, _I32, _P]),
    "soma_linear_backward_workspace": (_S, [_I32, _P, _I64, _P, _I64, _P, _I64, _I64, _I64, _I64, _I32, _I32,
                                            _I64P]),
    "soma_linear_backward": (_S, [_I32, _P, _I64, _P, _I64, _P, _I64, _P, _I64, _P, _I64, _P, _I64, _P, _P, _I64,
                                  _I64, _I64, _I64, _I32, _I32, _P]),
    "soma_ops_check": (_S, [_I32]),
    "soma_distill_forward": (_S, [_I32, _P, _I64, _P, _I64, _P, _I64, _P, _D, _P, _P, _I64, _I64, _I64, _I32, _I32,
                                  _I32, _P]),
    "soma_distill_backward": (_S, [_I32, _P, _P, _I64, _P, _P, _I64, _P, _I64, _P, _D, _P, _I64, _I64, _I64, _I64,
                                   _I32, _I32, _I32, _P]),
    "soma_distill_loss_grad": (_S, [_I32, _P, _I64, _P, _I64, _P, _I64, _P, _D, _P, _P, _P, _I64, _I64, _I64, _I64,
                                    _I32, _I32, _I32, _P]),
    "soma_embedding_forward": (_S, [_I32, _P, _I64, _P, _I64, _I64, _I64, _P, _I64, _I64, _I64, _I32, _I32, _D, _P]),
    "soma_embedding_backward_workspace": (_S, [_I32, _I64, _I64, _I64, _I64P]),
    "soma_embedding_backward": (_S, [_I32, _P, _I64, _P, _I64, _I64, _I64, _P, _I64, _I32, _P, _I64, _I64, _I64, _I32,
                                     _I32, _D, _P]),
    "soma_linear_cross_entropy_workspace": (_S, [_I32, _P, _I64, _I64, _I64, _I64, _I32, _I32, _I32, _I32, _I64P]),
    "soma_linear_cross_entropy_forward": (_S, [_I32, _P, _I64, _P, _I64, _P, _I64, _I64, _I64, _P, _P, _P, _P, _I64, _I64,
                                               _I64, _I32, _I32, _P]),
    "soma_linear_cross_entropy_backward": (_S, [_I32, _P, _P, _I64, _P, _I64, _P, _I64, _I64, _I64, _P, _P, _P, _I64, _P,
                                                _I64, _P, _I64, _I64, _I64, _I32, _I32, _P]),
    "soma_linear_cross_entropy_loss_grad": (_S, [_I32, _P, _I64, _P, _I64, _P, _I64, _I64, _I64, _P, _P, _P, _P, _I64, _P,
                                                 _I64, _P, _I64, _I64, _I64, _I32, _I32, _P]),
}

_lib = None


def load() -> ctypes.CDLL:
    """Load libsoma_opt.so (built by tensor_grad_clip_gb300.build) with this header's functions declared."""
    global _lib
    if _lib is None:
        lib = _abi.load()
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
            globals()[name] = fn
        _lib = lib
    return _lib
