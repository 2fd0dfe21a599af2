"""GB300-native C = ReLU(A . B): fp16 inputs, fp32 accumulation, fp16 output.

The compute path is a hand-written sm_103a CUDA library behind a C ABI
(``include/gemm_relu.h``); ``binding`` marshals torch tensors to it.  The
library is loaded lazily on first use so that importing this package (for
example to draw the seeded workloads in ``workloads``) needs no GPU.
"""
import importlib

__all__ = ["gemm_relu", "gemm_relu_host", "gemm_relu_grouped", "gemm_relu_grouped_dx", "gemm_relu_grouped_dw",
           "gemm_relu_adapters", "binding", "workloads"]

_FUNCTIONS = frozenset(__all__[:6]) | {"check_device_error"}


def __getattr__(name):
    if name in ("binding", "build", "workloads"):
        return importlib.import_module(f".{name}", __name__)
    if name in _FUNCTIONS:
        value = getattr(importlib.import_module(".binding", __name__), name)
        globals()[name] = value  # looked up once
        return value
    raise AttributeError(name)
