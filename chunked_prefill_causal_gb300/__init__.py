"""GB300 (sm_103a) chunked-prefill causal attention.

The compute path is the C-ABI library ``libvpp.so`` (hand-written CUDA for
sm_103a, declared in ``include/vpp.h``); ``chunked_prefill_causal_gb300.vpp``
is its thin binding (ctypes; the serving-step calls, a few microseconds of GPU
time each, go through a small compiled module, ``csrc/pycall.cpp``).  There is no CPU fallback: every binding call
raises if the library or a CUDA device is missing.
"""

__all__ = ["vpp", "workloads"]
