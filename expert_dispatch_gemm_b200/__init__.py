"""B200-native MoE routing-and-dispatch layer (sm_100a).

The compute lives in ``libmoe.so`` (hand-written CUDA behind a C ABI, see
``include/moe.h``); ``expert_dispatch_gemm_b200.moe`` is the thin ctypes
binding over torch-allocated device memory. The operators of the block around
the layer (``include/moe_block.h``, ``libmoe_block.so``) are bound in
``expert_dispatch_gemm_b200.block``. Importing this package does not load the
libraries; the bindings load them on first use and raise if one is missing.
"""
__all__ = ["block", "moe", "workloads"]
