"""B200-native (sm_100a) fused causal attention, forward and backward, and the operators
around it.

The library is a C ABI (include/) over hand-written CUDA kernels (csrc/).  ``_lib`` binds
the ABI under its own names; ``attention``, ``qkv`` (from the projection to the attention),
``grouped`` (linear products grouped by expert) and ``grads`` (gradient norm and clipping)
add torch-tensor front ends; ``workloads`` holds the benchmark shapes and seeded inputs.
Importing this package does not load the CUDA library; the first call does, and fails
loudly if it is missing.
"""
from . import workloads  # noqa: F401
from ._lib import ForgeAttnError, library_path, load  # noqa: F401
from .attention import (attn_bwd, attn_fwd, check_device_error, to_fp16,  # noqa: F401
                        workspace_bytes)
from .grads import grad_clip, grad_norm, grad_workspace_bytes  # noqa: F401
from .grouped import (linear_grouped_bwd_dw, linear_grouped_bwd_dx,  # noqa: F401
                      linear_grouped_fwd)
from .qkv import qkv_bwd, qkv_fwd, qkv_workspace_bytes  # noqa: F401
