"""MPQ row-batched post-training-quantisation solver for B200 (sm_100a).

The solver itself is libmpq.so (CUDA kernels behind a C ABI declared in
include/mpq.h); this package only binds it.  Importing the package loads the
library and raises ImportError if it has not been built.
"""
from ._lib import (Gram, MPQError, Plan, idx_to_numpy, kernel_launch_count, lib,  # noqa: F401
                   profile_start, profile_stop, rht)
from .layers import (layer_norm, layer_norm_backward, linear, linear_backward,  # noqa: F401
                     ops_status, token_logprobs, topk_distill)

__all__ = ["Plan", "Gram", "rht", "MPQError", "idx_to_numpy", "kernel_launch_count", "lib",
           "profile_start", "profile_stop", "linear", "linear_backward", "layer_norm",
           "layer_norm_backward", "token_logprobs", "topk_distill", "ops_status"]
