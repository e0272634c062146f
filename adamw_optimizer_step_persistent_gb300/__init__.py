"""Fused Adam/AdamW over one data-parallel rank's optimizer shard, and the
training operators that produce its gradients, for GB300.

The work happens in ``_build/libfadam.so`` (hand-written sm_103a kernels and
a C ABI declared in ``include/fadam.h`` and ``include/fadam_ops.h``); this
package is its thin Python binding.  Importing the package does not load the
library; the first call that needs it does, and fails loudly when it has not
been built.
"""
from ._abi import FadamError, lib  # noqa: F401
from .optimizer import FusedAdamShard, dtype_code, step_once  # noqa: F401
from .training import (BlockNorm, BlockNormGrads, Checkpoint8,  # noqa: F401
                       LinearCrossEntropy, block_norm, block_norm_backward, checkpoint8,
                       checkpoint8_restore, checkpoint8_weight_grad, linear_cross_entropy,
                       ops_status)

__all__ = ["FusedAdamShard", "FadamError", "step_once", "dtype_code", "lib",
           "linear_cross_entropy", "LinearCrossEntropy", "block_norm", "block_norm_backward",
           "BlockNorm", "BlockNormGrads", "checkpoint8", "checkpoint8_restore",
           "checkpoint8_weight_grad", "Checkpoint8", "ops_status"]
