"""POET-X orthogonal-equivalence linear layer for AMD MI355X (gfx950).

`poetx` is the ctypes binding of the C-ABI library libpoetx.so (built in-tree
by build_lib.build()); `PoetxLayer` wraps one layer's device buffers. Around the
linears of a block: `add_rms_norm` and `add_layer_norm` with their backward passes,
`dropout`, `linear` and `MergedLinear` (products with a weight that is no longer
trained), `linear_cross_entropy` and its backward, `clip_grads`. Importing the
package fails if the library has not been built.
"""
from . import poetx  # noqa: F401  (loads libpoetx.so, raises if missing)
from .block_ops import (MergedLinear, add_layer_norm, add_layer_norm_backward,  # noqa: F401
                        add_rms_norm, add_rms_norm_backward, clip_grads, dropout,
                        dropout_backward, linear, linear_cross_entropy,
                        linear_cross_entropy_backward)
from .layer import PoetxLayer, build_many, param_grad_many  # noqa: F401

__all__ = ["poetx", "PoetxLayer", "build_many", "param_grad_many", "add_rms_norm",
           "add_rms_norm_backward", "add_layer_norm", "add_layer_norm_backward", "dropout",
           "dropout_backward", "linear_cross_entropy", "linear_cross_entropy_backward", "linear",
           "MergedLinear", "clip_grads"]
