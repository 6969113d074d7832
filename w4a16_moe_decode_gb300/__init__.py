"""GB300-native (sm_103a) small-batch decode step of a Flint-style MoE FFN
layer with weight-only NVFP4 (W4A16) weights and BF16 activations, and what
fine-tuning needs beside the frozen weights: low-rank adapters of many requests
and the router's balance loss, with their gradients.

The computation lives in libflint_moe.so (C ABI: the headers in include/);
``binding`` exposes its entry points under the same names.
"""
from . import binding  # noqa: F401
from .build import LIB, build  # noqa: F401
