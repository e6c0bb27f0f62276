"""B200-native SVG-EAR sparse attention.

The operator runs entirely in libsvgear.so (hand-written CUDA for sm_100a,
C ABI in include/svgear.h); `svgear` is its ctypes binding, `block` an
attention block made of its operators and `synth` the seeded synthetic-input
generator.
"""
from . import block, svgear, synth  # noqa: F401

__all__ = ["block", "synth", "svgear"]
