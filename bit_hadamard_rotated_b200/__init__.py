"""Packed low-bit, Hadamard-rotated linears on B200 (sm_100a).

The compute lives in libhq.so (include/hq.h); this package is its Python
binding (``hq``; ``fp4`` for the 4-bit floating-point matrices, ``route`` for
the expert routing steps), the build script (``build``), the seeded synthetic
inputs (``synth``) and the multi-rank benchmark helpers (``dist``).
"""
from .hq import *  # noqa: F401,F403
from .fp4 import *  # noqa: F401,F403
from .route import *  # noqa: F401,F403
