"""B200-native coarse-to-fine key retrieval for top-k sparse attention at decode time.

HHR (Geometry-Aware Key Routing page bounds + Learned Hash Projection Hamming
ranking) and the HISA indexer variant (block filter + token refinement), with an
8-bit K/V cache, dense paged attention and block-sparse attention beside them, as
hand-written sm_100a CUDA kernels behind the C ABI in include/hhr.h.
"""
from . import hhr  # noqa: F401
from .hhr import HHRError, make_dims  # noqa: F401
from .step import BlockStep, DecodeStep, DenseStep, KV8Cache, LayerCache  # noqa: F401
