"""GB300 (sm_103a) persistent serial Markov draft walk, and the operators that
check its drafts against the target model's cache.

The CUDA library (``_build/libdspark_walk.so``) is the product; ``walk`` and
``tree`` are thin ctypes bindings of its C ABIs (``include/dspark_walk.h``,
``include/dspark_tree.h``).
"""
from . import tree, walk  # noqa: F401
from .tree import KVCache, Tree  # noqa: F401
from .walk import Walk, WalkError  # noqa: F401
