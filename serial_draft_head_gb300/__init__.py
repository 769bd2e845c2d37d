"""GB300 (sm_103a) persistent serial Markov draft walk, and the operators that
check its drafts against the target model's cache.

The CUDA library (``_build/libdspark_walk.so``) is the product; ``walk``, ``tree``
and ``pages`` are thin ctypes bindings of its C ABIs (``include/dspark_walk.h``,
``include/dspark_tree.h``, ``include/dspark_pages.h``).
"""
from . import pages, tree, walk  # noqa: F401
from .pages import Pages  # noqa: F401
from .tree import KVCache, Rotation, Tree  # noqa: F401
from .walk import Walk, WalkError  # noqa: F401
