"""GB300-native BEV pooling (depth-weighted scatter-reduce) and temporal
attention over BEV tokens.

The compute path is the C-ABI library ``libbevpool.so`` (hand-written CUDA
for sm_103a, declared in ``include/bevpool.h``).  ``bevpool`` is its thin
ctypes binding, ``attention`` that of the token operators (head norms with
rotary positions, paged key/value cache, attention over it); ``workloads``
draws seeded synthetic inputs.  Importing this package loads nothing;
importing ``bevpool`` or ``attention`` loads the library and raises if it has
not been built.
"""
__all__ = ["attention", "bevpool", "workloads"]
