"""B200-native (sm_100a) IndexCache decode hot path.

The compute lives in ``libindexcache.so`` (C ABI, ``include/indexcache.h``):
lightning indexer, top-k, sparse MLA decode with sink and gate, the F/S
layer-stack driver, and the paged latent cache (rotation, append, read-back,
dense and sparse attention; ``_front.so`` checks their tensors in C++). ``_abi`` binds it with ctypes under the same names;
``ops`` is a thin torch-tensor front end. ``workloads`` draws the seeded
synthetic inputs. Importing ``_abi``/``ops`` fails if the library has not
been built; there is no fallback implementation.
"""
__all__ = ["workloads", "ops", "_abi", "build"]
