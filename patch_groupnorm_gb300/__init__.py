"""libtileblend: GB300-native tile stitching, PatchGroupNorm and training norms.

The compute lives in the C-ABI shared library ``libtileblend.so`` (CUDA
kernels for sm_103a, declared in ``include/tileblend.h``); ``tileblend``
is its thin Python binding.  ``training`` has the layer norm and PatchGroupNorm
as autograd functions.  ``synth`` draws seeded synthetic inputs.
"""
__all__ = ["tileblend", "synth", "training"]
