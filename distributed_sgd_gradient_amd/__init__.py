"""MI355X-native Adasum gradient combiner.

The combine runs in the gfx950 HIP library ``libadasum.so`` (C ABI declared
in include/adasum.h); this package is its thin Python binding.  Importing it
loads the library and fails loudly when the library has not been built.
Next to the combine stand the layer operators that produce what it combines,
and what becomes of the combined gradient.
"""

from ._native import AdasumError, lib as _lib  # noqa: F401
from .combine import Combiner, combine, combine_cached, plain_sum, workspace_bytes  # noqa: F401
from .layers import (checkpoint_pack, checkpoint_unpack, embedding, embedding_grad, layer_norm,  # noqa: F401
                     layer_norm_grad, layer_norm_keep, layer_norm_keep_grad, linear_grad, relative_bias,
                     relative_bias_grad, rms_norm, rms_norm_grad, rms_norm_pack)
from .updates import orthogonalize  # noqa: F401

_lib()  # fail at import time when the HIP library is missing
