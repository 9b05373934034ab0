"""vidattn: the attention path of video diffusion transformers as hand-written
sm_100a CUDA behind a C ABI: multi-head attention (segment ids, causal, 3D
windows) with its backward pass, the layer norm and the 3D rotary embedding
ahead of it with theirs.  ``autograd`` has them as differentiable functions.

The Python layer only marshals arguments to the shared library
``csrc/libvidattn.so``; every step of the computation runs in its kernels.
"""
from .binding import (  # noqa: F401
    VIDATTN_OK, status_string, vidattn_fwd, vidattn_fwd_host, attention, attention_bwd,
    layer_norm, layer_norm_bwd, rope3d, rope3d_scaled, rope3d_scaled_bwd, library_path,
    load_library, exported_symbols,
)
