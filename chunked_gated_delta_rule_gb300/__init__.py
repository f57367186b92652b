"""GB300-native chunked gated-delta-rule forward and backward passes, the
paged cache and attention of the softmax layers beside them, and the operators
of state-space layers (short convolution, selective scan, norm).

The compute path is a C-ABI CUDA library (``include/gdr.h``, built in-tree
into ``_build/libgdr.so``); this package is its thin ctypes binding plus the
seeded synthetic input generator, and torch autograd functions over the
library's forward and backward entry points: ``chunk_gated_delta_rule``,
``short_conv``, ``selective_scan`` and ``rms_norm``.
There is no CPU fallback: every entry point raises if the CUDA library is
missing.
"""
from .api import (GdrError, LaunchTimer, gdr_chunk_fwd, gdr_chunk_fwd_host,  # noqa: F401
                  gdr_chunk_bwd, gdr_bwd_workspace_size,
                  gdr_chunk_fwd_noalloc, gdr_recurrent_fwd,
                  gdr_cache_write, gdr_cache_read, gdr_paged_attn, gdr_attn_workspace_size,
                  gdr_error_string, gdr_kernel_name, gdr_plan_query, gdr_release_cached,
                  gdr_version,
                  gdr_workspace_size, load_library)

from .layer import (gdr_short_conv_fwd, gdr_short_conv_bwd,  # noqa: F401
                    gdr_short_conv_bwd_workspace_size,
                    gdr_selective_scan_fwd, gdr_selective_scan_bwd,
                    gdr_selective_scan_workspace_size,
                    gdr_rms_norm_fwd, gdr_rms_norm_bwd, gdr_rms_norm_bwd_workspace_size)
from .autograd import (chunk_gated_delta_rule, rms_norm, selective_scan,  # noqa: F401,E402
                       short_conv)

# gdr_chunk_fwd_ex's options (scale, forced plan, workspace, status word) are
# keyword arguments of gdr_chunk_fwd in Python.
gdr_chunk_fwd_ex = gdr_chunk_fwd
