"""MI355X (gfx950) Gated DeltaNet chunked prefill.

``gdn`` holds the Python binding of the HIP library (``libgdn_mi355x.so``, built by
``python -m linear_attention_recurrence_prefill_amd.build``); the C ABI is ``include/gdn.h`` (and
``include/gdn_calib.h`` for the measurement kernels).  ``linattn`` holds linear attention with a
decay for each head (``include/gdn_linattn.h``) and ``pages`` the operators on a pool of states
(``include/gdn_pages.h``).
"""
from .gdn import (GdnError, calib_copy, calib_mfma_bf16, chunk_bwd, chunk_fwd, chunk_fwd_noalloc,
                  gdn_chunk_fwd_noalloc,
                  chunk_fwd_intermediates, chunk_fwd_plan, decode_step, device_faults,
                  gdn_calib_copy, gdn_calib_mfma_bf16, gdn_chunk_bwd, gdn_chunk_fwd,
                  gdn_chunk_fwd_intermediates, gdn_chunk_fwd_plan, gdn_decode_step,
                  gdn_device_faults, gdn_get_debug, gdn_set_debug, gdn_validate_cu_seqlens,
                  get_debug, load_library, set_debug, validate_cu_seqlens)
from .linattn import (gdn_linattn_bwd, gdn_linattn_bwd_workspace_size, gdn_linattn_fwd,
                      gdn_linattn_fwd_workspace_size, gdn_linattn_step, linattn_bwd, linattn_fwd,
                      linattn_step)
from .pages import (gdn_pages_compact, gdn_pages_copy, gdn_pages_fork, gdn_pages_free,
                    gdn_pages_workspace_size, pages_compact, pages_copy, pages_fork, pages_free)

__all__ = ["GdnError", "chunk_fwd", "chunk_fwd_noalloc", "gdn_chunk_fwd_noalloc", "chunk_bwd", "chunk_fwd_plan", "chunk_fwd_intermediates",
           "decode_step", "validate_cu_seqlens", "set_debug", "get_debug", "device_faults",
           "calib_copy", "calib_mfma_bf16", "load_library", "gdn_chunk_fwd",
           "gdn_chunk_fwd_plan", "gdn_chunk_fwd_intermediates", "gdn_chunk_bwd", "gdn_decode_step",
           "gdn_validate_cu_seqlens", "gdn_set_debug", "gdn_get_debug", "gdn_device_faults",
           "gdn_calib_copy", "gdn_calib_mfma_bf16", "linattn_fwd", "linattn_bwd", "linattn_step",
           "gdn_linattn_fwd", "gdn_linattn_bwd", "gdn_linattn_step",
           "gdn_linattn_fwd_workspace_size", "gdn_linattn_bwd_workspace_size", "pages_copy",
           "pages_fork", "pages_free", "pages_compact", "gdn_pages_copy", "gdn_pages_fork",
           "gdn_pages_free", "gdn_pages_compact", "gdn_pages_workspace_size"]
