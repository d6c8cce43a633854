"""GB300-native causal depthwise conv1d forward: varlen prefill with conv_state,
decode update (with the speculative-decoding extras), and the paged
sliding-window short conv; and the operators of the linear-attention layer
around it: the gated delta rule (prefill and decode), its gated norm, the
residual norm between blocks, and the verification of drafted tokens.

The compute path is the hand-written CUDA library ``libccv.so`` (C ABI in
``include/ccv.h`` and ``include/ccv_layer.h``); :mod:`.api` and :mod:`.layer`
are thin ctypes bindings over it with the same entry-point names.  Nothing here computes on the CPU: the binding rejects CPU
tensors and raises if the library has not been built.
"""
from .api import (PAD_SLOT_ID, Launch, ccv_fwd, ccv_update, ccv_update_spec,  # noqa: F401
                  paged_sconv_fwd, paged_sconv_fwd_streams, paged_sconv_fwd_with_metadata,
                  paged_sconv_seq_metadata, prepare_ccv_fwd, prepare_ccv_update,
                  prepare_ccv_update_spec, prepare_paged_sconv_fwd,
                  prepare_paged_sconv_fwd_streams, prepare_paged_sconv_fwd_with_metadata,
                  prepare_paged_sconv_seq_metadata)
from .layer import (gated_rms_norm, gdr_fwd, gdr_update, prepare_gated_rms_norm,  # noqa: F401
                    prepare_gdr_fwd, prepare_gdr_update, prepare_residual_rms_norm,
                    prepare_spec_verify, residual_rms_norm, spec_verify)
from ._lib import CcvError  # noqa: F401

__all__ = ["PAD_SLOT_ID", "ccv_fwd", "ccv_update", "ccv_update_spec", "paged_sconv_seq_metadata",
           "paged_sconv_fwd", "paged_sconv_fwd_with_metadata", "paged_sconv_fwd_streams",
           "prepare_paged_sconv_fwd_with_metadata", "prepare_paged_sconv_fwd_streams",
           "prepare_ccv_fwd", "prepare_ccv_update", "prepare_ccv_update_spec",
           "prepare_paged_sconv_seq_metadata", "prepare_paged_sconv_fwd", "Launch",
           "CcvError", "gdr_fwd", "gdr_update", "gated_rms_norm", "residual_rms_norm", "spec_verify",
           "prepare_gdr_fwd", "prepare_gdr_update", "prepare_gated_rms_norm",
           "prepare_residual_rms_norm", "prepare_spec_verify"]
