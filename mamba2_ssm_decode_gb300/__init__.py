"""GB300 (sm_103a) Mamba2 selective-state-update decode.

The C ABI lives in include/ssu.h and libssu_gb300.so (built in-tree by
``mamba2_ssm_decode_gb300.build``); this package binds it for CUDA torch
tensors:

  ssu_update         one-token decode step
  ssu_update_varlen  packed variable-length / speculative (MTP) step
  ssu_replay_update  ReplaySSM checkpointing update (ring caches, trackers)
  ssu_replay_update_static  the same for callers that cannot pass scratch memory
  ssd_combined_fwd_varlen  packed variable-length SSD prefill (chunk states)
  ssu_ring_update    ReplaySSM ring-tracker update or reset
  ssu_ring_commit    ReplaySSM ring-tracker commit of the previous window
  conv_update, conv_update_varlen, conv_fwd_varlen  the causal convolution in front of
                     the state update: one token, drafted tokens, packed prompts
  scan_update, scan_update_varlen, scan_fwd_varlen  the selective scan whose A varies
                     along dstate: one token, drafted tokens, packed prompts
  linattn_update, linattn_update_varlen, linattn_fwd_varlen  linear attention with a decay
                     for each head: one token, drafted tokens, packed prompts
  drafts_verify      drafted tokens against the target's probabilities
  prompt_maps        starts, chunks and row maps of a batch, from its lengths
  slots_copy, slots_clear, slots_compact  fork, zero and close up the slots of all pools
  slots_assign       fill slot tables with the lowest free slots
  ssu_device_error   the device error word of the bounded waits (diagnostic)
  ssu_selftest_bounded_wait  proves on the device that a bounded wait gives up
"""
from .api import (ssd_combined_fwd_varlen, ssd_workspace_bytes, ssu_device_error,
                  ssu_replay_update, ssu_replay_update_static,
                  ssu_ring_commit, ssu_ring_update, ssu_selftest_bounded_wait, ssu_update,
                  ssu_update_varlen)
from .layer_api import (PromptMaps, conv_fwd_varlen, conv_update, conv_update_varlen,
                        drafts_verify, linattn_fwd_varlen, linattn_update, linattn_update_varlen,
                        linattn_workspace_bytes, prompt_maps, scan_fwd_varlen, scan_update,
                        scan_update_varlen, slots_assign, slots_clear, slots_compact,
                        slots_compact_workspace_bytes, slots_copy)

__all__ = ["ssu_update", "ssu_update_varlen", "ssu_replay_update", "ssu_replay_update_static",
           "ssu_ring_update", "ssu_ring_commit", "ssd_combined_fwd_varlen", "ssd_workspace_bytes",
           "conv_update", "conv_update_varlen", "conv_fwd_varlen", "scan_update",
           "scan_update_varlen", "scan_fwd_varlen", "linattn_update", "linattn_update_varlen",
           "linattn_fwd_varlen", "linattn_workspace_bytes", "drafts_verify", "prompt_maps",
           "PromptMaps", "slots_assign", "slots_copy", "slots_clear", "slots_compact",
           "slots_compact_workspace_bytes", "ssu_device_error", "ssu_selftest_bounded_wait"]
