"""GB300 (sm_103a) Sparse Delta Memory forward hot path.

The compute lives in ``libsdm.so`` (CUDA C++, C ABI declared in include/sdm.h);
``api`` is a thin ctypes binding for torch tensors, ``layers`` has the layers beside
the memory (convolution, selective scan, linear attention, gated projections, norms and
projections with their gates and residuals), and ``workloads`` defines
the seeded synthetic configurations.  Importing the package does not load the
library; the first API call does (and fails loudly if it cannot).
"""
from .api import (BWD_DM0_ONLY, BWD_FINAL_ZERO, SELECT_AUTO, SELECT_COUNTING, SELECT_GENERAL, SDM_BF16, SDM_DEV_DUP_WRITE, SDM_DEV_INDEX_RANGE, SDM_DEV_TIMEOUT, SDM_F32, DecodeStep, SDMError,
                  backward_workspace_size, bounded_wait_check, copy_token_window, decode_step, decode_table, fill_state, forward,
                  forward_chunks, forward_workspace, scan_backward, scan_forward_train, select_backward,
                  gen_inputs, gen_M0, init_state_from_M0, lib, library_path, pinned_empty, project_kq, project_select, project_select_workspace,
                  project_stall_check, scan_forward,
                  scan_forward_noalloc, NOALLOC_SCRATCH_BYTES, scan_launch_info, scan_workspace, scan_workspace_size, select, side_stream)

from .layers import (causal_conv, causal_conv_step, gated_norm, gated_norm_backward, linear_attention,
                     linear_attention_step, linear_attention_workspace_size, project, project_backward,
                     project_backward_workspace_size, project_gated, project_gated_backward,
                     project_gated_backward_workspace_size, project_workspace_size, residual_norm,
                     residual_norm_backward, residual_norm_backward_workspace_size, selective_scan,
                     selective_scan_workspace_size, selective_step)

__all__ = ["gated_norm", "gated_norm_backward", "linear_attention", "linear_attention_step",
           "linear_attention_workspace_size", "project", "project_backward", "project_backward_workspace_size",
           "project_workspace_size", "residual_norm", "residual_norm_backward", "residual_norm_backward_workspace_size",
           "causal_conv", "causal_conv_step", "project_gated", "project_gated_backward",
           "project_gated_backward_workspace_size", "selective_scan", "selective_scan_workspace_size", "selective_step",
           "BWD_DM0_ONLY", "BWD_FINAL_ZERO", "SELECT_AUTO", "SELECT_COUNTING", "SELECT_GENERAL", "SDM_BF16", "SDM_DEV_DUP_WRITE", "SDM_DEV_INDEX_RANGE", "SDM_DEV_TIMEOUT", "SDM_F32", "DecodeStep", "SDMError",
           "backward_workspace_size", "bounded_wait_check", "copy_token_window", "decode_step", "decode_table", "fill_state", "forward",
           "forward_chunks", "forward_workspace", "scan_backward", "scan_forward_train", "select_backward",
           "gen_inputs", "gen_M0", "init_state_from_M0", "lib", "library_path", "pinned_empty", "project_kq", "project_select", "project_select_workspace",
           "project_stall_check", "scan_forward",
           "scan_forward_noalloc", "NOALLOC_SCRATCH_BYTES", "scan_launch_info", "scan_workspace", "scan_workspace_size", "select", "side_stream"]
