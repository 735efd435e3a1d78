"""GB300-native (sm_103a) normalised linear attention: forward and backward of one LA head batch,
and the operators of a recurrent layer around it.

The compute lives in ``csrc/`` (hand-written CUDA, C ABI in ``include/la.h``); ``la.py`` is a thin
ctypes binding over that ABI.  The library is loaded on first use and a missing or stale build raises
an error: there is no CPU fallback.
"""
from .la import (DecodeState, LAError, LA_BF16, LA_F32, RotaryFrequencies, SelectiveScanGradients, la_backward,
                 la_decode_step, la_decode_step_grouped, la_forward, la_gated_scan, la_gated_scan_backward,
                 la_gated_scan_step, la_get_status, la_launch_count, la_prompt, la_prompt_workspace_bytes,
                 la_rms_norm, la_rms_norm_8bit, la_rms_norm_backward, la_rotary, la_rotary_backward,
                 la_rotary_frequencies, la_selective_scan, la_selective_scan_backward, la_selective_scan_step,
                 la_short_conv, la_short_conv_backward, la_short_conv_step, la_state_append, la_status_string,
                 la_workspace_bytes, library_path, load_library, new_prompt_workspace, new_rms_norm_workspace,
                 new_selective_scan_marks, new_selective_scan_workspace, new_short_conv_workspace, new_workspace)

__all__ = ["DecodeState", "LAError", "LA_BF16", "LA_F32", "RotaryFrequencies", "SelectiveScanGradients",
           "la_backward", "la_decode_step", "la_decode_step_grouped", "la_forward", "la_gated_scan",
           "la_gated_scan_backward", "la_gated_scan_step", "la_get_status", "la_launch_count", "la_prompt",
           "la_prompt_workspace_bytes", "la_rms_norm", "la_rms_norm_8bit", "la_rms_norm_backward", "la_rotary",
           "la_rotary_backward", "la_rotary_frequencies", "la_selective_scan", "la_selective_scan_backward",
           "la_selective_scan_step", "la_short_conv", "la_short_conv_backward", "la_short_conv_step",
           "la_state_append", "la_status_string", "la_workspace_bytes", "library_path", "load_library",
           "new_prompt_workspace", "new_rms_norm_workspace", "new_selective_scan_marks",
           "new_selective_scan_workspace", "new_short_conv_workspace", "new_workspace"]
