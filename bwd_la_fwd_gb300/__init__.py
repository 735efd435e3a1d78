"""GB300-native (sm_103a) normalised linear attention: forward and backward of one LA head batch,
and the operators of a recurrent layer around it.

The compute lives in ``csrc/`` (hand-written CUDA, C ABI in ``include/la.h``); ``la.py`` is a thin
ctypes binding over that ABI.  The library is loaded on first use and a missing or stale build raises
an error: there is no CPU fallback.
"""
from .la import (LA_BF16, LA_F32, DecodeState, LAError, RotaryFrequencies, la_backward, la_decode_step,
                 la_decode_step_grouped, la_forward, la_gated_scan, la_gated_scan_backward, la_gated_scan_step,
                 la_get_status, la_launch_count, la_prompt, la_prompt_workspace_bytes, la_rotary, la_rotary_backward,
                 la_rotary_frequencies, la_state_append, la_status_string, la_workspace_bytes, library_path, load_library,
                 new_prompt_workspace, new_workspace)

__all__ = ["LA_BF16", "LA_F32", "DecodeState", "LAError", "RotaryFrequencies", "la_backward", "la_decode_step",
           "la_decode_step_grouped", "la_forward", "la_gated_scan", "la_gated_scan_backward", "la_gated_scan_step",
           "la_get_status", "la_launch_count", "la_prompt", "la_prompt_workspace_bytes", "la_rotary", "la_rotary_backward",
           "la_rotary_frequencies", "la_state_append", "la_status_string", "la_workspace_bytes", "library_path",
           "load_library", "new_prompt_workspace", "new_workspace"]
