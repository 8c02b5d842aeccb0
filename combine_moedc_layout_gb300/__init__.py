"""libmoedc: MoE expert-parallel layout, dispatch and combine on one GB300.

The compute runs in the CUDA library libmoedc.so (built by build.build());
this package holds its ctypes binding (moedc) and the seeded synthetic
workloads (synth).

Beside the layout, dispatch and combine it carries the language-model
operators around them: the top-k router (gate), the rows packed by expert
(sort, unsort), their gradients, and the experts' products with 4-bit weights
(matvec_int4).
"""
from .moedc import (BF16, FP8_E4M3, SCALES_COL_MAJOR, SCALES_PER_TOKEN, Layout, MoedcError, alloc_recv, combine,
                    combine_e4m3, dequant_e4m3, moedc_combine_e4m3,
                    dispatch, layout, layout_dispatch, layout_workspace, load, moedc_combine,
                    moedc_dequant_e4m3, moedc_dispatch, moedc_layout, moedc_layout_dispatch,
                    moedc_layout_static_scratch, moedc_layout_workspace_bytes,
                    moedc_layout_dispatch_workspace_bytes, layout_dispatch_workspace,
                    moedc_rank_combine, moedc_rank_dispatch, moedc_rank_layout, rank_combine,
                    rank_dispatch, rank_layout, strerror)
from .moedc import (F16, F32, GATE_BIAS_SCORE, GATE_NORMALIZE, GATE_SIGMOID, GATE_SOFTMAX, SWIGLU, Sorted, gate,
                    gate_grad, matvec_int4, moedc_gate, moedc_gate_grad, moedc_matvec_int4,
                    moedc_matvec_int4_workspace_bytes, moedc_sort, moedc_sort_rows, moedc_sort_workspace_bytes, moedc_unsort,
                    moedc_unsort_grad, sort, sort_grad, unsort, unsort_grad)

__all__ = ["BF16", "FP8_E4M3", "SCALES_COL_MAJOR", "SCALES_PER_TOKEN", "Layout", "MoedcError", "alloc_recv",
           "combine", "combine_e4m3", "dequant_e4m3", "moedc_combine_e4m3",
           "dispatch", "layout", "layout_dispatch", "layout_workspace", "load", "moedc_combine",
           "moedc_dequant_e4m3", "moedc_dispatch", "moedc_layout", "moedc_layout_dispatch",
           "moedc_layout_static_scratch", "moedc_layout_workspace_bytes",
           "moedc_layout_dispatch_workspace_bytes", "layout_dispatch_workspace", "moedc_rank_combine",
           "moedc_rank_dispatch", "moedc_rank_layout", "rank_combine", "rank_dispatch",
           "rank_layout", "strerror",
           "F16", "F32", "GATE_BIAS_SCORE", "GATE_NORMALIZE", "GATE_SIGMOID", "GATE_SOFTMAX", "SWIGLU",
           "Sorted", "gate", "gate_grad", "matvec_int4", "moedc_gate", "moedc_gate_grad",
           "moedc_matvec_int4", "moedc_matvec_int4_workspace_bytes", "moedc_sort", "moedc_sort_rows",
           "moedc_sort_workspace_bytes", "moedc_unsort", "moedc_unsort_grad", "sort", "sort_grad",
           "unsort", "unsort_grad"]
