"""The package's public names: everything that the binding offers is imported and
listed, and nothing is listed that is not there."""
import types

import combine_moedc_layout_gb300 as package
from combine_moedc_layout_gb300 import moedc


def test_all_names_exist_and_star_import_takes_them():
    assert len(set(package.__all__)) == len(package.__all__)
    into = {}
    exec("from combine_moedc_layout_gb300 import *", into)
    for name in package.__all__:
        assert into[name] is getattr(moedc, name)


def test_every_import_is_listed():
    ours = {n for n, v in vars(package).items()
            if not n.startswith("_") and not isinstance(v, types.ModuleType)}
    assert ours == set(package.__all__)


def test_the_operators_are_public():
    for name in ("gate", "gate_grad", "sort", "sort_grad", "unsort", "unsort_grad", "matvec_int4",
                 "Sorted", "GATE_SOFTMAX", "GATE_SIGMOID", "GATE_NORMALIZE", "GATE_BIAS_SCORE",
                 "SWIGLU", "F16", "F32", "moedc_gate", "moedc_gate_grad", "moedc_sort",
                 "moedc_sort_rows", "moedc_sort_workspace_bytes", "moedc_unsort",
                 "moedc_unsort_grad", "moedc_matvec_int4", "moedc_matvec_int4_workspace_bytes"):
        assert name in package.__all__, name
