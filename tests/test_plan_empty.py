"""A step plan of no matrices, with and without 4-bit forms: nothing to do, as for muon_step."""
import pytest

import newton_schulz_12_b200 as nsb


@pytest.mark.parametrize("forms", [False, True])
def test_no_matrices(forms):
    plan = nsb.MuonStepPlan([], [], [], mx_forms=forms)
    assert plan.mx_forms == ([] if forms else None)
    plan(stream=0)
