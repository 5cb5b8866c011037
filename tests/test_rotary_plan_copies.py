"""A rotary plan is kept by a model, which is copied (an average of weights) and pickled (checkpoints, worker processes)."""
import copy
import pickle

import pytest
import torch

import ulysses_dit_attention_gb300 as uaa

COPIES = [copy.copy, copy.deepcopy, lambda x: pickle.loads(pickle.dumps(x))]


@pytest.mark.parametrize("how", COPIES)
def test_a_copy_is_the_same_plan(how):
    plan = uaa.RotaryPlan([44, 42, 42], layout="interleaved", scaling="parts", factor=4.0)
    model = how(torch.nn.Module())
    model.plan = plan
    twin = how(model).plan
    assert bytes(twin._c) == bytes(plan._c)
    assert (twin.axes, twin.rot, twin.magnitude, twin.turns) == (plan.axes, plan.rot, plan.magnitude, plan.turns)


@pytest.mark.gpu
@pytest.mark.parametrize("how", COPIES)
def test_a_copy_rotates_alike(how):
    plan = uaa.RotaryPlan([64], scaling="linear", factor=2.0)
    q = torch.randn(2, 9, 3, 64, device="cuda").bfloat16()
    want, twin = uaa.rotary_fwd(q, None, plan, start=5)[0], how(plan)
    del plan
    assert torch.equal(uaa.rotary_fwd(q, None, twin, start=5)[0], want)
