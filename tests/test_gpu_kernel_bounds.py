"""Sizes on both sides of the bounds where the policy loss and the distillation change their kernels."""
import pytest

import rollout_x128_act_gb300 as jq
import test_gpu_linear_distill as distill
import test_gpu_policy as policy

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("nseg", [255, 256, 257])
@pytest.mark.parametrize("n", [4096, 4097])
@pytest.mark.parametrize("by_seg,per_token", [(False, False), (True, False), (True, True)])
def test_policy_loss_by_one_block_or_by_several(n, nseg, by_seg, per_token):
    """One block takes 4096 tokens and 256 sequences."""
    rng, old, nll, ref, adv = policy.data(n, n if per_token else nseg, n + nseg)
    off = policy.offsets(n, nseg, rng, tail=11, front=3)
    policy.check(nll, old, adv, off, ref, rng.random(n) < 0.8, 0.02, 0.03, 1.05, 0.05, by_seg, "segs",
                 per_token=per_token)


@pytest.mark.parametrize("n", [64, 65, 384, 385, 2048, 2049])
@pytest.mark.parametrize("renorm", [True, False])
def test_distillation_of_few_and_many_rows(n, renorm):
    """Products of a row's entries by several blocks up to 384 rows, a block a row in the join up to 2048."""
    x, w, ids, t, dloss = distill._inputs(n, 700, 136, 37, n, pad=8)
    if not renorm:
        t = distill._logprobs(t, ids, 700)
    _, lse, logp = distill._check_fwd(x, w, ids, t, 0.8, renorm)
    distill._check_bwd(x, w, ids, t, lse, logp, dloss, 0.8, renorm)
    again = jq.linear_distill(x, w, ids, t, scale=0.8, renorm=renorm)
    assert (again[1] == lse).all() and (again[2] == logp).all()
