"""The objectives on the GPU beside their numbers: batches of nothing, workspaces, autograd and flags."""
import numpy as np
import pytest
import torch

from tests.test_gpu_objectives import DT, U, gpu, near

pytestmark = pytest.mark.gpu


@pytest.fixture()
def Q(gpu_lib):
    from second_order_optimizer_amd import objectives
    return objectives


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("vocab", [5, 513, 2052, 4104, 32768, 140003])
def test_no_rows_of_any_length(Q, vocab, dtype):
    """No rows: empty outputs; every pair's sequences are empty, and its loss at h = 0 counts."""
    x, f = torch.empty(0, vocab, dtype=DT[dtype], device="cuda"), torch.empty(0, device="cuda")
    lab = torch.empty(0, dtype=torch.int64, device="cuda")
    assert Q.TokenLogp(0, vocab, dtype).run(x, lab).shape == (0,)
    stats, logp, grad = Q.PolicyLoss(0, vocab, dtype).run(x, lab, f)
    assert stats.tolist() == [0, 0, 0, 0] and grad.shape == (0, vocab)
    op = Q.PreferenceLoss(0, 3, vocab, dtype)
    stats, seq, logp, grad = op.run(x, lab, torch.zeros(7, dtype=torch.int32, device="cuda"))
    near(stats, np.array([np.log(2), 0, 0, 1]), 4 * U)
    assert not seq.any() and logp.shape == (0,) and grad.shape == (0, vocab) and op.flags() == 0
