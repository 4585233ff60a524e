"""What the objectives' classes refuse of autograd, on the host."""
import pytest
import torch

import second_order_optimizer_amd as K
from second_order_optimizer_amd import objectives as Q


def test_dropout_refuses_out_where_a_gradient_is_wanted():
    """It would cut the graph, or leave the dropout out of it."""
    op = Q.Dropout(4, 8, dtype="f32", device="cpu")
    x, g = torch.zeros(4, 8), torch.zeros(4, 8, requires_grad=True)
    for kw in (dict(x=g), dict(x=x, residual=g)):
        for out in (torch.zeros(4, 8), g):
            with pytest.raises(K.KfacError) as e:
                op.run(seed=1, out=out, **kw)
            assert e.value.status == K.KFAC_ERR_ARG
            with torch.no_grad(), pytest.raises(K.KfacError) as e:
                op.run(seed=1, out=out, **kw)
            assert e.value.status == K.KFAC_ERR_UNSUPPORTED        # as far as a GPU is needed
