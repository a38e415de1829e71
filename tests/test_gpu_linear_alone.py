"""bitlinear_linear of one matrix whose rows take just under 48 KB of dynamic shared memory a CTA, so that
dynamic and static shared memory together need the opt-in (the README's example has such a shape)."""
import numpy as np
import pytest
import torch

import bitlinear_w1_a8_gb300 as bl
import oracle
from bitlinear_w1_a8_gb300 import synth
from harness import Y_RTOL, max_rel_err

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N,K", [(10240, 2560), (9728, 2560), (8192, 2816), (10944, 2560)])
def test_one_token_one_matrix(N, K):
    W, x = synth.weight(N, K, 5), synth.activations(1, K, 6)
    Wq, sw_o, _ = oracle.weight_quant(W.numpy())
    packed = torch.from_numpy(oracle.pack(Wq)).cuda()
    sw = torch.tensor([sw_o], device="cuda")
    xq, sx = torch.empty(1, K, dtype=torch.int8, device="cuda"), torch.empty(1, device="cuda")
    y, acc = torch.empty(1, N, device="cuda"), torch.empty(1, N, dtype=torch.int32, device="cuda")
    bl.bitlinear_linear(x.cuda(), [(packed, sw, y, acc)], xq, sx)
    assert bl.bitlinear_device_status() == 0
    xq_o, sx_o = oracle.act_quant(x.numpy())
    acc_o, y_o = oracle.forward(xq_o, sx_o, oracle.pack(Wq), sw_o, N, K)
    np.testing.assert_array_equal(acc.cpu().numpy(), acc_o)
    assert max_rel_err(y.cpu().numpy(), y_o) <= Y_RTOL
