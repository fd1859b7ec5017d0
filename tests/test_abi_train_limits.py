"""The sizes up to which the operators that train and score a model take a call (host checks
only): what include/qpack.h names is taken, one more is refused."""
from __future__ import annotations

import pytest
import torch

import weight_only_quantized_qgemv_amd as qp
from test_abi_model import INVALID, UNSUPPORTED, refused
from test_abi_train import loss, loss_backward, norm, norm_backward


def test_rows_of_the_norms():
    for d in (8, 16384):
        assert qp.qblock_norm_backward_workspace_bytes(1 << 22, d, 0) > 0
        assert qp.qblock_norm_backward_workspace_bytes((1 << 22) + 1, d, 0) == 0
    refused(norm(m=(1 << 22) + 1), INVALID)
    refused(norm_backward(m=(1 << 22) + 1), INVALID)
    refused(norm(d=16385), UNSUPPORTED)


@pytest.mark.parametrize("size", [qp.qcross_entropy_workspace_bytes, qp.qcross_entropy_backward_workspace_bytes])
def test_rows_and_features_of_the_loss(size):
    assert size(1 << 20, 64, 1000, 4, 64, torch.bfloat16) > 0
    assert size((1 << 20) + 1, 64, 1000, 4, 64, torch.bfloat16) == 0
    assert size(2, 1 << 24, 1000, 4, 64, torch.bfloat16) > 0
    assert size(2, (1 << 24) + 64, 1000, 4, 64, torch.bfloat16) == 0
    refused(loss(m=(1 << 20) + 1), INVALID)
    refused(loss_backward(k=(1 << 24) + 64), INVALID)
