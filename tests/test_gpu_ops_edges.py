"""The operators around the layer on the GPU where their kernels could go wrong
unseen: forms that only some shapes take, sums of any length, values far out,
and calls that the C interface allows but the binding does not make."""
import math

import pytest
import torch

import combine_router_gemm_softmax_b200 as M
from oracle import ops as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32
CODE = {BF16: M.MOE_DTYPE_BF16, F32: M.MOE_DTYPE_F32}


def stream():
    return torch.cuda.current_stream().cuda_stream


@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("off,bad", [([0, 40, 9000, 50], True), ([-5, 10, 20, 64], True), ([0, 50, 20, 64], True),
                                     ([0, 0, 10, 64], False), ([3, 20, 20, 60], False)])
def test_bias_gradient_alone_reports_bad_offsets(dt, off, bad):
    """The C interface's weight gradient without dw: the bias sums are the only kernel, and right (small integers,
    so exactly), or the status says that the offsets were not."""
    g = torch.Generator().manual_seed(1)
    dy = torch.randint(-3, 4, (64, 48), generator=g).to(dt).to(DEV)
    x = torch.zeros((64, 40), dtype=dt, device=DEV)
    o = torch.tensor(off, dtype=torch.int32, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    db = torch.full((3, 48), math.nan, device=DEV)
    cfg = M.MoeGemmConfig(rows=64, n=48, k=40, groups=3, dtype=CODE[dt])
    assert M.lib().moe_grouped_gemm_wgrad(cfg, dy.data_ptr(), o.data_ptr(), x.data_ptr(), None, db.data_ptr(),
                                          status.data_ptr(), stream()) == M.MOE_OK
    assert int(status.item()) == (M.MOE_STATUS_BAD_OFFSETS if bad else 0)
    if not bad:
        want = torch.stack([dy[a:b].float().sum(0) for _, (a, b) in R.groups(off)])
        assert torch.equal(db, want)
