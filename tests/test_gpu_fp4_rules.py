"""The MXFP4 product on both sides of the rules that choose its kernel, against fp64."""
import pytest
import torch

from test_gpu_fp4 import test_gemm as check_gemm

pytestmark = pytest.mark.gpu


# 32 rows end the short K's few-row form, 64 the long one's; K 4064 and 4096 stand on both sides of long. N: K over 8, 4 and 2
# CTAs of a cluster, and whole.
@pytest.mark.parametrize("N,K", [(130, 4064), (130, 4096), (300, 96), (5000, 4128), (10000, 4128), (19000, 4128)])
def test_rows_on_both_sides(N, K):
    for M in (32, 33, 64, 65):
        check_gemm(M, N, K, torch.float32)
    check_gemm(40, N, K, torch.bfloat16)
