"""GPU runs of calls of qg_attention that a server makes: tables cut from wider ones, malformed offsets, mixed batches.

Bars and cases are those of test_gpu_attention.
"""
import numpy as np
import pytest
import torch

import quantized_gemm_amd as qg
from test_gpu_attention import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    qg.lib()
    yield


@pytest.mark.parametrize("counts", [None, [20, 90, 31]])
def test_a_table_cut_from_a_wider_one(counts):
    c = Case([100, 700, 31], 8, 2, 128, 16, counts=counts)
    table = c.table
    wide = torch.full((5, table.shape[1] + 9), 1 << 30, dtype=torch.int32, device="cuda")   # pages outside the cache
    c.table = wide[1:4, 3:3 + table.shape[1]]
    c.table.copy_(table)
    c.run().check()
    c.table = torch.cat([table, torch.full_like(table, -1)], 0)[:3]
    c.run().check()
