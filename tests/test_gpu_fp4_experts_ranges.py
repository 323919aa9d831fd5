"""The 4-bit operators and the token movement over their ranges: rows past 2^31
bytes."""

import pytest
import torch

from routed_expert_ffn_gemm_gb300 import api, build

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _library():
    build.build()
    api._lib()
    yield
    assert api.moe_read_device_status() == api.OK


# ------------------------------------------------------------------ dispatch

@pytest.mark.parametrize("d,dtype", [(1 << 30, torch.bfloat16), ((1 << 30) + 8, torch.bfloat16), (1 << 29, torch.float32)])
def test_rows_past_32_bits_of_bytes(d, dtype):
    x = torch.zeros(1, d, dtype=dtype, device=DEV)
    x[0, ::4097] = torch.arange(1, -(-d // 4097) + 1, device=DEV).remainder(251).to(dtype)
    idx = torch.tensor([[2, 0]], dtype=torch.int32, device=DEV)
    r = api.dispatch(x, idx, 3)
    assert torch.equal(r.rows[0], x[0]) and torch.equal(r.rows[1], x[0])
    assert r.inv_row.tolist() == [[1, 0]]
    out = api.combine(r.rows, r.inv_row)
    assert torch.equal(out, x + x)
