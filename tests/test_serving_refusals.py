"""Arguments that the binding of the serving operators hands on to the library's checks (no GPU needed)."""
import pytest
import torch

import tensor_core_gemm_tcgen05_gb300 as g
from tensor_core_gemm_tcgen05_gb300 import _build


@pytest.fixture(scope="module", autouse=True)
def lib():
    _build.build()
    return g.lib()


@pytest.mark.parametrize("given", [False, True], ids=["allocated", "workspace"])
@pytest.mark.parametrize("scale", [None, 0.5])
def test_heads_without_dimensions(given, scale):
    """The default scale of head_dim 0 is no number: the library's refusal, not an arithmetic error."""
    q, cache = torch.zeros(1, 2, 0, dtype=torch.float16), torch.zeros(2, 1, 16, 0, dtype=torch.float16)
    ints = torch.zeros(2, dtype=torch.int32)
    ws = torch.zeros(256, dtype=torch.uint8) if given else None
    with pytest.raises(g.GemmError) as e:
        g.paged_attention(None, q, cache, cache, ints, ints[:1], ints[None, :1], scale=scale, workspace=ws, stream=0)
    assert e.value.status == g.GEMM_ERR_ARG
