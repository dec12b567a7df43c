"""What the residual norm's binding refuses instead of leaving it unwritten."""
from __future__ import annotations

import pytest
import torch

from int8_quantized_02_b200 import llmint8 as L

pytestmark = pytest.mark.gpu


def test_a_y_without_a_norm():
    x = torch.randn((4, 64), device="cuda").half()
    y = torch.full_like(x, 7.0)
    with pytest.raises(ValueError, match="no Y"):
        L.llmint8_residual_norm(x, norm=None, Y=y)
    H, Y = L.llmint8_residual_norm(x, norm=None)
    assert Y is None and torch.equal(H, x) and (y == 7).all()
    with pytest.raises(L.LLMInt8Error):                 # nor an MXFP4 form of it
        L.llmint8_residual_norm_mxfp4(x, norm=None)
