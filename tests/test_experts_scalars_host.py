"""Scalar arguments beyond 32 bits are refused by the binding, where their lowest 32 bits would be
sizes that the library takes."""

import pytest

import w4a16_gemm_amd as w4
from test_experts_host import _good


@pytest.mark.parametrize("wrong", [2 ** 32 + 2, -2 ** 32 + 2, 2 ** 31, 2 ** 40 + 1])
@pytest.mark.parametrize("name,key", [("w4a16_route", "top_k"), ("w4a16_head_loss", "vocab"),
                                      ("w4a16_head_loss_backward", "vocab"), ("w4a16_experts_backward", "K"),
                                      ("w4a16_gemm_backward", "K"), ("w4a16_experts_gemm", "group_size"),
                                      ("w4a16_head_loss", "group_size")])
def test_binding_refuses_scalars_beyond_32_bits(name, key, wrong):
    with pytest.raises(ValueError):
        getattr(w4, name)(**dict(_good(name), **{key: wrong}))
