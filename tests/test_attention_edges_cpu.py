"""Refusals of the attention functions at the ends of their ranges, without a GPU."""
import pytest
import torch

from normalization_rmsnorm_fwd_gb300 import _abi
from normalization_rmsnorm_fwd_gb300 import build as nbuild
from test_attention_cpu import paged, prompt
from test_qk_rope_cpu import ARG, CUDA


@pytest.fixture(scope="module")
def L():
    if torch.cuda.is_available():
        pytest.skip("fake device addresses: only where no GPU could follow them")
    nbuild.build()
    return _abi.load()


@pytest.mark.parametrize("f", [prompt, paged])
def test_scales_whose_binary_form_leaves_fp32(L, f):
    # The kernels hold scale * log2(e).  Scores of 0 times infinity would be NaN, masked places times 0 too.
    assert f(L, scale=2.3e38) == CUDA and f(L, scale=2.4e38) == ARG and f(L, scale=3.4e38) == ARG
    assert f(L, scale=1e-45) == CUDA and f(L, scale=1e-38) == CUDA
