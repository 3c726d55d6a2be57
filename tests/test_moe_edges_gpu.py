"""The operators of a layer of experts at their edges: waits that run out, memory of the right
stream, values near the ends of fp32, layouts inside one buffer."""
import numpy as np
import pytest
import torch

from w8a8_int8_quantized_norm_b200 import sq

import _moe_reference as ref

pytestmark = pytest.mark.gpu

TIMEOUT = 6  # SQ_ERR_PIPELINE_TIMEOUT


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    sq.lib()
    assert sq.get_device_error() == 0
    yield
    sq.set_wait_limit(0)
    assert sq.get_device_error() == 0


def _rng(*key):
    return np.random.default_rng([17, *key])


def _cuda_of(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


def _np64(t):
    return t.double().cpu().numpy()


# ---------------------------------------------------------------------------
# block norm: waits that run out
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("limit", [1, 2, 4])
@pytest.mark.parametrize("quant", [True, False])
@pytest.mark.parametrize("pre", [sq.NORM_NONE, sq.NORM_RMS])
@pytest.mark.parametrize("top_k", [0, 2])
def test_block_norm_wait_limit(top_k, pre, quant, limit):
    """A wait that runs out is an error status: its group starts no further copy and leaves, and
    the next call is right.  A limit of 1 allows no probe and always runs out; 2 and 4 allow one
    and three that do not sleep, so that groups give up at some later row, or not at all."""
    M, K = 6000, 2048  # ten rows or more for every group
    x = torch.randn((M * max(1, top_k), K), device="cuda").to(torch.bfloat16)
    res = torch.randn((M, K), device="cuda").to(torch.bfloat16)
    kw = dict(post_norm=sq.NORM_RMS, pre_norm=pre, quant=quant)
    if top_k:
        kw.update(token_row=torch.randperm(M * top_k, device="cuda").to(torch.int32).view(M, top_k),
                  weights=torch.rand((M, top_k), device="cuda"))
    want = sq.block_norm_quant_per_token(x, res, **kw)
    torch.cuda.synchronize()
    assert sq.get_device_error() == 0
    sq.set_wait_limit(limit)
    try:
        sq.block_norm_quant_per_token(x, res, **kw)
        status = sq.get_device_error()
    finally:
        sq.set_wait_limit(0)
    assert status == TIMEOUT if limit == 1 else status in (0, TIMEOUT)
    got = sq.block_norm_quant_per_token(x, res, **kw)
    assert sq.get_device_error() == 0
    for a, b in zip(got, want):
        assert (a is None and b is None) or torch.equal(a, b)
