"""Backward passes at values where a formula that is right in exact numbers can go wrong in fp32.

Bounds are those of test_gpu_backward.py (its head derives them) unless a test says what comes on top."""

import math

import pytest
import torch

import block_sparse_self_b200 as vsa
from test_gpu_backward import DEV, U, check, inputs, reference, window_mask

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _no_device_errors():
    yield
    vsa.device_status()


# --------------------------------------------------------------------------
# centered dQ
# --------------------------------------------------------------------------

@pytest.mark.parametrize("mode", ["list", "window"])
def test_center_of_a_vanishing_mass(mode):
    """Keys 1 and 2 hold the weight, key 4 has e^-86 of it and the rest nothing: the columns that the mean key is
    weighted by (every fourth) have a mass of 16 e^-86, and the row's sum of dX over it is past fp32."""
    S, D = 128, 64
    g0 = torch.Generator(device=DEV).manual_seed(41)
    q = torch.zeros(1, 1, S, D, device=DEV)
    k = torch.zeros(1, 1, S, D, device=DEV)
    q[..., 0] = 8.0
    k[0, 0, :, 0] = -200.0          # logits of -200 and, at keys 1, 2 and 4, 86, 86 and 0 (exact in bf16 and fp32)
    k[0, 0, 1:3, 0] = 86.0
    k[0, 0, 4, 0] = 0.0
    k[..., 1:] = torch.randn(1, 1, S, D - 1, generator=g0, device=DEV)
    v = 100 * torch.randn(1, 1, S, D, generator=g0, device=DEV)
    g = 1000 * torch.randn(1, 1, S, D, generator=g0, device=DEV)
    q, k, v, g = (x.bfloat16() for x in (q, k, v, g))
    if mode == "list":
        lists = (torch.zeros(1, 1, dtype=torch.int32, device=DEV), torch.ones(1, dtype=torch.int32, device=DEV))
        o, lse = vsa.block_sparse_attention(q, k, v, *lists, 128, return_lse=True)
        got = vsa.block_sparse_attention_backward(g, q, k, v, o, lse, *lists, 128, grad_dtype=torch.float32)
    else:
        o, lse = vsa.window_attention(q, k, v, S, return_lse=True)
        got = vsa.window_attention_backward(g, q, k, v, o, lse, S, grad_dtype=torch.float32)
    ref = reference(q[0, 0], k[0, 0], v[0, 0], g[0, 0], torch.ones(S, S, dtype=torch.bool, device=DEV))
    # the sums that the center is meant to take off do leave the range of fp32 when divided by that mass
    mass = 16 * math.exp(-86)
    assert (ref["e_dX"].sum(1) / mass).max() > torch.finfo(torch.float32).max
    check([x[0, 0] for x in got], ref)
