"""Tensors of too few dimensions are refused as those of wrong shapes are."""
import pytest
import torch

import two_tier_sparse_gb300 as dsa
from two_tier_sparse_gb300 import build as dsa_build

BF, I32 = torch.bfloat16, torch.int32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    dsa_build.build()
    dsa.load()


@pytest.mark.parametrize("shape", [(), (2,), (2, 64), (2, 64, 512, 1, 1)])
def test_queries(shape):
    cfg, ws = dsa.config(), torch.zeros(256, dtype=torch.uint8)
    lat, n = torch.zeros((2, 64, 512), dtype=BF), torch.zeros((2,), dtype=I32)
    q, out = torch.zeros(shape, dtype=BF), torch.zeros(shape, dtype=BF)
    with pytest.raises(ValueError):
        dsa.full_attn_decode(cfg, q, lat, n, out, ws)
    with pytest.raises(ValueError):
        dsa.full_attn_multi(cfg, n, q, lat, out, ws)


@pytest.mark.parametrize("shape", [(), (512,), (64, 512), (1, 2, 64, 512)])
def test_caches(shape):
    cfg, ws = dsa.config(), torch.zeros(256, dtype=torch.uint8)
    n, q = torch.zeros((2,), dtype=I32), torch.zeros((2, 64, 512), dtype=BF)
    with pytest.raises(ValueError):
        dsa.full_attn_decode(cfg, q, torch.zeros(shape, dtype=BF), n, torch.zeros_like(q), ws)
    with pytest.raises(ValueError):
        dsa.full_attn_decode(cfg, q, torch.zeros((2, 64, 512), dtype=BF), n, torch.zeros_like(q), ws,
                             swa=torch.zeros(shape, dtype=BF), swa_len=n)


@pytest.mark.parametrize("shape", [(), (4,), (2, 0), (2, 4, 1)])
def test_random_numbers(shape):
    ws = torch.zeros(256, dtype=torch.uint8)
    n, x = torch.zeros((2,), dtype=I32), torch.zeros((2, 3), dtype=I32)
    with pytest.raises(ValueError):
        dsa.verify_drafts(torch.zeros((2, 4, 50)), x, torch.zeros(shape), torch.zeros((2, 4), dtype=I32), n, ws)


@pytest.mark.parametrize("shape", [(), (50,), (4, 50)])
def test_probabilities(shape):
    ws = torch.zeros(256, dtype=torch.uint8)
    n, x = torch.zeros((2,), dtype=I32), torch.zeros((2, 3), dtype=I32)
    u, tok = torch.zeros((2, 4)), torch.zeros((2, 4), dtype=I32)
    with pytest.raises(ValueError):
        dsa.verify_drafts(torch.zeros(shape), x, u, tok, n, ws)
    with pytest.raises(ValueError):
        dsa.verify_drafts(torch.zeros((2, 4, 50)), x, u, tok, n, ws, draft=torch.zeros(shape))
