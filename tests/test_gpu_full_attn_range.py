"""Attention over whole caches at the ends of what numbers its rows and queries may hold, and right
behind the calls that write its rows. Formulas and tolerances are those of test_gpu_full_attn.py;
where the inputs differ by powers of two alone, so do the outputs, bit for bit."""
import math

import pytest
import torch

import two_tier_sparse_gb300 as dsa
from test_gpu_full_attn import KV_SCALE, Case, cache_rows, check, config, i32

pytestmark = pytest.mark.gpu
FMTS = ["bf16", "e4m3", "mxfp4"]
TAU = 512 ** -0.5


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_device):
    from two_tier_sparse_gb300 import build
    build.build()
    dsa.load()
    torch.cuda.set_device(cuda_device)


@pytest.mark.parametrize("fmt", FMTS)
def test_rows_written_right_before(fmt):
    """Each step overwrites rows that the step before has read, with nothing between the calls."""
    B, n = 40, 700
    cfg = config(fmt)
    g = torch.Generator(device="cuda").manual_seed(1)
    width, dt = {"bf16": (512, torch.bfloat16), "e4m3": (512, torch.uint8), "mxfp4": (272, torch.uint8)}[fmt]
    cache = torch.zeros((B, 704, width), dtype=dt, device="cuda")
    slots = (704 * torch.arange(B, device="cuda")[:, None] + torch.arange(n, device="cuda")).view(-1).int()
    rows = [torch.randn((B * n, 512), generator=g, device="cuda").bfloat16() for _ in range(3)]
    q = torch.randn((B, 64, 512), generator=g, device="cuda").bfloat16()
    lens = i32([n] * B)
    ws = dsa.full_attn_workspace(cfg, B)

    def step(k, out, lse):
        dsa.kv_write(cfg, rows[k], slots, cache, ws)
        dsa.full_attn_decode(cfg, q, cache, lens, out, ws, lse=lse)
    want = []
    for k in range(3):
        out, lse = torch.empty_like(q), torch.empty((B, 64), device="cuda")
        step(k, out, lse)
        torch.cuda.synchronize()
        want.append((out, lse))
    assert not torch.equal(want[0][0], want[1][0])
    got = [(k % 3, torch.empty_like(q), torch.empty((B, 64), device="cuda")) for k in range(30)]
    for k, out, lse in got:
        step(k, out, lse)
    assert dsa.read_device_status(ws) == (0, 0)
    for k, out, lse in got:
        assert torch.equal(out, want[k][0]) and torch.equal(lse, want[k][1])
