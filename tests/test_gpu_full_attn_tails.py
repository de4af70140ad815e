"""Attention over whole caches where one row holds half of a head's weight and the rest lies in a
long tail of small probabilities, rows with a mean: what the tail adds must not get lost, however
long it is and wherever the large row lies.

Tolerances as in test_gpu_full_attn.py, but for the small probabilities of an E4M3 cache. P is
there a sum of two E4M3 numbers in units in which a tile's largest is at least 2^5, or the sum of the
tiles before at least 64 times the tiles of the query that a CTA has. A P is off by 2^-8 + 2^-11 of itself or by
2^-10 (half of E4M3's smallest step), whichever is more. The second, over the 128 rows of a tile, is
2^-3 c with c the mean of |v| over the tile: of a tile whose largest is at least 2^5, and so its sum,
2^-8 c; of the other tiles together 2^-3 / 64 = 2^-9 c of the whole sum. No term grows with the rows."""
import math

import pytest
import torch

import two_tier_sparse_gb300 as dsa
from test_gpu_full_attn import FMT, KV_SCALE, config, i32

pytestmark = pytest.mark.gpu
TAU = 512 ** -0.5
PAGE = 128  # rows, an E4M3 tile's


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_device):
    from two_tier_sparse_gb300 import build
    build.build()
    dsa.load()
    torch.cuda.set_device(cuda_device)


def encode(fmt, x):
    """Rows of fmt next to x [n, 512] (64 bits) and the values that they stand for."""
    if fmt == "bf16":
        r = x.bfloat16()
        return r.view(torch.int16), r.double()
    if fmt == "e4m3":
        r = (x / KV_SCALE).float().clamp(-448, 448).to(torch.float8_e4m3fn)
        return r.view(torch.uint8), r.double() * KV_SCALE
    b = x.view(-1, 16, 32)
    X = (torch.floor(torch.log2(b.abs().amax(dim=2))) - 2).clamp(-100, 100)
    y = b * torch.exp2(-X)[..., None]
    lut = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=x.device)
    code = (y.abs()[..., None] - lut).abs().argmin(dim=-1)
    v = (lut[code] * torch.sign(y) * torch.exp2(X)[..., None]).view(-1, 512)
    code = (code + 8 * (y < 0)).view(-1, 256, 2)
    return torch.cat([code[..., 0] + 16 * code[..., 1], (X + 127).long()], dim=1).to(torch.uint8), v


def peaked(fmt, n, spread, seed):
    """n rows, the first the large one, and four sets of queries that weigh it at about half (some
    heads less, some more) against the others, whose scores have this spread."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = 0.5 + torch.randn((n, 512), generator=g, device="cuda", dtype=torch.float64)
    x[:, :32] = 0.5 + spread * torch.randn((n, 32), generator=g, device="cuda", dtype=torch.float64)
    sign = torch.randint(0, 2, (32,), generator=g, device="cuda").double() * 2 - 1
    x[0, :32] = 4 * sign
    x[0, 32:] = -0.5 * torch.rand((480,), generator=g, device="cuda", dtype=torch.float64)
    rows, values = encode(fmt, x)
    gap = math.log(n) + 0.5 * (0.5 * spread) ** 2
    heads = 0.9 + 0.2 * torch.rand((4, 64, 1), generator=g, device="cuda", dtype=torch.float64)
    q = torch.zeros((4, 64, 512), device="cuda", dtype=torch.float64)
    q[..., :32] = heads * sign * gap / (TAU * 32 * 4)
    q[..., :32] *= 1 + 0.05 * torch.randn((4, 64, 32), generator=g, device="cuda", dtype=torch.float64)
    return rows, values, q.bfloat16()


def expect(fmt, q, v):
    """Outputs, lse, and how far off each may be, of queries [64, 512] over all of v [n, 512] in
    pages (a tile of E4M3 rows; the last may be shorter)."""
    q = q.double()
    z = q @ v.T * TAU
    lse = torch.logsumexp(z, dim=1)
    p = torch.exp(z - lse[:, None])
    o, A = p @ v, p @ v.abs()
    e_z = 520 * 2.0 ** -24 * TAU * (q.abs() @ v.abs().T).amax() + 2.0 ** -21 * (1 + z.abs().amax())
    tol = 2.0 ** -8 * o.abs() + 2.0 ** -8 * A
    if fmt == "e4m3":
        e_z = e_z + 2.0 ** -17.8 * TAU * q.abs().amax() * v.abs().sum(dim=1).amax()
        c = torch.stack([t.abs().sum(dim=0) / PAGE for t in v.split(PAGE)]).amax(dim=0)
        tol = tol + 2.0 ** -11 * A + (2.0 ** -8 + 2.0 ** -9) * c
    return o, lse, tol + 2 * e_z * A + 1e-30, 2 * e_z, p[:, 0]


@pytest.mark.parametrize("spread", [0.0, 2.0])
@pytest.mark.parametrize("B,n", [(152, 65536), (160, 8192), (16, 32768), (3, 131072), (1, 2048)])
@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "mxfp4"])
def test_one_large_row_and_a_long_tail(fmt, B, n, spread):
    rows, values, q4 = peaked(fmt, n - 37, spread, seed=n + B)
    pad = torch.full((37, rows.shape[1]), 0x7F, dtype=rows.dtype, device="cuda")  # (NaN in E4M3)
    latents = torch.cat([rows, pad]).contiguous()
    n_pages = n // PAGE
    # sequence b has the large row's page first, in the middle or just before the last
    table = torch.empty((B, n_pages), dtype=torch.int32)
    others = list(range(1, n_pages - 1))
    for b in range(B):
        order = others[b % len(others):] + others[:b % len(others)]
        order.insert((0, len(order) // 2, len(order))[b % 3], 0)
        table[b] = torch.tensor(order + [n_pages - 1])
    pages = dsa.Pages(table.cuda(), PAGE, n_pages)
    q = q4[torch.arange(B) % 4].contiguous()
    out, lse = torch.empty_like(q), torch.empty((B, 64), device="cuda")
    cfg = config(fmt)
    ws = dsa.full_attn_workspace(cfg, B)
    dsa.full_attn_decode(cfg, q, latents, i32([n - 37] * B), out, ws, pages=pages, lse=lse)
    assert dsa.read_device_status(ws) == (0, 0)
    for k in range(min(4, B)):
        o, want, tol, tol_lse, top = expect(fmt, q4[k], values)
        assert 0.2 < top.mean() < 0.8  # (about half is the tail's)
        worst = ((out[k::4].double() - o).abs() / tol).amax(dim=(1, 2))
        assert worst.max() <= 1, worst
        assert ((lse[k::4].double() - want).abs() <= tol_lse).all()


@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "mxfp4"])
def test_large_rows_now_and_then(fmt):
    """Heads whose largest score comes, goes and comes back: tiles whose largest scores lie 2^0 to
    2^30 below the head's largest, in any order, and a last tile far above all."""
    n = 64 * PAGE
    g = torch.Generator(device="cuda").manual_seed(3)
    x = 0.5 + torch.randn((n, 512), generator=g, device="cuda", dtype=torch.float64)
    level = torch.randint(0, 31, (64,), generator=g, device="cuda").double()
    level[5], level[63] = 30, 34
    x[:, 0] = (level / 4).repeat_interleave(PAGE)  # (quarters up to 8.5: of every format)
    x[:, 1:32] = 0
    rows, values = encode(fmt, x)
    q = torch.zeros((1, 64, 512), device="cuda", dtype=torch.float64)
    q[0, :, 0] = 4 * math.log(2) / TAU
    q = q.bfloat16()
    q[0, :, 32:] = (0.02 * torch.randn((64, 480), generator=g, device="cuda")).bfloat16()
    cfg = config(fmt)
    for B in (1, 152):
        qq = q.expand(B, 64, 512).contiguous()
        pages = dsa.Pages(torch.arange(64, dtype=torch.int32).repeat(B, 1).cuda(), PAGE, 64)
        out, lse = torch.empty_like(qq), torch.empty((B, 64), device="cuda")
        ws = dsa.full_attn_workspace(cfg, B)
        dsa.full_attn_decode(cfg, qq, rows.contiguous(), i32([n] * B), out, ws, pages=pages, lse=lse)
        assert dsa.read_device_status(ws) == (0, 0)
        o, want, tol, tol_lse, _ = expect(fmt, q[0], values)
        assert ((out.double() - o).abs() <= tol).all()
        assert ((lse.double() - want).abs() <= tol_lse).all()
