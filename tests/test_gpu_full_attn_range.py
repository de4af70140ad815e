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


def bits_of_scales(up, rows, q, fmt="e4m3"):
    """Outputs and lse over rows [n, 512] of E4M3 codes with the cache's scale times 2^up and the
    queries [B, 64, 512] times 2^-up: the same scores."""
    B, n = q.shape[0], rows.shape[0]
    cfg = dsa.config(kv_fmt=dsa.KV_FP8_E4M3, kv_scale=KV_SCALE * 2.0 ** up)
    pages = dsa.Pages(torch.arange(n // 64, dtype=torch.int32).repeat(B, 1).cuda(), 64, n // 64)
    ws = dsa.full_attn_workspace(cfg, B)
    out, lse = torch.empty_like(q), torch.empty((B, 64), device="cuda")
    qs = (q.double() * 2.0 ** -up).bfloat16()
    assert torch.equal(qs.double() * 2.0 ** up, q.double())
    dsa.full_attn_decode(cfg, qs, rows, i32([n] * B), out, ws, pages=pages, lse=lse)
    assert dsa.read_device_status(ws) == (0, 0)
    return out, lse


@pytest.mark.parametrize("B", [1, 152])
@pytest.mark.parametrize("up", [-112, -60, 90])
def test_any_scale_of_an_e4m3_cache(B, up):
    """The cache's scale times a power of two, the queries over it: the same lse, and outputs times
    the same power, where a sum is large (a first row of half the weight and a long tail) or not."""
    g = torch.Generator(device="cuda").manual_seed(2)
    n = 8192
    x = 2 + 2 * torch.randn((n, 512), generator=g, device="cuda")
    x[:, 0] = 0
    x[0, 0] = 64
    rows = x.to(torch.float8_e4m3fn).view(torch.uint8)
    q = 0.02 * torch.randn((B, 64, 512), generator=g, device="cuda")
    q[:, ::2, 0] = math.log(n) / (TAU * 64 * KV_SCALE)
    q = q.bfloat16()
    out, lse = bits_of_scales(0, rows, q)
    for b in sorted({0, B - 1}):
        check("e4m3", q[b], rows.view(torch.float8_e4m3fn).double() * KV_SCALE, TAU, out[b], lse[b])
    o2, l2 = bits_of_scales(up, rows, q)
    assert torch.equal(l2, lse)
    # (what falls below 2^-126 is rounded to a multiple of 2^-133: off by half of that, and out by 2^-8 of it)
    back = o2.double() * 2.0 ** -up
    small = out.double().abs() * 2.0 ** up < 2.0 ** -126
    assert torch.equal(back[~small], out.double()[~small])
    assert ((back - out.double()).abs()[small] <= 2.0 ** (-134 - up) + 2.0 ** -8 * out.double().abs()[small]).all()


@pytest.mark.parametrize("fmt", FMTS)
def test_heads_of_any_size(fmt):
    """Heads of zeros, of subnormal and of the largest elements, with one element far above the others,
    and with an infinity, beside ordinary ones."""
    n = 900
    c = Case(fmt, [n, n, 0], 960, 64, seed=3)
    q = torch.randn((3, 64, 512), generator=c.g, device="cuda").bfloat16()
    q[:, 1] = 0
    q[:, 2] = (q[:, 2].float() * 2.0 ** -126).bfloat16()  # (subnormal, many of them 0)
    q[:, 3] = (q[:, 3].float() * 2.0 ** -118).bfloat16()
    q[:, 4] = 0
    q[:, 4, 100] = 2.0 ** -133  # the smallest there is
    for h, at, big in ((5, 0, 64.0), (6, 511, -100.0), (7, 300, 250.0)):
        q[:, h] *= 2.0 ** -4
        q[:, h, at] = big  # (the others down to 2^-12 and less of it)
    q[:, 8, 3] = math.inf
    q[:, 9, 400] = -math.inf
    out, lse = torch.empty_like(q), torch.empty((3, 64), device="cuda")
    cfg = config(fmt)
    ws = dsa.full_attn_workspace(cfg, 3)
    sw = [128, 5, 0]
    dsa.full_attn_decode(cfg, q, c.latents, i32([n, n, 0]), out, ws, swa=c.swa, swa_len=i32(sw), pages=c.pages,
                         lse=lse)
    assert dsa.read_device_status(ws) == (0, 0)
    some = [h for h in range(64) if h not in (8, 9)]
    assert (out[2] == 0).all() and (lse[2] == -math.inf).all()
    for b in range(2):
        v = torch.cat([c.v[b], c.w[b, :sw[b]]])
        for h in some:  # (each by itself: a tolerance takes the largest of its heads)
            check(fmt, q[b, h:h + 1], v, TAU, out[b, h:h + 1], lse[b, h:h + 1])
        assert torch.isnan(out[b, 8:10]).all() and torch.isnan(lse[b, 8:10]).all()


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_the_largest_queries(fmt):
    """Elements up to 2^122 (and, over an E4M3 cache, to the largest of bf16) under a small tau."""
    n = 300
    c = Case(fmt, [n], 320, 64, seed=4)
    q = torch.randn((1, 64, 512), generator=c.g, device="cuda").clamp(-3.9, 3.9).bfloat16()
    up = 2.0 ** (120 if fmt == "e4m3" else 110)
    big = (q.float() * up).bfloat16()
    if fmt == "e4m3":
        big[:, :, 9] = torch.finfo(torch.bfloat16).max
    assert torch.isfinite(big.float()).all()
    tau = TAU / up
    cfg = config(fmt, sm_scale=tau)
    out, lse = torch.empty_like(q), torch.empty((1, 64), device="cuda")
    ws = dsa.full_attn_workspace(cfg, 1)
    dsa.full_attn_decode(cfg, big, c.latents, i32([n]), out, ws, pages=c.pages, lse=lse)
    assert dsa.read_device_status(ws) == (0, 0)
    # (tau as the configuration holds it, in 32 bits)
    check(fmt, big[0], c.v[0], float(torch.tensor(tau, dtype=torch.float32)), out[0], lse[0])


@pytest.mark.parametrize("B", [1, 40])
def test_any_scales_of_an_mxfp4_cache(B):
    """Blocks of 32 dims whose scales are 2^100 and 2^-60 times others', where the queries have
    zeros: the same scores, and outputs times those powers."""
    n = 640
    g = torch.Generator(device="cuda").manual_seed(5)
    rows, _ = cache_rows(n, "mxfp4", g)
    q = torch.randn((B, 64, 512), generator=g, device="cuda")
    q[..., :96] = 0
    q = q.bfloat16()
    cfg = config("mxfp4")
    ws = dsa.full_attn_workspace(cfg, B)
    pages = dsa.Pages(torch.arange(n // 64, dtype=torch.int32).repeat(B, 1).cuda(), 64, n // 64)
    got = []
    for up, down in ((0, 0), (100, 60)):
        r = rows.clone()
        r[:, 256] += up
        r[:, 257] -= down
        out, lse = torch.empty_like(q), torch.empty((B, 64), device="cuda")
        dsa.full_attn_decode(cfg, q, r, i32([n] * B), out, ws, pages=pages, lse=lse)
        assert dsa.read_device_status(ws) == (0, 0)
        got.append((out.double(), lse))
    (a, la), (b, lb) = got
    assert torch.equal(la, lb) and torch.equal(a[..., 64:], b[..., 64:])
    assert torch.equal(a[..., :32] * 2.0 ** 100, b[..., :32])
    assert torch.equal(a[..., 32:64] * 2.0 ** -60, b[..., 32:64])
