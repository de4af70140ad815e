"""Edges of the serving calls on the GPU: page ids that are no pages, frequencies and positions
of any size, cache elements that are no numbers, the binding without its compiled part, decode
steps right behind what writes their inputs. Tolerances as in test_gpu_serving.py, where
nothing else is said."""
from fractions import Fraction

import numpy as np
import pytest
import torch

import oracle as O
import two_tier_sparse_gb300 as dsa
from test_gpu_serving import frequencies, i32, small_ws

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_device):
    from two_tier_sparse_gb300 import build
    build.build()
    dsa.load()
    torch.cuda.set_device(cuda_device)


@pytest.mark.parametrize("max_new", [8, 20000])  # one CTA, several
@pytest.mark.parametrize("B,held", [(3, 3), (61, 37), (700, 9)])
def test_ids_outside_the_pool_do_not_enter_the_ring(B, held, max_new):
    """Requests end whose table rows hold ids that are no pages: the step is reported with such a
    request, the ring holds -1 for them, and who pops that is reported in turn."""
    rng = np.random.default_rng(B + max_new)
    n_pages = B * held + 5
    table = rng.permutation(n_pages)[:B * held].reshape(B, held).astype(np.int32)
    free = sorted(set(range(n_pages)) - set(table.ravel().tolist()))
    bad = rng.random((B, held)) < 0.2
    bad[0, 1] = True
    table[bad] = rng.choice([-1, -2 ** 31, n_pages, n_pages + 1, 2 ** 31 - 1], int(bad.sum()))
    table[0, 1] = n_pages
    head = n_pages - 3  # the free pages run over the ring's end
    ring = np.full(n_pages, -7, np.int32)
    ring[(head + np.arange(5)) % n_pages] = free
    pool = dsa.PagePool(i32(table), 64, i32(ring), torch.tensor([head, head + 5], device="cuda"))
    n = i32([held * 64] * B)
    plan, ws = dsa.StepPlan.empty(B, max_new, n_tokens=n), small_ws()
    ends = np.ones(B, bool)
    ends[2::5] = False  # these stay, and keep what they hold
    back = np.where(bad, -1, table)[ends].ravel().tolist()
    for new in (np.where(ends, -1, 0), np.zeros(B)):  # then a step in which nobody ends
        dsa.plan_step(dsa.config(), n, i32(new), pool, plan, ws)
        h, t = pool.ring_state.tolist()
        assert (h, t) == (head, head + 5 + len(back))
        r = pool.free_ring.cpu().numpy()
        assert [int(r[i % n_pages]) for i in range(h, t)] == free + back
        assert n.tolist() == np.where(ends, 0, held * 64).tolist()
        code, info = dsa.read_device_status(ws)
        if new.any():
            assert code == 6 and info >> 24 == 7
            b = info & 0xFFFFFF
            assert ends[b] and (bad[b] & (table[b] != -1)).any()
        else:
            assert code == 0


@pytest.mark.parametrize("bad", [-1, 8, 2 ** 31 - 1, -2 ** 31])
def test_a_ring_entry_outside_the_pool_gives_no_page(bad):
    pool = dsa.PagePool.empty(3, 64, 2, 8)
    pool.free_ring[1] = bad
    n, ws = i32([0, 0, 0]), small_ws()
    plan = dsa.StepPlan.empty(3, 300, n_tokens=n)
    dsa.plan_step(dsa.config(), n, i32([64, 65, 1]), pool, plan, ws)
    assert pool.table.tolist() == [[0, -1], [-1, 2], [3, -1]] and pool.ring_state.tolist() == [4, 8]
    slots = plan.latent_slots.tolist()
    assert slots[:64] == list(range(64)) and slots[64:128] == [-1] * 64
    assert slots[128:130] == [128, 192]
    code, info = dsa.read_device_status(ws)
    assert code == 6 and info == (7 << 24) + 1
    # its end: what it was given goes back, a page and none
    dsa.plan_step(dsa.config(), n, i32([0, -1, -1]), pool, plan, ws)
    assert pool.ring_state.tolist() == [4, 11]
    assert [int(pool.free_ring[i % 8]) for i in range(4, 11)] == [4, 5, 6, 7, -1, 2, 3]
    assert dsa.read_device_status(ws)[0] == 0


TWO_PI = Fraction("6.283185307179586476925286766559005768394338798750211641949889184615632812572417997256069650684234136")


def exact_rotation(x, pos, f, start, interleaved):
    """Pairs of x [n, heads, dim] (float64) turned by pos * f, each angle reduced exactly."""
    y = np.array(x, np.float64)
    half = len(f)
    i = np.arange(half)
    i0, i1 = (start + 2 * i, start + 2 * i + 1) if interleaved else (start + i, start + half + i)
    a = np.empty((len(pos), half))
    for t, p in enumerate(pos):
        for k, g in enumerate(f):
            turns = int(p) * Fraction(float(g)) / TWO_PI
            a[t, k] = float((turns - round(turns)) * TWO_PI)
    c, s = np.cos(a)[:, None], np.sin(a)[:, None]
    y0, y1 = y[..., i0], y[..., i1]
    y[..., i0], y[..., i1] = y0 * c - y1 * s, y0 * s + y1 * c
    size = np.abs(np.array(x, np.float64))
    size[..., i0] = size[..., i1] = np.abs(y0) + np.abs(y1)
    return y, size


@pytest.mark.parametrize("interleaved", [True, False])
def test_norm_rope_frequencies_and_positions_of_any_size(interleaved):
    """Frequencies above a turn a position, negative ones, subnormal ones and zero, and negative
    positions: an angle is off by at most 2^-33 turns (under 2^-30 radians) + |angle| 2^-62, the
    rest as above."""
    rng = np.random.default_rng(4)
    f = np.array([2 * np.pi, 6.2831853071795871, 7.5, 100.25, 9999.875, -3.25, -1e4, 2.0 ** 30,
                  0.0, 5e-324, 1e-310, 1.0, 160000.0 ** -0.5, 1e-9, 3e5, 2.0 ** -40])
    pos = np.array([0, 1, -1, 5, -77777, 2 ** 20, 2 ** 31 - 1, -2 ** 31])
    x = rng.standard_normal((len(pos), 3, 64)).astype(np.float32)
    want, size = exact_rotation(x, pos, f, 32, interleaved)
    out = torch.empty((len(pos), 3, 64), device="cuda")
    heads = dsa.Heads(torch.from_numpy(x).cuda(), out, norm=False, rope_start=32)
    dsa.norm_rope(i32(pos), dsa.HeadSet([heads]), dsa.Rope(torch.tensor(f, device="cuda"),
                                                           interleaved=interleaved))
    # the angles' error, for each pair
    off = 2.0 ** -30 + np.abs(pos[:, None].astype(np.float64) * f) * 2.0 ** -62
    i = np.arange(16)
    i0, i1 = (32 + 2 * i, 33 + 2 * i) if interleaved else (32 + i, 48 + i)
    tol = 2.0 ** -24 * np.abs(want) * (1 + 2.0 ** -10) + 2.0 ** -19 * size
    tol[..., i0] += off[:, None] * size[..., i0]
    tol[..., i1] += off[:, None] * size[..., i1]
    assert np.all(np.abs(out.double().cpu().numpy() - want) <= tol)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("interleaved", [True, False])
def test_norm_rope_frequencies_that_are_no_numbers(interleaved, dtype):
    """An infinite or NaN frequency has no angle: its pair is NaN, in every head and at every
    position, and the other pairs are as without it."""
    f = frequencies(16)
    x = torch.randn((4, 3, 64), device="cuda").to(dtype)
    outs = []
    for bad in ((), (2, 7, 11)):
        g = f.copy()
        g[list(bad)] = [float("inf"), float("nan"), -float("inf")][:len(bad)]
        out = torch.empty_like(x)
        dsa.norm_rope(i32([0, 1, 5, -3]), dsa.HeadSet([dsa.Heads(x, out, rope_start=32)]),
                      dsa.Rope(torch.tensor(g, device="cuda"), interleaved=interleaved))
        outs.append(out)
    nan = torch.zeros(64, dtype=torch.bool, device="cuda")
    for k in (2, 7, 11):
        nan[[32 + 2 * k, 33 + 2 * k] if interleaved else [32 + k, 48 + k]] = True
    assert torch.equal(outs[1].isnan(), nan.expand(4, 3, 64))
    assert torch.equal(outs[1][..., ~nan], outs[0][..., ~nan])


def test_the_calls_without_the_compiled_part(monkeypatch):
    """Plan, norm, rows in and out through the binding alone: as with the compiled part."""
    calls, plain = dsa._load_calls(), dsa._NoCalls
    assert calls is not plain
    cfg, ws = dsa.config(kv_fmt=dsa.KV_MXFP4), small_ws()
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn((5, 512), generator=g, device="cuda").bfloat16()
    rope = dsa.Rope(torch.tensor(frequencies(32), device="cuda"))
    got = []
    for part in (calls, plain):
        monkeypatch.setattr(dsa, "_calls", part)
        pool, plan = dsa.PagePool.empty(2, 64, 2, 4), dsa.StepPlan.empty(2, 5)
        dsa.plan_step(cfg, i32([0, 0]), i32([3, 2]), pool, plan, ws)
        y, cache = torch.zeros_like(x), torch.zeros((256, 272), dtype=torch.uint8, device="cuda")
        dsa.norm_rope(plan.positions, dsa.HeadSet([dsa.Heads(x, y, rope_start=448)]), rope,
                      n_valid=plan.n_valid)
        dsa.kv_write(cfg, y, plan.latent_slots, cache, ws)
        back = torch.zeros_like(x)
        dsa.kv_read(cfg, cache, plan.latent_slots, back, ws)
        got.append((pool.table, plan.latent_slots, y, cache, back))
    for a, b in zip(*got):
        assert torch.equal(a, b)
    assert got[0][4].any() and dsa.read_device_status(ws)[0] == 0


@pytest.mark.parametrize("scale", [1.0, 2.0 ** -6, 0.0173, 2.0 ** -61, 2.0 ** 61 * 1.1])
def test_e4m3_rows_of_nan_and_infinity(scale):
    """A NaN becomes a NaN code and an infinity the largest number, on both sides of what the
    reciprocal is used for; the elements beside them are as without them."""
    rows = torch.randn((2, 512), device="cuda").bfloat16()
    cfg, ws = dsa.config(kv_fmt=dsa.KV_FP8_E4M3, kv_scale=scale), small_ws()
    clean, cache = (torch.zeros((2, 512), dtype=torch.uint8, device="cuda") for _ in range(2))
    dsa.kv_write(cfg, rows, i32([0, 1]), clean, ws)
    rows[0, 3], rows[0, 4], rows[1, 511] = float("nan"), float("inf"), -float("inf")
    rows[1, 0] = torch.tensor([-1], dtype=torch.int16).view(torch.bfloat16)[0]  # a negative NaN
    dsa.kv_write(cfg, rows, i32([0, 1]), cache, ws)
    assert int(cache[0, 3]) & 0x7F == 0x7F and int(cache[1, 0]) & 0x7F == 0x7F
    assert int(cache[0, 4]) == 0x7E and int(cache[1, 511]) == 0xFE
    for r, c in ((0, 3), (0, 4), (1, 511), (1, 0)):
        cache[r, c] = clean[r, c]
    assert torch.equal(cache, clean)
    dsa.kv_write(cfg, rows, i32([0, 1]), cache, ws)
    out = torch.zeros_like(rows)
    dsa.kv_read(cfg, cache, i32([0, 1]), out, ws)
    nan = torch.zeros((2, 512), dtype=torch.bool, device="cuda")
    nan[0, 3] = nan[1, 0] = True
    assert torch.equal(out.isnan(), nan)
    assert dsa.read_device_status(ws)[0] == 0


def test_e4m3_rows_read_are_rounded_once():
    """Every code times scales of 24 bits, most of them such that the product lies next to the
    middle of two bf16 values (m / 8 times the scale, m odd, is one, or a step of fp32 beside
    it): rounded to fp32 first, it would come to lie on it. A product of 4 and 24 bits is exact in
    float64."""
    rng = np.random.default_rng(9)
    values = O.E4M3_TABLE[np.arange(256)]
    fin = np.isfinite(values)
    scales = [np.float32(rng.random() + 0.5) for _ in range(20)] + [np.float32(2.0 ** -100 / 3)]
    for m in (9, 11, 13, 15):
        for k in rng.integers(0, 128, 10):
            s = np.float32((1 + (2 * k + 1) * 2.0 ** -8) * 8 / m)
            scales += [s, np.nextafter(s, np.float32(9)), np.nextafter(s, np.float32(0))]
    cache = torch.from_numpy(np.resize(np.arange(256, dtype=np.uint8), (1, 512))).cuda()
    slot, ws, twice = i32([0]), small_ws(), 0
    out = torch.empty((1, 512), dtype=torch.bfloat16, device="cuda")
    for s in scales:
        dsa.kv_read(dsa.config(kv_fmt=dsa.KV_FP8_E4M3, kv_scale=float(s)), cache, slot, out, ws)
        got = out[0, :256].double().cpu().numpy()
        assert np.isnan(got[~fin]).all()
        exact = values[fin] * float(s)
        mant, e = np.frexp(exact)
        want = np.ldexp(np.rint(mant * 256), e - 8)  # 8 bits, ties to even
        assert np.array_equal(got[fin], want), s
        twice += int((want != O.bf16_to_f64(O.f32_to_bf16_rne(exact.astype(np.float32)))).sum())
    assert twice  # the cases are such
    assert dsa.read_device_status(ws)[0] == 0


KV_FORMATS = [dsa.KV_BF16, dsa.KV_FP8_E4M3, dsa.KV_MXFP4]


class LoneStep:
    """A decode step of one sequence over `n` latents of zeros and a window of two rows,
    contiguous caches; more blocks than the candidate stage keeps, so it scans them."""

    def __init__(self, fmt, n):
        self.cfg = dsa.config(kv_fmt=fmt, window=2, k_tokens=8, k_blocks=4)
        self.ws = dsa.workspace(self.cfg, 1, 256)
        row, dt = {dsa.KV_BF16: (512, torch.bfloat16), dsa.KV_FP8_E4M3: (512, torch.uint8),
                   dsa.KV_MXFP4: (272, torch.uint8)}[fmt]
        z = dict(device="cuda")
        self.swa = torch.zeros((1, 2, row), dtype=dt, **z)
        self.lat = torch.zeros((1, 256, row), dtype=dt, **z)
        self.keys = dsa.Keys("bf16", torch.zeros((1, 256, 128), dtype=torch.bfloat16, **z))
        self.pooled = dsa.Keys("bf16", torch.zeros((1, 32, 128), dtype=torch.bfloat16, **z))
        self.q_idx = torch.zeros((1, 16, 128), dtype=torch.bfloat16, **z)
        self.w = torch.zeros((1, 16), **z)
        self.n = i32([n])

    def __call__(self, q, swa_len, out, update_pool):
        dsa.decode_step(self.cfg, q, self.q_idx, self.w, self.keys, self.pooled, self.lat, self.n,
                        256, self.swa, swa_len, out, self.ws, update_pool=update_pool)


def outputs(n):
    return [torch.empty((1, 64, 512), dtype=torch.bfloat16, device="cuda") for _ in range(n)]


@pytest.mark.parametrize("update_pool", [False, True])
@pytest.mark.parametrize("n", [0, 256])
@pytest.mark.parametrize("fmt", KV_FORMATS)
def test_a_row_written_right_before_a_decode_step_is_read(fmt, n, update_pool):
    """kv_write of the one window row -> decode_step with nothing between, many times over. The query
    is zero, so the output is the row over the number of rows (itself and 8 latents of
    zeros): within 2^-7 of that, where neighbouring calls' rows differ by a factor of 2."""
    step = LoneStep(fmt, n)
    q, one, zero = torch.zeros((1, 64, 512), dtype=torch.bfloat16, device="cuda"), i32([1]), i32([0])
    rows = [torch.full((1, 512), 2.0 ** (i % 8), dtype=torch.bfloat16, device="cuda") for i in range(60)]
    outs = outputs(60)
    torch.cuda.synchronize()
    for r, o in zip(rows, outs):
        dsa.kv_write(step.cfg, r, zero, step.swa, step.ws)
        step(q, one, o, update_pool)
    torch.cuda.synchronize()
    share = 1.0 if n == 0 else 1.0 / 9
    for r, o in zip(rows, outs):
        want = float(r[0, 0]) * share
        assert bool(((o.float() - want).abs() <= 2.0 ** -7 * want).all())
    assert dsa.read_device_status(step.ws)[0] == 0


@pytest.mark.parametrize("update_pool", [False, True])
@pytest.mark.parametrize("fmt", KV_FORMATS)
def test_queries_normed_right_before_a_decode_step_are_read(fmt, update_pool):
    """norm_rope of the query in place -> decode_step with nothing between. The window holds a row
    of ones and its negative; a normed query of +-1 has scores +-22.6, so the output is the
    row of its sign (e^-45 of the other), while the query before its norm weighs both alike."""
    step = LoneStep(fmt, 0)
    both = torch.ones((2, 512), dtype=torch.bfloat16, device="cuda")
    both[1] = -1
    dsa.kv_write(step.cfg, both, i32([0, 1]), step.swa, step.ws)
    two = i32([2])
    signs = np.where(np.random.default_rng(6).random(60) < 0.5, -1.0, 1.0)
    qs = [torch.full((1, 64, 512), s * 2.0 ** -20, dtype=torch.bfloat16, device="cuda") for s in signs]
    sets = [dsa.HeadSet([dsa.Heads(q, eps=0.0)]) for q in qs]
    outs = outputs(60)
    torch.cuda.synchronize()
    for q, h, o in zip(qs, sets, outs):
        dsa.norm_rope(None, h)
        step(q, two, o, update_pool)
    torch.cuda.synchronize()
    for s, q, o in zip(signs, qs, outs):
        assert bool((q == s).all()) and bool((o == s).all())
    assert dsa.read_device_status(step.ws)[0] == 0
