"""The step plan, the norms with rotation and the cache rows on the GPU against plain
statements of them (loops and float64).

Tolerances. Plans and 4-bit rows are exact: lengths and slots are integers, and a
bf16 element times a power of two and its rounding to a code have no other
rounding. Norms and rotations: the sum of squares (at most 37 additions in a chain,
each 2^-24) enters with a half, then rsqrt (2 ulp), three products, the cosine and
sine (2 ulp, and an angle known to 2^-24 of half a turn, 2^-22.3) and two products and a sum:
under 2^-19 of |y0| + |y1|, before the rounding to the type, half a step of the result."""
import numpy as np
import pytest
import torch

import oracle as O
import two_tier_sparse_gb300 as dsa

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_device):
    from two_tier_sparse_gb300 import build
    build.build()
    dsa.load()
    torch.cuda.set_device(cuda_device)


def small_ws():
    return dsa.workspace(dsa.config(), 1, 0)


# ---------------------------------------------------------------------------
# Step plans
# ---------------------------------------------------------------------------


class PlanOracle:
    """A pool and its requests as lists."""

    def __init__(self, B, R, per_seq, n_pages, ratio, window, head=0):
        self.R, self.per_seq, self.ratio, self.window = R, per_seq, ratio, window
        self.n_pages = n_pages
        self.table = [[] for _ in range(B)]
        self.n = [0] * B
        self.free = list(range(n_pages))
        self.head, self.tail = head, head + n_pages

    def pages(self, n):
        return -(-(n // self.ratio) // self.R)

    def step(self, new):
        """Per-token rows (request, position, latent slot, window slot)."""
        back = []
        for b, a in enumerate(new):
            if a < 0:
                back += self.table[b]
                self.table[b] = []
                self.n[b] = 0
            else:
                for _ in range(self.pages(self.n[b] + a) - len(self.table[b])):
                    self.table[b].append(self.free.pop(0))
                    self.head += 1
        self.free += back
        self.tail += len(back)
        rows, cu = [], [0]
        for b, a in enumerate(new):
            end = self.n[b] + max(a, 0)
            for p in range(self.n[b], end):
                lat = wslot = -1
                if (p + 1) % self.ratio == 0:
                    j = (p + 1) // self.ratio - 1
                    lat = self.table[b][j // self.R] * self.R + j % self.R
                if p >= end - self.window:
                    wslot = b * self.window + p % self.window
                rows.append((b, p, lat, wslot))
            cu.append(len(rows))
            self.n[b] = end
        return rows, cu


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


def check_plan(o, rows, cu, plan, pool):
    assert plan.cu_new.tolist() == cu
    assert plan.n_tokens.tolist() == o.n
    assert plan.n_latents.tolist() == [n // o.ratio for n in o.n]
    assert plan.swa_len.tolist() == [min(n, o.window) for n in o.n]
    want = np.full((plan.max_new, 4), -1)
    want[:, 1] = 0
    want[:len(rows)] = rows if rows else want[:0]
    got = torch.stack([plan.token_seq, plan.positions, plan.latent_slots, plan.window_slots], 1)
    assert np.array_equal(got.cpu().numpy(), want)
    t = pool.table.cpu().numpy()
    for b, pages in enumerate(o.table):
        assert t[b, :len(pages)].tolist() == pages, b
    assert pool.ring_state_out.tolist() == [o.head, o.tail]
    ring = pool.free_ring.cpu().numpy()
    assert [int(ring[i % o.n_pages]) for i in range(o.head, o.tail)] == o.free


@pytest.mark.parametrize("B,R,ratio,window,most,max_new,seed", [
    (1, 64, 1, 128, 1, 1, 0),
    (3, 64, 2, 5, 40, 130, 1),
    (64, 64, 1, 128, 300, 5001, 2),       # several CTAs, a ragged tail of the arrays
    (700, 128, 2, 128, 90, 20000, 3),     # more requests than threads
    (4096, 192, 3, 1, 12, 40000, 4),      # the most requests
])
def test_plans_follow_a_run_of_steps(B, R, ratio, window, most, max_new, seed):
    rng = np.random.default_rng(seed)
    per_seq = 1 + 6 * most // (R * ratio) + 1
    n_pages = B * per_seq
    head = n_pages - 2  # the ring's positions wrap from the start
    o = PlanOracle(B, R, per_seq, n_pages, ratio, window, head)
    pool = dsa.PagePool.empty(B, R, per_seq, n_pages)
    pool.free_ring.copy_(torch.roll(pool.free_ring, head))
    pool.ring_state.add_(head)
    cfg = dsa.config(ratio=ratio, window=window)
    ws = small_ws()
    n = i32([0] * B)
    plan = dsa.StepPlan.empty(B, max_new, n_tokens=n)  # lengths and the ring in place
    for step in range(7):
        new = rng.integers(0, most + 1, B)
        new[rng.random(B) < 0.3] = 1
        new[rng.random(B) < 0.2] = 0
        if step:
            new[rng.random(B) < 0.2] = -1
        new[new.clip(0).cumsum() > max_new] = 0
        if step == 5:
            new[:] = 0
        dsa.plan_step(cfg, n, i32(new), pool, plan, ws)
        rows, cu = o.step(new.tolist())
        check_plan(o, rows, cu, plan, pool)
        assert dsa.read_device_status(ws)[0] == 0


def test_plan_with_separate_outputs_leaves_its_inputs():
    pool = dsa.PagePool(i32([[3, -1], [-1, -1]]), 64, i32([9, 0, 1, 2]),
                        torch.tensor([1, 4], device="cuda"),
                        ring_state_out=torch.zeros(2, dtype=torch.int64, device="cuda"))
    n, plan = i32([64, 0]), dsa.StepPlan.empty(2, 100)
    for _ in range(2):  # the same again: nothing of the state it reads has moved
        dsa.plan_step(dsa.config(), n, i32([2, 64]), pool, plan, small_ws())
        assert n.tolist() == [64, 0] and pool.ring_state.tolist() == [1, 4]
        assert plan.n_tokens.tolist() == [66, 64] and pool.ring_state_out.tolist() == [3, 4]
        assert pool.table.tolist() == [[3, 0], [1, -1]]
        assert plan.latent_slots[:3].tolist() == [0, 1, 64]


@pytest.mark.parametrize("what", ["pages", "rows", "per_seq", "negative", "ring", "overflow"])
def test_an_impossible_plan_changes_nothing(what):
    B, max_new = 5, 3000
    pool = dsa.PagePool.empty(B, 64, 8, 12)
    ws, cfg = small_ws(), dsa.config()
    n, new = i32([10, 64, 0, 3, 500]), [1, 1, 2, -1, 0]
    if what == "pages":
        pool.ring_state.copy_(torch.tensor([11, 12]))
    if what == "rows":
        new[2] = max_new
    if what == "per_seq":
        new[2] = 8 * 64 + 1
    if what == "negative":
        n[3] = -7
    if what == "ring":
        pool.ring_state.copy_(torch.tensor([3, 17]))
    if what == "overflow":
        new[4] = 2 ** 31 - 1
    plan = dsa.StepPlan.empty(B, max_new)
    n0, t0, r0, s0 = n.clone(), pool.table.clone(), pool.free_ring.clone(), pool.ring_state.clone()
    dsa.plan_step(cfg, n, i32(new), pool, plan, ws)
    assert torch.equal(plan.n_tokens, n0) and torch.equal(n, n0)
    assert torch.equal(pool.table, t0) and torch.equal(pool.free_ring, r0)
    assert torch.equal(pool.ring_state_out, s0)
    assert not plan.cu_new.any() and not plan.positions.any()
    for t in (plan.token_seq, plan.latent_slots, plan.window_slots):
        assert bool((t == -1).all())
    code, info = dsa.read_device_status(ws)
    assert code == 6 and info >> 24 == 7
    assert dsa.read_device_status(ws)[0] == 0
    # a possible one right after it, in the same workspace
    if what in ("rows", "per_seq", "overflow"):
        dsa.plan_step(cfg, n, i32([1, 1, 2, 0, 0]), pool, plan, ws)
        assert plan.cu_new.tolist() == [0, 1, 2, 4, 4, 4]


def test_a_table_entry_outside_the_pool_gives_no_slot():
    pool = dsa.PagePool.empty(2, 64, 4, 8)
    pool.table[0, 0] = 8
    pool.table[1, 0] = 5
    ws, plan = small_ws(), dsa.StepPlan.empty(2, 8)
    dsa.plan_step(dsa.config(), i32([10, 10]), i32([1, 1]), pool, plan, ws)
    assert plan.latent_slots[:2].tolist() == [-1, 5 * 64 + 10]
    code, info = dsa.read_device_status(ws)
    assert code == 6 and info == (7 << 24)


def test_plan_of_no_requests_and_no_rows():
    ws = small_ws()
    pool = dsa.PagePool.empty(2, 64, 4, 8)
    plan = dsa.StepPlan.empty(2, 0)
    dsa.plan_step(dsa.config(), i32([3, 4]), i32([0, -1]), pool, plan, ws)
    # request 1 would push a page onto a ring that already holds every page: refused
    assert plan.n_tokens.tolist() == [3, 4] and plan.cu_new.tolist() == [0, 0, 0]
    assert dsa.read_device_status(ws)[0] == 6
    pool.ring_state[0] += 2  # the two pages that the requests hold are not free
    dsa.plan_step(dsa.config(), i32([3, 4]), i32([0, -1]), pool, plan, ws)
    assert plan.n_tokens.tolist() == [3, 0] and plan.cu_new.tolist() == [0, 0, 0]
    assert pool.ring_state.tolist() == [2, 9]
    pool0 = dsa.PagePool(i32(np.zeros((0, 4))), 64, i32(range(8)), torch.tensor([0, 8], device="cuda"))
    plan0 = dsa.StepPlan.empty(0, 4)
    dsa.plan_step(dsa.config(), i32(np.zeros(0)), i32(np.zeros(0)), pool0, plan0, ws)
    assert plan0.cu_new.tolist() == [0] and plan0.token_seq.tolist() == [-1] * 4
    assert dsa.read_device_status(ws)[0] == 0


# ---------------------------------------------------------------------------
# Norms and rotation
# ---------------------------------------------------------------------------

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 0.0, torch.float16: 2.0 ** -25, torch.float32: 0.0}  # below the normals


def frequencies(half, base=160000.0):
    return base ** -(np.arange(half) / half)


def check_heads(got, x, w, eps, pos, f, start, interleaved, scale, norm=True):
    xs = x.double().cpu().numpy()
    wn = None if w is None else w.double().cpu().numpy()
    ref = O.norm_rope(xs, wn, eps, pos, f, start, interleaved, scale, norm)
    plain = np.abs(O.norm_rope(xs, wn, eps, pos, f, -1, interleaved, scale, norm))
    size = plain.copy()  # |y0| + |y1| of each rotated element's pair, times scale
    if start >= 0:
        half = len(f)
        i = np.arange(half)
        i0, i1 = (start + 2 * i, start + 2 * i + 1) if interleaved else (start + i, start + half + i)
        size[..., i0] = size[..., i1] = scale * (plain[..., i0] + plain[..., i1])
    tol = HALF_STEP[got.dtype] * np.abs(ref) * (1 + 2.0 ** -10) + 2.0 ** -19 * size + TINY[got.dtype]
    err = np.abs(got.double().cpu().numpy() - ref)
    assert np.all(err <= tol), f"{(err / np.maximum(tol, 1e-300)).max()} of the tolerance"


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("n,heads,dim,rope_dim,start,interleaved", [
    (1, 64, 512, 64, 448, True),
    (1, 1, 8, 8, 0, True),          # the smallest head
    (3, 5, 24, 16, 8, False),       # three of four lanes
    (7, 3, 64, 64, 0, False),
    (65, 2, 128, 48, 16, False),
    (2, 9, 192, 32, 160, True),
    (5, 4, 576, 64, 512, False),    # three chunks a lane, the last in part
    (4, 3, 512, 512, 0, False),     # halves in different chunks of a lane
    (2, 2, 1024, 1024, 0, False),   # the largest head and rotation
    (2, 2, 1000, 40, 8, True),
    (300, 16, 128, 128, 0, True),
])
def test_norm_rope(dtype, n, heads, dim, rope_dim, start, interleaved):
    g = torch.Generator(device="cuda").manual_seed(dim + n)
    x = (torch.randn((n, heads, dim), generator=g, device="cuda") * 3).to(dtype)
    x[0, 0] = 0  # a head of zeros stays zeros
    w = torch.randn((dim,), generator=g, device="cuda")
    pos = torch.randint(0, 1 << 20, (n,), generator=g, device="cuda").to(torch.int32)
    pos[0] = 2 ** 31 - 1 if n % 2 else 0
    f = frequencies(rope_dim // 2)
    out = torch.full_like(x, float("nan"))
    hs = dsa.HeadSet([dsa.Heads(x, out, weight=w, eps=1e-6, rope_start=start)])
    rope = dsa.Rope(torch.tensor(f, device="cuda"), interleaved=interleaved, scale=1.25)
    dsa.norm_rope(pos, hs, rope)
    check_heads(out, x, w, float(np.float32(1e-6)), pos.cpu().numpy(), f, start, interleaved, 1.25)
    assert not out[0, 0].any()


def test_norm_rope_groups_strides_in_place_and_padding():
    """Queries and keys as slices of one fused projection, some rotated, one without a weight,
    one rotated without a norm, one in place; rows behind n_valid stay."""
    g = torch.Generator(device="cuda").manual_seed(5)
    n, valid = 37, 29
    widths = [("q", 6, 128, 64, True), ("k", 2, 128, 64, True), ("i", 3, 64, None, True),
              ("v", 1, 64, 0, False)]
    total = sum(h * d for _, h, d, _, _ in widths)
    fused = torch.randn((n, total + 8), generator=g, device="cuda").bfloat16()
    before = fused.clone()
    pos = torch.randint(0, 5000, (n,), generator=g, device="cuda").to(torch.int32)
    f = frequencies(32)
    groups, at = [], 0
    for name, h, d, start, norm in widths:
        x = fused[:, at:at + h * d].view(n, h, d)
        out = x if name == "v" else torch.full((n, h, d), 7.0, dtype=torch.bfloat16, device="cuda")
        w = torch.randn((d,), generator=g, device="cuda") if name in "qk" else None
        groups.append(dsa.Heads(x, out, weight=w, eps=0.5, norm=norm, rope_start=start))
        at += h * d
    rope = dsa.Rope(torch.tensor(f, device="cuda"), interleaved=False)
    dsa.norm_rope(pos, dsa.HeadSet(groups), rope, n_valid=i32([valid]))
    at = 0
    for (name, h, d, start, norm), gr in zip(widths, groups):
        x = before[:, at:at + h * d].view(n, h, d)
        check_heads(gr.out[:valid], x[:valid], gr.weight, 0.5, pos[:valid].cpu().numpy(), f,
                    -1 if start is None else start, False, 1.0, norm)
        rest = gr.out[valid:]
        assert torch.equal(rest, x[valid:]) if name == "v" else bool((rest == 7.0).all())
        at += h * d
    assert torch.equal(fused[:, total:], before[:, total:])  # between the tokens' heads
    assert torch.equal(fused[:, :total - 64], before[:, :total - 64])


def test_norm_rope_two_dimensions_and_norm_alone():
    x = torch.randn((9, 512), device="cuda").bfloat16()
    out = torch.empty_like(x)
    dsa.norm_rope(None, dsa.HeadSet([dsa.Heads(x, out)]))
    check_heads(out[:, None], x[:, None], None, float(np.float32(1e-6)), None, [], -1, True, 1.0)
    bits = x.view(torch.int16).clone()  # bf16 as bits
    dsa.norm_rope(None, dsa.HeadSet([dsa.Heads(bits)]))
    assert torch.equal(bits.view(torch.bfloat16), out)


def test_norm_rope_keeps_a_bad_head_to_itself():
    x = torch.randn((2, 4, 128), device="cuda").bfloat16()
    clean = x.clone()
    x[0, 1, 5] = float("nan")
    x[1, 2, 7] = float("inf")
    out, ref = torch.empty_like(x), torch.empty_like(x)
    pos = i32([3, 4])
    rope = dsa.Rope(torch.tensor(frequencies(32), device="cuda"))
    dsa.norm_rope(pos, dsa.HeadSet([dsa.Heads(x, out, rope_start=64)]), rope)
    dsa.norm_rope(pos, dsa.HeadSet([dsa.Heads(clean, ref, rope_start=64)]), rope)
    keep = torch.ones((2, 4), dtype=torch.bool, device="cuda")
    keep[0, 1] = keep[1, 2] = False
    assert torch.equal(out[keep], ref[keep])
    assert bool(out[0, 1].isnan().all()) and bool(out[1, 2, 7].isnan())


# ---------------------------------------------------------------------------
# Cache rows
# ---------------------------------------------------------------------------


def bits(t):
    return t.view(torch.int16)


@pytest.mark.parametrize("n,n_rows", [(1, 1), (5, 40), (1999, 4001), (20000, 20003)])
@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "mxfp4"])
def test_rows_written_and_read(fmt, n, n_rows):
    rng = np.random.default_rng(n)
    g = torch.Generator(device="cuda").manual_seed(n)
    v = torch.randn((n, 512), generator=g, device="cuda")
    v *= torch.exp2(torch.randint(-30, 30, (n, 16), generator=g, device="cuda").float()
                    ).repeat_interleave(32, 1) if fmt == "mxfp4" else 1.0
    wide = torch.zeros((n, 520), dtype=torch.bfloat16, device="cuda")  # rows with a stride
    wide[:, :512] = v
    rows = wide[:, :512]
    rows[n // 2] = 0
    if n > 3:
        rows[1, :32] = 2.0 ** -126  # the smallest normals: the scale stops at 2^-127
        rows[1, 32:64] = 3.0e38     # the largest
        rows[1, 64:96] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 4.0] * 4)  # ties
        rows[3, ::2] = -0.0
    slots = rng.permutation(n_rows)[:n].astype(np.int32)
    if n > 100:
        slots[::7] = -1
    scale = 0.013 if fmt == "e4m3" else 1.0
    cfg = dsa.config(kv_fmt={"bf16": dsa.KV_BF16, "e4m3": dsa.KV_FP8_E4M3, "mxfp4": dsa.KV_MXFP4}[fmt],
                     kv_scale=scale)
    width = {"bf16": 512, "e4m3": 512, "mxfp4": 272}[fmt]
    cache = torch.full((n_rows, width), 0x5A, dtype=torch.int16 if fmt == "bf16" else torch.uint8,
                       device="cuda")
    ws = small_ws()
    dsa.kv_write(cfg, rows, i32(slots), cache, ws)
    got = cache.cpu().numpy()
    h = rows.float().cpu().numpy()
    with np.errstate(over="ignore", invalid="ignore"):
        want = {"bf16": lambda: rows.contiguous().view(torch.int16).cpu().numpy(),
                "e4m3": lambda: O.e4m3_encode((h / np.float32(scale)).astype(np.float64)),
                "mxfp4": lambda: O.latent_rows_mxfp4(h)}[fmt]()
    there = slots >= 0
    assert np.array_equal(got[slots[there]], want[there])
    rest = np.setdiff1d(np.arange(n_rows), slots[there])
    assert (got[rest] == 0x5A).all()
    out = torch.full((n, 512), 9.0, dtype=torch.bfloat16, device="cuda")
    dsa.kv_read(cfg, cache, i32(slots), out, ws)
    back = O.latent_values(want.view(np.uint16) if fmt == "bf16" else want,
                           "fp8" if fmt == "e4m3" else fmt, 1.0)
    if fmt == "e4m3":  # the code times the scale in fp32, then bf16
        ref = O.f32_to_bf16_rne(back.astype(np.float32) * np.float32(scale))
    else:  # exact
        ref = O.f32_to_bf16_rne(back.astype(np.float32))
    o = bits(out).cpu().numpy().view(np.uint16)
    assert np.array_equal(o[there] & 0x7FFF, ref[there] & 0x7FFF)
    assert np.array_equal(O.bf16_to_f64(o[there]), O.bf16_to_f64(ref[there]))
    assert (out[torch.from_numpy(~there).cuda()] == 9.0).all()
    assert dsa.read_device_status(ws)[0] == 0


@pytest.mark.parametrize("scale", [2.0 ** -6, 1.0 / 3, 0.0173, 1.9999999, 3e-5, 448.0, 2.0 ** -60 * 1.3,
                                   2.0 ** 59 * 1.7, 2.0 ** -61, 2.0 ** 61 * 1.1, 1.2e-38])
def test_e4m3_rows_of_every_bf16_value(scale):
    """Every finite bf16 value over a scale is the fp32 quotient's code (the scales on both
    sides of what the reciprocal is used for)."""
    x = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    x = torch.where(torch.isfinite(x.float()), x, torch.zeros_like(x)).view(128, 512)
    cfg = dsa.config(kv_fmt=dsa.KV_FP8_E4M3, kv_scale=scale)
    cache = torch.zeros((128, 512), dtype=torch.uint8, device="cuda")
    dsa.kv_write(cfg, x.cuda(), i32(np.arange(128)), cache, small_ws())
    with np.errstate(over="ignore", under="ignore"):
        q = x.float().numpy() / np.float32(cfg.kv_scale)
    want = O.e4m3_encode(np.clip(q, -1e4, 1e4).astype(np.float64))  # (saturates far below)
    assert np.array_equal(cache.cpu().numpy(), want)


def test_rows_past_the_cache_and_past_the_valid_ones():
    cfg, ws = dsa.config(kv_fmt=dsa.KV_MXFP4), small_ws()
    rows = torch.randn((6, 512), device="cuda").bfloat16()
    cache = torch.zeros((4, 272), dtype=torch.uint8, device="cuda")
    dsa.kv_write(cfg, rows, i32([0, 4, 2 ** 31 - 1, -5, 3, 1]), cache, ws, n_valid=i32([5]))
    code, info = dsa.read_device_status(ws)
    assert code == 6 and info >> 24 == 8 and info & 0xFFFFFF in (1, 2)
    assert cache[0].any() and cache[3].any() and not cache[1].any() and not cache[2].any()
    out = torch.zeros_like(rows)
    dsa.kv_read(cfg, cache, i32([4, 0, -1, 3, 2, 2]), out, ws, n_valid=i32([4]))
    code, info = dsa.read_device_status(ws)
    assert code == 6 and info == (8 << 24)
    assert out[1].any() and out[3].any()
    assert not out[0].any() and not out[2].any() and not out[4:].any()
    for nv in (0, -3, 100):
        out.zero_()
        dsa.kv_read(cfg, cache, i32([0] * 6), out, ws, n_valid=i32([nv]))
        assert out.any(dim=1).sum() == (6 if nv == 100 else 0)


def test_groups_with_nan_or_infinity_become_nan():
    cfg, ws = dsa.config(kv_fmt=dsa.KV_MXFP4), small_ws()
    rows = torch.ones((2, 512), dtype=torch.bfloat16, device="cuda")
    rows[0, 40] = float("nan")
    rows[1, 511] = -float("inf")
    cache = torch.zeros((2, 272), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(rows)
    dsa.kv_write(cfg, rows, i32([1, 0]), cache, ws)
    dsa.kv_read(cfg, cache, i32([1, 0]), out, ws)
    bad = torch.zeros((2, 512), dtype=torch.bool, device="cuda")
    bad[0, 32:64] = bad[1, 480:] = True
    assert torch.equal(out.isnan(), bad) and bool((out[~bad] == 1).all())


def test_serving_calls_on_a_stream_and_in_a_graph():
    """Plan, norms and rows captured in one graph on a side stream, replayed with
    other inputs: as the eager calls give it."""
    B, max_new, ws = 4, 16, small_ws()
    cfg = dsa.config(kv_fmt=dsa.KV_MXFP4)
    f = torch.tensor(frequencies(32), device="cuda")

    def state():
        pool = dsa.PagePool.empty(B, 64, 4, 16)
        n = i32([0] * B)
        kv = torch.zeros((max_new, 512), dtype=torch.bfloat16, device="cuda")
        return dict(pool=pool, n=n, new=i32([0] * B), kv=kv, plan=dsa.StepPlan.empty(B, max_new, n_tokens=n),
                    hs=dsa.HeadSet([dsa.Heads(kv, rope_start=448)]), ws=small_ws(),
                    lat=torch.zeros((16 * 64, 272), dtype=torch.uint8, device="cuda"),
                    win=torch.zeros((B, 128, 272), dtype=torch.uint8, device="cuda"))

    def step(s):
        dsa.plan_step(cfg, s["n"], s["new"], s["pool"], s["plan"], s["ws"])
        dsa.norm_rope(s["plan"].positions, s["hs"], rope, n_valid=s["plan"].n_valid)
        dsa.kv_write(cfg, s["kv"], s["plan"].latent_slots, s["lat"], s["ws"])
        dsa.kv_write(cfg, s["kv"], s["plan"].window_slots, s["win"], s["ws"])
    rope = dsa.Rope(f)
    eager, captured = state(), state()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(captured)  # once before the capture: sets limits; all lengths stay 0
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step(captured)
    torch.cuda.current_stream().wait_stream(side)
    rng = np.random.default_rng(0)
    for i in range(4):
        new = i32(rng.integers(0, 5, B) if i != 2 else [-1, 1, 4, 0])
        kv = torch.randn((max_new, 512), device="cuda").bfloat16()
        for s in (eager, captured):
            s["new"].copy_(new)
            s["kv"].copy_(kv)
        step(eager)
        graph.replay()
        torch.cuda.synchronize()
        for k in ("n", "kv", "lat", "win"):
            assert torch.equal(eager[k], captured[k]), (i, k)
        assert torch.equal(eager["pool"].table, captured["pool"].table)
        assert eager["lat"].any()
    assert dsa.read_device_status(captured["ws"])[0] == 0
    assert dsa.read_device_status(ws)[0] == 0


def test_tensors_of_another_device_are_refused():
    x = torch.zeros((2, 512), dtype=torch.bfloat16)  # on the host
    with pytest.raises(ValueError):
        dsa.norm_rope(None, dsa.HeadSet([dsa.Heads(x)]))
    with pytest.raises(ValueError):
        dsa.kv_write(dsa.config(), x, torch.zeros(2, dtype=torch.int32), x, small_ws())


def test_calls_with_a_host_tensor_among_their_tensors_are_refused():
    cfg, ws = dsa.config(), small_ws()

    def host(t):
        return t.cpu()
    rows = torch.zeros((2, 512), dtype=torch.bfloat16, device="cuda")
    slots = torch.zeros(2, dtype=torch.int32, device="cuda")
    one = torch.ones(1, dtype=torch.int32, device="cuda")
    cache = torch.zeros((4, 512), dtype=torch.bfloat16, device="cuda")
    for bad in range(4):
        a = [slots, cache, ws, one]
        a[bad] = host(a[bad])
        with pytest.raises(ValueError):
            dsa.kv_write(cfg, rows, a[0], a[1], a[2], n_valid=a[3])
        with pytest.raises(ValueError):
            dsa.kv_read(cfg, a[1], a[0], rows, a[2], n_valid=a[3])
    f = torch.ones(32, dtype=torch.float64, device="cuda")
    for bad in range(3):
        a = [slots, f, one]
        a[bad] = host(a[bad])
        with pytest.raises(ValueError):
            dsa.norm_rope(a[0], dsa.HeadSet([dsa.Heads(rows, rope_start=0)]), dsa.Rope(a[1]),
                          n_valid=a[2])
    plan, pool = dsa.StepPlan.empty(2, 2), dsa.PagePool.empty(2, 64, 2, 4)
    for bad in range(3):
        a = [slots, slots, ws]
        a[bad] = host(a[bad])
        with pytest.raises(ValueError):
            dsa.plan_step(cfg, a[0], a[1], pool, plan, a[2])
    with pytest.raises(ValueError):
        dsa.plan_step(cfg, slots, slots, dsa.PagePool.empty(2, 64, 2, 4, device="cpu"), plan, ws)
    with pytest.raises(ValueError):
        dsa.PagePool(pool.table, 64, host(pool.free_ring), pool.ring_state)
    with pytest.raises(ValueError):
        dsa.StepPlan(slots, slots, host(slots), torch.zeros(3, dtype=torch.int32, device="cuda"),
                     one, one, one, one)


@pytest.mark.parametrize("heads,n", [(1, 1), (1, 3), (2, 1), (2, 2), (3, 2), (2, 4), (3, 5)])
def test_norm_rope_takes_every_layout_whose_heads_are_apart(heads, n):
    """Strides from one element of 16 bytes on: refused when two heads share an element,
    normed as they lie otherwise. dim 16, bf16, weights of one, eps 0."""
    dim, step = 16, 8
    gen = torch.Generator().manual_seed(100 * heads + n)
    taken = refused = 0
    for hs in range(step, 13 * step, step):
        for ts in range(step, 13 * step, step):
            at = [h * hs + t * ts for t in range(n) for h in range(heads)]
            apart = all(abs(a - b) >= dim for i, a in enumerate(at) for b in at[:i])
            x = torch.randn((max(at) + dim,), generator=gen).to(torch.bfloat16).cuda()
            out = torch.full_like(x, 9.0)
            h = dsa._HeadsC(x=x.data_ptr(), out=out.data_ptr(), heads=heads, dim=dim,
                            x_token_stride=ts, x_head_stride=hs, out_token_stride=ts,
                            out_head_stride=hs, weight=None, eps=0.0, norm=1, rope_start=-1)
            import ctypes
            code = dsa.load().dsa_norm_rope(n, None, None, 0, ctypes.byref(h), 1, None,
                                            torch.cuda.current_stream().cuda_stream)
            assert code == (0 if apart else 1), (hs, ts)
            if not apart:
                refused += 1
                continue
            taken += 1
            want = torch.full(x.shape, 9.0, dtype=torch.float64)
            tol = torch.zeros(x.shape, dtype=torch.float64)
            xd = x.double().cpu()
            for a in at:
                v = xd[a:a + dim]
                y = v / v.square().mean().sqrt()
                want[a:a + dim] = y
                tol[a:a + dim] = y.abs() * (2.0 ** -8 + 2.0 ** -19)
            assert ((out.double().cpu() - want).abs() <= tol).all(), (hs, ts)
    assert taken and (refused or heads * n == 1)


def test_single_tokens_with_a_stride_of_any_size():
    """The stride of a dimension of one is not used, whatever it is."""
    big = torch.randn((4, 515), device="cuda").to(torch.bfloat16)
    x = big[:1, :512]
    assert x.stride(0) % 8
    w = torch.ones(512, device="cuda")
    out = torch.empty((1, 512), dtype=torch.bfloat16, device="cuda")
    dsa.norm_rope(None, dsa.HeadSet([dsa.Heads(x, out, w, eps=0.0)]))
    y = x.double() / x.double().square().mean().sqrt()
    assert ((out.double() - y).abs() <= y.abs() * (2.0 ** -8 + 2.0 ** -19)).all()
    cache = torch.zeros((2, 512), dtype=torch.bfloat16, device="cuda")
    one = torch.ones(1, dtype=torch.int32, device="cuda")
    dsa.kv_write(dsa.config(), x, one, cache, small_ws())
    assert torch.equal(cache[1], x[0]) and not cache[0].any()


def test_a_row_written_right_before_the_attention_is_read():
    """kv_write -> sparse_attn_decode with nothing between: many times over, every output
    that of the row just written (one visible row, so the output is the row)."""
    for fmt in (dsa.KV_BF16, dsa.KV_MXFP4):
        cfg = dsa.config(kv_fmt=fmt, window=4, k_tokens=8, k_blocks=8)
        ws = dsa.workspace(cfg, 1, 64)
        row = {dsa.KV_BF16: 512, dsa.KV_MXFP4: 272}[fmt]
        swa = torch.zeros((1, 4, row), device="cuda",
                          dtype=torch.bfloat16 if fmt == dsa.KV_BF16 else torch.uint8)
        lat = torch.zeros((1, 64, row), device="cuda", dtype=swa.dtype)
        q = torch.zeros((1, 64, 512), dtype=torch.bfloat16, device="cuda")
        zero, one = (torch.full((1,), v, dtype=torch.int32, device="cuda") for v in (0, 1))
        ids = torch.full((1, 8), -1, dtype=torch.int32, device="cuda")
        outs = [torch.empty((1, 64, 512), dtype=torch.bfloat16, device="cuda") for _ in range(60)]
        rows = [torch.full((1, 512), float(1 << (i % 8)), dtype=torch.bfloat16, device="cuda")
                for i in range(60)]
        torch.cuda.synchronize()
        for r, o in zip(rows, outs):
            dsa.kv_write(cfg, r, zero, swa, ws)
            dsa.sparse_attn_decode(cfg, q, lat, zero, ids, swa, one, o, ws)
        torch.cuda.synchronize()
        for r, o in zip(rows, outs):
            assert (o == r[0, 0]).all()
        assert dsa.read_device_status(ws)[0] == 0


def test_the_compiled_calls_and_the_binding_agree():
    """The plain case in C and the binding's own path (a stream given): same results; what is not
    plain (a stride, another type, another count, a host tensor) goes to the binding's path."""
    calls, cfg, ws = dsa._load_calls(), dsa.config(kv_fmt=dsa.KV_MXFP4), small_ws()
    s = torch.cuda.current_stream()
    g = torch.Generator(device="cuda").manual_seed(8)
    rows = torch.randn((5, 512), generator=g, device="cuda").bfloat16()
    slots, one = i32([3, 0, -1, 6, 2]), i32([4])
    a, b = (torch.zeros((7, 272), dtype=torch.uint8, device="cuda") for _ in range(2))
    for valid in (None, one):
        assert calls.rows(True, cfg, rows, slots, a, ws, valid) == 0
        dsa.kv_write(cfg, rows, slots, b, ws, n_valid=valid, stream=s)
        x, y = torch.zeros_like(rows), torch.zeros_like(rows)
        assert calls.rows(False, cfg, x, slots, a, ws, valid) == 0
        dsa.kv_read(cfg, b, slots, y, ws, n_valid=valid, stream=s)
        assert torch.equal(a, b) and torch.equal(bits(x), bits(y))
    wide = torch.zeros((5, 1024), dtype=torch.bfloat16, device="cuda")
    for bad in ((wide[:, :512], slots, a, ws, None), (rows.float(), slots, a, ws, None),
                (rows, slots.long(), a, ws, None), (rows, slots[:4], a, ws, None),
                (rows, slots, a[:, :256], ws, None), (rows, slots, a, ws.cpu(), None),
                (rows, slots, a, ws, slots), (rows, slots, a.view(-1), ws, None)):
        assert calls.rows(True, cfg, *bad) is None
    assert calls.rows(True, cfg, rows, slots, a, ws[8:], None) == 2  # the library's own answer
    x = torch.randn((5, 3, 64), generator=g, device="cuda")
    p, q = torch.zeros_like(x), torch.zeros_like(x)
    f = dsa.Rope(torch.tensor(frequencies(16), device="cuda"))
    hp, hq = (dsa.HeadSet([dsa.Heads(x, o, rope_start=0)]) for o in (p, q))
    assert calls.norm(slots, x, hp._key, f._key, one) == 0
    dsa.norm_rope(slots, hq, f, n_valid=one, stream=s)
    assert torch.equal(p, q) and p[:4].any() and not p[4].any()
    assert calls.norm(None, x, hp._key, f._key, None) is None
    assert calls.norm(slots.long(), x, hp._key, f._key, None) is None
    pools = [dsa.PagePool.empty(2, 64, 2, 4) for _ in range(2)]
    plans = [dsa.StepPlan.empty(2, 200) for _ in range(2)]
    n, new = i32([0, 0]), i32([100, 70])
    assert calls.plan(cfg, n, new, pools[0]._key, plans[0]._key, ws) == 0
    dsa.plan_step(cfg, n, new, pools[1], plans[1], ws, stream=s)
    for k in ("n_tokens", "n_latents", "swa_len", "cu_new", "positions", "latent_slots"):
        assert torch.equal(getattr(plans[0], k), getattr(plans[1], k)), k
    assert torch.equal(pools[0].table, pools[1].table)
    assert calls.plan(cfg, n[:1], new, pools[0]._key, plans[0]._key, ws) is None
    assert dsa.read_device_status(ws)[0] == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("dim,interleaved", [(128, True), (256, False), (512, True), (512, False),
                                             (576, False), (1024, True)])
def test_norm_rope_runs_over_many_units(dtype, dim, interleaved):
    """Calls of many more units than warps: a warp's run goes over heads, groups and tokens, with
    odd head counts (a warp's last heads missing), a group that is only rotated and one
    that is only normed, and tokens behind the last valid one."""
    n, valid, rope_dim = 800, 787, 64
    g = torch.Generator(device="cuda").manual_seed(dim + interleaved)
    f = frequencies(rope_dim // 2)
    pos = torch.randint(0, 1 << 20, (n,), generator=g, device="cuda").to(torch.int32)
    specs = [(11, dim, dim - 64, True), (1, dim, None, True), (5, 128, 64, True), (3, 72, 8, False)]
    groups, given = [], []
    for heads, d, start, norm in specs:
        x = torch.randn((n, heads, d), generator=g, device="cuda").to(dtype)
        w = torch.randn((d,), generator=g, device="cuda") if norm else None
        out = torch.full_like(x, 7.0)
        groups.append(dsa.Heads(x, out, weight=w, eps=1e-6, norm=norm, rope_start=start))
        given.append((x, out, w, start, norm))
    dsa.norm_rope(pos, dsa.HeadSet(groups), dsa.Rope(torch.tensor(f, device="cuda"),
                                                     interleaved=interleaved, scale=1.25),
                  n_valid=i32([valid]))
    for x, out, w, start, norm in given:
        assert (out[valid:] == 7.0).all()
        check_heads(out[:valid], x[:valid], w, float(np.float32(1e-6)), pos[:valid].cpu().numpy(), f,
                    -1 if start is None else start, interleaved, 1.25, norm=norm)
