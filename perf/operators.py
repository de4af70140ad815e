"""Cases for measuring the operators that keep and read a 4-bit KV cache.

Four operators, as a decode loop over the two-tier sparse attention calls them:

  plan       block tables and slot maps of a step from its request lengths (`plan_step`)
  norm_rope  norms of queries and keys for each head with the position rotation in the
             same pass (`norm_rope`)
  kv_rows    rows written to a cache in the cache's format through a slot map, and read
             back as the bf16 values they stand for (`kv_write`, `kv_read`)
  attn4      the sparse decode attention over a cache held in 4 bits (`sparse_attn_decode`
             and its paged form with `KV_MXFP4`)

With `own` false, `run` computes them from elementary torch operations; with `own` true it
calls the library. Both take the same state.
"""
import math

import torch

own = False

DEV = "cuda"
HEADS, LATENT, WINDOW = 64, 512, 128
ROW4 = LATENT // 2 + LATENT // 32  # bytes of an MXFP4 row: 256 of codes, then 16 scales
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZES = {"bf16": 2, "f16": 2, "f32": 4}
KV_SCALE = 2.0 ** -6  # of an E4M3 cache


def listed():
    return [
        # one token of one request: the latency of a decode step's plan
        {"name": "plan 64 x 1 token", "op": "plan", "B": 64, "new": 64, "ctx": 131072, "ratio": 1,
         "page_rows": 64, "release": 0, "ragged": False},
        # continuous batching: chunks of prompts beside single tokens, some requests ending
        {"name": "plan 301 ragged", "op": "plan", "B": 301, "new": 9973, "ctx": 32768, "ratio": 2,
         "page_rows": 128, "release": 37, "ragged": True},
        # many requests, whole prompts at once
        {"name": "plan 1024 x 128 tokens", "op": "plan", "B": 1024, "new": 131072, "ctx": 65536,
         "ratio": 1, "page_rows": 64, "release": 64, "ragged": True},
        # one request's token: 64 query heads, the latent, 16 index heads, the index key
        {"name": "norm_rope 1 token", "op": "norm_rope", "n": 1, "heads": 64, "kv_heads": 1,
         "dim": 512, "idx_heads": 16, "idx_dim": 128, "rope_dim": 64, "interleaved": True,
         "dtype": "bf16", "fused": False, "max_pos": 1048576},
        # a mixed batch out of one fused projection, halves rotated, f16
        {"name": "norm_rope 333 tokens", "op": "norm_rope", "n": 333, "heads": 64, "kv_heads": 8,
         "dim": 128, "idx_heads": 16, "idx_dim": 128, "rope_dim": 128, "interleaved": False,
         "dtype": "f16", "fused": True, "max_pos": 131072},
        # a prefill chunk
        {"name": "norm_rope 4096 tokens", "op": "norm_rope", "n": 4096, "heads": 64, "kv_heads": 1,
         "dim": 512, "idx_heads": 16, "idx_dim": 128, "rope_dim": 64, "interleaved": True,
         "dtype": "bf16", "fused": False, "max_pos": 65536 + 4096},
        # a decode step's window rows
        {"name": "kv_rows 64 mxfp4", "op": "kv_rows", "n": 64, "rows": 64 * WINDOW, "fmt": "mxfp4",
         "holes": False},
        # a ragged batch's new latents, some tokens completing none (8-bit cache)
        {"name": "kv_rows 1999 e4m3", "op": "kv_rows", "n": 1999, "rows": 16384, "fmt": "e4m3",
         "holes": True},
        # whole prompts
        {"name": "kv_rows 65536 mxfp4", "op": "kv_rows", "n": 65536, "rows": 131072,
         "fmt": "mxfp4", "holes": False},
        # one request of 4096 tokens at ratio 2
        {"name": "attn4 1 x 2048", "op": "attn4", "B": 1, "cap": 2048, "k": 512, "window": 128,
         "page_rows": 0, "ragged": False, "tau": 0.0},
        # the serving batch: 64 requests of 131072 tokens
        {"name": "attn4 64 x 131072", "op": "attn4", "B": 64, "cap": 131072, "k": 512,
         "window": 128, "page_rows": 0, "ragged": False, "tau": 0.0},
        # many short and long requests in 64-row pages, an empty one among them
        {"name": "attn4 200 paged ragged", "op": "attn4", "B": 200, "cap": 16384, "k": 512,
         "window": 128, "page_rows": 64, "ragged": True, "tau": 0.1},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["plan", "norm_rope", "kv_rows", "attn4"])
    if op == "plan":
        B = _log(rng, 1, 1024)
        return {"op": op, "B": B, "new": max(B, _log(rng, 1, 131072)), "ctx": _log(rng, 256, 65536),
                "ratio": rng.choice([1, 2]), "page_rows": rng.choice([64, 128, 192, 256]),
                "release": rng.randint(0, B // 4), "ragged": B > 1}
    if op == "norm_rope":
        dim = rng.choice([64, 128, 192, 256, 512, 576])
        heads = _log(rng, 1, 128)
        n = _log(rng, 1, max(1, min(16384, 4096 * 64 * 512 // (heads * dim * 4))))
        return {"op": op, "n": n, "heads": heads, "kv_heads": rng.choice([1, 2, 8]), "dim": dim,
                "idx_heads": rng.choice([8, 16]), "idx_dim": 128, "rope_dim": rng.choice([32, 64]),
                "interleaved": rng.random() < 0.5, "dtype": rng.choice(["bf16", "f16", "f32"]),
                "fused": rng.random() < 0.5, "max_pos": _log(rng, 1024, 1048576)}
    if op == "kv_rows":
        n = _log(rng, 1, 65536)
        return {"op": op, "n": n, "rows": n + _log(rng, 1, 65536),
                "fmt": rng.choice(["mxfp4", "mxfp4", "e4m3", "bf16"]),
                "holes": n >= 16 and rng.random() < 0.5}
    B = _log(rng, 1, 192)
    paged = rng.random() < 0.5
    cap = _log(rng, 8, 131072 if B <= 32 else 16384)
    page_rows = rng.choice([64, 128, 256]) if paged else 0
    return {"op": op, "B": B, "cap": -(-cap // 256) * 256 if paged else cap,
            "k": rng.choice([512, 512, rng.randint(1, 512)]),
            "window": rng.choice([128, rng.randint(1, 128)]), "page_rows": page_rows,
            "ragged": B > 1, "tau": rng.choice([0.0, 0.02, 0.2])}


# --- inputs -------------------------------------------------------------------------------


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _rand(shape, g, **kw):
    return torch.rand(shape, generator=g, device=DEV, **kw)


def _randn(shape, g, **kw):
    return torch.randn(shape, generator=g, device=DEV, **kw)


def _randint(lo, hi, shape, g):
    return torch.randint(lo, hi, shape, generator=g, device=DEV)


def _lengths(case, g):
    B = case["B"]
    top = case["cap"] if case["op"] == "attn4" else case["ctx"]
    if not case["ragged"]:
        return torch.full((B,), top, dtype=torch.int64, device=DEV)
    n = torch.exp(_rand((B,), g) * math.log(top + 1)).floor().long() - 1  # 0 .. top
    n = n.clamp(0, top)
    n[0] = 0
    return n[torch.randperm(B, generator=g, device=DEV)]


def _mxfp4_rows(n, g):
    """n rows of a normed, gained latent in MXFP4 (OCP MX v1.0): uint8 [n, 272]."""
    gain = torch.exp(0.5 * _randn((LATENT,), g))
    out = torch.empty((n, ROW4), dtype=torch.uint8, device=DEV)
    for at in range(0, n, 16384):
        m = min(16384, n - at)
        out[at:at + m] = _encode_mxfp4(_randn((m, LATENT), g) * gain)
    return out


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": case}
    {"plan": _prepare_plan, "norm_rope": _prepare_norm_rope, "kv_rows": _prepare_kv_rows,
     "attn4": _prepare_attn4}[case["op"]](case, g, s)
    return s


def _prepare_plan(case, g, s):
    B, R, ratio, new = case["B"], case["page_rows"], case["ratio"], case["new"]
    n = _lengths(case, g)
    # new tokens: one a request, the rest as prompt chunks of a few of them; some end
    n_new = torch.ones((B,), dtype=torch.int64, device=DEV)
    rest = new - B
    if rest > 0:
        share = torch.exp(3 * _randn((B,), g))
        n_new += (rest * share / share.sum()).floor().long()
    gone = torch.randperm(B, generator=g, device=DEV)[:case["release"]]
    n_new[gone] = -1
    most = case["ctx"] + (new if case["ragged"] else 1)
    per_seq = -(-most // (R * ratio)) + 1
    have = -(-(n // ratio) // R)
    need = -(-(torch.where(n_new < 0, 0 * n, n + n_new) // ratio) // R)
    used = int(have.sum())
    assert int((need - have).clamp(min=0).sum()) + used <= B * per_seq
    n_pages = B * per_seq + 61
    order = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
    cols = torch.arange(per_seq, device=DEV)
    held = cols[None, :] < have[:, None]
    at = (have.cumsum(0) - have)[:, None] + cols[None, :]
    table = torch.where(held, order[at.clamp(max=n_pages - 1)], torch.full_like(order[:1], -1))
    ring = torch.full((n_pages,), -1, dtype=torch.int32, device=DEV)
    head = n_pages - 7  # the free pages run over the ring's end
    free = order[used:]
    ring[(head + torch.arange(n_pages - used, device=DEV)) % n_pages] = free
    rows = -(-new // 64) * 64  # a padded batch
    i32 = dict(dtype=torch.int32, device=DEV)
    s.update(
        n_tokens=n.to(torch.int32), n_new=n_new.to(torch.int32), table=table.contiguous(),
        ring=ring, ring_state=torch.tensor([head, head + n_pages - used], device=DEV),
        n_pages=n_pages, rows=rows,
        out=dict(ring_state=torch.empty((2,), dtype=torch.int64, device=DEV),
                 n_tokens=torch.empty((B,), **i32), n_latents=torch.empty((B,), **i32),
                 swa_len=torch.empty((B,), **i32), cu_new=torch.empty((B + 1,), **i32),
                 token_seq=torch.empty((rows,), **i32), positions=torch.empty((rows,), **i32),
                 latent_slots=torch.empty((rows,), **i32),
                 window_slots=torch.empty((rows,), **i32)))
    if own:  # the handles a program keeps
        import two_tier_sparse_gb300 as dsa
        o = s["out"]
        s["cfg"] = dsa.config(ratio=ratio, window=WINDOW)
        s["ws"] = dsa.workspace(s["cfg"], B, 0, DEV)
        s["pool"] = dsa.PagePool(s["table"], R, ring, s["ring_state"],
                                 ring_state_out=o["ring_state"])
        s["plan"] = dsa.StepPlan(n_tokens=o["n_tokens"], n_latents=o["n_latents"],
                                 swa_len=o["swa_len"], cu_new=o["cu_new"],
                                 token_seq=o["token_seq"], positions=o["positions"],
                                 latent_slots=o["latent_slots"], window_slots=o["window_slots"])


def _inv_freq(rope_dim):
    """Base 160000, YaRN x16 over 65536 trained positions (frequencies in radians a position)."""
    half, base, factor, trained = rope_dim // 2, 160000.0, 16.0, 65536

    def at(turns):  # the pair that makes `turns` turns over the trained positions
        return rope_dim * math.log(trained / (turns * 2 * math.pi)) / (2 * math.log(base))

    lo, hi = max(math.floor(at(32.0)), 0), min(math.ceil(at(1.0)), rope_dim - 1)
    out = []
    for i in range(half):
        f = base ** (-2.0 * i / rope_dim)
        r = min(max((i - lo) / max(hi - lo, 1e-3), 0.0), 1.0)
        out.append(f / factor * r + f * (1.0 - r))
    return torch.tensor(out, dtype=torch.float64, device=DEV)


def _prepare_norm_rope(case, g, s):
    n, dt = case["n"], DTYPES[case["dtype"]]
    parts = [("q", case["heads"], case["dim"]), ("k", case["kv_heads"], case["dim"]),
             ("q_idx", case["idx_heads"], case["idx_dim"]), ("k_idx", 1, case["idx_dim"])]
    width = sum(h * d for _, h, d in parts)
    s["parts"] = []
    fused = _randn((n, width), g).mul_(2).to(dt) if case["fused"] else None
    at = 0
    for name, h, d in parts:
        x = (fused[:, at:at + h * d].view(n, h, d) if case["fused"]
             else _randn((n, h, d), g).mul_(2).to(dt))
        at += h * d
        w = 1 + 0.2 * _randn((d,), g)
        s["parts"].append((name, x, w, torch.empty((n, h, d), dtype=dt, device=DEV)))
    s["positions"] = _randint(0, case["max_pos"], (n,), g).to(torch.int32)
    s["positions"][0] = case["max_pos"] - 1
    s["inv_freq"] = _inv_freq(case["rope_dim"])
    s["scale"] = 1.0 + 0.1 * math.log(16.0)  # YaRN's factor on cos and sin
    if own:  # the handles a program keeps
        import two_tier_sparse_gb300 as dsa
        s["heads"] = dsa.HeadSet([dsa.Heads(x, out, weight=w, eps=1e-6,
                                            rope_start=x.shape[2] - case["rope_dim"])
                                  for _, x, w, out in s["parts"]])
        s["rope"] = dsa.Rope(s["inv_freq"], interleaved=case["interleaved"], scale=s["scale"])


def _prepare_kv_rows(case, g, s):
    n, rows = case["n"], case["rows"]
    gain = torch.exp(0.5 * _randn((LATENT,), g))
    kv = torch.empty((n, LATENT), dtype=torch.bfloat16, device=DEV)
    for at in range(0, n, 16384):
        m = min(16384, n - at)
        kv[at:at + m] = (_randn((m, LATENT), g) * gain).bfloat16()
    if n > 1:
        kv[n // 2] = 0  # a row of zeros
    s["kv"] = kv
    s["slots"] = torch.randperm(rows, generator=g, device=DEV)[:n].to(torch.int32)
    if case["holes"]:  # tokens without a slot
        s["slots"][_rand((n,), g) < 0.3] = -1
    width, dt = {"mxfp4": (ROW4, torch.uint8), "e4m3": (LATENT, torch.uint8),
                 "bf16": (LATENT, torch.bfloat16)}[case["fmt"]]
    s["cache"] = torch.zeros((rows, width), dtype=dt, device=DEV)
    s["out"] = torch.zeros((n, LATENT), dtype=torch.bfloat16, device=DEV)
    if own:  # the handles a program keeps
        import two_tier_sparse_gb300 as dsa
        s["cfg"] = dsa.config(kv_fmt={"mxfp4": dsa.KV_MXFP4, "e4m3": dsa.KV_FP8_E4M3,
                                      "bf16": dsa.KV_BF16}[case["fmt"]],
                              kv_scale=KV_SCALE if case["fmt"] == "e4m3" else 1.0)
        s["ws"] = dsa.workspace(s["cfg"], n, 0, DEV)


def _prepare_attn4(case, g, s):
    B, cap, k, window, R = case["B"], case["cap"], case["k"], case["window"], case["page_rows"]
    n = _lengths(case, g)
    base = _mxfp4_rows(min(cap * B, 131072), g)
    if R:
        per_seq = cap // R
        have = -(-n // R)
        n_pages = int(have.sum()) + 7
        order = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
        cols = torch.arange(per_seq, device=DEV)
        at = (have.cumsum(0) - have)[:, None] + cols[None, :]
        s["table"] = torch.where(cols[None, :] < have[:, None], order[at.clamp(max=n_pages - 1)],
                                 torch.full_like(order[:1], -1)).contiguous()
        s["n_pages"] = n_pages
        rows = n_pages * R
    else:
        rows = B * cap
    cache = torch.empty((rows, ROW4), dtype=torch.uint8, device=DEV)
    nb = base.shape[0]
    for i, at in enumerate(range(0, rows, nb)):  # the same rows in another order
        m = min(nb, rows - at)
        cache[at:at + m] = torch.roll(base, 7919 * i + 1, 0)[:m]
    s["latents"] = cache if R else cache.view(B, cap, ROW4)
    # k tokens of each request's n, ascending, -1 behind them
    ids = torch.full((B, k), -1, dtype=torch.int64, device=DEV)
    m = min(k, cap)
    for at in range(0, B, 32):
        sub = n[at:at + 32]
        score = _rand((sub.shape[0], cap), g)
        score[torch.arange(cap, device=DEV)[None, :] >= sub[:, None]] = -1
        top = score.topk(m, dim=1)
        got = torch.where(top.values >= 0, top.indices, torch.full_like(top.indices, cap))
        got = got.sort(dim=1).values
        ids[at:at + 32, :m] = torch.where(got < cap, got, torch.full_like(got, -1))
    s["token_ids"] = ids.to(torch.int32)
    s["n_latents"] = n.to(torch.int32)
    s["swa"] = _mxfp4_rows(B * window, g).view(B, window, ROW4)
    s["swa_len"] = n.clamp(max=window).to(torch.int32)
    s["q"] = _randn((B, HEADS, LATENT), g).bfloat16()
    s["out"] = torch.empty((B, HEADS, LATENT), dtype=torch.bfloat16, device=DEV)
    s["lse"] = torch.empty((B, HEADS), dtype=torch.float32, device=DEV)
    if own:  # the handles a program keeps
        import two_tier_sparse_gb300 as dsa
        s["cfg"] = dsa.config(k_tokens=k, window=window, sm_scale=case["tau"],
                              kv_fmt=dsa.KV_MXFP4)
        s["ws"] = dsa.workspace(s["cfg"], B, 0, DEV)
        s["pages"] = dsa.Pages(s["table"], R, s["n_pages"]) if R else None


# --- one pass -----------------------------------------------------------------------------


def run(s):
    op = s["case"]["op"]
    if own:
        return {"plan": _own_plan, "norm_rope": _own_norm_rope, "kv_rows": _own_kv_rows,
                "attn4": _own_attn4}[op](s)
    return {"plan": _plain_plan, "norm_rope": _plain_norm_rope, "kv_rows": _plain_kv_rows,
            "attn4": _plain_attn4}[op](s)


def _own_plan(s):
    import two_tier_sparse_gb300 as dsa
    dsa.plan_step(s["cfg"], s["n_tokens"], s["n_new"], s["pool"], s["plan"], s["ws"])
    return dict(s["out"], table=s["table"], ring=s["ring"])


def _own_norm_rope(s):
    import two_tier_sparse_gb300 as dsa
    dsa.norm_rope(s["positions"], s["heads"], s["rope"])
    return [p[3] for p in s["parts"]]


def _own_kv_rows(s):
    import two_tier_sparse_gb300 as dsa
    dsa.kv_write(s["cfg"], s["kv"], s["slots"], s["cache"], s["ws"])
    dsa.kv_read(s["cfg"], s["cache"], s["slots"], s["out"], s["ws"])
    return s["out"]


def _own_attn4(s):
    import two_tier_sparse_gb300 as dsa
    if s["pages"] is not None:
        dsa.sparse_attn_decode_paged(s["cfg"], s["q"], s["latents"], s["pages"], s["n_latents"],
                                     s["token_ids"], s["swa"], s["swa_len"], s["out"], s["ws"],
                                     lse=s["lse"])
    else:
        dsa.sparse_attn_decode(s["cfg"], s["q"], s["latents"], s["n_latents"], s["token_ids"],
                               s["swa"], s["swa_len"], s["out"], s["ws"], lse=s["lse"])
    return s["out"], s["lse"]


def _plain_plan(s):
    c, o = s["case"], s["out"]
    B, R, ratio, P = c["B"], c["page_rows"], c["ratio"], s["n_pages"]
    n, new = s["n_tokens"].long(), s["n_new"].long()
    gone = new < 0
    grow = new.clamp(min=0)
    after = torch.where(gone, torch.zeros_like(n), n + grow)
    p0 = (n // ratio + R - 1) // R
    p1 = (after // ratio + R - 1) // R
    alloc = torch.where(gone, torch.zeros_like(n), p1 - p0)
    freed = torch.where(gone, p0, torch.zeros_like(n))
    end = grow.cumsum(0)
    cu = torch.cat([torch.zeros_like(end[:1]), end])
    pa, pf = alloc.cumsum(0) - alloc, freed.cumsum(0) - freed
    head, tail = s["ring_state"][0], s["ring_state"][1]
    ring, table = s["ring"], s["table"]
    cols = torch.arange(table.shape[1], device=table.device)[None, :]
    taken = (cols >= p0[:, None]) & (cols < p1[:, None]) & ~gone[:, None]
    src = (head + pa[:, None] + cols - p0[:, None]).clamp(min=0) % P
    back = gone[:, None] & (cols < p0[:, None])
    dst = torch.where(back, (tail + pf[:, None] + cols) % P, torch.full_like(cols, P))
    table.copy_(torch.where(taken, ring[src], table))
    wide = torch.cat([ring, ring[:1]])
    wide[dst.reshape(-1)] = table.reshape(-1)
    ring.copy_(wide[:P])
    o["ring_state"].copy_(torch.stack([head + alloc.sum(), tail + freed.sum()]))
    o["n_tokens"].copy_(after)
    o["n_latents"].copy_(after // ratio)
    o["swa_len"].copy_(after.clamp(max=WINDOW))
    o["cu_new"].copy_(cu)
    i = torch.arange(s["rows"], device=n.device)
    seq = torch.searchsorted(end, i, right=True).clamp(max=B - 1)
    there = i < cu[B]
    t = n[seq] + i - cu[seq]
    j = (t + 1) // ratio - 1
    done = there & ((t + 1) % ratio == 0)
    page = table[seq, (j // R).clamp(0, table.shape[1] - 1)].long()
    none = torch.full_like(t, -1)
    o["token_seq"].copy_(torch.where(there, seq, none))
    o["positions"].copy_(torch.where(there, t, torch.zeros_like(t)))
    o["latent_slots"].copy_(torch.where(done, page * R + j % R, none))
    o["window_slots"].copy_(torch.where(there & (t >= after[seq] - WINDOW),
                                        seq * WINDOW + t % WINDOW, none))
    return dict(o, table=table, ring=ring)


def _plain_norm_rope(s):
    c = s["case"]
    rd = c["rope_dim"]
    a = s["positions"].double()[:, None] * s["inv_freq"][None, :]  # far positions: 64 bits
    cos = (a.cos() * s["scale"]).float()[:, None, :]
    sin = (a.sin() * s["scale"]).float()[:, None, :]
    outs = []
    for _, x, w, out in s["parts"]:
        v = x.float()
        v = v * torch.rsqrt((v * v).mean(dim=2, keepdim=True) + 1e-6) * w
        r = v[..., v.shape[2] - rd:]
        if c["interleaved"]:
            u = r.reshape(*r.shape[:2], rd // 2, 2)
            x0, x1 = u[..., 0], u[..., 1]
            r = torch.stack([x0 * cos - x1 * sin, x0 * sin + x1 * cos], dim=-1).reshape(r.shape)
        else:
            x0, x1 = r[..., :rd // 2], r[..., rd // 2:]
            r = torch.cat([x0 * cos - x1 * sin, x0 * sin + x1 * cos], dim=-1)
        out.copy_(torch.cat([v[..., :v.shape[2] - rd], r], dim=-1))
        outs.append(out)
    return outs


def _encode_mxfp4(v):
    """fp32 [n, 512] to MXFP4 rows (OCP MX v1.0): X = floor(log2 amax) - 2 for 32 values,
    elements v / 2^X to the nearest e2m1 value, ties to the even mantissa, at most 6."""
    u = v.reshape(-1, LATENT // 32, 32)
    e = torch.frexp(u.abs().amax(dim=2)).exponent - 1
    X = torch.where(u.abs().amax(dim=2) > 0, (e - 2).clamp(min=-127), torch.zeros_like(e))
    y = u * _pow2(-X)[..., None]
    m = y.abs()
    # steps of 0.5 below 2, of 1 below 4, of 2 above: round() takes ties to even
    q = torch.where(m < 2, (m * 2).round() / 2, torch.where(m < 4, m.round(), (m / 2).round() * 2))
    q = q.clamp(max=6)
    code = (q * 2).clamp(max=4) + (q - 2).clamp(0, 2) + (q - 4).clamp(0, 2) / 2
    code = code.to(torch.uint8) | (torch.signbit(y).to(torch.uint8) << 3)
    code = code.reshape(-1, LATENT // 2, 2)
    return torch.cat([code[..., 0] | (code[..., 1] << 4), (X + 127).to(torch.uint8)], dim=1)


def _pow2(e):
    """2^e in fp32, exactly, for whole e from -127 to 127."""
    return torch.where(e > -127, (e.int() + 127) << 23, torch.full_like(e.int(), 1 << 22)).view(
        torch.float32)


def _decode_mxfp4(rows):
    """MXFP4 rows uint8 [..., 272] to fp32 [..., 512]."""
    lut = torch.tensor(E2M1 + tuple(-x for x in E2M1), device=rows.device)
    c = rows[..., :LATENT // 2]
    v = torch.stack([lut[(c & 15).int()], lut[(c >> 4).int()]], dim=-1)
    v = v.reshape(*rows.shape[:-1], LATENT // 32, 32)
    f = _pow2(rows[..., LATENT // 2:].int() - 127)
    return (v * f[..., None]).reshape(*rows.shape[:-1], LATENT)


def _plain_kv_rows(s):
    fmt, cache, out = s["case"]["fmt"], s["cache"], s["out"]
    there = s["slots"] >= 0
    at = s["slots"][there].long()
    kv = s["kv"][there].float()
    if fmt == "mxfp4":
        cache[at] = _encode_mxfp4(kv)
        got = _decode_mxfp4(cache[at])
    elif fmt == "e4m3":
        y = (kv / KV_SCALE).clamp(-448, 448)
        cache[at] = y.to(torch.float8_e4m3fn).view(torch.uint8)
        got = cache[at].view(torch.float8_e4m3fn).float() * KV_SCALE
    else:
        cache[at] = kv.bfloat16()
        got = cache[at].float()
    out[there] = got.bfloat16()
    return out


def _rows_of(s):
    """Rows of the cache that each request's ids name, and which of them count."""
    c, ids = s["case"], s["token_ids"].long()
    there = ids >= 0
    at = ids.clamp(min=0)
    if c["page_rows"]:
        page = s["table"].long().gather(1, at // c["page_rows"]).clamp(min=0)
        return page * c["page_rows"] + at % c["page_rows"], there
    return at + c["cap"] * torch.arange(c["B"], device=ids.device)[:, None], there


def _plain_attn4(s):
    c = s["case"]
    tau = c["tau"] if c["tau"] > 0 else 1 / math.sqrt(LATENT)
    at, there = _rows_of(s)
    raw = torch.cat([s["swa"], s["latents"].reshape(-1, ROW4)[at]], dim=1)
    w = torch.arange(c["window"], device=at.device)[None, :] < s["swa_len"][:, None]
    mask = torch.cat([w, there], dim=1)
    v = _decode_mxfp4(raw) * mask[..., None]
    z = torch.matmul(s["q"].float(), v.transpose(1, 2)) * tau
    z = z.masked_fill(~mask[:, None, :], -math.inf)
    m = z.amax(dim=2, keepdim=True)
    m = torch.where(torch.isfinite(m), m, torch.zeros_like(m))
    p = torch.exp(z - m)
    l = p.sum(dim=2, keepdim=True)
    o = torch.matmul(p, v) / torch.where(l > 0, l, torch.ones_like(l))
    s["out"].copy_(o)
    s["lse"].copy_((torch.log(l) + m).squeeze(2))
    return s["out"], s["lse"]


# --- what a pass cannot do without ----------------------------------------------------------


def work(case):
    op = case["op"]
    if op == "plan":
        B, new = case["B"], case["new"]
        pages = new // (case["page_rows"] * case["ratio"]) + 1
        return {"bytes": B * 4 * 6 + new * 4 * 4 + pages * 8 + 32, "flops": 0}
    if op == "norm_rope":
        per = (case["heads"] + case["kv_heads"]) * case["dim"] + (case["idx_heads"] + 1) * case["idx_dim"]
        return {"bytes": case["n"] * (2 * per * SIZES[case["dtype"]] + 4), "flops": 6 * case["n"] * per}
    if op == "kv_rows":
        n = case["n"] * (0.7 if case["holes"] else 1.0)
        row = {"mxfp4": ROW4, "e4m3": LATENT, "bf16": 2 * LATENT}[case["fmt"]]
        return {"bytes": n * (2 * 2 * LATENT + 2 * row) + 8 * case["n"], "flops": 3 * n * LATENT}
    B = case["B"]
    mean = min(case["k"] + case["window"], 2 * case["cap"])
    if case["ragged"]:  # lengths spread over their logarithm
        top = math.log(case["cap"] + 1)
        part = lambda k: (min(k, case["cap"]) + max(0.0, (top - math.log(k + 1)) * k)) / top  # noqa: E731
        mean = min(mean, part(case["k"]) + part(case["window"]))
    rows = B * mean
    return {"bytes": rows * ROW4 + B * (4 * HEADS * LATENT + 4 * HEADS + 4 * case["k"] + 8),
            "flops": 4 * rows * HEADS * LATENT}


# --- the definitions in 64 bits ---------------------------------------------------------------


def exact(case, seed):
    op = case["op"]
    if op == "plan":
        return None  # whole numbers
    s = prepare(case, seed)
    if op == "norm_rope":
        return [_exact_heads(case, s, x, w) for _, x, w, _ in s["parts"]]
    if op == "kv_rows":
        return _exact_rows(case, s)
    outs, lses = [], []
    for b in range(case["B"]):
        o, l = _exact_attention(case, s, b)
        outs.append(o)
        lses.append(l)
    return torch.stack(outs), torch.stack(lses)


def _exact_heads(case, s, x, w):
    n, heads, d = x.shape
    half, first = case["rope_dim"] // 2, d - case["rope_dim"]
    y = torch.empty((n, heads, d), dtype=torch.float64, device=x.device)
    angle = torch.outer(s["positions"].double(), s["inv_freq"])
    turn = torch.polar(torch.full_like(angle, s["scale"]), angle)
    if case["interleaved"]:
        re = torch.arange(half, device=x.device) * 2 + first
        im = re + 1
    else:
        re = torch.arange(half, device=x.device) + first
        im = re + half
    for h in range(heads):
        v = x[:, h].double()
        norm = torch.linalg.vector_norm(v, dim=1) ** 2 / d + 1e-6
        v = v / norm.sqrt()[:, None] * w.double()
        z = torch.complex(v[:, re], v[:, im]) * turn
        v[:, re], v[:, im] = z.real, z.imag
        y[:, h] = v
    return y


def _nearest(y, values):
    """The nearest of the ascending `values` (ties to the even place) with y's sign."""
    t = torch.tensor(values, dtype=torch.float64, device=y.device)
    mid = (t[1:] + t[:-1]) / 2
    low = torch.bucketize(y.abs(), mid)  # mid below y: counted
    tie = torch.zeros_like(y, dtype=torch.bool)
    inside = low < len(mid)
    tie[inside] = y.abs()[inside] == mid[low[inside]]
    low = low + (tie & (low % 2 == 1)).long()
    return t[low] * torch.sign(y)


def _power(e):
    """2^e in fp64, exactly."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_rows(case, s):
    out = torch.zeros((case["n"], LATENT), dtype=torch.float64, device=DEV)
    for at in range(0, case["n"], 8192):
        x = s["kv"][at:at + 8192].double()
        if case["fmt"] == "mxfp4":
            u = x.view(-1, 16, 32)
            top = u.abs().amax(dim=2, keepdim=True)
            f = _power(torch.where(top > 0, torch.frexp(top).exponent - 3, 0 * top))
            y = (_nearest(u / f, E2M1) * f).view(-1, LATENT)
        elif case["fmt"] == "e4m3":
            table = [m / 512 for m in range(8)]
            table += [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)]
            y = _nearest(x / KV_SCALE, table[:-1]) * KV_SCALE
        else:
            y = x
        out[at:at + 8192] = y
    return out * (s["slots"] >= 0)[:, None]


def _exact_attention(case, s, b):
    """Request b's heads, over the rows that count and no others."""
    tau = case["tau"] if case["tau"] > 0 else LATENT ** -0.5
    ids = s["token_ids"][b]
    ids = ids[ids >= 0].long()
    if case["page_rows"]:
        R = case["page_rows"]
        lat = s["latents"].view(-1, R, ROW4)[s["table"][b].long()[ids // R], ids % R]
    else:
        lat = s["latents"][b][ids]
    raw = torch.cat([s["swa"][b, :int(s["swa_len"][b])], lat])
    if raw.shape[0] == 0:
        zero = torch.zeros((HEADS, LATENT), dtype=torch.float64, device=DEV)
        return zero, torch.full((HEADS,), -math.inf, dtype=torch.float64, device=DEV)
    code = torch.empty((raw.shape[0], LATENT), dtype=torch.int64, device=DEV)
    code[:, 0::2] = (raw[:, :LATENT // 2] % 16).long()
    code[:, 1::2] = (raw[:, :LATENT // 2] // 16).long()
    e, m = (code // 2) % 4, (code % 2).double()  # the bits of an e2m1 code: sign, 2 of exponent, 1
    mag = torch.where(e == 0, m / 2, (1 + m / 2) * _power(e - 1))
    power = raw[:, LATENT // 2:].long().repeat_interleave(32, dim=1) - 127
    v = torch.where(code >= 8, -mag, mag) * _power(power)
    z = (s["q"][b].double() @ v.T) * tau
    lse = torch.logsumexp(z, dim=1)
    return torch.exp(z - lse[:, None]) @ v, lse
