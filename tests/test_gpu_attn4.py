"""Attention over a 4-bit cache on the GPU against the oracle's attention over the
same rows' values in float64.

Tolerance, for each output o = sum_j p_j v_j / sum_j p_j with |v| weighted alike,
A = sum_j p_j |v_j| / sum_j p_j:
  * the output's rounding to bf16: 2^-8 |o|;
  * the probabilities' rounding to bf16 before the product: 2^-8 A;
  * a score off by dz moves its probability by a factor within e^(+-dz), and the sum by
    as much: 2 dz A. A score is an fp32 sum of 512 products of bf16 values (exact ones),
    at most 512 roundings (the tensor cores round towards zero: whole steps, 2^-23) of
    partial sums below tau sum |q k|, and one of its product with tau log2(e):
    dz = 2^-14 tau sum |q k| + 2^-22 |z|;
  * exp2, sums of up to 640 terms, the exchanged 24-bit parts and the merge:
    2^-12 A covers 640 sums at 2^-24 in O^T (2^-14.7), 2^-16 and a few 2^-22.
  * 2^x flushes below 2^-126: a probability under 2^-126 of the running maximum is 0, and
    that maximum is within 2^8 of the sum's largest term, so up to 640 terms of at most
    2^-118 each may be missing: 2^-108 max |v|, absolute.
The log-sum-exp is off by at most dz and 2^-16 (1 + |lse|)."""
import numpy as np
import pytest
import torch

import oracle as O
import synth
import two_tier_sparse_gb300 as dsa
from parity import DecodeOnDevice, dev, host_u16
from test_gpu_parity import check_step, run_step
from test_gpu_paged import PagedOnDevice

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_device):
    from two_tier_sparse_gb300 import build
    build.build()
    dsa.load()
    torch.cuda.set_device(cuda_device)


def rows4(rng, n, spread=0.0, gain=1.0):
    v = rng.standard_normal((n, 512)) * gain
    if spread:
        v = v * np.exp2(rng.integers(-spread, spread + 1, (n, 16))).repeat(32, axis=1)
    return O.latent_rows_mxfp4(v.astype(np.float32))


def check_attention(q_bits, rows, out_bits, lse, tau, label=""):
    q = O.bf16_to_f64(q_bits)
    got = O.bf16_to_f64(out_bits)
    if rows.shape[0] == 0:
        assert not got.any() and np.all(np.isneginf(lse)), label
        return
    v = O.latent_values(rows, "mxfp4")
    z = tau * (q @ v.T)
    zmax = z.max(axis=1, keepdims=True)
    p = np.exp(z - zmax)
    L = p.sum(axis=1, keepdims=True)
    o, A = p @ v / L, p @ np.abs(v) / L
    ref_lse = (np.log(L) + zmax)[:, 0]
    dz = (2.0 ** -14 * tau * (np.abs(q) @ np.abs(v).T) + 2.0 ** -22 * np.abs(z)).max(axis=1)
    tol = 2.0 ** -8 * np.abs(o) + (2.0 ** -8 + 2.0 ** -12 + 2 * dz[:, None]) * A \
        + 2.0 ** -108 * np.abs(v).max()
    err = np.abs(got - o)
    assert np.all(err <= tol), f"{label}: {(err / np.maximum(tol, 1e-300)).max():.3g} of the tolerance"
    assert np.all(np.abs(lse - ref_lse) <= dz + 2.0 ** -16 * (1 + np.abs(ref_lse))), label
    # and it is those rows, not merely something small
    assert ((got - o) ** 2).sum() <= 1e-4 * (o ** 2).sum() + 1e-30, label


class Case:
    """B sequences of n latents (a list) with k selected ids each, in 272-byte rows."""

    def __init__(self, n, k_tokens, window, seed, tau=0.0, q_scale=1.0, spread=0, swa=None,
                 stride=None, page_rows=0):
        rng = np.random.default_rng(seed)
        B = len(n)
        self.B, self.n, self.window = B, np.asarray(n, np.int32), window
        self.tau = tau if tau > 0 else 512 ** -0.5
        self.cfg = dsa.config(k_tokens=k_tokens, window=window, sm_scale=tau, kv_fmt=dsa.KV_MXFP4)
        self.q = O.f32_to_bf16_rne((rng.standard_normal((B, 64, 512)) * q_scale).astype(np.float32))
        self.swa_len = np.asarray([min(window, x) for x in n] if swa is None else swa, np.int32)
        cap = max(max(n), 1) if stride is None else stride
        # rows that no query may read: NaN scales, so that reading one shows
        self.latents = np.full((B, cap, 272), 255, np.uint8)
        self.swa = np.full((B, window, 272), 255, np.uint8)
        self.ids = np.full((B, k_tokens), -1, np.int32)
        for b in range(B):
            m = min(k_tokens, int(self.n[b]))
            pick = np.sort(rng.choice(int(self.n[b]), m, replace=False)) if m else []
            self.ids[b, :m] = pick
            self.latents[b, pick] = rows4(rng, m, spread)
            self.swa[b, :self.swa_len[b]] = rows4(rng, int(self.swa_len[b]), spread)
        self.page_rows = page_rows
        self.ws = dsa.workspace(self.cfg, B, 0)
        if page_rows:
            pad = -(-cap // page_rows) * page_rows
            lat = np.full((B, pad, 272), 255, np.uint8)
            lat[:, :cap] = self.latents
            pool, self.table = synth.paginate(lat, page_rows, seed)
            self.pages = dsa.Pages(dev(self.table), page_rows, pool.shape[0] // page_rows)
            self.dlat = dev(pool)
        else:
            self.dlat = dev(self.latents)

    def run(self, **over):
        a = dict(q=self.q, n=self.n, ids=self.ids, swa=self.swa, swa_len=self.swa_len)
        a = {k: over[k] if k in over else dev(x) for k, x in a.items()}
        out = torch.full((self.B, 64, 512), 0x7FC0, dtype=torch.int16, device="cuda")
        lse = torch.full((self.B, 64), float("nan"), device="cuda")
        if self.page_rows:
            dsa.sparse_attn_decode_paged(self.cfg, a["q"], self.dlat, self.pages, a["n"], a["ids"],
                                         a["swa"], a["swa_len"], out, self.ws, lse=lse)
        else:
            dsa.sparse_attn_decode(self.cfg, a["q"], self.dlat, a["n"], a["ids"], a["swa"],
                                   a["swa_len"], out, self.ws, lse=lse)
        return out, lse

    def rows(self, b):
        ids = self.ids[b][self.ids[b] >= 0]
        return np.concatenate([self.latents[b][ids], self.swa[b, :self.swa_len[b]]])

    def check(self, out, lse, seqs=None, label=""):
        o, l = host_u16(out), lse.cpu().numpy().astype(np.float64)
        for b in range(self.B) if seqs is None else seqs:
            check_attention(self.q[b], self.rows(b), o[b], l[b], self.tau, f"{label} seq {b}")


@pytest.mark.parametrize("n,k,window", [
    ([2048], 512, 128),                 # one sequence: eight CTAs
    ([1], 1, 1),                        # two rows
    ([1], 512, 128),                    # one latent, one window row
    ([63], 64, 1), ([64], 64, 64), ([65], 512, 127), ([700], 511, 3),
    ([5000, 0, 3, 129, 640], 512, 128),  # an empty sequence, ragged ones
    ([33] * 19, 40, 17), ([900] * 20, 512, 128), ([300] * 38, 129, 128),
    ([777] * 39, 512, 128), ([600] * 64, 512, 128), ([200] * 76, 100, 128),
    ([600] * 77, 512, 128), ([500, 0, 7] * 51, 512, 128), ([150] * 310, 64, 5),
])
def test_attention_over_four_bit_rows(n, k, window):
    c = Case(n, k, window, seed=len(n) + k)
    out, lse = c.run()
    assert dsa.read_device_status(c.ws)[0] == 0
    c.check(out, lse, seqs=range(len(n)) if len(n) < 80 else list(range(0, len(n), 7)) + [len(n) - 1])


@pytest.mark.parametrize("B", [2, 25, 50, 100])
def test_sharp_softmax_and_scales_far_apart(B):
    """Scores up to tens (the running maximum moves between tiles and differs between
    CTAs), scales of one row up to 2^12 apart, a dominant row in the last tile."""
    rng = np.random.default_rng(B)
    c = Case([int(x) for x in rng.integers(300, 2000, B)], 512, 128, seed=B, tau=0.05, q_scale=2.0,
             spread=6)
    for b in range(0, B, 3):
        q = O.bf16_to_f64(c.q[b, b % 64])
        last = c.ids[b][c.ids[b] >= 0][-1]
        c.latents[b, last] = O.latent_rows_mxfp4((q * 6).astype(np.float32)[None])[0]
    c.dlat = dev(c.latents)
    out, lse = c.run()
    c.check(out, lse, seqs=range(min(B, 30)))
    assert dsa.read_device_status(c.ws)[0] == 0


def test_ids_in_any_order_repeated_and_missing():
    """Ids need no order; a repeated id counts as often as it is given; -1 anywhere
    is skipped."""
    c = Case([400, 90, 10], 96, 7, seed=3)
    rng = np.random.default_rng(8)
    for b in range(3):
        ids = c.ids[b][c.ids[b] >= 0]
        c.ids[b] = rng.choice(np.concatenate([ids, [-1] * 20, ids[:1].repeat(9)]), 96)
    c.ids[2] = -1
    out, lse = c.run()
    c.check(out, lse)
    assert dsa.read_device_status(c.ws)[0] == 0


def test_no_rows_at_all():
    c = Case([0, 0, 50], 64, 16, seed=4, swa=[0, 3, 0])
    out, lse = c.run()
    c.check(out, lse)
    assert not out[0].any() and bool(torch.isneginf(lse[0]).all())


def test_bad_ids_lengths_and_pages_are_skipped_and_reported():
    c = Case([100, 60, 80], 64, 8, seed=5)
    ids = c.ids.copy()
    ids[0, 5], ids[2, 0] = 100, 2 ** 31 - 1     # past the sequence
    c2 = dict(ids=dev(ids))
    out, lse = c.run(**c2)
    code, info = dsa.read_device_status(c.ws)
    assert code == 6 and info >> 24 == 4
    c.ids = np.where(ids >= c.n[:, None], -1, ids)
    c.check(out, lse)
    # window lengths outside [0, window]
    out, lse = c.run(swa_len=dev(np.array([-1, 9, 8], np.int32)))
    assert dsa.read_device_status(c.ws)[0] == 6
    c.swa_len[0] = 0
    c.check(out, lse)
    # a page outside the pool
    p = Case([300, 200], 64, 8, seed=6, page_rows=64)
    t = p.table.copy()
    t[0, 1], t[1, 0] = -1, p.pages.c.n_pages
    p.pages = dsa.Pages(dev(t), 64, p.pages.c.n_pages)
    out, lse = p.run()
    assert dsa.read_device_status(p.ws)[0] == 6
    for b, page in ((0, 1), (1, 0)):
        p.ids[b] = np.where(p.ids[b] // 64 == page, -1, p.ids[b])
    p.check(out, lse)


@pytest.mark.parametrize("page_rows", [64, 128, 192])
def test_paged_equals_contiguous(page_rows):
    n = [1000, 64, 0, 65, 5, 777]
    a, b = Case(n, 512, 100, seed=9), Case(n, 512, 100, seed=9, page_rows=page_rows)
    for x, y in zip(a.run(), b.run()):
        assert torch.equal(x, y)
    assert dsa.read_device_status(b.ws)[0] == 0


def test_scales_at_the_ends_and_nan():
    """Scale bytes 0 (2^-127) and 252 (2^125, values up to 1.5 * 2^127) are exact; 255 is
    NaN, and stays with the queries that read it."""
    c = Case([40, 40, 40], 40, 4, seed=10, tau=1.0)
    code = np.full(256, 0x22, np.uint8)  # every element 1.0
    for b in range(3):
        c.latents[b, :40] = 0
        c.latents[b, :40, :256] = code
        c.swa[b, :4] = 0
        c.swa[b, :4, :256] = code
        c.q[b] = 0
    c.latents[1, :40, 256:] = 252
    c.swa[1, :4, 256:] = 252
    c.latents[2, 7, 256 + 3] = 255
    c.dlat = dev(c.latents)
    out, lse = c.run()
    got = out.view(torch.bfloat16).float()
    # 44 equal probabilities of equal rows; a probability's rounding does not show (1)
    assert bool((got[0] == 2.0 ** -127).all())
    assert bool((got[1] == 2.0 ** 125).all())
    bad = torch.zeros(512, dtype=torch.bool, device="cuda")
    bad[96:128] = True
    assert bool(got[2].isnan().any())
    assert not got[0].isnan().any() and not got[1].isnan().any()


def test_rows_past_two_to_the_31_bytes():
    """A cache of more than 2^31 bytes whose selected rows lie at both ends."""
    B, cap = 3, 2_700_000
    cfg = dsa.config(k_tokens=64, window=2, kv_fmt=dsa.KV_MXFP4)
    lat = torch.full((B, cap, 272), 255, dtype=torch.uint8, device="cuda")
    assert lat.numel() > 2 ** 31
    rng = np.random.default_rng(11)
    ids = np.stack([np.sort(np.concatenate([rng.choice(1000, 30, replace=False),
                                            cap - 1 - rng.choice(1000, 34, replace=False)]))
                    for _ in range(B)]).astype(np.int32)
    rows = rows4(rng, B * 64).reshape(B, 64, 272)
    for b in range(B):
        lat[b, dev(ids[b]).long()] = dev(rows[b])
    swa = rows4(rng, B * 2).reshape(B, 2, 272)
    q = O.f32_to_bf16_rne(rng.standard_normal((B, 64, 512)).astype(np.float32))
    out = torch.empty((B, 64, 512), dtype=torch.int16, device="cuda")
    lse = torch.empty((B, 64), device="cuda")
    ws = dsa.workspace(cfg, B, 0)
    dsa.sparse_attn_decode(cfg, dev(q), lat, dev(np.full(B, cap, np.int32)), dev(ids), dev(swa),
                           dev(np.full(B, 2, np.int32)), out, ws, lse=lse)
    assert dsa.read_device_status(ws)[0] == 0
    for b in range(B):
        check_attention(q[b], np.concatenate([rows[b], swa[b]]), host_u16(out)[b],
                        lse.cpu().numpy()[b].astype(np.float64), 512 ** -0.5, b)


def to_four_bits(inp):
    """The batch with its latents and window rows in the 4-bit format."""
    def enc(bits):
        v = O.bf16_to_f64(bits)
        v = np.where(np.isfinite(v), v, 0.0).astype(np.float32)
        return O.latent_rows_mxfp4(v)
    inp.latents, inp.swa, inp.kv_fmt = enc(inp.latents), enc(inp.swa), "mxfp4"
    return inp


@pytest.mark.parametrize("T,ratio,fmt,k_blocks,page_rows", [
    ([4096], 2, "bf16", 2048, 0),
    ([20000, 9001, 777, 64, 3], 1, "mxfp4", 128, 0),
    ([9000, 777, 64, 3], 1, "mxfp8", 128, 64),
    ([700] * 66, 2, "mxfp4", 20, 128),
])
def test_decode_step_with_a_four_bit_cache(T, ratio, fmt, k_blocks, page_rows):
    inp = to_four_bits(synth.decode_inputs(T, ratio, fmt, seed=70, q_scale=8.0))
    cfg = dsa.config(k_blocks=k_blocks, ratio=ratio, sm_scale=8.0, kv_fmt=dsa.KV_MXFP4)
    d = DecodeOnDevice(inp, cfg)
    d.pool()
    outs = run_step(d, cfg)
    assert d.status()[0] == 0
    check_step(inp, cfg, outs, range(min(len(T), 6)))
    if page_rows:
        p = PagedOnDevice(inp, cfg, page_rows, seed=71)
        p.pool()
        for x, y in zip(p.step(), outs):
            assert torch.equal(x, y)


def test_same_bits_each_time_in_a_graph_and_on_two_streams():
    a, b = Case([900] * 40, 512, 128, seed=20), Case([500] * 90, 300, 128, seed=21)
    want = [c.run() for c in (a, b)]
    torch.cuda.synchronize()
    for c, w in zip((a, b), want):
        for x, y in zip(c.run(), w):
            assert torch.equal(x, y)
    # two calls at once, each with its own workspace
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for c, s in zip((a, b), streams):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            for _ in range(5):
                r = c.run()
            got.append(r)
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert all(torch.equal(x, y) for x, y in zip(g, w))
    # replayed with another query in the captured buffer
    q, ids, n, swa, sl = (dev(x) for x in (a.q, a.ids, a.n, a.swa, a.swa_len))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = a.run(q=q, ids=ids, n=n, swa=swa, swa_len=sl)
    graph.replay()
    assert torch.equal(out, want[0][0]) and torch.equal(lse, want[0][1])
    q.copy_(dev(a.q[::-1].copy()))
    graph.replay()
    a.q = a.q[::-1].copy()
    a.check(out, lse, seqs=[0, 17, 39])


@pytest.mark.parametrize("ratio,page_rows", [(1, 0), (2, 64), (4, 0)])
def test_append_to_a_four_bit_cache(ratio, page_rows):
    """The pooled latent in the 4-bit format: for ratio 1 exactly the row's conversion; else
    the fp32 sum (ratio terms, a softmax weight each: within 2^-20 of the float64 one)
    may round to the neighbouring code where float64 lies that near a border."""
    T = np.array([4096, 1001, 64, 4, 17, 0], np.int64)
    B = len(T)
    inp = to_four_bits(synth.decode_inputs(T, ratio, "mxfp8", seed=90))
    cap = inp.cap
    kv = synth.normal_bf16(91, 4, 0, B * ratio * 512, 1 / np.sqrt(512)).reshape(B, ratio, 512)
    gate = (synth.uniform_f32(91, 3, 0, B * ratio) * 8 - 4).reshape(B, ratio)
    nk, ns = synth.normal_mxfp8(92, 9, 0, B, 128, 1 / np.sqrt(128))
    cfg = dsa.config(ratio=ratio, kv_fmt=dsa.KV_MXFP4)
    if page_rows:
        p = PagedOnDevice(inp, cfg, page_rows, seed=93)
        keys, pooled, latents, ws = p.keys, p.pooled, p.latents, p.ws

        def logical(t, b, rows):
            return O.gather_paged(t.cpu().numpy(), p.table_h[b], page_rows, rows)
    else:
        d = DecodeOnDevice(inp, cfg)
        keys, pooled, latents, ws = d.keys, d.pooled, d.latents, d.ws

        def logical(t, b, rows):
            return t.cpu().numpy()[b, :rows]
    before = latents.clone()
    dsa.compress_append(cfg, dev(T.astype(np.int32)), dev(kv), dev(gate),
                        dsa.Keys("mxfp8", dev(nk), dev(ns)), latents, keys, pooled, cap, ws)
    assert dsa.read_device_status(ws)[0] == 0
    for b in range(B):
        n = int(T[b]) // ratio
        got, was = logical(latents, b, max(n, 1)), logical(before, b, max(n, 1))
        if T[b] == 0 or T[b] % ratio:
            assert np.array_equal(got, was)
            continue
        assert np.array_equal(got[:n - 1], was[:n - 1])
        w = np.exp(gate[b].astype(np.float64) - gate[b].max())
        exact = ((w / w.sum())[:, None] * O.bf16_to_f64(kv[b])).sum(axis=0)
        if ratio == 1:
            assert np.array_equal(got[n - 1], O.latent_rows_mxfp4(exact.astype(np.float32)))
        lo = O.latent_values(O.latent_rows_mxfp4((exact - 2.0 ** -20 * np.abs(exact)).astype(np.float32)),
                             "mxfp4")
        hi = O.latent_values(O.latent_rows_mxfp4((exact + 2.0 ** -20 * np.abs(exact)).astype(np.float32)),
                             "mxfp4")
        v = O.latent_values(got[n - 1], "mxfp4")
        assert np.all((v == lo) | (v == hi)), b


@pytest.mark.parametrize("B", [1, 3, 20, 40, 77, 160])  # eight, four and two CTAs a sequence, one
@pytest.mark.parametrize("place", ["latent", "window"])
def test_a_nan_row_makes_every_head_of_its_sequence_nan(B, place):
    """Every score against a NaN row is NaN, and so are each head's sum, its output in every
    dim and its log-sum-exp; the other sequences are as without it."""
    c = Case([300 + b % 3 for b in range(B)], 200, 64, seed=B)
    want = c.run()
    hit = sorted({0, B // 2, B - 1})
    for b in hit:
        if place == "latent":
            c.latents[b, c.ids[b, (7 * b + 150) % 200], 256 + b % 16] = 255
        else:
            c.swa[b, (5 * b + 3) % 64, 256 + b % 16] = 255
    c.dlat = dev(c.latents)
    out, lse = c.run()
    got = out.view(torch.bfloat16)
    keep = [b for b in range(B) if b not in hit]
    assert bool(got[hit].isnan().all()) and bool(lse[hit].isnan().all())
    assert torch.equal(out[keep], want[0][keep]) and torch.equal(lse[keep], want[1][keep])
    assert not bool(want[0].view(torch.bfloat16).isnan().any()) and bool(want[1].isfinite().all())
    assert dsa.read_device_status(c.ws)[0] == 0


@pytest.mark.parametrize("B", [1, 20, 77, 160])
def test_a_head_of_nan_stays_with_itself(B):
    c = Case([300] * B, 200, 64, seed=B)
    want = c.run()
    hit = sorted({0, B - 1})
    for b in hit:
        c.q[b, 5, 17], c.q[b, 40, 0] = 0x7FC0, 0x7F80  # NaN, and an infinite element
    out, lse = c.run()
    got = out.view(torch.bfloat16)
    rest = [h for h in range(64) if h not in (5, 40)]
    for b in range(B):
        if b in hit:
            assert bool(got[b, [5, 40]].isnan().all()) and bool(lse[b, [5, 40]].isnan().all())
        else:
            assert torch.equal(out[b], want[0][b])
        assert torch.equal(out[b, rest], want[0][b, rest]) and torch.equal(lse[b, rest], want[1][b, rest])
