"""A decode loop with a 4-bit paged cache, its calls together as a server makes them: the
step's plan, norms and rotation of the step's queries and keys, the cache rows, the
selection and the attention; prompts first (their queries through the bf16 prefill over
rows read back), then single tokens, with requests that end and start meanwhile.

The reference keeps every request's rows in float64 from its own norms and rotations.
What the GPU rounds differently (a bf16 key whose fp32 value lay near a border, so one 4-bit
code in some thousands) stays with the row: so the reference takes the cache's rows as the
library wrote them, after checking that each is the row it expects to within one step of the
format, and holds the attention over those rows to the attention's tolerance."""
import numpy as np
import pytest
import torch

import oracle as O
import two_tier_sparse_gb300 as dsa
from parity import check_ids, host_u16
from test_gpu_attn4 import check_attention
from test_gpu_serving import frequencies, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_device):
    from two_tier_sparse_gb300 import build
    build.build()
    dsa.load()
    torch.cuda.set_device(cuda_device)


class Server:
    """B request slots over one pool: what a program keeps between steps."""

    def __init__(self, B, R, per_seq, n_pages, max_new, k_tokens, window, graph=False):
        self.B, self.max_new, self.window, self.R, self.per_seq = B, max_new, window, R, per_seq
        self.cfg = dsa.config(k_blocks=4096, k_tokens=k_tokens, window=window, kv_fmt=dsa.KV_MXFP4)
        self.cap = R * per_seq
        z = dict(device="cuda")
        self.n = i32([0] * B)
        self.new = i32([0] * B)
        self.pool = dsa.PagePool.empty(B, R, per_seq, n_pages)
        self.plan = dsa.StepPlan.empty(B, max_new, n_tokens=self.n)
        pages = self.pool.pages()
        rows = n_pages * R
        self.latents = torch.zeros((rows, 272), dtype=torch.uint8, **z)
        self.swa = torch.zeros((B, window, 272), dtype=torch.uint8, **z)
        self.keys = dsa.Keys("bf16", torch.zeros((rows, 128), dtype=torch.bfloat16, **z), None, pages)
        self.pooled = dsa.Keys("bf16", torch.zeros((rows // 8, 128), dtype=torch.bfloat16, **z), None,
                               pages)
        self.ws = dsa.workspace(self.cfg, max(B, max_new), self.cap)
        bf = dict(dtype=torch.bfloat16, **z)
        self.q = torch.zeros((max_new, 64, 512), **bf)
        self.kv = torch.zeros((max_new, 512), **bf)
        self.q_idx = torch.zeros((max_new, 16, 128), **bf)
        self.k_idx = torch.zeros((max_new, 128), **bf)
        self.w = torch.zeros((B, 16), **z)
        g = torch.Generator(device="cuda").manual_seed(1)
        self.weights = [1 + 0.2 * torch.randn((d,), generator=g, **z) for d in (512, 512, 128, 128)]
        self.f = frequencies(32)
        self.rope = dsa.Rope(torch.tensor(self.f, **z))
        self.heads = dsa.HeadSet([  # in place
            dsa.Heads(self.q, weight=self.weights[0], rope_start=448),
            dsa.Heads(self.kv, weight=self.weights[1], rope_start=448),
            dsa.Heads(self.q_idx, weight=self.weights[2], rope_start=64),
            dsa.Heads(self.k_idx, weight=self.weights[3], rope_start=64)])
        self.out = torch.zeros((B, 64, 512), **bf)
        self.lse = torch.zeros((B, 64), **z)
        self.ids = i32(np.zeros((B, k_tokens)))

    def take(self, x):
        """The step's projections, packed in request order."""
        for t, v in zip((self.q, self.kv, self.q_idx, self.k_idx), x):
            t[:v.shape[0]] = v

    def make(self):
        """Plan, norms with rotation, window rows: the same for prompts and single tokens."""
        dsa.plan_step(self.cfg, self.n, self.new, self.pool, self.plan, self.ws)
        dsa.norm_rope(self.plan.positions, self.heads, self.rope, n_valid=self.plan.n_valid)
        dsa.kv_write(self.cfg, self.kv, self.plan.window_slots, self.swa, self.ws)

    def prompts(self):
        self.make()
        dsa.kv_write(self.cfg, self.kv, self.plan.latent_slots, self.latents, self.ws)
        there = self.plan.latent_slots >= 0
        self.keys.data[self.plan.latent_slots[there].long()] = self.k_idx[there]
        dsa.pool_index_keys(self.cfg, self.keys, self.plan.n_latents, self.cap, self.pooled, self.ws)

    def decode(self):
        """One token for every request (ratio 1: each completes a latent)."""
        self.make()
        B = self.B
        gate = torch.zeros((B, 1), device="cuda")
        dsa.compress_append(self.cfg, self.plan.n_tokens, self.kv[:B], gate,
                            dsa.Keys("bf16", self.k_idx[:B]), self.latents, self.keys, self.pooled,
                            self.cap, self.ws)
        dsa.decode_step(self.cfg, self.q[:B], self.q_idx[:B], self.w, self.keys, self.pooled,
                        self.latents, self.plan.n_latents, self.cap, self.swa, self.plan.swa_len,
                        self.out, self.ws, lse=self.lse, token_ids=self.ids)


def bits(t):
    return host_u16(t.view(torch.int16))


def near_rows(got, want_v, label):
    """got: 4-bit rows; want_v: the float64 values they were made from. A row is off its
    values by half a step of the code at the group's scale (at most 1 of 6 in units of
    2^(s - 127): between 4 and 6), or 2 where the top saturates (6 for values below 8), and
    the bf16 rounding of the value before it, 2^-8 of it."""
    v = O.latent_values(got, "mxfp4")
    step = np.ldexp(1.0, got[..., 256:].astype(np.int64) - 127).repeat(32, axis=-1)
    err = np.abs(v - want_v)
    assert np.all(err <= np.where(np.abs(want_v) > 6 * step, 2.0, 1.0) * step + 2.0 ** -7 * np.abs(want_v)), label


@pytest.mark.parametrize("captured", [False, True])
def test_a_decode_loop_over_a_four_bit_cache(captured):
    B, window, k_tokens = 5, 16, 48
    s = Server(B, 64, 6, 40, 256, k_tokens, window)
    rng = np.random.default_rng(3)
    want = [dict(lat=np.zeros((0, 512)), key=np.zeros((0, 128))) for _ in range(B)]

    def projections(total):
        g = torch.Generator(device="cuda").manual_seed(int(rng.integers(1 << 30)))
        return [torch.randn(sh, generator=g, device="cuda").bfloat16()
                for sh in ((total, 64, 512), (total, 512), (total, 16, 128), (total, 128))]

    def expect(x, counts, lengths):
        """The reference's normed, rotated rows, appended to each request's."""
        pos = np.concatenate([np.arange(n, n + c) for n, c in zip(lengths, counts)] or [[]])
        eps = float(np.float32(1e-6))
        outs = [O.norm_rope(v.double().cpu().numpy().reshape(len(pos), -1, d), w.double().cpu().numpy(),
                            eps, pos, s.f, start, True)
                for v, w, d, start in zip(x, s.weights, (512, 512, 128, 128), (448, 448, 64, 64))]
        at = 0
        for b, c in enumerate(counts):
            want[b]["lat"] = np.concatenate([want[b]["lat"], outs[1][at:at + c, 0]])
            want[b]["key"] = np.concatenate([want[b]["key"], outs[3][at:at + c, 0]])
            at += c
        return outs

    # prompts: requests 1 and 4 come later
    counts = [100, 0, 7, 65, 0]
    x = projections(sum(counts))
    s.take(x)
    s.new.copy_(i32(counts))
    expect(x, counts, [0] * B)
    s.prompts()
    assert dsa.read_device_status(s.ws)[0] == 0
    assert s.n.tolist() == counts

    # the first request's prompt attends through the bf16 prefill, over its rows read back
    n0 = counts[0]
    slots = s.plan.latent_slots[:n0].contiguous()
    back = torch.zeros((n0, 512), dtype=torch.bfloat16, device="cuda")
    dsa.kv_read(s.cfg, s.latents, slots, back, s.ws)
    bf = dsa.config(k_blocks=64, k_tokens=k_tokens, window=window)
    win = torch.zeros((n0 + window - 1, 512), dtype=torch.bfloat16, device="cuda")
    win[window - 1:] = back
    keys = s.keys.data[slots.long()].contiguous()
    pooled = dsa.Keys("bf16", torch.zeros((1, (n0 + 7) // 8, 128), dtype=torch.bfloat16, device="cuda"))
    ws = dsa.workspace(bf, n0, n0)
    dsa.pool_index_keys(bf, dsa.Keys("bf16", keys[None]), i32([n0]), n0, pooled, ws)
    out = torch.zeros((n0, 64, 512), dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros((n0, 64), device="cuda")
    tok = i32(np.zeros((n0, k_tokens)))
    dsa.sparse_attn_prefill(bf, 0, s.q[:n0], s.q_idx[:n0], torch.ones((n0, 16), device="cuda"), back,
                            dsa.Keys("bf16", keys), dsa.Keys("bf16", pooled.data[0]), win, out, ws,
                            lse=lse, token_ids=tok)
    assert dsa.read_device_status(ws)[0] == 0
    rows = s.latents[slots.long()].cpu().numpy()
    for i in (0, 20, n0 - 1):
        sel = tok[i].cpu().numpy()
        sel = sel[sel >= 0]
        check_attention(bits(s.q)[i], np.concatenate([rows[sel], rows[max(0, i - window + 1):i + 1]]),
                        bits(out)[i], lse[i].cpu().numpy().astype(np.float64), 512 ** -0.5, f"prefill {i}")

    # single tokens; request 2 ends at the third step and starts anew, request 1 joins
    graph = None
    for step in range(5):
        counts = [1] * B
        lengths = s.n.tolist()
        if step == 2:
            s.new.copy_(i32([0, 0, -1, 0, 0]))
            dsa.plan_step(s.cfg, s.n, s.new, s.pool, s.plan, s.ws)
            want[2] = dict(lat=np.zeros((0, 512)), key=np.zeros((0, 128)))
            lengths[2] = 0
            assert s.n.tolist() == lengths
        x = projections(B)
        s.take(x)
        s.new.copy_(i32(counts))
        s.w.copy_(torch.from_numpy(rng.random((B, 16), np.float32)))
        outs = expect(x, counts, lengths)
        if captured and step == 1:
            # the graph's own first pass must not count: capture runs nothing
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                s.decode()
        if graph is not None:
            graph.replay()
        else:
            s.decode()
        code, info = dsa.read_device_status(s.ws)
        assert code == 0, hex(info)
        table = s.pool.table.cpu().numpy()
        lat, keys = s.latents.cpu().numpy(), bits(s.keys.data)
        swa, ids = s.swa.cpu().numpy(), s.ids.cpu().numpy()
        q = O.bf16_to_f64(bits(s.q)[:B])
        assert np.abs(q - outs[0]).max() <= 2.0 ** -8 * np.abs(outs[0]).max()
        for b in range(B):
            n = lengths[b] + 1
            row = O.gather_paged(lat, table[b], 64, n)
            near_rows(row, want[b]["lat"], f"latents of {b} at step {step}")
            key = O.bf16_to_f64(O.gather_paged(keys, table[b], 64, n))
            assert np.all(np.abs(key - want[b]["key"]) <= 2.0 ** -8 * np.abs(want[b]["key"]) + 2.0 ** -16)
            w = min(n, window)
            recent = np.stack([swa[b, p % window] for p in range(n - w, n)])
            assert np.array_equal(recent, row[n - w:]), f"window of {b}"
            scores = O.index_scores(O.bf16_to_f64(bits(s.q_idx)[b]), s.w[b].cpu().numpy(), key)
            best = O.topk_ids(scores, np.arange(n), k_tokens)
            best = np.concatenate([best, np.full(k_tokens - len(best), -1)])[:k_tokens]
            check_ids(ids[b], best, lambda i: scores[i], k_tokens, f"ids of {b} at step {step}")
            sel = ids[b][ids[b] >= 0]
            check_attention(bits(s.q)[b], np.concatenate([row[sel], recent]), bits(s.out)[b],
                            s.lse[b].cpu().numpy().astype(np.float64), 512 ** -0.5,
                            f"attention of {b} at step {step}")
    assert s.n.tolist() == [105, 5, 3, 70, 5]
    held = sum(-(-n // 64) for n in s.n.tolist())
    head, tail = s.pool.ring_state.tolist()
    assert tail - head == 40 - held


@pytest.mark.parametrize("captured", [False, True])
def test_a_refused_step_of_the_loop_leaves_the_caches(captured):
    """Too few free pages for a step: the plan refuses it, and the calls behind it, whose counts and
    slots are the plan's, write no cache row either (the append takes 0 tokens for requests that got
    none). With the pages there, the same step is the one that was never refused."""
    B, R = 3, 64
    runs = []
    for refuse in (True, False):
        s = Server(B, R, 3, 12, 200, 16, 8)
        g = torch.Generator(device="cuda").manual_seed(5)

        def projections(total):
            return [torch.randn(sh, generator=g, device="cuda").bfloat16()
                    for sh in ((total, 64, 512), (total, 512), (total, 16, 128), (total, 128))]

        def decode():
            s.make()
            grown = s.plan.n_tokens * (s.plan.cu_new[1:] > s.plan.cu_new[:-1])
            dsa.compress_append(s.cfg, grown, s.kv[:B], gate, dsa.Keys("bf16", s.k_idx[:B]), s.latents,
                                s.keys, s.pooled, s.cap, s.ws)
            dsa.decode_step(s.cfg, s.q[:B], s.q_idx[:B], s.w, s.keys, s.pooled, s.latents,
                            s.plan.n_latents, s.cap, s.swa, s.plan.swa_len, s.out, s.ws, lse=s.lse,
                            token_ids=s.ids)
        gate = torch.zeros((B, 1), device="cuda")
        s.take(projections(64 + 10 + 100))
        s.new.copy_(i32([64, 10, 100]))  # the first request's page is full
        s.prompts()
        s.new.copy_(i32([1] * B))
        x = projections(B)
        s.take(x)
        step = decode
        if captured:
            decode()  # (sets limits; taken back below)
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                decode()
            step = graph.replay
            s.n.sub_(1)
            s.pool.ring_state[0] -= 1
            s.take(x)
        if refuse:
            state = s.pool.ring_state.clone()
            s.pool.ring_state[0] = state[1]  # no page is free
            caches = (s.latents, s.swa, s.keys.data, s.pooled.data, s.pool.table, s.n)
            before = [t.clone() for t in caches]
            step()
            assert dsa.read_device_status(s.ws)[0] == 6
            for t, b in zip(caches, before):
                assert torch.equal(t, b)
            s.pool.ring_state.copy_(state)
            s.take(x)
        step()
        assert dsa.read_device_status(s.ws)[0] == 0
        assert s.n.tolist() == [65, 11, 101]
        runs.append([t.clone() for t in (s.out, s.lse, s.ids, s.latents, s.swa, s.pooled.data)])
    for a, b in zip(*runs):
        assert torch.equal(a, b)
