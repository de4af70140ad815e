"""Host-side argument checks of the step plan, the norms with rotation, the cache rows and
the 4-bit cache (no compute call runs here: every case stops in a check, or has
nothing to do)."""
import ctypes

import pytest
import torch

import two_tier_sparse_gb300 as dsa
from two_tier_sparse_gb300 import build as dsa_build

A = 1 << 12  # a fake device address, 256-byte aligned; never dereferenced


@pytest.fixture(scope="module")
def lib():
    dsa_build.build()
    return dsa.load()


def ref(x):
    return ctypes.byref(x) if x is not None else None


def test_four_bit_cache_is_a_format_of_the_decode_calls(lib):
    cfg = dsa.config(kv_fmt=dsa.KV_MXFP4)

    def decode(c, B):
        return lib.dsa_sparse_attn_decode(ref(c), A, A, 100, A, A, A, A, B, A, None, A, 1 << 30, None)
    assert decode(cfg, 0) == 0
    assert decode(dsa.config(kv_fmt=dsa.KV_MXFP4, kv_scale=float("nan")), 0) == 0  # not used
    for bad in (-1, 2, 4):
        assert decode(dsa.config(kv_fmt=bad), 0) == 1
    k = dsa._Keys(0, A, None, 100)
    p = dsa._Keys(0, A, None, 13)
    assert lib.dsa_sparse_attn_prefill(ref(cfg), 4, 96, A, A, A, A, ref(k), ref(p), A, A, None,
                                       None, A, 1 << 30, None) == 3
    assert lib.dsa_decode_multi(ref(cfg), 2, A, A, A, A, ref(k), ref(p), A, 100, 100, A, 1, A,
                                None, None, A, 1 << 30, None) == 3
    # the append takes 4-bit latents (B = 0: nothing to do) and still no E4M3 ones
    def append(c):
        return lib.dsa_compress_append(ref(c), 0, A, A, A, ref(k), A, 100, ref(k), ref(p), 100, A,
                                       1 << 30, None)
    assert append(cfg) == 0
    assert append(dsa.config(kv_fmt=dsa.KV_FP8_E4M3)) == 3


def test_plan_argument_errors(lib):
    cfg = dsa.config()

    def call(c=cfg, B=2, n=A, new=A, ws=A, wsb=256, pool=True, plan=True, **over):
        pl = dict(page_table=A, page_rows=64, pages_per_seq=4, n_pages=8, free_ring=A,
                  ring_state=A, ring_state_out=A)
        st = dict(n_tokens=A, n_latents=A, swa_len=A, cu_new=A, token_seq=A, positions=A,
                  latent_slots=A, window_slots=A, max_new=0)
        for k, v in over.items():
            (pl if k in pl else st)[k] = v
        return lib.dsa_plan_step(ref(c), B, n, new, ref(dsa._PagePool(**pl)) if pool else None,
                                 ref(dsa._StepPlan(**st)) if plan else None, ws, wsb, None)
    assert call(pool=False) == 1
    assert call(plan=False) == 1
    assert call(n=None) == 1
    assert call(new=None) == 1
    assert call(B=-1) == 1
    assert call(B=4097) == 3
    for f in ("page_table", "free_ring", "ring_state", "ring_state_out"):
        assert call(**{f: None}) == 1, f
        assert call(**{f: A + 2}) == 2, f
    assert call(ring_state=A + 4) == 2
    for f in ("n_tokens", "n_latents", "swa_len", "cu_new"):
        assert call(**{f: None}) == 1, f
        assert call(**{f: A + 2}) == 2, f
    for f in ("token_seq", "positions", "latent_slots", "window_slots"):
        assert call(max_new=5, **{f: None}) == 1, f
        assert call(max_new=5, **{f: A + 4}) == 2, f
    for over in (dict(page_rows=0), dict(page_rows=96), dict(pages_per_seq=0), dict(n_pages=0),
                 dict(n_pages=1 << 25), dict(n_pages=1 << 62), dict(max_new=-1),
                 dict(max_new=(1 << 30) + 1)):
        assert call(**over) == 1, over
    assert call(ws=None) == 4
    assert call(wsb=8) == 4
    assert call(ws=A + 16) == 2
    assert call(c=dsa.config(window=0)) == 1


def test_norm_rope_argument_errors(lib):
    def call(n=4, pos=A, dt=0, rope=dict(inv_freq=A, rope_dim=64, interleaved=1, scale=1.0),
             n_valid=None, groups=1, **over):
        h = dict(x=A, out=A, heads=2, dim=128, x_token_stride=256, x_head_stride=128,
                 out_token_stride=256, out_head_stride=128, weight=A, eps=1e-6, norm=1, rope_start=64)
        h.update(over)
        arr = (dsa._HeadsC * 9)(*[dsa._HeadsC(**h)] * 9)
        return lib.dsa_norm_rope(n, n_valid, pos, dt, arr if groups else None, abs(groups),
                                 ref(dsa._RopeC(**rope)) if rope else None, None)
    assert call(n=0) == 0
    assert call(n=0, heads=0) == 0
    assert call(heads=0) == 0  # nothing to do
    assert call(groups=0) == 0
    assert call(n=-1) == 1
    assert call(dt=3) == 1
    assert call(groups=9) == 3
    assert call(x=None) == 1
    assert call(out=None) == 1
    assert call(heads=-1) == 1
    for d in (0, 4, 12, 1032):
        assert call(dim=d, rope_start=-1) == 1, d
    assert call(x=A + 2) == 2
    assert call(out=A + 8) == 2
    assert call(weight=A + 4) == 2
    assert call(x_token_stride=252) == 2
    assert call(out_head_stride=132) == 2
    assert call(dt=2, x_head_stride=130) == 2
    assert call(out_token_stride=512) == 1         # in place with other strides
    assert call(x=2 * A, out_head_stride=0) == 1   # heads written over one another
    assert call(x=2 * A, out_token_stride=120) == 1
    assert call(x=2 * A, out_head_stride=-128) == 1
    assert call(eps=-1.0) == 1
    assert call(eps=float("nan")) == 1
    assert call(eps=float("inf")) == 1
    assert call(rope_start=4) == 1
    assert call(rope_start=72) == 1                # past the head's end
    assert call(rope=None) == 1                    # a group rotates, and there is no rotation
    assert call(pos=None) == 1
    assert call(pos=A + 2) == 2
    assert call(n_valid=A + 1) == 2

    def rope(**o):
        return dict(dict(inv_freq=A, rope_dim=64, interleaved=1, scale=1.0), **o)
    assert call(rope=rope(inv_freq=None)) == 1
    assert call(rope=rope(inv_freq=A + 4)) == 2
    assert call(rope=rope(rope_dim=0)) == 1
    assert call(rope=rope(rope_dim=12)) == 1
    assert call(rope=rope(rope_dim=24, interleaved=0)) == 1
    assert call(rope=rope(rope_dim=1032)) == 1
    assert call(rope=rope(scale=float("nan"))) == 1
    assert call(rope=rope(), n=0) == 0


@pytest.mark.parametrize("name", ["write", "read"])
def test_cache_row_argument_errors(lib, name):
    def call(c=dsa.config(kv_fmt=dsa.KV_MXFP4), n=3, nv=None, rows=A, stride=512, slots=A, cache=A,
             n_rows=100, ws=A, wsb=256):
        if name == "write":
            return lib.dsa_kv_write(ref(c), n, nv, rows, stride, slots, cache, n_rows, ws, wsb, None)
        return lib.dsa_kv_read(ref(c), n, nv, cache, n_rows, slots, rows, stride, ws, wsb, None)
    assert call(n=0) == 0
    assert call(n=-1) == 1
    assert call(rows=None) == 1
    assert call(slots=None) == 1
    assert call(cache=None) == 1
    assert call(n_rows=-1) == 1
    assert call(n_rows=1 << 31) == 1
    assert call(stride=504) == 1
    assert call(stride=516) == 2
    assert call(rows=A + 8) == 2
    assert call(cache=A + 8) == 2
    assert call(slots=A + 2) == 2
    assert call(nv=A + 2) == 2
    assert call(ws=None) == 4
    assert call(wsb=4) == 4
    assert call(ws=A + 16) == 2
    assert call(c=dsa.config(kv_fmt=2)) == 1
    assert call(c=dsa.config(kv_fmt=dsa.KV_FP8_E4M3, kv_scale=0.0)) == 1


def test_binding_refuses_what_it_cannot_pass(lib):
    i = dict(dtype=torch.int32)
    with pytest.raises(ValueError):
        dsa.PagePool(torch.zeros((2, 4)), 64, torch.zeros(8, **i), torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError):
        dsa.PagePool(torch.zeros((2, 4), **i), 64, torch.zeros(8, **i), torch.zeros(2, **i))
    with pytest.raises(ValueError):
        dsa.PagePool(torch.zeros((4, 2), **i).T, 64, torch.zeros(8, **i),
                     torch.zeros(2, dtype=torch.int64))
    t = [torch.zeros(3, **i) for _ in range(8)]
    with pytest.raises(ValueError):
        dsa.StepPlan(*t)  # cu_new has B + 1 entries
    plan = dsa.StepPlan.empty(3, 16, device="cpu")
    pool = dsa.PagePool.empty(3, 64, 4, 8, device="cpu")
    with pytest.raises(ValueError):
        dsa.plan_step(dsa.config(), torch.zeros(2, **i), torch.zeros(2, **i), pool, plan, None)
    x = torch.zeros((4, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        dsa.Heads(x.double())
    with pytest.raises(ValueError):
        dsa.Heads(x, out=torch.zeros((4, 2, 64)))
    with pytest.raises(ValueError):
        dsa.Heads(x.transpose(1, 2))
    with pytest.raises(ValueError):
        dsa.Heads(x, weight=torch.zeros(32))
    with pytest.raises(ValueError):
        dsa.HeadSet([])
    with pytest.raises(ValueError):
        dsa.HeadSet([dsa.Heads(x), dsa.Heads(torch.zeros((3, 2, 64), dtype=torch.bfloat16))])
    with pytest.raises(ValueError):
        dsa.Rope(torch.zeros(32))
    hs = dsa.HeadSet([dsa.Heads(x)])
    with pytest.raises(ValueError):
        dsa.norm_rope(torch.zeros(3, **i), hs)
    c = dsa.config(kv_fmt=dsa.KV_MXFP4)
    rows, cache = torch.zeros((3, 512), dtype=torch.bfloat16), torch.zeros((9, 272), dtype=torch.uint8)
    slots = torch.zeros(3, **i)
    for bad in (dict(rows=rows.float()), dict(rows=rows[:, :256]), dict(slots=slots.long()),
                dict(slots=slots[:2]), dict(cache=torch.zeros((9, 256), dtype=torch.uint8)),
                dict(n_valid=torch.zeros(2, **i))):
        kw = dict(dict(rows=rows, slots=slots, cache=cache, n_valid=None), **bad)
        with pytest.raises(ValueError):
            dsa.kv_write(c, kw["rows"], kw["slots"], kw["cache"], None, n_valid=kw["n_valid"])
        with pytest.raises(ValueError):
            dsa.kv_read(c, kw["cache"], kw["slots"], kw["rows"], None, n_valid=kw["n_valid"])


def test_heads_that_overlap_are_refused(lib):
    """Distances of two heads: every pair of spans, from their strides."""
    def call(heads, hs, n, ts, dim=128):
        h = dsa._HeadsC(x=2 * A, out=A, heads=heads, dim=dim, x_token_stride=ts, x_head_stride=hs,
                        out_token_stride=ts, out_head_stride=hs, weight=None, eps=0.0, norm=1,
                        rope_start=-1)
        return lib.dsa_norm_rope(n, None, None, 0, ctypes.byref(h), 1, None, None)
    assert call(2, 128, 2, 128) == 1     # head 1 of a token is head 0 of the next
    assert call(3, 256, 2, 256 + 64) == 1
    assert call(5, 300 * 8, 7, 600 * 8 + 64) == 1
    assert call(2, 1 << 62, 2, 128) == 1
    assert call(2, 128, 2, 1 << 62) == 1
    assert call(1, 129, 0, 129) == 0     # the stride of a single head or token is not used


def test_serving_tensors_of_two_devices_are_refused(lib):
    host, meta = torch.zeros(2, dtype=torch.int32), torch.zeros(2, dtype=torch.int32, device="meta")
    state = torch.zeros(2, dtype=torch.int64)
    with pytest.raises(ValueError):
        dsa._one_device(host, None, type("T", (), dict(get_device=lambda s: 0, device="cuda:0"))())
    dsa._one_device(host, None, meta)  # neither is on a CUDA device
    dsa.PagePool(host.view(1, 2), 64, host, state)


def test_the_compiled_calls_leave_everything_but_the_plain_case(lib):
    """Host tensors, and arguments that are no tensors at all, are not theirs: None, no error left
    behind, and the binding's own checks answer."""
    calls = dsa._load_calls()
    cfg = dsa.config(kv_fmt=dsa.KV_MXFP4)
    rows, slots = torch.zeros((2, 512), dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int32)
    cache, ws = torch.zeros((4, 272), dtype=torch.uint8), torch.zeros(256, dtype=torch.uint8)
    for a in ((True, cfg, rows, slots, cache, ws, None), (True, cfg, None, slots, cache, ws, None),
              (False, 3, "x", slots, cache, ws, None), (True, cfg, rows)):
        assert calls.rows(*a) is None
    pool = dsa.PagePool.empty(2, 64, 2, 4, device="cpu")
    plan = dsa.StepPlan.empty(2, 2, device="cpu")
    assert calls.plan(cfg, slots, slots, pool._key, plan._key, ws) is None
    assert calls.plan(cfg, None, slots, pool._key, plan._key, ws) is None
    heads = dsa.HeadSet([dsa.Heads(rows)])
    assert calls.norm(None, rows, heads._key, None, None) is None
    assert calls.norm(None, 7, heads._key, None, None) is None
    with pytest.raises(ValueError):
        calls.init(1, 2, 3, 4)


@pytest.mark.parametrize("dim,rope_dim", [(128, 64), (64, 64), (1024, 1024), (32, 64)])
def test_rotations_that_start_past_the_head_are_refused(lib, dim, rope_dim):
    """Starts up to the largest multiple of 8 that an int holds: start + rope_dim may pass 2^31."""
    rope = dsa._RopeC(inv_freq=A, rope_dim=rope_dim, interleaved=1, scale=1.0)
    last = dim - rope_dim
    for start in (last + 8, 1 << 20, (1 << 31) - rope_dim - 8, (1 << 31) - rope_dim, (1 << 31) - 8):
        if start < 0:
            continue
        h = dsa._HeadsC(x=A, out=A, heads=2, dim=dim, x_token_stride=2 * dim, x_head_stride=dim,
                        out_token_stride=2 * dim, out_head_stride=dim, weight=A, eps=1e-6, norm=1,
                        rope_start=start)
        assert lib.dsa_norm_rope(4, None, A, 0, ctypes.byref(h), 1, ctypes.byref(rope), None) == 1, start


def test_groups_that_write_what_another_reads_or_writes_are_refused(lib):
    """One launch runs the groups in no order: a group's output that is another's input (that
    group in place, say) or output is refused where they start at one address. Inputs may be shared."""
    def call(*groups, n=4):
        arr = (dsa._HeadsC * len(groups))()
        for h, (x, out, heads) in zip(arr, groups):
            h.x, h.out, h.heads, h.dim, h.rope_start, h.norm = x, out, heads, 64, -1, 1
            h.x_token_stride = h.out_token_stride = 128
            h.x_head_stride = h.out_head_stride = 64
        return lib.dsa_norm_rope(n, None, None, 0, arr, len(groups), None, None)
    x, y, z = A, 2 * A, 3 * A
    assert call((x, y, 2), (z, y, 2)) == 1        # two outputs
    assert call((x, x, 2), (x, y, 2)) == 1        # in place, and read by another
    assert call((x, y, 2), (x, x, 2)) == 1
    assert call((x, y, 2), (y, z, 1)) == 1        # one's output, another's input
    assert call((y, z, 1), (5 * A, 6 * A, 1), (x, y, 2)) == 1
    assert call((x, x, 2), (x, y, 2), n=0) == 0   # nothing is read or written
    assert call((x, x, 0), (x, y, 0)) == 0
