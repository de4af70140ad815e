"""Attention over whole caches and draft verification refuse outputs that overlap what the call reads or
another output (no compute call runs here: every case stops in the check)."""
import ctypes

import pytest

import two_tier_sparse_gb300 as dsa
from two_tier_sparse_gb300 import build as dsa_build

M = 1 << 20  # fake device addresses, each at a multiple of it; never dereferenced
REFUSED = 1


@pytest.fixture(scope="module")
def lib():
    dsa_build.build()
    return dsa.load()


def ref(x):
    return ctypes.byref(x) if x is not None else None


FULL = ["q", "lat", "n", "swa", "sl", "out", "lse"]  # (the workspace behind them)
B, CAP, NQ = 3, 64, 2


def full_call(lib, multi, fmt, paged, at):
    cfg = dsa.config(kv_fmt=fmt)
    pg = dsa._Pages(page_table=at["pages"], page_rows=64, pages_per_seq=1, n_pages=3) if paged else None
    end = (at["lse"], at["ws"], 1 << 26, None)
    if multi:
        return lib.dsa_full_attn_multi(ref(cfg), NQ, at["n"], at["q"], at["lat"], CAP, ref(pg), CAP,
                                       at["swa"], B, at["out"], *end)
    return lib.dsa_full_attn_decode(ref(cfg), at["q"], at["lat"], CAP, ref(pg), at["n"], CAP, at["swa"],
                                    at["sl"], B, at["out"], *end)


@pytest.mark.parametrize("multi", [False, True])
@pytest.mark.parametrize("fmt,row", [(dsa.KV_BF16, 1024), (dsa.KV_FP8_E4M3, 512), (dsa.KV_MXFP4, 272)])
@pytest.mark.parametrize("paged", [False, True])
def test_full_attention(lib, multi, fmt, row, paged):
    queries = B * (NQ if multi else 1)
    size = {"q": queries * 65536, "out": queries * 65536, "lse": queries * 256, "lat": B * 64 * row,
            "swa": B * (128 + (NQ - 1 if multi else 0)) * row, "n": 4 * B, "sl": 4 * B, "pages": 4 * B}
    apart = {k: (i + 1) * M for i, k in enumerate(FULL + ["pages", "ws"])}
    inputs = ["q", "lat", "n", "swa"] + ([] if multi else ["sl"]) + (["pages"] if paged else [])
    for w in ("out", "lse"):
        for r in inputs + (["lse"] if w == "out" else ["out"]):
            # from its start, over its last 16 bytes, and reaching into it from in front
            last = apart[r] + (size[r] - 1) // 16 * 16
            front = apart[r] - (size[w] - 16)
            for p in (apart[r], last, front):
                assert full_call(lib, multi, fmt, paged, {**apart, w: p}) == REFUSED, (w, r)
    for r in inputs + ["out", "lse"]:  # inside the workspace
        assert full_call(lib, multi, fmt, paged, {**apart, r: apart["ws"] + (40 << 20)}) == REFUSED, r


@pytest.mark.parametrize("dt,size", [(0, 2), (1, 2), (2, 4)])
@pytest.mark.parametrize("D", [0, 1, 4])
def test_verification(lib, dt, size, D):
    V, stride = 100, 104
    small = ["x", "n", "u", "tokens", "kept", "drop"]
    apart = {k: (i + 1) * M for i, k in enumerate(["p", "q"] + small + ["ws"])}
    nbytes = {"p": ((B * (D + 1) - 1) * stride + V) * size, "q": (max(B * D - 1, 0) * stride + V) * size,
              "x": 4 * B * D, "n": 4 * B, "u": 4 * B * (D + 1), "tokens": 4 * B * (D + 1), "kept": 4 * B,
              "drop": 4 * B}
    outputs = ["tokens", "kept", "drop"]

    def call(**over):
        a = {**apart, **over}
        return lib.dsa_verify_drafts(B, D, V, dt, a["p"], stride, a["q"], stride, a["x"], a["n"], a["u"],
                                     a["tokens"], a["kept"], a["drop"], a["ws"], 256, None)
    for w in outputs:
        for r in ["p", "n", "u"] + (["q", "x"] if D else []) + [o for o in outputs if o != w]:
            for p in (apart[r], apart[r] + (nbytes[r] - 1) // 4 * 4, apart[r] - (nbytes[w] - 4)):
                assert call(**{w: p}) == REFUSED, (w, r)
        assert call(ws=apart[w] // 256 * 256) == REFUSED
    assert call(n=apart["drop"]) == REFUSED  # a count that is updated in place
