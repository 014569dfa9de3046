"""The 8-bit cache at the ends of its ranges: queries of any size, keys that
decide a long row, appends of every width, rows that are not finite.

Tolerances are those of tests/test_cache_q8.py (their sums are written down
there)."""
from __future__ import annotations

import math

import pytest
import torch

from tests.test_cache_q8 import (ATTN, BF, attn_inputs, call, check_attn,
                                 dsa, reference)  # noqa: F401

gpu = pytest.mark.gpu

# of both attention kernels: over a selection and over all keys
KERNELS = [ATTN[1], ATTN[6], ATTN[9], ATTN[21], ATTN[5], ATTN[12], ATTN[13]]


@gpu
@pytest.mark.parametrize("power", [108, 112, 116, 120])
@pytest.mark.parametrize("case", KERNELS)
def test_large_queries_with_a_small_scale(dsa, case, power):
    """The scale brings the scores back to ordinary ones: the same softmax as
    that of ordinary queries, power for power.  (Powers of two: exact.)"""
    a = attn_inputs(case, 21)
    a["scale"] = 0.109375               # exact in fp32 after the power, too
    want = call(dsa, a)
    big = dict(a, q=(a["q"].float() * 2.0 ** power).to(BF),
               scale=a["scale"] * 2.0 ** -power)
    assert bool(torch.isfinite(big["q"].float()).all())
    o, lse, ws = call(dsa, big)
    assert dsa.dsa_indexer_check(ws) == 0
    r, T = reference(big)
    check_attn(r, o, lse, T)
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


@gpu
@pytest.mark.parametrize("power", [108, 112, 116, 120])
@pytest.mark.parametrize("case", [c for c in KERNELS if c[0] < 33 and
                                  c[2] // c[3] <= 16])
def test_rows_of_large_queries(dsa, case, power):
    """Large queries among ordinary ones: the row's largest score takes all of
    its weight, and a row of one key gives that key's value."""
    a = attn_inputs(case, 22)
    a["q_pos"][0] = 0
    a["q"][0, 0] = (a["q"][0, 0].float() * 2.0 ** power).to(BF)
    a["q"][-1, -1, 0] = (a["q"][-1, -1, 0].float() * 2.0 ** power).to(BF)
    o, lse, ws = call(dsa, a)
    assert dsa.dsa_indexer_check(ws) == 0
    r, T = reference(a)
    assert float(r["lse"][0, 0].abs().min()) > 2.0 ** (power - 20)
    check_attn(r, o, lse, T)


@gpu
@pytest.mark.parametrize("power", [20, 24, 26, 28, 31, 35, 40, 64, 100, 120])
@pytest.mark.parametrize("case", KERNELS)
def test_large_scores_of_one_key(dsa, case, power):
    """Rows of one key, with scores of either sign and any size."""
    a = attn_inputs(case, 23)
    a["q_pos"][0] = 0
    a["q"][0, 0] = (a["q"][0, 0].float() * 2.0 ** power).to(BF)
    o, lse, ws = call(dsa, a)
    assert dsa.dsa_indexer_check(ws) == 0
    r, T = reference(a)
    row = r["lse"][0, 0]
    assert row.numel() < 4 or bool((row < 0).any()) and bool((row > 0).any())
    check_attn(r, o, lse, T)
    assert bool((o[0, 0].double().cpu() - r["o"][0, 0]).abs().max() <= 2.0 ** -8
                * r["o"][0, 0].abs().max())


@gpu
@pytest.mark.parametrize("power", [64, 112, 120])
@pytest.mark.parametrize("case", [ATTN[5], ATTN[12], ATTN[13]])
def test_rows_of_large_queries_in_tiles(dsa, case, power):
    """(As above, of the kernel for many rows.)"""
    a = attn_inputs(case, 22)
    a["q"][0, 0] = (a["q"][0, 0].float() * 2.0 ** power).to(BF)
    a["q"][-1, -1, 0] = (a["q"][-1, -1, 0].float() * 2.0 ** power).to(BF)
    o, lse, ws = call(dsa, a)
    assert dsa.dsa_indexer_check(ws) == 0
    r, T = reference(a)
    check_attn(r, o, lse, T)
