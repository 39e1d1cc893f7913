"""What a K or V row that is not finite does to the rows that see it, dim by dim,
against the formula in 64 bits: infinities of one sign, of both, and NaN."""
import numpy as np
import pytest
import torch

from sparse_kv_cache_retrieval_gb300 import binding as spc
from tests.paged_cases import DEV, SCALE, bf16, f64, i32, prompt_tol

pytestmark = pytest.mark.gpu
LENS, AT = [150, 201], 150 + 100


def formula(q, k, v):
    """Each row over exactly the keys that it sees, in 64 bits: (out, sum of weights times |v|)."""
    q, k, v = f64(q), f64(k), f64(v)
    out, mag = np.zeros_like(q), np.zeros_like(q)
    for a, e in ((0, LENS[0]), (LENS[0], sum(LENS))):
        for i in range(a, e):
            for h in range(8):
                g = h // 4
                x = k[a:i + 1, g] @ q[i, h] * SCALE
                w = np.exp(x - x.max())
                w /= w.sum()
                out[i, h], mag[i, h] = w @ v[a:i + 1, g], w @ np.abs(v[a:i + 1, g])
    return out, mag


def attend(q, k, v):
    cu = [0, LENS[0], sum(LENS)]
    ws = torch.zeros(spc.spc_prompt_attn_workspace_size(sum(LENS), 2, 8, 2, 128), dtype=torch.uint8, device=DEV)
    out = torch.full((sum(LENS), 8, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    spc.spc_prompt_attn(q.to(DEV), k.to(DEV), v.to(DEV), i32(cu), sum(LENS), 2, 8, 2, 128, SCALE, out, ws)
    assert int(ws[:4].view(torch.int32).item()) == 0
    with np.errstate(all="ignore"):
        want, mag = formula(q, k, v)
    return f64(out), want, mag


def inputs(seed):
    rng = np.random.default_rng(seed)
    return [bf16(rng, sum(LENS), n, 128) for n in (8, 2, 2)]


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_a_key_row(bad):
    # every dim of one key: with queries of both signs the logit is inf - inf, NaN, for every row from there on
    q, k, v = inputs(110)
    clean, _, mag = attend(q, k, v)
    k[AT, 1] = bad
    got, want, _ = attend(q, k, v)
    seen = np.zeros(got.shape, bool)
    seen[AT:, 4:] = True
    assert np.array_equal(np.isnan(want), seen)
    assert np.all(np.isnan(got[seen])) and np.array_equal(got[~seen], clean[~seen])


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_one_value_of_a_key(bad):
    # its sign and the query's make the logit +inf (the row is NaN: inf - inf against the maximum) or -inf (the key
    # drops out); NaN reaches every row
    q, k, v = inputs(111)
    k[AT, 1, 3] = bad
    got, want, mag = attend(q, k, v)
    assert np.array_equal(np.isnan(got), np.isnan(want)) and np.all(np.isfinite(got) | np.isnan(got))
    rows = np.isnan(want[:, :, 0])
    assert 0 < rows[AT:, 4:].sum() and not rows[:AT].any() and not rows[:, :4].any()
    if not np.isnan(bad):
        assert rows[AT:, 4:].sum() < 0.7 * rows[AT:, 4:].size     # about half the queries
    ok = ~np.isnan(want)
    assert np.all(np.abs(got - want)[ok] <= prompt_tol(want, mag)[ok])


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_values(bad):
    # a whole row of V for one head, one value for the other: infinities keep their sign
    q, k, v = inputs(112)
    clean, cwant, cmag = attend(q, k, v)
    v[AT, 1], v[AT + 20, 0, 9] = bad, bad
    got, want, _ = attend(q, k, v)
    assert np.array_equal(np.isfinite(got), np.isfinite(want))
    odd = ~np.isfinite(want)
    assert np.array_equal(got[odd], want[odd], equal_nan=True)
    assert np.all(np.abs(got - cwant)[~odd] <= prompt_tol(cwant, cmag)[~odd])


@pytest.mark.parametrize("other", [-float("inf"), float("nan"), float("inf")])
def test_a_second_one_behind_the_first(other):
    # in one dim: it is in the block of keys of rows that see only the first
    q, k, v = inputs(113)
    v[AT, 1, 5], v[AT + 30, 1, 5] = float("inf"), other
    got, want, _ = attend(q, k, v)
    assert np.all(want[AT:AT + 30, 4:, 5] == np.inf)
    assert np.array_equal(np.isfinite(got), np.isfinite(want))
    odd = ~np.isfinite(want)
    assert np.array_equal(got[odd], want[odd], equal_nan=True)
