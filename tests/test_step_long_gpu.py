"""One-token attention where a worker walks many pages: every page exactly once.

q is zero, so every token has weight 1 and the products are exact; page p of a row holds 1 in value entry p mod Dv and 0
elsewhere.  out[d] is then the share of the row's tokens that lie in the pages with p mod Dv = d, and lse = ln(tokens): a page that
is lost or taken twice moves out[d] by a few per cent and the lse by 64 / tokens.

Bounds.  Sums of ones are exact below 2^24.  Each part's lse is off by a log2 (2 steps of a value up to 20: 4e-6), its scaling
and rounding (2e-6); the join adds up to 148 weights of such parts (148 * 2^-24 = 9e-6) and takes a logarithm (1e-6): 2e-5 in all,
for the lse as for the relative weight of a part.  bf16 results add half a step, 2^-8.
"""
import numpy as np
import pytest
import torch

from sparse_attention_long_dsa_b200 import binding as B
from test_step_gpu import _Cache, _i32

pytestmark = pytest.mark.gpu

DEV = "cuda"


def _marked(lens, f32=None, seed=0):
    """A cache whose values name their page; what no sequence holds stays NaN and infinity."""
    c = _Cache(lens, f32=f32, seed=seed)
    code = torch.zeros((c.blocks, c.dv), dtype=c.torch_dt, device=DEV)
    for b, n in enumerate(lens):
        p = np.arange(-(-n // 64))
        code[torch.tensor(c.table_h[b][p], device=DEV), torch.tensor(p % c.dv, device=DEV)] = 1
    pool = c.kv if c.v is None else c.v
    live = pool[:, :, 1].isfinite()
    pool[:, :, :c.dv] = torch.where(live[:, :, None], code[:, None], pool[:, :, :c.dv])
    return c


def _check_shares(c, out, lse, pages=None):
    rel = 2e-5 + (2.0 ** -8 if c.dt == B.DSA_BF16 else 0.0)
    for b, n in enumerate(c.lens_h):
        p = np.arange(-(-n // 64)) if pages is None else np.array([x for x in pages[b] if 0 <= x and 64 * x < n], dtype=int)
        tokens = np.minimum(64, n - 64 * p)
        o, l = out[b].double().cpu().numpy(), lse[b].double().cpu().numpy()
        if not len(p):
            assert (o == 0).all() and (l == -np.inf).all(), b
            continue
        ref = np.bincount(p % c.dv, weights=tokens, minlength=c.dv) / tokens.sum()
        assert (np.abs(o - ref) <= rel * ref).all(), (b, np.argwhere(np.abs(o - ref) > rel * ref)[:4])
        assert (np.abs(l - np.log(tokens.sum())) <= 2e-5).all(), (b, l[0] - np.log(tokens.sum()))


def _zero_q(c, heads):
    return torch.zeros((len(c.lens_h), heads, c.dqk), dtype=c.torch_dt, device=DEV)


@pytest.mark.parametrize("heads,f32", [(128, None), (5, None), (4, (64, 64)), (16, (32, 128))])
@pytest.mark.parametrize("lens", [
    [400001],                                              # 84 pages a worker of the latent path, 42 of the f32 path
    [64 * 74 * 32], [64 * 74 * 32 + 1], [64 * 74 * 33 - 63],           # 32 pages a worker, and around
    [4096 + 919 * i for i in range(32)],                   # about 124 pages a worker, several rows each
    [33] * 200 + [300000] + [70] * 100,
    [100000, 0, 1, 250000],
])
def test_every_page_of_long_rows_counts_once(heads, f32, lens):
    c = _marked(lens, f32=f32, seed=len(lens))
    out, lse = c.attend(_zero_q(c, heads), 0.07)
    B.dsa_read_device_status(c.ws)
    _check_shares(c, out, lse)


def _lists(rng, lens, kb, gaps):
    """Page lists in random order, a page now and then twice, with runs of -1 that begin and end around multiples of 32."""
    out = np.full((len(lens), kb), -1)
    for b, n in enumerate(lens):
        have = max(1, -(-n // 64))
        out[b] = np.resize(rng.permutation(have), kb)
        out[b, rng.random(kb) < 0.02] = rng.integers(0, have + 3)         # twice, or past the sequence
        at = 0
        while at < kb and gaps:
            start = at + 32 * int(rng.integers(0, 3)) + int(rng.integers(-2, 3))
            end = start + 32 * int(rng.integers(0, 4)) + int(rng.integers(-2, 3))
            out[b, max(0, start):max(0, end)] = -1
            at = max(end, at + 32)
    return out


@pytest.mark.parametrize("heads,f32", [(128, None), (16, None), (4, (64, 64))])
@pytest.mark.parametrize("lens,kb,gaps", [
    ([200000], 3001, False), ([200000], 7001, True), ([100000, 30000, 0, 77777], 2000, True), ([30000] * 32, 400, True),
    ([5000] * 90, 100, True),
])
def test_every_listed_page_counts_as_often_as_it_is_listed(heads, f32, lens, kb, gaps):
    rng = np.random.default_rng(kb + len(lens))
    c = _marked(lens, f32=f32, seed=kb)
    pages = _lists(rng, lens, kb, gaps)
    out, lse = c.attend(_zero_q(c, heads), 0.07, pages=_i32(pages))
    B.dsa_read_device_status(c.ws)
    _check_shares(c, out, lse, pages)


@pytest.mark.parametrize("heads", [128, 16])
def test_random_queries_over_many_pages_a_worker(heads):
    lens = [4096 + 919 * i for i in range(32)]
    c = _Cache(lens, seed=7)
    q = c.q(heads)
    out, lse = c.attend(q, 0.07)
    B.dsa_read_device_status(c.ws)
    c.check(q, 0.07, out, lse)
