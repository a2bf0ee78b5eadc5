"""Steps whose rows and sequences do not match one to one, on a GPU: rows behind the last sequence (a captured step that holds
fewer rows than its capacity), sequences without a new token between others, steps that are refused."""
import numpy as np
import pytest
import torch

from sparse_attention_long_dsa_b200 import binding as B
from sparse_attention_long_dsa_b200 import workloads as W
from sparse_attention_long_dsa_b200.paged_cache import PagedCache
from sparse_attention_long_dsa_b200.pipeline import DeviceBatch

pytestmark = pytest.mark.gpu

DEV = "cuda"


def _i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device=DEV)


# ------------------------------------------------------------------------------------------------ rows of no sequence
LENS, ROWS = [9000, 64, 700, 40], [3, 0, 5, 7]
REAL = 8                                      # the rows of the first three sequences; the last seven become padding


def _pair(kind, topk=64):
    """A batch of four sequences, and the same arrays described as three sequences with seven rows behind them."""
    kw = dict(H=4, Dqk=64, Dv=64, Hi=2, Di=32) if kind == "f32" else {}
    wl = W.make_workload("rows", kind=kind, seed=41, seq_lens=LENS, q_lens=ROWS, topk=topk, **kw)
    exact, padded = DeviceBatch(wl), DeviceBatch(wl)
    cut = (padded.block_table[:3], padded.seq_lens[:3], padded.cu_q[:4])
    padded.batch = B.make_batch(*cut, num_blocks=wl.num_blocks, page_size=64, total_q=wl.total_q,
                                max_q_per_seq=wl.max_q_per_seq, max_seq_len=wl.max_seq_len)
    for db in (exact, padded):
        db.scores.fill_(-77.0)
        db.idx.fill_(-5)
        db.out.fill_(5.0)
        db.lse.fill_(5.0)
    return exact, padded


@pytest.mark.parametrize("kind", ["mla", "f32"])
@pytest.mark.parametrize("fused", [False, True])
def test_rows_behind_the_last_sequence_select_nothing(kind, fused):
    exact, padded = _pair(kind)
    for db in (exact, padded):
        db.run(fused=fused)
        db.check_status()
    assert (padded.idx[REAL:] == -1).all() and (padded.scores[REAL:] == -77).all()
    assert (padded.out[REAL:] == 0).all() and (padded.lse[REAL:] == -float("inf")).all()
    for name in ("scores", "idx", "out", "lse"):
        assert torch.equal(getattr(padded, name)[:REAL], getattr(exact, name)[:REAL]), name


def test_rows_behind_the_last_sequence_in_the_other_selections():
    """The allocation-free top-k, and pages: scores, kept pages and positions."""
    exact, padded = _pair("mla")
    for db in (exact, padded):
        db.indexer()
        B.dsa_topk_noalloc(db.scores, db.ld, db.batch, 64, db.idx)
        db.block_select(4)
        db.check_status()
    assert (padded.idx[REAL:] == -1).all() and torch.equal(padded.idx[:REAL], exact.idx[:REAL])
    assert (padded.idx_blk[REAL:] == -1).all() and torch.equal(padded.idx_blk[:REAL], exact.idx_blk[:REAL])


@pytest.mark.parametrize("how", ["alone", "with the scores"])
def test_rows_behind_the_last_sequence_are_not_appended(how):
    exact, padded = _pair("mla")
    rng = np.random.default_rng(5)
    t = exact.wl.total_q
    kv = torch.tensor(rng.standard_normal((t, 576)), device=DEV).bfloat16()
    key = torch.tensor(rng.standard_normal((t, 128)), dtype=torch.float32, device=DEV)
    first = B.make_batch(exact.block_table[:3], exact.seq_lens[:3], exact.cu_q[:4], num_blocks=exact.wl.num_blocks, page_size=64,
                         total_q=REAL, max_q_per_seq=5, max_seq_len=exact.wl.max_seq_len)
    B.dsa_cache_append(kv[:REAL], B.DSA_BF16, key[:REAL], B.DSA_F32, 576, 128, first, exact.kv_pool, exact.kI_pool, exact.kS_pool,
                       exact.ws, exact.ws_bytes)
    if how == "alone":
        B.dsa_cache_append(kv, B.DSA_BF16, key, B.DSA_F32, 576, 128, padded.batch, padded.kv_pool, padded.kI_pool,
                           padded.kS_pool, padded.ws, padded.ws_bytes)
    else:
        padded.append_and_indexer(kv, key, B.DSA_F32)
        assert (padded.scores[REAL:] == -77).all()
    exact.check_status()
    padded.check_status()
    for name in ("kv_pool", "kI_pool", "kS_pool"):
        a, b = (getattr(db, name).view(torch.uint8) for db in (padded, exact))
        assert torch.equal(a, b), name


@pytest.mark.parametrize("kind", ["mla", "f32"])
def test_a_decode_row_of_a_sequence_without_tokens(kind):
    """Empty sequence slots of a decode batch: nothing selected, zeros from both attentions, other rows unchanged."""
    kw = dict(H=4, Dqk=64, Dv=64, Hi=2, Di=32) if kind == "f32" else {}
    wl = W.make_workload("slots", kind=kind, seed=42, seq_lens=[300, 65, 2100, 64], q_lens=[1] * 4, topk=64, **kw)
    full, some = DeviceBatch(wl), DeviceBatch(wl)
    some.seq_lens.copy_(_i32([300, 0, 2100, 0]))
    for fused in (False, True):
        for db in (full, some):
            db.idx.fill_(-5)
            db.out.fill_(5.0)
            db.run(fused=fused)
            db.check_status()
        assert (some.idx[1::2] == -1).all() and (some.out[1::2] == 0).all() and (some.lse[1::2] == -float("inf")).all()
        for name in ("idx", "out", "lse"):
            assert torch.equal(getattr(some, name)[::2], getattr(full, name)[::2]), name
    pages = {id(db): db.block_pages(3) for db in (full, some)}
    for db in (full, some):
        db.out.fill_(5.0)
        db.paged_attention(pages[id(db)])
    assert (some.out[1::2] == 0).all() and torch.equal(some.out[::2], full.out[::2])
    assert (some.block_select(3)[1::2] == -1).all()
    some.check_status()


# ------------------------------------------------------------------------------------------------ refused steps
@pytest.mark.parametrize("rows", [600, 5000])                # plan and rows in one launch, and in two
def test_a_refused_step_has_no_rows(rows):
    """A prompt that does not fit: cu_q is zero, so that the calls which follow in a captured step find rows of no sequence
    (the cached lengths with the prompt's rows would put them at negative positions)."""
    cache = PagedCache(3, 12, 40)
    cache.extend(_i32([100, 0, 70]), 170)
    cache.check_status()
    cache.extend(_i32([1, 2000, 1]), rows)
    with pytest.raises(B.DSAError) as e:
        cache.check_status()
    assert e.value.status == B.DSA_ERR_DEVICE_CHECK
    assert cache.cu_q.tolist() == [0] * 4 and cache.seq_lens.tolist() == [100, 0, 70]
    assert (cache.slots == -1).all() and (cache.positions == -1).all()
    batch = B.make_batch(cache.block_table, cache.seq_lens, cache.cu_q, num_blocks=12, page_size=64, total_q=rows,
                         max_q_per_seq=2000, max_seq_len=2560)
    ws = torch.zeros(B.dsa_workspace_size(B.DSA_OP_INDEXER_TOPK, batch, 64), dtype=torch.uint8, device=DEV)
    q, w = torch.zeros((rows, 64, 128), dtype=torch.uint8, device=DEV), torch.ones((rows, 64), device=DEV)
    scores, idx = torch.full((rows, 2560), -77.0, device=DEV), torch.zeros((rows, 64), dtype=torch.int32, device=DEV)
    B.dsa_indexer_topk(q, B.DSA_FP8_E4M3, w, cache.ki_pool, B.DSA_FP8_E4M3, cache.ks_pool, 64, 128, batch, 64, scores, 2560,
                       idx, ws, ws.numel())
    B.dsa_read_device_status(ws)
    assert (scores == -77).all() and (idx == -1).all()
