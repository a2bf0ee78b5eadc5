"""Steps whose rows and sequences do not match one to one, on a GPU: rows behind the last sequence (a captured step that holds
fewer rows than its capacity), sequences without a new token between others, steps that are refused."""
import numpy as np
import pytest
import torch

from sparse_attention_long_dsa_b200 import binding as B
from sparse_attention_long_dsa_b200 import workloads as W
from sparse_attention_long_dsa_b200.paged_cache import PagedCache
from sparse_attention_long_dsa_b200.pipeline import DeviceBatch
from test_step_gpu import _Cache, _check, _extend_ref, _freq, _random_tables, _rope_ref, _Tables, _view

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


# ------------------------------------------------------------------------------------------------ one row per sequence slot
@pytest.mark.parametrize("cached,add", [
    ([0], [1]),
    ([63, 64, 65, 0, 127, 128], [1, 0, 1, 1, 1, 0]),
    ([5, 64, 64], [0, 0, 0]),
    ([64 * (i % 3) for i in range(3000)], [i % 2 for i in range(3000)]),              # plan and rows in two launches
])
def test_a_decode_step_has_one_row_per_sequence(cached, add):
    n, rng = len(cached), np.random.default_rng(len(cached))
    width, blocks, table, free = _random_tables(rng, cached, add, spare=3)
    t = _Tables(n, width, blocks, free, table)
    seq, slots = torch.full((n,), -5, dtype=torch.int32, device=DEV), torch.full((n,), -5, dtype=torch.int64, device=DEV)
    pos, left = torch.full((n,), -5, dtype=torch.int32, device=DEV), torch.full((1,), -5, dtype=torch.int32, device=DEV)
    B.dsa_batch_extend(_i32(cached), _i32(add), 64, blocks, n, t.free, t.count, t.table, seq, None, slots, pos, left, t.ws,
                       t.ws.numel())
    ref_table, ref_left, cu, ref_slots, ref_pos = _extend_ref(cached, add, table, free, sum(add))
    assert t.status() == B.DSA_OK
    assert np.array_equal(t.table.cpu(), ref_table) and left.item() == ref_left
    assert np.array_equal(seq.cpu(), np.add(cached, add))
    has, row = np.array(add) > 0, np.array(cu[:-1])
    want = np.full((2, n), -1)
    want[:, has] = ref_slots[row[has]], ref_pos[row[has]]
    assert np.array_equal(slots.cpu(), want[0]) and np.array_equal(pos.cpu(), want[1])


@pytest.mark.parametrize("bad", ["two tokens", "blocks"])
def test_a_decode_step_that_does_not_fit(bad):
    cache = PagedCache(3, 3 if bad == "two tokens" else 2, 4, 4)
    cache.extend(_i32([64, 0, 64]), 128)
    cache.check_status()
    table, lens, count = cache.block_table.clone(), cache.seq_lens.clone(), cache.free_count.item()
    cache.extend(_i32([0, 0, 2] if bad == "two tokens" else [1, 1, 0]))
    with pytest.raises(B.DSAError) as e:
        cache.check_status()
    assert e.value.status == B.DSA_ERR_DEVICE_CHECK
    assert torch.equal(cache.block_table, table) and torch.equal(cache.seq_lens, lens) and cache.free_count.item() == count
    assert cache.slots.tolist() == cache.positions.tolist() == [-1] * 3


def _check_sparse(c, q, out, lse, idx, live):
    """Every position selected: the sparse attention of the live rows against the dense definition; others select nothing."""
    for b, n in enumerate(c.lens_h):
        if b in live:
            assert idx[b].tolist() == list(range(n)) + [-1] * (idx.shape[1] - n)
    keep = c.lens_h
    c.lens_h = [n if b in live else 0 for b, n in enumerate(keep)]
    masked, lm = out.clone(), lse.clone()
    dead = [b for b in range(len(keep)) if b not in live]
    masked[dead], lm[dead] = 0, -float("inf")
    c.check(q, 0.07, masked, lm)
    c.lens_h = keep


def test_a_captured_decode_step_with_pauses_from_store_to_both_attentions():
    """Tables, stores, scores, selection, sparse and dense attention of a decode step in one graph, q and the indexer's queries
    taken from store.  Slots pause in the middle and at the front; one stays empty.  Row b is slot b throughout."""
    n, heads, k = 5, 128, 256
    cache = PagedCache(n, 30, 4, heads)
    rng = np.random.default_rng(21)
    f = lambda *s: torch.tensor(rng.standard_normal(s), device=DEV).bfloat16()        # noqa: E731
    w_kv, w_ki, freq = f(512).abs() + 0.5, f(128).abs() + 0.5, torch.tensor(_freq(64), device=DEV)
    cache.extend(_i32([70, 100, 3, 62, 0]), 240)
    cache.store(f(240, 576), w_kv, freq, k_idx=f(240, 128), k_idx_weight=w_ki)
    new, kv, k_idx, q_rot, q_idx = _i32([0] * n), f(n, 576), f(n, 128), f(n, heads, 64), f(n, 64, 128)
    q, q_idx_out = f(n, heads, 576), torch.zeros((n, 64, 128), dtype=torch.uint8, device=DEV)
    w, scores = torch.rand((n, 64), device=DEV), torch.zeros((n, 256), device=DEV)
    idx = torch.zeros((n, k), dtype=torch.int32, device=DEV)
    outs = [torch.empty((n, heads, 512), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    lses = [torch.empty((n, heads), device=DEV) for _ in range(2)]
    sparse = cache.decode_batch()
    size = max(B.dsa_workspace_size(B.DSA_OP_INDEXER_TOPK, sparse, k), B.dsa_workspace_size(B.DSA_OP_ATTN_DECODE, sparse, k, heads, 512))
    ws = torch.zeros(size, dtype=torch.uint8, device=DEV)

    def step():
        cache.extend(new)
        cache.store(kv, w_kv, freq, k_idx=k_idx, k_idx_weight=w_ki, q_rot=q_rot, q=q, q_idx=q_idx, q_idx_out=q_idx_out)
        batch = cache.batch(n, 1, 256)
        B.dsa_indexer_topk(q_idx_out, B.DSA_FP8_E4M3, w, cache.ki_pool, B.DSA_FP8_E4M3, cache.ks_pool, 64, 128, batch, k, scores,
                           256, idx, ws, size)
        B.dsa_sparse_attn_decode(q, B.DSA_BF16, cache.kv_pool, None, heads, 576, 512, 0.07, idx, k, batch, outs[0], lses[0], ws, size)
        cache.attend(q, outs[1], 0.07, lse=lses[1])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()                                                         # no slot has a new token
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    lens = np.array([70, 100, 3, 62, 0])
    for add in ([1, 0, 1, 1, 0], [0, 1, 1, 1, 0], [1, 1, 0, 1, 0], [0, 0, 1, 0, 1], [1, 1, 1, 1, 1]):
        new.copy_(_i32(add))
        for x in (kv, k_idx, q_rot, q_idx, q):
            x.copy_(f(*x.shape))
        before = q.clone()
        graph.replay()
        lens += add
        cache.check_status()
        B.dsa_read_device_status(ws)
        live = [b for b in range(n) if add[b]]
        assert cache.seq_lens.tolist() == lens.tolist()
        assert cache.positions.tolist() == [lens[b] - 1 if add[b] else -1 for b in range(n)]
        ref, pre = _rope_ref(q_rot.double().cpu().numpy(), lens - 1, 1, (0, 0), 0, (0, 64), "pairs")
        _check(q[live][:, :, 512:], ref[live], pre[live], "bf16")
        rest = [b for b in range(n) if not add[b]]
        assert torch.equal(q[rest], before[rest]) and torch.equal(q[:, :, :512], before[:, :, :512])
        c = _view(cache, heads)
        c.check(q, 0.07, outs[1], lses[1])
        _check_sparse(c, q, outs[0], lses[0], idx, live)


def test_a_captured_packed_step_with_padding_and_pauses():
    """A packed step through batch: capacity above the rows, a slot without rows in the middle; scores, selection and sparse
    attention row by row.  With as many rows as slots the descriptor is still no decode batch."""
    n, heads, t, k = 3, 128, 7, 128
    cache = PagedCache(n, 20, 3, heads)
    rng = np.random.default_rng(22)
    f = lambda *s: torch.tensor(rng.standard_normal(s), device=DEV).bfloat16()        # noqa: E731
    w_kv, w_ki, freq = f(512).abs() + 0.5, f(128).abs() + 0.5, torch.tensor(_freq(64), device=DEV)
    lens = np.array([60, 1, 64])
    cache.extend(_i32(lens), 125)
    cache.store(f(125, 576), w_kv, freq, k_idx=f(125, 128), k_idx_weight=w_ki)
    for t, adds in ((7, ([2, 0, 3], [1, 1, 1], [0, 0, 0], [0, 0, 7])), (3, ([1, 0, 1], [0, 2, 1], [0, 1, 1]))):
        new, kv, k_idx, q_rot, q_idx = _i32([0] * n), f(t, 576), f(t, 128), f(t, heads, 64), f(t, 64, 128)
        q, q_idx_out = f(t, heads, 576), torch.zeros((t, 64, 128), dtype=torch.uint8, device=DEV)
        w, scores = torch.rand((t, 64), device=DEV), torch.zeros((t, 192), device=DEV)
        idx = torch.zeros((t, k), dtype=torch.int32, device=DEV)
        out = torch.empty((t, heads, 512), dtype=torch.bfloat16, device=DEV)
        lse = torch.empty((t, heads), device=DEV)

        def step():
            cache.extend(new, t)
            cache.store(kv, w_kv, freq, k_idx=k_idx, k_idx_weight=w_ki, q_rot=q_rot, q=q, q_idx=q_idx, q_idx_out=q_idx_out,
                        packed=True)
            batch = cache.batch(t, 1 if t == n else t, 192)
            size = max(B.dsa_workspace_size(B.DSA_OP_INDEXER_TOPK, batch, k),
                       B.dsa_workspace_size(B.DSA_OP_ATTN_PREFILL, batch, k, heads, 512))
            B.dsa_indexer_topk(q_idx_out, B.DSA_FP8_E4M3, w, cache.ki_pool, B.DSA_FP8_E4M3, cache.ks_pool, 64, 128, batch, k,
                               scores, 192, idx, ws, size)
            B.dsa_sparse_attn_prefill(q, B.DSA_BF16, cache.kv_pool, None, heads, 576, 512, 0.07, idx, k, batch, out, lse, ws, size)

        ws = torch.zeros(1 << 26, dtype=torch.uint8, device=DEV)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        for add in adds:
            new.copy_(_i32(add))
            graph.replay()
            lens = lens + add
            cache.check_status()
            B.dsa_read_device_status(ws)
            assert cache.seq_lens.tolist() == lens.tolist()
            c = _view(cache, heads)
            seq = np.repeat(np.arange(n), add)
            rows = [lens[b] - add[b] + i + 1 for b in range(n) for i in range(add[b])]
            c.table_h = np.concatenate([c.table_h[seq], np.zeros((t - len(seq), 3), int)])
            c.lens_h = rows + [0] * (t - len(rows))
            for r, m in enumerate(c.lens_h):
                m = min(m, k)
                if c.lens_h[r] <= k:
                    assert idx[r].tolist() == list(range(m)) + [-1] * (k - m)
            assert max(c.lens_h) <= k
            c.check(q, 0.07, out, lse)


def test_queries_of_a_packed_step_of_num_seqs_rows():
    """attend would take them with rows shifted behind a pause: refused, unless the caller says that packed rows are meant."""
    cache = PagedCache(3, 6, 2, 4)
    w, freq = torch.ones(512, device=DEV), torch.tensor(_freq(64), device=DEV)
    kv, q_rot = torch.randn((3, 576), device=DEV).bfloat16(), torch.randn((3, 4, 64), device=DEV).bfloat16()
    q = torch.zeros((3, 4, 576), dtype=torch.bfloat16, device=DEV)
    cache.extend(_i32([1, 0, 1]), 3)
    with pytest.raises(B.DSAError) as e:
        cache.store(kv, w, freq, q_rot=q_rot, q=q)
    assert e.value.status == B.DSA_ERR_INVALID_ARG
    cache.store(kv, w, freq)
    cache.store(kv, w, freq, q_rot=q_rot, q=q, packed=True)
    assert (q[:2, :, 512:] != 0).any(-1).all() and (q[2] == 0).all()                 # rows 0 and 1 are slots 0 and 2
    q.zero_()
    cache.extend(_i32([1, 0, 1]))
    cache.store(kv, w, freq, q_rot=q_rot, q=q)
    assert (q[::2, :, 512:] != 0).any(-1).all() and (q[1] == 0).all()
    with pytest.raises(B.DSAError):
        cache.batch(2, 1, 64)
    cache.check_status()


# ------------------------------------------------------------------------------------------------ which rows are cut
def _cut_rows(c, heads, dv):
    """The rows that were split, from what the attention left for its join in the workspace: (row, first worker) per worker."""
    workers = 74 if dv > 128 else 148
    info = c.ws[256:256 + 8 * workers].view(torch.int32).view(workers, 2).cpu().numpy()
    return set(info[info[:, 0] >= 0, 0].tolist())


_HALF = [10] * 100 + [0] * 500                             # more slots than threads, rows in a sixth of them


@pytest.mark.parametrize("heads,f32,pages,cut", [
    (128, None, [1] * 74 + [16], {74}),                    # a worker would wait for the one long row
    (128, None, [2] * 80 + [16], {80}),
    (128, None, [1] * 200 + [16, 16], {200, 201}),
    (128, None, [75] * 2 + [6] * 75, {0, 1}),
    (128, None, [16] * 75, None),                          # one worker would have two rows, 16 pages more than the others
    (128, None, [8] * 128, set()),
    (128, None, [8 + i % 6 for i in range(100)], set()),
    (128, None, _HALF, set()),
    (16, None, [8] * 75, None),
    (16, None, [8] * 128, set()),
    (16, (128, 128), [8] * 149, None),
    (16, (128, 128), [3] * 220, set()),
    (16, (128, 128), [1] * 150 + [8], {150}),
    (13, (32, 32), [1] * 150 + [8], set()),
    (4, (64, 64), [8] * 300, None),
    (4, (64, 64), [3] * 220 + [0] * 300, set()),
])
def test_rows_stay_whole_where_no_worker_waits_for_them(heads, f32, pages, cut):
    """More rows than workers.  cut: the rows in pieces; None: some are."""
    c = _Cache([max(0, 64 * p - 7 * (i % 9)) for i, p in enumerate(pages)], f32=f32, seed=len(pages))
    q = c.q(heads)
    out, lse = c.attend(q, 0.07)
    B.dsa_read_device_status(c.ws)
    got = _cut_rows(c, heads, c.dv)
    assert got == cut if cut is not None else got
    c.check(q, 0.07, out, lse)


def test_store_refusals():
    cache = PagedCache(2, 4, 2, 4)
    w, freq = torch.ones(512, device=DEV), torch.tensor(_freq(64), device=DEV)
    f = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device=DEV)                   # noqa: E731
    codes = torch.zeros((2, 64, 128), dtype=torch.uint8, device=DEV)
    with pytest.raises(B.DSAError) as e:
        cache.store(f(2, 576), w, freq)                                # no step yet: there are no slots to write to
    assert e.value.status == B.DSA_ERR_INVALID_ARG
    cache.extend(_i32([1, 1]))
    for bad in (dict(q_rot=f(2, 4, 64)), dict(q_idx=f(2, 64, 128)), dict(k_idx=f(2, 128)), dict(q_rot=f(2, 3, 64), q=f(2, 4, 576)), dict(q_rot=f(3, 4, 64), q=f(3, 4, 576))):
        with pytest.raises(B.DSAError) as e:
            cache.store(f(2, 576), w, freq, **bad)
        assert e.value.status == B.DSA_ERR_INVALID_ARG
    with pytest.raises(B.DSAError):
        cache.store(f(3, 576), w, freq)
    cache.store(f(2, 576), w, freq, q_rot=f(2, 4, 64), q=f(2, 4, 576), q_idx=f(2, 64, 128), q_idx_out=codes)
    cache.check_status()
