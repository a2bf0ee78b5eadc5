"""The serving step's calls on a GPU against plain implementations in 64 bits: block tables and slot maps from request
lengths, norm and rotation of query and key rows, one-token attention over the paged cache (whole, or a list of pages),
and a run of them together.

Bounds.  u = 2^-24 (half an fp32 step), a bf16 rounding is off by at most 2^-8 of the value, an e4m3 one by 2^-4 (2^-10
below the smallest normal).
* rotation: an angle in turns, |t| <= 1/2, is rounded to fp32 once (2^-26 turns = 9.4e-8 rad); sine and cosine add two
  fp32 steps (2.4e-7), the two products and the sum three more: 4e-7 (|a| + |b|) in all.
* norm: up to 1024 squares summed by lanes and a tree (under 40 additions in a row, 40 u), the square root halves that;
  division, root, product with the weight add 5 u: 25 u = 1.5e-6 of the value.
  Together at most 2e-6 (|a| + |b|) for a rotated pair (a, b) and 2e-6 |y| for an entry that is not rotated.
* attention: a dot product of D terms is off by at most D * 2^-23 * A, A the sum of the terms' magnitudes times the
  scale (2^-23: the tensor cores may truncate), a weight p by twice that plus 2^-21 (exponential and maximum), the sum
  of n weights and the products with v by (n + 64) u, and where P is held in bf16 each weight by 2^-8.
"""
import numpy as np
import pytest
import torch

import oracle
from sparse_attention_long_dsa_b200 import binding as B
from sparse_attention_long_dsa_b200 import workloads as W
from sparse_attention_long_dsa_b200.paged_cache import PagedCache
from sparse_attention_long_dsa_b200.pipeline import DeviceBatch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DEV = "cuda"


def _i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device=DEV)


def _zeros_ws(n):
    return torch.zeros(n, dtype=torch.uint8, device=DEV)


# ------------------------------------------------------------------------------------------------ block tables
class _Tables:
    """The device state of a cache's bookkeeping, and the call."""

    def __init__(self, seqs, width, blocks, free, table=None, cap=None):
        cap = len(free) if cap is None else cap
        self.blocks, self.n, self.width = blocks, seqs, width
        self.table = _i32(np.full((seqs, width), -7) if table is None else table)
        self.free = _i32(np.concatenate([free, np.full(cap - len(free), -9)]).astype(np.int32))
        self.count = _i32([len(free)])
        self.lens = _i32(np.zeros(seqs))
        self.ws = _zeros_ws(B.dsa_batch_workspace_size(B.DSA_OP_BATCH_EXTEND, seqs))

    def extend(self, cached, add, rows, lens=None, left=None, stream=None):
        cached = cached if isinstance(cached, torch.Tensor) else _i32(cached)
        add = add if isinstance(add, torch.Tensor) else _i32(add)
        self.seq = torch.full((self.n,), -5, dtype=torch.int32, device=DEV) if lens is None else lens
        self.cu = torch.full((self.n + 1,), -5, dtype=torch.int32, device=DEV)
        self.slots = torch.full((rows,), -5, dtype=torch.int64, device=DEV)
        self.pos = torch.full((rows,), -5, dtype=torch.int32, device=DEV)
        self.left = torch.full((1,), -5, dtype=torch.int32, device=DEV) if left is None else left
        B.dsa_batch_extend(cached, add, 64, self.blocks, rows, self.free, self.count, self.table, self.seq, self.cu,
                           self.slots, self.pos, self.left, self.ws, self.ws.numel(), stream)

    def status(self):
        try:
            B.dsa_read_device_status(self.ws)
        except B.DSAError as e:
            return e.status
        return B.DSA_OK


def _extend_ref(cached, add, table, free, rows):
    table, free = np.array(table), list(free)
    slots, pos, cu = np.full(rows, -1, np.int64), np.full(rows, -1, np.int64), [0]
    for b, (c, n) in enumerate(zip(cached, add)):
        for p in range(-(-c // 64), -(-(c + n) // 64)):
            table[b, p] = free.pop()
        for i in range(n):
            pos[cu[-1] + i] = c + i
            slots[cu[-1] + i] = int(table[b, (c + i) // 64]) * 64 + (c + i) % 64
        cu.append(cu[-1] + n)
    return table, len(free), cu, slots, pos


def _random_tables(rng, cached, add, spare, wide=2):
    held = [-(-c // 64) for c in cached]
    after = [-(-(c + n) // 64) for c, n in zip(cached, add)]
    width = max(max(after), 1) + wide
    blocks = sum(after) + spare
    ids = rng.permutation(blocks)
    table = np.full((len(cached), width), -7)
    at = 0
    for b, h in enumerate(held):
        table[b, :h] = ids[at:at + h]
        at += h
    return width, blocks, table, ids[at:]


@pytest.mark.parametrize("cached,add,pad", [
    ([0], [1], 0),
    ([63, 64, 65, 0, 127], [1, 1, 1, 0, 2], 0),
    ([0, 0, 0], [0, 0, 0], 3),
    ([100, 0, 64, 5], [0, 130, 64, 59], 7),
    ([0] * 5, [64, 1, 0, 63, 129], 0),
    ([7] * 1500, [1] * 1500, 5),
    ([3000, 57344, 0], [1, 8192, 4000], 1),            # past the rows that one CTA takes
    ([0] * 3000, [5] * 3000, 11),
])
def test_extend_against_a_plain_walk(cached, add, pad):
    rng = np.random.default_rng(len(cached) + sum(add))
    width, blocks, table, free = _random_tables(rng, cached, add, spare=3)
    rows = sum(add) + pad
    t = _Tables(len(cached), width, blocks, free, table)
    t.extend(cached, add, rows)
    ref_table, left, cu, slots, pos = _extend_ref(cached, add, table, free, rows)
    assert t.status() == B.DSA_OK
    assert np.array_equal(t.table.cpu(), ref_table)
    assert t.left.item() == left and t.count.item() == len(free)
    assert np.array_equal(t.cu.cpu(), cu) and np.array_equal(t.seq.cpu(), np.add(cached, add))
    assert np.array_equal(t.slots.cpu(), slots) and np.array_equal(t.pos.cpu(), pos)


def test_extend_in_place_over_steps_and_release():
    """Steps of random lengths with the state updated in place; sequences come and go; no block is ever held twice."""
    rng = np.random.default_rng(5)
    n, width, blocks = 37, 20, 400
    t = _Tables(n, width, blocks, rng.permutation(blocks))
    lens = np.zeros(n, int)
    for step in range(12):
        add = rng.integers(0, 60, n) * (rng.random(n) < 0.7)
        add = np.minimum(add, width * 64 - lens)
        rows = int(add.sum()) + step
        t.extend(t.lens, add, rows, lens=t.lens, left=t.count)
        assert t.status() == B.DSA_OK
        lens += add
        assert np.array_equal(t.lens.cpu(), lens)
        table, top = t.table.cpu().numpy(), t.count.item()
        held = [int(x) for b in range(n) for x in table[b, :-(-lens[b] // 64)]]
        assert sorted(held + t.free.cpu().tolist()[:top]) == list(range(blocks))
        pos, slots, cu = t.pos.cpu().numpy(), t.slots.cpu().numpy(), t.cu.cpu().numpy()
        for b in range(n):
            p = np.arange(lens[b] - add[b], lens[b])
            assert np.array_equal(pos[cu[b]:cu[b + 1]], p)
            assert np.array_equal(slots[cu[b]:cu[b + 1]], table[b, p // 64] * 64 + p % 64)
        done = rng.random(n) < 0.25
        B.dsa_batch_release(_i32(done), 64, blocks, t.table, t.lens, t.free, t.count, t.ws, t.ws.numel())
        assert t.status() == B.DSA_OK
        back = [int(x) for b in np.flatnonzero(done) for x in table[b, :-(-lens[b] // 64)]]
        assert t.count.item() == top + len(back)
        assert t.free.cpu().tolist()[top:top + len(back)] == back
        lens[done] = 0
        assert np.array_equal(t.lens.cpu(), lens)


@pytest.mark.parametrize("why", ["blocks", "long", "negative", "negative add", "rows", "count"])
def test_extend_refuses_a_step_that_does_not_fit(why):
    cached, add = [100, 64, 10], [30, 1, 60]
    rng = np.random.default_rng(3)
    width, blocks, table, free = _random_tables(rng, cached, add, spare=0)
    rows = 91
    if why == "blocks":
        free = free[1:]
    if why == "long":
        cached, add = [100, 64, width * 64], [30, 1, 1]
    if why == "negative":
        cached = [100, -3, 10]
    if why == "negative add":
        add = [30, -1, 60]
    if why == "rows":
        rows = 90
    t = _Tables(3, width, blocks, free, table)
    if why == "count":
        t.count += 1000
    count = t.count.item()
    t.extend(cached, add, rows)
    assert t.status() == B.DSA_ERR_DEVICE_CHECK
    assert np.array_equal(t.table.cpu(), table) and t.left.item() == count
    assert (t.slots.cpu() == -1).all() and (t.pos.cpu() == -1).all()
    assert np.array_equal(t.seq.cpu(), np.clip(cached, 0, width * 64))
    assert t.cu[0].item() == 0 and t.cu.max().item() <= rows
    assert t.status() == B.DSA_OK                                       # read and cleared


def test_extend_on_two_streams_at_once():
    rng = np.random.default_rng(1)
    add = [3000, 700, 1, 6000]
    width, blocks, table, free = _random_tables(rng, [5, 0, 64, 63], add, spare=4)
    a, b = (_Tables(4, width, blocks, free, table) for _ in range(2))
    cached, new = _i32([5, 0, 64, 63]), _i32(add)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(10):
        for t, s in ((a, s1), (b, s2)):
            with torch.cuda.stream(s):
                t.extend(cached, new, sum(add), stream=s)
    torch.cuda.synchronize()
    ref_table, left, cu, slots, pos = _extend_ref([5, 0, 64, 63], add, table, free, sum(add))
    for t in (a, b):
        assert t.status() == B.DSA_OK and np.array_equal(t.table.cpu(), ref_table) and t.left.item() == left
        assert np.array_equal(t.slots.cpu(), slots) and np.array_equal(t.pos.cpu(), pos)


def test_extend_reports_bad_ids():
    """An id outside the pool on the stack, and one in an entry that a row needs: those pages' rows get no slot."""
    table = np.array([[5, -7, -7], [99, -7, -7], [1, -7, -7]])
    t = _Tables(3, 3, 10, [2, 77], table)
    t.extend([64, 10, 20], [2, 3, 1], 6)
    assert t.status() == B.DSA_ERR_DEVICE_CHECK
    assert t.slots.cpu().tolist() == [-1, -1, -1, -1, -1, 84] and t.table.cpu().tolist()[0] == [5, -1, -7]


@pytest.mark.parametrize("why", ["capacity", "length", "count"])
def test_release_refusals(why):
    table = np.arange(12).reshape(3, 4)
    t = _Tables(3, 4, 12, [], table, cap=7 if why == "capacity" else 12)
    t.lens = _i32([256, 1, 300 if why == "length" else 256])
    if why == "count":
        t.count -= 1
    count, lens = t.count.item(), t.lens.clone()
    B.dsa_batch_release(_i32([1, 0, 1]), 64, 12, t.table, t.lens, t.free, t.count, t.ws, t.ws.numel())
    assert t.status() == B.DSA_ERR_DEVICE_CHECK
    assert t.count.item() == count and torch.equal(t.lens, lens) and (t.free.cpu() == -9).all()


# ------------------------------------------------------------------------------------------------ norm and rotation
def _freq(rot, base=10000.0):
    return base ** (-np.arange(0, rot, 2) / rot) if rot else np.zeros(0)


def _rope_ref(x, pos, weight, norm, eps, rope, style):
    """y in 64 bits, and the bound on what a 32-bit computation of it may be off by."""
    y = np.array(x, np.float64)
    off, n = norm
    if n:
        part = y[..., off:off + n]
        y[..., off:off + n] = part / np.sqrt((part ** 2).mean(-1, keepdims=True) + eps) * weight
    mag = np.abs(y)
    off, n = rope
    if n:
        theta = pos[:, None, None].astype(np.float64) * _freq(n)
        i = np.arange(n // 2)
        a, b = (off + 2 * i, off + 2 * i + 1) if style == "pairs" else (off + i, off + n // 2 + i)
        ya, yb = y[..., a].copy(), y[..., b].copy()
        y[..., a], y[..., b] = ya * np.cos(theta) - yb * np.sin(theta), yb * np.cos(theta) + ya * np.sin(theta)
        mag[..., a] = mag[..., b] = np.abs(ya) + np.abs(yb)
    return y, 2e-6 * mag


def _check(got, ref, pre, kind):
    got = got.double().cpu().numpy()
    step = {"f32": 2 * U, "bf16": 2.0 ** -8, "e4m3": 2.0 ** -4}[kind]
    tol = step * np.abs(ref) + 2 * pre + (2.0 ** -10 if kind == "e4m3" else 1e-30)
    bad = np.abs(got - np.clip(ref, -448, 448) if kind == "e4m3" else got - ref) > tol
    assert not bad.any(), (np.argwhere(bad)[:4], np.abs(got - ref)[bad][:4], tol[bad][:4])


_DT = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}


def _positions(rng, t):
    pos = rng.integers(0, 1 << 20, t).astype(np.int32)
    pos[: min(t, 3)] = [0, 1, 1048575][: min(t, 3)]
    return pos


@pytest.mark.parametrize("style", ["pairs", "halves"])
@pytest.mark.parametrize("t,h,d,norm,rope,xd,od", [
    (1, 1, 8, (0, 8), (0, 0), "f32", "f32"),
    (1, 3, 16, (0, 0), (0, 16), "bf16", "bf16"),
    (7, 5, 64, (0, 0), (0, 64), "bf16", "bf16"),
    (33, 128, 64, (0, 64), (0, 64), "bf16", "bf16"),
    (5, 37, 128, (0, 128), (0, 64), "bf16", "f32"),
    (3, 64, 128, (0, 0), (64, 64), "bf16", "e4m3"),
    (19, 2, 192, (8, 120), (128, 64), "f32", "bf16"),
    (9, 4, 256, (0, 256), (0, 256), "f32", "f32"),
    (6, 1, 576, (0, 512), (512, 64), "bf16", "bf16"),
    (11, 3, 264, (0, 264), (240, 16), "bf16", "bf16"),
    (4, 2, 1024, (0, 1024), (768, 256), "f32", "f32"),
    (300, 1, 128, (0, 128), (0, 64), "bf16", "e4m3"),
    (2, 1, 72, (64, 8), (0, 48), "f32", "bf16"),
    (3, 300, 64, (0, 64), (0, 32), "bf16", "bf16"),    # more heads than a CTA holds at a time
    (2, 150, 256, (0, 0), (128, 128), "bf16", "e4m3"),
    (2500, 128, 64, (0, 0), (0, 64), "bf16", "bf16"),  # several rows per CTA
    (9001, 1, 576, (0, 512), (512, 64), "bf16", "f32"),
])
def test_norm_and_rotation(style, t, h, d, norm, rope, xd, od):
    rng = np.random.default_rng(t * 1000 + d)
    x = torch.tensor(rng.standard_normal((t, h, d)) * 3, device=DEV).to(_DT[xd])
    w = torch.tensor(1 + 0.3 * rng.standard_normal(norm[1]), device=DEV).to(_DT["bf16" if d % 3 else "f32"])
    pos = _positions(rng, t)
    out = torch.zeros((t, h, d), dtype=_DT[od], device=DEV)
    ws = _zeros_ws(256)
    part = B.rope_part(x, out, weight=w if norm[1] else None, norm=norm, eps=1e-5, rope=rope, style=style)
    freq = torch.tensor(_freq(rope[1]), device=DEV) if rope[1] else None
    B.dsa_qk_norm_rope([part], _i32(pos), freq, ws, 256)
    ref, pre = _rope_ref(x.double().cpu().numpy(), pos, w.double().cpu().numpy(), norm, float(np.float32(1e-5)), rope, style)
    _check(out, ref, pre, od)
    B.dsa_read_device_status(ws)


def test_four_parts_to_slots_and_skipped_rows():
    """The step's whole prologue: query shares of a wider projection, latent rows and indexer keys to shuffled slots,
    indexer queries; rows with position -1 and rows with slot -1 stay as they were."""
    rng = np.random.default_rng(8)
    t, h, n = 21, 16, 40
    f = lambda *s: torch.tensor(rng.standard_normal(s), device=DEV).bfloat16()        # noqa: E731
    proj, kv, qi, ki = f(t, h, 192), f(t, 576), f(t, 64, 128), f(t, 128) * 5
    ki[4] = 0
    wkv, wki = f(512).abs(), f(128).float().abs() + 0.1
    q = torch.full((t, h, 576), 7.0, dtype=torch.bfloat16, device=DEV)
    pool = torch.full((n, 576), 9.0, dtype=torch.bfloat16, device=DEV)
    qi8 = torch.full((t, 64, 128), 0x55, dtype=torch.uint8, device=DEV)
    ki8, ks = torch.full((n, 128), 0x55, dtype=torch.uint8, device=DEV), torch.full((n,), 3.0, device=DEV)
    pos = _positions(rng, t)
    pos[6] = -1
    slots = rng.permutation(n)[:t].astype(np.int64)
    slots[9] = -1
    sl = torch.tensor(slots, device=DEV)
    ws = _zeros_ws(256)
    parts = [B.rope_part(proj[:, :, 128:], q[:, :, 512:], rope=(0, 64)),
             B.rope_part(kv, pool, weight=wkv, norm=(0, 512), rope=(512, 64), slots=sl),
             B.rope_part(qi, qi8, rope=(0, 64), style="halves"),
             B.rope_part(ki, ki8, weight=wki, norm=(0, 128), rope=(0, 64), style="halves", slots=sl, scale=ks)]
    B.dsa_qk_norm_rope(parts, _i32(pos), torch.tensor(_freq(64), device=DEV), ws, 256)
    B.dsa_read_device_status(ws)
    eps = float(np.float32(1e-6))
    ok = np.flatnonzero(pos >= 0)
    to = np.array([r for r in ok if slots[r] >= 0])
    num = lambda x: x.double().cpu().numpy()                                          # noqa: E731
    ref, pre = _rope_ref(num(proj[:, :, 128:]), pos, 1, (0, 0), 0, (0, 64), "pairs")
    _check(q[ok][:, :, 512:], ref[ok], pre[ok], "bf16")
    assert (q[:, :, :512] == 7).all() and (q[6] == 7).all()
    ref, pre = _rope_ref(num(kv)[:, None], pos, num(wkv), (0, 512), eps, (512, 64), "pairs")
    _check(pool[slots[to]], ref[to, 0], pre[to, 0], "bf16")
    rest = np.setdiff1d(np.arange(n), slots[to])
    assert (pool[rest] == 9).all() and (ki8[rest] == 0x55).all() and (ks[rest] == 3).all()
    ref, pre = _rope_ref(num(qi), pos, 1, (0, 0), 0, (0, 64), "halves")
    _check(qi8.view(_DT["e4m3"])[ok], ref[ok], pre[ok], "e4m3")
    assert (qi8[6] == 0x55).all()
    ref, pre = _rope_ref(num(ki)[:, None], pos, num(wki), (0, 128), eps, (0, 64), "halves")
    ref, pre = ref[to, 0], pre[to, 0]
    scale = np.abs(ref).max(-1) / 448
    scale[scale == 0] = 1
    got = num(ks)[slots[to]]
    assert (np.abs(got - scale) <= pre.max(-1) / 448 + 4 * U * scale).all()
    # codes of y / scale: the quotient is off by y's error over the scale and by the scale's own share
    q = ref / scale[:, None]
    _check(ki8.view(_DT["e4m3"])[slots[to]], q, pre / scale[:, None] + np.abs(q) * (pre.max(-1) / (448 * scale) + 4 * U)[:, None], "e4m3")
    assert (ki8[slots[4]].view(_DT["e4m3"]).float() == 0).all() and ks[slots[4]] == 1


@pytest.mark.parametrize("xd", ["f32", "bf16"])
def test_unaligned_and_transposed_views(xd):
    """Views that no 16-byte access may touch, heads before rows, and a row broadcast to every head."""
    rng = np.random.default_rng(2)
    t, h, d = 9, 3, 64
    pos, freq, ws = _positions(rng, t), torch.tensor(_freq(64), device=DEV), _zeros_ws(256)
    for layout in ("odd", "heads first", "broadcast"):
        if layout == "odd":
            x = torch.tensor(rng.standard_normal((t, h, d + 3)), device=DEV).to(_DT[xd])[:, :, 1:d + 1]
            out = torch.zeros((t, h, d + 5), dtype=_DT[xd], device=DEV)[:, :, 3:d + 3]
        elif layout == "heads first":
            x = torch.tensor(rng.standard_normal((h, t, d)), device=DEV).to(_DT[xd]).transpose(0, 1)
            out = torch.zeros((h, t, d), dtype=_DT[xd], device=DEV).transpose(0, 1)
        else:
            x = torch.tensor(rng.standard_normal((t, 1, d)), device=DEV).to(_DT[xd]).expand(t, h, d)
            out = torch.zeros((t, h, d), dtype=_DT[xd], device=DEV)
        w = torch.ones(d + 1, dtype=_DT[xd], device=DEV)[1:]
        B.dsa_qk_norm_rope([B.rope_part(x, out, weight=w, norm=(0, d), rope=(0, 64), style="halves")], _i32(pos), freq, ws, 256)
        ref, pre = _rope_ref(x.double().cpu().numpy(), pos, 1.0, (0, d), float(np.float32(1e-6)), (0, 64), "halves")
        _check(out, ref, pre, xd)


def test_rotation_in_place_matches_out_of_place():
    x = torch.randn(50, 7, 128, device=DEV).bfloat16()
    pos, freq, ws = torch.arange(50, dtype=torch.int32, device=DEV) * 997, torch.tensor(_freq(64), device=DEV), _zeros_ws(256)
    w, out, y = torch.rand(128, device=DEV) + 0.5, torch.empty_like(x), x.clone()
    for src, dst in ((x, out), (y, y)):
        B.dsa_qk_norm_rope([B.rope_part(src, dst, weight=w, norm=(0, 128), rope=(64, 64), style="pairs")], pos, freq, ws, 256)
    assert torch.equal(out, y)


def test_rotation_on_other_streams_and_in_a_graph():
    x = torch.randn(40, 6, 64, device=DEV).bfloat16()
    y = torch.randn(40, 6, 64, device=DEV).bfloat16()
    pos, freq = torch.arange(40, dtype=torch.int32, device=DEV) * 31, torch.tensor(_freq(64), device=DEV)
    outs = [torch.zeros_like(x) for _ in range(4)]
    ws = [_zeros_ws(256) for _ in range(2)]
    call = lambda i, o, w, s=None: B.dsa_qk_norm_rope([B.rope_part(i, o, rope=(0, 64))], pos, freq, w, 256, s)      # noqa: E731
    call(x, outs[0], ws[0])
    call(y, outs[1], ws[0])
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(20):
        call(x, outs[2], ws[0], s1)
        call(y, outs[3], ws[1], s2)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[2]) and torch.equal(outs[1], outs[3])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(x, outs[2], ws[0])
    pos.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[2], x)                                      # position 0 turns nothing


def test_slots_past_the_output_are_reported():
    x, out = torch.ones(3, 64, device=DEV), torch.zeros(5, 64, device=DEV)
    ws = _zeros_ws(256)
    B.dsa_qk_norm_rope([B.rope_part(x, out, slots=torch.tensor([4, 5, 0], device=DEV))], None, None, ws, 256)
    with pytest.raises(B.DSAError) as e:
        B.dsa_read_device_status(ws)
    assert e.value.status == B.DSA_ERR_DEVICE_CHECK
    assert out.sum(1).tolist() == [64, 0, 0, 0, 64]


def test_e4m3_saturates_and_keeps_nan():
    x = torch.tensor([[1e4, -1e4, 449, 464.1, 0, -0.0, 2.0 ** -11, float("nan")]], device=DEV)
    out = torch.zeros((1, 8), dtype=torch.float8_e4m3fn, device=DEV)
    B.dsa_qk_norm_rope([B.rope_part(x, out)], None, None, _zeros_ws(256), 256)
    assert out.float()[0, :7].tolist() == [448, -448, 448, 448, 0, 0, 0] and out.float()[0, 7].isnan()


# ------------------------------------------------------------------------------------------------ paged attention
class _Cache:
    """A paged cache with shuffled blocks; whatever no sequence holds is NaN and infinity."""

    def __init__(self, lens, f32=None, seed=0, spare=3, wide=1):
        rng = np.random.default_rng(seed)
        g = torch.Generator(device=DEV)
        g.manual_seed(seed)
        self.lens_h = list(lens)
        pages = [-(-n // 64) for n in lens]
        self.blocks = sum(pages) + spare
        width = max(max(pages), 1) + wide
        ids = rng.permutation(self.blocks)
        table = np.full((len(lens), width), self.blocks - 1)
        at = 0
        for b, p in enumerate(pages):
            table[b, :p] = ids[at:at + p]
            at += p
        self.table_h, self.table, self.lens = table, _i32(table), _i32(lens)
        self.dqk, self.dv, dt = (576, 512, torch.bfloat16) if f32 is None else (*f32, torch.float32)
        self.dt = B.DSA_BF16 if f32 is None else B.DSA_F32
        mk = lambda d: torch.randn((self.blocks, 64, d), generator=g, device=DEV).to(dt)          # noqa: E731
        self.kv, self.v = mk(self.dqk), None if f32 is None else mk(self.dv)
        live = torch.zeros(self.blocks * 64, dtype=torch.bool, device=DEV)
        for b, n in enumerate(lens):
            tok = np.arange(n)
            live[torch.tensor(table[b, tok // 64] * 64 + tok % 64, device=DEV)] = True
        for pool in (self.kv, self.v):
            if pool is not None:
                flat = pool.view(-1, pool.shape[-1])
                flat[~live] = float("nan")
                flat[~live, ::3] = float("inf")
        self.cu = torch.arange(len(lens) + 1, dtype=torch.int32, device=DEV)
        self.torch_dt = dt

    def q(self, heads, seed=1):
        g = torch.Generator(device=DEV)
        g.manual_seed(seed)
        return torch.randn((len(self.lens_h), heads, self.dqk), generator=g, device=DEV).to(self.torch_dt)

    def batch(self, table=None, lens=None):
        n = len(self.lens_h)
        return B.make_batch(self.table if table is None else table, self.lens if lens is None else lens, self.cu,
                            num_blocks=self.blocks, page_size=64, total_q=n, max_q_per_seq=1,
                            max_seq_len=self.table.shape[1] * 64)

    def attend(self, q, scale, pages=None, batch=None, lse=True, ws=None, stream=None, out=None):
        batch = batch or self.batch()
        heads, kb = q.shape[1], 0 if pages is None else pages.shape[1]
        size = B.dsa_workspace_size(B.DSA_OP_PAGED_DECODE, batch, kb, heads, self.dv)
        ws = _zeros_ws(size) if ws is None else ws
        out = torch.full((q.shape[0], heads, self.dv), 5.0, dtype=self.torch_dt, device=DEV) if out is None else out
        ls = torch.full((q.shape[0], heads), 5.0, device=DEV) if lse else None
        B.dsa_paged_attn_decode(q, self.dt, self.kv, self.v, heads, self.dqk, self.dv, scale, pages, kb, batch, out, ls, ws,
                                size, stream)
        self.ws = ws
        return out, ls

    def tokens(self, b, pages=None):
        n = self.lens_h[b]
        if pages is None:
            return np.arange(n)
        got = [np.arange(p * 64, min(n, p * 64 + 64)) for p in pages[b] if 0 <= p and p * 64 < n]
        return np.concatenate(got) if got else np.arange(0)

    def check(self, q, scale, out, lse, pages=None):
        for b in range(len(self.lens_h)):
            tok = self.tokens(b, pages)
            o, ls = out[b].double(), None if lse is None else lse[b].double()
            if not len(tok):
                assert (o == 0).all() and (ls is None or (ls == -float("inf")).all()), b
                continue
            blk, at = torch.tensor(self.table_h[b][tok // 64], device=DEV), torch.tensor(tok % 64, device=DEV)
            k = self.kv[blk, at].double()
            v = k[:, :self.dv] if self.v is None else self.v[blk, at].double()
            qb = q[b].double()
            z = qb @ k.T * scale
            p, ref, lref = torch.softmax(z, 1), torch.softmax(z, 1) @ v, torch.logsumexp(z, 1)
            zerr = (self.dqk * 2.0 ** -23 * (qb.abs() @ k.abs().T).amax(1) * scale)[:, None]      # per head
            bf = 2.0 ** -8 if self.dt == B.DSA_BF16 else 0.0
            tol = (bf + 2 * U) * ref.abs() + (bf + 2 * zerr + 2.0 ** -21 + (len(tok) + 64) * U) * (p @ v.abs())
            bad = (o - ref).abs() > tol
            assert not bad.any(), (b, len(tok), (o - ref).abs().max().item(), tol.min().item())
            if ls is not None:
                lt = zerr[:, 0] + 2.0 ** -21 + (len(tok) + 64) * U + 4 * U * lref.abs()
                assert ((ls - lref).abs() <= lt).all(), (b, (ls - lref).abs().max().item())


def _list(rng, lens, kb, empty=()):
    """Page lists in any order, with -1 among them, pages past the sequence, one page twice."""
    out = np.full((len(lens), kb), -1)
    for b, n in enumerate(lens):
        have = -(-n // 64)
        if b in empty:
            continue
        pick = rng.permutation(max(have, 1) + 2)[:kb]
        out[b, rng.permutation(kb)[:len(pick)]] = pick
    if kb > 2 and len(lens) > 1:
        out[1, 0] = out[1, 1]
        out[0, 2] = 1 << 30
    return out


LENS = [0, 1, 63, 64, 65, 127, 128, 129, 1000, 4097, 0, 300]


@pytest.mark.parametrize("heads", [1, 5, 16, 64, 65, 100, 128])
def test_latent_rows_of_every_length(heads):
    c = _Cache(LENS, seed=heads)
    q = c.q(heads)
    out, lse = c.attend(q, 0.07)
    B.dsa_read_device_status(c.ws)
    c.check(q, 0.07, out, lse)


@pytest.mark.parametrize("heads,dqk,dv", [(1, 1, 1), (4, 64, 64), (16, 128, 128), (5, 61, 50), (16, 32, 128), (3, 128, 7), (9, 6, 2)])
def test_f32_rows_of_every_length(heads, dqk, dv):
    c = _Cache(LENS, f32=(dqk, dv), seed=heads)
    q = c.q(heads)
    out, lse = c.attend(q, dqk ** -0.5)
    B.dsa_read_device_status(c.ws)
    c.check(q, dqk ** -0.5, out, lse)


@pytest.mark.parametrize("heads,f32", [(128, None), (16, None), (4, (64, 64))])
@pytest.mark.parametrize("kb", [1, 3, 32])
def test_page_lists(heads, f32, kb):
    rng = np.random.default_rng(kb)
    c = _Cache(LENS, f32=f32, seed=3)
    q = c.q(heads)
    pages = _list(rng, LENS, kb, empty=(4, 9))
    out, lse = c.attend(q, 0.07, pages=_i32(pages))
    B.dsa_read_device_status(c.ws)
    c.check(q, 0.07, out, lse, pages)


@pytest.mark.parametrize("heads,f32", [(128, None), (4, (64, 64))])
def test_long_runs_of_rows_whose_lists_hold_nothing(heads, f32):
    """Far more rows without a page than pages that a worker has in flight, between rows with one to five pages."""
    rng = np.random.default_rng(0)
    lens = [min(100 + 7 * i, 400) for i in range(2000)]
    pages = np.full((2000, 6), -1)
    for b in (0, 3, 40, 41, 42, 43, 700, 1400, 1999):
        have = -(-lens[b] // 64)
        n = min(have, int(rng.integers(1, 6)))
        pages[b, rng.permutation(6)[:n]] = rng.permutation(have)[:n]
    pages[5:30] = 1 << 20                                               # past every sequence
    c = _Cache(lens, f32=f32, seed=1)
    q = c.q(heads)
    out, lse = c.attend(q, 0.07, pages=_i32(pages))
    B.dsa_read_device_status(c.ws)
    c.check(q, 0.07, out, lse, pages)


@pytest.mark.parametrize("heads,f32", [(128, None), (32, None), (8, (64, 64))])
def test_one_long_row_and_many_short_ones(heads, f32):
    for lens in ([40001], [33] * 300, [1] * 200 + [30000] + [70] * 100, [0] * 7, ([0] * 50 + [65]) * 120, [0] * 40 + [500]):
        c = _Cache(lens, f32=f32, seed=len(lens))
        q = c.q(heads)
        out, lse = c.attend(q, 0.07)
        c.check(q, 0.07, out, lse)


@pytest.mark.parametrize("heads,f32", [(128, None), (4, (64, 64))])
def test_weights_that_grow_along_the_row(heads, f32):
    """Scores that rise steeply (the running maximum moves at every page) and fall steeply (later pages weigh nothing)."""
    for sign in (1, -1):
        c = _Cache([5000, 129], f32=f32, seed=6)
        q = c.q(heads)
        for b, n in enumerate(c.lens_h):
            tok = np.arange(n)
            blk, at = torch.tensor(c.table_h[b][tok // 64], device=DEV), torch.tensor(tok % 64, device=DEV)
            ramp = sign * torch.linspace(-8, 8, n, device=DEV)
            c.kv[blk, at, -8:] = ramp[:, None].to(c.torch_dt)
        q[:, :, -8:] = 16
        out, lse = c.attend(q, 0.07)
        c.check(q, 0.07, out, lse)


@pytest.mark.parametrize("heads,f32", [(128, None), (4, (64, 64))])
def test_same_bits_again_without_lse_on_other_streams_and_with_two_calls_at_once(heads, f32):
    c = _Cache([9000, 77, 0, 2500], f32=f32, seed=9)
    q1, q2 = c.q(heads, 1), c.q(heads, 2)
    ref1, _ = c.attend(q1, 0.07)
    ref2, _ = c.attend(q2, 0.07)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    batch = c.batch()
    size = B.dsa_workspace_size(B.DSA_OP_PAGED_DECODE, batch, 0, heads, c.dv)
    w1, w2 = _zeros_ws(size), _zeros_ws(size)
    o1, o2 = torch.empty_like(ref1), torch.empty_like(ref2)
    torch.cuda.synchronize()
    for _ in range(20):
        c.attend(q1, 0.07, lse=False, ws=w1, stream=s1, out=o1)
        c.attend(q2, 0.07, lse=False, ws=w2, stream=s2, out=o2)
    torch.cuda.synchronize()
    assert torch.equal(o1, ref1) and torch.equal(o2, ref2)


@pytest.mark.parametrize("heads,f32", [(128, None), (20, None), (4, (64, 64))])
@pytest.mark.parametrize("rows,lo,hi,empty", [
    (2, 16, 33, 0), (3, 100, 400, 0), (8, 87, 175, 0), (16, 0, 794, 0), (26, 1, 54, 9), (74, 1, 60, 0), (75, 1, 60, 1),
    (75, 1, 60, 0), (148, 64, 130, 0), (200, 1, 400, 150), (300, 1, 3000, 270), (390, 1, 90, 350), (6, 1035, 2070, 1),
    (40, 1, 900, 0), (30, 60, 70, 0), (100, 300, 1100, 0), (80, 700, 1000, 3), (160, 1, 640, 5), (128, 512, 512, 0), (151, 65, 800, 2),
])
def test_batches_of_rows_of_different_lengths(heads, f32, rows, lo, hi, empty):
    """Small batches are cut into pieces of rows, others into equal ranges of pages: both sides, and where they meet."""
    rng = np.random.default_rng(rows * 7 + hi)
    lens = rng.integers(lo, hi + 1, rows)
    lens[rng.permutation(rows)[:empty]] = 0
    c = _Cache(lens.tolist(), f32=f32, seed=rows)
    q = c.q(heads)
    out, lse = c.attend(q, 0.07)
    B.dsa_read_device_status(c.ws)
    c.check(q, 0.07, out, lse)


@pytest.mark.parametrize("heads,dqk,dv", [(1, 32, 32), (4, 20, 32), (3, 61, 64), (4, 128, 100), (2, 7, 5)])
@pytest.mark.parametrize("rows,hi", [(148, 500), (149, 500), (300, 40), (250, 1000)])
def test_f32_batches_around_the_number_of_workers(heads, dqk, dv, rows, hi):
    rng = np.random.default_rng(rows + heads)
    c = _Cache(rng.integers(0, hi + 1, rows).tolist(), f32=(dqk, dv), seed=rows)
    q = c.q(heads)
    out, lse = c.attend(q, dqk ** -0.5)
    B.dsa_read_device_status(c.ws)
    c.check(q, dqk ** -0.5, out, lse)


@pytest.mark.parametrize("heads,f32", [(128, None), (4, (64, 64))])
def test_a_head_that_is_nan_stays_nan_and_alone(heads, f32):
    """A NaN in one head's query: NaN in its result and its log-sum-exp, whether the row is split or not; the other heads keep
    their bits."""
    c = _Cache([5, 9000], f32=f32, seed=91)
    q = c.q(heads)
    out, lse = c.attend(q, 0.1)
    bad = q.clone()
    bad[:, 2, 3] = float("nan")
    o2, l2 = c.attend(bad, 0.1)
    assert o2[:, 2].isnan().all() and l2[:, 2].isnan().all()
    keep = [h for h in range(heads) if h != 2]
    assert torch.equal(o2[:, keep], out[:, keep]) and torch.equal(l2[:, keep], lse[:, keep])


def test_lengths_and_tables_may_change_under_a_captured_graph():
    c = _Cache([700, 64, 1], seed=12)
    q = c.q(128)
    batch = c.batch()
    size = B.dsa_workspace_size(B.DSA_OP_PAGED_DECODE, batch, 0, 128, 512)
    ws, out = _zeros_ws(size), torch.empty((3, 128, 512), dtype=torch.bfloat16, device=DEV)
    lse = torch.empty((3, 128), device=DEV)
    call = lambda: B.dsa_paged_attn_decode(q, B.DSA_BF16, c.kv, None, 128, 576, 512, 0.07, None, 0, batch, out, lse, ws,  # noqa: E731
                                           size)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for lens in ([700, 64, 1], [1, 0, 1], [699, 3, 0]):
        c.lens_h = lens
        c.lens.copy_(_i32(lens))
        g.replay()
        torch.cuda.synchronize()
        c.check(q, 0.07, out, lse)


def test_bad_block_ids_are_left_out_and_reported():
    c = _Cache([300, 200], seed=4)
    q = c.q(16)
    bad = c.table_h.copy()
    bad[0, 2] = c.blocks
    bad[1, 0] = -1
    table = _i32(bad)                                                   # the batch holds only its address
    out, lse = c.attend(q, 0.07, batch=c.batch(table=table))
    with pytest.raises(B.DSAError) as e:
        B.dsa_read_device_status(c.ws)
    assert e.value.status == B.DSA_ERR_DEVICE_CHECK
    c.check(q, 0.07, out, lse, pages=[[0, 1, 3, 4], [1, 2, 3]])


def test_a_length_past_the_table_is_cut_and_reported():
    c = _Cache([300, 128], seed=4, wide=0)
    q = c.q(16)
    table, cut = _i32(c.table_h[:, :2]), _i32([300, 128])
    batch = B.make_batch(table, cut, c.cu, num_blocks=c.blocks, page_size=64, total_q=2, max_q_per_seq=1,
                         max_seq_len=128)
    out, lse = c.attend(q, 0.07, batch=batch)
    with pytest.raises(B.DSAError):
        B.dsa_read_device_status(c.ws)
    c.lens_h = [128, 128]
    c.check(q, 0.07, out, lse)


@pytest.mark.parametrize("f32", [None, (64, 64)])
def test_blocks_far_into_a_pool_past_32_bit_offsets(f32):
    """A pool whose last blocks lie beyond 2^32 bytes (and 2^31 elements) of its start."""
    c = _Cache([200, 64], f32=f32, seed=2, spare=0)
    n = (1 << 32) // (64 * c.dqk * (2 if f32 is None else 4)) + 40
    n = max(n, (1 << 31) // (64 * c.dqk) + 40)
    if torch.cuda.mem_get_info()[0] < 3 * n * 64 * c.dqk * 4:
        pytest.skip("not enough device memory")
    far = torch.empty((n, 64, c.dqk), dtype=c.torch_dt, device=DEV)
    farv = None if c.v is None else torch.empty((n, 64, c.dv), dtype=c.torch_dt, device=DEV)
    shift = n - c.blocks
    far[shift:] = c.kv
    if farv is not None:
        farv[shift:] = c.v
    q = c.q(4)
    near, _ = c.attend(q, 0.07)
    c.kv, c.v, c.blocks, c.table_h = far, farv, n, c.table_h + shift
    c.table = _i32(c.table_h)
    out, lse = c.attend(q, 0.07)
    assert torch.equal(out, near)
    c.check(q, 0.07, out, lse)


# ------------------------------------------------------------------------------------------------ together
@pytest.mark.parametrize("heads", [128, 16])
def test_prompt_and_decode_steps_through_the_three_calls(heads):
    """Prompts, then decode steps with sequences of different ages: tables, slots and positions from the lengths, rows
    normed, rotated and written to their slots, attention over the cache; against 64-bit attention over the rows as
    stored, and the stored rows against the 64-bit norm and rotation.  The cache starts as NaN."""
    rng = np.random.default_rng(heads)
    n, width, blocks = 5, 12, 40
    t = _Tables(n, width, blocks, rng.permutation(blocks))
    pool = torch.full((blocks, 64, 576), float("nan"), dtype=torch.bfloat16, device=DEV)
    w = torch.tensor(1 + 0.1 * rng.standard_normal(512), device=DEV).bfloat16()
    freq, ws = torch.tensor(_freq(64), device=DEV), _zeros_ws(256)
    lens = np.zeros(n, int)
    inputs = [np.zeros((0, 576)) for _ in range(n)]
    for step, add in enumerate([[130, 64, 0, 1, 300], [1, 1, 65, 1, 1], [1, 0, 1, 62, 1], [1, 1, 1, 1, 20]]):
        add = np.array(add)
        rows = int(add.sum()) + 3                                       # three padding rows
        t.extend(t.lens, add, rows, lens=t.lens, left=t.count)
        kv = torch.tensor(rng.standard_normal((rows, 576)) * 2, device=DEV).bfloat16()
        part = B.rope_part(kv, pool.view(-1, 576), weight=w, norm=(0, 512), rope=(512, 64), slots=t.slots)
        B.dsa_qk_norm_rope([part], t.pos, freq, ws, 256)
        at = 0
        for b in range(n):
            inputs[b] = np.concatenate([inputs[b], kv[at:at + add[b]].double().cpu().numpy()])
            at += add[b]
        lens += add
        q = torch.tensor(rng.standard_normal((n, heads, 576)), device=DEV).bfloat16()
        c = _Cache.__new__(_Cache)
        c.lens_h, c.lens, c.table, c.table_h, c.blocks = list(lens), t.lens, t.table, t.table.cpu().numpy(), blocks
        c.kv, c.v, c.dqk, c.dv, c.dt, c.torch_dt = pool, None, 576, 512, B.DSA_BF16, torch.bfloat16
        c.cu = torch.arange(n + 1, dtype=torch.int32, device=DEV)
        out, lse = c.attend(q, 0.07)
        assert t.status() == B.DSA_OK
        B.dsa_read_device_status(ws)
        B.dsa_read_device_status(c.ws)
        c.check(q, 0.07, out, lse)
    for b in range(n):
        tok = np.arange(lens[b])
        got = pool.view(-1, 576)[torch.tensor(c.table_h[b][tok // 64] * 64 + tok % 64, device=DEV)]
        ref, pre = _rope_ref(inputs[b][:, None], tok, w.double().cpu().numpy(), (0, 512), float(np.float32(1e-6)), (512, 64), "pairs")
        _check(got, ref[:, 0], pre[:, 0], "bf16")


def _view(cache, heads):
    """A _Cache over a PagedCache's state, for its check."""
    c = _Cache.__new__(_Cache)
    c.table, c.lens, c.blocks = cache.block_table, cache.seq_lens, cache.num_blocks
    c.table_h, c.lens_h = cache.block_table.cpu().numpy(), cache.seq_lens.cpu().tolist()
    c.kv, c.v, c.dqk, c.dv, c.dt, c.torch_dt = cache.kv_pool, None, 576, 512, B.DSA_BF16, torch.bfloat16
    return c


def test_paged_cache_sparse_and_paged_attention_agree():
    """A prompt and a decode step in a PagedCache; the sparse path's calls on the same cache (scores, every position
    selected) and the paged attention give the same result, each within its rounding of the 64-bit one."""
    rng = np.random.default_rng(77)
    n, heads = 4, 128
    cache = PagedCache(n, 60, 12, heads)
    f = lambda *s: torch.tensor(rng.standard_normal(s), device=DEV).bfloat16()        # noqa: E731
    w_kv, w_ki, freq = f(512).abs() + 0.5, f(128).abs() + 0.5, torch.tensor(_freq(64), device=DEV)
    for add in ([70, 300, 1, 0], [1, 1, 1, 0]):
        t = sum(add) + 2
        cache.extend(_i32(add), t)
        q_idx_out = torch.zeros((t, 64, 128), dtype=torch.uint8, device=DEV)
        q = torch.zeros((t, heads, 576), dtype=torch.bfloat16, device=DEV)
        q[:, :, :512] = f(t, heads, 512)
        cache.store(f(t, 576), w_kv, freq, k_idx=f(t, 128), k_idx_weight=w_ki, q_rot=f(t, heads, 64), q=q, q_idx=f(t, 64, 128),
                    q_idx_out=q_idx_out)
        cache.check_status()
    q4 = torch.zeros((n, heads, 576), dtype=torch.bfloat16, device=DEV)
    q4[:3] = q[:3]
    out, lse = torch.empty((n, heads, 512), dtype=torch.bfloat16, device=DEV), torch.empty((n, heads), device=DEV)
    cache.attend(q4, out, 0.07, lse=lse)
    cache.check_status()
    c = _view(cache, heads)
    assert c.lens_h == [71, 301, 2, 0]
    c.check(q4, 0.07, out, lse)
    # the sparse path over the same cache: three sequences, 512 candidates at most, all of them selected
    batch = B.make_batch(cache.block_table[:3], cache.seq_lens[:3], cache.cu_q[:4], num_blocks=60, page_size=64, total_q=3,
                         max_q_per_seq=1, max_seq_len=301)
    scores = torch.zeros((3, 304), device=DEV)
    idx = torch.zeros((3, 512), dtype=torch.int32, device=DEV)
    size = max(B.dsa_workspace_size(B.DSA_OP_INDEXER_TOPK, batch, 512), B.dsa_workspace_size(B.DSA_OP_ATTN_DECODE, batch, 512, 128, 512))
    ws = _zeros_ws(size)
    wts = torch.rand((3, 64), device=DEV)
    B.dsa_indexer_topk(q_idx_out[:3].contiguous(), B.DSA_FP8_E4M3, wts, cache.ki_pool, B.DSA_FP8_E4M3, cache.ks_pool, 64, 128,
                       batch, 512, scores, 304, idx, ws, size)
    o2, l2 = torch.empty((3, heads, 512), dtype=torch.bfloat16, device=DEV), torch.empty((3, heads), device=DEV)
    B.dsa_sparse_attn_decode(q4[:3], B.DSA_BF16, cache.kv_pool, None, heads, 576, 512, 0.07, idx, 512, batch, o2, l2, ws, size)
    B.dsa_read_device_status(ws)
    for b, m in enumerate((71, 301, 2)):
        assert idx[b].tolist() == list(range(m)) + [-1] * (512 - m)
    full = torch.zeros_like(out)
    full[:3] = o2
    lfull = torch.full_like(lse, -float("inf"))
    lfull[:3] = l2
    c.check(q4, 0.07, full, lfull)


def test_a_captured_step_replays_as_the_cache_grows():
    """Tables, stores and attention of one decode step in a graph; replays advance the same state, across page borders,
    with slots that are empty and slots that pause."""
    n, heads = 3, 16
    cache = PagedCache(n, 12, 4, heads)
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    new = _i32([1, 1, 0])
    kv = torch.zeros((n, 576), dtype=torch.bfloat16, device=DEV)
    q = torch.randn((n, heads, 576), generator=g, device=DEV).bfloat16()
    w, freq = torch.ones(512, device=DEV), torch.tensor(_freq(64), device=DEV)
    out, lse = torch.empty((n, heads, 512), dtype=torch.bfloat16, device=DEV), torch.empty((n, heads), device=DEV)

    def step():
        cache.extend(new, n)
        cache.store(kv, w, freq)
        cache.attend(q, out, 0.07, lse=lse)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    want = np.array([1, 1, 0])
    for i in range(150):
        add = [1, int(i % 3 != 0), int(i >= 70)]
        new.copy_(_i32(add))
        kv.copy_(torch.randn((n, 576), generator=g, device=DEV))
        graph.replay()
        want += add
        if i in (0, 61, 62, 63, 80, 127, 149):
            cache.check_status()
            assert cache.seq_lens.tolist() == want.tolist()
            _view(cache, heads).check(q, 0.07, out, lse)


def test_two_captured_steps_of_one_cache_take_turns():
    """A decode step and a step of 40-row chunks, captured one after the other: they share the workspace, the tables and the
    descriptors, and are replayed in any order, padding rows among theirs."""
    n, heads = 3, 5
    cache = PagedCache(n, 60, 20, heads)
    g = torch.Generator(device=DEV)
    g.manual_seed(8)
    w, freq = torch.ones(512, device=DEV), torch.tensor(_freq(64), device=DEV)
    q = torch.randn((n, heads, 576), generator=g, device=DEV).bfloat16()
    out, lse = torch.empty((n, heads, 512), dtype=torch.bfloat16, device=DEV), torch.empty((n, heads), device=DEV)
    new = {3: _i32([0, 0, 0]), 40: _i32([0, 0, 0])}
    kv = {t: torch.zeros((t, 576), dtype=torch.bfloat16, device=DEV) for t in new}

    def step(t):
        cache.extend(new[t], t)
        cache.store(kv[t], w, freq)
        cache.attend(q, out, 0.07, lse=lse)

    graphs = {}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for t in new:
            step(t)
    torch.cuda.current_stream().wait_stream(side)
    for t in new:
        graphs[t] = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graphs[t]):
            step(t)
    want, rng = np.zeros(3, dtype=np.int64), np.random.default_rng(8)
    for i in range(30):
        t = 40 if rng.random() < 0.4 else 3
        add = rng.multinomial(rng.integers(0, t + 1), [0.5, 0.3, 0.2]) if t == 40 else rng.integers(0, 2, 3)
        new[t].copy_(_i32(add))
        kv[t].copy_(torch.randn((t, 576), generator=g, device=DEV))
        graphs[t].replay()
        want += add
        if i % 7 == 6 or i == 29:
            cache.check_status()
            assert cache.seq_lens.tolist() == want.tolist()
            assert cache.free_count.item() == 60 - int(sum(-(-want // 64)))
            _view(cache, heads).check(q, 0.07, out, lse)


def test_steps_of_many_sizes_share_buffers_and_keep_their_addresses():
    cache = PagedCache(2, 40, 30, 4)
    seen, total = {}, 0
    for t in (1, 2, 3, 5, 8, 7, 9, 100, 65, 128, 3, 1, 0):
        cache.extend(_i32([t // 2, t - t // 2]), t)
        cache.check_status()
        assert cache.slots.shape == cache.positions.shape == (t,)
        at = (cache.slots.data_ptr(), cache.positions.data_ptr())
        assert seen.setdefault(t, at) == at
        total += t
        assert cache.positions.tolist() == [cache.seq_lens[0].item() - t // 2 + i for i in range(t // 2)] + \
            [cache.seq_lens[1].item() - (t - t // 2) + i for i in range(t - t // 2)]
    assert cache.seq_lens.sum().item() == total and len(cache._rows) <= 8


@pytest.mark.parametrize("change", [
    dict(q=lambda q: q[:1]), dict(q=lambda q: q[:, :2]), dict(q=lambda q: q.float()), dict(out=lambda o: o[:1]),
    dict(out=lambda o: o.float()), dict(lse=lambda x: x[:1]), dict(lse=lambda x: x.bfloat16()),
    dict(pages=lambda p: p[:1]), dict(pages=lambda p: p.long()), dict(pages=lambda p: p[0]), dict(pages=lambda p: p.cpu()),
])
def test_attend_refuses_tensors_of_other_shapes_and_types(change):
    cache = PagedCache(2, 4, 2, 4)
    a = dict(q=torch.zeros((2, 4, 576), dtype=torch.bfloat16, device=DEV),
             out=torch.zeros((2, 4, 512), dtype=torch.bfloat16, device=DEV), lse=torch.zeros((2, 4), device=DEV),
             pages=_i32([[0, 1], [1, -1]]))
    cache.attend(a["q"], a["out"], 0.1, pages=a["pages"], lse=a["lse"])
    cache.check_status()
    for k, f in change.items():
        a[k] = f(a[k])
    with pytest.raises(B.DSAError) as e:
        cache.attend(a["q"], a["out"], 0.1, pages=a["pages"], lse=a["lse"])
    assert e.value.status == B.DSA_ERR_INVALID_ARG


@pytest.mark.parametrize("kind", ["mla", "f32"])
def test_device_batch_paged_attention(kind):
    """The batch's own paged attention: over every page, and over the pages that its block selection keeps, against the
    attention over their token positions."""
    if kind == "mla":
        wl = W.make_workload("paged", kind="mla", seed=31, seq_lens=[700, 64, 65, 1500, 1], q_lens=[1] * 5, topk=128)
    else:
        wl = W.make_workload("paged32", kind="f32", seed=32, seq_lens=[700, 64, 65, 1500, 1], q_lens=[1] * 5, topk=128, H=4,
                             Dqk=64, Dv=64, Hi=2, Di=32)
    db = DeviceBatch(wl)
    db.indexer()
    tol = 2e-2 if kind == "mla" else 1e-5
    for kb in (None, 3):
        if kb is None:
            db.paged_attention()
            idx = np.full((5, 1536), -1)
            for b, m in enumerate(wl.seq_lens):
                idx[b, :m] = np.arange(m)
        else:
            idx = db.block_select(kb).cpu().numpy()
            db.paged_attention(db.block_pages(kb))
        torch.cuda.synchronize()
        out, lse = db.out.float().cpu().numpy(), db.lse.cpu().numpy()
        for b in range(5):
            ref, ref_lse = oracle.sparse_attention_row(wl, b, idx[b])
            assert np.abs(out[b] - ref).max() <= tol and np.abs(lse[b] - ref_lse).max() <= (1e-3 if kind == "mla" else 1e-5)


@pytest.mark.parametrize("xd", ["f32", "bf16"])
@pytest.mark.parametrize("t,h,d,norm,rope,style,slots", [
    (5, 3, 64, (0, 64), (0, 64), "halves", True),          # 4, 8 and 32 lanes per row of a head
    (9, 64, 128, (0, 0), (64, 64), "pairs", False),
    (2, 150, 256, (0, 256), (0, 128), "halves", True),     # more heads than a CTA holds at a time
    (4, 2, 1024, (512, 512), (0, 256), "pairs", True),
    (600, 7, 128, (0, 128), (0, 64), "halves", True),
])
def test_a_scale_for_every_head(xd, t, h, d, norm, rope, style, slots):
    """e4m3 codes with a scale per row and head: scale[row, head], and codes of the head's own scale."""
    rng = np.random.default_rng(t + h)
    n = t + 5
    x = torch.tensor(rng.standard_normal((t, h, d)) * 10.0 ** rng.uniform(-2, 2, (t, h, 1)), device=DEV).to(_DT[xd])
    x[1, 0] = 0
    w = torch.tensor(1 + 0.3 * rng.standard_normal(max(norm[1], 1)), device=DEV).float() if norm[1] else None
    pos = _positions(rng, t)
    to = rng.permutation(n)[:t] if slots else np.arange(t)
    out = torch.full((n, h, d), 0x55, dtype=torch.uint8, device=DEV)
    scale = torch.full((n, h), 3.0, device=DEV)
    ws = _zeros_ws(256)
    part = B.rope_part(x, out, weight=w, norm=norm, rope=rope, style=style, scale=scale,
                       slots=torch.tensor(to, device=DEV) if slots else None)
    B.dsa_qk_norm_rope([part], _i32(pos), torch.tensor(_freq(rope[1]), device=DEV), ws, 256)
    B.dsa_read_device_status(ws)
    ref, pre = _rope_ref(x.double().cpu().numpy(), pos, 1 if w is None else w.double().cpu().numpy(), norm, float(np.float32(1e-6)),
                         rope, style)
    s = np.abs(ref).max(-1) / 448
    s[s == 0] = 1
    got = scale.double().cpu().numpy()[to]
    assert (np.abs(got - s) <= pre.max(-1) / 448 + 4 * U * s).all()
    q = ref / s[..., None]
    slack = pre / s[..., None] + np.abs(q) * (pre.max(-1) / (448 * s) + 4 * U)[..., None]
    _check(out.view(_DT["e4m3"])[torch.tensor(to, device=DEV)], q, slack, "e4m3")
    rest = np.setdiff1d(np.arange(n), to)
    assert (out[rest] == 0x55).all() and (scale[rest] == 3).all()
