"""Host-side checks of the serving step's calls (no GPU): sizes, and refusals before anything is enqueued."""
import ctypes

import pytest

from sparse_attention_long_dsa_b200 import binding as B

P = 1 << 24                                   # a 16-byte aligned address that is never read


def _lib():
    return B.load()


def _err():
    return _lib().dsa_last_error().decode()


def test_workspace_sizes():
    one = B.dsa_batch_workspace_size(B.DSA_OP_BATCH_EXTEND, 1)
    assert one >= 256 and B.dsa_batch_workspace_size(B.DSA_OP_BATCH_RELEASE, 5000) >= one + 8 * 4999
    for op, n in ((B.DSA_OP_TOPK, 4), (B.DSA_OP_BATCH_EXTEND, 0)):
        with pytest.raises(B.DSAError) as e:
            B.dsa_batch_workspace_size(op, n)
        assert e.value.status == B.DSA_ERR_INVALID_ARG
    b = _batch()
    small, large = (B.dsa_workspace_size(B.DSA_OP_PAGED_DECODE, b, 0, h, 512) for h in (1, 128))
    assert 256 < small < large
    assert B.dsa_workspace_size(B.DSA_OP_QK_NORM_ROPE, b) == 256
    assert B.dsa_workspace_size(B.DSA_OP_BATCH_EXTEND, b) == B.dsa_batch_workspace_size(B.DSA_OP_BATCH_EXTEND, b.num_seqs)
    with pytest.raises(B.DSAError) as e:
        B.dsa_workspace_size(B.DSA_OP_PAGED_DECODE, b, 0, 129, 512)
    assert e.value.status == B.DSA_ERR_INVALID_ARG


# ------------------------------------------------------------------------------------------------ block tables
def _extend(**kw):
    d = dict(cached=P, add=2 * P, n=4, page=64, width=8, blocks=100, rows=4, free=3 * P, cap=100, count=4 * P,
             table=5 * P, lens=P, cu=6 * P, slots=7 * P, pos=8 * P, left=4 * P, ws=9 * P, ws_bytes=1 << 20)
    d.update(kw)
    return _lib().dsa_batch_extend(*d.values(), None)


@pytest.mark.parametrize("bad,status", [
    (dict(n=0), B.DSA_ERR_INVALID_ARG),
    (dict(page=128), B.DSA_ERR_UNSUPPORTED),
    (dict(width=0), B.DSA_ERR_INVALID_ARG),
    (dict(width=1 << 26), B.DSA_ERR_UNSUPPORTED),
    (dict(blocks=0), B.DSA_ERR_INVALID_ARG),
    (dict(rows=-1), B.DSA_ERR_INVALID_ARG),
    (dict(rows=(1 << 30) + 1), B.DSA_ERR_UNSUPPORTED),
    (dict(cached=None), B.DSA_ERR_INVALID_ARG),
    (dict(free=None), B.DSA_ERR_INVALID_ARG),
    (dict(cap=-1), B.DSA_ERR_INVALID_ARG),
    (dict(slots=None), B.DSA_ERR_INVALID_ARG),
    (dict(add=P), B.DSA_ERR_INVALID_ARG),              # new_lens is the cached lengths' array
    (dict(ws_bytes=300), B.DSA_ERR_WORKSPACE),
    (dict(ws=None), B.DSA_ERR_WORKSPACE),
    (dict(ws=9 * P + 16), B.DSA_ERR_INVALID_ARG),
])
def test_extend_refusals(bad, status):
    assert _extend(**bad) == status


@pytest.mark.parametrize("rows", [3, 5, 0])
def test_without_cu_q_a_step_has_one_row_per_sequence(rows):
    assert _extend(cu=None, rows=rows) == B.DSA_ERR_INVALID_ARG and "one row per sequence" in _err()


@pytest.mark.parametrize("bad,status", [
    (dict(n=0), B.DSA_ERR_INVALID_ARG),
    (dict(page=32), B.DSA_ERR_UNSUPPORTED),
    (dict(done=None), B.DSA_ERR_INVALID_ARG),
    (dict(done=3 * P), B.DSA_ERR_INVALID_ARG),         # done is seq_lens
    (dict(count=None), B.DSA_ERR_INVALID_ARG),
    (dict(ws_bytes=0), B.DSA_ERR_WORKSPACE),
])
def test_release_refusals(bad, status):
    d = dict(done=P, n=4, page=64, width=8, blocks=100, table=2 * P, lens=3 * P, free=4 * P, cap=100, count=5 * P, ws=6 * P,
             ws_bytes=1 << 20)
    d.update(bad)
    assert _lib().dsa_batch_release(*d.values(), None) == status


# ------------------------------------------------------------------------------------------------ norm and rotation
def _part(**kw):
    d = dict(x=P, out=2 * P, weight=3 * P, x_row_stride=576, x_head_stride=576, out_row_stride=576, out_head_stride=576,
             out_rows=10, H=1, D=576, norm_off=0, norm_len=512, rope_off=512, rope_len=64, x_dt=B.DSA_BF16, w_dt=B.DSA_BF16,
             out_dt=B.DSA_BF16, eps=1e-6)
    d.update(kw)
    return B.dsa_rope_part_t(**d)


def _rope(parts, T=10, pos=4 * P, freq=5 * P, ws=6 * P, ws_bytes=256):
    arr = (B.dsa_rope_part_t * len(parts))(*parts)
    return _lib().dsa_qk_norm_rope(arr, len(parts), pos, T, freq, ws, ws_bytes, None)


@pytest.mark.parametrize("bad,status", [
    (dict(x=None), B.DSA_ERR_INVALID_ARG),
    (dict(H=0), B.DSA_ERR_INVALID_ARG),
    (dict(D=12), B.DSA_ERR_UNSUPPORTED),
    (dict(D=1032), B.DSA_ERR_UNSUPPORTED),
    (dict(x_dt=B.DSA_FP8_E4M3), B.DSA_ERR_UNSUPPORTED),
    (dict(out_dt=7), B.DSA_ERR_UNSUPPORTED),
    (dict(norm_len=584), B.DSA_ERR_INVALID_ARG),
    (dict(norm_len=500), B.DSA_ERR_UNSUPPORTED),
    (dict(weight=None), B.DSA_ERR_INVALID_ARG),
    (dict(w_dt=B.DSA_FP8_E4M3), B.DSA_ERR_UNSUPPORTED),
    (dict(eps=float("nan")), B.DSA_ERR_INVALID_ARG),
    (dict(eps=-1.0), B.DSA_ERR_INVALID_ARG),
    (dict(rope_off=520), B.DSA_ERR_INVALID_ARG),
    (dict(rope_off=508), B.DSA_ERR_UNSUPPORTED),
    (dict(rope_len=8), B.DSA_ERR_UNSUPPORTED),
    (dict(rope_off=0, rope_len=272), B.DSA_ERR_UNSUPPORTED),
    (dict(rope_style=2), B.DSA_ERR_INVALID_ARG),
    (dict(out_scale=P), B.DSA_ERR_INVALID_ARG),        # a scale goes with e4m3
    (dict(x_row_stride=-1), B.DSA_ERR_INVALID_ARG),
    (dict(out_row_stride=512), B.DSA_ERR_INVALID_ARG),
    (dict(H=2, out_head_stride=64), B.DSA_ERR_INVALID_ARG),
    (dict(out_rows=9), B.DSA_ERR_INVALID_ARG),
    (dict(slots=P, out_rows=0), B.DSA_ERR_INVALID_ARG),
    (dict(slots=P + 4), B.DSA_ERR_INVALID_ARG),
    (dict(x=P + 1), B.DSA_ERR_INVALID_ARG),
])
def test_rope_part_refusals(bad, status):
    assert _rope([_part(), _part(**bad)]) == status


def test_rope_call_refusals():
    assert _rope([_part()], pos=None) == B.DSA_ERR_INVALID_ARG
    assert _rope([_part()], freq=None) == B.DSA_ERR_INVALID_ARG
    assert _rope([_part(), _part(rope_len=32)]) == B.DSA_ERR_INVALID_ARG and "differs" in _err()
    assert _rope([_part()] * 5) == B.DSA_ERR_UNSUPPORTED
    assert _rope([_part()], T=-1) == B.DSA_ERR_INVALID_ARG
    assert _rope([_part(out_rows=1 << 31)], T=(1 << 30) + 1) == B.DSA_ERR_UNSUPPORTED
    assert _rope([_part()], ws_bytes=128) == B.DSA_ERR_WORKSPACE
    assert _rope([_part(x=None)], T=0) == B.DSA_OK                       # empty: checked only for its sizes
    assert _lib().dsa_qk_norm_rope(None, 1, P, 1, P, P, 256, None) == B.DSA_ERR_INVALID_ARG


@pytest.mark.parametrize("H,rows,row,head,ok", [
    (2, 10, 64, 64, False),                            # row t's second head is row t + 1's first
    (3, 10, 191, 64, False),
    (3, 10, 192, 64, True),
    (3, 10, 64, 639, False),                           # heads first
    (3, 10, 64, 640, True),
    (3, 10, 100, 963, False),
    (3, 10, 100, 964, True),
    (128, 10, 128 * 576, 576, True),                   # a view of 64 entries of wider rows
    (128, 10, 127 * 576 + 63, 576, False),
    (2, 1 << 40, 64, 1 << 46, True),                   # strides whose products pass 64 bits
    (2, 1 << 60, 1 << 60, 1 << 60, False),
    (2, 1 << 60, 1 << 60, 64, True),
    (1, 10, 64, 0, True),
])
def test_rope_output_rows_and_heads_may_not_overlap(H, rows, row, head, ok):
    part = _part(H=H, D=64, norm_len=0, rope_off=0, x_row_stride=64 * H, x_head_stride=64, out_rows=rows, out_row_stride=row,
                 out_head_stride=head)
    status = _rope([part], ws_bytes=128)               # the workspace is looked at after the parts
    assert status == (B.DSA_ERR_WORKSPACE if ok else B.DSA_ERR_INVALID_ARG)
    assert ok or "overlap" in _err()


@pytest.mark.parametrize("T,change,ok", [
    (10, dict(), True),
    (10, dict(x_dt=B.DSA_F32), False),                 # rows of f32 under rows of bf16: other rows' inputs are overwritten
    (1, dict(x_dt=B.DSA_F32), False),
    (10, dict(out_row_stride=1152), False),
    (1, dict(out_row_stride=1152), True),              # one row has no stride
    (10, dict(H=2, x_row_stride=1152, out_row_stride=1152), True),
    (10, dict(H=2, x_row_stride=1152, x_head_stride=0, out_row_stride=1152), False),
    (10, dict(slots=8 * P), False),
    (10, dict(out=4 * P, slots=8 * P), True),
])
def test_rope_in_place_needs_the_same_layout(T, change, ok):
    part = _part(**{**dict(out=P), **change})
    assert _rope([part], T=T, ws_bytes=128) == (B.DSA_ERR_WORKSPACE if ok else B.DSA_ERR_INVALID_ARG)


# ------------------------------------------------------------------------------------------------ paged attention
def _batch(**kw):
    d = dict(num_seqs=3, page_size=64, num_blocks=40, max_blocks_per_seq=4, block_table=1 << 20, seq_lens=1 << 21,
             cu_q=1 << 22, total_q=3, max_q_per_seq=1, max_seq_len=200)
    d.update(kw)
    return B.dsa_batch_t(**d)


def _attn(batch=None, **kw):
    d = dict(q=P, dt=B.DSA_BF16, kv=2 * P, v=None, H=128, Dqk=576, Dv=512, scale=0.1, pages=None, kb=0)
    d.update(kw)
    b = batch or _batch()
    ws = kw.pop("ws_bytes", 1 << 30)
    d.pop("ws_bytes", None)
    return _lib().dsa_paged_attn_decode(*d.values(), ctypes.byref(b), 3 * P, None, 4 * P, ws, None)


@pytest.mark.parametrize("bad,status", [
    (dict(q=None), B.DSA_ERR_INVALID_ARG),
    (dict(H=0), B.DSA_ERR_UNSUPPORTED),
    (dict(H=129), B.DSA_ERR_UNSUPPORTED),
    (dict(Dqk=512), B.DSA_ERR_UNSUPPORTED),
    (dict(v=P), B.DSA_ERR_UNSUPPORTED),
    (dict(dt=B.DSA_FP8_E4M3), B.DSA_ERR_UNSUPPORTED),
    (dict(dt=B.DSA_F32, H=17, Dqk=64, Dv=64, v=P), B.DSA_ERR_UNSUPPORTED),
    (dict(dt=B.DSA_F32, H=4, Dqk=64, Dv=64), B.DSA_ERR_UNSUPPORTED),      # f32 needs its own value cache
    (dict(scale=0.0), B.DSA_ERR_INVALID_ARG),
    (dict(scale=float("nan")), B.DSA_ERR_INVALID_ARG),
    (dict(kb=4), B.DSA_ERR_INVALID_ARG),
    (dict(pages=P, kb=0), B.DSA_ERR_INVALID_ARG),
    (dict(pages=P, kb=1 << 30), B.DSA_ERR_UNSUPPORTED),
    (dict(kv=2 * P + 8), B.DSA_ERR_INVALID_ARG),
    (dict(ws_bytes=1024), B.DSA_ERR_WORKSPACE),
])
def test_paged_attention_refusals(bad, status):
    assert _attn(**bad) == status


def test_paged_attention_batch_refusals():
    assert _attn(_batch(total_q=4, max_q_per_seq=2)) == B.DSA_ERR_INVALID_ARG and "one query row" in _err()
    assert _attn(_batch(page_size=32)) == B.DSA_ERR_UNSUPPORTED
    assert _attn(_batch(num_blocks=1 << 25)) == B.DSA_ERR_UNSUPPORTED
    assert _attn(_batch(total_q=0, max_q_per_seq=0), q=None) == B.DSA_OK


def test_binding_refuses_host_tensors():
    import torch
    t = torch.zeros(4, 64)
    with pytest.raises(B.DSAError) as e:
        B.rope_part(t, t)
    assert e.value.status == B.DSA_ERR_INVALID_ARG
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(B.DSAError) as e:
        B.dsa_batch_extend(i, i, 64, 4, 4, i, i, torch.zeros(4, 2, dtype=torch.int32), i, torch.zeros(5, dtype=torch.int32), i,
                           i, i, 1 << 24, 1 << 20)
    assert e.value.status == B.DSA_ERR_INVALID_ARG
    with pytest.raises(B.DSAError) as e:
        B.dsa_qk_norm_rope([], None, None, 1 << 24, 256)
    assert e.value.status == B.DSA_ERR_UNSUPPORTED


# ------------------------------------------------------------------------------------------------ devices
class _On:
    """What the binding looks at of a dense device tensor, without the device."""
    is_cuda = True

    def __init__(self, device, at=P):
        self.device_index, self.at = device, at

    def get_device(self):
        return self.device_index

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return self.at


class _Pages(_On):
    def __init__(self, shape, dtype, device=0):
        super().__init__(device, 0 if 0 in shape else P)          # an empty tensor's address is NULL
        self.shape, self.dtype = shape, dtype

    def dim(self):
        return len(self.shape)


@pytest.mark.parametrize("where", [None, "q", "kv_pool", "pages", "out", "lse", "ws"])
def test_paged_attention_takes_tensors_of_the_current_device(monkeypatch, where):
    import torch
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    t = {n: _On(int(n == where)) for n in ("q", "kv_pool", "out", "lse", "ws")}
    t["pages"] = _Pages((3, 4), torch.int32, int(where == "pages"))
    with pytest.raises(B.DSAError) as e:
        B.dsa_paged_attn_decode(t["q"], B.DSA_BF16, t["kv_pool"], None, 128, 576, 512, 0.1, t["pages"], 4, _batch(), t["out"],
                                t["lse"], t["ws"], 1024, stream=1)
    # all here: the library is asked, and finds the workspace too small
    assert e.value.status == (B.DSA_ERR_WORKSPACE if where is None else B.DSA_ERR_INVALID_ARG)
    assert where in (None, "pages") or "cuda:1" in str(e.value)


@pytest.mark.parametrize("call", ["extend", "release", "rotation"])
@pytest.mark.parametrize("device", [0, 1])
def test_workspaces_belong_to_the_current_device(monkeypatch, call, device):
    import torch
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    monkeypatch.setattr(B, "_dense", lambda what, dtype, *tensors: [P + 64 * i for i in range(len(tensors))])
    i, table, ws = torch.zeros(4, dtype=torch.int32), torch.zeros((4, 2), dtype=torch.int32), _On(device)
    with pytest.raises(B.DSAError) as e:
        if call == "extend":
            B.dsa_batch_extend(i, i, 64, 4, 4, i, i, table, i, torch.zeros(5, dtype=torch.int32), i, i, i, ws, 16, stream=1)
        elif call == "release":
            B.dsa_batch_release(i, 64, 4, table, i, i, i, ws, 16, stream=1)
        else:
            part = _part()
            part.rows, part.device, part.rotated = 10, 0, 64
            B.dsa_qk_norm_rope([part], torch.zeros(10, dtype=torch.int32), torch.zeros(32), ws, 16, stream=1)
    assert e.value.status == (B.DSA_ERR_WORKSPACE if device == 0 else B.DSA_ERR_INVALID_ARG)


@pytest.mark.parametrize("shape,kb,dtype", [
    ((3, 0), 0, "int32"),                                    # lists that hold nothing are no request for every page
    ((3, 4), 5, "int32"), ((2, 4), 4, "int32"), ((12,), 4, "int32"), ((3, 4), 4, "int64"),
])
def test_paged_attention_takes_page_lists_of_its_rows(monkeypatch, shape, kb, dtype):
    import torch
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    t = [_On(0) for _ in range(5)]
    with pytest.raises(B.DSAError) as e:
        B.dsa_paged_attn_decode(t[0], B.DSA_BF16, t[1], None, 128, 576, 512, 0.1, _Pages(shape, getattr(torch, dtype)), kb,
                                _batch(), t[2], t[3], t[4], 1024, stream=1)
    assert e.value.status == B.DSA_ERR_INVALID_ARG
