"""Cases of the serving step around the paged cache: what is measured, and the operators' plain forms.

Three operators that belong to one decode (or prefill) step over the paged cache:

* extend: block tables and slot maps built on the GPU from the requests' lengths (dsa_batch_extend);
* rope:   RMS norms and the position rotation of queries, latent rows and indexer rows in one pass, written as
          bf16, f32 or e4m3, densely or to the cache's slots (dsa_qk_norm_rope);
* attn:   softmax attention of one new token per sequence over the whole paged cache, or over the pages that a
          block selection kept (dsa_paged_attn_decode).

`own` false computes them with elementary torch operations in 32 bits (64 for angles), rounded once at the end;
`own` true makes the library's calls.
"""
import math
import random

import numpy as np
import torch

own = False

PAGE = 64
LATENT, VALUE, ROPE = 576, 512, 64          # a latent row: 512 value entries, then 64 rotated ones
IDX_H, IDX_D = 64, 128                      # indexer heads and key width
EPS = 1e-6
E4M3_MAX = 448.0


# ------------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # one decode step of 32 running requests: latency
        {"name": "extend_decode_32", "op": "extend", "seqs": 32, "lo": 4096, "hi": 32768, "new": 1, "chunks": 0, "chunk": 0},
        # a mixed step: 16 decodes and two 8192-token prefill chunks behind 57,344 cached tokens
        {"name": "extend_mixed", "op": "extend", "seqs": 16, "lo": 8192, "hi": 131072, "new": 1, "chunks": 2, "chunk": 8192},
        # a wave of 64 prompts of 1 to 16384 tokens admitted at once into an empty cache
        {"name": "extend_prompts", "op": "extend", "seqs": 64, "lo": 0, "hi": 0, "new": 16384, "chunks": 0, "chunk": 0},
        # the rotation step of a 32-row decode batch: 128 query heads, latent row, 64 indexer heads, indexer key
        {"name": "rope_decode_32", "op": "rope", "form": "mla", "rows": 32, "heads": 128, "far": 32768},
        # the same for a 16k-token prompt
        {"name": "rope_prefill_16k", "op": "rope", "form": "mla", "rows": 16384, "heads": 128, "far": 16384},
        # normed and rotated heads of a fused projection, odd counts, positions of a million-token context
        {"name": "rope_heads_1021", "op": "rope", "form": "heads", "rows": 1021, "heads": 5, "kheads": 1, "width": 128,
         "rot": 64, "style": "halves", "type": "bf16", "far": 1048576},
        # one short sequence: latency
        {"name": "attn_short", "op": "attn", "type": "bf16", "rows": 1, "lo": 130, "hi": 130, "heads": 128, "keep": 0},
        # the 32-row decode batch over contexts of 4K to 32K tokens
        {"name": "attn_decode_32", "op": "attn", "type": "bf16", "rows": 32, "lo": 4096, "hi": 32768, "heads": 128, "keep": 0},
        # a head shard of 16, many rows of odd lengths, empty rows among them (padding of a captured batch)
        {"name": "attn_shard_16", "op": "attn", "type": "bf16", "rows": 61, "lo": 0, "hi": 8191, "heads": 16, "keep": 0},
        # one row over 1,048,576 tokens
        {"name": "attn_1m", "op": "attn", "type": "bf16", "rows": 1, "lo": 1048576, "hi": 1048576, "heads": 128, "keep": 0},
        # the decode batch over the 32 pages per row that a block selection kept
        {"name": "attn_pages_32", "op": "attn", "type": "bf16", "rows": 32, "lo": 100, "hi": 32768, "heads": 128, "keep": 32},
        # the f32 path: separate keys and values of 64, four heads
        {"name": "attn_f32", "op": "attn", "type": "f32", "rows": 16, "lo": 256, "hi": 8192, "heads": 4, "dqk": 64, "dv": 64,
         "keep": 0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["extend", "rope", "rope", "attn", "attn", "attn"])
    if op == "extend":
        kind = rng.randrange(3)
        if kind == 0:
            return {"op": op, "seqs": _log(rng, 1, 512), "lo": 1, "hi": _log(rng, 64, 65536), "new": rng.choice([1, 1, 2, 5]),
                    "chunks": 0, "chunk": 0}
        if kind == 1:
            return {"op": op, "seqs": _log(rng, 1, 64), "lo": 0, "hi": _log(rng, 64, 131072), "new": 1,
                    "chunks": rng.randint(1, 4), "chunk": _log(rng, 17, 8192)}
        return {"op": op, "seqs": _log(rng, 1, 64), "lo": 0, "hi": 0, "new": _log(rng, 10, 16384), "chunks": 0, "chunk": 0}
    if op == "rope":
        if rng.random() < 0.5:
            return {"op": op, "form": "mla", "rows": _log(rng, 1, 16384), "heads": rng.choice([128, 64, 32, 16]),
                    "far": _log(rng, 16384, 1048576)}
        width = rng.choice([64, 128, 192, 256])
        return {"op": op, "form": "heads", "rows": _log(rng, 1, 16384), "heads": rng.randint(1, 40), "kheads": rng.randint(1, 8),
                "width": width, "rot": rng.choice([32, 64, width]), "style": rng.choice(["halves", "pairs"]),
                "type": rng.choice(["bf16", "bf16", "f32"]), "far": _log(rng, 16384, 1048576)}
    rows = _log(rng, 1, 256)
    top = _log(rng, 32, max(33, min(131072, (1 << 19) // rows)))
    lo = rng.choice([0, 1, top // 2])
    if rng.random() < 0.25:
        return {"op": op, "type": "f32", "rows": rows, "lo": lo, "hi": top, "heads": rng.randint(1, 16),
                "dqk": rng.choice([32, 61, 64, 128]), "dv": rng.choice([32, 50, 64, 128]), "keep": rng.choice([0, 0, 7])}
    return {"op": op, "type": "bf16", "rows": rows, "lo": lo, "hi": top, "heads": rng.choice([128, 128, 64, 100, 32, 16, 5, 1]),
            "keep": rng.choice([0, 0, 0, _log(rng, 1, 64)])}


def _lengths(case, n, lo, hi):
    """The lengths of a case's requests: fixed by the case, so that its work is too."""
    r = random.Random("%s %d %d %d %s" % (case["op"], n, lo, hi, case.get("heads", 0)))
    return [r.randint(lo, hi) for _ in range(n)]


def _extend_lengths(case):
    n = case["seqs"]
    cached = _lengths(case, n, case["lo"], case["hi"])
    new = [case["new"]] * n if case["hi"] else _lengths(case, n, 1, case["new"])
    return cached + [7 * case["chunk"]] * case["chunks"], new + [case["chunk"]] * case["chunks"]


def _attn_lengths(case):
    return _lengths(case, case["rows"], case["lo"], case["hi"])


# ------------------------------------------------------------------------------------------------ inputs
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(g, shape, dtype):
    """Standard normal values, drawn in pieces so that the 32-bit draws of a large pool do not add up."""
    out = torch.empty(shape, dtype=dtype, device="cuda")
    flat = out.view(-1)
    for at in range(0, flat.numel(), 1 << 27):
        flat[at:at + (1 << 27)] = torch.randn(min(1 << 27, flat.numel() - at), generator=g, device="cuda")
    return out


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _prepare_extend(case, g):
    cached, new = _extend_lengths(case)
    owned = [-(-n // PAGE) for n in cached]
    after = [-(-(c + n) // PAGE) for c, n in zip(cached, new)]
    width = max(after) + 3
    spare = sum(after) - sum(owned) + 17
    ids = torch.randperm(sum(owned) + spare, generator=g, device="cuda").to(torch.int32)
    col = torch.arange(width, device="cuda")[None]
    own_n = _ints(owned)[:, None]
    start = torch.cumsum(own_n, 0) - own_n
    held = col < own_n
    table = torch.where(held, ids[(start + col).clamp(max=len(ids) - 1)], torch.full((), -1, dtype=torch.int32, device="cuda"))
    free = torch.full((len(ids),), -1, dtype=torch.int32, device="cuda")
    free[:spare] = ids[sum(owned):]
    rows, n = sum(new), len(cached)
    return dict(cached=_ints(cached), new=_ints(new), table=table.contiguous(), free=free, count=_ints([spare]),
                blocks=len(ids), rows=rows, seq_lens=torch.empty(n, dtype=torch.int32, device="cuda"),
                cu_q=torch.empty(n + 1, dtype=torch.int32, device="cuda"),
                slots=torch.empty(rows, dtype=torch.int64, device="cuda"),
                positions=torch.empty(rows, dtype=torch.int32, device="cuda"), left=_ints([0]))


def _prepare_rope(case, g):
    t, rot = case["rows"], ROPE if case["form"] == "mla" else case["rot"]
    s = dict(positions=torch.randint(0, case["far"], (t,), generator=g, device="cuda", dtype=torch.int32),
             freq=10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot))
    bf16, u8 = torch.bfloat16, torch.uint8
    if case["form"] == "heads":
        dt = bf16 if case["type"] == "bf16" else torch.float32
        h, hk, d = case["heads"], case["kheads"], case["width"]
        proj = _normal(g, (t, h + 2 * hk, d), dt)               # queries, keys and values of one projection
        return dict(s, q_in=proj[:, :h], k_in=proj[:, h:h + hk], q_weight=1 + 0.1 * _normal(g, (d,), torch.float32),
                    k_weight=1 + 0.1 * _normal(g, (d,), torch.float32), q=torch.empty((t, h, d), dtype=dt, device="cuda"),
                    k=torch.empty((t, hk, d), dtype=dt, device="cuda"))
    h = case["heads"]
    tokens = -(-max(4 * t, 4096) // PAGE) * PAGE if t <= 4096 else -(-t // PAGE) * PAGE
    return dict(s, q_in=_normal(g, (t, h, 192), bf16)[:, :, 128:], q=torch.zeros((t, h, LATENT), dtype=bf16, device="cuda"),
                kv_in=2 * _normal(g, (t, LATENT), bf16), kv_weight=(1 + 0.1 * _normal(g, (VALUE,), torch.float32)).to(bf16),
                qi_in=_normal(g, (t, IDX_H, IDX_D), bf16), qi=torch.empty((t, IDX_H, IDX_D), dtype=u8, device="cuda"),
                ki_in=_normal(g, (t, IDX_D), bf16), ki_weight=1 + 0.1 * _normal(g, (IDX_D,), torch.float32),
                slots=torch.randperm(tokens, generator=g, device="cuda")[:t].contiguous(),
                kv_pool=_normal(g, (tokens, LATENT), bf16), ki_pool=torch.zeros((tokens, IDX_D), dtype=u8, device="cuda"),
                ks_pool=torch.ones((tokens,), dtype=torch.float32, device="cuda"))


def _prepare_attn(case, g):
    lens = _attn_lengths(case)
    pages = [-(-n // PAGE) for n in lens]
    width, blocks = max(max(pages), 1), sum(pages) + 3
    perm = torch.randperm(blocks, generator=g, device="cuda").to(torch.int32)
    col, n = torch.arange(width, device="cuda")[None], _ints(pages)[:, None]
    start = torch.cumsum(n, 0) - n
    table = torch.where(col < n, perm[(start + col).clamp(max=blocks - 1)], torch.zeros((), dtype=torch.int32, device="cuda"))
    f32 = case["type"] == "f32"
    dt, dqk, dv = (torch.float32, case["dqk"], case["dv"]) if f32 else (torch.bfloat16, LATENT, VALUE)
    rows, heads = case["rows"], case["heads"]
    kept = None
    if case["keep"]:
        # the kept pages of each row in ascending order, -1 behind them where the row has fewer: as the top-k gives them
        key = torch.rand((rows, width), generator=g, device="cuda").masked_fill(col >= n, 2.0)
        key = torch.nn.functional.pad(key, (0, max(0, case["keep"] - width)), value=2.0)
        best = torch.topk(key, case["keep"], dim=1, largest=False)
        at = torch.where(best.values < 2.0, best.indices, torch.full_like(best.indices, 1 << 30)).sort(dim=1).values
        kept = torch.where(at < (1 << 30), at, torch.full_like(at, -1)).to(torch.int32).contiguous()
    return dict(q=_normal(g, (rows, heads, dqk), dt), kv_pool=_normal(g, (blocks, PAGE, dqk), dt),
                v_pool=_normal(g, (blocks, PAGE, dv), dt) if f32 else None, table=table.contiguous(), lens=_ints(lens),
                cu_q=torch.arange(rows + 1, dtype=torch.int32, device="cuda"), kept=kept, top=max(max(lens), 1), dv=dv,
                scale=1 / math.sqrt(dqk if f32 else 192), out=torch.empty((rows, heads, dv), dtype=dt, device="cuda"),
                lse=torch.empty((rows, heads), dtype=torch.float32, device="cuda"))


def prepare(case, seed):
    g = _generator(seed)
    s = {"extend": _prepare_extend, "rope": _prepare_rope, "attn": _prepare_attn}[case["op"]](case, g)
    return dict(s, case=dict(case))


# ------------------------------------------------------------------------------------------------ the library's calls
def _plan_extend(s):
    from sparse_attention_long_dsa_b200 import binding as B
    size = B.dsa_batch_workspace_size(B.DSA_OP_BATCH_EXTEND, s["cached"].numel())
    return B, torch.zeros(size, dtype=torch.uint8, device="cuda"), size


def _own_extend(s):
    if "plan" not in s:
        s["plan"] = _plan_extend(s)
    B, ws, size = s["plan"]
    B.dsa_batch_extend(s["cached"], s["new"], PAGE, s["blocks"], s["rows"], s["free"], s["count"], s["table"], s["seq_lens"],
                       s["cu_q"], s["slots"], s["positions"], s["left"], ws, size)
    return {"table": s["table"], "seq_lens": s["seq_lens"], "cu_q": s["cu_q"], "slots": s["slots"],
            "positions": s["positions"], "left": s["left"]}


def _plan_rope(s):
    from sparse_attention_long_dsa_b200 import binding as B
    c, ws = s["case"], torch.zeros(256, dtype=torch.uint8, device="cuda")
    if c["form"] == "heads":
        d, rot = c["width"], (0, c["rot"])
        parts = [B.rope_part(s["q_in"], s["q"], weight=s["q_weight"], norm=(0, d), eps=EPS, rope=rot, style=c["style"]),
                 B.rope_part(s["k_in"], s["k"], weight=s["k_weight"], norm=(0, d), eps=EPS, rope=rot, style=c["style"])]
    else:
        parts = [B.rope_part(s["q_in"], s["q"][:, :, VALUE:], rope=(0, ROPE), style="pairs"),
                 B.rope_part(s["kv_in"], s["kv_pool"], weight=s["kv_weight"], norm=(0, VALUE), eps=EPS, rope=(VALUE, ROPE),
                             style="pairs", slots=s["slots"]),
                 B.rope_part(s["qi_in"], s["qi"], rope=(0, ROPE), style="halves"),
                 B.rope_part(s["ki_in"], s["ki_pool"], weight=s["ki_weight"], norm=(0, IDX_D), eps=EPS, rope=(0, ROPE),
                             style="halves", slots=s["slots"], scale=s["ks_pool"])]
    return B, parts, ws


def _own_rope(s):
    if "plan" not in s:
        s["plan"] = _plan_rope(s)
    B, parts, ws = s["plan"]
    B.dsa_qk_norm_rope(parts, s["positions"], s["freq"], ws, 256)
    return _rope_outputs(s)


def _rope_outputs(s):
    if s["case"]["form"] == "heads":
        return {"q": s["q"], "k": s["k"]}
    fp8 = torch.float8_e4m3fn
    return {"q": s["q"][:, :, VALUE:], "kv_pool": s["kv_pool"], "qi": s["qi"].view(fp8), "ki_pool": s["ki_pool"].view(fp8),
            "ks_pool": s["ks_pool"]}


def _plan_attn(s):
    from sparse_attention_long_dsa_b200 import binding as B
    rows, blocks = s["q"].shape[0], s["kv_pool"].shape[0]
    batch = B.make_batch(s["table"], s["lens"], s["cu_q"], num_blocks=blocks, page_size=PAGE, total_q=rows, max_q_per_seq=1,
                         max_seq_len=s["top"])
    size = B.dsa_workspace_size(B.DSA_OP_PAGED_DECODE, batch, s["case"]["keep"], s["q"].shape[1], s["dv"])
    return B, batch, torch.zeros(size, dtype=torch.uint8, device="cuda"), size


def _own_attn(s):
    if "plan" not in s:
        s["plan"] = _plan_attn(s)
    B, batch, ws, size = s["plan"]
    heads, dqk = s["q"].shape[1:]
    dt = B.DSA_BF16 if s["v_pool"] is None else B.DSA_F32
    B.dsa_paged_attn_decode(s["q"], dt, s["kv_pool"], s["v_pool"], heads, dqk, s["dv"], s["scale"], s["kept"],
                            s["case"]["keep"], batch, s["out"], s["lse"], ws, size)
    return {"out": s["out"], "lse": s["lse"]}


# ------------------------------------------------------------------------------------------------ plain forms
def _plain_extend(s):
    cached, new, table, free = s["cached"].long(), s["new"].long(), s["table"], s["free"]
    seq = cached + new
    held, after = (cached + PAGE - 1) // PAGE, (seq + PAGE - 1) // PAGE
    need = after - held
    ends = torch.cumsum(need, 0)
    col = torch.arange(table.shape[1], device="cuda")[None]
    nth = (ends - need)[:, None] + col - held[:, None]             # the step's how-manieth new page
    fresh = (col >= held[:, None]) & (col < after[:, None])
    count = s["count"].long()
    table = torch.where(fresh, free[(count - 1 - nth).clamp(0, free.numel() - 1)], table)
    cu = torch.nn.functional.pad(torch.cumsum(new, 0), (1, 0))
    row = torch.arange(s["rows"], device="cuda")
    b = torch.searchsorted(cu[1:], row, right=True)
    pos = cached[b] + row - cu[b]
    slots = table[b, pos // PAGE].long() * PAGE + pos % PAGE
    return {"table": table, "seq_lens": seq.int(), "cu_q": cu.int(), "slots": slots, "positions": pos.int(),
            "left": (count - ends[-1:]).int()}


def _rotate(x, cos, sin, style):
    """x [T, H, R] turned by the angles whose cosines and sines are [T, 1, R / 2]."""
    a, b = (x[..., 0::2], x[..., 1::2]) if style == "pairs" else x.chunk(2, dim=-1)
    u, v = a * cos - b * sin, b * cos + a * sin
    return torch.stack((u, v), dim=-1).flatten(-2) if style == "pairs" else torch.cat((u, v), dim=-1)


def _rms(x, weight):
    return x * torch.rsqrt((x * x).mean(dim=-1, keepdim=True) + EPS) * weight.float()


def _plain_rope(s):
    c = s["case"]
    angle = s["positions"].double()[:, None, None] * s["freq"]
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    if c["form"] == "heads":
        rot, style = c["rot"], c["style"]
        q, k = _rms(s["q_in"].float(), s["q_weight"]), _rms(s["k_in"].float(), s["k_weight"])
        s["q"].copy_(torch.cat((_rotate(q[..., :rot], cos, sin, style), q[..., rot:]), dim=-1))
        s["k"].copy_(torch.cat((_rotate(k[..., :rot], cos, sin, style), k[..., rot:]), dim=-1))
        return _rope_outputs(s)
    fp8 = torch.float8_e4m3fn
    s["q"][:, :, VALUE:] = _rotate(s["q_in"].float(), cos, sin, "pairs").bfloat16()
    kv = s["kv_in"].float()
    turned = _rotate(kv[:, None, VALUE:], cos, sin, "pairs")[:, 0]
    s["kv_pool"][s["slots"]] = torch.cat((_rms(kv[:, :VALUE], s["kv_weight"]), turned), dim=-1).bfloat16()
    qi = s["qi_in"].float()
    qi = torch.cat((_rotate(qi[..., :ROPE], cos, sin, "halves"), qi[..., ROPE:]), dim=-1)
    s["qi"].view(fp8).copy_(qi.clamp(-E4M3_MAX, E4M3_MAX))
    ki = _rms(s["ki_in"].float(), s["ki_weight"])
    ki = torch.cat((_rotate(ki[:, None, :ROPE], cos, sin, "halves")[:, 0], ki[:, ROPE:]), dim=-1)
    scale = ki.abs().amax(dim=-1) / E4M3_MAX
    scale = torch.where(scale == 0, torch.ones_like(scale), scale)
    s["ki_pool"][s["slots"]] = (ki / scale[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(fp8).view(torch.uint8)
    s["ks_pool"][s["slots"]] = scale
    return _rope_outputs(s)


def _plain_attn(s):
    q, lens = s["q"].float(), s["lens"].long()[:, None]
    rows, dv = q.shape[0], s["dv"]
    width = s["table"].shape[1]
    pages = s["kept"].long() if s["kept"] is not None else torch.arange(width, device="cuda").expand(rows, width)
    pos = (pages[:, :, None] * PAGE + torch.arange(PAGE, device="cuda")).flatten(1)
    seen = (pos >= 0) & (pos < lens)
    pos = torch.where(seen, pos, 0)
    at = torch.gather(s["table"].long(), 1, pos // PAGE) * PAGE + pos % PAGE
    keys = s["kv_pool"].flatten(0, 1)[at].float()
    values = keys[..., :dv] if s["v_pool"] is None else s["v_pool"].flatten(0, 1)[at].float()
    z = (torch.bmm(q, keys.transpose(1, 2)) * s["scale"]).masked_fill(~seen[:, None], -math.inf)
    top = z.amax(dim=-1, keepdim=True)
    p = torch.exp(z - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = p.sum(dim=-1, keepdim=True)
    out = torch.bmm(p, values) / torch.where(total == 0, torch.ones_like(total), total)
    return {"out": out.to(s["q"].dtype), "lse": (top + torch.log(total))[..., 0]}


def run(state):
    op = state["case"]["op"]
    if own:
        return _own_extend(state) if op == "extend" else _own_rope(state) if op == "rope" else _own_attn(state)
    return _plain_extend(state) if op == "extend" else _plain_rope(state) if op == "rope" else _plain_attn(state)


# ------------------------------------------------------------------------------------------------ what a pass cannot do without
def work(case):
    if case["op"] == "extend":
        cached, new = _extend_lengths(case)
        fresh = sum(-(-(c + n) // PAGE) - -(-c // PAGE) for c, n in zip(cached, new))
        tails = sum(1 for c in cached if c % PAGE)                  # a started page's id, read once
        return {"bytes": 16.0 * len(cached) + 4 * tails + 8 * fresh + 12 * sum(new) + 12, "flops": 0.0}
    if case["op"] == "rope":
        t = case["rows"]
        if case["form"] == "heads":
            size, n = (2 if case["type"] == "bf16" else 4), t * (case["heads"] + case["kheads"]) * case["width"]
            return {"bytes": 2.0 * size * n + 4 * t + 8 * case["width"], "flops": 8.0 * n}
        h = case["heads"]
        moved = 2 * 2 * h * ROPE + 2 * 2 * LATENT + 3 * IDX_H * IDX_D + 3 * IDX_D + 4 + 4 + 8
        return {"bytes": float(t * moved), "flops": float(t * (3 * h * ROPE + 4 * LATENT + 3 * IDX_H * ROPE + 6 * IDX_D))}
    lens = _attn_lengths(case)
    if case["keep"]:
        # a kept page holds 64 tokens, but for the row's last one
        seen = [n if -(-n // PAGE) <= case["keep"] else case["keep"] * PAGE for n in lens]
    else:
        seen = lens
    size, dqk, dv, both = (4, case["dqk"], case["dv"], 1) if case["type"] == "f32" else (2, LATENT, VALUE, 0)
    rows, h, tokens = case["rows"], case["heads"], sum(seen)
    held = sum(-(-n // PAGE) for n in seen)
    return {"bytes": float(size * (tokens * (dqk + both * dv) + rows * h * (dqk + dv)) + 4 * rows * h + 4 * held + 4 * rows),
            "flops": 2.0 * tokens * h * (dqk + dv)}


# ------------------------------------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    if case["op"] == "extend":
        return None                                                 # whole numbers only
    s = prepare(case, seed)
    return _exact_rope(s) if case["op"] == "rope" else _exact_attn(s)


def _exact_turned(x, s, first, length, style):
    """x [T, H, D] in 64 bits, the pairs of its entries [first, first + length) multiplied by e^(i * angle) as complex numbers."""
    half = length // 2
    i = torch.arange(half, device="cuda")
    re, im = (first + 2 * i, first + 2 * i + 1) if style == "pairs" else (first + i, first + half + i)
    turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), torch.outer(s["positions"].double(), s["freq"]))[:, None]
    z = torch.complex(x[:, :, re], x[:, :, im]) * turn
    out = x.clone()
    out[:, :, re], out[:, :, im] = z.real, z.imag
    return out


def _exact_norm(x, weight, first, length):
    part = x[:, :, first:first + length]
    out = x.clone()
    out[:, :, first:first + length] = part / torch.sqrt(part.square().sum(-1, keepdim=True) / length + EPS) * weight.double()
    return out


def _exact_rope(s):
    c = s["case"]
    if c["form"] == "heads":
        d = c["width"]
        return {n: _exact_turned(_exact_norm(s[n + "_in"].double(), s[n + "_weight"], 0, d), s, 0, c["rot"], c["style"])
                for n in ("q", "k")}
    kv = _exact_norm(s["kv_in"].double()[:, None], s["kv_weight"], 0, VALUE)
    kv_pool = s["kv_pool"].double()
    kv_pool[s["slots"]] = _exact_turned(kv, s, VALUE, ROPE, "pairs")[:, 0]
    ki = _exact_turned(_exact_norm(s["ki_in"].double()[:, None], s["ki_weight"], 0, IDX_D), s, 0, ROPE, "halves")[:, 0]
    scale = ki.abs().amax(-1) / E4M3_MAX
    ki_pool, ks_pool = torch.zeros(s["ki_pool"].shape, dtype=torch.float64, device="cuda"), s["ks_pool"].double()
    ki_pool[s["slots"]] = ki / scale[:, None]
    ks_pool[s["slots"]] = scale
    return {"q": _exact_turned(s["q_in"].double(), s, 0, ROPE, "pairs"), "kv_pool": kv_pool,
            "qi": _exact_turned(s["qi_in"].double(), s, 0, ROPE, "halves"), "ki_pool": ki_pool, "ks_pool": ks_pool}


def _exact_attn(s):
    rows, heads, dv = s["q"].shape[0], s["q"].shape[1], s["dv"]
    out = torch.zeros((rows, heads, dv), dtype=torch.float64, device="cuda")
    lse = torch.full((rows, heads), -math.inf, dtype=torch.float64, device="cuda")
    lens, table = s["lens"].tolist(), s["table"].cpu().numpy()
    kept = None if s["kept"] is None else s["kept"].cpu().numpy()
    for r in range(rows):
        n = lens[r]
        tokens = np.arange(n) if kept is None else np.concatenate(
            [np.arange(p * PAGE, min(n, (p + 1) * PAGE)) for p in kept[r] if p >= 0] or [np.arange(0)])
        if not len(tokens):
            continue
        block, slot = torch.from_numpy(table[r][tokens // PAGE]).cuda().long(), torch.from_numpy(tokens % PAGE).cuda()
        k = s["kv_pool"][block, slot].double()
        v = k[:, :dv] if s["v_pool"] is None else s["v_pool"][block, slot].double()
        z = s["q"][r].double() @ k.T * s["scale"]
        lse[r] = torch.logsumexp(z, dim=1)
        out[r] = torch.softmax(z, dim=1) @ v
    return {"out": out, "lse": lse}
