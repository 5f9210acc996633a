"""Measured cases of the rotary, paged-cache and paged-attention operators.

Four operators of a decode server's step over paged caches (pages of `page` rows, addressed by a
page table per sequence, held in bf16 or in 4 bits):

  rope     rotary positions of queries, keys, outputs and gradients
  append   new rows rotated, rounded to the cache's type and written into their pages
  scores   indexer scores of every cached key: sum_h w_h max(0, q_h . k_j)
  attn     sink-softmax attention of the selected cache rows

The 4-bit type holds groups of 16 values as n * s: s an e4m3 scale, n an integer in -7..7 stored as
n + 8. A 32-bit word holds 8 values, value i at bits 4 * (i // 2) + 16 * (i % 2). A page of 512-wide
rows is row-major, 256 bytes of values then 32 scales a row; a page of 128-wide rows is four planes
[page][16 bytes], plane c with values 32 c .. 32 c + 31 of each row, then [page][8] scales.
"""

import math

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
HEADS, KEY_DIM, KV_DIM = 64, 128, 512


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _rope(name, tokens, heads, dim, rot, first, layout, dtype, inplace, inverse, far, factor, original, magnitude):
    return dict(name=name, op="rope", tokens=tokens, heads=heads, dim=dim, rot=rot, first=first, layout=layout,
                dtype=dtype, inplace=inplace, inverse=inverse, far=far, factor=factor, original=original,
                magnitude=magnitude)


def _append(name, tokens, dim, form, page, dtype, rot, layout, seqs, padded):
    return dict(name=name, op="append", tokens=tokens, dim=dim, form=form, page=page, dtype=dtype, rot=rot,
                layout=layout, seqs=seqs, padded=padded)


def _scores(name, lens, form, page):
    return dict(name=name, op="scores", lens=lens, form=form, page=page)


def _attn(name, lens, widths, missing, form, page):
    return dict(name=name, op="attn", lens=lens, widths=widths, missing=missing, form=form, page=page)


def _text(v):
    return ",".join(str(x) for x in v)


def _numbers(s):
    return [int(x) for x in s.split(",")]


def listed():
    return [
        # Eight rows' attention queries of one decode step: the last 64 of 512 features, in place, far positions.
        _rope("rope_query_decode", 8, 64, 512, 64, 448, "interleaved", "bf16", True, False, 1 << 20, 16.0, 65536, 1.0),
        # The indexer's queries of a prompt chunk, out of place: half of each 128-wide head passes unrotated.
        _rope("rope_index_prefill", 4096, 64, 128, 64, 64, "half", "bf16", False, False, 131072, 4.0, 4096, 1.25),
        # The transposed rotation (the backward pass, and the attention's output before its projection), 32 bits.
        _rope("rope_inverse_fp32", 1021, 64, 512, 64, 448, "interleaved", "fp32", True, True, 32768, 1.0, 0, 1.0),
        # One new KV row of each of eight sequences into 4-bit pages.
        _append("append_kv_decode_int4", 8, 512, "int4", 64, "bf16", 64, "interleaved", 8, 0),
        # A long prompt's indexer keys into 4-bit pages, with a padded tail.
        _append("append_keys_prefill_int4", 32768, 128, "int4", 128, "bf16", 64, "half", 8, 100),
        # A prompt chunk's KV rows from the 32-bit projection into bf16 pages, an odd number of them.
        _append("append_kv_prefill_bf16", 8191, 512, "bf16", 64, "fp32", 64, "interleaved", 3, 0),
        # Eight short, ragged caches: the call's latency.
        _scores("scores_int4_short", "1,17,64,129,300,511,700,999", "int4", 64),
        # Eight full caches: a pure stream over a million 4-bit keys.
        _scores("scores_int4_long", _text([131072] * 8), "int4", 64),
        # Ragged caches in bf16 pages.
        _scores("scores_bf16_ragged", "4097,9000,16384,21111,30001,42000,55555,65536", "bf16", 64),
        # One new sequence: every cached row selected.
        _attn("attn_int4_one", "37", "37", 0, "int4", 16),
        # The decode step's attention over eight long 4-bit caches.
        _attn("attn_int4_long", _text([131072] * 8), _text([512] * 8), 0, "int4", 64),
        # Ragged rows in bf16 pages, some slots without a row.
        _attn("attn_bf16_ragged", "1,100,700,4097,9000,30001,65536,131072", "1,100,512,512,512,512,512,512", 5, "bf16",
              128),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    case = _drawn(rng)
    del case["name"]
    return case


def _drawn(rng):
    op = rng.choice(("rope", "append", "scores", "attn"))
    form = rng.choice(("bf16", "int4"))
    page = rng.choice((16, 32, 64, 128, 256))
    rows = rng.randint(1, 8)
    layout = rng.choice(("interleaved", "half"))
    if op == "rope":
        dim = rng.choice((64, 96, 128, 192, 256, 512))
        rot = rng.choice((dim, dim // 2, 64, 2 * rng.randint(1, dim // 2)))
        first = rng.choice((0, dim - rot, 2 * rng.randint(0, (dim - rot) // 2)))
        heads = rng.choice((1, 2, 7, 16, 64))
        dtype = rng.choice(tuple(TYPES))
        tokens = _log(rng, 1, min(16384, (4096 * 64 * 256) // (heads * dim * TYPES[dtype].itemsize)))
        inplace = rng.random() < 0.5
        factor = rng.choice((1.0, 4.0, 16.0, 40.0))
        return _rope("rope", tokens, heads, dim, rot, first, layout, dtype, inplace, rng.random() < 0.5,
                     _log(rng, 1000, 1 << 20), factor, rng.choice((0, 4096, 65536)),
                     1.0 if inplace else round(rng.uniform(0.5, 1.5), 3))
    if op == "append":
        dim = rng.choice((KEY_DIM, KV_DIM))
        tokens = _log(rng, 1, 32768 * KEY_DIM // dim)
        return _append("append", tokens, dim, form, page, rng.choice(tuple(TYPES)),
                       rng.choice((0, 64, dim // 4, 2 * rng.randint(1, dim // 2))), layout, rows,
                       rng.choice((0, tokens // 7)))
    if op == "scores":
        return _scores("scores", _text([_log(rng, 1, 131072 if form == "int4" else 60000) for _ in range(rows)]), form,
                       page)
    lens = [_log(rng, 1, 131072) for _ in range(rows)]
    widths = [min(n, 512) if rng.random() < 0.7 else rng.randint(1, min(n, 512)) for n in lens]
    return _attn("attn", _text(lens), _text(widths), rng.choice((0, 0, 1, 9)), form, page)


def work(case):
    if case["op"] == "rope":
        size = TYPES[case["dtype"]].itemsize
        vectors = case["tokens"] * case["heads"]
        width = case["rot"] if case["inplace"] else case["dim"]
        return {"bytes": 2 * vectors * width * size + 4 * case["tokens"], "flops": 3 * vectors * case["rot"]}
    if case["op"] == "append":
        n = case["tokens"] - case["padded"]
        row = _row_bytes(case["dim"], case["form"])
        values = 2 * case["dim"] if case["form"] == "int4" else 0
        return {"bytes": n * (case["dim"] * TYPES[case["dtype"]].itemsize + row + values) + 12 * case["tokens"],
                "flops": n * (3 * case["rot"] + 4 * case["dim"])}
    lens = _numbers(case["lens"])
    if case["op"] == "scores":
        keys = sum(lens)
        return {"bytes": keys * (_row_bytes(KEY_DIM, case["form"]) + 4) + len(lens) * HEADS * (2 * KEY_DIM + 4),
                "flops": keys * HEADS * (2 * KEY_DIM + 3)}
    slots = sum(max(0, w - case["missing"]) for w in _numbers(case["widths"]))
    return {"bytes": slots * (_row_bytes(KV_DIM, case["form"]) + 4) + len(lens) * HEADS * KV_DIM * 4,
            "flops": slots * HEADS * KV_DIM * 4}


# ---------------------------------------------------------------------------
# the cache's types
# ---------------------------------------------------------------------------

def _row_bytes(dim, form):
    return 2 * dim if form == "bf16" else dim // 2 + dim // 16


def _quantise(y):
    """Groups of 16 along the last axis: (n, s), n integers -7..7 and s the e4m3 scales, as `y`'s type."""
    g = y.reshape(*y.shape[:-1], -1, 16)
    bad = ~torch.isfinite(g).all(-1)
    g = torch.where(bad[..., None], 0.0, g)
    s = (g.abs().amax(-1).double() / 7).float().clamp(max=448.0)  # in 64 bits: next to a border
    s = s.to(torch.float8_e4m3fn).to(y.dtype)
    n = torch.where(s[..., None] > 0, g / torch.where(s > 0, s, 1.0)[..., None], 0.0).round().clamp(-7, 7)
    return n, torch.where(bad, float("nan"), s)


def _pack(n, s):
    """Rows [rows, dim] of (n, s) as bytes: values [rows, dim / 2] in the word order, scales [rows, dim / 16]."""
    rows = n.shape[0]
    c = (n.reshape(rows, -1, 4, 2) + 8).to(torch.int32)  # [rows, word, pair, side]
    shift = 4 * torch.arange(4, device=n.device, dtype=torch.int32)
    halves = (c << shift[:, None]).sum(2).to(torch.int32)  # [rows, word, side]: 16 bits each
    values = torch.stack((halves & 255, halves >> 8), -1).to(torch.uint8).reshape(rows, -1)
    return values, s.float().to(torch.float8_e4m3fn).view(torch.uint8)


def _blocks(pages, dim, page):
    """Views of a 4-bit pool: values and scales, one row's bytes at [page id, row] (keys: [page id, plane, row])."""
    if dim == KV_DIM:
        rows = pages.view(-1, page, 288)
        return rows[..., :256], rows[..., 256:]
    flat = pages.view(-1, page * 72)
    return flat[:, : page * 64].unflatten(1, (4, page, 16)), flat[:, page * 64:].unflatten(1, (page, 8))


def _store(pages, dim, form, page, ids, at, y):
    """Rows y [rows, dim] into page ids[i], row at[i]; returns the values that the cache then holds."""
    if form == "bf16":
        pages.view(-1, page, dim)[ids, at] = y.to(torch.bfloat16)
        return None
    n, s = _quantise(y)
    values, scales = _pack(n, s)
    v, sc = _blocks(pages, dim, page)
    if dim == KV_DIM:
        v[ids, at] = values
    else:
        v[ids, :, at] = values.view(-1, 4, 16)
    sc[ids, at] = scales
    return (n * s[..., None]).flatten(-2).to(torch.bfloat16)


def _fetch(pages, dim, form, page, ids, at):
    """Rows at[i] of pages ids[i] in 32 bits: [..., dim]."""
    if form == "bf16":
        return pages.view(-1, page, dim)[ids, at].float()
    v, sc = _blocks(pages, dim, page)
    values = v[ids, at] if dim == KV_DIM else v[ids, :, at].flatten(-2)
    halves = values.unflatten(-1, (-1, 2, 2)).to(torch.int32)  # [..., word, side, byte]
    halves = halves[..., 0] | halves[..., 1] << 8
    shift = 4 * torch.arange(4, device=pages.device, dtype=torch.int32)
    n = (halves[..., None, :] >> shift[:, None] & 15) - 8  # [..., word, pair, side]
    s = sc[ids, at].contiguous().view(torch.float8_e4m3fn).float()
    return (n.flatten(-3).unflatten(-1, (-1, 16)) * s[..., None]).flatten(-2)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _frequencies(rot, base, factor, original):
    """theta_i in 64 bits: plain, divided by `factor`, or (with `original`) blended by YaRN's ramp."""
    i = torch.arange(rot // 2, dtype=torch.float64)
    theta = base ** (-2 * i / rot)
    if factor == 1.0:
        return theta
    if not original:
        return theta / factor
    low, high = (rot * math.log(original / (2 * math.pi * r)) / (2 * math.log(base)) for r in (32.0, 1.0))
    low, high = max(math.floor(low), 0), min(math.ceil(high), rot - 1)
    ramp = ((i - low) / max(high - low, 0.001)).clamp(0, 1)
    return theta * (1 - ramp) + theta / factor * ramp


def _tables(lens, page, g):
    """A page table over a pool in which the sequences' pages lie in no order, with some pages unused."""
    need = [max(1, -(-n // page)) for n in lens]
    total = sum(need) + 3
    order = torch.randperm(total, generator=g, device=DEV).to(torch.int32)
    table = torch.full((len(lens), max(need)), -1, dtype=torch.int32, device=DEV)
    at = 0
    for e, n in enumerate(need):
        table[e, :n] = order[at:at + n]
        at += n
    return table, total


def _filled(lens, dim, form, page, g):
    table, total = _tables(lens, page, g)
    pages = torch.empty(total, page * _row_bytes(dim, form), dtype=torch.uint8, device=DEV)
    pages = pages.view(torch.bfloat16) if form == "bf16" else pages
    rows = torch.arange(total * page, device=DEV)
    for part in rows.split(1 << 18):
        y = torch.randn(len(part), dim, generator=g, device=DEV)
        _store(pages, dim, form, page, part // page, part % page, y)
    return pages, table


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    randn = lambda *shape: torch.randn(*shape, generator=g, device=DEV)  # noqa: E731
    bf16 = torch.bfloat16
    s = dict(case)
    if own:
        import deepseek_sparse_attention_ragged_gb300 as ds
        s["ds"] = ds
    if case["op"] == "rope":
        s["x"] = randn(case["tokens"], case["heads"], case["dim"]).to(TYPES[case["dtype"]])
        s["out"] = s["x"] if case["inplace"] else torch.empty_like(s["x"])
        s["positions"] = torch.randint(0, case["far"], (case["tokens"],), generator=g, device=DEV, dtype=torch.int32)
        s["theta"] = _frequencies(case["rot"], 10000.0, case["factor"], case["original"]).to(DEV)
        if own:
            s["rope"] = ds.Rope(case["rot"], first=case["first"], layout=case["layout"], base=10000.0,
                                factor=case["factor"], original_len=case["original"], magnitude=case["magnitude"])
    elif case["op"] == "append":
        n, seqs, page = case["tokens"], case["seqs"], case["page"]
        live = n - case["padded"]
        # The sequences append consecutive runs behind what their caches hold; padding lies at the end.
        start = torch.randint(0, 1000, (seqs,), generator=g, device=DEV)
        seq = torch.arange(n, device=DEV) * seqs // max(live, 1)
        run = torch.arange(n, device=DEV) - torch.searchsorted(seq, seq)
        slot = start[seq.clamp(max=seqs - 1)] + run
        seq[live:] = -1
        s["seq"], s["slot"] = seq.to(torch.int32), slot.to(torch.int32)
        s["positions"] = (4 * slot).to(torch.int32)  # a compressed row stands for four tokens
        table, total = _tables([1000 + -(-live // seqs) + 1] * seqs, page, g)
        pages = torch.zeros(total, page * _row_bytes(case["dim"], case["form"]), dtype=torch.uint8, device=DEV)
        s["pages"], s["table"] = pages.view(bf16) if case["form"] == "bf16" else pages, table
        s["x"] = randn(n, case["dim"]).to(TYPES[case["dtype"]])
        s["first"] = case["dim"] - case["rot"]
        s["theta"] = _frequencies(case["rot"], 10000.0, 4.0, 4096).to(DEV) if case["rot"] else None
        s["values"] = torch.zeros(n, case["dim"], dtype=bf16, device=DEV) if case["form"] == "int4" else None
        if own:
            s["cache"] = ds.PagedCache(s["pages"], table, page, case["dim"], case["form"])
            s["rope"] = ds.Rope(case["rot"], first=s["first"], layout=case["layout"], base=10000.0, factor=4.0,
                                original_len=4096) if case["rot"] else None
    else:
        lens = _numbers(case["lens"])
        rows, dim = len(lens), KEY_DIM if case["op"] == "scores" else KV_DIM
        s["pages"], s["table"] = _filled(lens, dim, case["form"], case["page"], g)
        s["kv_len"] = torch.tensor(lens, device=DEV)
        s["q"] = randn(rows, HEADS, dim).to(bf16)
        if own:
            s["cache"] = ds.PagedCache(s["pages"], s["table"], case["page"], dim, case["form"])
        if case["op"] == "scores":
            s["w"] = randn(rows, HEADS) / 8
            s["scores"] = torch.zeros(rows, max(lens), device=DEV)
            s["rows"] = [(n, min(n, 512), 512 * e, e) for e, n in enumerate(lens)]
        else:
            widths = _numbers(case["widths"])
            s["indices"] = torch.full((rows, max(widths)), -1, dtype=torch.int32, device=DEV)
            for e, (n, w) in enumerate(zip(lens, widths)):
                picked = torch.randperm(n, generator=g, device=DEV)[: max(0, w - case["missing"])]
                s["indices"][e, : len(picked)] = picked.to(torch.int32)
            s["sinks"] = randn(HEADS)
            s["scale"] = KV_DIM ** -0.5
            s["out"] = torch.empty(rows, HEADS, KV_DIM, dtype=bf16, device=DEV)
            s["rows"] = [(n, w, max(widths) * e, e) for e, (n, w) in enumerate(zip(lens, widths))]
            if own:
                s["workspace"] = ds.workspace(s["rows"])
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def _rotate(x, positions, theta, rot, first, layout, magnitude, inverse):
    """x [tokens, ..., dim] in 32 bits with features [first, first + rot) rotated; the angles are taken in 64 bits."""
    angle = positions.double()[:, None] * theta
    angle = angle.reshape(len(positions), *[1] * (x.dim() - 2), rot // 2)
    c, s = (angle.cos() * magnitude).float(), (angle.sin() * (-magnitude if inverse else magnitude)).float()
    part = x[..., first:first + rot].float()
    if layout == "interleaved":
        a, b = part[..., 0::2], part[..., 1::2]
        turned = torch.stack((a * c - b * s, a * s + b * c), -1).flatten(-2)
    else:
        a, b = part[..., : rot // 2], part[..., rot // 2:]
        turned = torch.cat((a * c - b * s, a * s + b * c), -1)
    return turned


def run(s):
    if s["op"] == "rope":
        if own:
            s["ds"].ds_rows_rope(s["rope"], s["x"], s["positions"], s["out"], inverse=s["inverse"])
            return s["out"]
        lo, hi = s["first"], s["first"] + s["rot"]
        turned = _rotate(s["x"], s["positions"], s["theta"], s["rot"], lo, s["layout"], s["magnitude"], s["inverse"])
        if not s["inplace"]:
            s["out"].copy_(s["x"])
        s["out"][..., lo:hi] = turned.to(s["out"].dtype)
        return s["out"]
    if s["op"] == "append":
        if own:
            s["ds"].ds_rows_append(s["cache"], s["x"], s["seq"], s["slot"], rope=s["rope"], positions=s["positions"],
                                   values=s["values"])
            return s["pages"] if s["values"] is None else s["values"]
        live = len(s["seq"]) - s["padded"]
        seq, slot, x = s["seq"][:live].long(), s["slot"][:live].long(), s["x"][:live].float()
        if s["rot"]:
            turned = _rotate(x, s["positions"][:live], s["theta"], s["rot"], s["first"], s["layout"], 1.0, False)
            x = torch.cat((x[..., : s["first"]], turned, x[..., s["first"] + s["rot"]:]), -1)
        ids, at = s["table"][seq, slot // s["page"]].long(), slot % s["page"]
        held = _store(s["pages"], s["dim"], s["form"], s["page"], ids, at, x)
        if held is None:
            return s["pages"]
        s["values"][:live] = held
        return s["values"]
    if s["op"] == "scores":
        if own:
            s["ds"].ds_rows_indexer_score_paged(s["rows"], s["q"], s["w"], s["cache"], s["scores"])
            return s["scores"]
        j = torch.arange(s["scores"].shape[1], device=DEV)
        there = j < s["kv_len"][:, None]
        ids = s["table"][:, j // s["page"]].long().clamp(min=0)
        k = _fetch(s["pages"], KEY_DIM, s["form"], s["page"], ids, (j % s["page"]).expand_as(ids))
        dots = torch.matmul(k, s["q"].float().transpose(1, 2)).clamp_(min=0)  # [rows, keys, heads]
        s["scores"].copy_(torch.where(there, torch.matmul(dots, s["w"][:, :, None])[..., 0], s["scores"]))
        return s["scores"]
    if own:
        s["ds"].ds_rows_sparse_attn_paged(s["rows"], s["q"], s["sinks"], 0, s["indices"], s["scale"], s["out"],
                                          s["cache"], workspace_t=s["workspace"])
        return s["out"]
    there = s["indices"] >= 0
    i = s["indices"].long().clamp(min=0)
    ids = s["table"].gather(1, i // s["page"]).long().clamp(min=0)
    kv = _fetch(s["pages"], KV_DIM, s["form"], s["page"], ids, i % s["page"])
    kv = torch.where(there[..., None], kv, 0.0)
    logits = torch.matmul(s["q"].float(), kv.transpose(1, 2)) * s["scale"]
    logits = torch.where(there[:, None], logits, float("-inf"))
    top = torch.maximum(logits.amax(-1), s["sinks"])[..., None]
    p = (logits - top).exp()
    den = p.sum(-1, keepdim=True) + (s["sinks"][:, None] - top).exp()
    s["out"].copy_(torch.matmul(p, kv) / den)
    return s["out"]


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------

def _turned64(x, positions, case, first, factor, original, magnitude, inverse):
    """Rows rotated pair by pair as complex numbers, from numpy's 64-bit angles."""
    rot = case["rot"]
    i = np.arange(rot // 2, dtype=np.float64)
    theta = np.power(10000.0, -2.0 * i / rot)
    if factor != 1.0 and not original:
        theta = theta / factor
    elif factor != 1.0:
        bound = [rot * np.log(original / (2 * np.pi * r)) / (2 * np.log(10000.0)) for r in (32.0, 1.0)]
        low, high = max(np.floor(bound[0]), 0.0), min(np.ceil(bound[1]), rot - 1.0)
        mix = np.clip((i - low) / max(high - low, 0.001), 0.0, 1.0)
        theta = theta * ((1.0 - mix) + mix / factor)
    angle = positions.cpu().numpy().astype(np.float64)[:, None] * theta
    turn = magnitude * np.exp((-1j if inverse else 1j) * angle)
    turn = torch.from_numpy(turn).to(DEV).view(len(positions), *[1] * (x.dim() - 2), rot // 2)
    y = x.double().clone()
    if case["layout"] == "interleaved":
        real, imag = slice(first, first + rot, 2), slice(first + 1, first + rot, 2)
    else:
        real, imag = slice(first, first + rot // 2), slice(first + rot // 2, first + rot)
    z = torch.complex(y[..., real], y[..., imag]) * turn
    y[..., real], y[..., imag] = z.real, z.imag
    return y


def _rows64(s, dim, e, j):
    """Rows j of sequence e, decoded value by value from the bytes."""
    page = s["page"]
    ids, at = s["table"][e, j // page].long(), j % page
    if s["form"] == "bf16":
        return s["pages"].reshape(-1, dim)[ids * page + at].double()
    f = torch.arange(dim, device=DEV)
    word, i = f // 8, f % 8
    bit = 4 * (i // 2) + 16 * (i % 2)
    byte = 4 * word + bit // 8
    raw = s["pages"].reshape(-1)
    start = ids[:, None] * page * (dim // 2 + dim // 16)
    if dim == KV_DIM:
        value_at = start + at[:, None] * 288 + byte
        scale_at = start + at[:, None] * 288 + 256 + f // 16
    else:
        value_at = start + byte // 16 * (page * 16) + at[:, None] * 16 + byte % 16
        scale_at = start + page * 64 + at[:, None] * 8 + f // 16
    n = (raw[value_at].long() >> bit % 8) % 16 - 8
    c = raw[scale_at].long()
    exponent, mantissa = c // 8 % 16, c % 8
    s64 = torch.where(exponent == 0, mantissa / 8 * 2.0 ** -6,
                      (1 + mantissa / 8) * torch.exp2((exponent - 7).double()))
    return n.double() * s64.double()


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _turned64(s["x"], s["positions"], case, case["first"], case["factor"], case["original"],
                         case["magnitude"], case["inverse"])
    if case["op"] == "append":
        live = case["tokens"] - case["padded"]
        y = s["x"][:live].double()
        if case["rot"]:
            y = _turned64(s["x"][:live], s["positions"][:live], case, s["first"], 4.0, 4096, 1.0, False)
        if case["form"] == "bf16":
            pages = s["pages"].double().reshape(-1, case["dim"])
            slot = s["slot"][:live].long()
            ids = s["table"][s["seq"][:live].long(), slot // case["page"]].long()
            pages[ids * case["page"] + slot % case["page"]] = y
            return pages.reshape(s["pages"].shape)
        group = y.reshape(live, -1, 16)
        scale = torch.clamp(group.abs().amax(-1) / torch.full((), 7.0, dtype=torch.float64, device=DEV), max=448.0)
        # e4m3: steps of 2^(exponent - 3), no exponent under -6; half goes to even.
        step = torch.exp2(torch.clamp(torch.floor(torch.log2(torch.clamp(scale, min=1e-30))), min=-6) - 3)
        scale = (torch.round(scale / step) * step)[..., None]
        n = torch.clamp(torch.round(group / torch.clamp(scale, min=1e-30)), -7, 7) * (scale > 0)
        out = torch.zeros(case["tokens"], case["dim"], dtype=torch.float64, device=DEV)
        out[:live] = (n * scale).reshape(live, -1)
        return out
    lens = _numbers(case["lens"])
    if case["op"] == "scores":
        out = s["scores"].double()
        for e, n in enumerate(lens):
            for j in torch.arange(n, device=DEV).split(16384):
                k = _rows64(s, KEY_DIM, e, j)
                out[e, j] = (torch.relu(k @ s["q"][e].double().T) * s["w"][e].double()).sum(1)
        return out
    out = torch.zeros(len(lens), HEADS, KV_DIM, dtype=torch.float64, device=DEV)
    for e in range(len(lens)):
        j = s["indices"][e][s["indices"][e] >= 0].long()
        kv = _rows64(s, KV_DIM, e, j)
        logits = torch.cat((s["q"][e].double() @ kv.T * s["scale"], s["sinks"].double()[:, None]), 1)
        out[e] = torch.softmax(logits, 1)[:, : len(j)] @ kv
    return out
