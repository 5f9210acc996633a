"""Measured cases of the 8-bit paged caches and of the attention over a shared prefix.

Operators beside the rotary and paged ones, for a server whose batch decodes from one long prompt:

  append   new rows rotated, rounded to 8-bit pages and written
  fetch    rows read back from their pages (bf16, 8 or 4 bits) into a contiguous buffer
  scores   indexer scores of every key of 8-bit pages: sum_h w_h max(0, q_h . k_j)
  prefix   sink-softmax attention over every cached row, for rows that share a long prefix

The 8-bit type holds blocks of 128 values as v * 2^e: v an e4m3 number of magnitude at most 448, e the
least exponent from -100 to 7 for which 448 * 2^e reaches the block, held as the byte e + 127. A page of
512-wide rows is [page][512 bytes] of values, then [page][4] exponents; a page of 128-wide rows is eight
planes [page][16 bytes], plane c with values 16 c .. 16 c + 15 of each row, then [page] exponents.

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

def _append(name, tokens, dim, page, dtype, rot, layout, seqs, padded):
    return dict(name=name, op="append", tokens=tokens, dim=dim, form="fp8", page=page, dtype=dtype, rot=rot,
                layout=layout, seqs=seqs, padded=padded)


def _fetch_case(name, tokens, dim, form, page, dtype, lens, whole, padded):
    return dict(name=name, op="fetch", tokens=tokens, dim=dim, form=form, page=page, dtype=dtype, lens=lens,
                whole=whole, padded=padded)


def _scores(name, lens, page):
    return dict(name=name, op="scores", lens=lens, dim=KEY_DIM, form="fp8", page=page)


def _prefix(name, prefix, tails, form, page):
    return dict(name=name, op="prefix", prefix=prefix, tails=tails, dim=KV_DIM, form=form, page=page)


def _text(v):
    return ",".join(str(x) for x in v)


def _numbers(s):
    return [int(x) for x in s.split(",")]


def listed():
    return [
        # One new KV row of each of eight sequences into 8-bit pages: a decode step.
        _append("append_kv_decode_fp8", 8, 512, 64, "bf16", 64, "interleaved", 8, 0),
        # A long prompt's indexer keys into 8-bit pages, with a padded tail.
        _append("append_keys_prefill_fp8", 32768, 128, 128, "bf16", 64, "half", 8, 100),
        # A few scattered rows of 4-bit pages, to look at or to move one short sequence: the call's latency.
        _fetch_case("fetch_kv_few_int4", 37, 512, "int4", 16, "bf16", "300,41", False, 3),
        # Whole 8-bit key caches back into contiguous bf16, for the calls that take contiguous keys.
        _fetch_case("fetch_keys_whole_fp8", 262144, 128, "fp8", 64, "bf16", _text([65536] * 4), True, 0),
        # KV rows of ragged sequences in 32 bits, in no order.
        _fetch_case("fetch_kv_rows_fp32", 20001, 512, "fp8", 128, "fp32", "30001,9000,511,1", False, 500),
        # Eight short, ragged caches: the call's latency.
        _scores("scores_fp8_short", "1,17,64,129,300,511,700,999", 64),
        # Eight full caches: a stream over a million 8-bit keys.
        _scores("scores_fp8_long", _text([131072] * 8), 64),
        # Three samples shortly after a short prompt.
        _prefix("prefix_few_short", 300, "1,17,40", "bf16", 16),
        # One sequence alone attends to its whole cache: the cache is split over the GPU.
        _prefix("prefix_one_long", 131072, "1", "bf16", 64),
        # Eight samples of a long prompt, each some hundred rows on.
        _prefix("prefix_eight_bf16", 65536, "1,64,100,129,300,511,700,999", "bf16", 64),
        # Five samples over 4-bit pages; the prompt ends inside a page.
        _prefix("prefix_five_int4", 40007, "1,2,33,250,1000", "int4", 64),
        # Many samples of one prompt, an odd number, over 8-bit pages.
        _prefix("prefix_many_fp8", 20001, _text([1 + 5 * i for i in range(63)]), "fp8", 128),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    case = _drawn(rng)
    del case["name"]
    return case


def _drawn(rng):
    op = rng.choice(("append", "fetch", "scores", "prefix", "prefix"))
    form = rng.choice(("bf16", "fp8", "int4"))
    page = rng.choice((16, 32, 64, 128, 256))
    if op == "append":
        dim = rng.choice((KEY_DIM, KV_DIM))
        tokens = _log(rng, 1, 32768 * KEY_DIM // dim)
        return _append(op, tokens, dim, page, rng.choice(tuple(TYPES)),
                       rng.choice((0, 64, dim // 4, 2 * rng.randint(1, dim // 2))), rng.choice(("interleaved", "half")),
                       rng.randint(1, 8), rng.choice((0, tokens // 7)))
    if op == "fetch":
        dim = rng.choice((KEY_DIM, KV_DIM))
        lens = [_log(rng, 1, 40000 * KEY_DIM // dim) for _ in range(rng.randint(1, 6))]
        whole = rng.random() < 0.5
        tokens = sum(lens) if whole else _log(rng, 1, 200000 * KEY_DIM // dim)
        return _fetch_case(op, tokens, dim, form, page, rng.choice(tuple(TYPES)), _text(lens), whole,
                           0 if whole else rng.choice((0, tokens // 9)))
    if op == "scores":
        return _scores(op, _text([_log(rng, 1, 131072) for _ in range(rng.randint(1, 8))]), page)
    rows = _log(rng, 1, 64)
    prefix = rng.choice((0, _log(rng, 1, min(131072, 1000000 // rows)), _log(rng, 1, min(131072, 1000000 // rows))))
    tails = [_log(rng, 1, 1000) - (1 if prefix and rng.random() < 0.3 else 0) for _ in range(rows)]
    return _prefix(op, prefix, _text(tails), form, page)


def _row_bytes(dim, form):
    return {"bf16": 2 * dim, "fp8": dim + dim // 128, "int4": dim // 2 + dim // 16}[form]


def work(case):
    row = _row_bytes(case["dim"], case["form"])
    if case["op"] in ("append", "fetch"):
        n = case["tokens"] - case["padded"]
        wide = case["dim"] * TYPES[case["dtype"]].itemsize
        if case["op"] == "fetch":
            return {"bytes": n * (row + wide) + 8 * case["tokens"], "flops": n * case["dim"]}
        return {"bytes": n * (wide + row + 2 * case["dim"]) + 12 * case["tokens"],
                "flops": n * (3 * case["rot"] + 3 * case["dim"])}
    if case["op"] == "scores":
        lens = _numbers(case["lens"])
        return {"bytes": sum(lens) * (row + 4) + len(lens) * HEADS * (2 * KEY_DIM + 4),
                "flops": sum(lens) * HEADS * (2 * KEY_DIM + 3)}
    tails = _numbers(case["tails"])
    attended = len(tails) * case["prefix"] + sum(tails)
    return {"bytes": (case["prefix"] + sum(tails)) * row + len(tails) * HEADS * KV_DIM * 4,
            "flops": attended * HEADS * KV_DIM * 4}


# ---------------------------------------------------------------------------
# the caches' types
# ---------------------------------------------------------------------------

def _quantise4(y):
    """Groups of 16 along the last axis: (n, s), n integers -7..7 and s the e4m3 scales, as `y`'s type."""
    g = y.reshape(*y.shape[:-1], -1, 16)
    s = (g.abs().amax(-1).double() / 7).float().clamp(max=448.0).to(torch.float8_e4m3fn).to(y.dtype)
    n = torch.where(s[..., None] > 0, g / torch.where(s > 0, s, 1.0)[..., None], 0.0).round().clamp(-7, 7)
    return n, s


def _quantise8(y):
    """Blocks of 128 along the last axis: (v, e), v the e4m3 numbers and e whole exponents."""
    g = y.reshape(*y.shape[:-1], -1, 128)
    m, x = torch.frexp(g.abs().amax(-1))  # m in [0.5, 1), and 448 = 0.875 * 2^9
    e = torch.where(m > 0.875, x - 8, x - 9).clamp(-100, 7)
    v = torch.ldexp(g, -e[..., None]).clamp(-448, 448).float().to(torch.float8_e4m3fn)
    return v, e


def _blocks(pages, dim, form, page):
    """Views of a pool of 8 or 4 bits: values and scales, one row's bytes at [page id, row] (keys: [page id, plane, row])."""
    if dim == KV_DIM and form == "int4":
        rows = pages.view(-1, page, 288)
        return rows[..., :256], rows[..., 256:]
    wide, few = (dim, dim // 128) if form == "fp8" else (dim // 2, dim // 16)
    flat = pages.view(-1, page * (wide + few))
    values, scales = flat[:, : page * wide], flat[:, page * wide:].unflatten(1, (page, few))
    return values.unflatten(1, (page, wide) if dim == KV_DIM else (wide // 16, page, 16)), scales


def _store(pages, dim, form, page, ids, at, y):
    """Rows y [rows, dim] into page ids[i], row at[i]; returns the values that the cache then holds."""
    if form == "bf16":
        pages.view(-1, page, dim)[ids, at] = y.to(torch.bfloat16)
        return None
    rows = y.shape[0]
    if form == "fp8":
        v, e = _quantise8(y)
        held = torch.ldexp(v.float(), e[..., None])
        values, scales = v.view(torch.uint8).reshape(rows, -1), (e + 127).to(torch.uint8)
    else:
        n, s = _quantise4(y)
        held = n * s[..., None]
        c = (n.reshape(rows, -1, 4, 2) + 8).to(torch.int32)  # [rows, word, pair, side]
        shift = 4 * torch.arange(4, device=n.device, dtype=torch.int32)
        halves = (c << shift[:, None]).sum(2).to(torch.int32)  # [rows, word, side]: 16 bits each
        values = torch.stack((halves & 255, halves >> 8), -1).to(torch.uint8).reshape(rows, -1)
        scales = s.float().to(torch.float8_e4m3fn).view(torch.uint8)
    to, sc = _blocks(pages, dim, form, page)
    if dim == KV_DIM:
        to[ids, at] = values
    else:
        to[ids, :, at] = values.unflatten(1, (-1, 16))
    sc[ids, at] = scales
    return held.flatten(-2).to(torch.bfloat16)


def _fetch(pages, dim, form, page, ids, at):
    """Rows at[i] of pages ids[i] in 32 bits: [..., dim]."""
    if form == "bf16":
        return pages.view(-1, page, dim)[ids, at].float()
    v, sc = _blocks(pages, dim, form, page)
    values = v[ids, at] if dim == KV_DIM else v[ids, :, at].flatten(-2)
    scales = sc[ids, at].contiguous()
    if form == "fp8":
        e = scales.to(torch.int32) - 127
        return torch.ldexp(values.contiguous().view(torch.float8_e4m3fn).float().unflatten(-1, (-1, 128)),
                           e[..., None]).flatten(-2)
    halves = values.unflatten(-1, (-1, 2, 2)).to(torch.int32)  # [..., word, side, byte]
    halves = halves[..., 0] | halves[..., 1] << 8
    shift = 4 * torch.arange(4, device=pages.device, dtype=torch.int32)
    n = (halves[..., None, :] >> shift[:, None] & 15) - 8  # [..., word, pair, side]
    s = scales.view(torch.float8_e4m3fn).float()
    return (n.flatten(-3).unflatten(-1, (-1, 16)) * s[..., None]).flatten(-2)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _frequencies(rot):
    """theta_i in 64 bits: base 10000, stretched four times from 4096 positions by YaRN's ramp."""
    i = torch.arange(rot // 2, dtype=torch.float64)
    theta = 10000.0 ** (-2 * i / rot)
    low, high = (rot * math.log(4096 / (2 * math.pi * r)) / (2 * math.log(10000.0)) for r in (32.0, 1.0))
    low, high = max(math.floor(low), 0), min(math.ceil(high), rot - 1)
    ramp = ((i - low) / max(high - low, 0.001)).clamp(0, 1)
    return theta * (1 - ramp) + theta / 4.0 * ramp


def _tables(need, shared, g):
    """A page table over a pool in which the sequences' pages lie in no order, with some pages unused;
    the first `shared` pages of every sequence are those of the first."""
    total = shared + sum(max(1, n) - shared for n in need) + 3
    order = torch.randperm(total, generator=g, device=DEV).to(torch.int32)
    table = torch.full((len(need), max(1, max(need))), -1, dtype=torch.int32, device=DEV)
    table[:, :shared] = order[:shared]
    at = shared
    for e, n in enumerate(need):
        n = max(1, n) - shared
        table[e, shared:shared + n] = order[at:at + n]
        at += n
    return table, total


def _filled(case, total, g):
    dim, form, page = case["dim"], case["form"], case["page"]
    pages = torch.empty(total, page * _row_bytes(dim, form), dtype=torch.uint8, device=DEV)
    pages = pages.view(torch.bfloat16) if form == "bf16" else pages
    rows = torch.arange(total * page, device=DEV)
    for part in rows.split(1 << 18):
        _store(pages, dim, form, page, part // page, part % page, torch.randn(len(part), dim, generator=g, device=DEV))
    return pages


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    randn = lambda *shape: torch.randn(*shape, generator=g, device=DEV)  # noqa: E731
    bf16, i32 = torch.bfloat16, torch.int32
    s = dict(case)
    dim, form, page = case["dim"], case["form"], case["page"]
    if case["op"] == "append":
        n, seqs = case["tokens"], case["seqs"]
        live = n - case["padded"]
        # The sequences append consecutive runs behind what their caches hold; padding lies at the end.
        start = torch.randint(0, 1000, (seqs,), generator=g, device=DEV)
        seq = torch.arange(n, device=DEV) * seqs // max(live, 1)
        run_at = torch.arange(n, device=DEV) - torch.searchsorted(seq, seq)
        slot = start[seq.clamp(max=seqs - 1)] + run_at
        seq[live:] = -1
        s["seq"], s["slot"] = seq.to(i32), slot.to(i32)
        s["positions"] = (4 * slot).to(i32)  # a compressed row stands for four tokens
        s["table"], total = _tables([-(-(1001 + -(-live // seqs)) // page)] * seqs, 0, g)
        s["pages"] = torch.zeros(total, page * _row_bytes(dim, form), dtype=torch.uint8, device=DEV)
        s["x"] = randn(n, dim).to(TYPES[case["dtype"]])
        s["first"] = dim - case["rot"]
        s["theta"] = _frequencies(case["rot"]).to(DEV)
        s["values"] = torch.zeros(n, dim, dtype=bf16, device=DEV)
    elif case["op"] == "prefix":
        tails = _numbers(case["tails"])
        lens = [case["prefix"] + t for t in tails]
        # Whole pages of the prompt are shared; a page that it shares with what follows is each row's own copy.
        s["table"], total = _tables([-(-n // page) for n in lens], case["prefix"] // page, g)
        s["pages"] = _filled(case, total, g)
        s["q"] = randn(len(lens), HEADS, dim).to(bf16)
        s["sinks"] = randn(HEADS)
        s["scale"] = dim ** -0.5
        s["rows"] = [(n, 1, 0, e) for e, n in enumerate(lens)]
        s["tail_len"] = torch.tensor(tails, device=DEV)
        s["tail_most"] = max(tails)
        s["out"] = torch.zeros(len(lens), HEADS, dim, dtype=bf16, device=DEV)
    else:
        lens = _numbers(case["lens"])
        s["table"], total = _tables([-(-n // page) for n in lens], 0, g)
        s["pages"] = _filled(case, total, g)
        s["kv_len"] = torch.tensor(lens, device=DEV)
        if case["op"] == "fetch":
            n, live = case["tokens"], case["tokens"] - case["padded"]
            if case["whole"]:
                seq = torch.repeat_interleave(torch.arange(len(lens), device=DEV), s["kv_len"])
                slot = torch.cat([torch.arange(x, device=DEV) for x in lens])
            else:
                seq = torch.randint(0, len(lens), (n,), generator=g, device=DEV)
                slot = (torch.rand(n, generator=g, device=DEV, dtype=torch.float64) * s["kv_len"][seq]).long()
            seq[live:] = -1
            s["seq"], s["slot"] = seq.to(i32), slot.to(i32)
            s["out"] = torch.zeros(n, dim, dtype=TYPES[case["dtype"]], device=DEV)
        else:
            s["q"] = randn(len(lens), HEADS, dim).to(bf16)
            s["w"] = randn(len(lens), HEADS) / 8
            s["scores"] = torch.zeros(len(lens), max(lens), device=DEV)
            s["rows"] = [(n, min(n, 512), 512 * e, e) for e, n in enumerate(lens)]
    if own:
        import deepseek_sparse_attention_ragged_gb300 as ds
        s["ds"] = ds
        s["cache"] = ds.PagedCache(s["pages"], s["table"], page, dim, form)
        if case["op"] == "append":
            s["rope"] = ds.Rope(case["rot"], first=s["first"], layout=case["layout"], base=10000.0, factor=4.0,
                                original_len=4096) if case["rot"] else None
        if case["op"] == "prefix":
            s["workspace"] = ds.prefix_attn_workspace(s["rows"], case["prefix"])
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def _rotated(s, x, positions):
    """Rows x [rows, dim] in 64 bits (the rounding that follows has borders) with their last `rot` features rotated."""
    angle = positions.double()[:, None] * s["theta"]
    c, sn = angle.cos(), angle.sin()
    kept, part = x[:, : s["first"]].double(), x[:, s["first"]:].double()
    if s["layout"] == "interleaved":
        a, b = part[:, 0::2], part[:, 1::2]
        return torch.cat((kept, torch.stack((a * c - b * sn, a * sn + b * c), -1).flatten(1)), 1)
    a, b = part[:, : s["rot"] // 2], part[:, s["rot"] // 2:]
    return torch.cat((kept, a * c - b * sn, a * sn + b * c), 1)


def _places(s, seq, slot):
    return s["table"][seq, slot // s["page"]].long().clamp(min=0), slot % s["page"]


def run(s):
    dim, form, page = s["dim"], s["form"], s["page"]
    if s["op"] == "append":
        if own:
            s["ds"].ds_rows_append(s["cache"], s["x"], s["seq"], s["slot"], rope=s["rope"], positions=s["positions"],
                                   values=s["values"])
            return s["values"]
        live = s["tokens"] - s["padded"]
        ids, at = _places(s, s["seq"][:live].long(), s["slot"][:live].long())
        y = _rotated(s, s["x"][:live], s["positions"][:live])
        s["values"][:live] = _store(s["pages"], dim, form, page, ids, at, y)
        return s["values"]
    if s["op"] == "fetch":
        if own:
            s["ds"].ds_rows_fetch(s["cache"], s["seq"], s["slot"], s["out"])
            return s["out"]
        live = s["tokens"] - s["padded"]
        ids, at = _places(s, s["seq"][:live].long(), s["slot"][:live].long())
        s["out"][:live] = _fetch(s["pages"], dim, form, page, ids, at).to(s["out"].dtype)
        return s["out"]
    if s["op"] == "scores":
        if own:
            s["ds"].ds_rows_indexer_score_paged(s["rows"], s["q"], s["w"], s["cache"], s["scores"])
            return s["scores"]
        j = torch.arange(s["scores"].shape[1], device=DEV)
        ids = s["table"][:, j // page].long().clamp(min=0)
        k = _fetch(s["pages"], dim, form, page, ids, (j % page).expand_as(ids))
        dots = torch.matmul(k, s["q"].float().transpose(1, 2)).clamp_(min=0)  # [rows, keys, heads]
        sums = torch.matmul(dots, s["w"][:, :, None])[..., 0]
        s["scores"].copy_(torch.where(j < s["kv_len"][:, None], sums, s["scores"]))
        return s["scores"]
    if own:
        s["ds"].ds_rows_prefix_attn(s["rows"], s["prefix"], s["q"], s["sinks"], 0, s["scale"], s["out"], s["cache"],
                                    workspace_t=s["workspace"])
        return s["out"]
    rows, prefix = len(s["rows"]), s["prefix"]
    q = s["q"].float()
    j = torch.arange(prefix, device=DEV)
    shared = _fetch(s["pages"], dim, form, page, *_places(s, torch.zeros_like(j), j))
    j = prefix + torch.arange(s["tail_most"], device=DEV).expand(rows, -1)
    there = j < prefix + s["tail_len"][:, None]
    j = torch.where(there, j, 0)  # a row that every sequence has
    e = torch.arange(rows, device=DEV)[:, None].expand_as(j)
    own_rows = _fetch(s["pages"], dim, form, page, *_places(s, e, j))
    a = torch.matmul(q.view(-1, dim), shared.T).view(rows, HEADS, prefix) * s["scale"]
    b = torch.matmul(q, own_rows.transpose(1, 2)) * s["scale"]
    b = torch.where(there[:, None], b, float("-inf"))
    logits = torch.cat((s["sinks"][None, :, None].expand(rows, -1, -1), a, b), -1)
    p = (logits - logits.amax(-1, keepdim=True)).exp()
    den = p.sum(-1, keepdim=True)
    acc = torch.matmul(p[..., 1:1 + prefix].reshape(rows * HEADS, prefix), shared).view(rows, HEADS, dim)
    s["out"].copy_((acc + torch.matmul(p[..., 1 + prefix:], own_rows)) / den)
    return s["out"]


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------

def _turned64(x, positions, case):
    """Rows with their last `rot` features rotated pair by pair as complex numbers, from numpy's 64-bit angles."""
    rot, y = case["rot"], x.double().clone()
    if rot == 0:
        return y
    i = np.arange(rot // 2, dtype=np.float64)
    theta = np.power(10000.0, -2.0 * i / rot)
    bound = [rot * np.log(4096 / (2 * np.pi * r)) / (2 * np.log(10000.0)) for r in (32.0, 1.0)]
    low, high = max(np.floor(bound[0]), 0.0), min(np.ceil(bound[1]), rot - 1.0)
    mix = np.clip((i - low) / max(high - low, 0.001), 0.0, 1.0)
    angle = positions.cpu().numpy().astype(np.float64)[:, None] * (theta * ((1.0 - mix) + mix / 4.0))
    turn = torch.from_numpy(np.exp(1j * angle)).to(DEV)
    first = case["dim"] - rot
    if case["layout"] == "interleaved":
        real, imag = slice(first, None, 2), slice(first + 1, None, 2)
    else:
        real, imag = slice(first, first + rot // 2), slice(first + rot // 2, None)
    z = torch.complex(y[:, real], y[:, imag]) * turn
    y[:, real], y[:, imag] = z.real, z.imag
    return y


def _e4m3(c):
    """The number that an e4m3 byte stands for."""
    exponent, mantissa = c // 8 % 16, c % 8
    v = torch.where(exponent == 0, mantissa / 8 * 2.0 ** -6, (1 + mantissa / 8) * torch.exp2((exponent - 7).double()))
    return torch.where(c >= 128, -v, v).double()


def _rows64(s, e, j):
    """Rows j of sequences e, decoded value by value from the bytes."""
    dim, page, form = s["dim"], s["page"], s["form"]
    ids, at = s["table"][e, j // page].long()[:, None], (j % page)[:, None]
    if form == "bf16":
        return s["pages"].reshape(-1, dim)[(ids * page + at)[:, 0]].double()
    f = torch.arange(dim, device=DEV)
    raw = s["pages"].reshape(-1)
    if form == "fp8":
        start = ids * page * (dim + dim // 128)
        value_at = start + (at * dim + f if dim == KV_DIM else f // 16 * (page * 16) + at * 16 + f % 16)
        scale = raw[start + page * dim + at * (dim // 128) + f // 128].double() - 127
        return _e4m3(raw[value_at].long()) * torch.exp2(scale)
    word, i = f // 8, f % 8
    bit = 4 * (i // 2) + 16 * (i % 2)
    byte = 4 * word + bit // 8
    start = ids * page * (dim // 2 + dim // 16)
    if dim == KV_DIM:
        value_at, scale_at = start + at * 288 + byte, start + at * 288 + 256 + f // 16
    else:
        value_at = start + byte // 16 * (page * 16) + at * 16 + byte % 16
        scale_at = start + page * 64 + at * 8 + f // 16
    return ((raw[value_at].long() >> bit % 8) % 16 - 8).double() * _e4m3(raw[scale_at].long())


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "append":
        live = case["tokens"] - case["padded"]
        block = _turned64(s["x"][:live], s["positions"][:live], case).reshape(live, -1, 128)
        top = torch.clamp(block.abs().amax(-1, keepdim=True), min=1e-37)
        e = torch.clamp(torch.ceil(torch.log2(top / 448)), -100, 7)
        e = torch.where((top <= 448 * torch.exp2(e - 1)) & (e > -100), e - 1, e)  # log2 is not exact next to a power
        v = block / torch.exp2(e)
        # e4m3: steps of 2^(exponent - 3), no exponent under -6; half goes to even.
        step = torch.exp2(torch.clamp(torch.floor(torch.log2(torch.clamp(v.abs(), min=1e-30))), min=-6) - 3)
        v = torch.clamp(torch.round(v / step) * step, -448, 448)
        out = torch.zeros(case["tokens"], case["dim"], dtype=torch.float64, device=DEV)
        out[:live] = (v * torch.exp2(e)).reshape(live, -1)
        return out
    if case["op"] == "fetch":
        live = case["tokens"] - case["padded"]
        out = torch.zeros(case["tokens"], case["dim"], dtype=torch.float64, device=DEV)
        for i in torch.arange(live, device=DEV).split(16384):
            out[i] = _rows64(s, s["seq"][i].long(), s["slot"][i].long())
        return out
    if case["op"] == "scores":
        out = s["scores"].double()
        for e, n in enumerate(_numbers(case["lens"])):
            for j in torch.arange(n, device=DEV).split(16384):
                k = _rows64(s, torch.full_like(j, e), j)
                out[e, j] = (torch.relu(k @ s["q"][e].double().T) * s["w"][e].double()).sum(1)
        return out
    prefix, tails = case["prefix"], _numbers(case["tails"])
    out = torch.zeros(len(tails), HEADS, KV_DIM, dtype=torch.float64, device=DEV)
    shared = [_rows64(s, torch.zeros_like(j), j) for j in torch.arange(prefix, device=DEV).split(16384)] if prefix else []
    for e, n in enumerate(tails):
        j = prefix + torch.arange(n, device=DEV)
        kv = torch.cat([*shared, _rows64(s, torch.full_like(j, e), j)])
        logits = torch.cat((s["q"][e].double() @ kv.T * s["scale"], s["sinks"].double()[:, None]), 1)
        out[e] = torch.softmax(logits, 1)[:, :-1] @ kv
    return out
