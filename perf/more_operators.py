"""Cases of the eight-bit attention layer's operators: heads normed, turned by positions of several axes and appended;
rows quantized into a paged E4M3 cache with a power-of-two scale per block of tokens and head; attention over that
cache; tokens quantized to 8-bit integers; the matrix product of 8-bit integers with scales per token and channel.

``own`` false computes each operator in elementary torch operations in 32 bits (64 for angles), rounded once at the
end; ``own`` true calls the library's entry points.  8 query heads on one key/value head of 256, 10 and 50 action
rows, 768 encoder tokens and the widths 1024, 2048, 4096 and 16384 are this library's own; the other layouts are
generic grouped-head ones.
"""
import itertools
import math
import random

import torch

own = False

PAGE = 16                       # cache rows per page unless a case says otherwise
# (query heads, key/value heads, head size)
HEADS = ((8, 1, 256), (32, 8, 128), (16, 2, 64), (28, 4, 128), (16, 16, 72), (12, 12, 80), (40, 8, 128), (8, 8, 64))
MOST_E4M3 = 448.0


# ---------------------------------------------------------------- cases

def _axes(name, frames, height, width, text, heads, rot, shares, interleaved, norm, base, append):
    """frames x height x width image tokens, then `text` tokens whose axes advance together; `shares`: how many of
    the pairs turn by each axis, in eighths of rot, one digit an axis (the last takes the rest)."""
    return {"name": name, "op": "axes", "frames": frames, "height": height, "width": width, "text": text,
            "heads": heads[0], "kv_heads": heads[1], "dim": heads[2], "rot": rot, "shares": shares,
            "interleaved": interleaved, "norm": norm, "base": base, "append": append}


def _append(name, sequences, rows, before, page, block, kv_heads, dim):
    """`rows` new rows of ragged sequences in all, behind up to `before` cached ones each."""
    return {"name": name, "op": "append", "sequences": sequences, "rows": rows, "before": before, "page": page,
            "block": block, "kv_heads": kv_heads, "dim": dim}


def _attend(name, sequences, rows, prefix, suffix, page, block, heads, causal):
    return {"name": name, "op": "attend", "sequences": sequences, "rows": rows, "prefix": prefix, "suffix": suffix,
            "page": page, "block": block, "heads": heads[0], "kv_heads": heads[1], "dim": heads[2], "causal": causal}


def _tokens(name, m, k):
    return {"name": name, "op": "tokens", "m": m, "k": k}


def _product(name, m, n, k, bias, residual):
    return {"name": name, "op": "product", "m": m, "n": n, "k": k, "bias": bias, "residual": residual}


def listed():
    return [
        # one camera's 16 x 16 patches inside the vision tower: two axes, no cache
        _axes("axes 256 patches", 1, 16, 16, 0, HEADS[4], 72, "4", False, False, 10000.0, False),
        # a clip's frames and the instruction behind them, time, height and width, into the language model's cache
        _axes("axes 12601 video tokens", 4, 56, 56, 57, HEADS[1], 128, "23", False, True, 1000000.0, True),
        # 64 sequences decode one token each: blocks that are partly filled, some of whose scales grow
        _append("append 64 tokens", 64, 64, 3000, 16, 16, 8, 128),
        # a batch of 16 ragged prompts, some behind earlier chunks
        _append("append 16 ragged prompts", 16, 9001, 700, 64, 32, 8, 128),
        # one denoising step: 10 action rows over the encoder's cached keys and their own
        _attend("attend 10 rows", 1, 10, 768, 10, PAGE, 16, HEADS[0], False),
        # one token of one sequence with a very long cache and no shared prefix
        _attend("attend one token long", 1, 1, 0, 131071, 64, 64, HEADS[1], True),
        # 64 sequences decode one token each behind one shared prompt, ragged histories of their own
        _attend("attend 64 sequences", 64, 1, 2051, 3000, PAGE, 16, HEADS[1], True),
        # the action rows before the decoder's GEMMs
        _tokens("tokens 50 x 1024", 50, 1024),
        # a batch of encoder tokens before the down-projection
        _tokens("tokens 8191 x 4096", 8191, 4096),
        # the decoder's up-projection for 50 action rows: the weights' bytes
        _product("product 50 x 4096 x 1024", 50, 4096, 1024, False, False),
        # the encoder's down-projection with bias and residual
        _product("product 768 x 2048 x 16384", 768, 2048, 16384, True, True),
        # a long prompt's up-projection
        _product("product 8191 x 16384 x 2048", 8191, 16384, 2048, False, False),
    ]


def _spread(rng, low, high):
    """A whole number between low and high, even over its logarithm."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    heads = rng.choice(HEADS)
    op = rng.choice(("axes", "append", "attend", "attend", "tokens", "product", "product"))
    if op == "axes":
        most = 12000 * 48 * 128 // ((heads[0] + 2 * heads[1]) * max(heads[2], 128))
        frames, text = rng.choice((1, 1, 2, 4, 7)), rng.choice((0, 1, _spread(rng, 1, 500)))
        side = max(1, int(math.sqrt(most / frames)))
        height, width = _spread(rng, 1, side), _spread(rng, 1, side)
        rots = [r for r in (heads[2], heads[2], 64, 32) if r <= heads[2]]
        case = _axes("", frames, height, width, text, heads, rng.choice(rots), rng.choice(("4", "23", "26", "8", "0")),
                     rng.random() < 0.4, rng.random() < 0.5, rng.choice((10000.0, 1000000.0)), rng.random() < 0.6)
    elif op == "append":
        sequences = _spread(rng, 1, 96)
        rows = rng.choice((sequences, _spread(rng, sequences, 9000)))
        page = rng.choice((16, 32, 64, 128))
        case = _append("", sequences, rows, rng.choice((0, _spread(rng, 1, 2000))), page,
                       rng.choice([b for b in (1, 16, 32, 64, 128) if b <= page]), min(heads[1], 8), min(heads[2], 128) if heads[1] > 1 else heads[2])
    elif op == "attend":
        rows = rng.choice((1, 1, 1, 2, 5, 10, 50))
        sequences = _spread(rng, 1, 64 if rows < 50 else 32)
        prefix = rng.choice((0, _spread(rng, 17, 8000)))
        most = max(64, min(60000, 120000 * 8 // (sequences * heads[1]))) if rows == 1 else 400
        suffix = max(rows, _spread(rng, 1, most))
        page = rng.choice((16, 64))
        case = _attend("", sequences, rows, prefix, suffix, page, rng.choice([b for b in (4, 16, 64) if b <= page]), heads,
                       rng.random() < 0.5)
    elif op == "tokens":
        k = 32 * _spread(rng, 1, 512)
        case = _tokens("", _spread(rng, 1, min(8191, 8191 * 4096 // k)), k)
    else:
        k, n = 32 * _spread(rng, 1, 512), 16 * _spread(rng, 1, 1024)
        most = 8191 * 16384 * 2048 // (n * k)
        case = _product("", _spread(rng, 1, max(1, min(8191, most))), n, k, rng.random() < 0.5, rng.random() < 0.5)
    del case["name"]
    return case


def _lengths(total, parts, least):
    """`total` split into `parts` ragged lengths, `least` at least, always the same ones for the same numbers."""
    rng = random.Random("%d in %d" % (total, parts))
    weights = [math.exp(rng.gauss(0.0, 0.8)) for _ in range(parts)]
    whole, spare = sum(weights), total - least * parts
    lengths = [least + int(spare * w / whole) for w in weights]
    lengths[0] += total - sum(lengths)
    rng.shuffle(lengths)
    return lengths


def _append_lengths(case):
    """(new rows, rows cached before) of each sequence."""
    rows = _lengths(case["rows"], case["sequences"], min(1, case["rows"] // case["sequences"]))
    rng = random.Random("before %d %d" % (case["before"], case["sequences"]))
    return rows, [rng.randint(0, case["before"]) for _ in rows]


def _suffix_lengths(case):
    """Cached rows of each sequence behind the prefix, the call's own rows among them."""
    if case["sequences"] == 1:
        return [case["suffix"]]
    rng = random.Random("suffix %d %d" % (case["suffix"], case["sequences"]))
    return [rng.randint(case["rows"], case["suffix"]) for _ in range(case["sequences"])]


def _count(case):
    return case["frames"] * case["height"] * case["width"] + case["text"]


def work(case):
    op = case["op"]
    if op == "axes":
        t, hq, hk, d = _count(case), case["heads"], case["kv_heads"], case["dim"]
        read = t * (hq + (2 if case["append"] else 1) * hk) * d * 2 + t * (4 * (len(case["shares"]) + 1)) + case["rot"] * 2
        written = t * (hq + hk) * d * 2 + (t * 2 * hk * d * 2 + 8 * t if case["append"] else 0)
        return {"bytes": read + written, "flops": t * (hq + hk) * (3 * case["rot"] + (4 * d if case["norm"] else 0))}
    if op == "append":
        rows, before = _append_lengths(case)
        block, width = case["block"], case["kv_heads"] * case["dim"]
        touched = sum((b + n - 1) // block - b // block + 1 for n, b in zip(rows, before) if n)
        return {"bytes": sum(rows) * width * 2 * 3 + touched * case["kv_heads"] * 2, "flops": sum(rows) * width * 4}
    if op == "attend":
        hq, hk, d, rows = case["heads"], case["kv_heads"], case["dim"], case["rows"]
        lengths = _suffix_lengths(case)
        own_pairs = [sum(max(0, min(n, i + 1 + n - rows)) for i in range(rows)) if case["causal"] else rows * n for n in lengths]
        cached = case["prefix"] + sum(lengths)
        scales = cached // case["block"] + 1
        return {"bytes": 2 * d * 2 * len(lengths) * rows * hq + 2 * hk * (cached * d + scales),
                "flops": 4 * d * hq * (len(lengths) * rows * case["prefix"] + sum(own_pairs))}
    if op == "tokens":
        return {"bytes": case["m"] * (3 * case["k"] + 4), "flops": 2 * case["m"] * case["k"]}
    m, n, k = case["m"], case["n"], case["k"]
    more = (2 * n if case["bias"] else 0) + (2 * m * n if case["residual"] else 0)
    return {"bytes": m * k + n * k + 4 * (m + n) + 2 * m * n + more, "flops": 2 * m * n * k}


# --------------------------------------------------------------- inputs

def _normal(gen, *shape, scale=1.0):
    return (torch.randn(*shape, device="cuda", generator=gen) * scale).to(torch.bfloat16)


def _offsets(lengths):
    return torch.tensor([0] + list(itertools.accumulate(lengths)), dtype=torch.int32, device="cuda")


def _shares(case):
    """How many pairs turn by each axis."""
    pairs = case["rot"] // 2
    first = [pairs * int(x) // 8 for x in case["shares"]]
    return first + [pairs - sum(first)]


def _prepare_axes(case, gen):
    hq, hk, d, rot = case["heads"], case["kv_heads"], case["dim"], case["rot"]
    t, axes = _count(case), len(case["shares"]) + 1
    at = torch.arange(case["frames"] * case["height"] * case["width"], device="cuda")
    frame, rest = at // (case["height"] * case["width"]), at % (case["height"] * case["width"])
    image = torch.stack((frame, rest // case["width"], rest % case["width"]))[3 - axes:]
    text = torch.arange(case["text"], device="cuda").expand(axes, -1) + max(case["frames"], case["height"], case["width"])
    shares = _shares(case)
    axis_of = torch.repeat_interleave(torch.arange(axes), torch.tensor(shares)).to(torch.uint8).cuda()
    j = torch.arange(rot // 2, device="cuda", dtype=torch.float64)
    qkv = _normal(gen, t, (hq + 2 * hk) * d)
    s = {"qkv": qkv, "q": qkv[:, :hq * d], "k": qkv[:, hq * d:(hq + hk) * d], "v": qkv[:, (hq + hk) * d:],
         "inv_freq": (case["base"] ** (-2.0 * j / rot)).float(), "axis_of": axis_of, "axes": axes, "eps": 1e-6,
         "positions": torch.cat((image, text), 1).to(torch.int32).contiguous(), "q_weight": None, "k_weight": None,
         "slots": None, "k_cache": None, "v_cache": None, "num_slots": 0,
         "q_out": torch.zeros(t, hq, d, dtype=torch.bfloat16, device="cuda"),
         "k_out": torch.zeros(t, hk, d, dtype=torch.bfloat16, device="cuda")}
    if case["append"]:
        pages = -(-t // PAGE) + 5
        table, row = torch.randperm(pages, device="cuda", generator=gen), torch.arange(t, device="cuda")
        s.update(slots=table[row // PAGE] * PAGE + row % PAGE, num_slots=pages * PAGE,
                 k_cache=_normal(gen, pages * PAGE, hk, d), v_cache=_normal(gen, pages * PAGE, hk, d))
    if case["norm"]:
        s["q_weight"], s["k_weight"] = (1 + _normal(gen, d, scale=0.2) for _ in range(2))
    return s


def _power(byte):
    """2^(byte - 127) in fp32, byte 0 being the subnormal 2^-127."""
    bits = byte.to(torch.int32) << 23
    return torch.where(bits == 0, torch.full_like(bits, 0x00400000), bits).view(torch.float32)


def _scale_byte(most):
    """The byte of the least power of two 2^e, e >= -127, with most <= 448 * 2^e; 0 for 0."""
    fraction, exponent = torch.frexp(most)
    byte = exponent - 9 + (fraction > 0.875).to(exponent.dtype) + 127
    return torch.where(most == 0, torch.zeros_like(byte), byte).clamp_(0, 254).to(torch.uint8)


def _encode(x, byte):
    """E4M3 codes of x (fp32) under the scales of `byte` (which broadcasts)."""
    return (x * _power(254 - byte.to(torch.int32))).to(torch.float8_e4m3fn).view(torch.uint8)


def _decode(code, byte):
    return code.view(torch.float8_e4m3fn).float() * _power(byte)


def _cache(gen, pages, page, block, kv_heads, dim):
    """A filled cache: codes and scale bytes.  Magnitudes differ from block to block and head to head."""
    x = torch.randn(pages * page // block, block, kv_heads, dim, device="cuda", generator=gen)
    x *= torch.exp(0.5 * torch.randn(x.shape[0], 1, kv_heads, 1, device="cuda", generator=gen))
    byte = _scale_byte(x.abs().amax((1, 3)))
    return _encode(x, byte[:, None, :, None]).reshape(pages * page, kv_heads, dim), byte


def _prepare_append(case, gen):
    hk, d, page = case["kv_heads"], case["dim"], case["page"]
    rows, before = _append_lengths(case)
    each = max(-(-(n + b) // page) for n, b in zip(rows, before)) + 1
    pages = each * len(rows) + 3
    table = torch.randperm(pages, device="cuda", generator=gen)[:each * len(rows)].to(torch.int32)
    total = sum(rows)
    kv = torch.randn(total, 2 * hk, d, device="cuda", generator=gen)
    kv *= torch.exp(0.7 * torch.randn(total, 2 * hk, 1, device="cuda", generator=gen))
    kv = kv.to(torch.bfloat16).reshape(total, 2 * hk * d)
    s = {"kv": kv, "k": kv[:, :hk * d], "v": kv[:, hk * d:], "cu_rows": _offsets(rows), "total": total, "longest": max(rows),
         "block_table": table.reshape(len(rows), each).contiguous(), "pages": (pages, each),
         "seq_lens": torch.tensor([n + b for n, b in zip(rows, before)], dtype=torch.int32, device="cuda")}
    for c in ("k", "v"):
        s[c + "_cache"], s[c + "_scales"] = _cache(gen, pages, page, case["block"], hk, d)
    return s


def _prepare_attend(case, gen):
    hq, hk, d, page, b = case["heads"], case["kv_heads"], case["dim"], case["page"], case["sequences"]
    lengths = _suffix_lengths(case)
    shared, each = -(-case["prefix"] // page), -(-case["suffix"] // page)
    pages = shared + each * b + 3
    table = torch.randperm(pages, device="cuda", generator=gen).to(torch.int32)
    # logits of a few units: rows attend to a minority of their keys
    s = {"q": _normal(gen, b * case["rows"], hq, d, scale=2.0),
         "prefix_pages": table[:shared].clone() if shared else None,
         "prefix_len": torch.tensor([case["prefix"]], dtype=torch.int32, device="cuda") if shared else None,
         "block_table": table[shared:shared + each * b].reshape(b, each).clone(),
         "seq_lens": torch.tensor(lengths, dtype=torch.int32, device="cuda"),
         "pages": (pages, shared, each), "scale": 1.0 / math.sqrt(d),
         "out": torch.zeros(b * case["rows"], hq, d, dtype=torch.bfloat16, device="cuda")}
    for c in ("k", "v"):
        s[c + "_cache"], s[c + "_scales"] = _cache(gen, pages, page, case["block"], hk, d)
    if own:
        import bf16_gemm_vla_amd as vla

        n = vla.vla_attn_shared_prefix_e4m3_workspace_bytes(b, case["rows"], hq, hk, d, shared * page, each * page)
        s["ws"] = torch.empty(n, dtype=torch.uint8, device="cuda")      # kept by the program
    return s


def _integers(x):
    """Rows of 8-bit integers and a scale for each: max |row| / 127, the nearest integer to x / scale, ties to even."""
    scale = x.abs().amax(1) / 127.0
    scale = torch.where(scale == 0, torch.ones_like(scale), scale)
    return torch.round(x / scale[:, None]).clamp_(-127, 127).to(torch.int8), scale


def _prepare_tokens(case, gen):
    m, k = case["m"], case["k"]
    x = torch.randn(m, k, device="cuda", generator=gen)
    # tokens of different magnitude, a few channels that stand out
    x *= torch.exp(0.7 * torch.randn(m, 1, device="cuda", generator=gen))
    x[:, :: max(1, k // 5)] *= 8.0
    return {"x": x.to(torch.bfloat16), "codes": torch.zeros(m, k, dtype=torch.int8, device="cuda"),
            "scales": torch.zeros(m, dtype=torch.float32, device="cuda")}


def _prepare_product(case, gen):
    m, n, k = case["m"], case["n"], case["k"]
    a, s_a = _integers(torch.randn(m, k, device="cuda", generator=gen) * torch.exp(0.5 * torch.randn(m, 1, device="cuda", generator=gen)))
    w, s_w = _integers(torch.randn(n, k, device="cuda", generator=gen) * 0.02)
    s = {"a": a, "s_a": s_a, "w": w, "s_w": s_w, "y": torch.zeros(m, n, dtype=torch.bfloat16, device="cuda"),
         "bias": _normal(gen, n, scale=0.5) if case["bias"] else None,
         "residual": _normal(gen, m, n) if case["residual"] else None}
    if own:
        import bf16_gemm_vla_amd as vla

        # laid out and zero-filled once, where the weights are loaded
        s["packed"] = torch.empty(n * k, dtype=torch.int8, device="cuda")
        vla.vla_pack_fp8(w, s["packed"], n, k)
        s["ws"] = torch.zeros(vla.vla_gemm_workspace_bytes(m, n, k, vla.VLA_WFMT_INT8), dtype=torch.uint8, device="cuda")
    return s


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    make = {"axes": _prepare_axes, "append": _prepare_append, "attend": _prepare_attend, "tokens": _prepare_tokens,
            "product": _prepare_product}[case["op"]]
    return dict(make(case, gen), case=case)


# ---------------------------------------------------------- plain forms

def _plain_heads(x, weight, cos, sin, rot, interleaved, eps):
    """Normed and rotated heads of x (tokens x heads x size), in fp32, rounded once."""
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * weight.float()
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
    turned = (a * cos - b * sin, b * cos + a * sin)
    turned = torch.stack(turned, -1).flatten(-2) if interleaved else torch.cat(turned, -1)
    return torch.cat((turned, x[..., rot:]), -1).to(torch.bfloat16)


def _plain_axes(s):
    case = s["case"]
    hq, hk, d, rot = case["heads"], case["kv_heads"], case["dim"], case["rot"]
    t = s["q"].shape[0]
    angle = (s["positions"].double()[s["axis_of"].long()].t() * s["inv_freq"].double())[:, None, :]
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    s["q_out"].copy_(_plain_heads(s["q"].reshape(t, hq, d), s["q_weight"], cos, sin, rot, case["interleaved"], s["eps"]))
    s["k_out"].copy_(_plain_heads(s["k"].reshape(t, hk, d), s["k_weight"], cos, sin, rot, case["interleaved"], s["eps"]))
    if case["append"]:
        s["k_cache"][s["slots"]] = s["k_out"]
        s["v_cache"][s["slots"]] = s["v"].reshape(t, hk, d)


def _plain_append(s):
    case = s["case"]
    hk, d, page, block = case["kv_heads"], case["dim"], case["page"], case["block"]
    at = torch.arange(s["total"], device="cuda", dtype=torch.int32)
    b = torch.searchsorted(s["cu_rows"], at, right=True) - 1
    position = (s["seq_lens"] - s["cu_rows"][1:])[b] + at
    slot = s["block_table"][b, (position // page).long()].long() * page + position % page
    of = slot // block
    blocks = s["k_cache"].shape[0] // block
    first = torch.full((blocks,), block, device="cuda").scatter_reduce_(0, of, (position % block).long(), "amin")
    touched = torch.nonzero(first < block)[:, 0]
    earlier = torch.arange(block, device="cuda") < first[touched][:, None]
    for c in ("k", "v"):
        x, cache, scales = s[c].reshape(-1, hk, d).float(), s[c + "_cache"], s[c + "_scales"]
        most = torch.zeros(blocks, hk, device="cuda").index_reduce_(0, of, x.abs().amax(-1), "amax")[touched]
        old = torch.where(first[touched][:, None] > 0, scales[touched], torch.zeros_like(scales[touched]))
        new = torch.maximum(_scale_byte(most), old)
        rows = cache.reshape(blocks, block, hk, d)
        codes = _encode(_decode(rows[touched], old[:, None, :, None]), new[:, None, :, None])
        rows[touched] = torch.where(earlier[:, :, None, None], codes, rows[touched])
        scales[touched] = new
        cache[slot] = _encode(x, scales[of][:, :, None])


def _plain_attend(s):
    """fp32 throughout; a row that sees nothing gives 0."""
    case = s["case"]
    b, rows, page, hq, hk, d = (case[c] for c in ("sequences", "rows", "page", "heads", "kv_heads", "dim"))
    inside = torch.arange(page, device="cuda")
    slot = (s["block_table"].long()[:, :, None] * page + inside).reshape(b, -1)
    j, i = torch.arange(slot.shape[1], device="cuda"), torch.arange(rows, device="cuda")
    length = s["seq_lens"][:, None, None]
    seen = (j < length).expand(b, rows, -1)
    if case["causal"]:
        seen = seen & (j <= i[:, None] + length - rows)
    if s["prefix_pages"] is not None:
        shared = (s["prefix_pages"].long()[:, None] * page + inside).reshape(1, -1).expand(b, -1)
        there = torch.arange(shared.shape[1], device="cuda") < s["prefix_len"]
        slot, seen = torch.cat((shared, slot), 1), torch.cat((there.expand(b, rows, -1), seen), 2)

    def rows_of(c):
        x = _decode(s[c + "_cache"][slot], s[c + "_scales"][slot // case["block"]][..., None])
        return x.permute(0, 2, 1, 3).contiguous()

    q = s["q"].float().reshape(b, rows, hk, hq // hk, d).permute(0, 2, 3, 1, 4).reshape(b, hk, -1, d)
    scores = torch.matmul(q, rows_of("k").transpose(2, 3).contiguous()).mul_(s["scale"]).reshape(b, hk, hq // hk, rows, -1)
    scores.masked_fill_(~seen[:, None, None], float("-inf"))
    top = scores.amax(-1, keepdim=True).clamp_(min=-3e38)
    scores.sub_(top).exp_()
    total = scores.sum(-1, keepdim=True).clamp_(min=1e-38)
    out = torch.matmul(scores.reshape(b, hk, -1, scores.shape[-1]), rows_of("v")).reshape(b, hk, hq // hk, rows, d) / total
    s["out"].copy_(out.permute(0, 3, 1, 2, 4).reshape(s["out"].shape).to(torch.bfloat16))


def _plain_tokens(s):
    codes, scales = _integers(s["x"].float())
    s["codes"].copy_(codes)
    s["scales"].copy_(scales)


def _plain_product(s):
    # products of up to 127 * 127, exact; their sums in fp32 are off by far less than the output's rounding
    y = torch.matmul(s["a"].float(), s["w"].float().t()) * s["s_a"][:, None] * s["s_w"]
    if s["bias"] is not None:
        y = y + s["bias"].float()
    y = y.to(torch.bfloat16)
    s["y"].copy_(y if s["residual"] is None else (s["residual"].float() + y.float()).to(torch.bfloat16))


def _own(s):
    import bf16_gemm_vla_amd as vla

    case = s["case"]
    op = case["op"]
    if op == "axes":
        hq, hk, d = case["heads"], case["kv_heads"], case["dim"]
        t, stride = s["qkv"].shape
        vla.vla_qk_norm_rope_axes_append(
            s["q"], s["k"], s["v"] if case["append"] else None, s["q_weight"], s["k_weight"], s["inv_freq"], s["axis_of"],
            s["positions"], s["slots"], s["q_out"], s["k_out"], s["k_cache"], s["v_cache"], t, hq, hk, d, case["rot"],
            s["axes"], stride, stride, stride, hq * d, hk * d, s["num_slots"],
            vla.VLA_ROPE_INTERLEAVED if case["interleaved"] else vla.VLA_ROPE_HALF, 1.0, s["eps"])
    elif op == "append":
        hk, d = case["kv_heads"], case["dim"]
        pages, each = s["pages"]
        vla.vla_kv_append_e4m3(
            s["k"], s["v"], s["cu_rows"], s["block_table"], s["seq_lens"], s["k_cache"], s["v_cache"], s["k_scales"],
            s["v_scales"], case["sequences"], s["longest"], s["total"], hk, d, pages, case["page"], case["block"], each,
            2 * hk * d, 2 * hk * d)
    elif op == "attend":
        hq, hk, d = case["heads"], case["kv_heads"], case["dim"]
        pages, shared, each = s["pages"]
        vla.vla_attn_shared_prefix_e4m3(
            s["q"], s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"], s["prefix_pages"], s["prefix_len"],
            s["block_table"], s["seq_lens"], s["out"], s["ws"], s["ws"].numel(), case["sequences"], case["rows"], hq, hk, d,
            pages, case["page"], case["block"], shared, each, hq * d, hq * d, case["causal"], s["scale"])
    elif op == "tokens":
        vla.vla_quantize_tokens_int8(s["x"], s["codes"], s["scales"], case["m"], case["k"])
    else:
        vla.vla_gemm_int8(s["a"], s["s_a"], s["packed"], s["s_w"], s["bias"], s["residual"], s["y"], s["ws"],
                          s["ws"].numel(), case["m"], case["n"], case["k"])


PLAIN = {"axes": _plain_axes, "append": _plain_append, "attend": _plain_attend, "tokens": _plain_tokens,
         "product": _plain_product}


def run(state):
    op = state["case"]["op"]
    if own:
        _own(state)
    else:
        PLAIN[op](state)
    if op == "axes":
        keys = ("q_out", "k_out") + (("k_cache", "v_cache") if state["case"]["append"] else ())
        return {c: state[c] for c in keys}
    if op == "append":
        out = {c: state[c].view(torch.float8_e4m3fn) for c in ("k_cache", "v_cache")}
        return dict(out, **{c: state[c].view(torch.float8_e8m0fnu) for c in ("k_scales", "v_scales")})
    if op == "attend":
        return {"out": state["out"]}
    return {c: state[c] for c in (("codes", "scales") if op == "tokens" else ("y",))}


# ------------------------------------------------------- 64-bit results

def _exact_axes(s):
    case = s["case"]
    t, rot = s["q"].shape[0], case["rot"]
    angle = torch.empty(t, rot // 2, dtype=torch.float64, device="cuda")
    for j, axis in enumerate(s["axis_of"].tolist()):
        angle[:, j] = s["positions"][axis].double() * s["inv_freq"][j].double()
    turn = torch.polar(torch.ones_like(angle), angle)[:, None]

    def head(x, weight):
        x = x.double().reshape(t, -1, case["dim"])
        if weight is not None:
            x = weight.double() * x / (x.pow(2).sum(-1, keepdim=True) / case["dim"] + s["eps"]).sqrt()
        y = x.clone()
        first, second = (slice(0, rot, 2), slice(1, rot, 2)) if case["interleaved"] else (slice(0, rot // 2), slice(rot // 2, rot))
        z = torch.complex(x[..., first], x[..., second]) * turn
        y[..., first], y[..., second] = z.real, z.imag
        return y

    out = {"q_out": head(s["q"], s["q_weight"]), "k_out": head(s["k"], s["k_weight"])}
    if case["append"]:
        for c, x in (("k", out["k_out"]), ("v", s["v"].double().reshape(t, -1, case["dim"]))):
            out[c + "_cache"] = s[c + "_cache"].double().index_copy(0, s["slots"], x)
    return out


def _e4m3_values():
    """The 256 values of the format by its definition (NaN where it has none)."""
    values = []
    for code in range(256):
        e, m = code >> 3 & 15, code & 7
        v = float("nan") if e == 15 and m == 7 else math.ldexp(m, -9) if e == 0 else math.ldexp(8 + m, e - 10)
        values.append(-v if code & 128 else v)
    return torch.tensor(values, dtype=torch.float64, device="cuda")


def _nearest_e4m3(x):
    """The format's value nearest to x, ties to the even one; |x| <= 448."""
    spacing = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(x / spacing) * spacing


def _exact_append(s):
    case = s["case"]
    block, page = case["block"], case["page"]
    values, out = _e4m3_values(), {}
    cu, lens, table = s["cu_rows"].tolist(), s["seq_lens"].tolist(), s["block_table"].tolist()
    places = []                                      # (block, its first new row's place, first row and number of new rows)
    for b, n in enumerate(lens):
        at, p = cu[b], n - (cu[b + 1] - cu[b])
        while p < n:
            some = min(n - p, block - p % block)
            places.append(((table[b][p // page] * page + p % page) // block, p % block, at, some))
            at, p = at + some, p + some
    which, start, row, some = (torch.tensor(c, device="cuda") for c in zip(*places))
    r = torch.arange(block, device="cuda")
    fresh = (r >= start[:, None]) & (r < (start + some)[:, None])
    source = (row[:, None] + r - start[:, None]).clamp(0, s["total"] - 1)
    for c in ("k", "v"):
        x = s[c].double().reshape(-1, case["kv_heads"], case["dim"])[source] * fresh[:, :, None, None]
        cached = values[s[c + "_cache"].long()].reshape(-1, block, case["kv_heads"], case["dim"])
        exponents = s[c + "_scales"].double() - 127
        least = torch.ceil(torch.log2((x.abs().amax((1, 3)) / MOST_E4M3).clamp(min=2.0 ** -127)))
        grown = torch.where(start[:, None] > 0, torch.maximum(least, exponents[which]), least)
        earlier = (r < start[:, None])[:, :, None, None]
        was = cached[which]
        moved = _nearest_e4m3(was * torch.exp2(exponents[which] - grown)[:, None, :, None])
        new = _nearest_e4m3(x / torch.exp2(grown)[:, None, :, None])
        cached[which] = torch.where(fresh[:, :, None, None], new, torch.where(earlier, moved, was))
        exponents[which] = grown
        out[c + "_cache"] = cached.reshape(s[c + "_cache"].shape)
        out[c + "_scales"] = torch.exp2(exponents)
    return out


def _exact_attend(s):
    case = s["case"]
    rows, page, prefix, block = case["rows"], case["page"], case["prefix"], case["block"]
    hq, hk = case["heads"], case["kv_heads"]
    values, out = _e4m3_values(), s["out"].double()

    def cached(c, pages, n, h):
        slot = (pages.long()[:, None] * page + torch.arange(page, device="cuda")).flatten()[:n]
        return values[s[c + "_cache"][slot, h].long()] * torch.exp2(s[c + "_scales"][slot // block, h].double() - 127)[:, None]

    for h in range(hk):
        shared = [cached(c, s["prefix_pages"], prefix, h) for c in ("k", "v")] if prefix else None
        for b, n in enumerate(s["seq_lens"].tolist()):
            k, v = (cached(c, s["block_table"][b], n, h) for c in ("k", "v"))
            if prefix:
                k, v = torch.cat((shared[0], k)), torch.cat((shared[1], v))
            limits = torch.full((rows,), prefix + n, device="cuda")
            if case["causal"]:
                limits = prefix + (torch.arange(rows, device="cuda") + 1 + n - rows).clamp(0, n)
            hidden = torch.arange(k.shape[0], device="cuda") >= limits[:, None, None]
            q = s["q"][b * rows:(b + 1) * rows, h * hq // hk:(h + 1) * hq // hk].double()
            weight = torch.softmax((q @ k.t() * s["scale"]).masked_fill_(hidden, -1e300), -1)
            out[b * rows:(b + 1) * rows, h * hq // hk:(h + 1) * hq // hk] = weight @ v * (limits > 0)[:, None, None]
    return {"out": out}


def _exact_tokens(s):
    # the scale is rounded to fp32, and the codes are those under the rounded scale
    scale = s["x"].double().abs().amax(1) / 127
    return {"codes": None, "scales": torch.where(scale == 0, 1.0, scale)}


def _exact_product(s):
    y = (s["a"].double() @ s["w"].double().t()) * (s["s_a"].double()[:, None] * s["s_w"].double()[None, :])
    for more in ("bias", "residual"):
        if s[more] is not None:
            y += s[more].double()
    return {"y": y}


def exact(case, seed):
    s = prepare(case, seed)
    return {"axes": _exact_axes, "append": _exact_append, "attend": _exact_attend, "tokens": _exact_tokens,
            "product": _exact_product}[case["op"]](s)
