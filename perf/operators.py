"""What is measured of the serving operators around the quantized products: appending keys and values to a
paged 8-bit cache, attention over that cache, and token log probabilities.

A case is a dict of plain values; `prepare` makes its inputs on the GPU from a seed, `run` does one pass (in
elementary torch operations, or through the package's entry points where `own` is set), `exact` states the
result in 64 bits, `work` the bytes and operations that a pass cannot do without.
"""
import math

import torch

own = False

DTYPE = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}


# ---------------------------------------------------------------- cases
def listed():
    return [
        # One decode step of a small batch: a token of each sequence goes into its partly filled page.
        dict(name="append step 16", op="append", batch=16, heads=8, dim=128, page=16, type="f32", new=1, past=1000, rot=128,
             adjacent=False),
        # One decode step of a full server: 256 sequences, fp16 projections, half of each head rotated, adjacent pairs.
        dict(name="append step 256", op="append", batch=256, heads=8, dim=128, page=32, type="f16", new=1, past=4000, rot=64,
             adjacent=True),
        # Ragged prompts that continue cached ones, pages entered and left in the middle, small heads, no rotation.
        dict(name="append ragged prompts", op="append", batch=7, heads=32, dim=64, page=64, type="bf16", new=700, past=333, rot=0,
             adjacent=False),
        # Long prompts into an empty cache: 4 x 8192 tokens of the 70B-class layer's k and v projections.
        dict(name="append long prompts", op="append", batch=4, heads=8, dim=128, page=64, type="f32", new=8192, past=0, rot=128,
             adjacent=False),
        # The smallest call: one token of one conversation, 32 query heads over 8 cached ones.
        dict(name="attend one token", op="attention", batch=1, q_heads=32, heads=8, dim=128, page=16, type="f32", new=1, len=777,
             rot=128, window=0),
        # One decode step of a full server: 64 sequences of up to 8192 tokens, the 70B-class layer's 64 query heads.
        dict(name="attend batch 64", op="attention", batch=64, q_heads=64, heads=8, dim=128, page=64, type="f32", new=1, len=8192,
             rot=128, window=0),
        # One token over one very long document, fp16.
        dict(name="attend long context", op="attention", batch=1, q_heads=32, heads=8, dim=128, page=64, type="f16", new=1,
             len=131071, rot=0, window=0),
        # Short ragged prompts of a small model: as many cached heads as query heads, 64 wide, a sliding window.
        dict(name="attend ragged prompts", op="attention", batch=7, q_heads=16, heads=16, dim=64, page=32, type="bf16", new=600,
             len=1500, rot=64, window=512),
        # A chunk of a long prompt of the 70B-class layer: 2048 new tokens over 8192 cached.
        dict(name="attend prompt chunk", op="attention", batch=1, q_heads=64, heads=8, dim=128, page=64, type="f32", new=2048,
             len=8192, rot=128, window=0),
        # The smallest call: the next token's candidates for one sequence.
        dict(name="logprobs one row", op="logprobs", rows=1, vocab=32768, type="f32", top=20, given=1),
        # One decode step of 64 sequences over a large odd vocabulary, few alternatives.
        dict(name="logprobs step 64", op="logprobs", rows=64, vocab=131073, type="f32", top=5, given=1),
        # A prompt's tokens scored at once from 16-bit logits.
        dict(name="logprobs prompt", op="logprobs", rows=4096, vocab=50001, type="bf16", top=8, given=1),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "attention", "logprobs"])
    kind = rng.choice(["f32", "f16", "bf16"])
    if op == "logprobs":
        vocab = _log(rng, 1000, 160000)
        rows = _log(rng, 1, max(1, min(4096, 200_000_000 // vocab)))
        return dict(op=op, rows=rows, vocab=vocab, type=kind, top=rng.choice([0, 1, 5, 8, 20, 32]), given=rng.choice([1, 1, 4]))
    dim = rng.choice([64, 96, 128, 128, 192, 256])
    heads = rng.choice([1, 2, 4, 8, 8, 16])
    rot = rng.choice([0, dim // 2, dim])
    page = rng.choice([16, 32, 64, 128])
    if op == "append":
        if rng.random() < 0.5:
            batch, new = _log(rng, 1, 256), 1
        else:
            batch = _log(rng, 1, 16)
            new = _log(rng, 2, 16384 // batch)
        return dict(op=op, batch=batch, heads=heads, dim=dim, page=page, type=kind, new=new, past=rng.choice([0, rng.randint(1, 3000)]),
                    rot=rot, adjacent=rng.random() < 0.5)
    q_heads = heads * rng.choice([1, 2, 4, 8]) if heads > 1 else rng.choice([1, 8, 12, 16])
    if rng.random() < 0.5:  # decode, a few tokens of each sequence
        batch, new = _log(rng, 1, 64), rng.choice([1, 1, 1, 4])
        length = _log(rng, 64, min(131072, 8192 * 64 * 8 * 128 // (batch * heads * dim)))
        length = max(length, new)
    else:
        batch = _log(rng, 1, 8)
        new = _log(rng, 16, 2048 // batch)
        length = new + rng.choice([0, rng.randint(1, 6000 // batch)])
    return dict(op=op, batch=batch, q_heads=q_heads, heads=heads, dim=dim, page=page, type=kind, new=new, len=length, rot=rot,
                window=rng.choice([0, 0, rng.randint(1, length)]))


# ---------------------------------------------------------------- sizes of a case
def _spread(n, lo, hi):
    """n whole numbers spread over lo .. hi, the first one hi."""
    return [hi - int((hi - lo + 1) * ((0.6180339887 * i) % 1.0)) for i in range(n)]


def _sizes(c):
    """(new tokens, tokens cached after them) of each sequence."""
    new = _spread(c["batch"], max(1, c["new"] // 4), c["new"])
    if c["op"] == "append":
        return new, [n + p for n, p in zip(new, _spread(c["batch"], c["past"] // 8, c["past"]))]
    return new, [max(n, m) for n, m in zip(new, _spread(c["batch"], max(1, c["len"] // 8), c["len"]))]


def _pairs(new, total, window):
    """Pairs of a query and a key that it sees."""
    seen = 0
    for n, m in zip(new, total):
        past = m - n
        if not window or window >= m:
            seen += n * past + n * (n + 1) // 2
        else:
            seen += sum(min(past + i + 1, window) for i in range(n))
    return seen


def work(c):
    if c["op"] == "logprobs":
        n = c["rows"] * c["vocab"]
        return {"bytes": n * SIZE[c["type"]] + c["rows"] * (8 + 8 * c["given"] + 8 * c["top"]), "flops": 5 * n}
    new, total = _sizes(c)
    rows, head = sum(new), c["heads"] * c["dim"]
    if c["op"] == "append":
        # the new rows in, the touched pages' codes out of the append and into the read, their values out of it
        pages = sum((m - 1) // c["page"] - (m - n) // c["page"] + 1 for n, m in zip(new, total))
        held = 2 * pages * c["page"] * head
        return {"bytes": 2 * rows * head * SIZE[c["type"]] + 4 * rows * c["rot"] + 2 * rows * head + held + held * SIZE[c["type"]]
                + 16 * pages * c["heads"], "flops": 2 * rows * head * 6}
    if c["window"]:
        seen = sum(min(m, n + c["window"] - 1) for n, m in zip(new, total))
    else:
        seen = sum(total)
    q = rows * c["q_heads"] * c["dim"]
    pairs = _pairs(new, total, c["window"])
    return {"bytes": 2 * seen * head + 8 * c["heads"] * (seen // c["page"] + 1) + 2 * q * SIZE[c["type"]] + 4 * rows * c["rot"]
            + 4 * rows * c["q_heads"], "flops": 4 * pairs * c["q_heads"] * c["dim"]}


# ---------------------------------------------------------------- inputs
def _rope_table(rows, rot):
    """cos and sin of position x frequency, [rows][rot / 2][2], base 10000."""
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    a = torch.arange(rows, dtype=torch.float64, device="cuda")[:, None] * f
    return torch.stack((a.cos(), a.sin()), -1).float().contiguous()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    c = case
    kind = DTYPE[c["type"]]
    if c["op"] == "logprobs":
        # logits of a trained head: a wide bulk, a few tokens that stand out, some that a grammar forbids
        x = rand(c["rows"], c["vocab"]).mul_(2.0)
        peak = torch.randint(0, c["vocab"], (c["rows"], 8), generator=g, device="cuda")
        x.scatter_add_(1, peak, rand(c["rows"], 8).abs_().mul_(6.0))
        off = torch.randint(0, c["vocab"], (c["rows"], max(1, c["vocab"] // 64)), generator=g, device="cuda")
        x.scatter_(1, off, float("-inf"))
        given = peak[:, : c["given"]].to(torch.int32).contiguous()
        out = lambda n, t: torch.empty(c["rows"], n, dtype=t, device="cuda")  # noqa: E731
        return dict(case=c, logits=x.to(kind), given=given, lse=out(1, torch.float32).view(-1), entropy=out(1, torch.float32).view(-1),
                    given_logp=out(c["given"], torch.float32), top_ids=out(c["top"], torch.int32), top_logp=out(c["top"], torch.float32))
    new, total = _sizes(c)
    page, heads, dim, batch = c["page"], c["heads"], c["dim"], c["batch"]
    per = [-(-m // page) for m in total]
    most = max(per)
    pages = sum(per) + 3
    ids = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    # a page table's unused entries hold no page
    used = torch.arange(most)[None, :] < torch.tensor(per)[:, None]
    table = torch.full((batch, most), -1, dtype=torch.int32, device="cuda")
    table[used.cuda()] = ids[: sum(per)]
    first = torch.tensor([0] + new).cumsum(0).to(torch.int32)
    s = dict(case=c, table=table, first=first.cuda(), length=torch.tensor(total, dtype=torch.int32, device="cuda"))
    # codes and scales as an append leaves them: values of a few units, each block's largest at 127
    s["k"] = rand(pages, heads, page, dim).mul_(40.0).round_().clamp_(-127, 127).to(torch.int8)
    s["v"] = rand(pages, heads, page, dim).mul_(40.0).round_().clamp_(-127, 127).to(torch.int8)
    s["k_scale"] = rand(pages, heads).mul_(0.2).exp_().mul_(3.2 / 127)
    s["v_scale"] = rand(pages, heads).mul_(0.2).exp_().mul_(3.2 / 127)
    s["rope"] = _rope_table(most * page, c["rot"]) if c["rot"] else None
    rows = sum(new)
    # what a scheduler knows of its rows: the sequence, the position
    n = torch.tensor(new)
    s["seq"] = torch.repeat_interleave(torch.arange(batch), n).cuda()
    s["pos"] = (torch.arange(rows) - torch.repeat_interleave(first[:-1].long() - (torch.tensor(total) - n), n)).cuda()
    if c["op"] == "append":
        s["key"] = rand(rows, heads, dim).to(kind)
        s["value"] = rand(rows, heads, dim).to(kind)
        at = torch.arange(most)[None, :]
        lo, hi = (torch.tensor(total) - n) // page, (torch.tensor(total) - 1) // page
        touched = (at >= lo[:, None]) & (at <= hi[:, None])
        s["pages"] = table[touched.cuda()].contiguous()
        s["key_out"] = torch.empty(s["pages"].numel(), heads, page, dim, dtype=kind, device="cuda")
        s["value_out"] = torch.empty_like(s["key_out"])
    else:
        s["q"] = rand(rows, c["q_heads"], dim).to(kind)
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(rows, c["q_heads"], dtype=torch.float32, device="cuda")
        s["new"], s["most"] = max(new), max(total)
    return s


# ---------------------------------------------------------------- the plain forms
def _rotated(x, pos, table, adjacent):
    """x [rows][heads][dim] with its first pairs turned by the table's rows at `pos`, in x's own precision."""
    if table is None:
        return x
    half = table.shape[1]
    cs = table[pos].to(x.dtype)[:, None]
    cos, sin = cs[..., 0], cs[..., 1]
    if adjacent:
        a, b = x[..., 0 : 2 * half : 2], x[..., 1 : 2 * half : 2]
        turned = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half : 2 * half]
        turned = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
    return torch.cat((turned, x[..., 2 * half :]), -1)


def _plain_append(x, codes, scale, pages, block, slot, fresh):
    """x [rows][heads][dim] into `slot` of the touched blocks `block` of codes[pages] [heads][page][dim], in place: a block's
    scale grows with its largest value, and the codes that it already held are rounded to the new scale."""
    held, old = codes[pages].float(), scale[pages]
    old = torch.where(fresh[:, None], torch.zeros_like(old), old)
    most = torch.zeros_like(old).index_reduce_(0, block, x.abs().amax(-1), "amax")
    d = torch.maximum(old, most / torch.full_like(most, 127.0))
    ratio = torch.where((d > old) & (old > 0), old / d, torch.ones_like(d))
    held = held * ratio[:, :, None, None]
    held = held.sign() * (held.abs() + 0.5).floor()
    inverse = torch.where(d > 0, torch.ones_like(d) / d, torch.zeros_like(d))
    y = x * inverse[block][:, :, None]
    held[block, :, slot] = (y.sign() * (y.abs() + 0.5).floor()).clamp(-127, 127)
    codes[pages] = held.to(torch.int8)
    scale[pages] = d


def _plain_attention(s, wide):
    """Softmax of the scaled products over the keys that each row sees, by padded sequences, in `wide`'s precision."""
    c = s["case"]
    page, heads, dim, group = c["page"], c["heads"], c["dim"], c["q_heads"] // c["heads"]
    table = s["table"].long().clamp(min=0)
    gather = lambda codes, scale: (codes[table].to(wide) * scale[table].to(wide)[..., None, None]).permute(0, 2, 1, 3, 4).flatten(2, 3)  # noqa: E731
    key, value = gather(s["k"], s["k_scale"]), gather(s["v"], s["v_scale"])  # [batch][heads][tokens][dim]
    q = _rotated(s["q"].to(wide), s["pos"], s["rope"], False)
    row = torch.arange(q.shape[0], device="cuda") - s["first"].long()[s["seq"]]
    padded = torch.zeros(c["batch"], s["new"], heads, group, dim, dtype=wide, device="cuda")
    padded[s["seq"], row] = q.view(-1, heads, group, dim)
    at = torch.full((c["batch"], s["new"]), -1, dtype=torch.long, device="cuda")
    at[s["seq"], row] = s["pos"]
    token = torch.arange(key.shape[2], device="cuda")
    sees = token <= at[..., None]
    if c["window"]:
        sees &= token > at[..., None] - c["window"]
    x = torch.matmul(padded.permute(0, 2, 3, 1, 4).flatten(2, 3), key.transpose(2, 3)) * dim ** -0.5
    x = x.view(c["batch"], heads, group, s["new"], -1).masked_fill(~sees[:, None, None], float("-inf"))
    top = x.amax(-1, keepdim=True).clamp(min=-1e30)
    p = (x - top).exp()
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p.flatten(2, 3), value).view(c["batch"], heads, group, s["new"], dim) / total.clamp(min=1e-30)
    lse = (total.log() + top).squeeze(-1)
    out = out.permute(0, 3, 1, 2, 4)[s["seq"], row].flatten(1, 2)
    return {"out": out, "lse": lse.permute(0, 3, 1, 2)[s["seq"], row].flatten(1, 2)}


def _ordered(x):
    """Whole numbers in the order of x's values."""
    i = (x + 0.0).view(torch.int32)
    return i ^ ((i >> 31) & 0x7FFFFFFF)


def _plain_logprobs(s):
    c = s["case"]
    x = s["logits"].float()
    top = x.amax(1, keepdim=True)
    lse = (x - top).exp().sum(1, keepdim=True).log() + top
    logp = x - lse
    p = logp.exp()
    entropy = -torch.where(p > 0, p * logp, torch.zeros_like(p)).sum(1)
    out = {"lse": lse[:, 0], "entropy": entropy, "given_logp": logp.gather(1, s["given"].long())}
    if c["top"]:
        place = 2**32 - 1 - torch.arange(x.shape[1], device="cuda")
        key = (_ordered(x).long() << 32) + place  # equal values: the lower index first
        ids = key.topk(c["top"], 1).indices
        out |= {"top_ids": ids.to(torch.int32), "top_logp": logp.gather(1, ids)}
    return out


def _run_plain(s):
    c = s["case"]
    kind = DTYPE[c["type"]]
    if c["op"] == "logprobs":
        return _plain_logprobs(s)
    if c["op"] == "attention":
        r = _plain_attention(s, torch.float32)
        return {"out": r["out"].to(kind), "lse": r["lse"]}
    pages = s["pages"].long()
    place = torch.empty(s["k"].shape[0], dtype=torch.long, device="cuda")
    place[pages] = torch.arange(pages.numel(), device="cuda")
    block = place[s["table"].long()[s["seq"], s["pos"] // c["page"]]]
    slot = s["pos"] % c["page"]
    # a page that this call fills from its first slot on keeps nothing of what was there
    fresh = torch.full_like(pages, c["page"]).index_reduce_(0, block, slot, "amin") == 0
    _plain_append(_rotated(s["key"].float(), s["pos"], s["rope"], c["adjacent"]), s["k"], s["k_scale"], pages, block, slot, fresh)
    _plain_append(s["value"].float(), s["v"], s["v_scale"], pages, block, slot, fresh)
    back = lambda codes, scale: (codes[pages].float() * scale[pages][..., None, None]).to(kind)  # noqa: E731
    return {"key": back(s["k"], s["k_scale"]), "value": back(s["v"], s["v_scale"])}


# ---------------------------------------------------------------- the package's entry points
def _run_own(s):
    import block_quantized_matmul_q4_gb300 as q

    c = s["case"]
    if c["op"] == "logprobs":
        q.qmm_logprobs(s["logits"], s["given"], s["lse"], s["entropy"], s["given_logp"], s["top_ids"], s["top_logp"])
        out = {"lse": s["lse"], "entropy": s["entropy"], "given_logp": s["given_logp"]}
        return out | {"top_ids": s["top_ids"], "top_logp": s["top_logp"]} if c["top"] else out
    cache = q.KvCache(s["k"], s["v"], s["k_scale"], s["v_scale"])
    batch = q.KvBatch(s["table"], s["first"], s["length"])
    if c["op"] == "attention":
        rope = q.Rope(s["rope"]) if c["rot"] else None
        q.qmm_kv_attention(cache, batch, rope, s["q"], s["out"], s["lse"], scale=c["dim"] ** -0.5, window=c["window"],
                           max_q=s["new"], max_kv=s["most"])
        return {"out": s["out"], "lse": s["lse"]}
    rope = q.Rope(s["rope"], adjacent=c["adjacent"]) if c["rot"] else None
    q.qmm_kv_append(cache, batch, rope, s["key"], s["value"])
    q.qmm_kv_read(cache, s["pages"], s["key_out"], s["value_out"])
    return {"key": s["key_out"], "value": s["value_out"]}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---------------------------------------------------------------- the definition in 64 bits
def _turn64(x, pos, table, adjacent):
    """Each pair (a, b) as the complex number a + ib, times cos + i sin."""
    if table is None:
        return x
    n = table.shape[1]
    w = torch.complex(table[pos, :, 0].double(), table[pos, :, 1].double())[:, None]
    y = x.clone()
    i = torch.arange(n, device=x.device)
    ia, ib = (2 * i, 2 * i + 1) if adjacent else (i, i + n)
    z = torch.complex(x[..., ia], x[..., ib]) * w
    y[..., ia], y[..., ib] = z.real, z.imag
    return y


def exact(case, seed):
    s = prepare(case, seed)
    c = case
    if c["op"] == "logprobs":
        n = c["rows"]
        out = {"lse": torch.empty(n, dtype=torch.float64), "entropy": torch.empty(n, dtype=torch.float64),
               "given_logp": torch.empty(n, c["given"], dtype=torch.float64)}
        if c["top"]:
            out |= {"top_ids": None, "top_logp": torch.empty(n, c["top"], dtype=torch.float64)}
        for r in range(0, n, 64):
            x = s["logits"][r : r + 64].double()
            lse = torch.logsumexp(x, 1)
            lp = x - lse[:, None]
            out["lse"][r : r + 64] = lse.cpu()
            out["entropy"][r : r + 64] = -torch.nan_to_num(lp.exp() * lp, nan=0.0).sum(1).cpu()
            out["given_logp"][r : r + 64] = lp.gather(1, s["given"][r : r + 64].long()).cpu()
            if c["top"]:
                out["top_logp"][r : r + 64] = lp.topk(c["top"], 1).values.cpu()
        return out
    new, total = _sizes(c)
    page, heads, dim = c["page"], c["heads"], c["dim"]
    table = s["table"].cpu().tolist()
    if c["op"] == "attention":
        group = c["q_heads"] // heads
        q = _turn64(s["q"].double(), s["pos"], s["rope"], False)
        out = torch.empty(q.shape, dtype=torch.float64)
        lse = torch.empty(q.shape[:2], dtype=torch.float64)
        if _pairs(new, total, 0) * c["q_heads"] * dim > 2e12:
            return None
        row = 0
        for b, (n, m) in enumerate(zip(new, total)):
            ids = torch.tensor(table[b][: -(-m // page)], device="cuda")
            pos = torch.arange(m - n, m, device="cuda")[:, None]
            t = torch.arange(m, device="cuda")[None]
            hidden = t > pos
            if c["window"]:
                hidden |= t <= pos - c["window"]
            for h in range(heads):
                k = (s["k"][ids, h].double() * s["k_scale"][ids, h].double()[:, None, None]).reshape(-1, dim)[:m]
                v = (s["v"][ids, h].double() * s["v_scale"][ids, h].double()[:, None, None]).reshape(-1, dim)[:m]
                for j in range(h * group, h * group + group):
                    x = (q[row : row + n, j] @ k.T / math.sqrt(dim)).masked_fill(hidden, float("-inf"))
                    out[row : row + n, j] = (torch.softmax(x, 1) @ v).cpu()
                    lse[row : row + n, j] = torch.logsumexp(x, 1).cpu()
            row += n
        return {"out": out, "lse": lse}
    result = {}
    for name, codes, scale, x in (("key", s["k"], s["k_scale"], _turn64(s["key"].double(), s["pos"], s["rope"], c["adjacent"])),
                                  ("value", s["v"], s["v_scale"], s["value"].double())):
        blocks, row = [], 0
        for b, (n, m) in enumerate(zip(new, total)):
            for i in range((m - n) // page, (m - 1) // page + 1):
                p = table[b][i]
                lo, hi = max(0, m - n - i * page), min(page, m - i * page)  # the slots that are new
                fresh = x[row : row + hi - lo].transpose(0, 1)  # [heads][slots][dim]
                row += hi - lo
                d0 = scale[p].double() if lo else torch.zeros(heads, dtype=torch.float64, device="cuda")
                d = torch.maximum(d0, fresh.abs().amax((1, 2)) / 127)[:, None, None]
                held = codes[p].double()
                grown = d > d0[:, None, None]
                held = torch.where(grown & (d0[:, None, None] > 0), torch.round(held * (d0[:, None, None] / d)), held)
                held[:, lo:hi] = torch.round(fresh / d).clamp(-127, 127)
                blocks.append(held * d)
        result[name] = torch.stack(blocks)
    return result
