"""qmm_kv_attention on the GPU against 64-bit attention over the cache's values.

Bound for each output (derived). Let e be the largest error of a score in
nats: q as two fp16 numbers (2^-22 relative), fp32 accumulation over the head
(at most 256 products) and the fp32 products with the scales, together less
than 2^-18 of scale * sum |q| |k|, plus 2^-22 of the score in log2 units (at
most twice that sum again). Probabilities are then off by 2 e relative, by
the exponential (2^-21) and by their own rounding: 2^-21 as two fp16 numbers,
2^-11 as one (fp16 and bf16 calls that are no decode step). Sums over n
tokens in fp32 add n 2^-24. So |out - exact| <= (2 e + 2^-19 + n 2^-24 [+
2^-11]) sum p |v| + the rounding to the output's type. lse: e + 2^-20 + 2^-22
|lse|."""
import math

import numpy as np
import pytest
import torch

from serving_ref import attend, rope_table, rotate
from test_gpu_kv_cache import TYPES, Case, q  # noqa: F401

pytestmark = pytest.mark.gpu
EPS = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}


def values(c):
    return [codes.astype(np.float64) * s[..., None, None].astype(np.float64) for codes, s in zip(c.codes, c.scales)]


def call(q, c, x, rope=None, **kw):
    out = torch.full_like(x, float("nan"), memory_format=torch.contiguous_format)
    lse = torch.full(x.shape[:2], float("nan"), device="cuda")
    kw = {"scale": c.dim ** -0.5, "max_q": max(n for n, _ in c.seqs), "max_kv": max(m for _, m in c.seqs)} | kw
    q.qmm_kv_attention(c.cache, c.batch, rope, x, out, lse, **kw)
    q.qmm_check_device_error()
    return out, lse


def check(c, x, kind, out, lse, rows=None, table=None, adjacent=False, causal=True, window=0, scale=None):
    """Every row in `rows` (default: all) of every head."""
    scale = c.dim ** -0.5 if scale is None else scale
    key, value = values(c)
    x64, out64, lse64 = x.double().cpu().numpy(), out.double().cpu().numpy(), lse.double().cpu().numpy()
    group = x.size(1) // c.heads
    for b, (n, m) in enumerate(c.seqs):
        pages = c.table[b, :-(-m // c.page)]
        k, v = (a[pages].transpose(0, 2, 1, 3).reshape(-1, c.heads, c.dim)[:m] for a in (key, value))
        for i in range(n):
            r = c.first[b] + i
            if rows is not None and r not in rows:
                continue
            for j in range(x.size(1)):
                qr = rotate(x64[r, j], m - n + i, table, adjacent)
                o, ls, size, xs = attend(qr, k[:, j // group], v[:, j // group], m - n + i, scale, causal, window)
                e = 2.0 ** -18 * xs + 2.0 ** -21 * xs
                rel = 2 * e + 2.0 ** -19 + m * 2.0 ** -24 + (0 if kind == "f32" else 2.0 ** -11)
                err = np.abs(out64[r, j] - o)
                assert np.all(err <= rel * size + EPS[kind] * np.abs(o) + 1e-30), (b, i, j, (err / (rel * size + EPS[kind] * np.abs(o))).max())
                assert abs(lse64[r, j] - ls) <= e + 2.0 ** -20 + 2.0 ** -22 * abs(ls), (b, i, j, lse64[r, j], ls)


def inputs(c, q_heads, kind, seed=1, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(c.rows, q_heads, c.dim, generator=g) * scale).to(TYPES[kind]).cuda()


DECODE = [(1, 1), (1, 15), (1, 16), (1, 17), (0, 5), (1, 63), (1, 64), (1, 65), (1, 200), (1, 777)]


@pytest.mark.parametrize("heads,group,page,dim,kind,rot", [
    (2, 4, 16, 128, "f32", 128), (1, 1, 32, 64, "f16", 0), (3, 8, 64, 128, "bf16", 64), (2, 16, 16, 64, "f32", 64), (1, 12, 128, 128, "f16", 128),
    (2, 2, 64, 96, "f32", 48), (1, 8, 16, 192, "bf16", 0), (1, 3, 32, 256, "f32", 256), (1, 32, 16, 96, "f16", 96), (1, 20, 128, 256, "f32", 8)])
def test_decode(q, heads, group, page, dim, kind, rot):  # noqa: F811
    c = Case(q, DECODE, heads, page, dim, seed=group)
    x = inputs(c, heads * group, kind)
    table = rope_table(c.most * page, rot) if rot else None
    out, lse = call(q, c, x, q.Rope(torch.from_numpy(table).cuda()) if rot else None)
    check(c, x, kind, out, lse, table=table)


@pytest.mark.parametrize("heads,group,page,dim,kind,window,causal", [
    (2, 4, 16, 64, "f32", 0, True), (1, 8, 64, 128, "f16", 0, True), (2, 1, 32, 64, "bf16", 100, True), (1, 2, 16, 128, "f32", 1, True),
    (2, 2, 64, 96, "f32", 33, True), (1, 4, 32, 256, "bf16", 0, True), (1, 3, 16, 192, "f16", 64, True), (2, 2, 32, 128, "f32", 0, False),
    (1, 4, 128, 64, "f16", 0, False), (1, 5, 128, 128, "bf16", 200, True)])
def test_prompts(q, heads, group, page, dim, kind, window, causal):  # noqa: F811
    seqs = [(1, 1), (1, 70), (2, 33), (0, 40), (130, 130), (65, 300), (17, 17), (200, 257)]
    c = Case(q, seqs, heads, page, dim, seed=group + page)
    x = inputs(c, heads * group, kind)
    out, lse = call(q, c, x, window=window, causal=causal)
    assert not out.isnan().any() and not lse.isnan().any()
    rows = set(range(0, c.rows, 7)) | {int(f) for f in c.first[:-1]} | {int(f) - 1 for f in c.first[1:]}
    check(c, x, kind, out, lse, rows=rows, window=window, causal=causal)


def test_hints_do_not_change_results(q):  # noqa: F811
    """max_q and max_kv that are wrong either way give the same rows within the bounds."""
    c = Case(q, [(1, 700), (9, 90), (40, 41)], 2, 16, 64, seed=2)
    x = inputs(c, 4, "f32")
    for max_q, max_kv in ((1, 1), (40, 700), (1, 100000), (1000, 64), (0, 0)):
        out, lse = call(q, c, x, max_q=max_q, max_kv=max_kv)
        check(c, x, "f32", out, lse)


@pytest.mark.parametrize("adjacent", [False, True])
def test_rotation(q, adjacent):  # noqa: F811
    c = Case(q, [(3, 50), (1, 9)], 2, 16, 96, seed=4)
    table = rope_table(c.most * 16, 48)
    x = inputs(c, 4, "f16")
    out, lse = call(q, c, x, q.Rope(torch.from_numpy(table).cuda(), adjacent=adjacent))
    check(c, x, "f16", out, lse, table=table, adjacent=adjacent)


def test_strided_rows(q):  # noqa: F811
    c = Case(q, [(3, 50), (1, 9)], 2, 16, 64, seed=4)
    wide = torch.full((c.rows, 9, 64), float("nan"), device="cuda")
    wide[:, 2:6] = inputs(c, 4, "f32")
    out, lse = call(q, c, wide[:, 2:6])
    check(c, wide[:, 2:6], "f32", out, lse)


@pytest.mark.parametrize("size", [1e-30, 1e-3, 300.0, 1e30])
def test_sizes_of_q(q, size):  # noqa: F811
    """Any magnitude of q that fp32 holds: the power of two per row comes off again."""
    c = Case(q, [(1, 300), (20, 40)], 1, 16, 64, seed=5)
    x = inputs(c, 2, "f32", scale=size)
    scale = 0.125 / size
    out, lse = call(q, c, x, scale=scale)
    check(c, x, "f32", out, lse, scale=scale)


def test_page_scales_far_apart(q):  # noqa: F811
    """Values of one page 10^12 times another's, pages of zeros, and scores that
    concentrate on the small ones."""
    c = Case(q, [(1, 90), (33, 90)], 1, 16, 64, seed=6)
    for b in range(2):
        c.scales[1][c.table[b, 1]] *= 1e-12
        c.scales[1][c.table[b, 2]] *= 1e6
        c.codes[1][c.table[b, 3]] = 0
        c.scales[1][c.table[b, 3]] = 0
        c.codes[0][c.table[b, 4]] = 0
        c.scales[0][c.table[b, 4]] = 0
    for t, a in zip(c.dev_codes + c.dev_scales, c.codes + c.scales):
        t.copy_(torch.from_numpy(a))
    x = inputs(c, 4, "f32", scale=2.0)
    out, lse = call(q, c, x)
    check(c, x, "f32", out, lse)


@pytest.mark.parametrize("n", [1, 40])
def test_what_no_row_sees_does_not_count(q, n):  # noqa: F811
    """Codes past a sequence's end, pages after it and poisoned pages outside
    the window leave no trace; a poisoned page inside it makes its head NaN."""
    c = Case(q, [(n, 100)], 2, 16, 64, seed=7)
    x = inputs(c, 4, "f32")
    want = call(q, c, x, window=20)
    c.dev_codes[0][c.table[0, 6], :, 4:] = 127
    c.dev_codes[1][c.table[0, 6], :, 4:] = -128
    first = (100 - n - 19) // 16  # the page of the first token that any row sees
    for i in range(first):
        for s in c.dev_scales:
            s[c.table[0, i]] = float("inf")
    got = call(q, c, x, window=20)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    c.dev_scales[1][c.table[0, 6], 1] = float("inf")
    out, _ = call(q, c, x, window=20)
    assert out[-1, 2:].isnan().all() and out[-1, :2].isfinite().all()
    # rows that do not reach the page are not touched by it
    if n > 20:
        assert torch.equal(out[:n - 20], want[0][:n - 20])


def test_missing_pages_are_reported(q):  # noqa: F811
    c = Case(q, [(1, 40), (1, 50)], 1, 16, 64, seed=8)
    x = inputs(c, 2, "f32")
    c.batch.tensors[0][1, 1] = 10 ** 6
    out = torch.full_like(x, 3.0)
    q.qmm_kv_attention(c.cache, c.batch, None, x, out, scale=0.125, max_q=1, max_kv=50)
    with pytest.raises(q.QmmError, match="outside"):
        q.qmm_check_device_error()
    lse = torch.empty(2, 2, device="cuda")
    c.seqs = c.seqs[:1]
    q.qmm_kv_attention(c.cache, c.batch, None, x, out, lse, scale=0.125, max_q=1, max_kv=50)
    check(c, x, "f32", out, lse)
    with pytest.raises(q.QmmError):
        q.qmm_check_device_error()


def test_callers_workspace_and_graph(q):  # noqa: F811
    """With a caller's workspace the call allocates nothing, so it can be captured; a replay sees new data."""
    c = Case(q, [(1, 500), (1, 900)], 2, 16, 128, seed=9)
    x = inputs(c, 8, "f32")
    want, want_lse = call(q, c, x)
    need = q.qmm_kv_attention_workspace_bytes(c.cache, 2, 8, 2, 1, 900)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    out, lse = torch.empty_like(x), torch.empty(2, 8, device="cuda")
    kw = dict(scale=128 ** -0.5, max_q=1, max_kv=900, workspace=ws, ws_bytes=need)
    q.qmm_kv_attention(c.cache, c.batch, None, x, out, lse, **kw)
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q.qmm_kv_attention(c.cache, c.batch, None, x, out, lse, **kw)
    x.copy_(inputs(c, 8, "f32", seed=2))
    graph.replay()
    torch.cuda.synchronize()
    check(c, x, "f32", out, lse)
    if need > 16:
        with pytest.raises(q.QmmError, match="workspace"):
            q.qmm_kv_attention(c.cache, c.batch, None, x, out, lse, **(kw | {"ws_bytes": 16}))


def test_cache_past_32_bit_offsets(q):  # noqa: F811
    """Pages beyond 2^32 bytes of codes and 2^31 elements."""
    pages = (1 << 32) // (8 * 64 * 128) + 40
    c = Case(q, [(1, 300), (70, 300)], 8, 64, 128, seed=10)
    big = [torch.zeros(pages, 8, 64, 128, dtype=torch.int8, device="cuda") for _ in range(2)]
    bs = [torch.zeros(pages, 8, device="cuda") for _ in range(2)]
    shift = pages - len(c.codes[0])
    for t, a in zip(big + bs, c.codes + c.scales):
        t[shift:] = torch.from_numpy(a).cuda()
    table = c.batch.tensors[0].clone()
    table[table >= 0] += shift
    small = call(q, c, inputs(c, 8, "f32"))
    c.cache = q.KvCache(*big, *bs)
    c.batch = q.KvBatch(table, *c.batch.tensors[1:])
    large = call(q, c, inputs(c, 8, "f32"))
    assert torch.equal(small[0], large[0]) and torch.equal(small[1], large[1])
    # and an append there reads back
    q.qmm_kv_append(c.cache, c.batch, None, *c.dev_x)
    k = torch.empty(1, 8, 64, 128, device="cuda")
    last = int(c.table[1, 4]) + shift
    q.qmm_kv_read(c.cache, torch.tensor([last], dtype=torch.int32, device="cuda"), k, torch.empty_like(k))
    rows = 300 - 256
    got, want = k[0, :, :rows].cpu().numpy(), c.x[0][-rows:].transpose(1, 0, 2)
    d = bs[0][last].cpu().numpy()[:, None, None]
    assert np.all(np.abs(got - want) <= 0.51 * d) and math.isfinite(got.sum())


@pytest.mark.parametrize("dim,page,rot", [(192, 32, 192), (256, 64, 0), (96, 16, 32), (128, 32, 128)])
def test_prompts_of_fp32_heads(q, dim, page, rot):  # noqa: F811
    """Two fp16 numbers each for Q and the weights at every width, over more than one split's tokens."""
    c = Case(q, [(150, 1300), (40, 40), (1, 600), (90, 91)], 2, page, dim, seed=dim)
    x = inputs(c, 8, "f32")
    table = rope_table(c.most * page, rot) if rot else None
    out, lse = call(q, c, x, q.Rope(torch.from_numpy(table).cuda()) if rot else None)
    rows = set(range(0, c.rows, 17)) | {int(f) - 1 for f in c.first[1:]}
    check(c, x, "f32", out, lse, rows=rows, table=table)


@pytest.mark.parametrize("dim,kind,window", [(128, "f32", 0), (64, "f32", 0), (128, "f16", 0), (64, "bf16", 500), (192, "f32", 0), (256, "bf16", 0)])
def test_long_prompts_agree_with_decode(q, dim, kind, window):  # noqa: F811
    """Thousands of tiles on the prompts' kernels against every row on the single tokens' one.

    Both are within the bound of the exact result, so within two of each other, with sum p |v| at most
    the largest |v| and sum |q| |k| at most |q|_1 max |k|."""
    c = Case(q, [(700, 2500), (1300, 1300), (64, 5000), (3, 9), (0, 7), (500, 9000)], 2, 32, dim, seed=dim)
    x = inputs(c, 16, kind)
    key, value = values(c)
    xs = c.dim ** -0.5 * float(x.double().abs().sum(-1).max()) * float(np.abs(key).max())
    top = float(np.abs(value).max())
    e = (2.0 ** -18 + 2.0 ** -21) * xs
    rel = 2 * e + 2.0 ** -19 + 9000 * 2.0 ** -24 + (0 if kind == "f32" else 2.0 ** -11)
    a, la = call(q, c, x, window=window)
    for _ in range(3):
        again, lagain = call(q, c, x, window=window)
        assert torch.equal(a, again) and torch.equal(la, lagain)
    b, lb = call(q, c, x, window=window, max_q=1)
    a, b = a.double(), b.double()
    assert ((a - b).abs() <= 2 * (rel * top + EPS[kind] * (b.abs() + rel * top))).all()
    assert ((la - lb).abs() <= 2 * (e + 2.0 ** -20 + 2.0 ** -22 * lb.abs())).all()


@pytest.mark.parametrize("seqs,q_heads,dim,kind", [([(1, 5200)], 2, 64, "f32"), ([(1, 9000), (1, 300)], 4, 128, "f16"), ([(90, 5000), (1, 40)], 4, 64, "bf16"),
                                                   ([(70, 4100)], 2, 192, "f32")])
def test_nothing_is_written_past_the_workspace(q, seqs, q_heads, dim, kind):  # noqa: F811
    """Windows change how a call splits: whatever they are, it keeps to the size that was asked for."""
    c = Case(q, seqs, 2, 32, dim, seed=dim)
    x = inputs(c, q_heads, kind)
    max_q, max_kv = max(n for n, _ in seqs), max(m for _, m in seqs)
    need = q.qmm_kv_attention_workspace_bytes(c.cache, len(seqs), q_heads, c.rows, max_q, max_kv)
    rows = {0, c.rows // 2, c.rows - 1}
    for window in (0, 1, 100, 600, 1000, 1700, 2500, 3300, 4500):
        ws = torch.full((need + (1 << 20),), 0xAB, dtype=torch.uint8, device="cuda")
        out, lse = call(q, c, x, window=window, workspace=ws, ws_bytes=need)
        assert bool((ws[need:] == 0xAB).all()), window
        check(c, x, kind, out, lse, rows=rows, window=window)
