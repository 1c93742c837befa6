"""The paged 8-bit cache on the GPU: qmm_kv_append and qmm_kv_read against
64-bit forms of the definition in include/qmm.h.

Bounds (derived, not fitted). With d the block's scale: a new value x becomes
round(x / d) d, off by at most d / 2; fp32 rounding of the rotation, of 1 / d
and of the product moves x / d (at most 127) by less than 127 * 2^-20, which
may tip a rounding. A kept value q d_old is rounded once more: q d_old / d
within 127 * 2^-22 of the exact quotient. Scales: a maximum, one division and
the rotation's fp32 roundings, 2^-21 relative."""
import numpy as np
import pytest
import torch

from serving_ref import rope_table, rotate

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def q():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import block_quantized_matmul_q4_gb300 as q
    return q


class Case:
    """Sequences given as (new, total) pairs over a cache of random content."""

    def __init__(self, q, seqs, heads, page, dim, kind="f32", seed=0, scale=1.0, spare=3):
        self.rng = np.random.default_rng(seed)
        self.seqs, self.heads, self.page, self.dim = seqs, heads, page, dim
        per = [-(-m // page) for _, m in seqs]
        self.most = max(per + [1])
        pages = sum(per) + spare
        ids = self.rng.permutation(pages)
        self.table = np.full((len(seqs), self.most), -1, np.int32)
        at = 0
        for b, n in enumerate(per):
            self.table[b, :n] = ids[at:at + n]
            at += n
        self.rows = sum(n for n, _ in seqs)
        self.first = np.cumsum([0] + [n for n, _ in seqs]).astype(np.int32)
        shape = (pages, heads, page, dim)
        self.codes = [self.rng.integers(-127, 128, shape).astype(np.int8) for _ in range(2)]
        self.scales = [np.exp(self.rng.normal(0, 0.5, shape[:2])).astype(np.float32) * np.float32(0.02) for _ in range(2)]
        self.dev_codes = [torch.from_numpy(c.copy()).cuda() for c in self.codes]
        self.dev_scales = [torch.from_numpy(s.copy()).cuda() for s in self.scales]
        self.cache = q.KvCache(*self.dev_codes, *self.dev_scales)
        self.batch = q.KvBatch(torch.from_numpy(self.table).cuda(), torch.from_numpy(self.first).cuda(),
                               torch.tensor([m for _, m in seqs], dtype=torch.int32, device="cuda"))
        x = [torch.from_numpy(self.rng.normal(0, scale, (self.rows, heads, dim))).to(TYPES[kind]) for _ in range(2)]
        self.x = [t.double().numpy() for t in x]
        self.dev_x = [t.cuda() for t in x]

    def blocks(self):
        """(page id, kept slots, new rows of x, their positions) of every touched page."""
        for b, (n, m) in enumerate(self.seqs):
            start = m - n
            for i in range(start // self.page, -(-m // self.page)):
                lo, hi = max(start, i * self.page), min(m, (i + 1) * self.page)
                if lo < hi:
                    r0 = self.first[b] + lo - start
                    yield self.table[b, i], lo - i * self.page, range(r0, r0 + hi - lo), range(lo, hi)


def check_append(c, table=None, adjacent=False):
    got_codes = [t.cpu().numpy() for t in c.dev_codes]
    got_scales = [t.cpu().numpy() for t in c.dev_scales]
    touched = set()
    for side in range(2):
        for page, kept, rows, positions in c.blocks():
            touched.add(int(page))
            for h in range(c.heads):
                x = np.stack([rotate(c.x[side][r, h], p, table if side == 0 else None, adjacent) for r, p in zip(rows, positions)])
                old = float(c.scales[side][page, h]) if kept else 0.0
                want = max(old, np.abs(x).max() / 127.0)
                d = float(got_scales[side][page, h])
                assert abs(d - want) <= 2.0 ** -21 * want
                codes = got_codes[side][page, h].astype(np.float64)
                assert np.abs(codes).max() <= 127
                err = np.abs(codes[kept:kept + len(rows)] * d - x)
                assert np.all(err <= d * (0.5 + 127 * 2.0 ** -20)), f"page {page} head {h}: {err.max() / d}"
                before = c.codes[side][page, h]
                other = np.r_[:kept, kept + len(rows):c.page]  # slots that are not new
                if d == old or kept == 0:
                    assert np.array_equal(got_codes[side][page, h, other], before[other])
                else:
                    err = np.abs(codes[other] - before[other].astype(np.float64) * (old / d))
                    assert np.all(err <= 0.5 + 127 * 2.0 ** -22)
        rest = [p for p in range(len(c.codes[side])) if p not in touched]
        assert np.array_equal(got_codes[side][rest], c.codes[side][rest])
        assert np.array_equal(got_scales[side][rest], c.scales[side][rest])


SEQS = [(1, 1), (1, 16), (0, 9), (1, 130), (5, 5), (37, 40), (3, 130), (200, 333), (2, 129)]


@pytest.mark.parametrize("heads,page,dim,kind,rot,adjacent", [
    (1, 16, 64, "f32", 64, False), (3, 32, 128, "f16", 128, True), (8, 64, 128, "bf16", 64, False), (2, 128, 256, "f32", 256, False),
    (5, 16, 96, "bf16", 48, True), (2, 64, 192, "f16", 0, False), (1, 128, 96, "f32", 8, False)])
def test_append(q, heads, page, dim, kind, rot, adjacent):
    c = Case(q, SEQS, heads, page, dim, kind, seed=dim + page)
    table = rope_table(c.most * page, rot) if rot else None
    rope = q.Rope(torch.from_numpy(table).cuda(), adjacent=adjacent) if rot else None
    q.qmm_kv_append(c.cache, c.batch, rope, *c.dev_x)
    q.qmm_check_device_error()
    check_append(c, table, adjacent)
    # the same rows again change nothing: every scale already covers them
    before = [t.clone() for t in c.dev_codes + c.dev_scales]
    q.qmm_kv_append(c.cache, c.batch, rope, *c.dev_x)
    assert all(torch.equal(a, b) for a, b in zip(before, c.dev_codes + c.dev_scales))


@pytest.mark.parametrize("scale,grows", [(1e-3, False), (50.0, True)])
def test_kept_codes(q, scale, grows):
    """Small new values leave the kept codes and the scale bit for bit; large ones re-round them."""
    c = Case(q, [(1, 20), (4, 60)], 4, 16, 128, seed=3, scale=scale)
    q.qmm_kv_append(c.cache, c.batch, None, *c.dev_x)
    check_append(c)
    page = c.table[0, 1]
    assert (c.dev_scales[0][page].cpu().numpy() > c.scales[0][page]).all() == grows


def test_token_by_token_equals_definition(q):
    """Forty appends of one token: each value within half a step of the final
    scale plus half a step for every time its block's scale grew."""
    c = Case(q, [(40, 40)], 2, 16, 64, seed=11)
    steps = {}
    for i in range(40):
        b = q.KvBatch(c.batch.tensors[0], torch.tensor([0, 1], dtype=torch.int32, device="cuda"),
                      torch.tensor([i + 1], dtype=torch.int32, device="cuda"))
        q.qmm_kv_append(c.cache, b, None, c.dev_x[0][i:i + 1], c.dev_x[1][i:i + 1])
        steps[i] = c.dev_scales[0].cpu().numpy().astype(np.float64)
    codes, scales = c.dev_codes[0].cpu().numpy(), steps[39]
    for i in range(40):
        page = c.table[0, i // 16]
        for h in range(2):
            seen = [steps[j][page, h] for j in range(i, min(40, (i // 16 + 1) * 16))]
            bound = 0.5 * seen[0] + sum(0.5 * b for a, b in zip(seen, seen[1:]) if b > a) + 1e-4 * scales[page, h]
            assert np.all(np.abs(codes[page, h, i % 16] * scales[page, h] - c.x[0][i, h]) <= bound)


def test_rows_of_a_fused_projection(q):
    """K and V as strided slices of one product's rows, on a stream that is not the current one."""
    c = Case(q, SEQS, 2, 32, 128, seed=5)
    fused = torch.empty(c.rows, 7, 128, device="cuda")
    fused[:, 3:5], fused[:, 5:7] = c.dev_x[0], c.dev_x[1]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    q.qmm_kv_append(c.cache, c.batch, None, fused[:, 3:5], fused[:, 5:7], stream=side)
    side.synchronize()
    check_append(c)


def test_zero_tiny_and_non_finite_blocks(q):
    c = Case(q, [(16, 16), (16, 16), (16, 16), (16, 16)], 2, 16, 64, seed=6)
    k = c.dev_x[0]
    k[:16] = 0.0
    k[16:32] *= 1e-39
    k[32, 0, 5] = float("inf")
    k[48, 1, 0] = float("nan")
    q.qmm_kv_append(c.cache, c.batch, None, *c.dev_x)
    q.qmm_check_device_error()
    codes, scales = c.dev_codes[0].cpu().numpy(), c.dev_scales[0].cpu().numpy()
    pages = c.table[:, 0]
    assert np.all(scales[pages[0]] == 0) and np.all(codes[pages[0]] == 0)
    assert np.all(scales[pages[1]] == 0) and np.all(codes[pages[1]] == 0)
    for page, head in ((pages[2], 0), (pages[3], 1)):
        assert np.isposinf(scales[page, head]) and np.all(codes[page, head] == 0)
        assert np.isfinite(scales[page, 1 - head]) and codes[page, 1 - head].any()
    out = torch.empty(2, 2, 16, 64, device="cuda")
    q.qmm_kv_read(c.cache, torch.tensor(pages[2:], device="cuda"), out, torch.empty_like(out))
    assert out[0, 0].isnan().all() and out[1, 1].isnan().all() and out[0, 1].isfinite().all() and out[1, 0].isfinite().all()


@pytest.mark.parametrize("kind", list(TYPES))
def test_read(q, kind):
    c = Case(q, [(1, 100)], 3, 32, 96, seed=8)
    pages = torch.tensor([4, 0, 2], dtype=torch.int32, device="cuda")
    k = torch.full((3, 3, 32, 96), float("nan"), dtype=TYPES[kind], device="cuda")
    v = torch.full_like(k, float("nan"))
    q.qmm_kv_read(c.cache, pages, k, v)
    for got, codes, scales in ((k, c.codes[0], c.scales[0]), (v, c.codes[1], c.scales[1])):
        want = torch.from_numpy(codes[[4, 0, 2]].astype(np.float32) * scales[[4, 0, 2]][..., None, None]).to(TYPES[kind])
        assert torch.equal(got.cpu(), want)


def test_offsets_outside_their_arrays_are_reported(q):
    """A sequence whose length, rows or page ids do not fit is left out, the others are done."""
    good = [(3, 20), (2, 2)]
    for spoil in ("length", "rows", "page"):
        c = Case(q, good + [(4, 36)], 2, 16, 64, seed=9)
        table, first, length = (t.clone() for t in c.batch.tensors)
        if spoil == "length":
            length[2] = c.most * 16 + 1
        elif spoil == "rows":
            first[3] = c.rows + 1
        else:
            table[2, 2] = c.cache.num_pages
        q.qmm_kv_append(c.cache, q.KvBatch(table, first, length), None, *c.dev_x)
        with pytest.raises(q.QmmError, match="outside"):
            q.qmm_check_device_error()
        q.qmm_check_device_error()  # read once
        c.seqs = good
        check_append(c)


def test_nothing_to_do(q):
    c = Case(q, [(0, 5), (0, 0)], 2, 16, 64)
    q.qmm_kv_append(c.cache, c.batch, None, *c.dev_x)
    empty = torch.empty(0, 2, 16, 64, device="cuda")
    q.qmm_kv_read(c.cache, torch.empty(0, dtype=torch.int32, device="cuda"), empty, empty)
    q.qmm_check_device_error()
    check_append(c)


@pytest.mark.parametrize("heads,page,dim,kind,rot", [(3, 16, 128, "f32", 128), (1, 32, 96, "bf16", 32), (2, 128, 256, "f16", 0), (5, 64, 64, "f32", 16),
                                                     (1, 16, 192, "f16", 192)])
def test_append_few_rows(q, heads, page, dim, kind, rot):
    """Many sequences of one or two new rows, some of none, one of many: a warp takes each touched page."""
    seqs = [(1, 1 + 7 * b) for b in range(30)] + [(0, 5), (2, 2), (0, 0), (2, page + 1), (2, 2 * page), (40, 47 + page)]
    seqs += [(b % 3, 40 + b) for b in range(40)]
    c = Case(q, seqs, heads, page, dim, kind, seed=dim + heads)
    assert c.rows <= 2 * min(len(seqs), c.rows)
    table = rope_table(c.most * page, rot) if rot else None
    q.qmm_kv_append(c.cache, c.batch, q.Rope(torch.from_numpy(table).cuda()) if rot else None, *c.dev_x)
    q.qmm_check_device_error()
    check_append(c, table)
