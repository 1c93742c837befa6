"""qmm_logprobs on the GPU against 64-bit log probabilities.

Bounds (derived): exponentials are relative to the row's largest logit; each
is off by 2^-21 relative plus what rounding (x - max) log2 e costs, so lse by
less than 2^-20 + 2^-22 |lse| and log probabilities by that and one rounding
of x - lse. Entropy = log l - t / l: t sums p times distances of at most about
100 nats, each rounded once: 2^-18 of (1 + the entropy's largest possible
value ln V). Ids are exact: they are compared by (logit, index)."""
import math

import numpy as np
import pytest
import torch

from serving_ref import logprobs

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def q():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import block_quantized_matmul_q4_gb300 as q
    return q


def run(q, x, given, top, **kw):
    M, G = given.shape
    out = {"lse": torch.full((M,), 7.0, device="cuda"), "entropy": torch.full((M,), 7.0, device="cuda"),
           "given_logp": torch.full((M, G), 7.0, device="cuda"),
           "top_ids": torch.full((M, top), -1, dtype=torch.int32, device="cuda"), "top_logp": torch.full((M, top), 7.0, device="cuda")}
    q.qmm_logprobs(x, given, **out, **kw)
    q.qmm_check_device_error()
    return {k: t.cpu().numpy() for k, t in out.items()}


def check(got, x, given, top):
    x64, V = x.double().cpu().numpy(), x.size(1)
    for m in range(x.size(0)):
        lse, ent, glp, ids, tlp = logprobs(x64[m], given[m].cpu().numpy(), top)
        near = 2.0 ** -20 + 2.0 ** -22 * abs(lse) if math.isfinite(lse) else 0.0

        def close(a, b, tol):
            a, b = np.float64(a), np.float64(b)
            same = (a == b) | (np.abs(a - b) <= tol + 2.0 ** -22 * np.abs(np.where(np.isfinite(b), b, 0)))
            assert np.all(same), (a, b, tol)

        close(got["lse"][m], lse, near)
        close(got["entropy"][m], ent, 2.0 ** -18 * (1 + math.log(V)))
        with np.errstate(invalid="ignore"):
            close(got["given_logp"][m], glp, near)
            close(got["top_logp"][m], tlp, near)
        assert np.array_equal(got["top_ids"][m], ids), (got["top_ids"][m], ids)


@pytest.mark.parametrize("M,V,kind,top,G", [
    (1, 1, "f32", 1, 1), (1, 7, "f16", 7, 2), (3, 33, "bf16", 32, 1), (2, 1000, "f32", 20, 3), (5, 4093, "f16", 5, 1),
    (1, 32768, "f32", 32, 1), (4, 16384, "f32", 8, 1), (3, 16385, "bf16", 20, 4), (2, 131073, "f32", 20, 1), (200, 513, "f32", 0, 1),
    (200, 20001, "bf16", 3, 1), (1, 1048576, "f16", 32, 1), (160, 16390, "f32", 32, 2)])
def test_logprobs(q, M, V, kind, top, G):
    g = torch.Generator().manual_seed(M + V)
    x = (torch.randn(M, V, generator=g) * 3).to(TYPES[kind]).cuda()
    given = torch.randint(0, V, (M, G), generator=g).to(torch.int32).cuda()
    check(run(q, x, given, top), x, given, top)


@pytest.mark.parametrize("V", [40, 20000, 70000])
def test_ties_and_masks(q, V):
    """Equal logits by rising id; masked ones (-inf, or the type's lowest value) where they belong; rows that are all masked."""
    rows = [torch.zeros(V), torch.full((V,), -math.inf), torch.full((V,), torch.finfo(torch.float32).min), torch.zeros(V), torch.zeros(V),
            torch.randint(0, 3, (V,), generator=torch.Generator().manual_seed(1)).float(), torch.full((V,), -math.inf)]
    rows[3][::2] = -0.0
    rows[4][5:] = -math.inf
    rows[6][V - 1] = -3.0
    rows.append(torch.full((V,), torch.finfo(torch.float32).min))
    rows[7][V // 2] = 2.0
    x = torch.stack(rows).cuda()
    given = torch.tensor([[0, V - 1]] * len(rows), dtype=torch.int32).cuda()
    got = run(q, x, given, 20)
    check(got, x, given, 20)
    assert got["lse"][1] == -np.inf and got["entropy"][1] == 0 and np.all(got["top_logp"][1] == -np.inf)


def test_nan_and_infinity(q):
    x = torch.randn(3, 5000, generator=torch.Generator().manual_seed(2)).cuda()
    x[0, 77] = math.nan
    x[1, 4999] = math.inf
    got = run(q, x, torch.zeros(3, 1, dtype=torch.int32, device="cuda"), 4)
    for m, first in ((0, 77), (1, 4999)):
        assert np.isnan(got["lse"][m]) and np.isnan(got["entropy"][m]) and np.isnan(got["given_logp"][m]).all()
        assert got["top_ids"][m, 0] == first
    check({k: v[2:] for k, v in got.items()}, x[2:], torch.zeros(1, 1, dtype=torch.int32), 4)


@pytest.mark.parametrize("kind,offset,stride", [("f32", 1, 1005), ("f16", 3, 1001), ("bf16", 1, 1002), ("f32", 0, 2000)])
def test_rows_of_any_alignment(q, kind, offset, stride):
    """Rows apart by more than their length, starting anywhere: nothing outside them counts."""
    g = torch.Generator().manual_seed(4)
    flat = torch.full((offset + 9 * stride,), 1000.0, dtype=TYPES[kind])
    view = flat.cuda()[offset:offset + 9 * stride].view(9, stride)[:, :1000]
    view.copy_(torch.randn(9, 1000, generator=g) * 2)
    given = torch.randint(0, 1000, (9, 1), generator=g).to(torch.int32).cuda()
    check(run(q, view, given, 6), view, given, 6)


def test_ids_outside_the_vocabulary(q):
    x = torch.randn(2, 100, device="cuda")
    given = torch.tensor([[-1, 5], [100, 99]], dtype=torch.int32, device="cuda")
    lp = run(q, x, given, 0)["given_logp"]
    assert np.isnan(lp[0, 0]) and np.isnan(lp[1, 0]) and np.isfinite(lp[:, 1]).all()


def test_outputs_are_optional_and_workspace_is_the_callers(q):
    x = torch.randn(3, 40000, device="cuda")
    given = torch.tensor([[1], [2], [3]], dtype=torch.int32, device="cuda")
    want = run(q, x, given, 5)
    need = q.qmm_logprobs_workspace_bytes(3, 40000, 5)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    got = run(q, x, given, 5, workspace=ws, ws_bytes=need)
    assert all(np.array_equal(want[k], got[k]) for k in want)
    lse = torch.empty(3, device="cuda")
    q.qmm_logprobs(x, lse=lse)
    assert np.array_equal(lse.cpu().numpy(), want["lse"])
    with pytest.raises(q.QmmError, match="workspace"):
        q.qmm_logprobs(x, given, lse, workspace=ws, ws_bytes=16)
    q.qmm_logprobs(torch.empty(0, 10, device="cuda"))


@pytest.mark.parametrize("M,V,kind,top", [(920, 25000, "f32", 8), (920, 26001, "f32", 3), (920, 51301, "bf16", 1), (40, 262147, "f16", 32)])
def test_large_chunks(q, M, V, kind, top):
    """Rows of one, two and many chunks, where there are enough rows for large ones."""
    g = torch.Generator().manual_seed(V)
    x = (torch.randn(M, V, generator=g) * 3).to(TYPES[kind]).cuda()
    given = torch.randint(0, V, (M, 1), generator=g, dtype=torch.int32).cuda()
    got = run(q, x, given, top)
    rows = list(range(0, M, max(1, M // 12)))
    check({k: v[rows] for k, v in got.items()}, x[rows], given[rows], top)
