"""examples/serve.py: every attention call and log probability of a few steps
against their 64-bit forms, with the bounds of the operators' own tests."""
import importlib.util
import os

import numpy as np
import pytest
import torch

from serving_ref import attend, logprobs, rotate

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "serve.py")


@pytest.fixture(scope="module")
def serve():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    spec = importlib.util.spec_from_file_location("serve_example", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_steps(serve, monkeypatch):
    server = serve.Server(layers=2, hidden=512, q_heads=8, heads=2, dim=64, vocab=3000, pages=32, page=32, positions=512)
    q = serve.qmm
    calls, plain = [], q.qmm_kv_attention

    def recorded(cache, batch, rope, x, out, **kw):
        plain(cache, batch, rope, x, out, **kw)
        pages = torch.arange(cache.num_pages, dtype=torch.int32, device="cuda")
        k, v = (torch.empty(cache.num_pages, cache.heads, cache.page_tokens, cache.head_dim, device="cuda") for _ in range(2))
        q.qmm_kv_read(cache, pages, k, v)
        calls.append([t.double().cpu().numpy() for t in (x, out, k, v)] + [t.cpu().numpy() for t in batch.tensors] + [kw["scale"]])

    monkeypatch.setattr(q, "qmm_kv_attention", recorded)
    table = server.rope.tensors[0].cpu().numpy()
    g = torch.Generator().manual_seed(3)
    prompts = [torch.randint(0, 3000, (n,), generator=g).tolist() for n in (150, 1, 31, 33)]
    seqs = [server.add() for _ in prompts]
    logits, ids, logp = server.step(seqs, prompts)
    for step in range(3):
        for row in range(len(seqs)):
            lse, _, _, top, tlp = logprobs(logits[row].double().cpu().numpy(), np.array([0]), 5)
            assert np.array_equal(ids[row].cpu().numpy(), top)
            near = 2.0 ** -20 + 2.0 ** -22 * abs(lse) + 2.0 ** -22 * np.abs(tlp)
            assert np.all(np.abs(logp[row].double().cpu().numpy() - tlp) <= near)
        if step < 2:
            logits, ids, logp = server.step(seqs, [[t] for t in ids[:, 0].tolist()])
    assert server.lengths == [152, 3, 33, 35] and [len(t) for t in server.tables] == [5, 1, 2, 2]
    assert len(calls) == 6
    for x, out, k, v, pages, first, length, scale in calls:
        for b, m in enumerate(length):
            mine = pages[b, :-(-m // 32)]
            kb, vb = (a[mine].transpose(0, 2, 1, 3).reshape(-1, 2, 64)[:m] for a in (k, v))
            rows = range(first[b], first[b + 1])
            for r in set(rows[::13]) | {rows[-1]}:
                pos = m - len(rows) + r - first[b]
                for j in range(8):
                    o, _, size, xs = attend(rotate(x[r, j], pos, table, False), kb[:, j // 4], vb[:, j // 4], pos, scale)
                    # (the cache's values were rounded to fp32 by the read: 2^-24 of a score, and of v)
                    rel = 2 * (2.0 ** -18 + 2.0 ** -21 + 2.0 ** -24) * xs + 2.0 ** -19 + m * 2.0 ** -24 + 2.0 ** -24
                    assert np.all(np.abs(out[r, j] - o) <= rel * size + 2.0 ** -24 * np.abs(o) + 1e-30)
