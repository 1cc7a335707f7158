"""The drafted-token operators as a serving step uses them: projection rows through
qkv_norm_rope, attention of the tree, verification, commit of the accepted path, all on
the device and captured once as a graph, beside a twin cache that takes the accepted
tokens through oscar_quant_append."""

import numpy as np
import pytest
import torch

import oracle
from bit_rotated_kv_oscar_gb300 import abi, build
from tests.draft_harness import check_rows, parents, tree_reference
from tests.gpu_harness import D, Layer
from tests.test_gpu_verify_draft import reference as verify_reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "the gpu-marked tests need a CUDA device"
    build.build()
    abi.lib()


def test_speculative_steps():
    lengths, hq, hkv, t, vocab, steps = [180, 0, 66], 8, 2, 7, 50, 6
    b = len(lengths)
    ref, spec = (Layer(hq, hkv, 4, 64, b, 400, seed=51) for _ in range(2))
    for layer in (ref, spec):
        layer.cache.pool.zero_()
        for r, n in enumerate(lengths):
            layer.stream_id = 10 * r
            if n:
                layer.append(r, *layer.draw(n))
            layer.cache.reserve(r, n + steps * t)
    dev = lambda *s, d=torch.bfloat16: torch.zeros(s, dtype=d, device="cuda")  # noqa: E731
    i32 = torch.int32
    width = (hq + 2 * hkv) * D
    qkv, depth = dev(b * t, width), dev(b, t, d=i32)
    q, k, v, o = dev(b, t, hq, D), dev(b, t, hkv, D), dev(b, t, hkv, D), dev(b, t, hq, D)
    wq, wk = (torch.ones(D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    turns = abi.rope_turns(1e4 ** (-np.arange(0, D, 2) / D)).cuda()
    parent, used, tokens = dev(b, t, d=i32), dev(b, d=i32), dev(b, t, d=i32)
    probs, ua, us = dev(b, t, vocab, d=torch.float32), dev(b, t, d=torch.float32), dev(b, d=torch.float32)
    path, count, nxt = dev(b, t, d=i32), dev(b, d=i32), dev(b, d=i32)
    ws = torch.empty(spec.ctx.tree_attn_workspace_bytes(b, t), dtype=torch.uint8, device="cuda")
    ctx, cache = spec.ctx, spec.cache

    def step():
        pos = (cache.state[:, :1] + depth).view(-1)
        abi.qkv_norm_rope(qkv, pos, turns, q.view(-1, hq, D), k.view(-1, hkv, D), v.view(-1, hkv, D), q_weight=wq,
                          k_weight=wk)
        ctx.tree_attn(q, k, v, parent, cache.page_table, cache.state, o, b, t, ws, draft_len=used)
        abi.verify_draft(probs, tokens, parent, ua, us, path, count, nxt, draft_len=used)
        ctx.commit_draft(cache.page_table, cache.state, k, v, path, count, b, t)

    keep = [x.clone() for x in (cache.state, cache.pool, cache.window)]
    used.fill_(0)
    step()                                   # nothing used: nothing changes
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(keep, (cache.state, cache.pool, cache.window)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    rng = np.random.default_rng(2)
    total = 0
    for s in range(steps):
        par = np.stack([parents(rng, t, 3) for _ in range(b)])
        n = rng.integers(1, t + 1, b)
        dep = np.zeros((b, t), np.int64)
        for i in range(1, t):
            dep[:, i] = dep[np.arange(b), par[:, i]] + 1
        p = rng.dirichlet(np.full(vocab, 0.1), (b, t)).astype(np.float32)
        tok = np.zeros((b, t), np.int64)
        for r in range(b):
            for i in range(1, t):
                tok[r, i] = np.argsort(-p[r, par[r, i]])[(par[r, 1:i] == par[r, i]).sum()]
        a, w = rng.random((b, t), np.float32), rng.random(b, np.float32)
        for buf, x in ((parent, par), (used, n), (depth, dep), (tokens, tok), (probs, p), (ua, a), (us, w),
                       (qkv, rng.standard_normal((b * t, width)))):
            buf.copy_(torch.from_numpy(np.ascontiguousarray(x)).to(buf.dtype))
        before = [(spec.len[r], spec.e[r]) for r in range(b)]
        caches = [ref.oracle_cache_resolved(r) for r in range(b)]
        graph.replay()
        torch.cuda.synchronize()
        host = [x.float().cpu().numpy().astype(np.float64) for x in (q, k, v)]
        for r in range(b):
            want, bound = tree_reference(caches[r], host[0][r], host[1][r], host[2][r], par[r], n[r])
            check_rows(o[r, :n[r]].float().cpu().numpy(), want, bound)
            steps_, x = verify_reference(p[r], None, tok[r], par[r], n[r], a[r], w[r])
            assert path[r].tolist()[:len(steps_)] == steps_ and int(count[r]) == len(steps_) and int(nxt[r]) == x
            total += len(steps_)
            rows = torch.tensor(steps_, device="cuda")
            kr, vr = k[r][rows].contiguous(), v[r][rows].contiguous()
            ref.append(r, kr.float().cpu(), vr.float().cpu())
            spec._record(r, kr.float().cpu(), vr.float().cpu())
            assert (spec.len[r], spec.e[r]) == oracle.next_state(*before[r], len(steps_), 64, 4)
        assert torch.equal(ref.cache.state, cache.state) and torch.equal(ref.cache.pool, cache.pool)
        assert torch.equal(ref.cache.window.view(torch.int16), cache.window.view(torch.int16))
    assert total > steps * b            # drafts were accepted
    assert ctx.error_flags() == 0 and ref.ctx.error_flags() == 0
    # the plain decode step goes on from there
    qd = ref.queries(b, 99)
    got = spec.decode(qd)
    for r in range(b):
        want = spec.oracle_decode(qd[r].numpy(), r)
        assert np.linalg.norm(got[r] - want) <= 2e-3 * np.linalg.norm(want)
