"""oscar_commit_draft leaves the cache that oscar_quant_append of the gathered rows leaves,
byte for byte: pool, window and state of a twin that appends request by request."""

import numpy as np
import pytest
import torch

from bit_rotated_kv_oscar_gb300 import abi, build
from tests.gpu_harness import D, Layer

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "the gpu-marked tests need a CUDA device"
    build.build()
    abi.lib()


def _twins(lengths, *args, **kw):
    pair = [Layer(*args, **kw) for _ in range(2)]
    for layer in pair:
        layer.cache.pool.zero_()
        for b, n in enumerate(lengths):
            layer.stream_id = 10 * b
            k, v = layer.draw(max(n, 1))
            if n:
                layer.append(b, k, v)
    return pair


def _same(a, b):
    assert torch.equal(a.cache.state, b.cache.state)
    assert torch.equal(a.cache.pool, b.cache.pool)
    assert torch.equal(a.cache.window.view(torch.int16), b.cache.window.view(torch.int16))


def _rows(layer, b, t, seed):
    layer.stream_id = 800 + seed
    k, v = layer.draw(b * t)
    return tuple(x.view(b, t, layer.hkv, D).to(torch.bfloat16).cuda().contiguous() for x in (k, v))


def _step(ref, com, counts, t, seed):
    rng = np.random.default_rng(seed)
    b = len(counts)
    k, v = _rows(ref, b, t, seed)
    path = np.full((b, t), -1, np.int32)
    for r, n in enumerate(counts):
        path[r, :n] = np.sort(rng.permutation(t)[:n])
    for layer in (ref, com):
        for r, n in enumerate(counts):
            layer.cache.reserve(r, layer.len[r] + n, upload=False)
        layer.cache.upload()
    for r, n in enumerate(counts):
        if n:
            rows = torch.from_numpy(path[r, :n]).long().cuda()
            ref.ctx.quant_append(ref.cache.page_table[r:], ref.cache.state[r:], k[r][rows].contiguous(),
                                 v[r][rows].contiguous(), 1, n)
    com.ctx.commit_draft(com.cache.page_table, com.cache.state, k, v, torch.from_numpy(path).cuda(),
                         torch.tensor(counts, dtype=torch.int32, device="cuda"), b, t)
    torch.cuda.synchronize()
    _same(ref, com)
    for layer in (ref, com):
        for r, n in enumerate(counts):
            layer.len[r] += n
    assert ref.ctx.error_flags() == 0 and com.ctx.error_flags() == 0


@pytest.mark.parametrize("sink,recent,group", [(4, 128, 32), (64, 256, 64), (0, 1, 32), (7, 5, 32), (3, 33, 64)])
def test_ragged_counts(sink, recent, group):
    lengths = [0, 1, sink, sink + recent - 1, sink + recent, 400, 611]
    ref, com = _twins(lengths, 4, 2, sink, recent, len(lengths), 900, seed=31, group=group)
    rng = np.random.default_rng(1)
    for s in range(4):
        _step(ref, com, rng.integers(0, 12, len(lengths)).tolist(), 11, s)


@pytest.mark.parametrize("t", [1, 9, 64])
def test_every_row_accepted(t):
    ref, com = _twins([300, 20], 8, 8, 4, 64, 2, 600, seed=32)
    for s in range(3):
        _step(ref, com, [t, t], t, s)


def test_fold_rv_and_spikes():
    ref, com = _twins([300], 4, 2, 4, 64, 1, 400, seed=33, fold_rv=1, spikes=True)
    _step(ref, com, [13], 16, 0)


def test_more_requests_than_ctas():
    lengths = [70 + 3 * i for i in range(40)]
    ref, com = _twins(lengths, 8, 8, 4, 64, 40, 400, seed=34, n_cal=128)
    _step(ref, com, [(5 * i) % 7 for i in range(40)], 6, 0)
    _step(ref, com, [(3 * i + 1) % 7 for i in range(40)], 6, 1)


def test_bad_requests_keep_their_cache():
    ref, com = _twins([200, 200, 200, 200, 200], 4, 2, 4, 64, 5, 300, seed=35)
    k, v = _rows(ref, 5, 6, 0)
    for layer in (ref, com):
        for r in range(5):
            layer.cache.reserve(r, 210)
    before = [x.clone() for x in (com.cache.pool, com.cache.window, com.cache.state)]
    path = torch.tensor([[0, 6, 2, -1, -1, -1], [0, 1, 2, 3, 4, 5], [0, -1, 1, 2, 3, 4], [0, 1, 2, 3, 4, 5],
                         [1, 3, 77, 77, 77, 77]], dtype=torch.int32, device="cuda")
    count = torch.tensor([3, 7, 4, -1, 2], dtype=torch.int32, device="cuda")
    com.ctx.commit_draft(com.cache.page_table, com.cache.state, k, v, path, count, 5, 6)
    torch.cuda.synchronize()
    assert com.ctx.error_flags() == abi.FLAG_BAD_TREE
    assert torch.equal(com.cache.state[:4], before[2][:4])
    rows = torch.tensor([1, 3], device="cuda")
    ref.ctx.quant_append(ref.cache.page_table[4:], ref.cache.state[4:], k[4][rows].contiguous(), v[4][rows].contiguous(),
                         1, 2)
    torch.cuda.synchronize()
    _same(ref, com)   # only request 4 changed
    com.cache.state[1, 0] = -5
    com.ctx.commit_draft(com.cache.page_table, com.cache.state, k, v, path, torch.zeros_like(count), 5, 6)
    torch.cuda.synchronize()
    assert com.ctx.error_flags() == abi.FLAG_BAD_STATE and int(com.cache.state[1, 0]) == -5


def test_bad_page_id_is_reported():
    ref, com = _twins([200], 4, 2, 4, 64, 1, 300, seed=36)
    k, v = _rows(ref, 1, 4, 0)
    com.cache.page_table[0] = -1
    pool = com.cache.pool.clone()
    path = torch.arange(4, dtype=torch.int32, device="cuda")[None]
    com.ctx.commit_draft(com.cache.page_table, com.cache.state, k, v, path, torch.tensor([4], dtype=torch.int32).cuda(), 1, 4)
    torch.cuda.synchronize()
    assert com.ctx.error_flags() == abi.FLAG_BAD_PAGE_ID and torch.equal(pool, com.cache.pool)


def test_captured_and_replayed():
    ref, com = _twins([150], 4, 2, 4, 64, 1, 400, seed=37)
    t = 5
    k, v = _rows(ref, 1, t, 0)
    path, count = torch.arange(t, dtype=torch.int32, device="cuda")[None], torch.tensor([3], dtype=torch.int32).cuda()
    for layer in (ref, com):
        layer.cache.reserve(0, 200)
    keep = com.cache.state.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        com.ctx.commit_draft(com.cache.page_table, com.cache.state, k, v, path, count, 1, t)
    com.cache.state.copy_(keep)
    for n in (3, 5, 0, 1):
        count.fill_(n)
        graph.replay()
        if n:
            ref.ctx.quant_append(ref.cache.page_table, ref.cache.state, k[:, :n].contiguous(), v[:, :n].contiguous(), 1, n)
    torch.cuda.synchronize()
    _same(ref, com)


def test_two_streams_and_repeated_rows():
    # two commits of one context at the same time, on different requests; a row may be
    # taken twice
    lengths = [70 + 31 * i for i in range(12)]
    ref, com = _twins(lengths, 8, 8, 4, 64, 12, 600, seed=39, n_cal=128)
    t = 6
    path = torch.tensor([[0, 2, 2, 5, 5, 5]] * 12, dtype=torch.int32, device="cuda")
    for layer in (ref, com):
        for r in range(12):
            layer.cache.reserve(r, 520, upload=False)
        layer.cache.upload()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in range(6):
        k, v = _rows(ref, 12, t, s)
        count = torch.tensor([(5 * r + s) % (t + 1) for r in range(12)], dtype=torch.int32, device="cuda")
        torch.cuda.synchronize()
        for i, stream in enumerate(streams):
            a = slice(6 * i, 6 * i + 6)
            com.ctx.commit_draft(com.cache.page_table[a], com.cache.state[a], k[a], v[a], path[a], count[a], 6, t, stream=stream)
        for r, n in enumerate(count.tolist()):
            if n:
                rows = path[r, :n].long()
                ref.ctx.quant_append(ref.cache.page_table[r:], ref.cache.state[r:], k[r][rows].contiguous(),
                                     v[r][rows].contiguous(), 1, n)
        torch.cuda.synchronize()
        _same(ref, com)


def test_refusals():
    ref, _ = _twins([10], 4, 2, 4, 64, 1, 100, seed=38)
    k, v = _rows(ref, 1, 4, 0)
    path, count = torch.zeros((1, 4), dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    pt, st = ref.cache.page_table, ref.cache.state
    odd = torch.empty(k.numel() + 8, dtype=k.dtype, device="cuda")[1:k.numel() + 1].view_as(k)
    with pytest.raises(abi.OscarError) as e:
        ref.ctx.commit_draft(pt, st, odd, v, path, count, 1, 4)
    assert e.value.status == -1
    with pytest.raises(ValueError):
        ref.ctx.commit_draft(pt, st, k, v, path.long(), count, 1, 4)
    with pytest.raises(ValueError):
        ref.ctx.commit_draft(pt, st, k, v[:, :3], path, count, 1, 4)
    with pytest.raises(abi.OscarError) as e:
        abi.Context(ref.cfg).commit_draft(pt, st, k, v, path, count, 1, 4)
    assert e.value.status == -2
