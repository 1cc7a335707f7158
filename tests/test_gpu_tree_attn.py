"""GPU parity of the attention of drafted-token trees (oscar_tree_attn) against the
float64 oracle, at the sizes and masks where it can go wrong."""

import numpy as np
import pytest
import torch

from bit_rotated_kv_oscar_gb300 import abi, build
from tests.draft_harness import check_rows, draft, parents, tree_call, tree_reference
from tests.gpu_harness import D, Layer

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "the gpu-marked tests need a CUDA device"
    build.build()
    abi.lib()


def _layer(lengths, *args, **kw):
    layer = Layer(*args, **kw)
    layer.cache.pool.fill_(0xFF)   # slots never written are NaN scales
    for b, n in enumerate(lengths):
        if n:
            layer.stream_id = 10 * b
            layer.append(b, *layer.draw(n))
    return layer


def _check(layer, lengths, t, width, used=None, seed=0):
    rng = np.random.default_rng(seed)
    b = len(lengths)
    host, dev = draft(layer, b, t, seed)
    par = np.stack([parents(rng, t, width) for _ in range(b)])
    length = None if used is None else torch.tensor(used, dtype=torch.int32, device="cuda")
    o = tree_call(layer, dev, torch.from_numpy(par).cuda(), length)
    torch.cuda.synchronize()
    got = o.float().cpu().numpy()
    for r in range(b):
        n = t if used is None else used[r]
        assert np.isnan(got[r, n:]).all()           # rows of unused nodes are left as they were
        if n:
            cache = layer.oracle_cache_resolved(r)
            want, bound = tree_reference(cache, *(x[r].astype(np.float64) for x in host), par[r], n)
            check_rows(got[r, :n], want, bound)
    assert layer.ctx.error_flags() == 0
    return host, dev, par, o


# query group sizes x numbers of nodes: one row to 512 rows per cached head
@pytest.mark.parametrize("hq,hkv,t", [(2, 2, 1), (8, 1, 1), (2, 2, 17), (4, 2, 8), (4, 2, 9), (8, 2, 8), (8, 2, 13),
                                      (8, 1, 5), (8, 1, 16), (8, 1, 64), (4, 1, 33)])
def test_heads_and_nodes(hq, hkv, t):
    layer = _layer([501], hq, hkv, 4, 64, 1, 640, seed=3)
    _check(layer, [501], t, 3, seed=t)


# cached tokens around the sink, the ring, a page and the warps' page pairs
@pytest.mark.parametrize("n", [0, 1, 3, 4, 5, 67, 68, 69, 79, 80, 81, 95, 96, 97, 260, 333])
def test_lengths(n):
    layer = _layer([n], 8, 2, 4, 64, 1, 400, seed=5)
    _check(layer, [n], 6, 2, seed=n)


@pytest.mark.parametrize("sink,recent", [(0, 1), (0, 64), (7, 33), (64, 256), (500, 524)])
def test_windows(sink, recent):
    n = sink + recent + 203
    layer = _layer([n], 8, 2, sink, recent, 1, n + 16, seed=6)
    _check(layer, [n], 9, 3)


@pytest.mark.parametrize("width", [1, 2, 64])
def test_chains_and_stars(width):
    layer = _layer([300], 4, 2, 4, 64, 1, 400, seed=7)
    _check(layer, [300], 64, width, seed=width)


@pytest.mark.parametrize("hq,t", [(16, 3), (8, 21)])
def test_groups_of_64(hq, t):
    layer = _layer([700, 391], hq, 2, 64, 256, 2, 800, seed=8, group=64, clip_percentiles=(96.0, 92.0))
    _check(layer, [700, 391], t, 3)


@pytest.mark.parametrize("hq", [4, 16])
def test_ragged_batch(hq):
    lengths, used = [900, 0, 3, 130, 417], [7, 5, 1, 0, 11]
    layer = _layer(lengths, hq, 2, 4, 128, 5, 1024, seed=9)
    _check(layer, lengths, 11, 3, used)


@pytest.mark.parametrize("splits", [1, 2, 37, 200])
@pytest.mark.parametrize("hq", [4, 16])
def test_split_counts(splits, hq):
    layer = _layer([3000], hq, 2, 4, 64, 1, 3100, seed=10, num_splits=splits)
    _check(layer, [3000], 5, 2)


def test_more_pages_than_one_batch_of_ids():
    # one split: each warp walks 94 pages, three registers' worth of page ids
    layer = _layer([12000], 8, 1, 4, 64, 1, 12032, seed=11, num_splits=1)
    _check(layer, [12000], 5, 2)


# Many requests of 17 .. 32 query rows per cached head take another kernel, whose warps share
# page pairs: 10 requests x 8 heads are more than one wave of 16-row tiles on 152 SMs.
_MANY = [700, 0, 3, 68, 69, 84, 85, 260, 333, 196]


@pytest.mark.parametrize("hq,t", [(8, 17), (8, 32), (16, 9), (16, 16), (32, 5), (64, 3), (64, 4)])
def test_many_requests(hq, t):
    layer = _layer(_MANY, hq, 8, 4, 64, 10, 704, seed=23)
    _check(layer, _MANY, t, 3, seed=t)


@pytest.mark.parametrize("group,fold", [(32, 1), (64, 0), (64, 1)])
def test_many_ragged_requests(group, fold):
    # some use 16 rows or fewer, one none
    used = [11, 11, 1, 9, 8, 5, 0, 10, 4, 3]
    layer = _layer(_MANY, 16, 8, 4, 64, 10, 704, seed=24, group=group, fold_rv=fold)
    _check(layer, _MANY, 11, 3, used)


@pytest.mark.parametrize("splits", [1, 3, 40, 256])
def test_many_requests_split(splits):
    # one split of the longest: 70 pages for each warp, three batches of page ids
    lengths = [9000] + _MANY[1:]
    layer = _layer(lengths, 16, 8, 4, 64, 10, 9040, seed=25, num_splits=splits)
    _check(layer, lengths, 9, 2)


def test_many_requests_token_spikes():
    layer = _layer(_MANY, 16, 8, 4, 64, 10, 704, seed=26, spikes=True)
    _check(layer, _MANY, 12, 3)


def test_many_requests_bad_page_ids_and_replay():
    layer = _layer([400] * 10, 16, 8, 4, 64, 10, 512, seed=27)
    host, dev = draft(layer, 10, 9, 0)
    par = torch.tensor([[-1, 0, 0, 1, 2, 2, 3, 6, 7]] * 10, dtype=torch.int32, device="cuda")
    good = tree_call(layer, dev, par)
    ws = torch.empty(layer.ctx.tree_attn_workspace_bytes(10, 9), dtype=torch.uint8, device="cuda")
    pt, state, o = layer.cache.page_table[:10].clone(), layer.cache.state[:10], torch.zeros_like(dev[0])
    call = lambda: layer.ctx.tree_attn(*dev, par, pt, state, o, 10, 9, ws)  # noqa: E731
    call()
    torch.cuda.synchronize()
    assert torch.equal(o, good)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    o.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, good) and layer.ctx.error_flags() == 0
    pt[4, 5], pt[4, 6] = layer.cache.num_pages, -4
    graph.replay()
    torch.cuda.synchronize()
    assert layer.ctx.error_flags() == abi.FLAG_BAD_PAGE_ID
    assert torch.equal(o[:4], good[:4]) and torch.equal(o[5:], good[5:])
    # the positions of those pages take no part, whatever they hold
    pages = layer.cache.pool.view(layer.cache.num_pages, -1)
    for i in (5, 6):
        pages[int(layer.cache.page_table_host[4, i])] = 0xFF
    pt[4, 5:7] += 2 * layer.cache.num_pages
    skipped = o[4].clone()
    graph.replay()
    torch.cuda.synchronize()
    assert layer.ctx.error_flags() == abi.FLAG_BAD_PAGE_ID
    assert torch.equal(o[4], skipped) and torch.isfinite(o).all() and not torch.equal(o[4], good[4])


@pytest.mark.parametrize("hq,hkv,batch", [(4, 2, 3), (16, 8, 10), (16, 2, 3)])
def test_unused_rows_and_workspace_may_hold_anything(hq, hkv, batch):
    # 22 (one wave and many requests) and 88 query rows per cached head
    lengths, used = [300, 3, 130] + _MANY[3:batch], ([7, 11, 2] * 4)[:batch]
    layer = _layer(lengths, hq, hkv, 4, 64, batch, 704, seed=28)
    host, dev = draft(layer, batch, 11, 0)
    par = torch.tensor([[-1] + [max(0, i - 1 - i % 3) for i in range(1, 11)]] * batch, dtype=torch.int32, device="cuda")
    length = torch.tensor(used, dtype=torch.int32, device="cuda")
    want = tree_call(layer, dev, par, length)
    for b, n in enumerate(used):
        par[b, n:] = 99
        for x in dev:
            x[b, n:] = float("nan")
    size = layer.ctx.tree_attn_workspace_bytes(batch, 11)
    for fill in (0xFF, 0x7F, 0):
        ws = torch.full((size,), fill, dtype=torch.uint8, device="cuda")
        got = tree_call(layer, dev, par, length, workspace=ws)
        for b, n in enumerate(used):
            assert torch.isfinite(got[b, :n]).all() and torch.equal(got[b, :n], want[b, :n])
            assert got[b, n:].isnan().all()
    assert layer.ctx.error_flags() == 0


@pytest.mark.parametrize("fold", [0, 1])
def test_many_rows(fold):
    # 104 rows for each of 8 heads of 6 requests: the merge of more rows than two CTAs per SM
    # hold at a time; some rows unused
    lengths, used = [200, 68, 0, 133, 417, 90], [13, 13, 12, 13, 2, 13]
    layer = _layer(lengths, 64, 8, 4, 64, 6, 448, seed=30, fold_rv=fold)
    _check(layer, lengths, 13, 3, used)


def test_fold_rv():
    layer = _layer([400], 8, 2, 4, 64, 1, 512, seed=12, fold_rv=1)
    _check(layer, [400], 9, 2)


def test_token_spikes():
    layer = _layer([600], 8, 2, 4, 64, 1, 640, seed=13, spikes=True)
    _check(layer, [600], 12, 3)


def test_values_beyond_fp16_in_the_window():
    # BF16 keys and values keep their own range: the draft's values reach 1e30
    layer = _layer([40], 4, 2, 4, 64, 1, 128, seed=14)
    host, dev = draft(layer, 1, 4, 0)
    q, k, v = dev
    v.mul_(1e30)
    par = torch.tensor([[-1, 0, 1, 2]], dtype=torch.int32, device="cuda")
    got = tree_call(layer, (q, k, v), par).float().cpu().numpy()[0]
    want, bound = tree_reference(layer.oracle_cache(0), host[0][0].astype(np.float64), host[1][0].astype(np.float64),
                                 v[0].float().cpu().numpy().astype(np.float64), par[0].cpu().numpy(), 4)
    assert np.isfinite(got).all()
    assert (np.abs(got - want) <= bound + 2.0 ** -8 * (np.abs(want) + bound)).all()


def test_high_page_ids():
    # page blocks past 2^31 bytes of the pool
    layer = Layer(8, 8, 4, 64, 1, 400, seed=15, extra_pages=190000, shuffled=False)
    layer.cache.free = list(layer.cache.free)[::-1]     # highest ids first
    layer.stream_id = 0
    layer.append(0, *layer.draw(400))
    assert int(layer.cache.page_table_host[0, 0]) * 8 * 1536 > 2 ** 31
    _check(layer, [400], 3, 2)


def test_same_call_twice_and_other_rows_do_not_matter():
    # bitwise the same result again; a request alone gives what it gives in a batch of ragged
    # requests, up to the fp32 merge of another split count
    layer = _layer([900, 333], 8, 2, 4, 128, 2, 1024, seed=16, num_splits=3)
    host, dev, par, o = _check(layer, [900, 333], 7, 2)
    again = tree_call(layer, dev, torch.from_numpy(par).cuda())
    assert torch.equal(o, again)


def test_a_chain_is_what_appending_and_decoding_gives():
    # node i of a chain attends to what the cache would hold after appending nodes 0 .. i;
    # with a ring large enough to hold them nothing is quantised in between
    layer = _layer([100], 8, 2, 4, 256, 1, 512, seed=17)
    host, dev = draft(layer, 1, 5, 0)
    par = torch.tensor([[-1, 0, 1, 2, 3]], dtype=torch.int32, device="cuda")
    got = tree_call(layer, dev, par).float().cpu().numpy()[0]
    for i in range(5):
        layer.append(0, torch.from_numpy(host[1][0, i:i + 1]), torch.from_numpy(host[2][0, i:i + 1]))
        want = layer.decode(torch.from_numpy(host[0][:, i]))[0]
        assert np.linalg.norm(got[i] - want) <= (2e-3 + 2.0 ** -8) * np.linalg.norm(want)


def test_bad_trees_and_states():
    layer = _layer([200, 200, 200, 200], 8, 2, 4, 64, 4, 256, seed=18)
    host, dev = draft(layer, 4, 5, 0)
    par = torch.tensor([[-1, 0, 1, 2, 3]] * 4, dtype=torch.int32, device="cuda")
    good = tree_call(layer, dev, par).clone()
    for bad in ([0, 0, 1, 2, 3], [-1, 0, 2, 2, 3], [-1, -1, 1, 2, 3], [-1, 0, 1, 2, 9], [-1, 0, 1, 2, -7]):
        p = par.clone()
        p[1] = torch.tensor(bad, dtype=torch.int32)
        o = tree_call(layer, dev, p)
        assert (o[1] == 0).all() and torch.equal(o[0], good[0]) and torch.equal(o[2:], good[2:])
        assert layer.ctx.error_flags() == abi.FLAG_BAD_TREE
    for n in (-1, 6):
        o = tree_call(layer, dev, par, torch.tensor([5, 5, n, 5], dtype=torch.int32, device="cuda"))
        assert (o[2] == 0).all() and torch.equal(o[3], good[3])
        assert layer.ctx.error_flags() == abi.FLAG_BAD_TREE
    # a parent past the used nodes' own check is not read
    p = par.clone()
    p[1, 4] = 77
    o = tree_call(layer, dev, p, torch.tensor([5, 4, 5, 5], dtype=torch.int32, device="cuda"))
    assert torch.equal(o[1, :4], good[1, :4]) and layer.ctx.error_flags() == 0
    keep = layer.cache.state.clone()
    layer.cache.state[3, 2] = 9   # window row outside the batch
    o = tree_call(layer, dev, par)
    assert (o[3] == 0).all() and torch.equal(o[:3], good[:3])
    assert layer.ctx.error_flags() == abi.FLAG_BAD_STATE
    layer.cache.state.copy_(keep)


def test_bad_page_ids_are_skipped():
    layer = _layer([400], 8, 2, 4, 64, 1, 512, seed=19)
    host, dev = draft(layer, 1, 4, 0)
    par = torch.tensor([[-1, 0, 0, 1]], dtype=torch.int32, device="cuda")
    layer.cache.page_table[0, 5] = layer.cache.num_pages
    layer.cache.page_table[0, 6] = -4
    got = tree_call(layer, dev, par).float().cpu().numpy()[0]
    assert layer.ctx.error_flags() == abi.FLAG_BAD_PAGE_ID
    # the positions of those pages take no part
    cache = layer.oracle_cache_resolved(0)
    from tests.draft_harness import ancestors
    see = ancestors(par[0].cpu().numpy(), 4)
    for h in range(2):
        kh, vh = cache.raw_kv(h)
        keep = np.r_[0:80, 112:400]
        kk, vv = np.concatenate([kh[keep], host[1][0, :, h]]), np.concatenate([vh[keep], host[2][0, :, h]])
        for m in range(4):
            s = host[0][0, :, 4 * h + m].astype(np.float64) @ kk.T / np.sqrt(D)
            s[:, len(keep):][~see] = -np.inf
            p = np.exp(s - s.max(1, keepdims=True))
            want = (p / p.sum(1, keepdims=True)) @ vv
            assert np.linalg.norm(got[:, 4 * h + m] - want) <= (2e-3 + 2.0 ** -8) * np.linalg.norm(want)


def test_captured_and_replayed_on_other_inputs():
    layer = _layer([500], 8, 2, 4, 64, 1, 640, seed=20)
    host, dev = draft(layer, 1, 6, 0)
    par = torch.tensor([[-1, 0, 0, 1, 1, 2]], dtype=torch.int32, device="cuda")
    ws = torch.empty(layer.ctx.tree_attn_workspace_bytes(1, 6), dtype=torch.uint8, device="cuda")
    pt, state, o = layer.cache.page_table[:1].contiguous(), layer.cache.state[:1], torch.zeros_like(dev[0])
    call = lambda: layer.ctx.tree_attn(*dev, par, pt, state, o, 1, 6, ws)  # noqa: E731
    call()
    torch.cuda.synchronize()
    first = o.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    host2, dev2 = draft(layer, 1, 6, 1)
    for x, y in zip(dev, dev2):
        x.copy_(y)
    layer.append(0, *layer.draw(40))    # the cache moved on as well
    graph.replay()
    torch.cuda.synchronize()
    got = o.clone()
    o.zero_()
    call()
    torch.cuda.synchronize()
    assert torch.equal(got, o) and not torch.equal(got, first)


def test_two_streams_with_their_own_workspaces():
    layer = _layer([800], 8, 2, 4, 64, 1, 1024, seed=21)
    sets = [draft(layer, 1, 8, s)[1] for s in range(2)]
    par = torch.tensor([[-1, 0, 0, 1, 1, 2, 5, 6]], dtype=torch.int32, device="cuda")
    want = [tree_call(layer, d, par).clone() for d in sets]
    ws = [torch.empty(layer.ctx.tree_attn_workspace_bytes(1, 8), dtype=torch.uint8, device="cuda") for _ in sets]
    outs = [torch.zeros_like(d[0]) for d in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    for _ in range(10):
        for d, w, o, s in zip(sets, ws, outs, streams):
            tree_call(layer, d, par, o=o, workspace=w, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(want, outs))


def test_refusals():
    layer = _layer([40], 8, 2, 4, 64, 2, 128, seed=22)
    host, dev = draft(layer, 1, 4, 0)
    q, k, v = dev
    par = torch.tensor([[-1, 0, 0, 1]], dtype=torch.int32, device="cuda")
    pt, state, o = layer.cache.page_table[:1].contiguous(), layer.cache.state[:1], torch.zeros_like(q)
    n = layer.ctx.tree_attn_workspace_bytes(1, 4)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")

    def status(**kw):
        a = dict(q=q, k=k, v=v, parent=par, page_table=pt, state=state, o=o, batch=1, n_draft=4, workspace=ws)
        a.update(kw)
        with pytest.raises(abi.OscarError) as e:
            layer.ctx.tree_attn(**a)
        return e.value.status
    assert status(workspace=ws[:n - 1]) == -3
    odd = torch.empty(n + 16, dtype=torch.uint8, device="cuda")[1:n + 1]
    assert status(workspace=odd) == -1
    shifted = torch.empty(q.numel() + 8, dtype=q.dtype, device="cuda")[1:q.numel() + 1].view_as(q)
    assert status(q=shifted) == -1
    big = torch.zeros((1, 65, 8, D), dtype=q.dtype, device="cuda")
    kv = torch.zeros((1, 65, 2, D), dtype=q.dtype, device="cuda")
    par65 = torch.zeros((1, 65), dtype=torch.int32, device="cuda")
    assert status(q=big, k=kv, v=kv, o=big.clone(), parent=par65, n_draft=65) == -5
    assert layer.ctx.tree_attn_workspace_bytes(1, 65) == 0 and layer.ctx.tree_attn_workspace_bytes(3, 4) == 0
    for kw in (dict(q=q.float()), dict(k=v.transpose(1, 2)), dict(parent=par.long()), dict(o=o[:, :3]),
               dict(q=q.cpu()), dict(v=v.expand(1, 4, 2, D)[:, ::2])):
        with pytest.raises(ValueError):
            status(**kw)
    fresh = abi.Context(layer.cfg)
    with pytest.raises(abi.OscarError) as e:
        fresh.tree_attn(q, k, v, par, pt, state, o, 1, 4, ws)
    assert e.value.status == -2
