"""oscar_verify_draft against a float64 restatement: paths and tokens must be equal.

Equality holds by arithmetic: acceptance compares exact products (or 2^-44 fixed-point sums
against float32 numbers), and the running sums of at most 2^18 weights, each off by at most
2^-45, differ from the float64 ones by at most 2^-27, so a draw changes only where u falls
within 2^-27 of a border; the draws here keep 2^-20 away from every border."""

import numpy as np
import pytest
import torch

from bit_rotated_kv_oscar_gb300 import abi, build
from tests.draft_harness import parents

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "the gpu-marked tests need a CUDA device"
    build.build()
    abi.lib()


def reference(p, q, tok, par, n, ua, us):
    """(path, token) of one request; p, q [t, V]."""
    if n == 0:
        return [], -1
    path = [0]
    while True:
        i = path[-1]
        kids = [j for j in range(1, n) if par[j] == i]
        to, mass, seen = None, 0.0, set()
        for j in kids:
            x = tok[j]
            if q is not None:
                if np.float64(ua[i]) * np.float64(q[i, x]) < np.float64(p[i, x]):
                    to = j
            elif x not in seen:
                seen.add(x)
                mass += np.float64(p[i, x])
                if ua[i] < mass:
                    to = j
            if to is not None:
                break
        if to is None:
            break
        path.append(to)
    w = np.clip(p[i].astype(np.float64), 0, 1)
    if kids and q is not None:
        w = np.maximum(w - q[i], 0)
    elif kids:
        w[[tok[j] for j in kids]] = 0
    if w.sum() == 0:
        w = p[i].astype(np.float64)
    run = np.cumsum(w)
    if run[-1] == 0:
        return path, -1
    return path, int(np.flatnonzero((run > us * run[-1]) & (w > 0))[0])


def clear_of_borders(p, q, tok, par, n, ua, us):
    """Move us off the borders of the reference's draw by at least 2^-20 of the total."""
    path, x = reference(p, q, tok, par, n, ua, us)
    i = path[-1]
    kids = [j for j in range(1, n) if par[j] == i]
    w = p[i].astype(np.float64)
    if kids and q is not None:
        w = np.maximum(w - q[i], 0)
    elif kids:
        w[[tok[j] for j in kids]] = 0
    if w.sum() == 0:
        w = p[i].astype(np.float64)
    run = np.concatenate([[0], np.cumsum(w)]) / w.sum()
    big = int(np.argmax(w))
    if run[x] + 2.0 ** -20 < us < run[x + 1] - 2.0 ** -20:
        return us
    return np.float32((run[big] + run[big + 1]) / 2)


def run(p, q, tok, par, used, ua, us, base=0, dbase=0):
    """The device call; `base` shifts probs by that many floats (rows off 16-byte alignment)."""
    b, t, v = p.shape

    def put(x, shift):
        buf = torch.zeros(x.size + 4, dtype=torch.float32, device="cuda")
        view = buf[shift:shift + x.size].view(b, t, v)
        view.copy_(torch.from_numpy(x))
        return view
    path = torch.full((b, t), -9, dtype=torch.int32, device="cuda")
    count = torch.full((b,), -9, dtype=torch.int32, device="cuda")
    nxt = torch.full((b,), -9, dtype=torch.int32, device="cuda")
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    dev = lambda x, d: torch.from_numpy(np.ascontiguousarray(x, dtype=d)).cuda()  # noqa: E731
    abi.verify_draft(put(p, base), dev(tok, np.int32), dev(par, np.int32), dev(ua, np.float32), dev(us, np.float32), path,
                     count, nxt, draft_probs=None if q is None else put(q, dbase),
                     draft_len=None if used is None else dev(used, np.int32), err_flags=flags)
    torch.cuda.synchronize()
    return path.cpu().numpy(), count.cpu().numpy(), nxt.cpu().numpy(), int(flags.item())


def case(seed, b, t, v, width, sampled, ragged=True, sharp=2.0):
    rng = np.random.default_rng(seed)
    logits = rng.standard_normal((b, t, v)) * sharp
    soft = lambda x: (lambda e: (e / e.sum(-1, keepdims=True)).astype(np.float32))(np.exp(x - x.max(-1, keepdims=True)))  # noqa: E731
    p = soft(logits)
    guess = logits + rng.standard_normal(logits.shape) * 0.7
    par = np.stack([parents(rng, t, width) for _ in range(b)])
    tok = np.zeros((b, t), np.int32)
    q = soft(guess) if sampled else None
    for r in range(b):
        seen = {}
        for i in range(1, t):
            at = par[r, i]
            if sampled:
                c = np.cumsum(q[r, at].astype(np.float64))
                tok[r, i] = min(int(np.searchsorted(c, rng.random() * c[-1])), v - 1)
            else:
                k = seen.get(at, 0)
                seen[at] = k + 1
                tok[r, i] = np.argsort(-guess[r, at])[min(k, v - 1)]
    used = rng.integers(1, t + 1, b) if ragged else np.full(b, t)
    ua, us = rng.random((b, t), np.float32), rng.random(b, np.float32)
    us = np.array([clear_of_borders(p[r], None if q is None else q[r], tok[r], par[r], used[r], ua[r], us[r])
                   for r in range(b)], np.float32)
    return p, q, tok, par, used, ua, us


def check(p, q, tok, par, used, ua, us, **kw):
    path, count, nxt, flags = run(p, q, tok, par, used, ua, us, **kw)
    for r in range(len(p)):
        want, x = reference(p[r], None if q is None else q[r], tok[r], par[r], used[r], ua[r], us[r])
        assert path[r].tolist() == want + [-1] * (p.shape[1] - len(want)), r
        assert count[r] == len(want) and nxt[r] == x, (r, nxt[r], x)
    assert flags == 0
    return count


@pytest.mark.parametrize("sampled", [True, False])
@pytest.mark.parametrize("b,t,v", [(1, 1, 1), (1, 2, 2), (3, 5, 3), (1, 5, 127), (2, 4, 129), (4, 7, 1000), (2, 3, 4099),
                                   (1, 4, 50001), (300, 2, 517), (1, 64, 96)])
def test_sizes(b, t, v, sampled):
    check(*case(b + t + v, b, t, v, 1 if sampled else 4, sampled))


def test_long_paths_are_reached():
    counts = check(*case(5, 64, 9, 257, 1, True, ragged=False))
    assert counts.max() >= 6
    counts = check(*case(6, 64, 20, 8, 6, False, ragged=False))
    assert counts.max() >= 4


@pytest.mark.parametrize("base,dbase", [(0, 1), (1, 1), (2, 3), (3, 0)])
def test_unaligned_rows(base, dbase):
    check(*case(7, 3, 4, 1003, 1, True), base=base, dbase=dbase)


def test_largest_vocabulary():
    check(*case(8, 1, 2, 1 << 18, 1, True))
    with pytest.raises(abi.OscarError) as e:
        z = torch.zeros((1, 1, (1 << 18) + 1), device="cuda")
        i = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
        f = torch.zeros((1, 1), device="cuda")
        abi.verify_draft(z, i, i - 1, f, f[0], i.clone(), i[0].clone(), i[0].clone())
    assert e.value.status == -5


def test_children_that_repeat_a_token():
    # the same token under one node twice counts once, and is drawn at most from one of them
    p = np.zeros((1, 4, 4), np.float32)
    p[0, 0] = [0.25, 0.25, 0.25, 0.25]
    p[0, 1:] = [0.5, 0.5, 0, 0]
    par, tok = np.array([[-1, 0, 0, 0]]), np.array([[0, 2, 2, 1]])
    for u, path, nxt in ((0.2, [0, 1], 0), (0.3, [0, 3], 0), (0.49, [0, 3], 0), (0.51, [0], 0), (0.99, [0], 0)):
        got = run(p, None, tok, par, None, np.full((1, 4), u), np.array([0.1]))
        assert got[0][0, :len(path)].tolist() == path and got[1][0] == len(path) and got[2][0] == nxt
    # the weights left after refusal: tokens 0 and 3
    assert run(p, None, tok, par, None, np.full((1, 4), 0.9), np.array([0.6]))[2][0] == 3


def test_uniform_numbers_at_their_ends():
    p = np.zeros((1, 2, 5), np.float32)
    p[0, 0] = [0, 0.5, 0, 0.5, 0]
    p[0, 1] = [0, 0, 1, 0, 0]
    par, tok = np.array([[-1, 0]]), np.array([[0, 0]])    # a child of mass 0 is never taken
    below = np.nextafter(np.float32(1), np.float32(0))
    for us, x in ((0.0, 1), (0.4999, 1), (0.5, 3), (below, 3), (1.0, 3), (2.0, 3), (-1.0, 1), (np.nan, 1)):
        got = run(p, None, tok, par, None, np.zeros((1, 2)), np.array([us]))
        assert got[1][0] == 1 and got[2][0] == x, us
    for ua in (0.0, below, 1.0, np.nan):
        got = run(p, None, tok, par, None, np.full((1, 2), ua), np.array([0.1]))
        assert got[1][0] == 1
    # with draft probabilities: p equal to q is always accepted for u < 1
    got = run(p, p, np.array([[0, 3]]), par, None, np.full((1, 2), below), np.array([0.1]))
    assert got[0][0].tolist() == [0, 1] and got[2][0] == 2


def test_weights_that_vanish():
    p = np.zeros((3, 2, 6), np.float32)
    p[:, 0, 4] = 1.0
    par, tok = np.array([[-1, 0]] * 3), np.array([[0, 4]] * 3)
    q = p.copy()
    # refused although p = q there (u = 1): no residual, the target's own distribution is used
    got = run(p, q, tok, par, None, np.ones((3, 2)), np.full(3, 0.3))
    assert got[1].tolist() == [1, 1, 1] and got[2].tolist() == [4, 4, 4] and got[3] == 0
    # no probability at all: no token, and a flag
    got = run(np.zeros_like(p), None, tok, par, np.array([1, 2, 2]), np.ones((3, 2)), np.full(3, 0.3))
    assert got[2].tolist() == [-1, -1, -1] and got[3] == abi.FLAG_BAD_TREE
    nan = np.full_like(p, np.nan)
    nan[:, 0, 2] = 0.25
    got = run(nan, None, tok, par, None, np.full((3, 2), 0.9), np.full(3, 0.5))
    assert got[2].tolist() == [2, 2, 2] and got[3] == 0


def test_bad_requests_and_empty_drafts():
    p, q, tok, par, used, ua, us = case(9, 6, 4, 100, 2, False, ragged=False)
    good = run(p, None, tok, par, used, ua, us)
    for change in (("par", (0, 0), 0), ("par", (1, 2), 2), ("par", (1, 3), -1), ("tok", (2, 1), 100), ("tok", (2, 1), -1),
                   ("used", (3,), 5), ("used", (3,), -2)):
        a = {"par": par.copy(), "tok": tok.copy(), "used": used.copy()}
        a[change[0]][change[1]] = change[2]
        path, count, nxt, flags = run(p, None, a["tok"], a["par"], a["used"], ua, us)
        r = change[1][0]
        assert flags == abi.FLAG_BAD_TREE and count[r] == 0 and nxt[r] == -1 and (path[r] == -1).all()
        others = [i for i in range(6) if i != r]
        assert (count[others] == good[1][others]).all() and (nxt[others] == good[2][others]).all()
    a = used.copy()
    a[4] = 0
    path, count, nxt, flags = run(p, None, tok, par, a, ua, us)
    assert flags == 0 and count[4] == 0 and nxt[4] == -1 and (path[4] == -1).all()
    # a second child needs the draft's distribution without the first: refused
    star = np.array([[-1, 0, 0, 1]] * 6)
    path, count, nxt, flags = run(p, p.copy(), tok, star, used, ua, us)
    assert flags == abi.FLAG_BAD_TREE and (count == 0).all()


def test_the_result_is_distributed_like_the_target():
    # over a grid of uniform numbers the first token after node 0 (the accepted child's, or the
    # one drawn) has the target's distribution; each of the n grid cells can be off by one
    # border per axis, so a token's share is off by at most 2 / n per axis and token
    v, n = 6, 100
    rng = np.random.default_rng(3)
    p0 = rng.dirichlet(np.ones(v)).astype(np.float32)
    q0 = rng.dirichlet(np.ones(v)).astype(np.float32)
    grid = ((np.arange(n) + 0.5) / n).astype(np.float32)
    ua, us = (x.reshape(-1) for x in np.meshgrid(grid, grid))
    b = n * n
    p = np.broadcast_to(p0, (b, 4, v)).copy()
    par, tok = np.tile([-1, 0, 0, 0], (b, 1)), np.tile([0, 3, 1, 3], (b, 1))
    path, count, nxt, _ = run(p, None, tok, par, None, np.repeat(ua[:, None], 4, 1), us)
    first = np.where(count > 1, tok[np.arange(b), path[:, 1]], nxt)
    assert np.abs(np.bincount(first, minlength=v) / b - p0).max() <= 4 / n
    # chain: the child's token is drawn from q
    total = np.zeros(v)
    q = np.broadcast_to(q0, (b, 2, v)).copy()
    for x in range(v):
        path, count, nxt, _ = run(p[:, :2].copy(), q, np.tile([0, x], (b, 1)), np.tile([-1, 0], (b, 1)), None,
                                  np.repeat(ua[:, None], 2, 1), us)
        first = np.where(count > 1, x, nxt)
        total += q0[x] * np.bincount(first, minlength=v) / b
    assert np.abs(total - p0).max() <= 4 / n


def test_captured_and_replayed():
    b, t, v = 2, 5, 3001
    inputs = [case(20 + s, b, t, v, 3, False, ragged=False) for s in range(2)]
    bufs = [torch.from_numpy(np.ascontiguousarray(x)).cuda() for x in
            (inputs[0][0], inputs[0][2], inputs[0][3], inputs[0][5], inputs[0][6])]
    path = torch.zeros((b, t), dtype=torch.int32, device="cuda")
    count, nxt = (torch.zeros(b, dtype=torch.int32, device="cuda") for _ in range(2))
    call = lambda: abi.verify_draft(bufs[0], bufs[1], bufs[2], bufs[3], bufs[4], path, count, nxt)  # noqa: E731
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for c in inputs:
        for buf, x in zip(bufs, (c[0], c[2], c[3], c[5], c[6])):
            buf.copy_(torch.from_numpy(np.ascontiguousarray(x)))
        graph.replay()
        torch.cuda.synchronize()
        for r in range(b):
            want, x = reference(c[0][r], None, c[2][r], c[3][r], t, c[5][r], c[6][r])
            assert path[r].tolist()[:len(want)] == want and int(count[r]) == len(want) and int(nxt[r]) == x
