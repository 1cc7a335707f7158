"""Cases and plain forms of the speculative-decoding operators.

One round of speculative decoding over an OSCAR cache is four operators:

  qkv_norm_rope  the layer's fused q / k / v projection split into q, k and v, with a
                 root-mean-square norm of every q and k head and the position rotation
  tree_attn      attention of a tree of drafted tokens over the paged INT2 cache, the
                 BF16 sink and recent tokens and the tree's own keys and values
  verify_draft   which drafted tokens the target accepts, and the token sampled after them
  commit_draft   the accepted tokens' keys and values appended to the cache (sink, ring,
                 and the ring entries that leave it rotated, clipped and quantised)

`run` computes them in elementary torch operations, or with `own` set through the
library. `exact` gives the same results from the definitions in 64 bits.
"""

from __future__ import annotations

import math

import numpy as np
import torch

own = False

D, PAGE = 128, 16
DEV = "cuda"


# ---------------------------------------------------------------------------- cases
def listed():
    return [
        # one chat request in the middle of its answer, a chain of 4 guesses after the last token
        {"name": "tree_bs1_4k_chain5", "op": "tree_attn", "batch": 1, "hq": 32, "hkv": 8, "lo": 4099, "hi": 4099,
         "sink": 4, "recent": 128, "group": 32, "nodes": 5, "width": 1, "ragged": False},
        # one long document, a wide tree
        {"name": "tree_bs1_32k_tree26", "op": "tree_attn", "batch": 1, "hq": 32, "hkv": 8, "lo": 32768, "hi": 32768,
         "sink": 4, "recent": 128, "group": 32, "nodes": 26, "width": 4, "ragged": False},
        # a serving batch of unequal requests, small trees of unequal size
        {"name": "tree_bs16_ragged_tree8", "op": "tree_attn", "batch": 16, "hq": 32, "hkv": 8, "lo": 8192, "hi": 32768,
         "sink": 4, "recent": 128, "group": 32, "nodes": 8, "width": 2, "ragged": True},
        # the long-context batch of the benchmark with short chains
        {"name": "tree_bs28_100k_chain4", "op": "tree_attn", "batch": 28, "hq": 64, "hkv": 8, "lo": 100000,
         "hi": 100000, "sink": 4, "recent": 128, "group": 32, "nodes": 4, "width": 1, "ragged": False},
        # the method's own constants with the widest trees: 488 query rows for each cache head
        {"name": "tree_bs8_16k_g64_tree61", "op": "tree_attn", "batch": 8, "hq": 64, "hkv": 8, "lo": 16001, "hi": 16001,
         "sink": 64, "recent": 256, "group": 64, "nodes": 61, "width": 3, "ragged": False},
        # one request: a sampled chain against the draft's own distributions
        {"name": "verify_bs1_chain5_sampled", "op": "verify_draft", "batch": 1, "nodes": 5, "width": 1, "vocab": 151936,
         "sampled": True, "ragged": False},
        # a batch of wide trees, children fixed by the draft model's best guesses
        {"name": "verify_bs64_tree26", "op": "verify_draft", "batch": 64, "nodes": 26, "width": 4, "vocab": 151936,
         "sampled": False, "ragged": True},
        # many requests, an odd vocabulary (rows that are not 16-byte aligned)
        {"name": "verify_bs256_chain5_odd", "op": "verify_draft", "batch": 256, "nodes": 5, "width": 1, "vocab": 32003,
         "sampled": True, "ragged": True},
        # one request's accepted chain
        {"name": "commit_bs1_chain5", "op": "commit_draft", "batch": 1, "hkv": 8, "lo": 4099, "hi": 4099, "sink": 4,
         "recent": 128, "group": 32, "nodes": 5},
        # a serving batch of accepted paths of unequal length
        {"name": "commit_bs64_g64_tree16", "op": "commit_draft", "batch": 64, "hkv": 8, "lo": 300, "hi": 2100,
         "sink": 64, "recent": 256, "group": 64, "nodes": 16},
        # the single token of a plain decode step, far into its context
        {"name": "rope_1_token", "op": "qkv_norm_rope", "tokens": 1, "hq": 32, "hkv": 8, "rotary": 128,
         "interleaved": False, "norm": True, "pad": 0, "far": 131072},
        # a long prompt, the projection's rows padded
        {"name": "rope_prompt_32769", "op": "qkv_norm_rope", "tokens": 32769, "hq": 64, "hkv": 8, "rotary": 128,
         "interleaved": False, "norm": True, "pad": 64, "far": 131072},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tree_attn", "tree_attn", "verify_draft", "commit_draft", "qkv_norm_rope"])
    if op == "qkv_norm_rope":
        hkv = rng.choice([1, 2, 4, 8])
        return {"op": op, "tokens": _log(rng, 1, 32768), "hq": hkv * rng.choice([1, 2, 4, 8]), "hkv": hkv,
                "rotary": rng.choice([32, 64, 96, 128]), "interleaved": rng.random() < 0.5,
                "norm": rng.random() < 0.75, "pad": rng.choice([0, 8, 64]), "far": _log(rng, 64, 1 << 20)}
    nodes = rng.randint(1, 64)
    if op == "verify_draft":
        sampled = rng.random() < 0.5
        vocab = rng.randint(1000, 152000)
        nodes = min(nodes, 26)
        return {"op": op, "batch": _log(rng, 1, max(1, min(256, int(2.5e8) // (nodes * vocab)))), "nodes": nodes,
                "width": 1 if sampled else rng.randint(1, 5), "vocab": vocab, "sampled": sampled,
                "ragged": rng.random() < 0.5}
    preset = rng.random() < 0.5
    sink, recent, group = (64, 256, 64) if preset else (4, 128, 32)
    hkv = rng.choice([1, 2, 4, 8])
    if op == "commit_draft":
        hi = _log(rng, 16, 8000)
        return {"op": op, "batch": _log(rng, 1, 64), "hkv": hkv, "lo": rng.randint(0, hi), "hi": hi, "sink": sink,
                "recent": recent, "group": group, "nodes": min(nodes, 16)}
    hq = hkv * rng.choice([1, 2, 4, 8])
    batch = _log(rng, 1, 16)
    most = int(2.0e9) // (batch * hq * nodes)            # query rows x positions of the largest listed cases
    hi = _log(rng, 64, min(100000, max(65, most), 400000 // batch))
    lo = rng.randint(0, hi) if rng.random() < 0.5 else hi
    return {"op": op, "batch": batch, "hq": hq, "hkv": hkv, "lo": lo, "hi": hi, "sink": sink, "recent": recent,
            "group": group, "nodes": nodes, "width": rng.randint(1, 5), "ragged": rng.random() < 0.5}


def _lengths(case, seed):
    """Cached tokens of every request: uniform in [lo, hi]."""
    r = np.random.RandomState(seed % (1 << 31))
    return r.randint(case["lo"], case["hi"] + 1, case["batch"])


def work(case):
    op = case["op"]
    if op == "qkv_norm_rope":
        n, heads = case["tokens"], case["hq"] + 2 * case["hkv"]
        return {"bytes": 2 * n * heads * D * 2 + 4 * n, "flops": 10 * n * (case["hq"] + case["hkv"]) * D}
    if op == "verify_draft":
        # the row of the last accepted node (with the draft's row beside it), and the drafted tokens' entries
        rows = case["batch"] * (2 if case["sampled"] else 1)
        return {"bytes": rows * case["vocab"] * 4 + case["batch"] * case["nodes"] * 20,
                "flops": 2 * rows * case["vocab"]}
    mean = (case["lo"] + case["hi"]) / 2
    ng = D // case["group"]
    token = 64 + 8 * ng                              # codes and metadata of one cached token of one head
    if op == "commit_draft":
        n = case["batch"] * case["hkv"] * (case["nodes"] + 1) / 2
        return {"bytes": n * (512 * 3 + token) + 2 * case["hkv"] * D * D * 4, "flops": n * 4 * D * D}
    win = min(mean, case["sink"] + case["recent"])
    keys = case["batch"] * case["hkv"]
    rows = case["nodes"] * case["hq"] // case["hkv"]
    return {"bytes": keys * ((mean - win) * token + (win + case["nodes"]) * 512 + 2 * rows * D * 2),
            "flops": keys * rows * (mean + case["nodes"] / 2) * 4 * D}


# ------------------------------------------------------------------------ preparation
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 7919 + 17)
    return g


def _parents(case, seed):
    """Parents of every request's tree, node 0 the last sampled token: each further node hangs on one of
    the `width` nodes before it (width 1: a chain); and how many of the nodes the request uses."""
    r = np.random.RandomState((seed + 1) % (1 << 31))
    b, t = case["batch"], case["nodes"]
    parent = np.full((b, t), -1, np.int32)
    for i in range(1, t):
        parent[:, i] = np.maximum(0, i - 1 - r.randint(0, case.get("width", 1), b))
    used = r.randint(1, t + 1, b) if case.get("ragged") else np.full(b, t)
    return torch.from_numpy(parent).to(DEV), torch.from_numpy(used.astype(np.int32)).to(DEV)


def _cache(case, seed, g, headroom):
    """A paged cache as a request's prompt leaves it: random 2-bit codes, scales and zeros of the size that
    rotated activations have, BF16 window rows, shuffled pages, random orthogonal rotations."""
    b, hkv, sink, recent, group = (case[k] for k in ("batch", "hkv", "sink", "recent", "group"))
    ng = D // group
    lens = _lengths(case, seed)
    pages = (int(case["hi"]) + headroom + PAGE - 1) // PAGE
    num = b * pages
    block = 1024 + 128 * ng
    pool = torch.randint(-2 ** 31, 2 ** 31 - 1, (num * hkv * block // 4,), dtype=torch.int32, device=DEV, generator=g)
    half = pool.view(torch.float16).view(num, hkv, block // 2)

    def meta(n, sign):
        u = torch.rand((num, hkv, n), device=DEV, generator=g)
        return (u * 0.8 + 2.0 if sign else -(u * 2.0 + 5.0)).to(torch.float16)
    half[:, :, 512:512 + 16 * ng] = meta(16 * ng, True)                                # K scales
    half[:, :, 512 + 16 * ng:512 + 32 * ng] = meta(16 * ng, False)                     # K zeros
    vm = half[:, :, 512 + 32 * ng:].view(num, hkv, 4 * ng, 2, 4)
    vm[:, :, :, 0] = meta(16 * ng, True).view(num, hkv, 4 * ng, 4)
    vm[:, :, :, 1] = meta(16 * ng, False).view(num, hkv, 4 * ng, 4)
    window = torch.randn((b, hkv, 2, sink + recent, D), device=DEV, generator=g)
    window[..., :4] *= 20.0                                                            # outlier channels
    window = window.to(torch.bfloat16)
    table = torch.randperm(num, device=DEV, generator=g).to(torch.int32).view(b, pages)
    state = np.zeros((b, 4), np.int32)
    state[:, 0] = lens
    state[:, 1] = np.maximum(sink, lens - recent)
    state[:, 2] = np.arange(b)[::-1]
    rot = torch.linalg.qr(torch.randn((2, hkv, D, D), device=DEV, generator=g, dtype=torch.float64))[0]
    rot = rot.to(torch.float32).contiguous()
    clip = torch.full((2, hkv), 12.0, device=DEV)
    return {"pool": pool, "pages": num, "window": window, "table": table, "lens": lens,
            "state": torch.from_numpy(state).to(DEV), "rot": rot, "clip": clip}


def _context(case, s, hq):
    """The library's context with the same cache and rotations."""
    from bit_rotated_kv_oscar_gb300 import abi
    cfg = abi.make_config(hq, case["hkv"], case["sink"], case["recent"], case["batch"], s["table"].shape[1],
                          group_size=case["group"])
    ctx = abi.Context(cfg)
    ctx.bind_cache(s["pool"], s["pages"], s["window"])
    ctx.load_rotations(s["rot"][0].cpu().numpy(), s["rot"][1].cpu().numpy(), s["clip"][0].cpu().numpy(),
                       s["clip"][1].cpu().numpy())
    return ctx


def _prepare_tree(case, seed):
    g = _gen(seed)
    b, t, hq, hkv = case["batch"], case["nodes"], case["hq"], case["hkv"]
    s = _cache(case, seed, g, 0)
    s["parent"], s["used"] = _parents(case, seed)
    s["q"] = (torch.randn((b, t, hq, D), device=DEV, generator=g) * 0.3).to(torch.bfloat16)
    kv = torch.randn((2, b, t, hkv, D), device=DEV, generator=g)
    kv[..., :4] *= 20.0
    s["k"], s["v"] = kv.to(torch.bfloat16)
    s["o"] = torch.zeros((b, t, hq, D), dtype=torch.bfloat16, device=DEV)
    if own:
        s["ctx"] = _context(case, s, hq)
        s["ws"] = torch.empty(s["ctx"].tree_attn_workspace_bytes(b, t), dtype=torch.uint8, device=DEV)
    return s


def _prepare_verify(case, seed):
    g = _gen(seed)
    b, t, v = case["batch"], case["nodes"], case["vocab"]
    s = {}
    s["parent"], s["used"] = _parents(case, seed)
    logits = torch.randn((b, t, v), device=DEV, generator=g) * 3.0
    s["p"] = torch.softmax(logits, -1)
    # the draft model: the target's logits with an error of its own
    logits += torch.randn((b, t, v), device=DEV, generator=g) * 0.7
    par = s["parent"].long().clamp(min=0)
    rows = torch.arange(b, device=DEV)[:, None]
    tokens = torch.zeros((b, t), dtype=torch.int64, device=DEV)
    if case["sampled"]:
        qd = torch.softmax(logits, -1)
        drawn = torch.multinomial(qd.view(b * t, v), 1, generator=g).view(b, t)
        tokens[:, 1:] = drawn[rows, par[:, 1:]]                  # a chain: one child for each node
        s["qd"] = qd
    else:
        # the n-th child of a node is the draft's n-th best guess there
        best = torch.topk(logits, min(t, v), -1).indices
        same = (par[:, None, :] == par[:, :, None]) & (torch.arange(t, device=DEV)[:, None] > torch.arange(t, device=DEV))
        same[:, :, 0] = False
        rank = same.sum(-1)
        tokens[:, 1:] = best[rows, par[:, 1:], rank[:, 1:]]
        s["qd"] = None
    del logits
    s["tokens"] = tokens.to(torch.int32)
    s["ua"] = torch.rand((b, t), device=DEV, generator=g)
    s["us"] = torch.rand((b,), device=DEV, generator=g)
    if own:
        s["path"] = torch.empty((b, t), dtype=torch.int32, device=DEV)
        s["count"] = torch.empty((b,), dtype=torch.int32, device=DEV)
        s["next"] = torch.empty((b,), dtype=torch.int32, device=DEV)
    return s


def _prepare_commit(case, seed):
    g = _gen(seed)
    b, t, hkv = case["batch"], case["nodes"], case["hkv"]
    s = _cache(case, seed, g, t)
    s["state0"] = s["state"].clone()
    kv = torch.randn((2, b, t, hkv, D), device=DEV, generator=g)
    kv[..., :4] *= 20.0
    s["k"], s["v"] = kv.to(torch.bfloat16)
    r = np.random.RandomState((seed + 2) % (1 << 31))
    count = r.randint(1, t + 1, b)
    path = np.full((b, t), -1, np.int32)
    for i in range(b):                                  # node 0 and some of the others, in order
        path[i, 1:count[i]] = 1 + np.sort(r.permutation(t - 1)[:count[i] - 1])
        path[i, 0] = 0
    s["path"], s["count"] = torch.from_numpy(path).to(DEV), torch.from_numpy(count.astype(np.int32)).to(DEV)
    if own:
        s["ctx"] = _context(case, s, hkv)
    return s


def _prepare_rope(case, seed):
    g = _gen(seed)
    n, hq, hkv = case["tokens"], case["hq"], case["hkv"]
    width = (hq + 2 * hkv) * D
    s = {"qkv": torch.randn((n, width + case["pad"]), device=DEV, generator=g).to(torch.bfloat16)[:, :width]}
    s["wq"] = (1 + 0.2 * torch.randn(D, device=DEV, generator=g)).to(torch.bfloat16) if case["norm"] else None
    s["wk"] = (1 + 0.2 * torch.randn(D, device=DEV, generator=g)).to(torch.bfloat16) if case["norm"] else None
    s["pos"] = torch.randint(0, case["far"], (n,), device=DEV, generator=g, dtype=torch.int32)
    s["inv_freq"] = 1e6 ** (-np.arange(0, case["rotary"], 2, dtype=np.float64) / case["rotary"])
    s["freq"] = torch.from_numpy(s["inv_freq"]).to(DEV)
    if own:
        from bit_rotated_kv_oscar_gb300 import abi
        s["turns"] = abi.rope_turns(s["inv_freq"]).to(DEV)
        s["q"] = torch.empty((n, hq, D), dtype=torch.bfloat16, device=DEV)
        s["k"] = torch.empty((n, hkv, D), dtype=torch.bfloat16, device=DEV)
        s["v"] = torch.empty((n, hkv, D), dtype=torch.bfloat16, device=DEV)
    return s


_PREPARE = {"tree_attn": _prepare_tree, "verify_draft": _prepare_verify, "commit_draft": _prepare_commit,
            "qkv_norm_rope": _prepare_rope}


def prepare(case, seed):
    torch.backends.cuda.matmul.allow_tf32 = False
    s = _PREPARE[case["op"]](case, seed)
    s["case"] = case
    return s


# -------------------------------------------------------------------------- plain forms
def _ancestors(parent, used):
    """[b, t, t] whether node j is node i or above it, among the used nodes."""
    b, t = parent.shape
    up = torch.nn.functional.one_hot(parent.long().clamp(min=0), t).float() * (parent >= 0).float()[..., None]
    reach = up + torch.eye(t, device=parent.device)
    for _ in range(max(1, (t - 1).bit_length())):
        reach = ((reach @ reach) > 0).float()
    live = torch.arange(t, device=parent.device) < used[:, None]
    return (reach > 0) & live[:, :, None] & live[:, None, :]


def _codes(words, value):
    """2-bit codes [..., 16 tokens, 128 channels] of the packed words [..., 128] (int32) of a block's keys or values."""
    lead = words.shape[:-1]
    w = words.view(lead + (8, 4, 2, 2, 1, 1))                         # a, b, token half or pair, x
    hi = torch.tensor([0, 16], dtype=torch.int32, device=words.device).view(2, 1)
    i = torch.arange(8, dtype=torch.int32, device=words.device) * 2
    c = (w >> (hi + i)) & 3                                           # a, b, th, x, hi, i
    n = len(lead)
    order = (2, 1, 4, 5, 3, 0) if value else (2, 0, 5, 3, 1, 4)
    return c.permute(tuple(range(n)) + tuple(n + k for k in order)).reshape(lead + (PAGE, D))


def _dequant(blocks, ng, dtype):
    """Keys and values [n, h, 16, 128] that page blocks [n, h, words] stand for, in the rotated bases."""
    lead = blocks.shape[:-1]
    m = blocks[..., 256:].contiguous().view(torch.float16).to(dtype)
    ks = m[..., :16 * ng].reshape(lead + (8, ng, 2)).permute(0, 1, 4, 2, 3).reshape(lead + (PAGE, ng, 1))
    kz = m[..., 16 * ng:32 * ng].reshape(lead + (PAGE, ng, 1))
    vm = m[..., 32 * ng:].reshape(lead + (ng, 4, 2, 2, 2)).permute(0, 1, 4, 5, 3, 6, 2)
    vm = vm.reshape(lead + (2, PAGE, ng, 1))
    kc = _codes(blocks[..., :128].contiguous(), False).view(lead + (PAGE, ng, D // ng))
    vc = _codes(blocks[..., 128:256].contiguous(), True).view(lead + (PAGE, ng, D // ng))
    k = (kc * ks + kz).view(lead + (PAGE, D))
    v = (vc * vm[:, :, 0] + vm[:, :, 1]).view(lead + (PAGE, D))
    return k, v


def _plain_tree(s):
    case = s["case"]
    b, t, hq, hkv, sink, recent = (case[k] for k in ("batch", "nodes", "hq", "hkv", "sink", "recent"))
    g = hq // hkv
    blocks = s["pool"].view(s["pages"], hkv, -1)[s["table"].long().view(-1)]          # [b pages, hkv, words]
    pages = s["table"].shape[1]
    k2, v2 = _dequant(blocks, D // case["group"], torch.float32)
    k2, v2 = (x.view(b, pages, hkv, PAGE, D).transpose(1, 2).reshape(b, hkv, pages * PAGE, D) for x in (k2, v2))
    del blocks
    q = s["q"].float().view(b, t, hkv, g, D).permute(0, 2, 1, 3, 4).reshape(b, hkv, t * g, D)
    L, E, row = (s["state"][:, i].long() for i in (0, 1, 2))
    win = s["window"][row].float()                                                    # [b, hkv, 2, S + W, D]
    kd, vd = (s[x].float().transpose(1, 2) for x in "kv")                             # [b, hkv, t, D]
    # positions of the window rows: the sink, then for each ring row the one position in [E, L) it holds
    slot = torch.arange(sink + recent, device=DEV)
    first = torch.maximum(E, torch.tensor(sink, device=DEV))[:, None]
    ring = first + (slot - sink - first) % recent
    in_win = torch.where(slot < sink, slot < L[:, None], ring < L[:, None])
    pos = torch.arange(pages * PAGE, device=DEV)
    in_int2 = (pos >= sink) & (pos < torch.minimum(E, L)[:, None])
    mask = _ancestors(s["parent"], s["used"]).repeat_interleave(g, 1)                 # [b, t g, t]
    qr = q @ s["rot"][0]
    sc = torch.cat([(qr @ k2.transpose(2, 3)).masked_fill_(~in_int2[:, None, None], -math.inf),
                    (q @ win[:, :, 0].transpose(2, 3)).masked_fill_(~in_win[:, None, None], -math.inf),
                    (q @ kd.transpose(2, 3)).masked_fill_(~mask[:, None], -math.inf)], -1)
    del k2
    sc *= D ** -0.5
    top = sc.max(-1, keepdim=True).values.clamp(min=-3e38)                            # rows of unused nodes: none
    sc.sub_(top).exp_()
    total = sc.sum(-1, keepdim=True).clamp(min=1e-30)
    n2, nw = pages * PAGE, sink + recent
    o = (sc[..., :n2] @ v2) @ s["rot"][1].transpose(1, 2)
    o += sc[..., n2:n2 + nw] @ win[:, :, 1] + sc[..., n2 + nw:] @ vd
    o /= total
    o = o.view(b, hkv, t, g, D).permute(0, 2, 1, 3, 4).reshape(b, t, hq, D).to(torch.bfloat16)
    used = torch.arange(t, device=DEV) < s["used"][:, None]
    return torch.where(used[:, :, None, None], o, s["o"])                             # other rows stay as they were


def _plain_verify(s):
    case = s["case"]
    b, t, v = case["batch"], case["nodes"], case["vocab"]
    rows = torch.arange(b, device=DEV)
    par, tok = s["parent"].long(), s["tokens"].long()
    live = torch.arange(t, device=DEV) < s["used"].long()[:, None]
    pc = par.clamp(min=0)
    p_tok = s["p"][rows[:, None], pc, tok].double()                                   # the target's mass of each node's token
    node = torch.zeros(b, dtype=torch.long, device=DEV)
    path = torch.full((b, t), -1, dtype=torch.int32, device=DEV)
    path[:, 0] = 0
    count = torch.ones(b, dtype=torch.int32, device=DEV)
    going = torch.ones(b, dtype=torch.bool, device=DEV)
    idx = torch.arange(t, device=DEV)
    earlier = (tok[:, :, None] == tok[:, None, :]) & (idx[:, None] > idx)             # [b, i, j < i] the same token
    # a sibling's token counted once: nodes that repeat an earlier child of the same parent add nothing
    again = (earlier & (par[:, :, None] == par[:, None, :]) & (idx > 0)).any(-1)
    for d in range(1, t):
        child = (par == node[:, None]) & live & (idx > 0)
        u = s["ua"].double()[rows, node]
        if s["qd"] is not None:
            q_tok = s["qd"][rows[:, None], pc, tok].double()
            good = child & (u[:, None] * q_tok < p_tok)
        else:
            mass = torch.where(child & ~again, p_tok, 0.0).cumsum(-1)
            good = child & ~again & (u[:, None] < mass)
        hit = going & good.any(-1)
        first = torch.where(good, idx, t).min(-1).values.clamp(max=t - 1)
        node = torch.where(hit, first, node)
        path[:, d] = torch.where(hit, node.int(), -1)
        count += hit.int()
        going = hit
    # the weights the next token is drawn from: the last node's distribution, less what was refused there
    w = s["p"][rows, node].double()
    child = (par == node[:, None]) & live & (idx > 0)
    if s["qd"] is not None:
        w = torch.where(child.any(-1, keepdim=True), (w - s["qd"][rows, node].double()).clamp(min=0), w)
    else:
        out = torch.zeros((b, v + 1), dtype=torch.bool, device=DEV)
        out.scatter_(1, torch.where(child, tok, v), True)
        w = w.masked_fill(out[:, :v], 0.0)
    run_ = w.cumsum(-1)
    past = run_ > s["us"].double()[:, None] * run_[:, -1:]
    at = torch.arange(v, device=DEV)
    nxt = torch.where(past & (w > 0), at, v).min(-1).values
    return {"path": path, "count": count, "next": nxt.int()}


def _rotate32(x, rot):
    """x rot as the write path defines it: two sums of 64 products each, every product added with one
    rounding to 32 bits, and then the two added. A code next to a rounding border depends on this order,
    so it is kept: each step's exact sum in 64 bits, rounded to 32."""
    lo = torch.zeros(x.shape, device=DEV)
    hi = torch.zeros(x.shape, device=DEV)
    x, rot = x.double(), rot.double()
    for i in range(D // 2):
        lo = (x[..., i:i + 1] * rot[:, i] + lo).float()
        hi = (x[..., i + 64:i + 65] * rot[:, i + 64] + hi).float()
    return lo + hi


def _plain_commit(s):
    case = s["case"]
    b, t, hkv, sink, recent, group = (case[k] for k in ("batch", "nodes", "hkv", "sink", "recent", "group"))
    ng = D // group
    s["state"].copy_(s["state0"])
    L, E, row = (s["state"][:, i].long()[:, None] for i in (0, 1, 2))                 # [b, 1]
    n = s["count"].long()[:, None]
    E2 = torch.maximum(torch.maximum(E, L + n - recent), torch.tensor(sink, device=DEV))
    j = torch.arange(t, device=DEV)[None]
    path = s["path"].long().clamp(min=0)
    new = torch.stack([s["k"], s["v"]], 3)[torch.arange(b, device=DEV)[:, None], path]  # [b, t, hkv, 2, D]
    # positions E + j < E2 go to INT2: from the ring while cached, else straight from the accepted rows
    pos = E + j
    rot_on = pos < E2
    old = s["window"][row, :, :, (sink + pos % recent)]                               # [b, t, hkv, 2, D]
    src = torch.where((pos < L)[..., None, None, None], old,
                      new.gather(1, (pos - L).clamp(0, t - 1)[..., None, None, None].expand_as(new)))
    x = _rotate32(src.transpose(2, 3), s["rot"][0]), _rotate32(src.transpose(2, 3), s["rot"][1])
    x = torch.stack([x[0][:, :, 0], x[1][:, :, 1]], 2)                                # [b, t, 2, hkv, D]
    clip = s["clip"][:, :, None]
    xg = torch.minimum(torch.maximum(x, -clip), clip).view(b, t, 2, hkv, ng, group)
    mn, mx = xg.amin(-1), xg.amax(-1)
    s16, z16 = ((mx - mn) / 3).half(), mn.half()
    sf, zf = s16.float()[..., None], z16.float()[..., None]
    code = torch.where(sf == 0, 0.0, ((xg - zf) * (1 / sf)).round().clamp(0, 3)).int().view(b, t, 2, hkv, 8, 2, 8)
    bits = (code << (2 * torch.arange(8, device=DEV, dtype=torch.int32)).view(8, 1, 1)).sum(4)  # [b, t, 2, hkv, x, 8]
    # where each token's half-words lie in its block
    a, half, quad = pos % 8, (pos % PAGE) // 8, (pos % 8) // 2
    x_, r = torch.arange(2, device=DEV)[:, None], torch.arange(8, device=DEV)
    at_k = (8 * (4 * a[..., None, None] + r // 2) + 2 * (2 * half[..., None, None] + x_) + r % 2).expand(b, t, 2, 8)
    at_v = 256 + 8 * (4 * r + quad[..., None, None]) + 2 * (2 * half[..., None, None] + x_) + (pos % 2)[..., None, None]
    gq = torch.arange(ng, device=DEV)
    at_ks = 512 + 2 * ng * a[..., None] + 2 * gq + half[..., None]
    at_kz = 512 + 16 * ng + ng * (pos % PAGE)[..., None] + gq
    at_vs = 512 + 32 * ng + 8 * (4 * gq + quad[..., None]) + 2 * half[..., None] + (pos % 2)[..., None]
    at = torch.cat([at_k.flatten(2), at_v.flatten(2), at_ks, at_kz, at_vs, at_vs + 4], -1)
    to16 = lambda h: h.contiguous().view(torch.int16)  # noqa: E731
    val = torch.cat([bits[:, :, 0].flatten(3).to(torch.int16), bits[:, :, 1].flatten(3).to(torch.int16),
                     to16(s16[:, :, 0]), to16(z16[:, :, 0]), to16(s16[:, :, 1]), to16(z16[:, :, 1])], -1)
    table = s["table"].long()
    page = table.gather(1, (pos // PAGE).clamp(max=table.shape[1] - 1))
    size = 512 + 64 * ng
    flat = ((page[..., None, None] * hkv + torch.arange(hkv, device=DEV)[:, None]) * size + at[:, :, None])
    pool = s["pool"].view(torch.int16)
    on = rot_on[:, :, None, None].expand_as(flat)
    pool[flat[on]] = val[on]
    # the window: sink positions and those that stay in the ring
    q = L + j
    keep = (j < n) & ((q < sink) | (q >= E2))
    slot = torch.where(q < sink, q, sink + q % recent)
    who = torch.nonzero(keep, as_tuple=True)
    s["window"][row.expand(b, t)[who], :, :, slot[who]] = new[who]
    s["state"][:, 0] += s["count"]
    s["state"][:, 1] = E2[:, 0].int()
    return {"pool": s["pool"], "window": s["window"], "state": s["state"]}


def _plain_rope(s):
    case = s["case"]
    n, hq, hkv, rot = (case[k] for k in ("tokens", "hq", "hkv", "rotary"))
    x = s["qkv"].float().view(n, hq + 2 * hkv, D)
    qk, v = x[:, :hq + hkv], x[:, hq + hkv:]
    if case["norm"]:
        w = torch.cat([s["wq"].float().expand(hq, D), s["wk"].float().expand(hkv, D)])
        qk = qk * torch.rsqrt(qk.square().mean(-1, keepdim=True) + 1e-6) * w
    angle = s["pos"].double()[:, None] * s["freq"]                                    # far positions need 64 bits
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    if case["interleaved"]:
        a, c = qk[..., 0:rot:2], qk[..., 1:rot:2]
        turned = torch.stack([a * cos - c * sin, c * cos + a * sin], -1).flatten(2)
    else:
        a, c = qk[..., :rot // 2], qk[..., rot // 2:rot]
        turned = torch.cat([a * cos - c * sin, c * cos + a * sin], -1)
    qk = torch.cat([turned, qk[..., rot:]], -1).to(torch.bfloat16)
    return {"q": qk[:, :hq], "k": qk[:, hq:], "v": v.to(torch.bfloat16)}


_PLAIN = {"tree_attn": _plain_tree, "verify_draft": _plain_verify, "commit_draft": _plain_commit,
          "qkv_norm_rope": _plain_rope}


def run(s):
    op = s["case"]["op"]
    if not own:
        return _PLAIN[op](s)
    from bit_rotated_kv_oscar_gb300 import abi
    if op == "tree_attn":
        s["ctx"].tree_attn(s["q"], s["k"], s["v"], s["parent"], s["table"], s["state"], s["o"], s["case"]["batch"],
                           s["case"]["nodes"], s["ws"], draft_len=s["used"])
        return s["o"]
    if op == "verify_draft":
        abi.verify_draft(s["p"], s["tokens"], s["parent"], s["ua"], s["us"], s["path"], s["count"], s["next"],
                         draft_probs=s["qd"], draft_len=s["used"])
        return {"path": s["path"], "count": s["count"], "next": s["next"]}
    if op == "commit_draft":
        s["state"].copy_(s["state0"])                                                 # every pass from the same lengths
        s["ctx"].commit_draft(s["table"], s["state"], s["k"], s["v"], s["path"], s["count"], s["case"]["batch"],
                              s["case"]["nodes"])
        return {"pool": s["pool"], "window": s["window"], "state": s["state"]}
    abi.qkv_norm_rope(s["qkv"], s["pos"], s["turns"], s["q"], s["k"], s["v"], q_weight=s["wq"], k_weight=s["wk"],
                      eps=1e-6, interleaved=s["case"]["interleaved"])
    return {"q": s["q"], "k": s["k"], "v": s["v"]}


# -------------------------------------------------------------------- definitions, in 64 bits
def _exact_tree(case, s):
    """Request by request: every cached key and value in its raw basis, then softmax attention of each node
    over the cache and its own ancestors."""
    b, t, hq, hkv, sink, recent, group = (case[k] for k in ("batch", "nodes", "hq", "hkv", "sink", "recent", "group"))
    g, ng = hq // hkv, D // group
    out = torch.zeros((b, t, hq, D), dtype=torch.float64, device=DEV)
    rot = s["rot"].double()
    c, tt = np.meshgrid(np.arange(D), np.arange(PAGE))
    kbit = 8 * (16 * (4 * (tt % 8) + (c % 8) // 2) + 4 * (2 * (tt // 8) + c % 16 // 8)) + 16 * (c % 2) + 2 * (c // 16)
    vbit = 8 * (16 * (4 * (c % 8) + tt % 8 // 2) + 4 * (2 * (tt // 8) + c % 16 // 8)) + 16 * (tt % 2) + 2 * (c // 16)
    gq = c // group
    kso = 4 * ng * (tt % 8) + 4 * gq + 2 * (tt // 8)
    kzo = 32 * ng + 2 * ng * tt + 2 * gq
    vso = 64 * ng + 16 * (4 * gq + tt % 8 // 2) + 4 * (tt // 8) + 2 * (tt % 2)
    dev = lambda x: torch.from_numpy(x.astype(np.int64)).to(DEV)  # noqa: E731
    bytes_ = s["pool"].view(torch.uint8).view(s["pages"], hkv, -1)
    state, parent, used = s["state"].cpu().numpy(), s["parent"].cpu().numpy(), s["used"].cpu().numpy()
    for r in range(b):
        n, e, row = (int(x) for x in state[r, :3])
        e2 = min(e, n)
        ks, vs = [], []
        w = s["window"][row].double()
        if n:
            ks.append(w[:, 0, :min(sink, n)])
            vs.append(w[:, 1, :min(sink, n)])
        if e2 > sink:
            blk = bytes_[s["table"][r, sink // PAGE:(e2 + PAGE - 1) // PAGE].long()]
            f16 = blk[..., 1024:].contiguous().view(torch.float16)
            for to, base, bit, so, zo, turn in ((ks, 0, kbit, kso, kzo, rot[0]), (vs, 512, vbit, vso, vso + 8, rot[1])):
                code = (blk[..., dev(base + bit // 8)] >> dev(bit % 8).to(torch.uint8)) & 3
                x = code.double() * f16[..., dev(so // 2)].double() + f16[..., dev(zo // 2)].double()
                x = x.transpose(0, 1).reshape(hkv, -1, D)[:, sink % PAGE:][:, :e2 - sink]
                to.append(x @ turn.transpose(1, 2))
        first = max(e, sink)
        if n > first:
            slots = sink + torch.arange(first, n, device=DEV) % recent
            ks.append(w[:, 0, slots])
            vs.append(w[:, 1, slots])
        ks.append(s["k"][r].double().transpose(0, 1))
        vs.append(s["v"][r].double().transpose(0, 1))
        kk, vv = torch.cat(ks, 1), torch.cat(vs, 1)
        see = np.zeros((t, t), bool)
        for i in range(t):
            at = i
            while at >= 0:
                see[i, at] = True
                at = parent[r, at]
        see = torch.from_numpy(see).to(DEV).repeat_interleave(g, 0)
        q = s["q"][r].double().view(t, hkv, g, D).transpose(0, 1).reshape(hkv, t * g, D)
        sc = q @ kk.transpose(1, 2) / math.sqrt(D)
        sc[:, :, n:].masked_fill_(~see, -math.inf)
        o = torch.softmax(sc, -1) @ vv
        out[r] = o.view(hkv, t, g, D).permute(1, 0, 2, 3).reshape(t, hq, D)
        out[r, int(used[r]):] = 0
    return out


def _exact_verify(case, s):
    """Request by request on the host."""
    b, t, v = case["batch"], case["nodes"], case["vocab"]
    par, tok, used = (s[x].cpu().numpy() for x in ("parent", "tokens", "used"))
    ua, us = s["ua"].double().cpu().numpy(), s["us"].double().cpu().numpy()
    path, count, nxt = np.full((b, t), -1, np.int32), np.zeros(b, np.int32), np.zeros(b, np.int32)
    for r in range(b):
        node, steps, kids = 0, [0], []
        while True:
            kids = [i for i in range(1, used[r]) if par[r, i] == node]
            if not kids:
                break
            p = s["p"][r, node].double().cpu().numpy()
            to, seen, mass = None, set(), 0.0
            for i in kids:
                x = int(tok[r, i])
                if s["qd"] is not None:
                    if ua[r, node] * float(s["qd"][r, node, x]) < p[x]:
                        to = i
                elif x not in seen:
                    seen.add(x)
                    mass += p[x]
                    if ua[r, node] < mass:
                        to = i
                if to is not None:
                    break
            if to is None:
                break
            node = to
            steps.append(node)
        p = s["p"][r, node].double().cpu().numpy()
        if kids and s["qd"] is not None:
            p = np.maximum(p - s["qd"][r, node].double().cpu().numpy(), 0)
        elif kids:
            p[[int(tok[r, i]) for i in kids]] = 0
        run_ = np.cumsum(p)
        path[r, :len(steps)], count[r] = steps, len(steps)
        nxt[r] = int(np.flatnonzero((run_ > us[r] * run_[-1]) & (p > 0))[0])
    return {"path": path, "count": count, "next": nxt}


def _exact_commit(case, s):
    """State and window row by row. The packed words have no 64-bit value of their own."""
    sink, recent = case["sink"], case["recent"]
    window, state = s["window"].double(), s["state0"].cpu().numpy().copy()
    path, count = s["path"].cpu().numpy(), s["count"].cpu().numpy()
    for r in range(case["batch"]):
        n, e, row = (int(x) for x in state[r, :3])
        e2 = max(e, sink, n + int(count[r]) - recent)
        for j in range(int(count[r])):
            at = n + j
            if at < sink or at >= e2:
                slot = at if at < sink else sink + at % recent
                window[row, :, 0, slot] = s["k"][r, path[r, j]].double()
                window[row, :, 1, slot] = s["v"][r, path[r, j]].double()
        state[r, 0], state[r, 1] = n + int(count[r]), e2
    return {"pool": None, "window": window, "state": state}


def _exact_rope(case, s):
    n, hq, hkv, rot = (case[k] for k in ("tokens", "hq", "hkv", "rotary"))
    x = s["qkv"].double().reshape(n, hq + 2 * hkv, D)
    y = x.clone()
    if case["norm"]:
        size = (x[:, :hq + hkv] ** 2).sum(-1, keepdim=True) / D + 1e-6
        y[:, :hq + hkv] = x[:, :hq + hkv] / size.sqrt()
        y[:, :hq] *= s["wq"].double()
        y[:, hq:hq + hkv] *= s["wk"].double()
    angle = (s["pos"].double()[:, None] * torch.from_numpy(s["inv_freq"]).to(DEV))[:, None]
    i = torch.arange(rot // 2, device=DEV)
    a, c = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + rot // 2)
    qk = y[:, :hq + hkv]
    z = torch.complex(qk[..., a], qk[..., c]) * torch.polar(torch.ones_like(angle), angle)
    qk = qk.clone()
    qk[..., a], qk[..., c] = z.real, z.imag
    return {"q": qk[:, :hq], "k": qk[:, hq:], "v": x[:, hq + hkv:]}


_EXACT = {"tree_attn": _exact_tree, "verify_draft": _exact_verify, "commit_draft": _exact_commit,
          "qkv_norm_rope": _exact_rope}


def exact(case, seed):
    s = prepare(case, seed)
    return _EXACT[case["op"]](case, s)
