"""oscar_qkv_norm_rope against a float64 restatement.

Tolerance: everything is fp32 but the bf16 output, half a step of which is 2^-8 of a value.
The fp32 part: the norm's sum of 128 squares, the root and the products are off by at most
about 140 * 2^-24 of the value, cos and sin (2 ulp, and an angle off by 2^-26 turns) by
2^-22 of the pair's length, so 2^-16 of the pair's length covers them."""

import numpy as np
import pytest
import torch

from bit_rotated_kv_oscar_gb300 import abi, build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "the gpu-marked tests need a CUDA device"
    build.build()
    abi.lib()


def reference(x, pos, inv_freq, w, eps, rotary, interleaved):
    """x [n, heads, 128] float64 -> (y, length of each channel's pair)."""
    y = x.copy()
    if w is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * w
    i = np.arange(rotary // 2)
    a, c = (2 * i, 2 * i + 1) if interleaved else (i, i + rotary // 2)
    # the angle modulo a turn in exact integers of 2^-200 turns
    from fractions import Fraction
    two_pi = Fraction(6.283185307179586476925286766559) + Fraction(2.4492935982947064e-16)
    turn = np.array([[float((Fraction(int(p)) * Fraction(float(f)) / two_pi) % 1) for f in inv_freq] for p in pos])
    cos, sin = np.cos(2 * np.pi * turn)[:, None], np.sin(2 * np.pi * turn)[:, None]
    out = y.copy()
    out[..., a] = y[..., a] * cos - y[..., c] * sin
    out[..., c] = y[..., c] * cos + y[..., a] * sin
    size = np.abs(y)
    size[..., a] = size[..., c] = np.hypot(y[..., a], y[..., c])
    return out, size


def check(n, hq, hkv, rotary=128, interleaved=False, norm=True, pad=0, far=100000, eps=1e-6, seed=0, pos=None, scale=1.0):
    rng = np.random.default_rng(seed)
    width = (hq + 2 * hkv) * 128
    buf = torch.from_numpy(rng.standard_normal((n, width + pad)).astype(np.float32) * scale).to(torch.bfloat16).cuda()
    qkv = buf[:, :width]
    w = [torch.from_numpy(1 + 0.3 * rng.standard_normal(128)).to(torch.bfloat16).cuda() if norm else None for _ in range(2)]
    pos = rng.integers(0, far, n) if pos is None else np.asarray(pos)
    inv = 1e6 ** (-np.arange(0, rotary, 2) / rotary)
    out = [torch.full((n, h, 128), float("nan"), dtype=torch.bfloat16, device="cuda") for h in (hq, hkv, hkv)]
    abi.qkv_norm_rope(qkv, torch.from_numpy(pos.astype(np.int32)).cuda(), abi.rope_turns(inv).cuda(), *out, q_weight=w[0],
                      k_weight=w[1], eps=eps, interleaved=interleaved)
    torch.cuda.synchronize()
    x = qkv.double().cpu().numpy().reshape(n, -1, 128)
    for part, got, wt in ((slice(0, hq), out[0], w[0]), (slice(hq, hq + hkv), out[1], w[1])):
        want, size = reference(x[:, part], pos, inv, None if wt is None else wt.double().cpu().numpy(), eps, rotary,
                               interleaved)
        err = np.abs(got.double().cpu().numpy() - want)
        fine = 2.0 ** -16 * size
        assert (err <= fine + 2.0 ** -8 * (np.abs(want) + fine)).all()
    assert torch.equal(out[2].view(n, -1), qkv[:, (hq + hkv) * 128:])


@pytest.mark.parametrize("hq,hkv", [(1, 1), (2, 1), (8, 2), (32, 8), (64, 8)])
@pytest.mark.parametrize("n", [1, 2, 7])
def test_heads(n, hq, hkv):
    check(n, hq, hkv, seed=n + hq)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rotary", [16, 48, 64, 96, 128])
def test_rotary_dims(rotary, interleaved):
    check(5, 4, 2, rotary=rotary, interleaved=interleaved)


@pytest.mark.parametrize("pad", [8, 24, 128])
def test_padded_rows(pad):
    check(9, 4, 2, pad=pad)


def test_without_norm():
    check(6, 4, 2, norm=False)


def test_many_tokens():
    check(4097, 2, 1, rotary=32)   # several tokens per CTA, the last CTA cut short


def test_far_and_negative_positions():
    check(6, 2, 1, pos=[0, 1, 1 << 20, (1 << 31) - 1, -1, -(1 << 31)])


def test_small_and_zero_rows():
    check(4, 2, 1, scale=1e-4, eps=1e-6)
    check(4, 2, 1, scale=0.0, eps=1e-5)


def test_no_tokens():
    z = torch.zeros((0, 512), dtype=torch.bfloat16, device="cuda")
    q, k = (torch.zeros((0, h, 128), dtype=torch.bfloat16, device="cuda") for h in (2, 1))
    abi.qkv_norm_rope(z, torch.zeros(0, dtype=torch.int32, device="cuda"), abi.rope_turns(np.ones(64)).cuda(), q, k, k.clone())


def test_refusals():
    n, hq, hkv = 2, 2, 1
    t = dict(qkv=torch.zeros((n, 512), dtype=torch.bfloat16, device="cuda"), pos=torch.zeros(n, dtype=torch.int32, device="cuda"),
             turns=abi.rope_turns(np.ones(64)).cuda(), q=torch.zeros((n, hq, 128), dtype=torch.bfloat16, device="cuda"),
             k=torch.zeros((n, hkv, 128), dtype=torch.bfloat16, device="cuda"),
             v=torch.zeros((n, hkv, 128), dtype=torch.bfloat16, device="cuda"))
    w = torch.ones(128, dtype=torch.bfloat16, device="cuda")

    def status(**kw):
        with pytest.raises(abi.OscarError) as e:
            abi.qkv_norm_rope(**{**t, **kw})
        return e.value.status
    assert status(turns=abi.rope_turns(np.ones(20)).cuda()) == -5      # rotary_dim 40
    assert status(turns=abi.rope_turns(np.ones(72)).cuda()) == -5
    assert status(q_weight=w) == -1
    assert status(eps=-1.0) == -1 and status(eps=float("nan")) == -1
    assert status(qkv=torch.zeros((n, 516), dtype=torch.bfloat16, device="cuda")[:, :512]) == -1   # stride 516
    assert status(qkv=torch.zeros((n, 520), dtype=torch.bfloat16, device="cuda")[:, 4:516]) == -1  # 8-byte base
    for kw in (dict(qkv=t["qkv"].float()), dict(qkv=t["qkv"].t()), dict(pos=t["pos"].long()), dict(v=t["v"].cpu()),
               dict(qkv=t["qkv"][:1].expand(2, 512)), dict(k=t["k"].float())):
        with pytest.raises(ValueError):
            status(**kw)
