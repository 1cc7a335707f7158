"""Host side of the drafted-token operators: statuses, refusals and the frequency table,
without a GPU."""

import ctypes
from fractions import Fraction

import numpy as np
import pytest
import torch

from bit_rotated_kv_oscar_gb300 import abi, build


@pytest.fixture(scope="module")
def lib():
    build.build()
    return abi.lib()


def test_null_contexts_and_pointers(lib):
    n = None
    assert lib.oscar_tree_attn(n, n, n, n, n, n, n, n, n, 1, 1, n, 0, n) == -1
    assert lib.oscar_commit_draft(n, n, n, n, n, n, n, 1, 1, n) == -1
    assert lib.oscar_tree_attn_workspace_bytes(n, 1, 1) == 0
    assert lib.oscar_verify_draft(n, n, n, n, n, n, n, 1, 1, 8, n, n, n, n, n) == -1
    assert lib.oscar_qkv_norm_rope(n, 512, n, n, 128, 0, n, n, 1e-6, n, n, n, 1, 2, 1, n) == -1
    assert lib.oscar_rope_turns(n, 1, n) == -1


def test_verify_sizes_are_checked_before_anything_is_read(lib):
    x = ctypes.c_void_p(16)   # never dereferenced on the host
    call = lambda b, t, v: lib.oscar_verify_draft(x, None, x, x, None, x, x, b, t, v, x, x, x, None, None)  # noqa: E731
    assert call(0, 1, 8) == call(1, 0, 8) == call(1, 1, 0) == -1
    assert call(1, 65, 8) == call(1, 1, (1 << 18) + 1) == -5
    assert call((1 << 20) + 1, 1, 8) == -3


def test_rope_shapes_are_checked_before_anything_is_read(lib):
    x = ctypes.c_void_p(16)

    def call(stride=512, rotary=128, w=(None, None), eps=1e-6, n=1, hq=2, hkv=1, qkv=x):
        return lib.oscar_qkv_norm_rope(qkv, stride, x, x, rotary, 0, w[0], w[1], eps, x, x, x, n, hq, hkv, None)
    assert call(rotary=8) == call(rotary=40) == call(rotary=144) == -5
    assert call(stride=511) == call(stride=516) == call(stride=0) == -1
    assert call(w=(x, None)) == call(eps=-1.0) == call(n=-1) == call(hq=0) == call(qkv=ctypes.c_void_p(8)) == -1
    assert call(n=0) == 0


def test_rope_turns_are_fractions_of_a_turn(lib):
    inv = np.concatenate([1e6 ** (-np.arange(0, 128, 2) / 128), [0.0, 2 * np.pi, 7.0, -1.0]])
    got = abi.rope_turns(inv).numpy().view(np.uint64)
    two_pi = Fraction(6.283185307179586476925286766559) + Fraction(2.4492935982947064e-16)
    for f, t in zip(inv, got):
        want = (Fraction(float(f)) / two_pi) % 1
        off = abs(Fraction(int(t), 1 << 64) - want)
        # the quotient carries 53 bits of |f| / 2 pi (two roundings, and 2 pi's own)
        assert min(off, 1 - off) <= Fraction(3, 1 << 53) * max(abs(want), Fraction(abs(float(f)))) + Fraction(1, 1 << 63), f
    with pytest.raises(abi.OscarError):
        abi.rope_turns([1.0, float("inf")])


def test_the_binding_refuses_host_tensors(lib):
    f, i = torch.zeros((1, 2, 8)), torch.zeros((1, 2), dtype=torch.int32)
    with pytest.raises(ValueError):
        abi.verify_draft(f, i, i, f[:, :, 0].contiguous(), f[:, 0, 0].contiguous(), i.clone(), i[:, 0].contiguous(),
                         i[:, 0].contiguous())
    b = torch.zeros((1, 512), dtype=torch.bfloat16)
    q = torch.zeros((1, 2, 128), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        abi.qkv_norm_rope(b, i[:, 0].contiguous(), torch.zeros(64, dtype=torch.int64), q, q[:, :1].contiguous(),
                          q[:, :1].contiguous())
