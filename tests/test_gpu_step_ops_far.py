"""Rotary positions whose angles are thousands of millions of turns, against angles reduced
in rational arithmetic; tolerances as in test_gpu_step_ops."""
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

import paged_kv_cache_98_gb300 as pkv
from test_gpu_step_ops import DEV, TD, ints, near

pytestmark = pytest.mark.gpu
TWO_PI = 2 * Fraction("3.14159265358979323846264338327950288419716939937510582097494459")


@pytest.fixture(scope="module", autouse=True)
def _library():
    from paged_kv_cache_98_gb300 import _build
    _build.build()
    pkv.load()
    torch.cuda.init()


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_rotary_far_positions_and_high_frequencies(layout, dtype):
    inv = np.concatenate([[1000.0, -1000.0, 999.7, 123.456, 1.0, -1e-9, 1e-3, 0.9], np.geomspace(1000.0, 1e-6, 24)])
    pos = np.array([0, 1, 7, 12345, 131071, 2 ** 24 + 1, 123456789, 2 ** 30 - 1, 2 ** 30, 2 ** 31 - 1])
    T, H, D = len(pos), 16, 64
    g = torch.Generator(device=DEV).manual_seed(3)
    q, k, v = (torch.randn((T, n, D), generator=g, device=DEV).to(TD[dtype]) for n in (H, 2, 2))
    kc, vc = (torch.zeros((1, 2, 16, D), dtype=TD[dtype], device=DEV) for _ in range(2))
    out = torch.empty_like(q)
    pkv.rotary_and_cache(out, q, k, v, kc, vc, ints(np.arange(T), torch.int64), ints(pos), inv, layout)
    turn = [[float((Fraction(float(f)) * int(t) / TWO_PI) % 1) for f in inv] for t in pos]
    ang = torch.tensor(turn, dtype=torch.float64)[:, None] * 2 * math.pi
    c, s = torch.cos(ang), torch.sin(ang)
    i = torch.arange(32)
    ia, ib = (i, i + 32) if layout == "half" else (2 * i, 2 * i + 1)
    for got, x in ((out, q), (kc[0, :, :T].transpose(0, 1), k)):
        x = x.double().cpu()
        a, b = x[..., ia], x[..., ib]
        want, off = torch.empty_like(x), torch.empty_like(x)
        want[..., ia], want[..., ib] = a * c - b * s, b * c + a * s
        off[..., ia] = off[..., ib] = (a.abs() + b.abs()) * 2.0 ** -21
        near(got, want, off, "q" if x.shape[1] == H else "k")
