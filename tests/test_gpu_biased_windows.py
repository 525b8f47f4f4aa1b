"""Prefill chunks under windows on both sides of where the kernel changes the order of its
matrix products, against the plain 64-bit softmax of test_gpu_biased."""
import pytest
import torch

import paged_kv_cache_98_gb300 as pkv
from test_gpu_biased import Batch, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library():
    from paged_kv_cache_98_gb300 import _build
    _build.build()
    pkv.load()
    torch.cuda.init()


@pytest.mark.parametrize("window", [511, 512, 700])
@pytest.mark.parametrize("kw", [dict(H=8, hkv=2), dict(H=4, hkv=4, alibi=True, dtype="fp16"), dict(H=7, hkv=1, D=64),
                                dict(H=8, hkv=2, softcap=20.0), dict(H=4, hkv=1, kv="e4m3")],
                         ids=lambda k: "-".join(f"{a}{b}" for a, b in k.items()))
def test_windows(kw, window):
    run(Batch(131, [(129, 1153), (40, 640), (1, 513), (520, 520)], window=window, **kw))


def test_windows_and_items_of_many_lengths():
    run(Batch(133, [(n, n + c) for n, c in ((5, 0), (600, 0), (0, 40), (70, 900), (33, 520), (130, 2000), (1, 1))],
              H=8, hkv=8, window=600, alibi=True))
