"""Ways of calling the biased attention: from two threads at once without workspaces of
their own, and captured with every length left out."""
import threading

import pytest
import torch

import paged_kv_cache_98_gb300 as pkv
from test_gpu_biased import DEV, Batch, Decode

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library():
    from paged_kv_cache_98_gb300 import _build
    _build.build()
    pkv.load()
    torch.cuda.init()


def test_decode_from_two_threads():
    """Each thread's calls allocate and give back a workspace on the same stream, beside the
    other's allocations and writes of the same size."""
    batches = [Decode(141 + i, [900, 40, 1400, 2000], H=8, hkv=2, softcap=20.0) for i in range(2)]
    want = [b.call().cpu() for b in batches]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        b = batches[i]
        q, (bt, cl) = b.q.to(DEV), b.dev[:2]
        n = pkv.decode_biased_workspace_size(4, 8, 128, 2000)
        outs = []
        for _ in range(60):
            out = torch.empty_like(q)
            pkv.paged_attention_decode_biased(out, q, b.kc, b.vc, bt, cl, b.scale, softcap=20.0,
                                              max_context_len=2000)
            torch.empty(n, dtype=torch.uint8, device=DEV).fill_(255)
            outs.append(out)
        if not all(torch.equal(o.cpu(), want[i]) for o in outs):
            bad.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


@pytest.mark.parametrize("kw", [dict(window=90), dict(alibi=True, dtype="fp16"), dict(kv="e4m3", softcap=20.0)],
                         ids=lambda k: "-".join(k))
def test_prefill_captured_without_lengths(kw):
    b = Batch(143, [(70, 200), (1, 33), (130, 513)], H=8, hkv=2, **kw)
    b.check(b.call())
    q, (bt, cl, qsl) = b.q.to(DEV), b.dev[:3]
    out = torch.empty_like(q)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        pkv.paged_attention_prefill_biased(out, q, b.kc, b.vc, bt, cl, qsl, b.scale, softcap=b.softcap,
                                           window=b.window, alibi_slopes=b.dev[5], k_scale=b.ks, v_scale=b.vs)
    b.q = (-b.q).roll(5, 0)
    q.copy_(b.q)
    g.replay()
    torch.cuda.synchronize()
    b.check(out)
