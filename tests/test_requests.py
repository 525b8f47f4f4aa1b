"""Host side of the calls on requests whose block lists live on the GPU, and on the caches
of all layers: refusals before anything is launched, and how the binding takes caches."""
import contextlib
import ctypes

import pytest
import torch

import paged_kv_cache_98_gb300 as pkv
from paged_kv_cache_98_gb300 import _build


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return pkv.load()


def _fork(lib, **over):
    a = dict(tables_out=1 << 12, lens_out=1 << 13, tables=1 << 14, lens=1 << 15, counts=1 << 16,
             parents=1 << 17, num_out=4, num_in=3, width=8, block_size=16, num_blocks=64, errors=None,
             stream=None)
    a.update(over)
    return lib.pkv_fork_requests(*a.values())


@pytest.mark.parametrize("over,status", [
    (dict(tables_out=None), -1), (dict(lens_out=None), -1), (dict(tables=None), -1), (dict(lens=None), -1),
    (dict(counts=None), -1), (dict(parents=None), -1), (dict(num_out=-1), -1), (dict(num_in=-1), -1),
    (dict(width=0), -1), (dict(num_blocks=0), -1), (dict(parents=(1 << 17) + 2), -1),
    (dict(errors=(1 << 18) + 1), -1), (dict(counts=(1 << 16) + 1), -1),
    # outputs over inputs and over one another
    (dict(tables_out=1 << 14), -1), (dict(tables_out=(1 << 14) + 8), -1), (dict(lens_out=1 << 15), -1),
    (dict(parents=1 << 13), -1), (dict(counts=(1 << 12) + 124), -1), (dict(lens=(1 << 16) + 252), -1),
    (dict(block_size=32), -2), (dict(num_out=65537), -2), (dict(num_in=65537), -2), (dict(width=1 << 27), -2),
])
def test_fork_refusals(lib, over, status):
    assert _fork(lib, **over) == status


def test_fork_of_nothing(lib):
    assert _fork(lib, num_out=0, num_in=0, tables_out=None, lens_out=None, tables=None, lens=None,
                 counts=None, parents=None) == 0


def _resize(lib, **over):
    a = dict(tables=1 << 14, counts=1 << 16, rows=512, cached=768, lens=1024, granted=1 << 17,
             new_blocks=1 << 18, pairs=1 << 19, num_seqs=4, num_rows=6, width=8, num_new=5, block_size=16,
             num_blocks=64, errors=None, stream=None)
    a.update(over)
    return lib.pkv_resize_requests(*a.values())


@pytest.mark.parametrize("over,status", [
    (dict(tables=None), -1), (dict(counts=None), -1), (dict(rows=None), -1), (dict(cached=None), -1),
    (dict(lens=None), -1), (dict(granted=None), -1), (dict(new_blocks=None), -1), (dict(pairs=None), -1),
    (dict(num_seqs=-1), -1), (dict(num_rows=0), -1), (dict(width=0), -1), (dict(num_new=-1), -1),
    (dict(num_blocks=0), -1), (dict(granted=(1 << 17) + 1), -1), (dict(errors=(1 << 20) + 3), -1),
    # lengths in place, a list over the tables, counts over pairs
    (dict(granted=768), -1), (dict(granted=1024 + 12), -1), (dict(new_blocks=(1 << 14) + 188), -1),
    (dict(pairs=(1 << 16) + 252), -1), (dict(rows=(1 << 19) + 28), -1), (dict(granted=1 << 18), -1),
    (dict(block_size=8), -2), (dict(num_seqs=16385), -2), (dict(num_blocks=(1 << 30) - 1), -2),
    (dict(width=1 << 27), -2),
])
def test_resize_refusals(lib, over, status):
    assert _resize(lib, **over) == status


def test_resize_of_nothing(lib):
    assert _resize(lib, num_seqs=0, num_new=0, tables=None, counts=None, rows=None, cached=None, lens=None,
                   granted=None, new_blocks=None, pairs=None) == 0


def _caches(n, at=1 << 24, step=1 << 20):
    return ctypes.cast((ctypes.c_void_p * max(n, 1))(*[at + i * step for i in range(n)]), ctypes.c_void_p)


def _copy(lib, k=None, v=None, layers=3, pairs=4096, num=2, heads=2, d=128, bs=16, nb=8, dt=1, errors=None):
    k = _caches(layers) if k is None else k
    v = _caches(layers, 1 << 28) if v is None else v
    return lib.pkv_copy_blocks_layers(k, v, layers, pairs, num, heads, d, bs, nb, dt, errors, None)


def _compact(lib, **over):
    a = dict(k=_caches(3), v=_caches(3, 1 << 28), layers=3, tables=4096, context=8192, base=8448, starts=8704,
             keep=12288, new=8960, counts=None, num_seqs=2, num_keep=9, heads=2, d=128, bs=16, width=8, nb=8,
             dt=1, errors=None, stream=None)
    a.update(over)
    return lib.pkv_compact_tokens(*a.values())


@pytest.mark.parametrize("over,status", [
    (dict(layers=-1), -1), (dict(pairs=None), -1), (dict(num=-1), -1), (dict(heads=0), -1), (dict(nb=0), -1),
    (dict(d=0), -1), (dict(pairs=4097), -1), (dict(errors=2), -1), (dict(bs=32), -2), (dict(dt=3), -2),
    (dict(k=_caches(3, (1 << 24) + 8)), -1),            # off the 16-byte boundary
    (dict(v=_caches(3, (1 << 24) + (1 << 19))), 0),     # between K's caches of 65536 bytes
    (dict(v=_caches(3, (1 << 24) + 65520)), -1),        # over the end of K's
    (dict(k=_caches(3, step=0)), -1),                   # one cache twice
    (dict(k=_caches(129, step=65536), v=_caches(129, 1 << 28, 65536), layers=129, num=0), 0),
    (dict(k=_caches(129, step=65536), v=_caches(129, (1 << 24) + 128 * 65536 + 16, 65536), layers=129, num=0), -1),
])
def test_copy_refusals(lib, over, status):
    if status == 0:
        over = dict(over, num=0)
    assert _copy(lib, **over) == status


def test_copy_of_nothing(lib):
    assert _copy(lib, num=0, pairs=None) == 0
    assert lib.pkv_copy_blocks_layers(None, None, 0, 4096, 2, 2, 128, 16, 8, 1, None, None) == 0
    assert lib.pkv_copy_blocks_layers(None, None, 1, 4096, 2, 2, 128, 16, 8, 1, None, None) == -1


@pytest.mark.parametrize("over,status", [
    (dict(layers=0), -1), (dict(tables=None), -1), (dict(context=None), -1), (dict(base=None), -1),
    (dict(starts=None), -1), (dict(keep=None), -1), (dict(new=None), -1), (dict(num_seqs=-1), -1),
    (dict(num_keep=-1), -1), (dict(heads=0), -1), (dict(width=0), -1), (dict(nb=0), -1), (dict(k=None), -1),
    (dict(keep=12289), -1), (dict(errors=1), -1), (dict(counts=3), -1),
    (dict(new=8192), -1), (dict(new=8704 + 8), -1), (dict(counts=8960 - 28), -1), (dict(new=4096 + 60), -1),
    (dict(v=_caches(3, (1 << 24) + 65520)), -1),
    (dict(bs=32), -2), (dict(d=96), -2), (dict(dt=3), -2), (dict(width=1 << 27), -2),
])
def test_compact_refusals(lib, over, status):
    assert _compact(lib, **over) == status


def test_compact_of_nothing(lib):
    assert _compact(lib, num_seqs=0, num_keep=0, tables=None, context=None, base=None, starts=None, keep=None,
                    new=None) == 0


# ---- the binding -----------------------------------------------------------------------------

@pytest.fixture
def on_cpu(monkeypatch):
    monkeypatch.setattr(pkv, "_stream_on", lambda device, stream, tensors: (7, contextlib.nullcontext()))
    return monkeypatch


def test_layers_as_lists_and_as_one_tensor(on_cpu):
    """Either way the library gets every layer's address, in order."""
    seen = []

    class Lib:
        @staticmethod
        def pkv_copy_blocks_layers(k, v, L, pairs, n, h, d, bs, nb, dt, err, stream):
            seen.append((list(k[:L]), list(v[:L]), L, n, h, d, bs, nb, dt))
            return 0

    on_cpu.setattr(pkv, "_lib", Lib())
    both = torch.zeros(3, 2, 5, 4, 16, 64, dtype=torch.float16)
    pairs = torch.zeros(7, 2, dtype=torch.int32)
    pkv.copy_blocks_layers(both[:, 0], both[:, 1], pairs)
    pkv.copy_blocks_layers([x[0] for x in both], [x[1] for x in both], pairs)
    assert seen[0] == seen[1]
    assert seen[0] == ([x[0].data_ptr() for x in both], [x[1].data_ptr() for x in both], 3, 7, 4, 64, 16, 5,
                       pkv.F16)


@pytest.mark.parametrize("k,v", [
    (lambda x: x[:, 0], lambda x: x[:2, 1]),                          # fewer layers
    (lambda x: x[:, 0], lambda x: x[:, 1].to(torch.bfloat16)),        # another dtype
    (lambda x: x[:, 0], lambda x: x[:, 1, :4]),                       # fewer blocks
    (lambda x: x[:, 0].transpose(2, 3), lambda x: x[:, 1].transpose(2, 3)),  # layers not contiguous
    (lambda x: [y[0] for y in x], lambda x: [y[1].transpose(0, 1) for y in x]),
    (lambda x: [], lambda x: []),
    (lambda x: x[0, 0], lambda x: x[0, 1]),                           # no layers' dimension
])
def test_layers_refused(on_cpu, k, v):
    x = torch.zeros(3, 2, 5, 4, 16, 64, dtype=torch.float16)
    with pytest.raises(ValueError):
        pkv.copy_blocks_layers(k(x), v(x), torch.zeros(7, 2, dtype=torch.int32))
