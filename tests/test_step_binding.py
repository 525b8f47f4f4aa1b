"""What the Python binding of the serving-step operators holds and does around a launch,
shown on the CPU: the library is replaced by one that looks instead of launching."""
import contextlib
import ctypes
import weakref

import pytest
import torch

import paged_kv_cache_98_gb300 as pkv


class Watcher:
    """Stands in for the library: a workspace of `need` bytes, and `launched` called where
    a kernel would be."""

    def __init__(self, need, launched):
        self.need, self.launched = need, launched

    def pkv_decode_biased_workspace_size(self, *a):
        return self.need

    def pkv_paged_attention_decode_biased(self, *a):
        return self.launched(a) or 0


def _decode_args():
    return dict(out=torch.empty(2, 8, 128, dtype=torch.bfloat16), q=torch.empty(2, 8, 128, dtype=torch.bfloat16),
                k_cache=torch.empty(4, 2, 16, 128, dtype=torch.bfloat16),
                v_cache=torch.empty(4, 2, 16, 128, dtype=torch.bfloat16),
                block_tables=torch.zeros(2, 64, dtype=torch.int32),
                context_lens=torch.zeros(2, dtype=torch.int32), scale=0.1)


@pytest.fixture
def on_cpu(monkeypatch):
    """The binding's calls as they run on the GPU, on CPU tensors."""
    monkeypatch.setattr(pkv, "_stream_on", lambda device, stream, tensors: (7, contextlib.nullcontext()))
    return monkeypatch


def test_decode_workspace_lives_until_the_launch(on_cpu):
    """The workspace that the call allocates is still the call's own when the kernel is
    launched: another thread may allocate while the library runs without the
    interpreter's lock."""
    made, alive = [], []
    empty = torch.empty

    def watched(*a, **k):
        t = empty(*a, **k)
        made.append((weakref.ref(t), t.data_ptr()))
        return t

    def launched(args):
        (ref, ptr), = made
        alive.append(ref() is not None)
        assert getattr(args[20], "value", args[20]) == ptr and args[21] == 4096

    t = _decode_args()
    on_cpu.setattr(pkv, "_lib", Watcher(4096, launched))
    on_cpu.setattr(torch, "empty", watched)
    pkv.paged_attention_decode_biased(max_context_len=1024, **t)
    assert alive == [True]


def test_prefill_reads_nothing_back(on_cpu):
    """Lengths that are left out are bounded by what the host knows: no wait for the GPU
    (which a capture could not hold)."""
    seen = {}

    class Prefill:
        @staticmethod
        def pkv_paged_attention_prefill_biased(*a):
            seen.update(seqs=a[8], rows=a[9], max_q_len=a[10], max_context_len=a[17])
            return 0

    def read(*a, **k):
        raise AssertionError("a device value was read")

    t = _decode_args()
    t["query_start_loc"] = torch.tensor([0, 1, 2], dtype=torch.int32)
    on_cpu.setattr(pkv, "_lib", Prefill())
    on_cpu.setattr(torch.Tensor, "item", read)
    pkv.paged_attention_prefill_biased(**t)
    assert seen == dict(seqs=2, rows=2, max_q_len=2, max_context_len=64 * 16)
    pkv.paged_attention_prefill_biased(max_context_len=100, **t)
    assert seen["max_context_len"] == 100


def test_decode_reads_lengths_on_the_stream_it_launches_on(on_cpu):
    """A left-out max_context_len is read behind the work that fills context_lens, which the
    caller ordered before `stream`, not before the current one."""
    inside, seen = [], []

    @contextlib.contextmanager
    def stream(s):
        inside.append(s)
        yield
        inside.pop()

    most = torch.Tensor.max

    def watched(t, *a, **k):
        seen.append(list(inside))
        return most(t, *a, **k)

    t = _decode_args()
    t["context_lens"] += 40
    on_cpu.setattr(pkv, "_lib", Watcher(0, lambda a: seen.append(a[14])))
    on_cpu.setattr(torch.cuda, "stream", stream)
    on_cpu.setattr(torch.Tensor, "max", watched)
    pkv.paged_attention_decode_biased(stream="side", **t)
    assert seen == [["side"], 40]
    seen.clear()
    pkv.paged_attention_decode_biased(**t)
    assert seen == [[], 40] or seen == [[None], 40]


def test_empty_batches_are_nothing_to_do():
    """No sequences, or sequences without queries: tensors of no elements have no address,
    and the calls return what they were given."""
    from paged_kv_cache_98_gb300 import _build
    _build.build()
    lib = pkv.load()
    tail = [8, 2, 128, 16, 4, 8, 64, 0.1, 1, 1, 1.0, 1.0]  # heads .. v_scale
    kc, vc = 1 << 22, 1 << 23
    decode = lambda n, head_dim=128: lib.pkv_paged_attention_decode_biased(  # noqa: E731
        None, None, kc, vc, None, None, None, n, *tail[:2], head_dim, *tail[3:], None, 0, None, None)
    prefill = lambda n, rows, bt, cl: lib.pkv_paged_attention_prefill_biased(  # noqa: E731
        None, None, kc, vc, bt, cl, 4096, None, n, rows, 0, *tail, None, None)
    assert decode(0) == 0
    assert decode(0, 96) == -2 and decode(1) == -1  # other arguments are still looked at
    assert prefill(0, 0, None, None) == 0
    assert prefill(3, 0, 1024, 2048) == 0
    assert prefill(3, 1, 1024, 2048) == -1 and prefill(3, 0, None, 2048) == -1


def test_error_words_off_their_alignment_are_refused():
    """The error word is written by a 32-bit atomic: an address between words would fault."""
    from paged_kv_cache_98_gb300 import _build
    _build.build()
    lib = pkv.load()
    tail = [2, 8, 2, 128, 16, 4, 8, 64, 0.1, 1, 1, 1.0, 1.0]
    for word in (4096 + 1, 4096 + 2):
        assert lib.pkv_paged_attention_decode_biased(
            1 << 20, 1 << 21, 1 << 22, 1 << 23, 1024, 2048, None, *tail, None, 0, word, None) == -1
        assert lib.pkv_paged_attention_prefill_biased(
            1 << 20, 1 << 21, 1 << 22, 1 << 23, 1024, 2048, 3584, None, 2, 6, 4, *tail[1:], word, None) == -1
        assert lib.pkv_build_step_maps(
            4096, 8192, 8448, 8704, 8960, 12288, 512, 768, 1024, 1280, 2, 4, 8, 4, 2, 16, 64, word, None) == -1
        inv = (ctypes.c_double * 64)(*([1.0] * 64))
        assert lib.pkv_rotary_and_cache(
            1 << 20, 1 << 22, 1 << 23, 1 << 24, 1 << 25, 1 << 26, 256, 256, ctypes.cast(inv, ctypes.c_void_p),
            1024, 256, 256, 4, 8, 2, 128, 16, 8, 128, 0, 1.0, 1, 1, 1.0, 1.0, word, None) == -1


def test_empty_batches_through_the_binding(on_cpu):
    """Tensors without rows, through the library itself: nothing is launched."""
    from paged_kv_cache_98_gb300 import _build
    _build.build()
    e = lambda *shape, dtype=torch.bfloat16: torch.empty(shape, dtype=dtype)  # noqa: E731
    kc, vc = e(4, 2, 16, 128), e(4, 2, 16, 128)
    i32 = dict(dtype=torch.int32)
    assert pkv.paged_attention_decode_biased(e(0, 8, 128), e(0, 8, 128), kc, vc, e(0, 3, **i32), e(0, **i32),
                                             0.1, softcap=30.0).shape[0] == 0
    for n in (0, 3):
        assert pkv.paged_attention_prefill_biased(
            e(0, 8, 128), e(0, 8, 128), kc, vc, e(n, 3, **i32), torch.zeros(n, **i32),
            torch.zeros(n + 1, **i32), 0.1, window=20).shape[0] == 0
    assert pkv.rotary_and_cache(e(0, 8, 128), e(0, 8, 128), e(0, 2, 128), e(0, 2, 128), kc, vc,
                                e(0, dtype=torch.int64), e(0, **i32), [1.0] * 64).shape[0] == 0
