"""Host side of the serving-step operators (step maps, rotary positions with the
cache write, attention with score modifiers): refusals before anything is
launched, workspace sizes, and the rotary frequencies against their formulas."""
import ctypes
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_98_gb300 as pkv
from paged_kv_cache_98_gb300 import _build


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return pkv.load()


# ---- step maps -------------------------------------------------------------------------------

def _maps(lib, **over):
    a = dict(block_tables=4096, context_lens=8192, query_start_loc=8448, slot_mapping=8704,
             positions=8960, request_tables=12288, rows=512, cached_lens=768, q_lens=1024,
             new_blocks=1280, num_seqs=2, num_request_rows=4, max_blocks=8, num_tokens=4,
             num_new=2, block_size=16, num_blocks=64, errors=None, stream=None)
    a.update(over)
    return lib.pkv_build_step_maps(*a.values())


@pytest.mark.parametrize("over,status", [
    (dict(block_tables=None), -1), (dict(context_lens=None), -1),
    (dict(query_start_loc=None), -1), (dict(slot_mapping=None), -1), (dict(positions=None), -1),
    (dict(request_tables=None), -1), (dict(rows=None), -1), (dict(cached_lens=None), -1),
    (dict(q_lens=None), -1), (dict(new_blocks=None), -1), (dict(num_seqs=-1), -1),
    (dict(num_request_rows=0), -1), (dict(max_blocks=0), -1), (dict(num_tokens=-1), -1),
    (dict(num_new=-1), -1), (dict(num_blocks=0), -1), (dict(slot_mapping=260), -1),
    # outputs over inputs (lengths in place) and over one another
    (dict(context_lens=768), -1), (dict(context_lens=1020), -1), (dict(query_start_loc=1028), -1),
    (dict(block_tables=12288), -1), (dict(request_tables=4096 - 4), -1), (dict(positions=8704 + 28), -1),
    (dict(slot_mapping=1280), -1), (dict(positions=8196), -1),
    (dict(block_size=32), -2), (dict(num_seqs=16385), -2), (dict(max_blocks=1 << 27), -2),
])
def test_maps_refusals(lib, over, status):
    assert _maps(lib, **over) == status


# ---- rotary ----------------------------------------------------------------------------------

def _rot(lib, **over):
    a = dict(q_out=1 << 20, q=1 << 22, k=1 << 23, v=1 << 24, k_cache=1 << 25, v_cache=1 << 26,
             slots=256, positions=256, inv=(ctypes.c_double * 64)(*([1.0] * 64)), qs=1024, ks=256,
             vs=256, tokens=4, heads=8, kv_heads=2, head_dim=128, block_size=16, num_blocks=8,
             rot=128, layout=0, attn=1.0, src=1, cache=1, k_scale=1.0, v_scale=1.0, errors=None,
             stream=None)
    a.update(over)
    if a["inv"] is not None:
        a["inv"] = ctypes.cast(a["inv"], ctypes.c_void_p)
    return lib.pkv_rotary_and_cache(*a.values())


@pytest.mark.parametrize("over,status", [
    (dict(q_out=None), -1), (dict(q=None), -1), (dict(k=None), -1), (dict(v=None), -1),
    (dict(k_cache=None), -1), (dict(v_cache=None), -1), (dict(slots=None), -1),
    (dict(positions=None), -1), (dict(inv=None), -1), (dict(tokens=-1), -1), (dict(heads=0), -1),
    (dict(kv_heads=0), -1), (dict(q=(1 << 22) + 2), -1), (dict(qs=1020), -1), (dict(qs=1028), -1),
    (dict(ks=128), -1), (dict(vs=260), -1), (dict(rot=0), -1), (dict(rot=3), -1),
    (dict(rot=130), -1), (dict(layout=2), -1), (dict(attn=math.inf), -1),
    (dict(cache=2, k_scale=0.0), -1), (dict(cache=2, v_scale=math.nan), -1),
    (dict(head_dim=96), -2), (dict(block_size=8), -2), (dict(src=2), -2), (dict(src=0), -2),
    (dict(heads=1 << 20, qs=1 << 27), -2),
    (dict(inv=(ctypes.c_double * 64)(*([math.nan] * 64))), -1),
    (dict(inv=(ctypes.c_double * 64)(*([2e3] * 64))), -1),
    # q_out over q with another layout, over k, over v
    (dict(q_out=1 << 22, qs=1536), -1), (dict(q_out=(1 << 22) + 2048), -1),
    (dict(q_out=(1 << 23) + 512), -1), (dict(q_out=(1 << 24) - 4096), -1),
    (dict(k_cache=1 << 26), -1), (dict(v_cache=(1 << 25) + 64), -1), (dict(k_cache=1 << 20), -1),
    (dict(v_cache=1 << 24), -1),
    (dict(tokens=0), 0),
])
def test_rotary_refusals(lib, over, status):
    assert _rot(lib, **over) == status


def test_rotary_binding_refusals():
    inv = np.ones(64)
    t = dict(q_out=torch.empty(3, 8, 128, dtype=torch.bfloat16),
             q=torch.empty(3, 8, 128, dtype=torch.bfloat16),
             k=torch.empty(3, 2, 128, dtype=torch.bfloat16),
             v=torch.empty(3, 2, 128, dtype=torch.bfloat16),
             k_cache=torch.empty(4, 2, 16, 128, dtype=torch.bfloat16),
             v_cache=torch.empty(4, 2, 16, 128, dtype=torch.bfloat16),
             slot_mapping=torch.zeros(3, dtype=torch.int64),
             positions=torch.zeros(3, dtype=torch.int32), inv_freq=inv)
    for over, exc in [
            (dict(slot_mapping=torch.zeros(3, dtype=torch.int32)), TypeError),
            (dict(positions=torch.zeros(4, dtype=torch.int32)), ValueError),
            (dict(k=torch.empty(3, 2, 64, dtype=torch.bfloat16)), ValueError),
            (dict(v=torch.empty(3, 2, 128, dtype=torch.float16)), ValueError),
            (dict(q=torch.empty(3, 128, 8, dtype=torch.bfloat16).transpose(1, 2)), ValueError),
            (dict(q_out=torch.empty(3, 8, 256, dtype=torch.bfloat16)[..., :128]), ValueError),
            (dict(layout="neither"), ValueError),
            (dict(inv_freq=np.ones((2, 32))), ValueError),
            (dict(), ValueError)]:  # on the CPU
        with pytest.raises(exc):
            pkv.rotary_and_cache(**{**t, **over})


def test_rotary_frequencies_formulas():
    r, base, f, n = 128, 10000.0, 8.0, 4096
    plain = np.array([base ** (-2 * i / r) for i in range(r // 2)])
    got, attn = pkv.rotary_frequencies(r, base)
    np.testing.assert_allclose(got, plain, rtol=1e-14)
    assert attn == 1.0
    np.testing.assert_allclose(pkv.rotary_frequencies(r, base, "linear", f)[0], plain / f, rtol=1e-14)
    np.testing.assert_allclose(
        pkv.rotary_frequencies(r, base, "ntk", f)[0],
        [(base * f ** (r / (r - 2))) ** (-2 * i / r) for i in range(r // 2)], rtol=1e-13)
    # the longest wavelength of the base change is the interpolated one
    assert pkv.rotary_frequencies(r, base, "ntk", f)[0][-1] == pytest.approx(plain[-1] / f, rel=1e-12)
    lo, hi = 1.0, 4.0
    want = []
    for inv in plain:
        wave = 2 * math.pi / inv
        m = (n / wave - lo) / (hi - lo)
        want.append(inv if wave < n / hi else inv / f if wave > n / lo else (1 - m) * inv / f + m * inv)
    np.testing.assert_allclose(pkv.rotary_frequencies(r, base, "bands", f, lo, hi, n)[0], want, rtol=1e-12)
    got, attn = pkv.rotary_frequencies(r, base, "yarn", f, 1.0, 32.0, n)
    assert attn == pytest.approx(0.1 * math.log(f) + 1, rel=1e-6)
    turns = n * plain / (2 * math.pi)
    assert np.all(got[:20] == plain[:20]) and np.all(turns[:20] > 32)
    np.testing.assert_allclose(got[turns < 0.9], plain[turns < 0.9] / f, rtol=1e-14)
    share = (got - plain / f) / (plain - plain / f)
    mid = (turns < 30) & (turns > 1.1)
    step = np.diff(share[mid])
    np.testing.assert_allclose(step, step[0], rtol=1e-6)  # linear in the index
    assert step[0] < 0


@pytest.mark.parametrize("args", [
    (128, 1.0), (128, math.nan), (3, 1e4), (128, 1e4, "linear", 0.5), (128, 1e4, "ntk", math.inf),
    (128, 1e4, "bands", 2.0, 4.0, 1.0, 4096), (128, 1e4, "yarn", 2.0, 1.0, 32.0, 0)])
def test_rotary_frequencies_refusals(args):
    with pytest.raises(pkv.PagedKVError):
        pkv.rotary_frequencies(*args)
    with pytest.raises(ValueError):
        pkv.rotary_frequencies(128, 1e4, "other")
    with pytest.raises(ValueError):
        pkv.rotary_frequencies(0)


# ---- attention under score modifiers --------------------------------------------------------------

def _mods(**over):
    m = pkv._ScoreMods(over.pop("softcap", 0.0), over.pop("alibi", None), over.pop("window", 0),
                       over.pop("key_start", None), over.pop("prefix", None))
    assert not over
    return m


def _decode(lib, mods=None, **over):
    a = dict(out=1 << 20, q=1 << 21, k_cache=1 << 22, v_cache=1 << 23, block_tables=1024, context_lens=2048,
             mods=ctypes.addressof(mods) if mods else None, num_seqs=2, num_heads=8,
             num_kv_heads=2, head_dim=128, block_size=16, max_blocks_per_seq=4, num_blocks=8,
             max_context_len=64, scale=0.1, q_dtype=1, kv_dtype=1, k_scale=1.0, v_scale=1.0,
             workspace=None, workspace_bytes=0, errors=None, stream=None)
    a.update(over)
    return lib.pkv_paged_attention_decode_biased(*a.values())


def _prefill(lib, mods=None, **over):
    a = dict(out=1 << 20, q=1 << 21, k_cache=1 << 22, v_cache=1 << 23, block_tables=1024, context_lens=2048,
             qsl=4096, mods=ctypes.addressof(mods) if mods else None, num_seqs=2, total_q=6,
             max_q_len=4, num_heads=8, num_kv_heads=2, head_dim=128, block_size=16,
             max_blocks_per_seq=4, num_blocks=8, max_context_len=64, scale=0.1, q_dtype=1,
             kv_dtype=1, k_scale=1.0, v_scale=1.0, errors=None,
             stream=None)
    a.update(over)
    return lib.pkv_paged_attention_prefill_biased(*a.values())


@pytest.mark.parametrize("call", [_decode, _prefill])
@pytest.mark.parametrize("mods,over,status", [
    (dict(softcap=-1.0), {}, -1), (dict(softcap=math.nan), {}, -1), (dict(softcap=math.inf), {}, -1),
    (dict(softcap=1e-45), {}, -1), (dict(softcap=1e-30), dict(scale=1e30), -1),
    (dict(window=-1), {}, -1), (None, dict(head_dim=96), -2), (None, dict(block_size=32), -2),
    (None, dict(num_heads=6, num_kv_heads=4), -1), (None, dict(num_heads=34), -2),
    (None, dict(q_dtype=2), -2), (None, dict(q_dtype=0), -2), (None, dict(out=None), -1),
    (None, dict(q=264), -1), (None, dict(scale=math.nan), -1),
    (None, dict(out=1 << 21), -1), (None, dict(out=(1 << 21) + 2048), -1), (None, dict(out=1 << 22), -1),
    (None, dict(out=(1 << 23) + 4096), -1),
    (None, dict(kv_dtype=2, k_scale=-1.0), -1), (None, dict(num_seqs=0), 0)])
def test_biased_refusals(lib, call, mods, over, status):
    assert call(lib, _mods(**mods) if mods else None, **over) == status


def test_biased_refusals_of_one_kind(lib):
    assert _decode(lib, _mods(prefix=4096)) == -1  # a decode row is the last token
    assert _decode(lib, None, max_context_len=4096, max_blocks_per_seq=256) == -3
    assert _prefill(lib, None, qsl=None) == -1
    assert _prefill(lib, None, total_q=-1) == -1
    assert _prefill(lib, None, total_q=0) == 0


def test_biased_workspace_sizes(lib):
    def split(heads, parts, d):
        return -(-heads * parts * 4 // 256) * 256 + -(-heads * parts * d * 4 // 256) * 256

    assert pkv.decode_biased_workspace_size(64, 32, 128, 512) == 0
    assert pkv.decode_biased_workspace_size(64, 32, 128, 4096) == split(64 * 32, 8, 128)
    # a window bounds the partitions, wherever in a block it starts
    assert pkv.decode_biased_workspace_size(64, 32, 128, 131072, 497) == 0
    assert pkv.decode_biased_workspace_size(64, 32, 128, 131072, 498) == split(64 * 32, 2, 128)
    assert pkv.decode_biased_workspace_size(64, 32, 128, 131072, 2 ** 31 - 1) == split(64 * 32, 256, 128)
    assert pkv.decode_biased_workspace_size(64, 32, 128, 4096, -1) == 0


def test_biased_binding_refusals():
    t = dict(out=torch.empty(2, 8, 128, dtype=torch.bfloat16),
             q=torch.empty(2, 8, 128, dtype=torch.bfloat16),
             k_cache=torch.empty(4, 2, 16, 128, dtype=torch.bfloat16),
             v_cache=torch.empty(4, 2, 16, 128, dtype=torch.bfloat16),
             block_tables=torch.zeros(2, 2, dtype=torch.int32),
             context_lens=torch.zeros(2, dtype=torch.int32), scale=0.1, max_context_len=32)
    for over, exc in [(dict(alibi_slopes=torch.zeros(8, dtype=torch.float64)), TypeError),
                      (dict(alibi_slopes=torch.zeros(2)), ValueError),
                      (dict(key_start=torch.zeros(2, dtype=torch.int64)), TypeError),
                      (dict(key_start=torch.zeros(3, dtype=torch.int32)), ValueError),
                      (dict(context_lens=torch.zeros(3, dtype=torch.int32)), ValueError),
                      (dict(out=torch.empty(2, 8, 128, dtype=torch.float16)), TypeError),
                      (dict(device_errors=torch.zeros(3, dtype=torch.uint8)), ValueError),
                      (dict(), ValueError)]:  # on the CPU
        with pytest.raises(exc):
            pkv.paged_attention_decode_biased(**{**t, **over})
    with pytest.raises(TypeError):
        pkv.paged_attention_prefill_biased(query_start_loc=torch.tensor([0, 1, 2]), max_q_len=1, **t)
    with pytest.raises(ValueError):
        pkv.paged_attention_prefill_biased(
            query_start_loc=torch.tensor([0, 1, 2], dtype=torch.int32),
            prefix_lens=torch.zeros(1, dtype=torch.int32), max_q_len=1, **t)
