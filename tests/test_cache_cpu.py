"""The paged cache's host layer (no GPU needed): what the C ABI and the tensor helpers refuse, and the reference's
4-bit rows against their definition."""
from __future__ import annotations

import ctypes

import pytest
import torch

from tests import cache_ref as ref


@pytest.fixture(scope="module")
def abi():
    from shifted_sparse_attention_b200 import build
    build.build()
    from shifted_sparse_attention_b200 import binding
    return binding


FAKE = 1 << 20  # never dereferenced: validation fails first


def structs(**over):
    from shifted_sparse_attention_b200.cache import _BatchStruct, _CacheStruct
    c = dict(k=FAKE, v=FAKE, k_scale=None, v_scale=None, pages=8, heads=2, page_size=16, D=128, format=0)
    b = dict(page_table=FAKE, seq_lens=FAKE, q_starts=FAKE, seqs=3, tokens=7, table_width=4, max_new=5, max_len=64)
    for name, value in over.items():
        (c if name in c else b)[name] = value
    return _CacheStruct(**c), _BatchStruct(**b)


DESCRIPTORS = [
    (dict(format=2), -1), (dict(k=None), -1), (dict(v=None), -1), (dict(k=FAKE + 8), -1), (dict(k_scale=FAKE), -1),
    (dict(format=1), -1), (dict(format=1, k_scale=FAKE, v_scale=FAKE + 4), -1), (dict(page_table=None), -1),
    (dict(seq_lens=None), -1), (dict(seq_lens=FAKE + 2), -1), (dict(q_starts=FAKE + 1), -1),
    (dict(pages=0), -2), (dict(heads=0), -2), (dict(seqs=0), -2), (dict(tokens=0, max_new=0), -2),
    (dict(table_width=0), -2), (dict(max_new=8), -2), (dict(max_new=-1), -2), (dict(max_len=65), -2),
    (dict(max_len=-1), -2), (dict(q_starts=None), -2), (dict(table_width=1 << 28, max_len=0), -2),
    (dict(D=96), -3), (dict(D=256), -3), (dict(page_size=8), -3), (dict(page_size=48), -3), (dict(page_size=256), -3),
    (dict(pages=1 << 31), -3), (dict(pages=1 << 30), -3), (dict(tokens=1 << 30), -3), (dict(seqs=1 << 30), -3),
]


@pytest.mark.parametrize("over,code", DESCRIPTORS)
def test_descriptors_are_checked_by_every_call(abi, over, code):
    L = abi.lib()
    c, b = structs(**over)
    pc, pb = ctypes.byref(c), ctypes.byref(b)
    assert L.s2attn_cache_append(pc, pb, None, 0, FAKE, 256, FAKE, 256, None, 0, None, 1e4, 1.0, None) == code
    assert abi.s2attn_last_error()
    assert L.s2attn_cache_read(pc, pb, FAKE, FAKE, None) == code
    assert L.s2attn_cache_attn(pc, pb, FAKE, 1024, FAKE, None, 8, FAKE, 1 << 40, None) == code
    assert L.s2attn_cache_attn_workspace_size(pc, pb, 8) == 0


def test_append_arguments(abi):
    L = abi.lib()
    c, b = structs()
    good = dict(q=FAKE, ldq=1024, k=FAKE, ldk=256, v=FAKE, ldv=256, q_out=FAKE, heads=8, positions=None, base=1e4,
                scale=1.0)
    for over, code in [
        (dict(k=None), -1), (dict(v=FAKE + 4), -1), (dict(q_out=None), -1), (dict(q=None), -1), (dict(q=FAKE + 2), -1),
        (dict(base=1.0), -1), (dict(base=-2.0), -1), (dict(base=float("nan")), -1), (dict(base=float("inf")), -1),
        (dict(scale=0.0), -1), (dict(scale=float("inf")), -1), (dict(base=0.0), -1), (dict(positions=FAKE + 2), -1),
        (dict(ldk=255), -2), (dict(ldk=260), -2), (dict(ldv=128), -2), (dict(ldq=1000), -2), (dict(heads=3), -2),
        (dict(heads=0), -2), (dict(heads=258, ldq=258 * 128), -3),
    ]:
        rc = L.s2attn_cache_append(ctypes.byref(c), ctypes.byref(b), *{**good, **over}.values(), None)
        assert rc == code, (over, rc, abi.s2attn_last_error())


def test_attention_and_read_arguments(abi):
    L = abi.lib()
    c, b = structs()
    pc, pb = ctypes.byref(c), ctypes.byref(b)
    need = L.s2attn_cache_attn_workspace_size(pc, pb, 8)
    assert need > 0
    good = dict(q=FAKE, ldq=1024, o=FAKE, lse=None, heads=8, ws=FAKE, n=need)
    for over, code in [
        (dict(q=None), -1), (dict(o=None), -1), (dict(o=FAKE + 8), -1), (dict(lse=FAKE + 2), -1), (dict(ws=None), -1),
        (dict(ws=FAKE + 128), -1), (dict(n=need - 1), -1), (dict(n=0), -1), (dict(ldq=1016), -2), (dict(ldq=1028), -2),
        (dict(heads=5), -2), (dict(heads=258, ldq=258 * 128), -3),
    ]:
        rc = L.s2attn_cache_attn(pc, pb, *{**good, **over}.values(), None)
        assert rc == code, (over, rc, abi.s2attn_last_error())
    for kv in ((None, FAKE), (FAKE, None), (FAKE + 8, FAKE)):
        assert L.s2attn_cache_read(pc, pb, *kv, None) == -1
    assert L.s2attn_cache_read(None, pb, FAKE, FAKE, None) == -1
    assert L.s2attn_cache_read(pc, None, FAKE, FAKE, None) == -1


@pytest.mark.parametrize("D,format", [(128, 0), (64, 0), (128, 1), (64, 1)])
def test_one_workspace_serves_every_batch_of_a_cache(abi, D, format):
    """What a program learns of its sequences as they grow (and how many take part, with how many tokens) chooses
    kernels; the workspace that it keeps must do for all of them."""
    L = abi.lib()
    scales = dict(k_scale=FAKE, v_scale=FAKE) if format else {}
    sizes = set()
    for seqs, tokens, max_new in [(1, 1, 1), (16, 80, 5), (64, 64, 1), (3, 2000, 1000), (1, 2048, 2048), (9, 700, 0)]:
        for width, max_len in [(4, 0), (1 << 12, 0), (1 << 12, 40), (1 << 12, 3800), (1 << 12, 3900), (1 << 12, 65536)]:
            for heads in (2, 8, 32):
                c, b = structs(D=D, format=format, seqs=seqs, tokens=tokens, max_new=max_new, table_width=width,
                               max_len=max_len, **scales)
                n = L.s2attn_cache_attn_workspace_size(ctypes.byref(c), ctypes.byref(b), heads)
                assert n > 0
                sizes.add(n)
    assert len(sizes) == 1


def test_tensor_helpers_refuse_host_tensors(abi):
    import shifted_sparse_attention_b200 as s2
    x = torch.zeros(2, 2, 16, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        s2.KVCache(x, x)
    with pytest.raises(ValueError):
        s2.KVCache(x, x, x[..., :2])
    with pytest.raises(ValueError):
        s2.KVCache.empty(2, 16, 2, 128, bits=8)
    t = torch.zeros(2, 4, dtype=torch.int32)
    with pytest.raises(ValueError):
        s2.CacheBatch(t, t[:, 0])


def test_tensors_that_want_a_gradient_are_refused():
    """There is no backward: a result without a gradient must not come in silence."""
    from types import SimpleNamespace
    from shifted_sparse_attention_b200.cache import _rows
    cache, batch = SimpleNamespace(index=-1, dim=64), SimpleNamespace(tokens=3)  # -1: host tensors
    leaf = torch.zeros(3, 2, 64, dtype=torch.bfloat16, requires_grad=True)
    for t in (leaf, leaf * 2):
        with pytest.raises(ValueError, match="gradient"):
            _rows("q", t, cache, batch, 2)
        with torch.no_grad():
            assert _rows("q", t, cache, batch, 2) == 128
        assert _rows("q", t.detach(), cache, batch, 2) == 128
    with torch.inference_mode():
        assert _rows("q", leaf * 2, cache, batch, 2) == 128


def test_reference_rows_of_four_bits():
    x = torch.randn(50, 128, generator=torch.Generator().manual_seed(0)).bfloat16()
    c, s, m = ref.pack(x)
    assert c.min() == 0 and c.max() == 15 and torch.equal(ref.split_codes(ref.join_codes(c)), c)
    v = m[:, None] + s[:, None] * c
    # half a step, and at the upper end what the scale's rounding to bf16 moves the grid: 15 s 2^-8 at most
    assert ((v - x.double()).abs() <= s[:, None] * (0.5 + 15 * 2.0 ** -8)).all()


def test_reference_attention_is_a_softmax_over_the_visible_rows():
    for bits in (16, 4):
        p = ref.Paged([37, 5], 2, 64, 16, bits)
        q = torch.randn(4, 4, 64).bfloat16()
        o, lse, _, _ = ref.attention(p, q, torch.tensor([0, 3, 4]))
        k, v, _, _ = p.rows(0, 1)
        z = (q[1, 2].double() @ k[:36].T) / 8.0
        assert torch.allclose(o[1, 2], torch.softmax(z, 0) @ v[:36]) and torch.allclose(lse[1, 2], torch.logsumexp(z, 0))
