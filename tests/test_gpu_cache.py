"""The paged cache of keys and values on the GPU (needs a B200): append, read and attention against the 64-bit
reference (tests/cache_ref.py), which also derives the tolerances."""
from __future__ import annotations

import pytest
import torch

import shifted_sparse_attention_b200 as s2
from tests import cache_ref as ref

pytestmark = pytest.mark.gpu


def starts_of(news):
    return torch.tensor([0] + list(news)).cumsum(0).to(torch.int32)


def on_gpu(c):
    return s2.KVCache(*[t.cuda() for t in (c.k, c.v, c.ks, c.vs) if t is not None])


def batch_of(c, news, plain=False, extra=0, wide=False, **hints):
    """wide: a table with room for a million keys, which the call then has to reckon with (it takes the kernel for
    many rows, whatever the lengths are)."""
    lens = torch.tensor(c.lens, dtype=torch.int32).cuda()
    starts = None if plain else starts_of(news).cuda()
    table = c.table
    if wide:
        table = torch.nn.functional.pad(table, (0, (1 << 20) // c.S), value=-7)
    return s2.CacheBatch(table.cuda(), lens, starts, sum(news) + extra, **hints)


def check_attention(c, news, H, seed=0, plain=False, wide=False, **hints):
    T = sum(news)
    g = torch.Generator().manual_seed(seed)
    q = torch.randn(T, H, c.dim, generator=g).bfloat16()
    o, lse, to, tl = ref.attention(c, q, starts_of(news))
    got_lse = torch.empty(T, H, device="cuda")
    got = s2.cache_attention(on_gpu(c), batch_of(c, news, plain, wide=wide, **hints), q.cuda(), lse=got_lse)
    s2.check_status()
    got, got_lse = got.double().cpu(), got_lse.double().cpu()
    assert torch.isfinite(got).all()
    over = (got - o).abs() - to
    assert (over <= 0).all(), ("o", float(over.max()), int((over > 0).sum()))
    empty = lse.isinf()
    assert torch.equal(got_lse.isinf(), empty)
    off = ((got_lse - lse).abs() - tl)[~empty]
    assert off.numel() == 0 or (off <= 0).all(), ("lse", float(off.max()))
    return got


STEPS = [  # (lens, new tokens)
    ([1], [1]),
    ([15], [1]),
    ([16], [1]),
    ([17], [1]),
    ([513], [1]),
    ([128, 129, 1, 127, 64], [1] * 5),
    ([20000], [1]),
    ([5000, 3, 9001, 700], [1, 1, 2, 3]),
]


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("D,H,Hkv,S", [(128, 8, 2, 16), (64, 3, 3, 64)])
@pytest.mark.parametrize("lens,news", STEPS)
def test_few_new_tokens(bits, D, H, Hkv, S, lens, news):
    # without and with the host's knowledge of the lengths: units are cut for long sequences, whole for short ones
    c = ref.Paged(lens, Hkv, D, S, bits, seed=len(lens) + lens[0])
    for max_len in (0, max(lens)):
        check_attention(c, news, H, plain=all(n == 1 for n in news), max_new=max(news), max_len=max_len)


@pytest.mark.parametrize("bits", [16, 4])
def test_whole_units_of_uneven_batches(bits):
    # more sequences than threads look at the lengths at once, rows in several blocks, empty sequences among them
    lens = [(37 * i) % 300 for i in range(200)]
    news = [min(n, 1 + i % 3) if i % 7 else 0 for i, n in enumerate(lens)]
    c = ref.Paged(lens, 1, 64, 16, bits)
    check_attention(c, news, 9, max_new=3, max_len=300)
    check_attention(c, news, 9, max_new=3)


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("D,H,Hkv,lens,news", [  # how many units there are decides how many CTAs share one
    (128, 4, 1, [2048], [1]),
    (128, 32, 32, [513], [1]),
    (64, 24, 2, [1900, 0, 1, 70, 15], [2, 1, 1, 0, 3]),       # blocks of 16 rows, some of them of no token
    (128, 4, 4, [1000, 64, 0, 1, 512, 333, 17, 900, 2, 5], [1, 2, 1, 1, 1, 1, 1, 1, 1, 1]),
    (64, 8, 8, [(97 * i) % 513 for i in range(20)], [1] * 20),
])
def test_whole_units_shared_by_clusters(bits, D, H, Hkv, lens, news):
    c = ref.Paged(lens, Hkv, D, 16, bits, seed=H + lens[0])
    for max_len in (max(lens), 130):  # 130: longer than the host knows
        check_attention(c, news, H, max_new=max(news), max_len=max_len)


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("D", [128, 64])
@pytest.mark.parametrize("H,Hkv", [(7, 1), (16, 1), (17, 1), (40, 2), (12, 4)])
def test_heads_shared_by_key_heads(bits, D, H, Hkv):
    c = ref.Paged([700, 31], Hkv, D, 32, bits, seed=H)
    check_attention(c, [1, 1], H, max_new=1)
    check_attention(c, [3, 2], H, max_new=3)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("D,H,Hkv,S", [(128, 4, 2, 128), (64, 6, 2, 16), (128, 5, 1, 64)])
@pytest.mark.parametrize("lens,news", [
    ([200], [200]),                 # a whole prompt: the first token sees one key
    ([129, 1000], [129, 130]),
    ([640, 64, 1], [256, 64, 1]),   # chunks beside a single token
    ([1200], [700]),
])
def test_chunks_of_prompts(bits, D, H, Hkv, S, lens, news, wide):
    c = ref.Paged(lens, Hkv, D, S, bits, seed=lens[0])
    check_attention(c, news, H, wide=wide, max_new=max(news), max_len=0 if wide else max(lens))


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("lens,news", [
    ([9000], [300]),                            # units cut over several CTAs
    ([2500, 700, 31, 4000], [64, 700, 31, 5]),
    ([128, 256, 384] * 12, [128, 1, 300] * 12),  # many units for a CTA
])
def test_units_cut_over_ctas(bits, lens, news):
    c = ref.Paged(lens, 2, 128, 64, bits, seed=lens[0])
    check_attention(c, news, 6, wide=True, max_new=max(news))


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("H,Hkv", [(8, 1), (3, 3), (7, 1), (128, 1), (48, 2), (20, 4)])
def test_chunks_with_heads_shared_by_key_heads(bits, H, Hkv):
    c = ref.Paged([333, 150], Hkv, 64, 32, bits, seed=H)
    check_attention(c, [40, 150], H, wide=True, max_new=150)


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("max_new,wide", [(1, False), (0, False), (5, True)])
def test_rows_that_see_nothing_and_sequences_left_out(bits, max_new, wide):
    # lengths of zero (a padded batch), fewer rows than new tokens, no new token
    lens, news = [0, 40, 2, 300, 0], [1, 1, 5, 0, 3]
    c = ref.Paged(lens, 2, 128, 16, bits)
    got = check_attention(c, news, 8, wide=wide, max_new=max_new)
    assert (got[0] == 0).all() and (got[2:5] == 0).all() and (got[5] != 0).any()


@pytest.mark.parametrize("max_new", [1, 200])
def test_hints_change_no_result_and_runs_repeat_bitwise(max_new):
    lens, news = [1500, 260, 77], [1, 200, 3]
    c = ref.Paged(lens, 2, 128, 64, 16)
    a = check_attention(c, news, 8, max_new=max_new)
    b = check_attention(c, news, 8, wide=True, max_new=200)
    assert torch.equal(a, check_attention(c, news, 8, max_new=max_new)) and (a - b).abs().max() < 2e-2
    assert torch.equal(b, check_attention(c, news, 8, wide=True, max_new=200))


def test_lengths_beyond_the_hints_are_served():
    lens, news = [1500, 3, 700], [2, 1, 1]
    c = ref.Paged(lens, 2, 128, 64, 16)
    for hints in (dict(max_new=1, max_len=40), dict(max_new=2, max_len=600), dict(max_new=0, max_len=1)):
        check_attention(c, news, 8, **hints)


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("wide", [False, True])
def test_pages_shared_by_sequences(bits, wide):
    # two conversations with one beginning: the same pages in both tables
    c = ref.Paged([256, 300, 290], 2, 128, 32, bits)
    c.table[1, :8] = c.table[0, :8]
    c.table[2, :8] = c.table[0, :8]
    check_attention(c, [1, 44, 34], 8, wide=wide, max_new=44)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("bits", [16, 4])
def test_tokens_of_no_sequence_are_left_as_they_were(bits, wide):
    c = ref.Paged([90, 33], 2, 64, 16, bits)
    news, extra, before = [2, 1], 4, 3
    T = sum(news) + extra + before
    starts = (starts_of(news) + before).to(torch.int32).cuda()
    table = torch.nn.functional.pad(c.table, (0, 1 << 16), value=-7) if wide else c.table
    batch = s2.CacheBatch(table.cuda(), torch.tensor(c.lens, dtype=torch.int32).cuda(), starts, T, max_new=T)
    H = 32 if wide else 4
    q = torch.randn(T, H, 64).bfloat16().cuda()
    out, lse = torch.full((T, H, 64), 7.0).bfloat16().cuda(), torch.full((T, H), 7.0).cuda()
    s2.cache_attention(on_gpu(c), batch, q, out=out, lse=lse)
    rows = [torch.full((T, 2, 64), 7.0).bfloat16().cuda() for _ in range(2)]
    s2.cache_read(on_gpu(c), batch, out=rows)
    cache = on_gpu(c)
    rq = torch.full_like(q, 7.0)
    s2.cache_append(cache, batch, *[torch.randn(T, 2, 64).bfloat16().cuda() for _ in range(2)], q, out=rq)
    s2.check_status()
    for t in (out, lse, *rows, rq):
        assert (t[:before] == 7).all() and (t[before + sum(news):] == 7).all()
        assert (t[before:before + sum(news)] != 7).any()


def test_extreme_scores():
    # a key so large that one weight is all, or none
    c = ref.Paged([64], 1, 128, 16, 16)
    c.k[c.table[0, 1].long(), 0, 3] *= 100
    for seed in range(4):
        check_attention(c, [1], 1, seed=seed, plain=True)


def test_infinite_value_in_a_visible_row():
    # an infinite value reaches its channel and no other (its weight is far from 0 here)
    c = ref.Paged([64], 1, 128, 16, 16)
    cache, batch = on_gpu(c), batch_of(c, [1], plain=True)
    cache.v[c.table[0, 3].long(), 0, 15, 5] = float("inf")
    q = 0.1 * torch.randn(1, 1, 128, generator=torch.Generator().manual_seed(0))
    got = s2.cache_attention(cache, batch, q.bfloat16().cuda())
    assert torch.isinf(got[0, 0, 5]) and torch.isfinite(got[0, 0, :5]).all() and torch.isfinite(got[0, 0, 6:]).all()


def test_strided_queries():
    c = ref.Paged([77, 400], 2, 128, 32, 16)
    wide = torch.randn(2, 8 * 128 + 64).bfloat16()
    q = wide[:, 64:].unflatten(1, (8, 128))
    batch = batch_of(c, [1, 1], plain=True)
    a = s2.cache_attention(on_gpu(c), batch, wide.cuda()[:, 64:].unflatten(1, (8, 128)))
    b = s2.cache_attention(on_gpu(c), batch, q.contiguous().cuda())
    assert torch.equal(a, b)


def test_rows_beyond_32_bit_offsets():
    # 2^18 pages of 64 rows of 128 channels x 2 heads in bf16: 4.3e9 elements a tensor (8.6 GB); the sequence lives at
    # its end
    pages, S, Hkv, D = (1 << 18) + 8, 64, 2, 128
    cache = s2.KVCache.empty(pages, S, Hkv, D)
    c = ref.Paged([150, 64], Hkv, D, S, 16, spare=0)
    shift = pages - c.k.shape[0]
    cache.k[shift:], cache.v[shift:] = c.k.cuda(), c.v.cuda()
    table = torch.where(c.table >= 0, c.table + shift, c.table).cuda()
    lens = torch.tensor(c.lens, dtype=torch.int32).cuda()
    for news in ([1, 1], [150, 64]):
        starts = starts_of(news)
        q = torch.randn(sum(news), 4, D).bfloat16()
        o, _, to, _ = ref.attention(c, q, starts)
        wide = torch.nn.functional.pad(table, (0, 1 << 13), value=-7) if max(news) > 1 else table
        batch = s2.CacheBatch(wide.contiguous(), lens, starts.cuda(), sum(news), max_new=max(news))
        got = s2.cache_attention(cache, batch, q.cuda())
        assert ((got.double().cpu() - o).abs() <= to).all()
    k, _ = s2.cache_read(cache, batch)
    assert torch.equal(k[:150, 1].cpu().double(), c.rows(0, 1)[0])
    s2.check_status()


# ---------------------------------------------------------------- append and read


def check_append(lens, news, H, Hkv, D, S, bits, base=10000.0, scale=1.0, positions=None, seed=0):
    c = ref.Paged(lens, Hkv, D, S, bits, seed=seed)
    T = sum(news)
    g = torch.Generator().manual_seed(seed + 1)
    qkv = torch.randn(T, (H + 2 * Hkv) * D, generator=g).bfloat16()
    q, k, v = qkv.split([H * D, Hkv * D, Hkv * D], 1)
    q, k, v = q.unflatten(1, (H, D)), k.unflatten(1, (Hkv, D)), v.unflatten(1, (Hkv, D))
    place = torch.cat([n - m + torch.arange(m) for n, m in zip(lens, news)])
    pos = place if positions is None else positions
    cache, batch = on_gpu(c), batch_of(c, news)
    before = [t.clone() for t in (cache.k, cache.v)]
    dev = qkv.cuda()
    dq, dk, dv = (t.unflatten(1, (-1, D)) for t in dev.split([H * D, Hkv * D, Hkv * D], 1))
    kw = {} if positions is None else {"positions": positions.to(torch.int32).cuda()}
    out = s2.cache_append(cache, batch, dk, dv, dq if base else None, base=base, scale=scale, **kw)
    rk, rv = s2.cache_read(cache, batch)
    s2.check_status()
    stored = place >= 0

    def near(got, want, pair):
        # the rotation: sine and cosine to 3e-7 (angle in turns rounded to 32 bits), two products and a sum, a rounding
        slack = 6e-7 * pair + 2.0 ** -23 * want.abs()
        assert ((got - want).abs() <= ref.U * (want.abs() + slack) + slack).all()

    def pair_size(x):
        h = D // 2
        s = x.double()[..., :h].abs() + x.double()[..., h:].abs()
        return torch.cat([s, s], -1)

    kr = ref.rotate(k, pos, base, scale) if base else k.double()
    if base:
        near(out.double().cpu(), ref.rotate(q, pos, base, scale), pair_size(q))
    else:
        assert out is None
    gk, gv = rk.double().cpu()[stored], rv.double().cpu()[stored]
    if bits == 16:
        near(gk, kr[stored], pair_size(k)[stored]) if base else None
        assert base or torch.equal(gk, kr[stored])
        assert torch.equal(gv, v.double()[stored])
    else:
        # values: exactly what the definition makes of them
        cv, sv, mv = ref.pack(v[stored])
        assert torch.equal(gv, (mv[..., None] + sv[..., None] * cv).float().bfloat16().double())
        # keys: the rotated row may differ from the reference's by a step of bf16, so a code by one
        ck, sk, mk = ref.pack(kr[stored].bfloat16())
        want = mk[..., None] + sk[..., None] * ck
        assert ((gk - want).abs() <= 1.1 * sk[..., None] + 2 * ref.U * want.abs()).all()
        assert ((gk - want).abs() > ref.U * want.abs() + 2.0 ** -7 * sk[..., None] + 1e-6).double().mean() < 1e-3
        # half a step of the grid, the scale's rounding, and the row's own roundings to bf16
        size = kr[stored].abs().amax(-1, keepdim=True)
        assert ((gk - kr[stored]).abs() <= 0.55 * sk[..., None] + 3 * ref.U * size).all()
    # nothing else was written
    touched = torch.zeros(c.k.shape[:3], dtype=torch.bool)
    at = 0
    for b, (n, m) in enumerate(zip(lens, news)):
        for i in range(m):
            p = n - m + i
            if p >= 0:
                touched[int(c.table[b, p // S]), :, p % S] = True
        at += m
    for t, old in zip((cache.k, cache.v), before):
        a, o = t.cpu()[~touched], old.cpu()[~touched]
        assert torch.equal(a.view(torch.uint8), o.view(torch.uint8))
    return cache, batch


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("D,H,Hkv,S", [(128, 4, 2, 16), (64, 5, 5, 128), (128, 9, 1, 64)])
@pytest.mark.parametrize("lens,news", [
    ([1], [1]), ([257], [1]), ([130, 1, 64], [130, 1, 33]), ([900, 17, 0, 3], [2, 17, 1, 0]), ([5, 40], [9, 1]),
])
def test_append_and_read(bits, D, H, Hkv, S, lens, news):
    check_append(lens, news, H, Hkv, D, S, bits, seed=lens[0])


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("D,H,Hkv,S,lens,news", [
    (128, 4, 2, 64, [900, 17, 0, 64], [690, 17, 0, 33]),  # the last call of one token to a CTA,
    (128, 4, 2, 64, [900, 17, 0, 64], [691, 17, 0, 33]),  # and the first of several
    (64, 8, 8, 16, [8300, 90], [8200, 3]),
])
def test_append_and_read_of_many_tokens(bits, D, H, Hkv, S, lens, news):
    check_append(lens, news, H, Hkv, D, S, bits, seed=news[0])


@pytest.mark.parametrize("bits", [16, 4])
def test_append_at_given_positions_and_unrotated(bits):
    pos = torch.tensor([0, 1, 8191, 99999, 1000000, 2 ** 31 - 1, 7])
    check_append([40, 9], [4, 3], 4, 2, 128, 32, bits, base=500000.0, scale=0.25, positions=pos)
    check_append([40, 9], [4, 3], 4, 2, 64, 32, bits, base=0.0)


def test_packing_of_flat_and_broken_rows():
    cache = s2.KVCache.empty(1, 16, 1, 64, bits=4)
    lens = torch.tensor([4], dtype=torch.int32).cuda()
    batch = s2.CacheBatch(torch.zeros(1, 1, dtype=torch.int32).cuda(), lens,
                          torch.tensor([0, 4], dtype=torch.int32).cuda(), 4)
    x = torch.randn(4, 1, 64).bfloat16()
    x[0] = -3.0                       # all equal: scale 0
    x[1, 0, 5] = float("nan")
    x[2, 0, 63] = float("inf")
    s2.cache_append(cache, batch, x.cuda(), x.cuda(), base=0.0)
    k, v = s2.cache_read(cache, batch)
    for t in (k, v):
        assert (t[0] == -3.0).all() and torch.isnan(t[1:3]).all() and torch.isfinite(t[3]).all()


def test_codes_at_borders_and_of_all_sizes():
    """Rows whose numbers lie right between two codes, and rows from the smallest numbers to large ones: the codes are
    those of the 32-bit definition, to the last bit."""
    g = torch.Generator().manual_seed(3)
    rows = [torch.randint(-200, 200, (200, 128), generator=g).float() * 2.0 ** e for e in (-130, -126, -100, -8, 0, 60, 100)]
    rows += [torch.arange(128).float()[None] * 0.5 ** k for k in range(6)]
    x = torch.cat(rows).bfloat16()
    T = len(x)
    cache = s2.KVCache.empty(-(-T // 16), 16, 1, 128, bits=4)
    batch = s2.CacheBatch(torch.arange(-(-T // 16), dtype=torch.int32)[None].cuda(),
                          torch.tensor([T], dtype=torch.int32).cuda(), torch.tensor([0, T], dtype=torch.int32).cuda(), T)
    s2.cache_append(cache, batch, x[:, None].cuda(), x[:, None].cuda(), base=0.0)
    f = x.float()
    mn, mx = f.amin(-1, keepdim=True), f.amax(-1, keepdim=True)
    s = ((mx - mn) / 15).bfloat16().float()
    c = torch.where(s > 0, torch.round((f - mn) / torch.where(s > 0, s, 1.0)), 0.0).clamp(0, 15)
    assert torch.equal(cache.v.view(-1, 64)[:T].cpu(), ref.join_codes(c))
    assert torch.equal(cache.v_scale.view(-1, 2)[:T].cpu().float(), torch.cat([s, mn], -1))


def test_numbers_out_of_range_are_reported_and_touch_nothing():
    c = ref.Paged([40, 33], 2, 64, 16, 16)
    T = 2

    def batch(**kw):
        a = dict(page_table=c.table.clone(), seq_lens=torch.tensor([40, 33], dtype=torch.int32),
                 q_starts=torch.tensor([0, 1, 2], dtype=torch.int32))
        for name, (at, value) in kw.items():
            a[name][at] = value
        return s2.CacheBatch(*[t.cuda() for t in a.values()], T)

    x = torch.randn(T, 2, 64).bfloat16().cuda()
    good = s2.cache_attention(on_gpu(c), batch(), x)
    s2.check_status()
    for kw in (dict(page_table=((0, 2), 10 ** 6)), dict(page_table=((0, 2), -1)), dict(seq_lens=(0, 10 ** 6)),
               dict(seq_lens=(0, -3)), dict(q_starts=(0, 2)), dict(q_starts=(0, -1))):
        cache = on_gpu(c)
        got = s2.cache_attention(cache, batch(**kw), x)
        with pytest.raises(s2.S2AttnError) as e:
            s2.check_status()
        assert e.value.code == -6
        assert torch.equal(got[1], good[1])  # the other sequence is served
        s2.cache_append(cache, batch(**kw), x, x, base=0.0)
        with pytest.raises(s2.S2AttnError):
            s2.check_status()
        at = c.table[0, 2].long()
        assert torch.equal(cache.k[at].cpu().view(torch.int16), c.k[at].view(torch.int16))
    s2.check_status()


# ---------------------------------------------------------------- a serving program


@pytest.mark.parametrize("bits", [16, 4])
def test_prompt_in_chunks_and_steps_match_the_dense_forward(bits):
    """A prompt appended in two chunks, then single steps, against the framework's dense-causal forward over the keys
    and values that the cache holds."""
    N, H, Hkv, D, S = 640, 8, 2, 128, 64
    g = torch.Generator().manual_seed(5)
    q, k, v = (torch.randn(N, h, D, generator=g).bfloat16().cuda() for h in (H, Hkv, Hkv))
    cache = s2.KVCache.empty(12, S, Hkv, D, bits=bits)
    table = torch.randperm(12, generator=g)[: N // S].to(torch.int32)[None].cuda()
    lens = torch.zeros(1, dtype=torch.int32).cuda()
    outs, rq = [], []
    at = 0
    for n in (300, 329) + (1,) * 11:
        lens += n
        batch = s2.CacheBatch(table, lens, torch.tensor([0, n], dtype=torch.int32).cuda(), n, max_new=n)
        r = s2.cache_append(cache, batch, k[at:at + n], v[at:at + n], q[at:at + n])
        outs.append(s2.cache_attention(cache, batch, r))
        rq.append(r)
        at += n
    whole = s2.CacheBatch(table, lens, torch.tensor([0, N], dtype=torch.int32).cuda(), N)
    ck, cv = s2.cache_read(cache, whole)
    s2.check_status()
    fk, fv = (t.repeat_interleave(H // Hkv, 1)[None].contiguous() for t in (ck, cv))
    o, _ = s2.forward(torch.cat(rq)[None].contiguous(), fk, fv, N, s2.DENSE_CAUSAL)
    got = torch.cat(outs).double()
    # both sides round weights and results (4 U), and the read-back rows of 4 bits once more (2 U)
    off = (got - o[0].double()).abs()
    assert (off <= 6 * ref.U * (fv[0].abs().double().amax())).all() and off.mean() < 2e-3


@pytest.mark.parametrize("bits", [16, 4])
def test_steps_captured_in_a_graph(bits):
    """One captured step, replayed while the program moves lengths and tokens on, against eager calls."""
    Hkv, H, D, S = 2, 8, 128, 16
    lens0 = [5, 130, 47]
    c = ref.Paged([n + 40 for n in lens0], Hkv, D, S, bits, fill=0.0)
    cache, twin = on_gpu(c), on_gpu(c)
    lens = torch.tensor(lens0, dtype=torch.int32).cuda()
    batch = s2.CacheBatch(c.table.cuda(), lens, max_len=170)
    q, k, v = (torch.zeros(3, h, D, dtype=torch.bfloat16, device="cuda") for h in (H, Hkv, Hkv))
    rq, o = torch.empty_like(q), torch.empty_like(q)
    ws = s2.cache_attention_workspace(cache, batch, H)
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        s2.cache_append(cache, batch, k, v, q, out=rq)
        s2.cache_attention(cache, batch, rq, out=o, workspace=ws)
    torch.cuda.current_stream().wait_stream(side)
    with torch.cuda.graph(graph):
        s2.cache_append(cache, batch, k, v, q, out=rq)
        s2.cache_attention(cache, batch, rq, out=o, workspace=ws)
    cache.k.copy_(c.k), cache.v.copy_(c.v)
    if bits == 4:
        cache.k_scale.copy_(c.ks), cache.v_scale.copy_(c.vs)
    g = torch.Generator().manual_seed(1)
    for _ in range(35):
        for t in (q, k, v):
            t.copy_(torch.randn(t.shape, generator=g))
        lens += 1
        graph.replay()
        want = s2.cache_attention(twin, batch, s2.cache_append(twin, batch, k, v, q))
        assert torch.equal(o, want)
    assert torch.equal(cache.k.view(torch.uint8), twin.k.view(torch.uint8))
    s2.check_status()


@pytest.mark.parametrize("bits", [16, 4])
def test_chunks_captured_in_a_graph(bits):
    """A captured call of the kernel for many rows, replayed with other lengths, starts and pages."""
    c = ref.Paged([700, 400], 2, 128, 64, bits, fill=0.0)
    cache = on_gpu(c)
    batch = batch_of(c, [200, 100], wide=True, max_new=200)
    q = torch.randn(300, 8, 128, generator=torch.Generator().manual_seed(2)).bfloat16()
    out, ws, dev = torch.empty(300, 8, 128).bfloat16().cuda(), s2.cache_attention_workspace(cache, batch, 8), q.cuda()
    s2.cache_attention(cache, batch, dev, out=out, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s2.cache_attention(cache, batch, dev, out=out, workspace=ws)
    table = batch.page_table.clone()
    for lens, news in (([700, 400], [200, 100]), ([650, 77], [250, 50]), ([300, 0], [1, 299])):
        batch.seq_lens.copy_(torch.tensor(lens)), batch.q_starts.copy_(starts_of(news))
        batch.page_table.copy_(table)
        graph.replay()
        c.lens = lens
        o, _, to, _ = ref.attention(c, q, starts_of(news))
        assert ((out.double().cpu() - o).abs() <= to).all()
    s2.check_status()


def test_calls_on_other_streams():
    """Calls given a stream allocate on it and run there, two at once with a workspace each."""
    c = ref.Paged([3000, 200], 2, 128, 64, 16)
    cache, batch = on_gpu(c), batch_of(c, [1, 1], plain=True)
    q = torch.randn(2, 8, 128).bfloat16().cuda()
    want = s2.cache_attention(cache, batch, q)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = []
    for _ in range(20):
        for s in streams:
            outs.append(s2.cache_attention(cache, batch, q, stream=s))
        outs.append(s2.cache_attention(cache, batch, q, stream=streams[0].cuda_stream))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    s2.check_status()


def test_one_token_of_any_stride():
    # the rows of one token are nowhere apart: what the tensor says their distance is does not matter
    c = ref.Paged([77], 2, 128, 32, 16)
    batch, q, kv = batch_of(c, [1], plain=True), torch.randn(1, 4, 128).bfloat16(), torch.randn(1, 2, 128).bfloat16()

    def odd(t):
        return torch.as_strided(t.cuda(), t.shape, (3, 128, 1))

    a, b = on_gpu(c), on_gpu(c)
    assert torch.equal(s2.cache_append(a, batch, odd(kv), odd(kv), odd(q)),
                       s2.cache_append(b, batch, kv.cuda(), kv.cuda(), q.cuda()))
    for x, y in ((a.k, b.k), (a.v, b.v)):  # as bits: rows that hold nothing hold NaN
        assert torch.equal(x.view(torch.int16), y.view(torch.int16))
    assert torch.equal(s2.cache_attention(a, batch, odd(q)), s2.cache_attention(b, batch, q.cuda()))


def test_packing_of_rows_wider_than_32_bits():
    cache = s2.KVCache.empty(1, 16, 1, 64, bits=4)
    cache.k.fill_(255)
    batch = s2.CacheBatch(torch.zeros(1, 1, dtype=torch.int32).cuda(), torch.tensor([2], dtype=torch.int32).cuda(),
                          torch.tensor([0, 2], dtype=torch.int32).cuda(), 2)
    x = torch.randn(2, 1, 64).bfloat16()
    x[0, 0, 3], x[0, 0, 40] = 3e38, -3e38  # finite, but their distance is not
    s2.cache_append(cache, batch, x.cuda(), x.cuda(), base=0.0)
    for t in s2.cache_read(cache, batch):
        assert torch.isnan(t[0]).all() and torch.isfinite(t[1]).all()


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("H,Hkv,lens,news", [
    (3, 1, [700], [1]), (1, 1, [513], [1]), (5, 1, [1000, 40], [1, 3]), (7, 1, [900, 0, 333], [1, 1, 1]),
])
def test_clusters_whose_rows_end_inside_a_warp(bits, H, Hkv, lens, news):
    # rows of 64 channels are half a warp's work: an odd number of them ends the last turn of a warp's lanes apart, and
    # the lanes that write lse part as well, right before the cluster's CTAs meet
    c = ref.Paged(lens, Hkv, 64, 16, bits, seed=H)
    check_attention(c, news, H, max_new=max(news), max_len=max(lens))


def check_not_finite(c, news, H, q, **kw):
    """As check_attention for queries and keys that hold NaN or infinities: o and lse are NaN and infinite where the
    definition's are, and near it elsewhere.  Returns o, lse and the definition's."""
    T, wide = sum(news), kw.pop("wide", False)
    o, lse, to, tl = ref.attention(c, q, starts_of(news))
    got_lse = torch.empty(T, H, device="cuda")
    got = s2.cache_attention(on_gpu(c), batch_of(c, news, wide=wide, **kw), q.cuda(), lse=got_lse)
    s2.check_status()
    got, got_lse = got.double().cpu(), got_lse.double().cpu()
    assert torch.equal(got.isnan(), o.isnan())
    assert torch.equal(got_lse.isnan(), lse.isnan())
    assert torch.equal(got_lse.nan_to_num(0, 1, -1).where(got_lse.isinf(), 0.0), lse.nan_to_num(0, 1, -1).where(lse.isinf(), 0.0))
    some = o.isfinite()
    assert ((got - o).abs() <= to)[some].all()
    some = lse.isfinite()
    assert ((got_lse - lse).abs() <= tl)[some].all()
    return got, got_lse, o, lse


# units taken whole by one CTA or by a cluster, cut over CTAs, and the kernel for many rows (whole and cut)
PATHS = ["whole", "cut", "many"]


def heads_of(path, news, few):
    """Query heads (on two key heads) with which the path is taken: rows enough for the kernel for many."""
    return few if path != "many" else 128 if max(news) < 16 else 48


def hints_of(path, lens, news):
    return {"whole": dict(max_new=max(news), max_len=min(max(lens), 512)), "cut": dict(max_new=max(news)),
            "many": dict(max_new=max(news), wide=True)}[path]


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("lens,news", [([1], [1]), ([16], [1]), ([17], [1]), ([33], [1]), ([513], [1]), ([40, 9001], [3, 5]),
                                       ([129], [2]), ([9000], [300])])
def test_a_query_that_holds_nan(bits, lens, news, path):
    c = ref.Paged(lens, 2, 128, 16, bits, seed=lens[0])
    T, H = sum(news), heads_of(path, news, 6)
    q = torch.randn(T, H, 128, generator=torch.Generator().manual_seed(T)).bfloat16()
    q[T - 1, H - 2, 77] = float("nan")  # one row, on the second key head
    got, _, _, _ = check_not_finite(c, news, H, q, **hints_of(path, lens, news))
    assert got[T - 1, H - 2].isnan().all() and got.isnan().sum() == 128


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("lens,news,at", [  # the newest key alone in its step, tile or piece; and one far from both ends
    ([1], [1], 0), ([16], [1], 15), ([17], [1], 16), ([33], [1], 32), ([513], [1], 512), ([129], [1], 128),
    ([300], [40], 290), ([9001], [3], 9000), ([9000], [300], 8999), ([9000], [300], 4321), ([9000], [300], 0),
])
def test_a_key_that_holds_nan(bits, lens, news, at, path):
    # a 4-bit row is NaN as append leaves a broken one
    c = ref.Paged(lens, 2, 128, 16, bits, seed=lens[0])
    page = int(c.table[0, at // 16])
    if bits == 16:
        c.k[page, 1, at % 16, 5] = float("nan")
    else:
        c.ks[page, 1, at % 16] = float("nan")
    H = heads_of(path, news, 4)
    q = torch.randn(sum(news), H, 128, generator=torch.Generator().manual_seed(at)).bfloat16()
    got, _, _, _ = check_not_finite(c, news, H, q, **hints_of(path, lens, news))
    seen = lens[0] - news[0] + torch.arange(news[0]) >= at
    assert got[seen][:, H // 2:].isnan().all() and got[:, :H // 2].isfinite().all()


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("lens,news,at", [
    ([1], [1], [0]), ([17], [1], [16]), ([17], [1], [3, 4, 16]), ([513], [1], [512]), ([300], [40], [290]),
    ([9001], [3], [5000, 17]), ([9000], [300], [8900, 4321]), ([20], [1], range(20)), ([700], [300], range(700)),
])
def test_scores_that_are_infinite(lens, news, at, path):
    """A key with an infinity meets queries of both signs in its channel: a score of inf makes lse inf and o NaN
    (inf / inf), one of -inf has no weight, and where all are -inf, o is 0 / 0 and lse -inf."""
    c = ref.Paged(lens, 2, 128, 16, 16, seed=lens[0])
    H, T = heads_of(path, news, 4), sum(news)
    q = torch.randn(T, H, 128, generator=torch.Generator().manual_seed(at[0])).bfloat16()
    q[:, ::2, 0], q[:, 1::2, 0] = 1.0, -1.0
    # what the keys of score -inf leave: as if it were about -1000 / sqrt(128) = -88, a weight below 2^-100
    for p in at:
        c.k[int(c.table[0, p // 16]), 1, p % 16, 0] = 1000.0
    o, lse, to, tl = ref.attention(c, q, starts_of(news))
    for p in at:
        c.k[int(c.table[0, p // 16]), 1, p % 16, 0] = float("inf")
    hints = hints_of(path, lens, news)
    got_lse = torch.empty(T, H, device="cuda")
    got = s2.cache_attention(on_gpu(c), batch_of(c, news, wide=hints.pop("wide", False), **hints), q.cuda(), lse=got_lse)
    s2.check_status()
    got, got_lse = got.double().cpu(), got_lse.double().cpu()
    place = lens[0] - news[0] + torch.arange(T)
    on_second = torch.arange(H) >= H // 2
    hit = (place >= min(at))[:, None] & on_second  # rows that see such a key
    up, down = hit & (torch.arange(H) % 2 == 0), hit & (torch.arange(H) % 2 == 1)
    none = down & torch.tensor([all(j in at for j in range(int(p) + 1)) for p in place])[:, None]  # and no other
    assert got[up].isnan().all() and (got_lse[up] == float("inf")).all()
    assert got[none].isnan().all() and (got_lse[none] == -float("inf")).all()
    rest = ~up & ~none
    assert ((got - o).abs() <= to)[rest].all() and ((got_lse - lse).abs() <= tl)[rest].all()


@pytest.mark.parametrize("bits", [16, 4])
def test_one_workspace_over_a_conversation(bits):
    """A prompt in chunks, then steps whose bound of the lengths grows past where another kernel is chosen: the program
    keeps the workspace that it made for its first step."""
    H, Hkv, D, S = 16, 2, 128, 16
    lens = [5000, 300, 2, 77]
    c = ref.Paged(lens, Hkv, D, S, bits)
    cache = on_gpu(c)
    first = batch_of(c, [1] * 4, max_new=1, max_len=5000)
    ws = s2.cache_attention_workspace(cache, first, H)
    for news, max_len in ([1] * 4, 5000), ([300, 300, 2, 70], 5000), ([5, 5, 2, 5], 5008), ([40, 1, 1, 1], 5008), ([1] * 4, 0):
        batch = batch_of(c, news, max_new=max(news), max_len=max_len)
        q = torch.randn(sum(news), H, D, generator=torch.Generator().manual_seed(max_len)).bfloat16()
        o, _, to, _ = ref.attention(c, q, starts_of(news))
        got = s2.cache_attention(cache, batch, q.cuda(), workspace=ws)
        assert ((got.double().cpu() - o).abs() <= to).all()
    s2.check_status()


@pytest.mark.parametrize("H,wide", [(4, False), (128, True)])
@pytest.mark.parametrize("length", [-1, 10 ** 6, 2 ** 31 - 1])
def test_sequences_without_new_tokens_take_no_part(length, H, wide):
    # a slot that no conversation holds: neither its length nor its pages are looked at
    c = ref.Paged([40, 33, 64], 2, 64, 16, 16)
    news = [2, 0, 1]
    q = torch.randn(3, H, 64, generator=torch.Generator().manual_seed(H)).bfloat16()
    o, _, to, _ = ref.attention(c, q, starts_of(news))
    c.lens[1] = length
    c.table[1] = -7
    for hints in (dict(max_new=2), dict(max_new=2, max_len=64)):
        cache, batch = on_gpu(c), batch_of(c, news, wide=wide, **hints)
        got = s2.cache_attention(cache, batch, q.cuda())
        s2.check_status()
        assert ((got.double().cpu() - o).abs() <= to).all()
        x = torch.randn(3, 2, 64).bfloat16().cuda()
        s2.cache_append(cache, batch, x, x, base=0.0)
        k, _ = s2.cache_read(cache, batch)
        s2.check_status()
        assert torch.equal(k, x)


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("D", [128, 64])
@pytest.mark.parametrize("power", [123, 120, 100, 0, -100])
def test_four_bit_keys_of_all_sizes(D, power, path):
    # rows up to 2^127 wide: their scale times 128, which the products go through, is beyond 32 bits
    lens, news = [700, 33], [3, 1]
    c = ref.Paged(lens, 2, D, 16, 4, seed=D)
    c.ks *= 2.0 ** power
    H = heads_of(path, news, 6)
    q = (torch.randn(4, H, D, generator=torch.Generator().manual_seed(7)) * 2.0 ** -power).bfloat16()
    check_not_finite(c, news, H, q, **hints_of(path, lens, news))
    rows, _ = s2.cache_read(on_gpu(c), batch_of(c, lens))
    assert rows.isfinite().all()


@pytest.mark.parametrize("first,second,scale,value", [  # largest errors among the bf16 numbers, were both roundings made
    (39.25, 50.0, 1.9609375, 5), (42.5, 44.75, 1.3359375, 4), (43.75, 50.0, 1.1171875, 6),
])
def test_four_bit_weights_are_rounded_once(first, second, scale, value):
    """The kernel for many rows writes the weights of a tile's first half before it knows the second half's maximum.
    Where that grows, they are scaled down, which must not round them again: all weight is the first half's here."""
    c = ref.Paged([256], 1, 64, 128, 4)
    pages = c.table[0, :2].long()
    score = torch.zeros(2, 128)
    score[1, :64], score[1, 64:] = first, second  # over sqrt(64): in powers of two 0, 7.1 to 7.9, 8.1 to 9
    B = 200  # so many conversations with the same pages that many are not cut between their two tiles
    c.table, c.lens = c.table.expand(B, -1).contiguous(), [256] * B
    c.k.zero_()  # rows whose channels are all their smallest value
    c.ks[pages, 0, :, 0], c.ks[pages, 0, :, 1] = 0.0, score.bfloat16()
    codes = torch.full((2, 128), 8, dtype=torch.uint8)
    codes[1, :64] += value
    c.v[pages, 0] = (codes | codes << 4)[..., None]
    c.vs[pages, 0, :, 0], c.vs[pages, 0, :, 1] = scale, -8 * scale
    q = torch.zeros(B, 64, 64).bfloat16()
    q[..., 0] = 1.0
    check_not_finite(c, [1] * B, 64, q, wide=True, max_new=1)
