"""The 4-bit paged cache on the GPU: bytes written, values read back and attention over them, against numpy in 64 bits.

Tolerances: stored bytes and rotated queries are compared bit for bit with the documented fp32 arithmetic.  Values read
back are rounded once in fp32 and once to the element type.  The attention's bounds are derived in
kv4_reference.attention; its output is then rounded to the element type, by half a step at most.
"""
import numpy as np
import pytest
import torch

import row_wise_online_gb300 as rwo
from kv4_reference import Cache, attention, np_of, rotate

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _built():
    from row_wise_online_gb300 import _build

    _build.build()
    torch.cuda.set_device(0)


def dev(a, dtype=torch.int32):
    return torch.as_tensor(np.asarray(a), dtype=dtype).cuda()


def pool(lens, heads, page, d, seed, width=None):
    """Random codes, sensible scales, and NaN bytes in every place that holds no token; tables, with -1 behind a sequence."""
    rng = np.random.default_rng(seed)
    need = [-(-n // page) for n in lens]
    total = sum(need) + 2
    data = rng.integers(0, 256, (total, heads, page // 16, 20 * d), dtype=np.uint8)
    half = data.view(np.float16)
    s = np.exp(0.7 * rng.standard_normal(data.shape[:3] + (2, d // 2))) * 0.25
    z = -8 * s * (1 + 0.2 * rng.standard_normal(s.shape))
    half[..., 8 * d:] = np.stack([s, z], axis=-2).reshape(data.shape[:3] + (-1,))
    c = Cache(data)
    order = rng.permutation(total)
    table = np.full((len(lens), width or max(1, max(need))), -1, np.int32)
    used = np.zeros(total * page, bool)
    at = 0
    for b, n in enumerate(lens):
        table[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
        pos = np.arange(n)
        used[table[b][pos // page].astype(np.int64) * page + pos % page] = True
    for place in np.flatnonzero(~used):  # scales and zeros NaN
        p, x = divmod(int(place), page)
        for h in range(heads):
            hb = data[p, h, x // 16].view(np.float16)
            for hf in (c.k_half[x % 16], c.v_half[x % 16]):
                hb[hf] = hb[hf + 16 * c.G] = np.nan
    return c, table


def cu_of(news):
    return np.concatenate([[0], np.cumsum(news)]).astype(np.int32)


# ---- append and read back -------------------------------------------------------------------------------------

APPENDS = [
    # lens (with the new tokens), new tokens, kv heads, q heads, d, page, rotated, neighbours, dtype
    ([1], [1], 1, 1, 128, 16, 128, False, BF),
    ([17, 16, 33], None, 2, 6, 128, 16, 128, False, BF),
    ([40, 1, 64, 65], [40, 0, 3, 17], 3, 3, 64, 32, 64, False, FP),
    ([100, 31, 16], [100, 31, 1], 2, 4, 128, 48, 64, True, FP),
    ([50, 20], [9, 20], 1, 5, 64, 16, 8, True, BF),
    ([200], [133], 4, 0, 128, 64, 0, False, BF),
    ([30, 70], [2, 70], 5, 1, 64, 16, 32, False, BF),
]


@pytest.mark.parametrize("lens,news,heads,q_heads,d,page,rot,nb,dt", APPENDS)
def test_append_writes_the_documented_bytes(lens, news, heads, q_heads, d, page, rot, nb, dt):
    c, table = pool(lens, heads, page, d, seed=sum(lens) + d)
    cu = None if news is None else cu_of(news)
    T = len(lens) if cu is None else int(cu[-1])
    gen = torch.Generator().manual_seed(7)
    pad = 3 if cu is not None else 0  # rows behind the last sequence
    fused = torch.randn(T + pad, q_heads + 2 * heads, d, generator=gen).mul_(torch.exp(torch.randn(T + pad, q_heads + 2 * heads, 1, generator=gen)))
    fused = fused.to(dt).cuda()  # q, k, v of a token side by side
    q, k, v = fused[:, :q_heads], fused[:, q_heads:q_heads + heads], fused[:, q_heads + heads:]
    cs = None
    if rot:
        ang = np.arange(max(lens))[:, None] * 0.9 ** np.arange(rot // 2)
        cs = np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)
    data = torch.from_numpy(c.data).cuda()
    q_out = torch.full((T + pad, q_heads, d), 7.0, dtype=dt, device="cuda") if q_heads else None
    out = rwo.kv4_append(k, v, data, dev(table), dev(lens), cu_tokens=None if cu is None else dev(cu), q=q if q_heads else None, q_out=q_out,
                         cos_sin=None if cs is None else torch.from_numpy(cs).cuda(), interleaved=nb)
    assert rwo.get_status() == rwo.OK
    kf, vf, qf = (t.float().cpu().numpy() for t in (k, v, q))
    starts = np.arange(len(lens) + 1) if cu is None else cu
    want_q = np.full((T + pad, q_heads, d), 7.0, np.float32)
    for b, n in enumerate(lens):
        for i in range(starts[b], starts[b + 1]):
            pos = n - (starts[b + 1] - i)
            turn = (lambda x: rotate(x, cs[pos], nb)) if rot else (lambda x: x)
            for h in range(heads):
                c.put(table[b], pos, h, turn(kf[i, h]), vf[i, h])
            for h in range(q_heads):
                want_q[i, h] = turn(qf[i, h])
    assert np.array_equal(data.cpu().numpy(), c.data)
    if q_heads:
        assert out is q_out and torch.equal(q_out.cpu(), torch.from_numpy(want_q).to(dt))
        same = q.contiguous()  # in place
        rwo.kv4_append(k, v, data, dev(table), dev(lens), cu_tokens=None if cu is None else dev(cu), q=same, q_out=same,
                       cos_sin=None if cs is None else torch.from_numpy(cs).cuda(), interleaved=nb)
        assert torch.equal(same[:T], q_out[:T])


def test_append_groups_at_the_border():
    """Equal elements, zeros, one outlier, half-way quotients, subnormal ranges and values beyond fp16."""
    d = 128
    x = np.zeros((8, 1, d), np.float32)
    x[0] = 3.0
    x[1, 0, 5] = 1e4
    x[2] = np.tile(np.arange(32) * 0.5, 4)  # steps of 31/30: many near half-way
    x[3] = np.tile(np.arange(32) % 31 * 0.5, 4)  # range 15: s = 1, every odd one a tie
    x[4] = np.linspace(-1e-7, 1e-7, d)
    x[5] = np.linspace(-3e38, 3e38, d)
    x[6] = -x[3]
    x[7] = np.linspace(1e-3, 2e-3, d)
    k = torch.from_numpy(x).to(BF).cuda()
    data = rwo.kv4_cache_empty(1, 1, 16, d)
    rwo.kv4_append(k, k.flip(2), data, dev([[0]]), dev([8]), cu_tokens=dev([0, 8]))
    assert rwo.get_status() == rwo.OK
    want = Cache(np.zeros((1, 1, 1, 20 * d), np.uint8))
    kf = k.float().cpu().numpy()
    for i in range(8):
        want.put([0], i, 0, kf[i, 0], kf[i, 0, ::-1])
    assert np.array_equal(data.cpu().numpy(), want.data)


@pytest.mark.parametrize("heads,d,page,dt", [(1, 64, 16, BF), (3, 64, 48, FP), (2, 128, 32, BF), (5, 128, 16, FP)])
def test_gather_reads_the_values(heads, d, page, dt):
    lens, news = [65, 1, 40, 16], [65, 1, 7, 0]
    c, table = pool(lens, heads, page, d, seed=heads + d)
    cu = cu_of(news)
    T = int(cu[-1])
    # outputs as attention_forward takes them: [heads][tokens][d] underneath, with a row behind the last sequence
    k, v = (torch.full((heads, T + 1, d), 9.0, dtype=dt, device="cuda") for _ in range(2))
    rwo.kv4_gather(torch.from_numpy(c.data).cuda(), dev(table), dev(lens), cu_tokens=dev(cu), k=k.transpose(0, 1), v=v.transpose(0, 1))
    assert rwo.get_status() == rwo.OK
    assert (k[:, T] == 9).all() and (v[:, T] == 9).all()
    step = torch.finfo(dt).eps / 2
    for h in range(heads):
        for b, n in enumerate(lens):
            for got, ref in zip((k, v), c.sequence(table[b], n, h)):
                ref = ref[n - news[b]:]
                err = np.abs(np_of(got[h, cu[b]:cu[b + 1]]) - ref)
                assert (err <= (step * (1 + 2.0 ** -20) + 2.0 ** -23) * np.abs(ref) + (2.0 ** -25 if dt == FP else 0)).all()


# ---- attention ------------------------------------------------------------------------------------------------


def check_attention(c, table, lens, news, q_heads, dt, seed, scale=None, q_sd=1.0, cu_given=True, stream=None, spread=None):
    cu = cu_of(news)
    T = int(cu[-1])
    pad = 2 if cu_given else 0
    gen = torch.Generator().manual_seed(seed)
    fused = (q_sd * torch.randn(T + pad, q_heads + 2, c.d, generator=gen)).to(dt).cuda()
    q = fused[:, :q_heads]
    o = torch.full((T + pad, q_heads, c.d), 5.0, dtype=dt, device="cuda")
    lse = torch.full((T + pad, q_heads), 5.0, device="cuda")
    rwo.attention_kv4(q, torch.from_numpy(c.data).cuda(), dev(table), dev(lens), cu_tokens=dev(cu) if cu_given else None, o=o, lse_out=lse,
                      scale=scale, stream=stream)
    assert rwo.get_status(stream) == rwo.OK
    f32 = float(np.float32(scale if scale else 1 / np.sqrt(c.d)))
    want, want_lse, do, dl = attention(c, table, lens, cu, np_of(q)[:T], f32)
    assert (o[T:] == 5).all() and (lse[T:] == 5).all()
    got, got_lse = np_of(o)[:T], np_of(lse)[:T]
    none = np.isneginf(want_lse)
    assert np.isneginf(got_lse[none]).all() and (got[none] == 0).all()
    bound = do + torch.finfo(dt).eps / 2 * (np.abs(want) + do) + 2.0 ** -24
    off = np.abs(got - want)
    assert (off <= bound).all(), (off.max(), (off / bound).max(), np.unravel_index(np.argmax(off / bound), off.shape))
    off = np.abs(got_lse - want_lse)[~none]
    assert (off <= dl[~none]).all(), (off / dl[~none]).max()


LENS = [[1], [16], [63], [64, 65], [1, 2, 15, 16, 17, 31, 33, 47, 48, 127, 128, 129], [0, 5, 0, 300, 0], [700, 3, 1500, 40]]


@pytest.mark.parametrize("dt", [BF, FP])
@pytest.mark.parametrize("d,heads,group,page", [(128, 1, 1, 16), (128, 2, 4, 32), (128, 2, 8, 16), (64, 3, 3, 48), (64, 1, 7, 64),
                                                (128, 1, 16, 16), (64, 2, 9, 16), (128, 1, 33, 32)])
@pytest.mark.parametrize("lens", LENS, ids=lambda v: "-".join(map(str, v)))
def test_decode_against_64_bits(lens, d, heads, group, page, dt):
    c, table = pool(lens, heads, page, d, seed=sum(lens) + d + group)
    check_attention(c, table, lens, [1] * len(lens), heads * group, dt, seed=group, cu_given=len(lens) % 2 == 0)


@pytest.mark.parametrize("dt,d", [(BF, 128), (FP, 64)])
@pytest.mark.parametrize("lens,news", [([5], [5]), ([40, 7, 80], [2, 0, 5]), ([16, 64, 130], [16, 3, 17]), ([3, 9], [5, 9]),
                                       ([200, 1, 90, 33], [4, 1, 4, 4]), ([300], [100])])
@pytest.mark.parametrize("group", [1, 4, 12])
def test_several_tokens_a_sequence(lens, news, group, dt, d):
    """Drafts and short prompts: each token sees the ones before it; a sequence with no tokens here, one shorter than its rows."""
    c, table = pool(lens, 2, 16, d, seed=sum(lens) + group)
    check_attention(c, table, lens, news, 2 * group, dt, seed=group)


def test_sharp_rows_and_scales():
    """Scores spread over hundreds, so that the maximum moves often, in both directions along the keys."""
    lens = [900, 2000]
    c, table = pool(lens, 2, 16, 128, seed=5)
    check_attention(c, table, lens, [1, 1], 8, BF, seed=3, q_sd=12.0, cu_given=False)
    check_attention(c, table, lens, [3, 2], 8, FP, seed=4, q_sd=0.01, scale=3.0)
    check_attention(c, table, lens, [3, 2], 8, BF, seed=4, q_sd=1e-20, scale=0.7)  # nearly uniform weights, tiny q
    check_attention(c, table, lens, [1, 2], 8, BF, seed=4, q_sd=1e15, scale=1e-15)


@pytest.mark.parametrize("grow", [1.002, 0.998])
def test_value_scales_that_grow_or_shrink(grow):
    """V's scales run over many powers of two along the keys; some are zero, some as large as fp16 has."""
    lens = [3000]
    c, table = pool(lens, 1, 32, 128, seed=9)
    for pos in range(lens[0]):
        hb, hf = c.block(table[0], pos, 0).view(np.float16), c.v_half[pos % 16]
        f = np.float16(grow ** pos * (0.02 if grow > 1 else 1.0))
        hb[hf], hb[hf + 64] = hb[hf] * f, hb[hf + 64] * f
        if pos % 7 == 0:
            hb[hf] = 0
    check_attention(c, table, lens, [2], 4, BF, seed=1)
    hb, hf = c.block(table[0], 1234, 0).view(np.float16), c.v_half[1234 % 16]
    hb[hf] = 4000.0
    check_attention(c, table, lens, [2], 4, FP, seed=1)


def test_all_scales_zero():
    lens = [70]
    c, table = pool(lens, 1, 16, 64, seed=2)
    for pos in range(70):
        hb = c.block(table[0], pos, 0).view(np.float16)
        hb[c.v_half[pos % 16]] = 0
        hb[c.k_half[pos % 16]] = 0
    check_attention(c, table, lens, [1], 2, BF, seed=1)


def test_long_and_short_together():
    """One long sequence among short ones: its keys are spread over many runs and merged, theirs are not."""
    lens = [37, 60000, 5, 0, 900]
    c, table = pool(lens, 2, 64, 64, seed=11)
    check_attention(c, table, lens, [1, 2, 1, 1, 3], 8, BF, seed=8)


def test_many_sequences():
    lens = [int(n) for n in np.random.default_rng(1).integers(0, 90, 300)]
    c, table = pool(lens, 1, 16, 64, seed=12, width=9)
    check_attention(c, table, lens, [1] * 300, 2, FP, seed=8, cu_given=False)


@pytest.mark.parametrize("dt,d,group", [(BF, 128, 8), (FP, 128, 16), (BF, 64, 4), (BF, 64, 16)])
@pytest.mark.parametrize("most,batch", [(900, 150), (3000, 60)])
def test_many_ragged_sequences(most, batch, dt, d, group):
    """More (sequence, head)s than runs, of one to many tiles: runs that start and end at any place, and some between."""
    rng = np.random.default_rng(most + d + group)
    lens = [int(n) for n in rng.integers(0, most, batch)]
    news = [int(n) for n in rng.integers(0, 4, batch)]
    c, table = pool(lens, 4, 32, d, seed=batch, width=-(-most // 32))
    check_attention(c, table, lens, news, 4 * group, dt, seed=group)


def test_results_do_not_change_from_call_to_call():
    lens = [5000, 700]
    c, table = pool(lens, 2, 16, 128, seed=4)
    q = torch.randn(2, 16, 128, device="cuda").to(BF)
    a = (q, torch.from_numpy(c.data).cuda(), dev(table), dev(lens))
    first = rwo.attention_kv4(*a)
    ws = rwo.attention_kv4_workspace(2, 2, 16, 2, 128)
    ws.fill_(255)  # nothing in the workspace is kept from call to call
    for _ in range(5):
        assert torch.equal(rwo.attention_kv4(*a, workspace=ws), first)


def test_another_stream_and_two_at_once():
    lens = [4000, 3]
    c, table = pool(lens, 2, 16, 128, seed=21)
    s = torch.cuda.Stream()
    check_attention(c, table, lens, [1, 1], 8, BF, seed=2, cu_given=False, stream=s)
    check_attention(c, table, lens, [1, 1], 8, BF, seed=2, cu_given=False, stream=int(s.cuda_stream))
    data, tab, ln = torch.from_numpy(c.data).cuda(), dev(table), dev(lens)
    qs = [torch.randn(2, 8, 128, device="cuda").to(BF) for _ in range(2)]
    alone = [rwo.attention_kv4(q, data, tab, ln) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[], []]
    for _ in range(20):
        for k in range(2):
            outs[k].append(rwo.attention_kv4(qs[k], data, tab, ln, stream=streams[k]))
    torch.cuda.synchronize()
    assert all(torch.equal(o, alone[k]) for k in range(2) for o in outs[k])


# ---- values on the device that are out of range: reported, nothing followed -----------------------------------


def test_bad_pages_lengths_and_offsets_are_reported():
    d, heads = 64, 2
    lens = [40, 20]
    c, table = pool(lens, heads, 16, d, seed=3)
    data = torch.from_numpy(c.data).cuda()
    before = data.clone()
    k = torch.randn(2, heads, d, device="cuda").to(BF)
    q = torch.randn(2, 4, d, device="cuda").to(BF)
    good = rwo.attention_kv4(q, data, dev(table), dev(lens))
    assert rwo.get_status() == rwo.OK
    cs = torch.ones(30, 16, device="cuda")
    last = table.copy()
    last[0, 2] = 10 ** 6  # position 39
    low = table.copy()
    low[0, 2] = -5
    for tab, ln, kw in [(last, lens, {}), (low, lens, {}), (table, [0, 20], {}), (table, [10 ** 6, 20], {}), (table, [-3, 20], {}),
                        (table, lens, {"cos_sin": cs})]:
        data.copy_(before)
        rwo.kv4_append(k, k, data, dev(tab), dev(ln), **kw)
        assert rwo.get_status() == rwo.ERR_INVALID_ARG
        assert rwo.get_status() == rwo.OK
        changed = (data != before).flatten(1).any(1).cpu().numpy()
        assert set(np.flatnonzero(changed)) == {int(table[1, 1])}  # the other sequence's token alone
        data.copy_(before)
        out = [torch.full((2, heads, d), 3.0, dtype=BF, device="cuda") for _ in range(2)]
        if not kw:
            rwo.kv4_gather(data, dev(tab), dev(ln), k=out[0], v=out[1])
            assert rwo.get_status() == rwo.ERR_INVALID_ARG
            assert (out[0][0] == 3).all() and not (out[0][1] == 3).all()
        if not kw and ln[0]:
            o = rwo.attention_kv4(q, data, dev(tab), dev(ln))
            assert rwo.get_status() == rwo.ERR_INVALID_ARG
            assert torch.equal(o[1], good[1])
    for cu in ([0, 5, 2], [-1, 1, 2], [0, 1, 9], [1, 0, 2]):
        rwo.kv4_append(k, k, data, dev(table), dev(lens), cu_tokens=dev(cu))
        assert rwo.get_status() == rwo.ERR_INVALID_ARG
        rwo.attention_kv4(q, data, dev(table), dev(lens), cu_tokens=dev(cu))
        assert rwo.get_status() == rwo.ERR_INVALID_ARG


def test_bad_lengths_among_runs_of_tokens():
    """The same where sequences bring many tokens: one too long for its table, one of negative length, one shorter than its
    rows, a page that is none, positions without angles."""
    d, heads = 128, 2
    lens, news = [40, 40, 40, 40, 90], [20, 20, 20, 30, 90]
    c, table = pool([40, 40, 40, 40, 90], heads, 16, d, seed=5)
    table[3, 1] = 10 ** 6
    cu, told = dev(cu_of(news)), [10 ** 6, -7, 9, 40, 90]
    before = torch.from_numpy(c.data).cuda()
    gen = torch.Generator(device="cuda").manual_seed(2)
    k, v = (torch.randn(180, heads, d, generator=gen, device="cuda").to(BF) for _ in range(2))
    q = torch.randn(180, 3, d, generator=gen, device="cuda").to(BF)
    cs = torch.ones(80, 64, device="cuda")
    data, out = before.clone(), torch.full((180, 3, d), 5.0, dtype=BF, device="cuda")
    rwo.kv4_append(k, v, data, dev(table), dev(told), cu_tokens=cu, q=q, q_out=out, cos_sin=cs)
    assert rwo.get_status() == rwo.ERR_INVALID_ARG
    # sequence 2 (9 tokens for 20 rows): its last 9 rows; 3: positions 10 .. 15 and 32 ..; 4: positions below 80
    written = [i for i in range(180) if 51 <= i < 60 or 60 <= i < 66 or 82 <= i < 90 or 90 <= i < 170]
    where = [(2, i - 51) for i in range(51, 60)] + [(3, 10 + i - 60) for i in range(60, 66)] + \
            [(3, 10 + i - 60) for i in range(82, 90)] + [(4, i - 90) for i in range(90, 170)]
    kf, vf, ones = k.float().cpu().numpy(), v.float().cpu().numpy(), np.ones(64, np.float32)
    for i, (b, pos) in zip(written, where):
        for h in range(heads):
            c.put(table[b], pos, h, rotate(kf[i, h], ones, False), vf[i, h])
    assert np.array_equal(data.cpu().numpy(), c.data)
    touched = (out != 5).flatten(1).any(1).cpu().numpy()
    assert list(np.flatnonzero(touched)) == written
    ks, vs = (torch.full((180, heads, d), 5.0, dtype=BF, device="cuda") for _ in range(2))
    rwo.kv4_gather(data, dev(table), dev(told), cu_tokens=cu, k=ks, v=vs)
    assert rwo.get_status() == rwo.ERR_INVALID_ARG
    touched = (ks != 5).flatten(1).any(1).cpu().numpy()
    assert list(np.flatnonzero(touched)) == written + list(range(170, 180))  # (reading back needs no angles)


def test_offsets_that_descend_do_not_overflow():
    """Offsets 0, T, 0, T, ...: half of the sequences claim every row, more units than 32 bits count."""
    T, B, heads, d = 200000, 20000, 16, 64
    data = rwo.kv4_cache_empty(1, heads, T, d)
    k = torch.zeros(T, heads, d, dtype=BF, device="cuda")
    cu = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    cu[1::2] = T
    lens = torch.full((B,), T, dtype=torch.int32, device="cuda")
    table = torch.zeros(B, 1, dtype=torch.int32, device="cuda")
    rwo.kv4_append(k, k, data, table, lens, cu_tokens=cu)
    assert rwo.get_status() == rwo.ERR_INVALID_ARG
    assert not data.any()


def test_binding_errors():
    data = rwo.kv4_cache_empty(4, 2, 16, 64)
    tab, ln = dev([[0]]), dev([3])
    k = torch.zeros(1, 2, 64, dtype=BF, device="cuda")
    rwo.kv4_append(k, k, data, tab, ln)
    for bad in (lambda: rwo.kv4_append(k, k[:, :1], data, tab, ln), lambda: rwo.kv4_append(k, k.half(), data, tab, ln),
                lambda: rwo.kv4_append(k, k, data, tab.long(), ln), lambda: rwo.kv4_append(k, k, data.int(), tab, ln),
                lambda: rwo.kv4_append(k, k, data, tab, ln, q_out=k), lambda: rwo.kv4_append(k[..., ::2], k, data, tab, ln),
                lambda: rwo.attention_kv4(k.repeat(2, 1, 1), data, tab, ln), lambda: rwo.attention_kv4(k, data, tab, ln.cpu()),
                lambda: rwo.attention_kv4(k, data, tab, ln, lse_out=torch.zeros(1, 2)), lambda: rwo.kv4_gather(data, tab, ln, cu_tokens=dev([0, 1]))):
        with pytest.raises((ValueError, TypeError)):
            bad()
    with pytest.raises(rwo.SoftmaxError) as e:
        rwo.attention_kv4(torch.zeros(1, 3, 64, dtype=BF, device="cuda"), data, tab, ln)
    assert e.value.status == rwo.ERR_INVALID_ARG
    with pytest.raises(TypeError):
        rwo.attention_kv4(k.double(), data, tab, ln)
    with pytest.raises(rwo.SoftmaxError) as e:
        rwo.attention_kv4(k.float(), data, tab, ln)
    assert e.value.status == rwo.ERR_UNSUPPORTED
    with pytest.raises(rwo.SoftmaxError):
        rwo.attention_kv4(k, data, tab, ln, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
