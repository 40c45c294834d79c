"""logits_process_rows against float64.

Tolerances: l is made of a division or product, a product and a sum for the penalties, one sum for each bias, and a
product: 8 fp32 roundings of the magnitudes added up (``big``), so |delta l| <= 8 2^-24 big; written as logits, half a step
of the element type besides.  softmax: relative 2 max|delta l| + 1e-5 (the library's bound for the softmax itself) + half
a step; log softmax and LSE: the same, absolute against max(1, |value|).  Masked entries are exact.
"""
import numpy as np
import pytest
import torch

import row_wise_online_gb300 as rwo

pytestmark = pytest.mark.gpu
F32, BF, FP = torch.float32, torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _built():
    from row_wise_online_gb300 import _build

    _build.build()
    torch.cuda.set_device(0)


def dev(a, dtype=torch.int32):
    return torch.as_tensor(np.asarray(a), dtype=dtype).cuda()


def make(M, N, dt, seed, L=0, K=0, mask=False, params=True):
    rng = np.random.default_rng(seed)
    s = {"x": torch.from_numpy(rng.standard_normal((M, N)).astype(np.float32) * 3).to(dt)}
    if L:
        total = rng.integers(0, L + 1, M)
        total[0] = L
        tokens = np.minimum((N * rng.random((M, L)) ** 4).astype(np.int64), N - 1)
        tokens[rng.random((M, L)) < 0.05] = -1
        s |= {"tokens": tokens, "token_lens": total, "prompt_lens": (total * rng.random(M)).astype(np.int64)}
        if params:
            s |= {"repetition": 0.7 + rng.random(M), "frequency": rng.random(M) - 0.2, "presence": rng.random(M) - 0.3}
    if K:
        ids = rng.integers(-1, N, (M, K))
        ids[:, K // 2:] = np.where(rng.random((M, K - K // 2)) < 0.5, ids[:, :K - K // 2], ids[:, K // 2:])  # some twice
        s |= {"bias_ids": ids, "bias_values": 4 * rng.standard_normal((M, K))}
    if mask:
        s["mask"] = rng.integers(0, 2 ** 32, (M, (N + 31) // 32), dtype=np.uint64).astype(np.uint32)
    if params:
        s["scale"] = 0.5 + rng.random(M)
    return s


F = ("repetition", "frequency", "presence", "bias_values", "scale")


def args(s):
    a = {}
    for k, v in s.items():
        if k == "x":
            continue
        a[k] = dev(v.view(np.int32)) if k == "mask" else dev(v, F32 if k in F else torch.int32)
    return a


def reference(s):
    """(l, bound on |delta l|) in float64."""
    x = s["x"].double().numpy()
    M, N = x.shape
    f = {k: np.asarray(v).astype(np.float32).astype(np.float64) for k, v in s.items() if k in F}
    big = np.abs(x)
    if "tokens" in s:
        for r in range(M):
            toks = s["tokens"][r, :s["token_lens"][r]]
            gen = toks[s["prompt_lens"][r]:] if "prompt_lens" in s else toks
            seen = np.zeros(N, bool)
            seen[toks[(toks >= 0) & (toks < N)]] = True
            count = np.bincount(gen[(gen >= 0) & (gen < N)], minlength=N)
            rep, fr, pr = (f[k][r] if k in f else dflt for k, dflt in (("repetition", 1.0), ("frequency", 0.0), ("presence", 0.0)))
            x[r] = np.where(seen, np.where(x[r] > 0, x[r] / rep, x[r] * rep), x[r])
            big[r] = np.abs(x[r]) + (np.abs(fr) * count + abs(pr)) * (count > 0)
            x[r] -= (fr * count + pr) * (count > 0)
    if "bias_ids" in s:
        for r in range(M):
            ok = (s["bias_ids"][r] >= 0) & (s["bias_ids"][r] < N)
            np.add.at(x[r], s["bias_ids"][r][ok], f["bias_values"][r][ok])
            np.add.at(big[r], s["bias_ids"][r][ok], 2 * np.abs(f["bias_values"][r][ok]))
    if "scale" in f:
        x *= f["scale"][:, None]
        big = big * f["scale"][:, None]
    if "mask" in s:
        bits = np.unpackbits(np.ascontiguousarray(s["mask"]).view(np.uint8), axis=1, bitorder="little")[:, :N]
        x[bits == 0] = -np.inf
    return x, 8 * 2.0 ** -24 * np.where(np.isfinite(big), big, 0)


def check(s, y, lse, out, dt):
    l, dl = reference(s)
    y, lse = y.double().cpu().numpy(), lse.double().cpu().numpy()
    step = torch.finfo(dt).eps / 2
    small = 2.0 ** -25 if dt == FP else 2.0 ** -126
    dead = np.isneginf(l).all(1)
    m = np.where(dead, 0, l.max(1))
    d = np.exp(l - m[:, None]).sum(1)
    with np.errstate(divide="ignore"):
        want_lse = np.where(dead, -np.inf, m + np.log(d))
    worst = dl.max(1)
    assert np.array_equal(np.isneginf(lse), dead)
    off = np.abs(lse - want_lse)[~dead]
    assert (off <= (2 * worst + 1e-5 * np.maximum(1, np.abs(want_lse)))[~dead]).all()
    if out == "logits":
        none = np.isneginf(l)
        assert np.array_equal(np.isneginf(y), none)
        off = np.abs(y - l)[~none]
        assert (off <= (dl + step * (np.abs(l) + dl) + small)[~none]).all(), off.max()
    elif out == "softmax":
        want = np.where(dead[:, None], 0, np.exp(l - m[:, None]) / np.where(dead, 1, d)[:, None])
        assert (y[np.isneginf(l)] == 0).all() and (y[dead] == 0).all()
        assert (np.abs(y - want) <= (2 * worst[:, None] + 1e-5 + step * (1 + 1e-3)) * want + small).all()
    else:
        none = np.isneginf(l)
        assert np.array_equal(np.isneginf(y), none)
        with np.errstate(invalid="ignore"):
            want = l - want_lse[:, None]
        tol = 2 * worst[:, None] + 1e-5 * np.maximum(1, np.abs(want)) + step * np.abs(want) * (1 + 1e-3)
        assert (np.abs(y - want)[~none] <= tol[~none]).all()


@pytest.mark.parametrize("dt", [F32, BF, FP])
@pytest.mark.parametrize("out", ["logits", "softmax", "log_softmax"])
@pytest.mark.parametrize("M,N,L,K,mask", [(1, 1, 1, 1, True), (3, 7, 20, 3, True), (2, 33, 0, 0, True), (5, 1000, 64, 0, False), (4, 5003, 300, 40, True),
                                          (2, 32768, 500, 7, True), (3, 50021, 900, 1024, False), (1, 131072, 2000, 16, True), (1, 140001, 50, 5, True)])
def test_against_64_bits(M, N, L, K, mask, out, dt):
    s = make(M, N, dt, seed=M + N + L, L=L, K=K, mask=mask)
    lse = torch.full((M,), 9.0, device="cuda")
    y = rwo.logits_process_rows(s["x"].cuda(), out=out, lse_out=lse, **args(s))
    assert rwo.get_status() == rwo.OK
    check(s, y, lse, out, dt)


@pytest.mark.parametrize("out", ["logits", "softmax", "log_softmax"])
def test_rows_longer_than_a_cluster_holds(out):
    s = make(2, 600001, BF, seed=6, L=3000, K=33, mask=True)
    lse = torch.empty(2, device="cuda")
    y = rwo.logits_process_rows(s["x"].cuda(), out=out, lse_out=lse, **args(s))
    assert rwo.get_status() == rwo.OK
    check(s, y, lse, out, BF)


@pytest.mark.parametrize("out", ["logits", "softmax", "log_softmax"])
@pytest.mark.parametrize("N,L,K,mask", [(400003, 20000, 9, True), (300000, 70000, 0, False), (5000011, 40, 3, True)])
def test_parts_taken_in_chunks(N, L, K, mask, out):
    """More listed tokens, or a longer mask, than a CTA holds for its part; also in place, where the second pass reads what
    the first has not changed."""
    s = make(1, N, BF, seed=7, L=L, K=K, mask=mask)
    lse = torch.empty(1, device="cuda")
    a = args(s)
    x = s["x"].cuda()
    y = rwo.logits_process_rows(x, out=out, lse_out=lse, **a)
    assert rwo.get_status() == rwo.OK
    check(s, y, lse, out, BF)
    rwo.logits_process_rows(x, y=x, out=out, **a)
    assert torch.equal(x, y)


@pytest.mark.parametrize("M", [77, 151, 152, 400])
def test_row_counts_around_the_sms(M):
    """One CTA a row, two, or more rows than are resident."""
    s = make(M, 20011, FP, seed=M, L=300, K=20, mask=True)
    lse = torch.empty(M, device="cuda")
    y = rwo.logits_process_rows(s["x"].cuda(), lse_out=lse, **args(s))
    assert rwo.get_status() == rwo.OK
    check(s, y, lse, "softmax", FP)


def test_many_rows_and_no_options():
    s = make(700, 4100, FP, seed=8, params=False)
    lse = torch.empty(700, device="cuda")
    y = rwo.logits_process_rows(s["x"].cuda(), lse_out=lse)
    check(s, y, lse, "softmax", FP)
    ref = rwo.softmax_rows(s["x"].cuda())
    assert ((y.float() - ref.float()).abs() <= 2.0 ** -10 * ref.float() + 2.0 ** -24).all()  # two roundings of fp16, half a step each
    z = rwo.logits_process_rows(s["x"].cuda(), out="logits")
    assert torch.equal(z.cpu(), s["x"])  # nothing to do leaves every bit


def test_pitched_rows_in_place_and_odd_starts():
    for dt, a in ((BF, 3), (F32, 1), (FP, 8)):
        s = make(6, 2001, dt, seed=31, L=90, K=5, mask=True)
        wide = torch.full((6, 2100), 4.0, dtype=dt, device="cuda")
        view = wide[:, a:a + 2001]
        view.copy_(s["x"])
        lse = torch.empty(6, device="cuda")
        y = rwo.logits_process_rows(view, out="log_softmax", lse_out=lse, **args(s))
        check(s, y, lse, "log_softmax", dt)
        rwo.logits_process_rows(view, y=view, out="log_softmax", lse_out=lse, **args(s))
        assert torch.equal(view, y)
        assert (wide[:, :a] == 4).all() and (wide[:, a + 2001:] == 4).all()


def test_rows_that_the_mask_leaves_empty():
    s = make(3, 777, BF, seed=2, L=10, mask=True)
    s["mask"][1] = 0
    s["mask"][2] = 0
    s["mask"][2, 24] = 1 << 8  # element 776 alone
    for out in ("softmax", "log_softmax", "logits"):
        lse = torch.empty(3, device="cuda")
        y = rwo.logits_process_rows(s["x"].cuda(), out=out, lse_out=lse, **args(s))
        check(s, y, lse, out, BF)
    assert float(rwo.logits_process_rows(s["x"].cuda(), **args(s))[2, 776]) == 1.0


def test_infinite_entries_and_nan_under_the_mask():
    s = make(2, 300, F32, seed=4, L=30, mask=True)
    s["mask"][:] = 0xFFFFFFFF
    s["mask"][0, 1] = 0  # 32 .. 63
    s["x"][0, 32:64] = float("nan")
    s["x"][1, 5:9] = -float("inf")
    s["tokens"][1, :4] = [5, 6, 7, 8]
    s["token_lens"][1] = 30
    a = args(s)
    lse = torch.empty(2, device="cuda")
    y = rwo.logits_process_rows(s["x"].cuda(), lse_out=lse, **a)
    s["x"][0, 32:64] = 0.0  # whatever is masked does not count
    check(s, y, lse, "softmax", F32)


def test_counts_are_whole_and_repeated_tokens_add_up():
    """A token that occurs thousands of times, and every bias on one token."""
    N, L = 2000, 9000
    x = torch.zeros(1, N, device="cuda")
    tokens = np.full((1, L), 1234)
    tokens[0, :100] = 7
    y = rwo.logits_process_rows(x, out="logits", tokens=dev(tokens), token_lens=dev([L]), prompt_lens=dev([50]), frequency=dev([0.25], F32),
                                presence=dev([1.0], F32), bias_ids=dev([[3] * 5 + [-1]]), bias_values=dev([[1.0, 2.0, 4.0, 8.0, 16.0, 99.0]], F32))
    want = torch.zeros(N)
    want[1234], want[7], want[3] = -(0.25 * 8900 + 1), -(0.25 * 50 + 1), 31
    assert torch.equal(y[0].cpu(), want)
    s = make(2, 3001, BF, seed=3, L=5000, K=300, mask=True)
    first = rwo.logits_process_rows(s["x"].cuda(), **args(s))
    for _ in range(5):
        assert torch.equal(rwo.logits_process_rows(s["x"].cuda(), **args(s)), first)


def test_tokens_out_of_range_are_reported_and_ignored():
    s = make(2, 500, F32, seed=5, L=12, K=4)
    clean = {k: (v.copy() if hasattr(v, "copy") else v) for k, v in s.items()}
    clean["token_lens"][:] = 12
    dirty = {k: (v.copy() if hasattr(v, "copy") else v) for k, v in clean.items()}
    for key, val in (("tokens", 500), ("tokens", 2 ** 31 - 1), ("bias_ids", 500)):
        clean[key][0, 2] = -1
        dirty[key][0, 2] = val
        lse = torch.empty(2, device="cuda")
        y = rwo.logits_process_rows(s["x"].cuda(), out="log_softmax", lse_out=lse, **args(dirty))
        assert rwo.get_status() == rwo.ERR_INVALID_ARG
        check(clean, y, lse, "log_softmax", F32)
    dirty["token_lens"][1] = 13
    rwo.logits_process_rows(s["x"].cuda(), **args(dirty))
    assert rwo.get_status() == rwo.ERR_INVALID_ARG
    dirty["token_lens"][1], dirty["prompt_lens"][1] = 5, 6
    dirty["tokens"][0, 2] = dirty["bias_ids"][0, 2] = 0
    rwo.logits_process_rows(s["x"].cuda(), **args(dirty))
    assert rwo.get_status() == rwo.ERR_INVALID_ARG
    assert rwo.get_status() == rwo.OK


def test_binding_errors():
    x = torch.zeros(2, 64, device="cuda")
    t, n = dev([[1], [2]]), dev([1, 1])
    for bad in (dict(out="max"), dict(tokens=t), dict(token_lens=n), dict(frequency=dev([1, 1], F32)), dict(tokens=t.long(), token_lens=n),
                dict(bias_ids=t), dict(bias_ids=t, bias_values=dev([[1.0]], F32)), dict(mask=dev([[1], [1]])), dict(scale=dev([1], F32)),
                dict(y=torch.zeros(2, 63, device="cuda")), dict(y=torch.zeros(2, 64)), dict(lse_out=torch.zeros(2)), dict(scale=dev([1.0, 1.0], F32).cpu())):
        with pytest.raises(ValueError):
            rwo.logits_process_rows(x, **bad)
    with pytest.raises(TypeError):
        rwo.logits_process_rows(x.double())
