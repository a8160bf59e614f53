"""The attention side on the GPU against its oracle (oracle/attention.py):
qk_norm_rope, KVCache4 (write, read, attend) and prompt_attention, alone and
together.

Cache contents are bit-exact.  Bounds of the computed outputs, per element,
u = 2^-24 (half a step of float32) and h = 2^-8 (half a step of bfloat16):
- norm_rope: h |y| for the rounding of the output, and 32 u times the sum of
  the magnitudes joined by the last addition (a mean over at most 8 + 6
  additions in a row enters with half its relative error; a reciprocal square
  root, three products and one addition of at most 2 u each).
- attention: a score is off by at most e = (D + 8) u reach (reach = largest
  sum |q||k| scale; D products and sums, the scaling and the exponent's
  argument), a probability by 2 e + 16 u relative (its own and the sum's; the
  exponential 4 u, a float32 sum over few partial sums) and by h where it is
  rounded to bfloat16 for the second product: out within
  (h + 2 e + 64 u) spread + h |out|, spread = sum p |v|.  lse within
  e + 64 u + 4 u |lse|.
"""

import numpy as np
import pytest
import torch

import moe_layer_05_amd as mm
from moe_layer_05_amd import workloads
from oracle import attention as oa
from tests.helpers import np_f32

pytestmark = pytest.mark.gpu
DEV = "cuda"
U, H = 2.0 ** -24, 2.0 ** -8


def say(*a):
    print("[case]", *a, flush=True)


def gen(seed):
    return torch.Generator().manual_seed(seed)


def normal(g, *shape, scale=1.0):
    return (torch.randn(*shape, generator=g) * scale).to(torch.bfloat16)


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def close(got, ref, bound, what=""):
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    assert np.array_equal(np.isnan(got), np.isnan(ref)), what
    fine = np.isfinite(ref)
    assert np.array_equal(got[~fine & ~np.isnan(ref)], ref[~fine & ~np.isnan(ref)]), what
    off = np.abs(got[fine] - ref[fine]) - np.asarray(np.broadcast_to(bound, ref.shape))[fine]
    assert off.size == 0 or off.max() <= 0, f"{what}: over the bound by {off.max():.3g}"


# ------------------------------------------------------------------ norms and rotation

_TABLES = {}


def table(max_pos, R):
    if (max_pos, R) not in _TABLES:
        _TABLES[max_pos, R] = workloads.rope_table(max_pos, R)
    return _TABLES[max_pos, R]


def check_heads(x, w, y, pos, tab, R, inter, eps):
    ref, size = oa.norm_rope(np_f32(x), None if w is None else f64(w), eps, pos.numpy(),
                             tab.numpy(), R, inter)
    close(f64(y), ref, H * np.abs(ref) + 32 * U * size, "norm_rope")


@pytest.mark.parametrize("T,NHq,NHk,D,R,inter,wdt", [
    (1, 1, 1, 8, 8, True, torch.bfloat16), (5, 3, 0, 16, 16, False, torch.float32),
    (16, 16, 2, 128, 128, False, torch.bfloat16), (33, 7, 3, 64, 32, False, None),
    (9, 16, 16, 192, 64, True, None), (7, 5, 5, 200, 112, False, torch.bfloat16),
    (3, 40, 8, 256, 256, True, torch.float32), (2, 9, 1, 512, 512, False, torch.bfloat16),
    (11, 65, 13, 40, 16, True, torch.bfloat16), (1200, 33, 4, 128, 64, False, torch.bfloat16),
])
def test_norm_rope(T, NHq, NHk, D, R, inter, wdt):
    say("norm_rope", T, NHq, NHk, D, R, inter, wdt)
    g = gen(T * 1000 + D)
    q, k = normal(g, T, NHq, D, scale=3.0), normal(g, T, NHk, D) if NHk else None
    pos = torch.randint(0, 300, (T,), generator=g, dtype=torch.int64)
    tab = table(300, R)
    w = [None, None] if wdt is None else [(1 + 0.3 * torch.randn(D, generator=g)).to(wdt) for _ in range(2)]
    dev = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    wk = w[1] if NHk else None
    qo, ko = mm.qk_norm_rope(dev(q), dev(k), pos.to(DEV), tab.to(DEV), R, dev(w[0]), dev(wk), 1e-5,
                             interleaved=inter)
    rows = slice(0, T) if T <= 64 else np.r_[0:8, T - 8:T]
    check_heads(q[rows], w[0], qo.cpu()[rows], pos[rows], tab, R, inter, 1e-5)
    if NHk:
        check_heads(k[rows], wk, ko.cpu()[rows], pos[rows], tab, R, inter, 1e-5)
    else:
        assert ko is None


def test_norm_rope_in_place_and_strided():
    """The heads of a fused projection normed where they lie; the value part
    and the row behind stay as they are; clamped positions."""
    say("norm_rope in place")
    g = gen(5)
    T, NHq, NHk, D, R = 21, 6, 2, 64, 64
    qkv = normal(g, T + 1, (NHq + 2 * NHk) * D).to(DEV)
    before = qkv.clone()
    q = qkv[:T, :NHq * D].view(T, NHq, D)
    k = qkv[:T, NHq * D:(NHq + NHk) * D].view(T, NHk, D)
    pos = torch.arange(T, dtype=torch.int64) * 3
    pos[0], pos[1] = -7, 10 ** 12
    w = normal(g, D)
    a, b = mm.qk_norm_rope(q, k, pos.to(DEV), table(40, R).to(DEV), R, w.to(DEV), w.to(DEV), q_out=q, k_out=k)
    assert a is q and b is k
    bc = before.cpu()
    check_heads(bc[:T, :NHq * D].view(T, NHq, D), w, q.cpu(), pos, table(40, R), R, False, 1e-6)
    check_heads(bc[:T, NHq * D:(NHq + NHk) * D].view(T, NHk, D), w, k.cpu(), pos, table(40, R), R, False, 1e-6)
    assert torch.equal(qkv[:T, (NHq + NHk) * D:], before[:T, (NHq + NHk) * D:])
    assert torch.equal(qkv[T], before[T])


def test_norm_rope_extremes():
    """Zero heads (eps alone), tiny and large values, a NaN and an infinity
    that stay in their heads."""
    say("norm_rope extremes")
    g = gen(6)
    q = normal(g, 6, 2, 64)
    q[0, 0] = 0
    q[1] *= 1e-18
    q[2] *= 1e15
    q[3, 0, 5] = float("nan")
    q[4, 1, 63] = float("inf")
    pos = torch.zeros(6, dtype=torch.int64)
    w = torch.ones(64)
    y, _ = mm.qk_norm_rope(q.to(DEV), None, pos.to(DEV), table(40, 64).to(DEV), 64, w.to(DEV))
    bad = torch.zeros(6, 2, dtype=torch.bool)
    bad[3, 0] = bad[4, 1] = True
    y = y.cpu()
    assert torch.isnan(y[3, 0]).all() and torch.isnan(y[4, 1]).any()
    ref, size = oa.norm_rope(np_f32(torch.where(bad[..., None], torch.zeros(()).to(q), q)), f64(w), 1e-6, pos.numpy(),
                             table(40, 64).numpy(), 64, False)
    keep = ~bad.numpy()
    close(f64(y)[keep], ref[keep], (H * np.abs(ref) + 32 * U * size)[keep])


# ------------------------------------------------------------------ the cache

def paged(g, lens, page, extra=2):
    """A table of shuffled distinct pages for sequences of ``lens``."""
    per = [-(-n // page) for n in lens]
    order = torch.randperm(sum(per) + extra, generator=g).tolist()
    t = torch.full((len(lens), max(per + [1])), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(per):
        t[b, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
        at += n
    return t, sum(per) + extra


def cu(lens):
    return np.concatenate([[0], np.cumsum(lens)]).astype(np.int32).tolist()


@pytest.mark.parametrize("D,NKV,page,new,before", [
    (64, 1, 16, [1], [0]), (128, 2, 16, [1, 1, 1], [0, 15, 16]), (192, 3, 32, [17, 0, 5], [3, 9, 40]),
    (256, 1, 48, [50], [31]), (128, 4, 64, [64, 1, 130, 0], [0, 63, 1, 0]), (64, 2, 4096, [33], [4090]),
])
def test_cache_bit_exact(D, NKV, page, new, before):
    """Writing changes exactly the bytes of the new tokens, to the oracle's;
    reading gives the values the bytes stand for, in bfloat16."""
    say("cache", D, NKV, page, new, before)
    g = gen(D + page)
    total = [a + b for a, b in zip(before, new)]
    tab, n = paged(g, total, page)
    pages = torch.randint(0, 251, (n, NKV, page // 16, 17 * D), generator=g, dtype=torch.uint8)
    T = sum(new)
    k, v = normal(g, T, NKV, D), normal(g, T, NKV, D, scale=20.0)
    k[T // 2] *= 1e-3
    ref = pages.numpy().copy()
    for b in range(len(new)):
        for i in range(new[b]):
            pos = before[b] + i
            for h in range(NKV):
                t = cu(new)[b] + i
                oa.put(ref, int(tab[b, pos // page]), h, pos % page, f64(k[t, h]), f64(v[t, h]))
    c = mm.KVCache4.of(pages.to(DEV))
    c.write(k.to(DEV), v.to(DEV), tab.to(DEV), i32(before), i32(cu(new)))
    assert np.array_equal(c.pages.cpu().numpy(), ref)
    kb, vb = c.read(tab.to(DEV), i32([0] * len(new)), i32(cu(total)), sum(total))
    rows = range(sum(total)) if sum(total) < 300 else [0, 1, sum(total) - 1]
    for t in rows:
        b = int(np.searchsorted(cu(total)[1:], t, side="right"))
        pos = t - cu(total)[b]
        for h in range(NKV):
            x, y = oa.get(ref, int(tab[b, pos // page]), h, pos % page)
            assert np.array_equal(f64(kb[t, h]), x) and np.array_equal(f64(vb[t, h]), y), (t, h)


def test_cache_every_bfloat16():
    """All finite bfloat16 values as members of groups of many scales, ties
    included, and groups with an infinity or NaN."""
    say("cache values")
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    bits = bits[torch.isfinite(bits.float())]
    g = gen(3)
    x = bits[torch.randperm(len(bits), generator=g)][:65024].view(-1, 1, 64)
    near = normal(g, 512, 1, 64) * torch.exp2(torch.randint(-100, 100, (512, 1, 1), generator=g).float()).to(torch.bfloat16)
    ties = (torch.randint(-28, 29, (64, 1, 64), generator=g) / 4).to(torch.bfloat16)
    odd = normal(g, 4, 1, 64)
    odd[0, 0, 3], odd[1, 0, 40], odd[2, 0, 31], odd[3] = float("inf"), float("nan"), float("-inf"), 0.0
    x = torch.cat([x, near, ties, odd])
    T = len(x)
    tab = torch.arange((T + 255) // 256, dtype=torch.int32)[None]
    c = mm.KVCache4(tab.numel(), 256, 1, 64)
    c.write(x.to(DEV), x.flip(0).contiguous().to(DEV), tab.to(DEV), i32([0]), i32([0, T]))
    k, v = c.read(tab.to(DEV), i32([0]), i32([0, T]), T)
    want = oa.values(*oa.quantise(f64(x[:, 0])))
    assert np.array_equal(f64(k)[:, 0], want, equal_nan=True)
    assert np.array_equal(f64(v)[:, 0], want[::-1], equal_nan=True)


def test_cache_reads_into_parts_of_rows():
    """k and v as the two parts of the rows of one tensor."""
    say("cache into parts")
    g = gen(9)
    D, NKV, n = 64, 2, 20
    k, v = normal(g, n, NKV, D).to(DEV), normal(g, n, NKV, D).to(DEV)
    c, tab = mm.KVCache4(2, 16, NKV, D), i32([[1, 0]])
    c.write(k, v, tab, i32([0]), i32([0, n]))
    a, b = c.read(tab, i32([0]), i32([0, n]), n)
    rows = torch.full((n, 3 * NKV * D), 5.0, dtype=torch.bfloat16, device=DEV)
    parts = rows.view(n, 3, NKV, D)
    c.read(tab, i32([0]), i32([0, n]), n, k=parts[:, 0], v=parts[:, 2])
    assert torch.equal(parts[:, 0], a) and torch.equal(parts[:, 2], b) and (parts[:, 1] == 5.0).all()


def test_cache_skips_what_has_no_place():
    """Negative starts, positions behind the table, page ids outside the
    cache: nothing is written there and zeros are read; rows behind the last
    sequence stay in given tensors and are zero in new ones."""
    say("cache without places")
    g = gen(8)
    D, NKV, page, n = 128, 2, 16, 5
    pages = torch.randint(0, 251, (n, NKV, 1, 17 * D), generator=g, dtype=torch.uint8)
    tab = torch.tensor([[0, -1], [1, 5], [2, 2 ** 31 - 1], [3, -2 ** 31]], dtype=torch.int32)
    start, new = [-3, 14, 30, -2 ** 31], [6, 5, 4, 2]
    T = sum(new) + 3
    k, v = normal(g, T, NKV, D), normal(g, T, NKV, D)
    ref = pages.numpy().copy()
    for b in range(4):
        for i in range(new[b]):
            pos, t = start[b] + i, cu(new)[b] + i
            if 0 <= pos < 32 and 0 <= int(tab[b, pos // 16]) < n:
                for h in range(NKV):
                    oa.put(ref, int(tab[b, pos // 16]), h, pos % 16, f64(k[t, h]), f64(v[t, h]))
    c = mm.KVCache4.of(pages.to(DEV))
    c.write(k.to(DEV), v.to(DEV), tab.to(DEV), i32(start), i32(cu(new)))
    assert np.array_equal(c.pages.cpu().numpy(), ref)
    mine = normal(g, T, NKV, D).to(DEV)
    ko, vo = mine.clone(), mine.clone()
    c.read(tab.to(DEV), i32(start), i32(cu(new)), T, k=ko, v=vo)
    kz, vz = c.read(tab.to(DEV), i32(start), i32(cu(new)), T)
    for b in range(4):
        for i in range(new[b]):
            pos, t = start[b] + i, cu(new)[b] + i
            has = 0 <= pos < 32 and 0 <= int(tab[b, pos // 16]) < n
            want = oa.get(ref, int(tab[b, pos // 16]), 1, pos % 16)[0] if has else np.zeros(D)
            assert np.array_equal(f64(ko[t, 1]), want) and np.array_equal(f64(kz[t, 1]), want)
    assert torch.equal(ko[-3:], mine[-3:]) and torch.equal(vo[-3:], mine[-3:])
    assert not kz[-3:].any() and not vz[-3:].any()


def filled(g, tab, n, lens, page, NKV, D):
    """A cache with noise everywhere (NaN scales among it) and tokens written
    at the sequences' places; (cache, keys, values) as its values."""
    pages = torch.randint(0, 256, (n, NKV, page // 16, 17 * D), generator=g, dtype=torch.uint8)
    pages[..., 8 * D:8 * D + D // 2] = 255                 # whatever lies behind a sequence reads as NaN
    pages[..., 16 * D + D // 2:] = 255
    c = mm.KVCache4.of(pages.to(DEV))
    T = sum(lens)
    k, v = normal(g, max(T, 1), NKV, D, scale=1.5), normal(g, max(T, 1), NKV, D)
    c.write(k.to(DEV), v.to(DEV), tab.to(DEV), i32([0] * len(lens)), i32(cu(lens)))
    val = lambda x: oa.values(*oa.quantise(f64(x)))  # noqa: E731
    return c, val(k), val(v)


def check_attend(out, lse, q, k, v, lens, scale, D):
    B, NHq, _ = q.shape
    NKV = k.shape[1]
    at = cu(lens)
    for b in range(B):
        for h in range(NHq):
            s = slice(at[b], at[b] + lens[b])
            o, z, spread, reach = oa.attend(f64(q[b, h])[None], k[s, h // (NHq // NKV)],
                                            v[s, h // (NHq // NKV)], scale)
            e = (D + 8) * U * reach[0]
            close(f64(out[b, h]), o[0], (H + 2 * e + 64 * U) * spread[0] + H * np.abs(o[0]), f"out {b} {h}")
            close(f64(lse[b, h]), z[0], e + 64 * U + 4 * U * abs(z[0]) if lens[b] else 0.0, f"lse {b} {h}")


@pytest.mark.parametrize("D,NHq,NKV,page,lens", [
    (64, 1, 1, 16, [1]), (128, 4, 2, 16, [0, 1, 2, 15, 16, 17, 31, 32, 33]),
    (192, 6, 3, 32, [63, 64, 65, 127, 0]), (256, 16, 1, 48, [100, 200]),
    (128, 34, 2, 64, [129, 500]), (64, 40, 1, 16, [300]), (128, 16, 2, 128, [1025, 7, 2000]),
    (256, 5, 5, 256, [777]), (192, 8, 8, 16, [260, 3]),
])
def test_attend(D, NHq, NKV, page, lens):
    say("attend", D, NHq, NKV, page, lens)
    g = gen(D * 7 + NHq)
    tab, n = paged(g, lens, page)
    c, k, v = filled(g, tab, n, lens, page, NKV, D)
    q = normal(g, len(lens), NHq, D)
    out, lse = c.attend(q.to(DEV), tab.to(DEV), i32(lens), return_lse=True)
    check_attend(out, lse, q, k, v, lens, D ** -0.5, D)
    # a wider table: more splits, the same sequences
    wide = torch.full((len(lens), tab.shape[1] + 4000 // page), -1, dtype=torch.int32)
    wide[:, :tab.shape[1]] = tab
    out2, lse2 = c.attend(q.to(DEV), wide.to(DEV), i32(lens), return_lse=True)
    check_attend(out2, lse2, q, k, v, lens, D ** -0.5, D)


def test_attend_long_and_peaked():
    """A long sequence over many splits, with scores that grow along it (the
    maximum moves in every step) and a scale of its own."""
    say("attend long")
    g = gen(11)
    D, NKV, page, lens = 128, 1, 64, [5003]
    tab, n = paged(g, lens, page)
    T = lens[0]
    q = normal(g, 1, 4, D)
    k = normal(g, T, NKV, D) + (q[0, :1].float() * torch.linspace(0, 3, T)[:, None, None]).to(torch.bfloat16)
    v = normal(g, T, NKV, D)
    c = mm.KVCache4(n, page, NKV, D)
    c.write(k.to(DEV), v.to(DEV), tab.to(DEV), i32([0]), i32([0, T]))
    out, lse = c.attend(q.to(DEV), tab.to(DEV), i32(lens), scale=0.7, return_lse=True)
    val = lambda x: oa.values(*oa.quantise(f64(x)))  # noqa: E731
    check_attend(out, lse, q, val(k), val(v), lens, 0.7, D)


def test_attend_bad_pages_and_lengths():
    """Page ids outside the cache hold no tokens; lengths are brought into
    the table; strided queries and a strided output, whose other columns
    stay."""
    say("attend bad pages")
    g = gen(12)
    D, NHq, NKV, page = 128, 4, 2, 16
    lens = [40, 48, 48, 20]
    tab, n = paged(g, lens, page)
    c, k, v = filled(g, tab, n, lens, page, NKV, D)
    bad = tab.clone()
    bad[0, 1], bad[1, :], bad[2, 2] = n, -1, 2 ** 31 - 1
    told = [40, 10 ** 9, 2 ** 31 - 1, -5]
    at = cu(lens)
    rows = [np.r_[0:16, 32:40], [], np.r_[0:32], []]
    keep = np.concatenate([at[b] + np.asarray(r, int) for b, r in enumerate(rows)])
    big = normal(g, 4, 2 * NHq * D).to(DEV)
    q = big[:, NHq * D:].view(4, NHq, D)
    res = torch.full((4, 2 * NHq * D), 7.0, dtype=torch.bfloat16, device=DEV)
    out = res[:, :NHq * D].view(4, NHq, D)
    o, lse = c.attend(q, bad.to(DEV), i32(told), out=out, return_lse=True)
    assert o is out and (res[:, NHq * D:] == 7.0).all()
    check_attend(out, lse, q.cpu(), k[keep], v[keep], [len(r) for r in rows], D ** -0.5, D)


def test_attend_non_finite():
    """A NaN key reaches the heads of its kv head only, a NaN query its own
    head only, a NaN value the features of its group only."""
    say("attend non-finite")
    g = gen(13)
    D, NHq, NKV, page, lens = 128, 4, 2, 16, [70, 33]
    tab, n = paged(g, lens, page)
    T = sum(lens)
    k, v, q = normal(g, T, NKV, D), normal(g, T, NKV, D), normal(g, 2, NHq, D)
    c = mm.KVCache4(n, page, NKV, D)
    args = (tab.to(DEV), i32([0, 0]), i32(cu(lens)))
    c.write(k.to(DEV), v.to(DEV), *args)
    base = c.attend(q.to(DEV), tab.to(DEV), i32(lens))
    k2, v2, q2 = k.clone(), v.clone(), q.clone()
    k2[5, 0, 9] = float("nan")              # sequence 0, heads 0 and 1
    v2[80, 1, 40] = float("inf")            # sequence 1, heads 2 and 3, features 32..63
    q2[1, 0, 0] = float("nan")
    c.write(k2.to(DEV), v2.to(DEV), *args)
    out, lse = c.attend(q2.to(DEV), tab.to(DEV), i32(lens), return_lse=True)
    nan = torch.zeros(2, NHq, D, dtype=torch.bool)
    nan[0, :2] = nan[1, 0] = True
    nan[1, 2:, 32:64] = True
    assert torch.equal(torch.isnan(out).cpu(), nan)
    assert torch.equal(out.cpu()[~nan], base.cpu()[~nan])
    assert torch.isnan(lse.cpu()[nan[..., 0]]).all() and torch.isfinite(lse.cpu()[1, 1:]).all()


# ------------------------------------------------------------------ prompts

def check_prompt(out, lse, q, k, v, nq, nk, causal, scale, rows=None):
    NHq, NKV, D = q.shape[1], k.shape[1], q.shape[2]
    cq, ck = cu(nq), cu(nk)
    for b in range(len(nq)):
        i = np.arange(nq[b])
        if rows is not None and nq[b] > 2 * rows:
            i = np.r_[0:rows, nq[b] - rows:nq[b]]
        if len(i) == 0:
            continue
        sees = i + 1 + nk[b] - nq[b] if causal else np.full(len(i), nk[b])
        ks = slice(ck[b], ck[b] + nk[b])
        for h in range(NHq):
            kh = h // (NHq // NKV)
            o, z, spread, reach = oa.attend(f64(q[cq[b] + i, h]), f64(k[ks, kh]), f64(v[ks, kh]), scale, sees)
            e = ((D + 8) * U * reach)[:, None]
            close(f64(out[cq[b] + i, h]), o, (H + 2 * e + 64 * U) * spread + H * np.abs(o), f"out {b} {h}")
            zb = np.where(np.isfinite(z), z, 0.0)
            close(f64(lse[cq[b] + i, h]), z, e[:, 0] + 64 * U + 4 * U * np.abs(zb), f"lse {b} {h}")


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("D,NHq,NKV,nq,nk", [
    (64, 1, 1, [1], [1]), (128, 2, 1, [1, 2, 31, 32, 33], [1, 2, 31, 32, 33]),
    (128, 3, 3, [127, 128, 129, 0, 5], [127, 128, 129, 0, 5]), (64, 4, 2, [63, 64, 65, 200], [63, 64, 65, 200]),
    (192, 2, 1, [95, 130], [95, 130]), (256, 2, 2, [33, 257], [33, 257]),
    (128, 4, 2, [1, 5, 64, 3], [300, 64, 65, 0]), (64, 2, 1, [40, 200, 7], [20, 70, 7]),
    (192, 3, 1, [1, 70], [500, 90]), (256, 1, 1, [129], [200]),
])
def test_prompt(D, NHq, NKV, nq, nk, causal):
    """One token to several tiles, tile edges, empty sequences, keys behind
    cached prefixes (nk > nq), and more queries than keys (causal: the first
    rows see nothing)."""
    say("prompt", D, NHq, NKV, nq, nk, causal)
    g = gen(D + NHq + sum(nq))
    q = normal(g, sum(nq), NHq, D)
    k, v = normal(g, sum(nk), NKV, D), normal(g, sum(nk), NKV, D)
    out, lse = mm.prompt_attention(q.to(DEV), k.to(DEV), v.to(DEV), i32(cu(nq)), i32(cu(nk)),
                                   causal=causal, return_lse=True)
    check_prompt(out, lse, q, k, v, nq, nk, causal, D ** -0.5)


@pytest.mark.parametrize("D,NHq,NKV,nq,nk,causal", [
    (128, 8, 1, [1], [5000], True), (64, 7, 1, [40, 3], [1500, 2500], True), (256, 10, 2, [1, 30], [700, 33], True),
    (192, 6, 2, [2, 0, 60], [900, 50, 61], False), (128, 3, 1, [90], [2000], True), (64, 5, 5, [70, 2], [70, 1600], True),
    (128, 5, 1, [300], [260], True),
])
def test_prompt_groups_and_splits(D, NHq, NKV, nq, nk, causal):
    """Groups whose rows do not divide a tile, and few queries over many keys
    (the keys are split and joined, some sequences by one split alone)."""
    say("prompt groups", D, NHq, NKV, nq, nk, causal)
    g = gen(D + NHq + sum(nk))
    q = normal(g, sum(nq), NHq, D)
    k, v = normal(g, sum(nk), NKV, D), normal(g, sum(nk), NKV, D)
    out, lse = mm.prompt_attention(q.to(DEV), k.to(DEV), v.to(DEV), i32(cu(nq)), i32(cu(nk)),
                                   causal=causal, return_lse=True)
    check_prompt(out, lse, q, k, v, nq, nk, causal, D ** -0.5)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("D,NHq,NKV", [(64, 4, 2), (128, 2, 1), (128, 8, 1), (192, 4, 2), (256, 2, 2)])
def test_prompt_few_and_many_rows(D, NHq, NKV, causal):
    """Few rows and keys and many (of padding behind the last sequence) take
    workgroups of different sizes and tiles, and in some of them waves share a
    tile's keys: all are held to the oracle, and NaN and infinity, in masked and
    seen places, to theirs."""
    say("prompt rows", D, NHq, NKV, causal)
    g = gen(D + NHq)
    nq, nk = [300, 0, 33, 1, 129, 70], [300, 9, 500, 70, 129, 20]
    q = normal(g, sum(nq), NHq, D)
    k, v = normal(g, sum(nk), NKV, D), normal(g, sum(nk), NKV, D)
    clean = [t.clone() for t in (q, k, v)]
    v[299, 0, 5] = float("nan")                # seen by the first sequence's last query
    k[280, 0, 7] = float("inf")
    q[320, 0, 3] = float("nan")
    n = sum(nq)
    same = lambda a, b: bool(((a == b) | (a.isnan() & b.isnan())).all())  # noqa: E731
    for c, (x, y, z) in enumerate((clean, (q, k, v))):
        cus = i32(cu(nq)), i32(cu(nk))
        few, lse = mm.prompt_attention(x.to(DEV), y.to(DEV), z.to(DEV), *cus, causal=causal, return_lse=True)
        if c == 0:
            check_prompt(few, lse, x, y, z, nq, nk, causal, D ** -0.5)
        else:
            assert few[299, 0].isnan().any() and few[320, 0].isnan().all()
        pad = lambda t, rows: torch.cat([t, torch.full((rows, *t.shape[1:]), float("nan"), dtype=t.dtype)]).to(DEV)  # noqa: E731
        for rows, keys in ((20000, 0), (40000, 0), (40000, 9000), (80000, 0), (80000, 9000), (160000, 9000)):
            many, lse2 = mm.prompt_attention(pad(x, rows // NHq - n), pad(y, keys), pad(z, keys), *cus,
                                             causal=causal, return_lse=True)
            if c == 0:
                check_prompt(many[:n], lse2[:n], x, y, z, nq, nk, causal, D ** -0.5)
            assert same(few.isnan(), many[:n].isnan()) and same(lse.isnan(), lse2[:n].isnan())
            assert not many[n:].any() and torch.isneginf(lse2[n:]).all()


def test_prompt_splits_non_finite():
    """A value that is not finite in the last split's masked part, a NaN key
    that some rows see, and a query that is NaN throughout."""
    say("prompt splits non-finite")
    g = gen(29)
    D, NHq, NKV, nq, nk = 128, 4, 2, [6], [3000]
    q, k, v = normal(g, 6, NHq, D), normal(g, 3000, NKV, D), normal(g, 3000, NKV, D)
    v[2999, 0, 7] = float("nan")            # the last query alone sees it
    k[2998, 1, 0] = float("nan")            # the last two queries
    q[1, 0] = float("nan")
    out, lse = mm.prompt_attention(q.to(DEV), k.to(DEV), v.to(DEV), i32([0, 6]), i32([0, 3000]), return_lse=True)
    nan = torch.zeros(6, NHq, D, dtype=torch.bool)
    nan[5, :2, 7] = nan[4:, 2:] = nan[1, 0] = True
    assert torch.equal(torch.isnan(out).cpu(), nan)
    assert torch.isnan(lse[1, 0]) and torch.isnan(lse[4:, 2:]).all() and torch.isfinite(lse[0]).all()
    rows = [0, 2, 3]
    clean = lambda x: torch.nan_to_num(x, nan=0.0)  # noqa: E731
    for r in rows:
        check_prompt(out[r:r + 1], lse[r:r + 1], q[r:r + 1], clean(k)[:2995 + r], clean(v)[:2995 + r], [1], [2995 + r],
                     True, D ** -0.5)


def test_prompt_long():
    say("prompt long")
    g = gen(21)
    n, D = 2500, 128
    q, k, v = normal(g, n, 2, D), normal(g, n, 1, D), normal(g, n, 1, D)
    k = k + (torch.linspace(0, 2, n)[:, None, None] * q[:, :1].float()).to(torch.bfloat16)
    out, lse = mm.prompt_attention(q.to(DEV), k.to(DEV), v.to(DEV), i32([0, n]), scale=0.5, return_lse=True)
    check_prompt(out, lse, q, k, v, [n], [n], True, 0.5, rows=40)


def test_prompt_strides_and_tail():
    """Heads of a fused projection, packed with padding behind the last
    sequence: the padding's NaN reaches nothing, a given output keeps its
    rows there, a new one has zeros."""
    say("prompt strides")
    g = gen(22)
    NHq, NKV, D, nq = 4, 2, 128, [70, 1, 150]
    T, pad = sum(nq), 200
    qkv = normal(g, T + pad, (NHq + 2 * NKV) * D)
    qkv[T:] = float("nan")
    dev = qkv.to(DEV)
    parts = lambda x: (x[:, :NHq * D].view(-1, NHq, D), x[:, NHq * D:(NHq + NKV) * D].view(-1, NKV, D),  # noqa: E731
                       x[:, (NHq + NKV) * D:].view(-1, NKV, D))
    out, lse = mm.prompt_attention(*parts(dev), i32(cu(nq)), return_lse=True)
    check_prompt(out, lse, *parts(qkv), nq, nq, True, D ** -0.5)
    assert not out[T:].any() and (lse[T:] == -float("inf")).all()
    wide = torch.full((T + pad, 2 * NHq * D), 3.0, dtype=torch.bfloat16, device=DEV)
    given = wide[:, NHq * D:].view(T + pad, NHq, D)
    _, lse2 = mm.prompt_attention(*parts(dev), i32(cu(nq)), out=given, return_lse=True)
    assert torch.equal(given[:T], out[:T]) and torch.equal(lse2, lse)
    assert (wide[T:] == 3.0).all() and (wide[:, :NHq * D] == 3.0).all()


@pytest.mark.parametrize("T,first", [(300, 40), (300, 300), (30000, 500)])
def test_prompt_rows_before_the_first_sequence(T, first):
    """A batch whose first sequence starts behind row 0: the rows before it
    are like those behind the last one."""
    say("prompt rows before", T, first)
    g = gen(T + first)
    D, NHq, NKV, n = 64, 4, 2, min(70, T - first)
    q, k, v = (normal(g, T, h, D) for h in (NHq, NKV, NKV))
    at = i32([first, first + n])
    out, lse = mm.prompt_attention(q.to(DEV), k.to(DEV), v.to(DEV), at, return_lse=True)
    mine = slice(first, first + n)
    check_prompt(out[mine], lse[mine], q[mine], k[mine], v[mine], [n], [n], True, D ** -0.5)
    free = torch.ones(T, dtype=torch.bool, device=DEV)
    free[mine] = False
    assert not out[free].any() and torch.isneginf(lse[free]).all()
    given = torch.full_like(out, 3.0)
    mm.prompt_attention(q.to(DEV), k.to(DEV), v.to(DEV), at, out=given)
    assert torch.equal(given[mine], out[mine]) and (given[free] == 3.0).all()


@pytest.mark.parametrize("D", [64, 128, 192, 256])
@pytest.mark.parametrize("what", ["nan", "inf"])
def test_prompt_future_tokens_stay_out(D, what):
    """Keys and values that are not finite at some token: rows before it are
    what they are without them, rows from it on see them; other sequences are
    untouched bit for bit.  (Rows that share a tile with such a token are
    computed in another order, without the rounding of the probabilities, so
    they are held to the attention's bound, which counts that rounding.)"""
    say("prompt future", D, what)
    g = gen(23)
    NHq, NKV, nq = 4, 2, [150, 60]
    q, k, v = normal(g, 210, NHq, D), normal(g, 210, NKV, D), normal(g, 210, NKV, D)
    run = lambda k, v: mm.prompt_attention(q.to(DEV), k.to(DEV), v.to(DEV), i32(cu(nq)), return_lse=True)  # noqa: E731
    base, base_lse = run(k, v)
    cut = 77
    v2, k2 = v.clone(), k.clone()
    v2[cut, 0, 3] = float(what)
    k2[cut + 20, 1, 5] = float("nan")
    v2[cut + 20, 1, :] = float(what)
    out, lse = run(k2, v2)
    clean = lambda x: torch.where(torch.isfinite(x), x, torch.zeros_like(x))  # noqa: E731
    first = lambda x, n: x[:n]  # noqa: E731
    check_prompt(first(out, cut), first(lse, cut), *(first(x, cut) for x in (q, k, v)), [cut], [cut], True, D ** -0.5)
    check_prompt(out[:cut + 20, 2:], lse[:cut + 20, 2:], q[:cut + 20, 2:], clean(k2)[:cut + 20, 1:],
                 clean(v2)[:cut + 20, 1:], [cut + 20], [cut + 20], True, D ** -0.5)
    assert torch.equal(out[150:], base[150:]) and torch.equal(lse[150:], base_lse[150:])
    got = out[cut:150].float().cpu()
    assert not torch.isfinite(got[:, :2, 3]).any()
    assert torch.isfinite(got[:, :2, 4:]).all()
    assert torch.isnan(got[20:, 2:]).all()


def test_prompt_large_scores():
    """Scores far beyond the exponential's range: the maximum keeps every
    probability finite, and rows of one dominant key return its value.  The
    maximum is rounded to float32 (scores reach 2^20, half a step 2^-5), so
    the one probability left is p = 2^d, |d| <= 2^-5, not 1: the output is
    bf16(p) / p times the value, off by h for the rounding of p and h for its
    own."""
    say("prompt large scores")
    g = gen(24)
    n, D = 130, 128
    q = normal(g, n, 1, D, scale=60.0)
    k, v = q.clone(), normal(g, n, 1, D)
    out, lse = mm.prompt_attention(q.to(DEV), k.to(DEV), v.to(DEV), i32([0, n]), return_lse=True)
    close(f64(out), f64(v), (2 * H + H * H) * np.abs(f64(v)))
    assert torch.isfinite(lse).all()
    check_prompt(out, lse, q, k, v, [n], [n], True, D ** -0.5)


# ------------------------------------------------------------------ together, streams, graphs

def decode_step(c, layer, qkv, logits, pos, tab, cs, w, NHq, NKV, D):
    """One decode step around the cache and into the layer."""
    B = qkv.shape[0]
    q = qkv[:, :NHq * D].view(B, NHq, D)
    k = qkv[:, NHq * D:(NHq + NKV) * D].view(B, NKV, D)
    v = qkv[:, (NHq + NKV) * D:].view(B, NKV, D)
    qn, kn = mm.qk_norm_rope(q, k, pos.long(), cs, D, w, w)
    c.write(kn, v, tab, pos)
    a = c.attend(qn, tab, pos + 1)
    return a, layer(a.view(B, NHq * D), logits)


def test_a_prompt_then_decode_steps():
    """A prompt through its attention into the cache, then decode steps over
    what was written, into the layer: each attention against the oracle on
    the values that the cache holds, and the layer on its output."""
    say("chain")
    g = gen(31)
    NHq, NKV, D, page, nq = 4, 2, 64, 16, [20, 1, 37]
    B, R = 3, 64
    cfg = workloads.CONFIGS["tiny"]
    tab, n = paged(g, [60] * B, page)
    w = (1 + 0.1 * torch.randn(D, generator=g)).to(torch.bfloat16)
    cs = table(300, R)
    qkv = normal(g, sum(nq), (NHq + 2 * NKV) * D)
    dev = qkv.to(DEV)
    pos = torch.cat([torch.arange(x) for x in nq])
    parts = lambda x: (x[:, :NHq * D].view(-1, NHq, D), x[:, NHq * D:(NHq + NKV) * D].view(-1, NKV, D),  # noqa: E731
                       x[:, (NHq + NKV) * D:].view(-1, NKV, D))
    q, k, v = parts(dev)
    qn, kn = mm.qk_norm_rope(q, k, pos.to(DEV), cs.to(DEV), R, w.to(DEV), w.to(DEV))
    out, lse = mm.prompt_attention(qn, kn, v, i32(cu(nq)), return_lse=True)
    check_prompt(out, lse, qn.cpu(), kn.cpu(), v.cpu(), nq, nq, True, D ** -0.5)
    c = mm.KVCache4(n, page, NKV, D)
    td = tab.to(DEV)
    c.write(kn, v, td, i32([0] * B), i32(cu(nq)))
    H = NHq * D
    w13 = (torch.randn(cfg.E, 2 * cfg.I, H, generator=g) / H ** 0.5).to(torch.bfloat16).to(DEV)
    w2 = (torch.randn(cfg.E, H, cfg.I, generator=g) / cfg.I ** 0.5).to(torch.bfloat16).to(DEV)
    layer = mm.FusedMoE(w13, w2, cfg.K)
    lens = list(nq)
    for step in range(3):
        new = normal(g, B, (NHq + 2 * NKV) * D).to(DEV)
        logits = torch.randn(B, cfg.E, generator=g).to(DEV)
        a, y = decode_step(c, layer, new, logits, i32(lens), td, cs.to(DEV), w.to(DEV), NHq, NKV, D)
        lens = [x + 1 for x in lens]
        kc, vc = c.read(td, i32([0] * B), i32(cu(lens)), sum(lens))
        qn, _ = mm.qk_norm_rope(parts(new)[0], None, i32(lens).long() - 1, cs.to(DEV), R, w.to(DEV))
        a2, lse = c.attend(qn, td, i32(lens), return_lse=True)
        assert torch.equal(a, a2)
        check_attend(a, lse, qn.cpu(), f64(kc), f64(vc), lens, D ** -0.5, D)
        # the same keys and values in bfloat16 through the prompt's path
        o2, _ = mm.prompt_attention(qn, kc, vc, i32(list(range(B + 1))), i32(cu(lens)), return_lse=True)
        close(f64(o2), f64(a), 4 * H * (np.abs(f64(a)) + 1))
        assert torch.equal(y, mm.fused_forward(a.view(B, H), logits, w13, w2, cfg.K))


def test_prefix_and_chunk_join_by_lse():
    """A chunk's own causal attention joined with its attention to a cached
    prefix by their lse equals the attention over both."""
    say("lse join")
    g = gen(32)
    D, NH, n = 128, 2, 50
    q, k, v = (normal(g, n, NH, D).to(DEV) for _ in range(3))
    cut = 30
    whole, z = mm.prompt_attention(q, k, v, i32([0, n]), return_lse=True)
    a, za = mm.prompt_attention(q[cut:], k[cut:], v[cut:], i32([0, n - cut]), return_lse=True)
    b, zb = mm.prompt_attention(q[cut:], k[:cut], v[:cut], i32([0, n - cut]), i32([0, cut]), causal=False, return_lse=True)
    zz = torch.logaddexp(za, zb)
    joined = a.float() * (za - zz).exp()[..., None] + b.float() * (zb - zz).exp()[..., None]
    # z: two sums' errors; out: three outputs of (2 h) each, joined by factors that sum to 1
    assert (zz - z[cut:]).abs().max() < 1e-4
    assert (joined - whole[cut:].float()).abs().max() <= 6 * H * v.float().abs().max()


def test_other_stream_and_determinism():
    """Calls on a stream of their own give the same bits as on the current
    one, again and again."""
    say("streams")
    g = gen(33)
    D, NHq, NKV, page, lens = 128, 8, 2, 32, [700, 90, 3000]
    tab, n = paged(g, lens, page)
    c, _, _ = filled(g, tab, n, lens, page, NKV, D)
    q = normal(g, 3, NHq, D).to(DEV)
    td, ld = tab.to(DEV), i32(lens)
    p = normal(g, 300, NHq, D).to(DEV)
    kv = normal(g, 300, NKV, D).to(DEV)
    base, pbase = c.attend(q, td, ld), mm.prompt_attention(p, kv, kv, i32([0, 100, 300]))
    cus = i32([0, 100, 300])
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    for _ in range(3):
        a = c.attend(q, td, ld, stream=st)
        b = mm.prompt_attention(p, kv, kv, cus, stream=st)
        x = c.attend(q, td, ld)
        st.synchronize()
        assert torch.equal(a, base) and torch.equal(b, pbase) and torch.equal(x, base)


def test_graph_replays_follow_lengths():
    """A captured decode step replays with new lengths, pages and inputs, and
    matches the eager step; two captured graphs do not share scratch."""
    say("graphs")
    g = gen(34)
    D, NHq, NKV, page, B = 64, 8, 2, 16, 4
    cfg = workloads.CONFIGS["tiny"]
    H = NHq * D
    w13 = (torch.randn(cfg.E, 2 * cfg.I, H, generator=g) / H ** 0.5).to(torch.bfloat16).to(DEV)
    w2 = (torch.randn(cfg.E, H, cfg.I, generator=g) / cfg.I ** 0.5).to(torch.bfloat16).to(DEV)
    layer = mm.FusedMoE(w13, w2, cfg.K)
    lens = [300, 17, 0, 64]
    tab, n = paged(g, [600] * B, page)
    td = tab.to(DEV)
    c, _, _ = filled(g, tab, n, lens, page, NKV, D)
    cs, w = table(2000, D).to(DEV), normal(g, D).to(DEV)
    qkv, logits, pos = normal(g, B, (NHq + 2 * NKV) * D).to(DEV), torch.randn(B, cfg.E, generator=g).to(DEV), i32(lens)
    step = lambda: decode_step(c, layer, qkv, logits, pos, td, cs, w, NHq, NKV, D)  # noqa: E731
    step()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs = step()
        graphs.append((gr, outs))
    for r in range(4):
        qkv.copy_(normal(g, *qkv.shape))
        pos.copy_(torch.tensor([x + r for x in lens], dtype=torch.int32) if r != 2 else i32([-1, 17, 5, 599]))
        torch.cuda.synchronize()
        for gr, _ in graphs:
            gr.replay()
        torch.cuda.synchronize()
        a, y = step()
        torch.cuda.synchronize()
        # places between the written tokens hold noise that reads as NaN; the
        # layer's outputs are defined for the other rows (in the last round every
        # sequence has such a place: the round before left one out)
        rows = torch.isfinite(a).flatten(1).all(1)
        assert rows.sum() == (4, 4, 2, 0)[r]
        for _, (ga, gy) in graphs:
            assert np.array_equal(f64(ga), f64(a), equal_nan=True) and torch.equal(gy[rows], y[rows]), r
        if r == 2:
            assert not a[0].any()


def test_binding_refusals():
    """Wrong types, shapes, strides, overlaps and streams raise before
    anything is launched."""
    say("refusals")
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16, device=DEV)
    pos = torch.zeros(4, dtype=torch.int64, device=DEV)
    cs = torch.zeros(8, 64, device=DEV)
    x2, wide = torch.zeros_like(x), torch.zeros(4, 256, dtype=torch.bfloat16, device=DEV)
    c = mm.KVCache4(3, 16, 2, 64)
    tab, one = torch.zeros(4, 1, dtype=torch.int32, device=DEV), i32([0, 0, 0, 0])
    wrong = [
        lambda: mm.qk_norm_rope(x.float(), x, pos, cs, 64),
        lambda: mm.qk_norm_rope(x, x[:3], pos, cs, 64),
        lambda: mm.qk_norm_rope(x, x, pos[:3], cs, 64),
        lambda: mm.qk_norm_rope(x, x, pos.int(), cs, 64),
        lambda: mm.qk_norm_rope(x, x, pos, cs, 32),
        lambda: mm.qk_norm_rope(x, x, pos, cs, 64, torch.ones(32, device=DEV)),
        lambda: mm.qk_norm_rope(x, x, pos, cs, 64, torch.ones(64, device=DEV), torch.ones(64, device=DEV).bfloat16()),
        lambda: mm.qk_norm_rope(x, None, pos, cs, 64, None, torch.ones(64, device=DEV)),
        lambda: mm.qk_norm_rope(x.transpose(1, 2), None, pos, cs, 64),
        lambda: mm.qk_norm_rope(x[1:], None, pos[1:], cs, 64, q_out=x[:3]),
        lambda: mm.qk_norm_rope(x, x2, pos, cs, 64, q_out=x2),
        lambda: mm.qk_norm_rope(x, x2, pos, cs, 64, k_out=x),
        lambda: c.read(tab, one, None, 4, k=x, v=x),
        lambda: c.read(tab, one, None, 4, k=wide[:, :128].view(4, 2, 64), v=wide[:, 64:192].view(4, 2, 64)),
        lambda: c.write(x, x[:3], tab, one),
        lambda: c.write(x[:3], x[:3], tab, one),
        lambda: c.write(x, x, tab.long(), one),
        lambda: c.write(x, x, tab[:3], one),
        lambda: c.write(x, x, tab, one.long()),
        lambda: c.read(tab, one, None, 5),
        lambda: c.read(tab, one, None, 4, k=x),
        lambda: c.attend(x, tab, one[:3]),
        lambda: c.attend(x[:, :1], tab, one),
        lambda: c.attend(x, tab, one, scale=0.0),
        lambda: c.attend(x, tab, one, out=x),
        lambda: mm.prompt_attention(x, x, x, i32([0, 4]), out=x),
        lambda: mm.prompt_attention(x, x[:3], x[:3], i32([0, 4])),
        lambda: mm.prompt_attention(x, x, x, i32([0, 4]), i32([0, 2, 4])),
        lambda: mm.prompt_attention(x, x, x, i32([0, 4]).long()),
        lambda: mm.prompt_attention(x[:, :1], x, x, i32([0, 4])),
        lambda: mm.prompt_attention(x, x, x, i32([0, 4]), scale=-1.0),
        lambda: mm.KVCache4.of(torch.zeros(2, 2, 1, 100, dtype=torch.uint8, device=DEV)),
    ]
    for i, f in enumerate(wrong):
        with pytest.raises((TypeError, ValueError, mm.MoEError)):
            f()
            print("not refused:", i)
    torch.cuda.synchronize()


def test_empty_calls():
    say("empty")
    x = torch.zeros(0, 2, 64, dtype=torch.bfloat16, device=DEV)
    a, b = mm.qk_norm_rope(x, x, torch.zeros(0, dtype=torch.int64, device=DEV), torch.zeros(8, 64, device=DEV), 64)
    assert a.shape == b.shape == (0, 2, 64)
    c = mm.KVCache4(3, 16, 2, 64)
    e = torch.zeros(0, dtype=torch.int32, device=DEV)
    tab = torch.zeros(0, 2, dtype=torch.int32, device=DEV)
    c.write(x, x, tab, e)
    k, v = c.read(tab, e, i32([0]), 3)
    assert k.shape == (3, 2, 64) and not k.any() and not v.any()
    assert c.attend(x, tab, e).shape == (0, 2, 64)
    y = torch.ones(5, 2, 64, dtype=torch.bfloat16, device=DEV)
    out, lse = mm.prompt_attention(y, y, y, i32([0]), return_lse=True)
    assert not out.any() and (lse == -float("inf")).all()
    out = mm.prompt_attention(y, x, x, i32([0, 5]), i32([0, 0]))
    assert not out.any()
    # a table without columns: no tokens
    o = c.attend(y, torch.zeros(5, 0, dtype=torch.int32, device=DEV), i32([3] * 5))
    assert not o.any()
