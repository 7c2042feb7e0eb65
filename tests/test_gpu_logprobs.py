"""zo_logprobs against log-softmax in 64 bits; the alternatives exactly.

Tolerances: a sum of n nonnegative fp32 terms, each within 2^-21 (exponential and its argument),
taken by 128 or more threads one after another and joined in at most 16 steps, is within
E = (n / 128 / 4 + 4 + 16) 2^-24 4 + 2^-21 relative when four partial chains are not assumed: the
bound used is E = (n / 128 + 24) 2^-24 + 2^-21.  With c the fp32 log2 e (2^-26 off),
|logprob - ref| <= E + 2^-25 (max - x_t) + 2^-24 |ref|, and the entropy's two sums give
|H - ref| <= E (1 + 2 sum_j p_j (max - x_j)) + 2^-24 |ref|.
"""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def ctx(zo):
    c = zo.zo_create(torch.zeros(64, dtype=torch.bfloat16, device="cuda"))
    yield c
    c.close()


def buffers(rows, top):
    return (torch.full((rows,), 9.0, device="cuda"), torch.full((rows,), 9.0, device="cuda"),
            torch.full((rows, top), -9, dtype=torch.int32, device="cuda"), torch.full((rows, top), 9.0, device="cuda"))


def call(zo, ctx, x, targets, top, vocab=None, rows=None):
    rows = x.shape[0] if rows is None else rows
    vocab = x.shape[1] if vocab is None else vocab
    lp, ent, ids, tlp = buffers(rows, top)
    zo.zo_logprobs(ctx, x, rows, vocab, x.stride(0), targets, lp, ent, top, ids, tlp)
    return lp, ent, ids, tlp


def order(x):
    """Indices by value, largest first (NaN before all), equal ones by index."""
    key = x.double()
    key = torch.where(torch.isnan(key), torch.full_like(key, math.inf), key)
    nan_first = torch.isnan(x).to(torch.int32)
    idx = torch.sort(key, dim=1, descending=True, stable=True).indices
    return idx.gather(1, torch.sort(nan_first.gather(1, idx), dim=1, descending=True, stable=True).indices)


def check(x, targets, got, top):
    lp, ent, ids, tlp = got
    x = x.double()
    n = x.shape[1]
    big = x.amax(1, keepdim=True)
    ref = torch.log_softmax(x, 1)
    p = ref.exp()
    spread = torch.where(p > 0, big - x, torch.zeros_like(x))
    E = (n / 128 + 24) * 2.0 ** -24 + 2.0 ** -21
    t = targets.long()
    want = torch.where(t >= 0, ref.gather(1, t.clamp(min=0)[:, None])[:, 0], torch.zeros_like(ref[:, 0]))
    gap = (big[:, 0] - x.gather(1, t.clamp(min=0)[:, None])[:, 0])
    gap = torch.where(torch.isfinite(gap), gap, torch.zeros_like(gap))
    tol = E + 2.0 ** -25 * gap + 2.0 ** -24 * want.abs()
    same = (lp.double() == want) | ((lp.double() - want).abs() <= tol)
    assert torch.all(same), (lp.double() - want).abs().max()
    H = -(p * torch.where(p > 0, ref, torch.zeros_like(ref))).sum(1)
    tol = E * (1 + 2 * (p * spread).sum(1)) + 2.0 ** -24 * H.abs()
    assert torch.all((ent.double() - H).abs() <= tol), (ent.double() - H).abs().max()
    if top:
        idx = order(x)[:, :top]
        assert torch.equal(ids.long(), idx)
        want = ref.gather(1, idx)
        gap = torch.where(torch.isfinite(want), big - x.gather(1, idx), torch.zeros_like(want))
        same = (tlp.double() == want) | ((tlp.double() - want).abs() <= E + 2.0 ** -25 * gap + 2.0 ** -24 * want.abs())
        assert torch.all(same)


def logits(rows, vocab, dtype, seed=0, scale=3.0):
    g = torch.Generator(device="cuda").manual_seed(seed + rows + vocab)
    x = torch.randn(rows, vocab, generator=g, device="cuda") * scale
    t = torch.randint(0, vocab, (rows,), generator=g, device="cuda", dtype=torch.int32)
    return x.to(TYPES[dtype]), t


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,vocab", [(1, 1), (3, 2), (5, 7), (4, 31), (2, 33), (9, 256), (3, 1000), (2, 4095),
                                        (2, 8191), (2, 8192), (3, 32001), (1, 50272), (5, 151936), (300, 777),
                                        (1000, 8200)])
def test_logprobs_match(zo, ctx, dtype, rows, vocab):
    x, t = logits(rows, vocab, dtype)
    for top in sorted({0, 1, min(5, vocab), min(32, vocab)}):
        check(x, t, call(zo, ctx, x, t, top), top)
    assert zo.zo_sync(ctx) == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("pad,shift", [(1, 0), (3, 1), (8, 0), (13, 5)])
def test_strides_and_alignments(zo, ctx, dtype, pad, shift):
    """Rows that start anywhere; what lies between them is not read as logits (NaN there)."""
    for vocab in (6, 100, 9001):
        x, t = logits(7, vocab, dtype)
        wide = torch.full((7 * (vocab + pad) + shift,), math.nan, device="cuda").to(TYPES[dtype])
        view = wide[shift:].view(7, vocab + pad)
        view[:, :vocab] = x
        check(x, t, call(zo, ctx, view, t, min(6, vocab), vocab=vocab), min(6, vocab))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_ties_go_to_the_lowest_index(zo, ctx, dtype):
    n = 20000
    g = torch.Generator(device="cuda").manual_seed(1)
    rows = [torch.zeros(n, device="cuda"),                                     # all equal
            torch.randint(0, 3, (n,), generator=g, device="cuda").float(),     # three values
            torch.where(torch.arange(n, device="cuda") % 1000 == 999, 5.0, 1.0),
            torch.where(torch.arange(n, device="cuda") % 2 == 0, -0.0, 0.0),   # -0 equals +0
            torch.arange(n, device="cuda").float().div(100).floor(),           # runs, growing
            -torch.arange(n, device="cuda").float().div(4000).floor(),         # runs, falling
            torch.where(torch.arange(n, device="cuda") < 9, 2.0, -1.0)]
    x = torch.stack(rows).to(TYPES[dtype])
    t = torch.zeros(len(rows), dtype=torch.int32, device="cuda")
    for top in (1, 8, 32):
        check(x, t, call(zo, ctx, x, t, top), top)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_largest_logits_crowded_into_few_places(zo, ctx, dtype):
    """Thousands of logits above any bound that the threads' own largest ones give."""
    n, step = 60000, {"f32": 4, "bf16": 8}[dtype]
    base = torch.zeros(n, device="cuda")
    at = torch.arange(n, device="cuda")
    crowd = (at // step) % 512 < 24          # 24 of 512 vectors in a row: the same 24 threads' ones
    x = torch.stack([torch.where(crowd, 10.0 + (at % 97).float() / 64, base),
                     torch.where(crowd, 10.0, base - (at % 7).float()),
                     torch.where((at // step) % 512 < 40, 8.0, base)]).to(TYPES[dtype])
    t = torch.tensor([0, 5, n - 1], dtype=torch.int32, device="cuda")
    for top in (20, 32):
        check(x, t, call(zo, ctx, x, t, top), top)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,rows", [(20000, 200), (3000, 160), (700, 30), (700, 4100), (3000, 4003), (9000, 900)])
def test_ties_masks_and_bad_rows_where_a_block_has_a_row_of_its_own(zo, ctx, dtype, n, rows):
    """The same kinds of rows with enough of them that none is split, and with rows of one warp."""
    g = torch.Generator(device="cuda").manual_seed(n)
    at = torch.arange(n, device="cuda")
    low = torch.finfo(TYPES[dtype]).min
    kinds = [torch.zeros(n, device="cuda"), torch.randint(0, 3, (n,), generator=g, device="cuda").float(),
             at.float().div(100).floor(), -at.float().div(n // 5).floor(), torch.where(at == n - 1, 0.0, -math.inf),
             torch.where(at % 97 == 5, at.float() / n, torch.full((n,), -math.inf, device="cuda")),
             torch.full((n,), low, device="cuda"), torch.where((at // 8) % 128 < 9, 10.0 + (at % 7).float(), 0.0)]
    x = torch.stack([kinds[i % len(kinds)] for i in range(rows)]).to(TYPES[dtype])
    t = torch.full((rows,), n - 1, dtype=torch.int32, device="cuda")
    for top in (5, 20, 32):
        check(x, t, call(zo, ctx, x, t, top), top)
    x[3, n // 2] = math.nan
    x[11, 0] = math.inf
    x[rows - 1] = -math.inf
    lp, ent, ids, tlp = call(zo, ctx, x, t, 2)
    bad = [3, 11, rows - 1]
    assert torch.isnan(lp[bad]).all() and torch.isnan(ent[bad]).all() and torch.isnan(tlp[bad]).all()
    assert ids[3, 0] == n // 2 and ids[11, 0] == 0 and ids[rows - 1].tolist() == [0, 1]
    keep = [i for i in range(rows) if i not in bad]
    check(x[keep], t[keep], (lp[keep], ent[keep], ids[keep], tlp[keep]), 2)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,vocab", [(2, 60000), (200, 20000), (900, 9000), (4000, 3000)])
def test_sorted_rows(zo, ctx, dtype, rows, vocab):
    """Rising and falling logits: far more than the alternatives lie within 1 % of the largest."""
    up = torch.arange(vocab, device="cuda").float() / 64
    x = torch.stack([up if i % 2 else 1000.0 - up for i in range(rows)]).to(TYPES[dtype])
    t = torch.arange(rows, dtype=torch.int32, device="cuda") % vocab
    for top in (1, 32):
        check(x, t, call(zo, ctx, x, t, top), top)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,vocab", [(1, 4099), (3, 9000), (40, 8300), (148, 5000), (149, 5000)])
@pytest.mark.parametrize("shift", [0, 3])
def test_rows_split_over_blocks(zo, ctx, dtype, rows, vocab, shift):
    """A row's largest logits, masks and target in each of its parts."""
    x, t = logits(rows, vocab + 16, dtype, seed=shift)
    x = x[:, shift: shift + vocab]
    at = torch.linspace(0, vocab - 1, 9, device="cuda").long()
    x[:, at[:-1]] += torch.randperm(8, device="cuda").to(x.dtype) + 9
    x[0, vocab // 3: vocab // 2] = -math.inf
    t = at[torch.arange(rows, device="cuda") % 9].to(torch.int32)
    lp, ent, ids, tlp = buffers(rows, 7)
    zo.zo_logprobs(ctx, x, rows, vocab, x.stride(0), t, lp, ent, 7, ids, tlp)
    check(x, t, (lp, ent, ids, tlp), 7)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_masked_rows(zo, ctx, dtype):
    """-inf and the type's lowest value as masks; one token left; rows that only masks fill."""
    n, low = 9000, torch.finfo(TYPES[dtype]).min
    x, t = logits(8, n, dtype)
    x[0, 1:] = -math.inf                       # one token left, the first
    x[1, :-1] = -math.inf                      # the last
    x[2, ::2] = -math.inf
    x[3, 100:] = low
    x[4, :] = low                              # only lowest values: uniform
    x[5, :] = low
    x[5, 7] = low / 2                          # all but one weight vanish
    x[6, :20] = -math.inf
    t[0], t[1], t[2], t[3], t[4], t[5], t[6] = 0, n - 1, 4, 3, 17, 7, 3
    check(x, t, call(zo, ctx, x, t, 32), 32)
    t2 = t.clone()
    t2[0], t2[3] = 5, 5000                     # given tokens that are masked
    check(x, t2, call(zo, ctx, x, t2, 3), 3)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rows_without_a_distribution_are_nan(zo, ctx, dtype):
    n = 9000
    x, t = logits(6, n, dtype)
    x[0] = -math.inf
    x[1, 77] = math.nan
    x[2, 8999] = math.inf
    x[3, :] = math.nan
    x[4, 5] = -math.nan
    x[4, 3] = math.inf
    lp, ent, ids, tlp = call(zo, ctx, x, t, 4)
    assert torch.isnan(lp[:5]).all() and torch.isnan(ent[:5]).all() and torch.isnan(tlp[:5]).all()
    check(x[5:], t[5:], (lp[5:], ent[5:], ids[5:], tlp[5:]), 4)
    assert ids[0].tolist() == [0, 1, 2, 3] and ids[3].tolist() == [0, 1, 2, 3]
    assert ids[1, 0] == 77 and ids[2, 0] == 8999 and ids[4, :2].tolist() == [5, 3]
    assert torch.equal(ids[1, 1:].long(), order(x[1:2])[0, 1:4])


def test_huge_values_of_both_signs(zo, ctx):
    """Largest logits beyond +-1e30: differences count, nothing overflows."""
    n = 8300
    x = torch.zeros(5, n, device="cuda")
    x[0] = 3.0e38
    x[1] = -3.0e38
    x[1, 9] = -2.9e38
    x[2, 4] = 3.0e38
    x[3] = 2.0e30
    x[4] = -2.0e30
    t = torch.tensor([3, 9, 4, 1, 8299], dtype=torch.int32, device="cuda")
    check(x, t, call(zo, ctx, x, t, 5), 5)


def test_targets_outside_and_not_scored(zo, ctx):
    x, _ = logits(6, 500, "f32")
    t = torch.tensor([-1, 500, -2, 2 ** 31 - 1, -2 ** 31, 499], dtype=torch.int32, device="cuda")
    lp, ent, _, _ = call(zo, ctx, x, t, 0)
    assert lp[0] == 0 and torch.isnan(lp[1:5]).all()
    check(x[5:], t[5:], (lp[5:], ent[5:], None, None), 0)
    assert torch.isfinite(ent).all()


def test_some_outputs_only(zo, ctx):
    x, t = logits(4, 3000, "bf16")
    lp, ent, ids, tlp = call(zo, ctx, x, t, 7)
    a, b, i, v = buffers(4, 7)
    zo.zo_logprobs(ctx, x, 4, 3000, 3000, t, a, None, 0)
    zo.zo_logprobs(ctx, x, 4, 3000, 3000, None, None, b)
    zo.zo_logprobs(ctx, x, 4, 3000, 3000, None, None, None, 7, i, None)
    zo.zo_logprobs(ctx, x, 4, 3000, 3000, None, None, None, 7, None, v)
    assert torch.equal(a, lp) and torch.equal(b, ent) and torch.equal(i, ids) and torch.equal(v, tlp)


def test_replayed_and_repeatable(zo):
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        c = zo.zo_create(torch.zeros(64, device="cuda"), stream=s)
        x, t = logits(3, 60000, "f32")
        outs = buffers(3, 5)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        zo.zo_logprobs(c, x, 3, 60000, 60000, t, outs[0], outs[1], 5, outs[2], outs[3])
    for seed in range(2):
        with torch.cuda.stream(s):
            x.copy_(logits(3, 60000, "f32", seed=seed)[0])
            g.replay()
        s.synchronize()
        check(x, t, outs, 5)
        first = [o.clone() for o in outs]
        with torch.cuda.stream(s):
            g.replay()
        s.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, outs))
    del g
    c.close()


def test_offsets_beyond_32_bits(zo, ctx):
    """Rows whose first element lies past 2^31 elements."""
    rows, vocab = 2200, 1000000
    x = torch.zeros(rows, vocab, dtype=torch.bfloat16, device="cuda")
    pick = [0, 2146, 2147, 2148, 2199]
    for r in pick:
        x[r] = torch.randn(vocab, device="cuda").to(torch.bfloat16)
    t = torch.full((rows,), 999999, dtype=torch.int32, device="cuda")
    lp, ent, ids, tlp = call(zo, ctx, x, t, 3)
    check(x[pick], t[pick], (lp[pick], ent[pick], ids[pick], tlp[pick]), 3)


def test_logprobs_refusals(zo, ctx):
    x, t = logits(4, 100, "f32")
    lp, ent, ids, tlp = buffers(4, 5)
    base = dict(x=x, rows=4, vocab=100, ld=100, t=t, lp=lp, ent=ent, top=5, ids=ids, tlp=tlp, dtype=0)

    def refused(**k):
        a = dict(base, **k)
        with pytest.raises(zo.ZoError) as e:
            zo.zo_logprobs(ctx, a["x"], a["rows"], a["vocab"], a["ld"], a["t"], a["lp"], a["ent"], a["top"],
                           a["ids"], a["tlp"], a["dtype"])
        assert e.value.status == zo.ZO_ERR_INVALID

    refused(x=0)
    refused(vocab=2 ** 31 - 16, ld=2 ** 31 - 1)
    refused(t=None)
    refused(dtype=5)
    refused(rows=0)
    refused(rows=1 << 31)
    refused(vocab=0)
    refused(vocab=101)
    refused(ld=1 << 31)
    refused(top=-1)
    refused(top=33)
    refused(vocab=4, ld=100)               # top above the vocabulary
    refused(lp=None, ent=None, ids=None, tlp=None)
    refused(lp=None, ent=None, top=0)
    refused(x=x.data_ptr() + 2)
    refused(ids=ids.data_ptr() + 1)
    torch.cuda.synchronize()
    assert torch.all(lp == 9.0) and torch.all(ids == -9)


@pytest.mark.parametrize("rows,vocab,dtype", [(1, 1 << 28, "bf16"), (1, (1 << 27) + 5, "f32"), (150, 1 << 22, "f32"),
                                              (900, 1 << 20, "bf16"), (4000, 9001, "bf16")])
def test_sums_over_very_many_equal_terms(zo, ctx, rows, vocab, dtype):
    """Every 997th logit is 1, the others 0: nearly every vector of a thread adds the same, and the
    roundings of a long fp32 sum would add up, to some 1e-4.  Joined in fp64, what is left are the sums of
    at most 64 batches of vectors (2^-24 each, and in a batch some 10 steps) in s and u, whose errors enter
    the entropy as they are, two exponentials (2^-22 each) and the output's rounding."""
    x = torch.zeros(rows, vocab, dtype=TYPES[dtype], device="cuda")
    x[:, ::997] = 1.0
    t = torch.full((rows,), 5, dtype=torch.int32, device="cuda")
    lp, ent, _, _ = call(zo, ctx, x, t, 0)
    ones = (vocab + 996) // 997
    z = ones * math.e + (vocab - ones)
    H = math.log(z) - ones * math.e / z
    assert torch.all((lp.double() + math.log(z)).abs() <= 10 * 2.0 ** -24 + 2.0 ** -22 + 2.0 ** -24 * math.log(z))
    assert torch.all((ent.double() - H).abs() <= 84 * 2.0 ** -24 + 2.0 ** -21 + 2.0 ** -24 * H)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,vocab", [(1, 151936), (3, 50272), (300, 50272), (1000, 20000), (4100, 5000)])
def test_statistics_are_joined_in_64_bits(zo, ctx, dtype, rows, vocab):
    """Tighter than the bound above, which takes fp32 sums along a thread: a sum is off by its terms
    (exponential 2^-22, argument two roundings of 2^-24) and the fp32 chains of 4 vectors (s: 8 terms in
    each of four, and 2 joins) or of a sixteenth of a thread's rounds and those (u), at most 10 + 40."""
    x, t = logits(rows, vocab, dtype)
    lp, ent, _, tlp = call(zo, ctx, x, t, 4)
    for a in range(0, rows, 500):
        X, T = x[a: a + 500].double(), t[a: a + 500].long()
        ref = torch.log_softmax(X, 1)
        p = ref.exp()
        spread = (p * (X.amax(1, keepdim=True) - X)).sum(1)
        E = 2.0 ** -22 + 10 * 2.0 ** -24 + 2.0 ** -23 * spread
        want = ref.gather(1, T[:, None])[:, 0]
        assert torch.all((lp[a: a + 500].double() - want).abs() <= E + 2.0 ** -24 * want.abs())
        best = ref.topk(4, 1).values
        assert torch.all((tlp[a: a + 500].double() - best).abs() <= E[:, None] + 2.0 ** -24 * best.abs())
        H = -(p * ref).sum(1)
        assert torch.all((ent[a: a + 500].double() - H).abs() <= E * (1 + 2 * spread) + 40 * 2.0 ** -24 * spread + 2.0 ** -24 * H)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,vocab,top", [(1, 151936, 20.0), (2, 50272, 20.0), (300, 50272, 18.0), (1000, 20000, 20.0),
                                            (4100, 5000, 16.0)])
def test_entropy_where_one_token_has_nearly_all(zo, ctx, dtype, rows, vocab, top):
    """One logit stands far above the others, all 0: its exponential is 1 exactly, and of the others only
    those of its own 4 vectors (32 at most) can vanish beside it in fp32; the rest is relative: 2^-22 of the
    exponential, two roundings of an argument of 29 at most, chains of 10 and 40."""
    x = torch.zeros(rows, vocab, device="cuda")
    at = (torch.arange(rows, device="cuda") * 7919) % vocab
    x[torch.arange(rows, device="cuda"), at] = top
    x = x.to(TYPES[dtype])
    t = at.to(torch.int32)
    lp, ent, _, _ = call(zo, ctx, x, t, 0)
    rest = (vocab - 1) * math.exp(-top)
    H = math.log1p(rest) + rest * top / (1 + rest)
    lost = 32 * math.exp(-top)
    rel = 2.0 ** -22 + 2 * 29 * 2.0 ** -24 + 50 * 2.0 ** -24
    assert torch.all((lp.double() + math.log1p(rest)).abs() <= lost + rel * rest)
    assert torch.all((ent.double() - H).abs() <= lost + rel * H)


@pytest.mark.parametrize("rows", [5, 300, 4100])
def test_tokens_that_are_not_scored_give_0_whatever_the_row_holds(zo, ctx, rows):
    x, t = logits(rows, 700, "f32")
    x[1, 5], x[2] = math.nan, -math.inf
    t[:3] = -1
    lp, ent, _, _ = call(zo, ctx, x, t, 0)
    assert torch.all(lp[:3] == 0) and torch.isnan(ent[1:3]).all() and torch.isfinite(ent[0])
