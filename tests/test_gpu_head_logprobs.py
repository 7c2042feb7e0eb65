"""zo_head_logprobs against the product and log-softmax in 64 bits.

Tolerances: a logit is an fp32 sum of `width` exact products, off by at most
e_x = width 2^-23 max_j sum_i |h_i w_ji| whatever the order (2^-23: truncation); it moves lse and
the given logit by e_x each.  The statistics add E = (vocab / 16 + 24) 2^-24 + 2^-21 at most (a
thread sums every fourth or rarer column of its range; the bound takes one in 16 of all), as in
the tests of zo_logprobs:
    |logprob - ref| <= 2 e_x + E + 2^-25 (max - x_t) + 2^-24 |ref|,
    |H - ref| <= (E + 2 e_x) (1 + 2 sum_j p_j (max - x_j)) + 2^-24 |ref| + 2 e_x.
"""
import math

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def ctx(zo):
    c = zo.zo_create(torch.zeros(64, dtype=torch.bfloat16, device="cuda"))
    yield c
    c.close()


def make(rows, vocab, width, seed=0, scale=None, pad=0):
    g = torch.Generator(device="cuda").manual_seed(seed + rows + vocab + width)
    h = torch.randn(rows, width + pad, generator=g, device="cuda").to(torch.bfloat16)
    w = torch.randn(vocab, width + pad, generator=g, device="cuda") * (2.0 / math.sqrt(width) if scale is None else scale)
    t = torch.randint(0, vocab, (rows,), generator=g, device="cuda", dtype=torch.int32)
    return h, w.to(torch.bfloat16), t


def call(zo, ctx, h, w, t, width=None, guard=256):
    rows, vocab = len(h), len(w)
    width = h.shape[1] if width is None else width
    n = zo.zo_head_logprobs_workspace(rows, vocab)
    space = torch.full((n + guard,), 0xAB, dtype=torch.uint8, device="cuda")
    lp, ent = torch.full((rows,), 9.0, device="cuda"), torch.full((rows,), 9.0, device="cuda")
    zo.zo_head_logprobs(ctx, h, w, rows, vocab, width, h.stride(0), w.stride(0), t, lp, ent, space, n)
    assert zo.zo_sync(ctx) == 0
    assert torch.all(space[n:] == 0xAB)  # nothing behind the workspace
    return lp, ent


def check(h, w, t, got):
    lp, ent = got
    vocab, width = w.shape
    E = (vocab / 16 + 24) * 2.0 ** -24 + 2.0 ** -21
    for a in range(0, len(h), 512):
        H, T = h[a: a + 512].double(), t[a: a + 512].long()
        x = H @ w.double().T
        e = width * 2.0 ** -23 * (H.abs() @ w.double().abs().T).amax(1)
        ref = torch.log_softmax(x, 1)
        p = ref.exp()
        big = x.amax(1, keepdim=True)
        spread = (p * (big - x)).sum(1)
        want = torch.where(T >= 0, ref.gather(1, T.clamp(min=0)[:, None])[:, 0], torch.zeros_like(spread))
        gap = big[:, 0] - x.gather(1, T.clamp(min=0)[:, None])[:, 0]
        tol = 2 * e + E + 2.0 ** -25 * gap + 2.0 ** -24 * want.abs()
        off = (lp[a: a + 512].double() - want).abs()
        assert torch.all(off <= tol), (off / tol).max()
        ref_h = -(p * ref).sum(1)
        tol = (E + 2 * e) * (1 + 2 * spread) + 2.0 ** -24 * ref_h + 2 * e
        off = (ent[a: a + 512].double() - ref_h).abs()
        assert torch.all(off <= tol), (off / tol).max()


SIZES = [(1, 1, 8), (1, 2, 8), (3, 31, 16), (5, 32, 64), (1, 33, 72), (7, 257, 128), (127, 1000, 64), (128, 4736, 64),
         (129, 5000, 136), (16, 50272, 768), (1, 30001, 1024), (200, 9999, 512), (300, 500, 264), (1000, 3001, 64),
         (2049, 1200, 128), (513, 40000, 192), (4096, 20011, 64), (5, 1000, 1032), (200, 3000, 2056), (130, 1000, 4096),
         (257, 64, 8), (129, 63, 1024)]


@pytest.mark.parametrize("rows,vocab,width", SIZES)
def test_head_logprobs_match(zo, ctx, rows, vocab, width):
    h, w, t = make(rows, vocab, width)
    check(h, w, t, call(zo, ctx, h, w, t))


@pytest.mark.parametrize("scale", [1e-4, 1.0])
def test_flat_and_peaked_distributions(zo, ctx, scale):
    h, w, t = make(70, 7000, 256, scale=scale)
    t[:35] = (h[:35].double() @ w.double().T).argmax(1).to(torch.int32)
    check(h, w, t, call(zo, ctx, h, w, t))


@pytest.mark.parametrize("rows,vocab", [(40, 3000), (700, 3000), (1200, 9000)])
def test_strides(zo, ctx, rows, vocab):
    """Padded rows full of NaN behind the width."""
    h, w, t = make(rows, vocab, 200, pad=24)
    h[:, 200:] = math.nan
    w[:, 200:] = math.nan
    check(h[:, :200], w[:, :200], t, call(zo, ctx, h, w, t, width=200))


@pytest.mark.parametrize("rows", [3, 600])
def test_each_target_position_is_found(zo, ctx, rows):
    """Targets on every unit and tile edge, the first and the last."""
    vocab = 4111
    h, w, t = make(rows, vocab, 64)
    edges = [0, 1, 31, 32, 63, 64, 127, 128, 255, 256, 257, 4095, 4096, 4110]
    for a in range(0, len(edges), rows):
        part = torch.tensor(edges[a: a + rows], dtype=torch.int32, device="cuda")
        t[: len(part)] = part
        check(h, w, t, call(zo, ctx, h, w, t))


@pytest.mark.parametrize("rows", [6, 400])
def test_targets_outside_and_not_scored(zo, ctx, rows):
    h, w, t = make(rows, 500, 64)
    t[:5] = torch.tensor([-1, 500, -2, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32)
    lp, ent = call(zo, ctx, h, w, t)
    assert lp[0] == 0 and torch.isnan(lp[1:5]).all() and torch.isfinite(ent).all()
    check(h[5:], w, t[5:], (lp[5:], ent[5:]))


@pytest.mark.parametrize("rows", [9, 500])
def test_bad_rows_stay_their_own(zo, ctx, rows):
    h, w, t = make(rows, 2000, 128)
    want = call(zo, ctx, h, w, t)
    h[2, 5] = math.nan
    h[4] = math.inf
    lp, ent = call(zo, ctx, h, w, t)
    assert torch.isnan(lp[[2, 4]]).all() and torch.isnan(ent[[2, 4]]).all()
    keep = [i for i in range(rows) if i not in (2, 4)]
    assert torch.equal(lp[keep], want[0][keep]) and torch.equal(ent[keep], want[1][keep])


@pytest.mark.parametrize("rows", [9, 500])
@pytest.mark.parametrize("where", [0, 31, 1000, 1984, 1999])
@pytest.mark.parametrize("count", [1, 40, 600])
def test_a_bad_row_of_the_head_is_seen_by_every_row(zo, ctx, rows, where, count):
    """NaN in one or many rows of W, whole ranges of a CTA among them."""
    h, w, t = make(rows, 2000, 128)
    w[where: where + count] = math.nan
    lp, ent = call(zo, ctx, h, w, t)
    assert torch.isnan(lp).all() and torch.isnan(ent).all()


@pytest.mark.parametrize("rows", [9, 500])
@pytest.mark.parametrize("where,count", [(0, 1), (100, 40), (1300, 700)])
def test_ruled_out_tokens_leave_the_others_scores(zo, ctx, rows, where, count):
    """W rows that give a logit of -inf: probability 0, as if they were not there; a row without any
    other has no distribution."""
    h, w, t = make(rows, 2000, 128)
    h[:, 0] = 1.0
    w[where: where + count] = 0.0
    w[where: where + count, 0] = -math.inf
    t[:] = torch.arange(rows, device="cuda") % 50 + 50
    got = call(zo, ctx, h, w, t)
    keep = torch.ones(2000, dtype=torch.bool, device="cuda")
    keep[where: where + count] = False
    tk = (torch.cumsum(keep.int(), 0) - 1)[t.long()].to(torch.int32)
    check(h, w[keep], tk, got)
    t[:] = where
    lp, _ = call(zo, ctx, h, w, t)
    assert torch.all(lp == -math.inf)
    w[:] = w[where]
    lp, ent = call(zo, ctx, h, w, t)
    assert torch.isnan(lp).all() and torch.isnan(ent).all()


@pytest.mark.parametrize("rows", [4, 900])
def test_repeatable_and_one_output_only(zo, ctx, rows):
    h, w, t = make(rows, 20000, 256)
    lp, ent = call(zo, ctx, h, w, t)
    again = call(zo, ctx, h, w, t)
    assert torch.equal(lp, again[0]) and torch.equal(ent, again[1])
    n = zo.zo_head_logprobs_workspace(rows, 20000)
    space = torch.empty(n, dtype=torch.uint8, device="cuda")
    a, b = torch.zeros_like(lp), torch.zeros_like(ent)
    zo.zo_head_logprobs(ctx, h, w, rows, 20000, 256, 256, 256, t, a, None, space)
    zo.zo_head_logprobs(ctx, h, w, rows, 20000, 256, 256, 256, None, None, b, space)
    assert torch.equal(a, lp) and torch.equal(b, ent)


def test_agrees_with_logits_in_memory(zo, ctx):
    """The same rows through zo_gemm_bf16 (fp32 output) and zo_logprobs."""
    h, w, t = make(256, 5000, 512)
    x = torch.zeros(256, 5000, device="cuda")
    zo.zo_gemm_bf16(ctx, h, w, None, x, 256, 5000, 512, 5000, zo.ZO_EPI_RESID_F32)
    a, b = torch.zeros(256, device="cuda"), torch.zeros(256, device="cuda")
    zo.zo_logprobs(ctx, x, 256, 5000, 5000, t, a, b)
    lp, ent = call(zo, ctx, h, w, t)
    e = 512 * 2.0 ** -23 * (h.double().abs() @ w.double().abs().T).amax(1)
    assert torch.all((lp.double() - a).abs() <= 4 * e + 1e-4) and torch.all((ent.double() - b).abs() <= 20 * e + 1e-4)


@pytest.mark.parametrize("rows", [20, 512])
def test_replayed(zo, rows):
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        c = zo.zo_create(torch.zeros(64, device="cuda"), stream=s)
        h, w, t = make(rows, 4000, 128)
        lp, ent = torch.zeros(rows, device="cuda"), torch.zeros(rows, device="cuda")
        space = torch.empty(zo.zo_head_logprobs_workspace(rows, 4000), dtype=torch.uint8, device="cuda")
        # once before the capture, as any kernel's first launch sets it up
        zo.zo_head_logprobs(c, h, w, rows, 4000, 128, 128, 128, t, lp, ent, space)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        zo.zo_head_logprobs(c, h, w, rows, 4000, 128, 128, 128, t, lp, ent, space)
    for seed in (5, 6):
        with torch.cuda.stream(s):
            h.copy_(make(rows, 4000, 128, seed=seed)[0])
            g.replay()
        s.synchronize()
        check(h, w, t, (lp, ent))
    del g
    c.close()


def test_head_refusals(zo, ctx):
    h, w, t = make(4, 100, 64)
    lp, ent = torch.full((4,), 9.0, device="cuda"), torch.full((4,), 9.0, device="cuda")
    n = zo.zo_head_logprobs_workspace(4, 100)
    space = torch.zeros(n, dtype=torch.uint8, device="cuda")
    base = dict(h=h, w=w, rows=4, vocab=100, width=64, ldh=64, ldw=64, t=t, lp=lp, ent=ent, space=space, n=n)

    def refused(**k):
        a = dict(base, **k)
        with pytest.raises(zo.ZoError) as e:
            zo.zo_head_logprobs(ctx, a["h"], a["w"], a["rows"], a["vocab"], a["width"], a["ldh"], a["ldw"], a["t"],
                                a["lp"], a["ent"], a["space"], a["n"])
        assert e.value.status == zo.ZO_ERR_INVALID

    for name in ("h", "w", "space"):
        refused(**{name: 0})
    for name in ("h", "w", "space"):
        refused(**{name: a.data_ptr() + 8 if (a := base[name]) is not None else 0})
    for name in ("rows", "vocab", "width"):
        refused(**{name: 0})
    refused(rows=1 << 31)
    refused(vocab=1 << 31)
    refused(width=60)
    refused(width=72)
    refused(ldh=60)
    refused(ldw=68)
    refused(t=None)
    refused(lp=None, ent=None)
    refused(n=n - 1)
    refused(lp=lp.data_ptr() + 2)
    torch.cuda.synchronize()
    assert torch.all(lp == 9.0)


def exact_scores(x, t):
    """(logprob, entropy, sum_j p_j (max - x_j)) of exact logits, in 64 bits."""
    ref = torch.log_softmax(x, 1)
    p = ref.exp()
    spread = torch.where(p > 0, p * (x.amax(1, keepdim=True) - x), torch.zeros_like(x)).sum(1)
    return ref.gather(1, t.long()[:, None])[:, 0], -(p * torch.where(p > 0, ref, torch.zeros_like(ref))).sum(1), spread


@pytest.mark.parametrize("rows", [5, 200])
@pytest.mark.parametrize("width", [2048, 4096, 4104])
def test_small_products_stand_beside_large_ones_over_wide_widths(zo, ctx, rows, width):
    """Logits of 1024 from the first column, and 2^-19 from every one behind the first accumulator: one
    accumulator over the whole width would lose all of those (16 at a time are a quarter of its last bit),
    accumulators of 1024 or 512 hold them exactly, and so does their sum (whole multiples of 2^-13)."""
    part, vocab = 1024 if width <= 2048 else 512, 700
    h, w = torch.zeros(rows, width, device="cuda"), torch.zeros(vocab, width, device="cuda")
    h[:, 0], h[:, part:] = 32.0, 2.0 ** -9
    w[:, 0] = 31.75
    w[::7, 0] = 32.0
    w[::14, part: width // 64 * 64] = 2.0 ** -10
    h, w = h.to(torch.bfloat16), w.to(torch.bfloat16)
    t = (torch.arange(rows, device="cuda") % 50 * 7).to(torch.int32)
    lp, ent = call(zo, ctx, h, w, t)
    want, want_h, spread = exact_scores(h.double() @ w.double().T, t)
    # exponentials (2^-22), chains of 10, arguments up to 14 (2^-24 each): the small products matter 2e-3
    E = 2.0 ** -22 + 10 * 2.0 ** -24 + 2.0 ** -24 * (1 + spread)
    assert torch.all((lp.double() - want).abs() <= E + 2.0 ** -24 * want.abs())
    assert torch.all((ent.double() - want_h).abs() <= E * (3 + 2 * spread) + 2.0 ** -24 * want_h)
    assert (want[0] - want[1]).abs() > 1e-3  # (tokens 0 and 7: with the small products and without)


@pytest.mark.parametrize("rows,vocab", [(3, 50272), (300, 50272), (5, 151936)])
def test_statistics_of_exact_logits(zo, ctx, rows, vocab):
    """Logits that are one product each, so that only the statistics are off: 32 columns at a time in fp32
    (exponentials 2^-22, four chains of 8 and their sum, arguments 2^-24 of their size), beyond in fp64."""
    g = torch.Generator(device="cuda").manual_seed(rows)
    x = (torch.randn(vocab, generator=g, device="cuda") * 3).to(torch.bfloat16)
    h, w = torch.zeros(rows, 8, device="cuda"), torch.zeros(vocab, 8, device="cuda", dtype=torch.bfloat16)
    h[:, 0] = torch.tensor([1.0, 0.5, 1.25], device="cuda")[torch.arange(rows, device="cuda") % 3]
    w[:, 0] = x
    h = h.to(torch.bfloat16)
    t = torch.randint(0, vocab, (rows,), generator=g, device="cuda", dtype=torch.int32)
    lp, ent = call(zo, ctx, h, w, t)
    for r in (0, 1, 2):
        want, want_h, spread = exact_scores(h[r: r + 1].double() @ w.double().T, t[r: r + 1])
        E = 2.0 ** -22 + 10 * 2.0 ** -24 + 2.0 ** -24 * (1 + spread)
        gap = 2.0 ** -25 * 40
        assert (lp[r].double() - want).abs() <= E + gap + 2.0 ** -24 * want.abs()
        assert (ent[r].double() - want_h).abs() <= E * (3 + 2 * spread) + 2.0 ** -24 * want_h
    same = torch.arange(rows, device="cuda") % 3
    assert torch.equal(ent, ent[:3][same])


@pytest.mark.parametrize("rows", [4, 200])
def test_entropy_where_one_token_has_nearly_all(zo, ctx, rows):
    """One logit of 20, the others 0: entropies of 2e-3 and less, off by the largest token's exponential
    (2^-22) and the chains that it stands in (10 steps each of s and u)."""
    vocab = 50272
    h, w = torch.zeros(rows, 8, device="cuda"), torch.zeros(vocab, 8, device="cuda")
    h[:, 0], w[777, 0] = 1.0, 20.0
    w[778, 1] = 4.0
    h[:, 1] = (torch.arange(rows, device="cuda") % 5).float()
    h, w = h.to(torch.bfloat16), w.to(torch.bfloat16)
    t = torch.full((rows,), 777, dtype=torch.int32, device="cuda")
    lp, ent = call(zo, ctx, h, w, t)
    want, want_h, _ = exact_scores(h.double() @ w.double().T, t)
    assert torch.all((lp.double() - want).abs() <= 2.0 ** -22 + 10 * 2.0 ** -24 + 2.0 ** -19 * want.abs())
    assert torch.all((ent.double() - want_h).abs() <= 2.0 ** -22 + 20 * 2.0 ** -24 + 2.0 ** -19 * want_h)


@pytest.mark.parametrize("rows", [5, 300])
def test_tokens_that_are_not_scored_give_0_whatever_the_row_holds(zo, ctx, rows):
    h, w, t = make(rows, 700, 64)
    h[1, 5] = math.nan
    t[:2] = -1
    lp, ent = call(zo, ctx, h, w, t)
    assert torch.all(lp[:2] == 0) and torch.isnan(ent[1]) and torch.isfinite(ent[0])
