"""zo_attention_packed against softmax attention in 64 bits, sequence by sequence.

Tolerance per output, with w the exact weights and A = sum_j w_j |v_j|: the probabilities of
P V are rounded to bf16 (2^-8 each), the exponentials are approximate to 2^-21, a score's error
moves every weight by at most e_s relative, and the output is rounded to bf16 once:
    |out - ref| <= A (2^-8 + 2^-20 + 2 e_s) + 2^-8 |ref| + 2^-8 A (second order, absorbed by 1.02),
with e_s = 2 head_dim 2^-23 max_j sum_e |q_e k_je| scale + 2^-23 max |score| (fp32 sums of exact
products, truncated at worst, and the scaling).
"""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def ctx(zo):
    c = zo.zo_create(torch.zeros(64, dtype=torch.bfloat16, device="cuda"))
    yield c
    c.close()


def offsets(lens):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")


def reference(q, k, v, lens, H, Hk, hd, scale):
    """(fp64 output, tolerance) of the rows inside the sequences."""
    at, outs, tols = 0, [], []
    for n in lens:
        if n == 0:
            continue
        sl = slice(at, at + n)
        at += n
        Q = q[sl].double().reshape(n, H, hd).transpose(0, 1)
        K = k[sl].double().reshape(n, Hk, hd).transpose(0, 1).repeat_interleave(H // Hk, 0)
        V = v[sl].double().reshape(n, Hk, hd).transpose(0, 1).repeat_interleave(H // Hk, 0)
        s = Q @ K.transpose(1, 2) * scale
        size = Q.abs() @ K.abs().transpose(1, 2) * scale
        mask = torch.ones(n, n, dtype=torch.bool, device="cuda").triu(1)
        s = s.masked_fill(mask, -math.inf)
        w = torch.softmax(s, -1)
        o, A = w @ V, w @ V.abs()
        e = 2 * hd * 2.0 ** -23 * size.masked_fill(mask, 0).amax(-1) \
            + 2.0 ** -23 * s.masked_fill(mask, 0).abs().amax(-1)
        tol = 1.02 * (A * (2.0 ** -8 + 2.0 ** -20 + 2 * e[..., None]) + 2.0 ** -8 * o.abs()) + 1e-30
        outs.append(o.transpose(0, 1).reshape(n, H * hd))
        tols.append(tol.transpose(0, 1).reshape(n, H * hd))
    return torch.cat(outs), torch.cat(tols)


def make(lens, H, Hk, hd, extra=0, seed=0, scale_q=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed + sum(lens) + H + hd)
    total = sum(lens) + extra
    qkv = torch.randn(total, (H + 2 * Hk) * hd, generator=g, device="cuda")
    qkv[:, : H * hd] *= scale_q
    return qkv.to(torch.bfloat16)


def split(qkv, H, Hk, hd):
    return qkv[:, : H * hd], qkv[:, H * hd: (H + Hk) * hd], qkv[:, (H + Hk) * hd:]


def call(zo, ctx, qkv, out, cu, H, Hk, hd, scale=None):
    q, k, v = split(qkv, H, Hk, hd)
    ld = qkv.shape[1]
    zo.zo_attention_packed(ctx, q, k, v, out, cu, cu.numel() - 1, qkv.shape[0], ld, ld, ld, H * hd, H, Hk, hd,
                           1 / math.sqrt(hd) if scale is None else scale)


def check(zo, ctx, qkv, out, lens, H, Hk, hd, scale=None):
    n = sum(lens)
    q, k, v = split(qkv, H, Hk, hd)
    ref, tol = reference(q, k, v, lens, H, Hk, hd, 1 / math.sqrt(hd) if scale is None else scale)
    bad = ~((out[:n].double() - ref).abs() <= tol)
    assert not bad.any(), (bad.sum().item(), ((out[:n].double() - ref).abs() / tol).max().item())


LENS = [[1], [2], [17], [64], [65], [127], [128], [129], [191, 1, 0, 193], [256, 255, 257], [0, 0, 3, 0],
        [640, 5, 1, 1, 1, 300], [1] * 70, [700], [130, 1026]]


@pytest.mark.parametrize("lens", LENS, ids=lambda v: "-".join(map(str, v[:6])))
@pytest.mark.parametrize("H,Hk,hd", [(4, 2, 128), (3, 3, 64), (8, 1, 64), (1, 1, 128), (4, 4, 64), (6, 2, 64),
                                     (2, 2, 128), (6, 2, 128)])
def test_packed_attention_matches(zo, ctx, lens, H, Hk, hd):
    qkv = make(lens, H, Hk, hd)
    out = torch.zeros(max(1, sum(lens)), H * hd, dtype=torch.bfloat16, device="cuda")
    call(zo, ctx, qkv, out, offsets(lens), H, Hk, hd)
    assert zo.zo_sync(ctx) == 0
    check(zo, ctx, qkv, out, lens, H, Hk, hd)


@pytest.mark.parametrize("hd", [64, 128])
def test_packed_attention_long_sequences(zo, ctx, hd):
    lens = [2500, 4097]
    qkv = make(lens, 2, 1, hd)
    out = torch.zeros(sum(lens), 2 * hd, dtype=torch.bfloat16, device="cuda")
    call(zo, ctx, qkv, out, offsets(lens), 2, 1, hd)
    assert zo.zo_sync(ctx) == 0
    check(zo, ctx, qkv, out, lens, 2, 1, hd)
    again = torch.zeros_like(out)
    call(zo, ctx, qkv, again, offsets(lens), 2, 1, hd)
    assert torch.equal(out, again)


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("scale_q", [30.0, 1e-3])
def test_packed_attention_sharp_and_flat_scores(zo, ctx, hd, scale_q):
    """Scores up to some hundreds (the running maximum grows far from tile to tile) and near 0."""
    lens = [300, 77, 513]
    qkv = make(lens, 4, 4, hd, scale_q=scale_q)
    out = torch.zeros(sum(lens), 4 * hd, dtype=torch.bfloat16, device="cuda")
    call(zo, ctx, qkv, out, offsets(lens), 4, 4, hd)
    check(zo, ctx, qkv, out, lens, 4, 4, hd)


@pytest.mark.parametrize("hd", [64, 128])
def test_packed_attention_growing_scores(zo, ctx, hd):
    """Scores that grow by 2^16 from one group of 64 keys to the next: rescaled every time."""
    lens, H = [520, 260], 2
    total = sum(lens)
    r = np.random.default_rng(hd)
    q = np.ones((total, H, hd)) * 2.0 / np.sqrt(hd) + 0.1 * r.standard_normal((total, H, hd))
    pos = np.concatenate([np.arange(n) for n in lens])
    k = q.mean(axis=0, keepdims=True) * (pos[:, None, None] / 2.0) + 0.1 * r.standard_normal((total, H, hd))
    v = r.standard_normal((total, H, hd))
    qkv = torch.from_numpy(np.concatenate([x.reshape(total, -1) for x in (q, k, v)], 1).astype(np.float32))
    qkv = qkv.to(torch.bfloat16).cuda()
    out = torch.zeros(total, H * hd, dtype=torch.bfloat16, device="cuda")
    call(zo, ctx, qkv, out, offsets(lens), H, H, hd)
    check(zo, ctx, qkv, out, lens, H, H, hd)


def test_packed_attention_separate_tensors_strides_and_scale(zo, ctx):
    lens, H, Hk, hd = [33, 140, 200], 4, 2, 64
    n = sum(lens)
    g = torch.Generator(device="cuda").manual_seed(3)

    def t(cols, pad):
        return torch.randn(n, cols + pad, generator=g, device="cuda").to(torch.bfloat16)

    q, k, v = t(H * hd, 8), t(Hk * hd, 64), t(Hk * hd, 0)
    out = torch.full((n, H * hd + 16), 5.0, dtype=torch.bfloat16, device="cuda")
    zo.zo_attention_packed(ctx, q, k, v, out, offsets(lens), len(lens), n, H * hd + 8, Hk * hd + 64, Hk * hd,
                           H * hd + 16, H, Hk, hd, 0.3)
    ref, tol = reference(q[:, : H * hd], k[:, : Hk * hd], v, lens, H, Hk, hd, float(np.float32(0.3)))
    assert torch.all((out[:, : H * hd].double() - ref).abs() <= tol)
    assert torch.all(out[:, H * hd:] == 5.0)


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("what", [math.nan, math.inf])
def test_rows_outside_a_sequence_do_not_reach_it(zo, ctx, hd, what):
    """Neighbour sequences and padding full of NaN or infinities; rows behind the last sequence
    are left as they were."""
    lens, H, Hk = [100, 30, 129, 64, 3], 2, 1
    qkv = make(lens, H, Hk, hd, extra=150)
    clean = qkv.clone()
    at = np.cumsum([0] + lens)
    qkv[at[1]: at[2]] = what
    qkv[at[3]: at[4]] = what
    qkv[at[-1]:] = what
    out = torch.full((len(qkv), H * hd), 3.0, dtype=torch.bfloat16, device="cuda")
    call(zo, ctx, qkv, out, offsets(lens), H, Hk, hd)
    want = torch.full_like(out, 3.0)
    call(zo, ctx, clean, want, offsets(lens), H, Hk, hd)
    assert zo.zo_sync(ctx) == 0
    for i in (0, 2, 4):
        assert torch.equal(out[at[i]: at[i + 1]], want[at[i]: at[i + 1]])
    for i in (1, 3):
        assert not torch.isfinite(out[at[i]: at[i + 1]]).any()
    assert torch.all(out[at[-1]:] == 3.0)


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("where", ["k", "v", "q", "kv"])
@pytest.mark.parametrize("what", [math.nan, math.inf, -math.inf])
def test_a_later_token_does_not_reach_earlier_rows(zo, ctx, hd, where, what):
    lens, H, Hk, bad = [300, 200], 2, 1, 170
    qkv = make(lens, H, Hk, hd)
    clean = qkv.clone()
    q, k, v = split(qkv, H, Hk, hd)
    for name, t in (("q", q), ("k", k), ("v", v)):
        if name in where:
            t[bad] = what
    out = torch.zeros(len(qkv), H * hd, dtype=torch.bfloat16, device="cuda")
    call(zo, ctx, qkv, out, offsets(lens), H, Hk, hd)
    assert zo.zo_sync(ctx) == 0
    cq, ck, cv = split(clean, H, Hk, hd)
    ref, tol = reference(cq, ck, cv, lens, H, Hk, hd, 1 / math.sqrt(hd))
    rows = list(range(bad)) + list(range(300, 500))
    if where == "q":
        rows += list(range(bad + 1, 300))
    err = (out.double() - ref).abs()
    assert torch.all(err[rows] <= tol[rows])
    if "v" in where or where == "q":
        assert not torch.isfinite(out[bad]).any()


@pytest.mark.parametrize("hd", [64, 128])
def test_single_bad_values_stay_in_their_column(zo, ctx, hd):
    """One infinite feature of one value row: earlier rows finite, its own and later rows infinite
    in that column of the sharing heads only."""
    lens, H, Hk = [260], 4, 2
    qkv = make(lens, H, Hk, hd)
    q, k, v = split(qkv, H, Hk, hd)
    v[200, hd + 7] = math.inf
    out = torch.zeros(260, H * hd, dtype=torch.bfloat16, device="cuda")
    call(zo, ctx, qkv, out, offsets(lens), H, Hk, hd)
    bad = ~torch.isfinite(out)
    want = torch.zeros_like(bad)
    want[200:, 2 * hd + 7] = want[200:, 3 * hd + 7] = True
    assert torch.equal(bad, want)
    v[200, hd + 7] = 0.0
    ref, tol = reference(q, k, v, lens, H, Hk, hd, 1 / math.sqrt(hd))
    assert torch.all(((out.double() - ref).abs() <= tol)[:200])


def test_matches_equal_lengths_without_packing(zo, ctx):
    """The batch of equal lengths that zo_attention_gqa takes."""
    B, S, H, Hk, hd = 3, 200, 4, 2, 128
    qkv = make([S] * B, H, Hk, hd)
    a = torch.zeros(B * S, H * hd, dtype=torch.bfloat16, device="cuda")
    b = torch.zeros_like(a)
    call(zo, ctx, qkv, a, offsets([S] * B), H, Hk, hd)
    zo.zo_attention_gqa(ctx, qkv, b, B, S, H, Hk, hd)
    q, k, v = split(qkv, H, Hk, hd)
    _, tol = reference(q, k, v, [S] * B, H, Hk, hd, 1 / math.sqrt(hd))
    assert torch.all((a.double() - b.double()).abs() <= 2 * tol)


def test_many_short_sequences(zo, ctx):
    r = np.random.default_rng(0)
    lens = r.integers(0, 4, 2000).tolist() + [129]
    qkv = make(lens, 2, 2, 64)
    out = torch.zeros(sum(lens), 128, dtype=torch.bfloat16, device="cuda")
    call(zo, ctx, qkv, out, offsets(lens), 2, 2, 64)
    assert zo.zo_sync(ctx) == 0
    check(zo, ctx, qkv, out, lens, 2, 2, 64)


@pytest.mark.parametrize("cu,kept", [([0, 50, 40, 90], [(0, 50), (40, 90)]), ([0, 60, 200], [(0, 60)]),
                                     ([-5, 10, 100], [(10, 100)])])
def test_bad_offsets_raise_the_flag_and_are_skipped(zo, ctx, cu, kept):
    """Pairs that decrease or leave the buffer: reported by zo_sync, nothing written for them."""
    H, hd, total = 2, 64, 100
    qkv = make([total], H, H, hd)
    out = torch.full((total, H * hd), 4.0, dtype=torch.bfloat16, device="cuda")
    call(zo, ctx, qkv, out, torch.tensor(cu, dtype=torch.int32, device="cuda"), H, H, hd)
    with pytest.raises(zo.ZoError) as e:
        zo.zo_sync(ctx)
    assert e.value.status == zo.ZO_ERR_INVALID
    assert zo.zo_sync(ctx) == 0  # cleared
    inside = torch.zeros(total, dtype=torch.bool, device="cuda")
    for a, b in kept:
        inside[a:b] = True
    assert torch.all(out[~inside] == 4.0)
    a, b = kept[-1]
    q, k, v = split(qkv[a:b], H, H, hd)
    ref, tol = reference(q, k, v, [b - a], H, H, hd, 1 / math.sqrt(hd))
    if len(kept) == 1:
        assert torch.all((out[a:b].double() - ref).abs() <= tol)


@pytest.mark.parametrize("H,Hk,hd", [(2, 2, 64), (2, 2, 128), (3, 1, 64)])
@pytest.mark.parametrize("what", [math.nan, math.inf])
def test_bad_rows_stay_out_however_heads_are_paired(zo, ctx, H, Hk, hd, what):
    """Neighbour sequences, padding and a later token full of NaN or infinities, with pairs of heads
    that share no key/value head and with two tiles of one head."""
    lens, late = [100, 30, 300, 64, 3, 390], 250
    qkv = make(lens, H, Hk, hd, extra=150)
    clean = qkv.clone()
    at = np.cumsum([0] + lens)
    qkv[at[1]: at[2]] = what
    qkv[at[3]: at[4]] = what
    qkv[at[2] + late, H * hd:] = what          # a key and value row of the third sequence
    qkv[at[-1]:] = what
    out = torch.full((len(qkv), H * hd), 3.0, dtype=torch.bfloat16, device="cuda")
    call(zo, ctx, qkv, out, offsets(lens), H, Hk, hd)
    assert zo.zo_sync(ctx) == 0
    q, k, v = split(clean, H, Hk, hd)
    ref, tol = reference(q, k, v, lens, H, Hk, hd, 1 / math.sqrt(hd))
    err = (out[: at[-1]].double() - ref).abs()
    for i in (0, 4, 5):
        assert torch.all(err[at[i]: at[i + 1]] <= tol[at[i]: at[i + 1]])
    assert torch.all(err[at[2]: at[2] + late] <= tol[at[2]: at[2] + late])
    assert torch.all(out[at[-1]:] == 3.0)


@pytest.mark.parametrize("H,Hk,hd", [(4, 2, 128), (4, 4, 64), (3, 3, 64)])
def test_many_sequences_of_several_tiles(zo, ctx, H, Hk, hd):
    """More than 32 sequences with up to four tiles: several rounds of items on every CTA."""
    r = np.random.default_rng(1)
    lens = r.integers(0, 450, 110).tolist()
    qkv = make(lens, H, Hk, hd, extra=9)
    out = torch.full((len(qkv), H * hd), 3.0, dtype=torch.bfloat16, device="cuda")
    call(zo, ctx, qkv, out, offsets(lens), H, Hk, hd)
    assert zo.zo_sync(ctx) == 0
    check(zo, ctx, qkv, out, lens, H, Hk, hd)
    assert torch.all(out[sum(lens):] == 3.0)


def test_two_graphs_of_one_context_and_changed_lengths(zo):
    """Captured once, replayed with other offsets in the same buffers; two graphs in turn."""
    s = torch.cuda.Stream()
    H, hd = 2, 128
    with torch.cuda.stream(s):
        c = zo.zo_create(torch.zeros(64, device="cuda"), stream=s)
        qkv = make([400], H, H, hd)
        outs = [torch.zeros(400, H * hd, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        cus = [offsets([100, 200, 100]), offsets([399, 1, 0])]
    s.synchronize()
    graphs = []
    for o, cu in zip(outs, cus):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            call(zo, c, qkv, o, cu, H, H, hd)
        graphs.append(g)
    for lens in ([100, 200, 100], [1, 398, 1], [0, 0, 400]):
        with torch.cuda.stream(s):
            cus[0].copy_(offsets(lens))
            for g in graphs:
                g.replay()
        s.synchronize()
        check(zo, c, qkv, outs[0], lens, H, H, hd)
        check(zo, c, qkv, outs[1], [399, 1, 0], H, H, hd)
    assert zo.zo_sync(c) == 0
    del graphs, g
    c.close()


def test_packed_attention_refusals(zo, ctx):
    H, hd, n = 2, 64, 20
    qkv = make([n], H, H, hd)
    out = torch.full((n, H * hd), 2.0, dtype=torch.bfloat16, device="cuda")
    base = dict(q=qkv, k=qkv, v=qkv, out=out, cu=offsets([n]), n=1, total=n, ldq=384, ldk=384, ldv=384, ldo=128,
                H=H, Hk=H, hd=hd, scale=0.1)

    def refused(status=None, **k):
        a = dict(base, **k)
        with pytest.raises(zo.ZoError) as e:
            zo.zo_attention_packed(ctx, a["q"], a["k"], a["v"], a["out"], a["cu"], a["n"], a["total"], a["ldq"],
                                   a["ldk"], a["ldv"], a["ldo"], a["H"], a["Hk"], a["hd"], a["scale"])
        assert e.value.status == (zo.ZO_ERR_INVALID if status is None else status)

    for name in ("q", "k", "v", "out", "cu"):
        refused(**{name: 0})
    for name in ("q", "k", "v", "out"):
        refused(**{name: qkv.data_ptr() + 2})
    for name in ("ldq", "ldk", "ldv", "ldo"):
        refused(**{name: 120})
        refused(**{name: 388})
    refused(n=0)
    refused(n=(1 << 24) + 1)
    refused(total=0)
    refused(total=1 << 31)
    refused(H=0)
    refused(H=3, Hk=2, ldo=192)
    refused(Hk=0)
    for scale in (0.0, -1.0, math.inf, math.nan):
        refused(scale=scale)
    refused(status=zo.ZO_ERR_UNSUPPORTED, hd=96)
    torch.cuda.synchronize()
    assert torch.all(out == 2.0)


def by_definition(q, k, v, lens, H, Hk, hd, scale):
    """(fp64 output with infinities and NaN where the sum over a row's own keys has them, tolerance of
    the finite ones).  Weights are taken as positive wherever the score is not -inf or NaN."""
    fill = torch.where(torch.isfinite(v), v, torch.zeros_like(v))
    ref, tol = reference(q, k, fill, lens, H, Hk, hd, scale)
    at = 0
    for n in lens:
        V = v[at: at + n].reshape(n, Hk, hd).repeat_interleave(H // Hk, 1).reshape(n, H * hd)
        up, down = (V == math.inf).cumsum(0) > 0, (V == -math.inf).cumsum(0) > 0
        nan = (torch.isnan(V).cumsum(0) > 0) | (up & down)
        o = ref[at: at + n]
        o[up] = math.inf
        o[down] = -math.inf
        o[nan] = math.nan
        at += n
    return ref, tol


def same_or_close(out, ref, tol):
    """Where the reference is finite, within tol; elsewhere the same infinity, or NaN."""
    out = out.double()
    close = torch.isfinite(ref) & ((out - ref).abs() <= tol)
    return close | (out == ref) | (torch.isnan(out) & torch.isnan(ref))


# sequences, and (row, own column's value) before (row, later value) of one sequence
OWN_AND_LATER = [([260], 0, 130, 170),           # inside the second tile's diagonal
                 ([40, 500, 300], 1, 3, 100),    # the first tile, between other sequences
                 ([700], 0, 10, 650),            # own value tiles ahead of the diagonal one
                 ([30, 9], 0, 3, 9),             # short sequences: one group of 16 keys
                 ([30, 9], 0, 3, 25)]            # the second group


@pytest.mark.parametrize("H,Hk,hd", [(4, 2, 128), (4, 2, 64), (2, 2, 64), (3, 3, 64), (1, 1, 128)])
@pytest.mark.parametrize("lens,seq,own,late", OWN_AND_LATER)
@pytest.mark.parametrize("first", [math.inf, -math.inf])
@pytest.mark.parametrize("then", [math.nan, math.inf, -math.inf])
def test_own_infinities_stand_beside_later_bad_values(zo, ctx, H, Hk, hd, lens, seq, own, late, first, then):
    """A value column with an infinity of a row's own and a bad value of a later token: the infinity, up to
    the later token.  Columns that hold nothing bad keep the bits that they have without it."""
    qkv = make(lens, H, Hk, hd)
    clean = torch.zeros(sum(lens), H * hd, dtype=torch.bfloat16, device="cuda")
    call(zo, ctx, qkv, clean, offsets(lens), H, Hk, hd)
    q, k, v = split(qkv, H, Hk, hd)
    row0 = sum(lens[:seq])
    v[row0 + own, 5] = first
    v[row0 + late, 5] = then
    v[row0 + late, hd - 3] = then     # a column with nothing bad before
    v[row0 + own, 9] = first          # one with nothing bad behind
    out = torch.zeros_like(clean)
    call(zo, ctx, qkv, out, offsets(lens), H, Hk, hd)
    assert zo.zo_sync(ctx) == 0
    ref, tol = by_definition(q, k, v, lens, H, Hk, hd, 1 / math.sqrt(hd))
    ok = same_or_close(out, ref, tol)
    assert ok.all(), (~ok).nonzero()[:8].tolist()
    good = [c for c in range(H * hd) if c % hd not in (5, 9, hd - 3)]
    assert torch.equal(out[:, good], clean[:, good])


@pytest.mark.parametrize("H,Hk,hd", [(4, 2, 128), (2, 2, 64), (3, 3, 64), (1, 1, 128)])
@pytest.mark.parametrize("lens", [[300, 150], [12, 30, 1]])
def test_rows_whose_every_score_is_ruled_out_are_nan(zo, ctx, H, Hk, hd, lens):
    """Keys that give a score of -inf have no weight; a row with no other key has no softmax."""
    qkv = make(lens, H, Hk, hd)
    q, k, v = split(qkv, H, Hk, hd)
    q.view(-1, H, hd)[:, :, 0] = 1.0
    dead = {0: lens[0] // 2, 1: 2}                     # leading keys of the first two sequences
    at = np.cumsum([0] + lens)
    for i, n in dead.items():
        k.view(-1, Hk, hd)[at[i]: at[i] + n, :, 0] = -math.inf
    k.view(-1, Hk, hd)[at[1] + 5, :, 0] = -math.inf    # one key among others
    out = torch.zeros(sum(lens), H * hd, dtype=torch.bfloat16, device="cuda")
    call(zo, ctx, qkv, out, offsets(lens), H, Hk, hd)
    assert zo.zo_sync(ctx) == 0
    none = torch.zeros(sum(lens), dtype=torch.bool, device="cuda")
    for i, n in dead.items():
        none[at[i]: at[i] + n] = True
    assert torch.isnan(out[none]).all()
    # the others as if those keys were not there
    alive = torch.isfinite(k[:, 0]).tolist()
    for i, n in enumerate(lens):
        for r in range(n):
            if none[at[i] + r] or (r % 7 and r < n - 3):
                continue
            keep = [j for j in range(at[i], at[i] + r + 1) if alive[j]]
            for h in range(H):
                g = h // (H // Hk)
                K, V = k[keep, g * hd: (g + 1) * hd].double(), v[keep, g * hd: (g + 1) * hd].double()
                Q = q[at[i] + r, h * hd: (h + 1) * hd].double()
                s = K @ Q / math.sqrt(hd)
                w = torch.softmax(s, 0)
                ref, A = w @ V, w @ V.abs()
                e = 2 * hd * 2.0 ** -23 * (K.abs() @ Q.abs()).max() / math.sqrt(hd) + 2.0 ** -23 * s.abs().max()
                tol = 1.02 * (A * (2.0 ** -8 + 2.0 ** -20 + 2 * e) + 2.0 ** -8 * ref.abs())
                assert torch.all((out[at[i] + r, h * hd: (h + 1) * hd].double() - ref).abs() <= tol)


def scattered(n_seqs, lens, seed=0):
    """n_seqs lengths, all 0 but `lens`, which lie at random places, the last of all among them."""
    r = np.random.default_rng(seed)
    at = np.sort(r.choice(n_seqs - 1, len(lens) - 1, replace=False)).tolist() + [n_seqs - 1]
    out = np.zeros(n_seqs, dtype=np.int64)
    out[at] = lens
    return out


@pytest.mark.parametrize("H,Hk,hd", [(2, 1, 128), (2, 2, 64), (1, 1, 64)])
@pytest.mark.parametrize("n_seqs,lens", [
    (3000, [2000]), (3000, [1, 700, 33, 2000, 129]), (300000, [5000, 3, 1100, 64, 1100, 400]),
    (40000, [40 * k + 33 for k in range(60)]),            # more long ones than lanes, many distinct lengths
    ((1 << 20) + 77, [1300, 40, 900, 300, 2000, 128, 129, 700]),  # items of no tiles between the others
    ((1 << 20) + 77, [150 * k + 40 for k in range(40)])])
def test_few_long_sequences_among_many_empty_ones(zo, ctx, H, Hk, hd, n_seqs, lens):
    qkv = make(lens, H, Hk, hd)
    out = torch.zeros(sum(lens), H * hd, dtype=torch.bfloat16, device="cuda")
    call(zo, ctx, qkv, out, offsets(scattered(n_seqs, lens)), H, Hk, hd)
    assert zo.zo_sync(ctx) == 0
    check(zo, ctx, qkv, out, lens, H, Hk, hd)


def test_a_long_sequence_among_many_empty_ones_costs_few_scans(zo):
    """16384 tokens among 131072 sequences: 128 numbers of tiles, of which two occur.  A scan for every one
    of them takes more than 100 ms, one for every one that occurs a few."""
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        c = zo.zo_create(torch.zeros(64, device="cuda"), stream=s)
        qkv = make([16384], 2, 1, 64)
        out = torch.zeros(16384, 128, dtype=torch.bfloat16, device="cuda")
        cu = offsets(scattered(131072, [16384]))
        times = []
        for _ in range(4):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record(s)
            call(zo, c, qkv, out, cu, 2, 1, 64)
            b.record(s)
            s.synchronize()
            times.append(a.elapsed_time(b))
    assert zo.zo_sync(c) == 0
    assert min(times) < 30.0, times
    c.close()


@pytest.mark.parametrize("H,Hk,hd", [(1, 1, 64), (2, 1, 128)])
def test_a_late_bad_token_of_a_very_long_sequence_ends_no_wait(zo, ctx, H, Hk, hd):
    """Rows of its tile take seconds to compute again from 600000 keys: nothing in the kernel waits
    for them, and they come out right."""
    n, H_all = 600001, H + 2 * Hk
    g = torch.Generator(device="cuda").manual_seed(hd)
    qkv = torch.randn(n, H_all * hd, generator=g, device="cuda", dtype=torch.bfloat16)
    q, k, v = split(qkv, H, Hk, hd)
    v[n - 1] = math.nan
    out = torch.zeros(n, H * hd, dtype=torch.bfloat16, device="cuda")
    call(zo, ctx, qkv, out, offsets([n]), H, Hk, hd)
    assert zo.zo_sync(ctx) == 0
    assert torch.isnan(out[n - 1]).all() and torch.isfinite(out[: n - 1]).all()
    for r in (n - 2, n - 3, n - 34, n // 128 * 128 - 1, 300000):
        for h in range(H):
            Q = q[r, h * hd: (h + 1) * hd].double()
            K, V = k[: r + 1, :hd].double(), v[: r + 1, :hd].double()
            s = K @ Q / math.sqrt(hd)
            w = torch.softmax(s, 0)
            ref, A = w @ V, w @ V.abs()
            # as above, and a sum of r + 1 fp32 terms in chains of n / 32 at most
            e = 2 * hd * 2.0 ** -23 * (K.abs() @ Q.abs()).max() / math.sqrt(hd) + 2.0 ** -23 * s.abs().max() + n / 32 * 2.0 ** -23
            tol = 1.02 * (A * (2.0 ** -8 + 2.0 ** -20 + 2 * e) + 2.0 ** -8 * ref.abs())
            assert torch.all((out[r, h * hd: (h + 1) * hd].double() - ref).abs() <= tol)


@pytest.mark.parametrize("H,Hk,hd", [(4, 2, 128), (2, 2, 64), (3, 3, 64)])
@pytest.mark.parametrize("lens", [[500, 40, 9], [30, 9, 17]])
def test_infinities_in_many_rows(zo, ctx, H, Hk, hd, lens):
    """Value columns that are infinite in every row, from a row on, up to a row, or with either sign in turn:
    every row is looked at again, for several columns and with several rows at a time."""
    qkv = make(lens, H, Hk, hd)
    q, k, v = split(qkv, H, Hk, hd)
    at = torch.arange(sum(lens), device="cuda")
    v[:, 5] = math.inf
    v[:, 6] = torch.where(at % 2 == 0, math.inf, -math.inf).to(torch.bfloat16)
    v[:, hd - 1] = -math.inf
    v[lens[0] - 7:, 8] = math.inf
    v[:13, 9] = -math.inf
    v[20:, 9] = math.nan
    v[7:, 33] = math.nan
    out = torch.zeros(sum(lens), H * hd, dtype=torch.bfloat16, device="cuda")
    call(zo, ctx, qkv, out, offsets(lens), H, Hk, hd)
    assert zo.zo_sync(ctx) == 0
    ref, tol = by_definition(q, k, v, lens, H, Hk, hd, 1 / math.sqrt(hd))
    ok = same_or_close(out, ref, tol)
    assert ok.all(), (~ok).nonzero()[:8].tolist()


def test_as_many_sequences_as_there_may_be(zo, ctx):
    """2^24 of them, a few long: the warps that wait for items wait for scans of all."""
    lens = [1300, 40, 900, 300, 2000, 128, 700]
    qkv = make(lens, 2, 1, 64)
    out = torch.zeros(sum(lens), 128, dtype=torch.bfloat16, device="cuda")
    call(zo, ctx, qkv, out, offsets(scattered(1 << 24, lens)), 2, 1, 64)
    assert zo.zo_sync(ctx) == 0
    check(zo, ctx, qkv, out, lens, 2, 1, 64)
