"""Host side of the packed-prompt operators, without a GPU: rotary frequencies and their
refusals, the workspace size, null contexts, and the block-to-work arithmetic of the kernels
restated in Python."""
import ctypes
import math

import numpy as np
import pytest

PLAIN = dict(theta=1.0e4, rot_dim=64)
BANDS = dict(theta=1.0e6, rot_dim=128, scaling="bands", factor=4.0, orig_len=4096.0, band_low=1.0,
             band_high=32.0)


def _formula(c):
    i = np.arange(c["rot_dim"] // 2)
    f = c["theta"] ** (-2.0 * i / c["rot_dim"])
    if c.get("scaling") == "linear":
        return f / c["factor"]
    if c.get("scaling") == "bands":
        wavelength = 2.0 * math.pi / f
        g = np.clip((c["orig_len"] / wavelength - c["band_low"]) / (c["band_high"] - c["band_low"]), 0, 1)
        return g * f + (1 - g) * f / c["factor"]
    return f


@pytest.mark.parametrize("cfg", [PLAIN, dict(PLAIN, rot_dim=2), dict(PLAIN, rot_dim=256, theta=5.0e5),
                                 dict(PLAIN, scaling="linear", factor=8.0), BANDS,
                                 dict(BANDS, band_high=4.0, factor=32.0, rot_dim=80)])
def test_rope_frequencies_follow_the_formula(zo, cfg):
    got = zo.zo_rope_frequencies(cfg)
    # pow, two products and a division in fp64: a handful of half steps of 2^-53
    np.testing.assert_allclose(got, _formula(cfg), rtol=16 * 2.0 ** -53, atol=0)


def test_rope_bands_keep_fast_and_interpolate_slow_frequencies(zo):
    plain = zo.zo_rope_frequencies(dict(theta=BANDS["theta"], rot_dim=128))
    scaled = zo.zo_rope_frequencies(BANDS)
    turns = BANDS["orig_len"] * plain / (2 * math.pi)
    assert np.array_equal(scaled[turns >= 32], plain[turns >= 32])
    assert np.array_equal(scaled[turns <= 1], plain[turns <= 1] / 4.0)
    assert np.all(np.diff(scaled) < 0)


@pytest.mark.parametrize("bad", [dict(theta=0.0), dict(theta=-1.0), dict(theta=math.inf), dict(theta=math.nan),
                                 dict(rot_dim=0), dict(rot_dim=3), dict(rot_dim=258), dict(rot_dim=-2),
                                 dict(scaling=7), dict(scaling="linear", factor=0.0),
                                 dict(scaling="linear", factor=math.nan),
                                 dict(scaling="bands", factor=2.0, orig_len=0.0, band_low=1.0, band_high=4.0),
                                 dict(scaling="bands", factor=2.0, orig_len=64.0, band_low=4.0, band_high=4.0),
                                 dict(magnitude=math.inf)])
def test_rope_configuration_refusals(zo, bad):
    with pytest.raises(zo.ZoError) as e:
        zo.zo_rope_frequencies({**PLAIN, **bad})
    assert e.value.status == zo.ZO_ERR_INVALID


def test_rope_interleaved_must_be_zero_or_one(zo):
    c = zo.zo_rope_cfg.from_dict(PLAIN)
    c.interleaved = 2
    out = np.zeros(32)
    assert zo.lib.zo_rope_frequencies(ctypes.byref(c), out.ctypes.data) == zo.ZO_ERR_INVALID
    assert zo.lib.zo_rope_frequencies(None, out.ctypes.data) == zo.ZO_ERR_INVALID
    assert zo.lib.zo_rope_frequencies(ctypes.byref(zo.zo_rope_cfg.from_dict(PLAIN)), None) == zo.ZO_ERR_INVALID


def test_null_contexts_are_refused(zo):
    c = zo.zo_rope_cfg.from_dict(PLAIN)
    L = zo.lib
    assert L.zo_rope(None, 16, 32, 0, None, ctypes.byref(c), 1, 64, 64, 1, 64) == zo.ZO_ERR_INVALID
    assert L.zo_attention_packed(None, 16, 16, 16, 16, 16, 1, 1, 64, 64, 64, 64, 1, 1, 64, 1.0) == zo.ZO_ERR_INVALID
    assert L.zo_logprobs(None, 16, 0, 1, 8, 8, 16, 16, 16, 0, None, None) == zo.ZO_ERR_INVALID
    assert L.zo_head_logprobs(None, 16, 16, 1, 8, 8, 8, 8, 16, 16, 16, 16, 1 << 20) == zo.ZO_ERR_INVALID


@pytest.mark.parametrize("rows,vocab", [(0, 8), (-1, 8), (1, 0), (1 << 31, 8), (1, 1 << 31)])
def test_head_workspace_refusals(zo, rows, vocab):
    with pytest.raises(zo.ZoError):
        zo.zo_head_logprobs_workspace(rows, vocab)
    n = ctypes.c_int64(-7)
    assert zo.lib.zo_head_logprobs_workspace(rows, vocab, ctypes.byref(n)) == zo.ZO_ERR_INVALID
    assert n.value == -7
    assert zo.lib.zo_head_logprobs_workspace(1, 8, None) == zo.ZO_ERR_INVALID


@pytest.mark.parametrize("vocab", [1, 31, 32, 1000, 50272, 151936])
def test_head_workspace_is_far_below_the_logits(zo, vocab):
    """It grows with the rows, and at large vocabularies stays far below rows x vocab fp32."""
    last = 0
    for rows in (1, 127, 128, 129, 1000, 4096, 20000):
        n = zo.zo_head_logprobs_workspace(rows, vocab)
        assert n > 0 and n % 4 == 0
        if vocab >= 50272:
            assert n < rows * vocab * 4 // 32
        last = max(last, n)
    assert last == n


def _items(cu, total, rows, group, grid):
    """The items that each CTA of the packed attention takes, in its order: (sequence, tile, head group)
    by falling tile number, heads fastest, to and fro over the CTAs, a last partial round from the back."""
    tiles = []
    for s, e in zip(cu[:-1], cu[1:]):
        bad = s < 0 or e < s or e > total
        tiles.append(0 if bad else (e - s + rows - 1) // rows)
    count = sum(tiles) * group
    for cta in range(grid):
        level = max(tiles) - 1
        base = n = 0
        while True:
            back = n % 2 == 1 or (n > 0 and (n + 1) * grid >= count)
            slot = n * grid + (grid - 1 - cta if back else cta)
            n += 1
            while level >= 0 and slot >= base + sum(t > level for t in tiles) * group:
                base += sum(t > level for t in tiles) * group
                level -= 1
            if level < 0:
                break
            index = slot - base
            yield cta, [i for i, t in enumerate(tiles) if t > level][index // group], level, index % group


@pytest.mark.parametrize("lens", [[1], [0], [0, 0, 5], [128, 129, 127], [1] * 300, [0, 1000, 0, 1, 2],
                                  [2000, 3, 700, 700, 128, 256, 257]])
@pytest.mark.parametrize("rows,group", [(128, 3), (256, 2)])
def test_every_tile_of_every_sequence_is_one_item(lens, rows, group):
    cu = [0] + np.cumsum(lens).tolist()
    total = max(1, cu[-1])
    most = ((total + rows - 1) // rows + len(lens)) * group
    for grid in (min(148, most), min(7, most)):
        seen = [(s, t, g) for _, s, t, g in _items(cu, total, rows, group, grid)]
        want = [(s, t, g) for s, n in enumerate(lens) for t in range((n + rows - 1) // rows) for g in range(group)]
        assert sorted(seen) == want


def test_long_items_are_spread():
    """The work (key tiles) of the busiest CTA stays near the mean."""
    lens = [2048, 129, 1777, 64, 1023, 2000, 300, 5]
    cu = [0] + np.cumsum(lens).tolist()
    load = np.zeros(148)
    for cta, _, tile, _ in _items(cu, cu[-1], 128, 6, 148):
        load[cta] += tile + 1
    assert load.max() <= 1.2 * load.mean()


@pytest.mark.parametrize("cu", [[0, 10, 5, 20], [-3, 10, 20], [0, 10, 40], [2 ** 31 - 1, -2 ** 31, 4]])
def test_bad_offsets_have_no_items(cu):
    good = {i for i, (s, e) in enumerate(zip(cu[:-1], cu[1:])) if 0 <= s <= e <= 32}
    assert {s for _, s, _, _ in _items(cu, 32, 128, 1, 4)} == {i for i in good if cu[i + 1] > cu[i]}


def _items_by_distinct_lengths(cu, total, rows, group, grid):
    """_items with a scan of the offsets only where the set of long enough sequences changes: it is the
    same from a number of tiles down to the next one that occurs.  Yields (scans so far, item)."""
    tiles = []
    for s, e in zip(cu[:-1], cu[1:]):
        bad = s < 0 or e < s or e > total
        tiles.append(0 if bad else (e - s + rows - 1) // rows)
    items = sum(tiles) * group

    def scan(level):
        return [i for i, t in enumerate(tiles) if t > level], max((t for t in tiles if t <= level), default=0)

    for cta in range(grid):
        level = max(tiles) - 1
        base = n = 0
        scans = 1
        held, below = scan(level) if level >= 0 else ([], 0)
        while True:
            back = n % 2 == 1 or (n > 0 and (n + 1) * grid >= items)
            slot = n * grid + (grid - 1 - cta if back else cta)
            n += 1
            while level >= 0 and slot >= base + len(held) * group:
                base += len(held) * group
                level -= 1
                if 0 <= level < below:
                    held, below = scan(level)
                    scans += 1
            if level < 0:
                break
            index = slot - base
            yield scans, (cta, held[index // group], level, index % group)


@pytest.mark.parametrize("lens", [[1], [0], [0, 0, 5], [128, 129, 127], [0, 1000, 0, 1, 2], [5000, 0, 0, 0, 1],
                                  [2000, 3, 700, 700, 128, 256, 257], [300 * k for k in range(9)]])
@pytest.mark.parametrize("rows,group", [(128, 3), (256, 1)])
def test_scans_of_distinct_lengths_find_the_same_items(lens, rows, group):
    cu = [0] + np.cumsum(lens).tolist()
    total = max(1, cu[-1])
    distinct = len({(n + rows - 1) // rows for n in lens if n})
    for grid in (1, 7, 148):
        got = list(_items_by_distinct_lengths(cu, total, rows, group, grid))
        assert [i for _, i in got] == list(_items(cu, total, rows, group, grid))
        assert all(s <= distinct for s, _ in got)


@pytest.mark.parametrize("vocab", [1, 33, 1000, 2400, 50272, 151936])
def test_head_workspace_serves_smaller_calls(zo, vocab):
    """A workspace for so many rows (or tokens) is enough for fewer."""
    need = [zo.zo_head_logprobs_workspace(rows, vocab) for rows in range(1, 1300)]
    assert need == sorted(need)
    for rows in (1, 128, 129, 600):
        need = [zo.zo_head_logprobs_workspace(rows, v) for v in range(max(1, vocab - 300), vocab + 300)]
        assert need == sorted(need)


def _calls(zo, torch):
    """The operators with tensors of the right types: name of an argument -> a call with it replaced.  The
    context is closed, so that a call whose types pass is refused by the library without a launch."""
    ctx = type("Closed", (), dict(handle=None, check=staticmethod(lambda st: (_ for _ in ()).throw(zo.ZoError(st, "")))))()
    f32, bf, i32 = (lambda n, d=d: torch.zeros(n, dtype=d) for d in (torch.float32, torch.bfloat16, torch.int32))

    def rope(**k):
        a = dict(dict(x=bf(64), out=bf(64), positions=i32(1)), **k)
        zo.zo_rope(ctx, a["x"], a["out"], a["positions"], PLAIN, 1, 64, 64, 1, 64)

    def attention(**k):
        a = dict(dict(q=bf(64), k=bf(64), v=bf(64), out=bf(64), cu_seqlens=i32(2)), **k)
        zo.zo_attention_packed(ctx, a["q"], a["k"], a["v"], a["out"], a["cu_seqlens"], 1, 1, 64, 64, 64, 64, 1, 1, 64, 1.0)

    def logprobs(**k):
        a = dict(dict(targets=i32(1), logprob=f32(1), entropy=f32(1), top_ids=i32(2), top_logprobs=f32(2)), **k)
        zo.zo_logprobs(ctx, f32(8), 1, 8, 8, a["targets"], a["logprob"], a["entropy"], 2, a["top_ids"], a["top_logprobs"])

    def head(**k):
        a = dict(dict(hidden=bf(8), W=bf(64), targets=i32(1), logprob=f32(1), entropy=f32(1)), **k)
        zo.zo_head_logprobs(ctx, a["hidden"], a["W"], 1, 8, 8, 8, 8, a["targets"], a["logprob"], a["entropy"], 16, 1 << 20)

    return dict(rope=rope, attention=attention, logprobs=logprobs, head=head)


@pytest.mark.parametrize("op,name,wrong", [
    ("rope", "positions", "int64"), ("rope", "out", "float32"), ("rope", "x", "float16"), ("rope", "out", "float16"),
    ("attention", "cu_seqlens", "int64"), ("attention", "q", "float16"), ("attention", "k", "float32"),
    ("attention", "v", "float16"), ("attention", "out", "float32"),
    ("logprobs", "targets", "int64"), ("logprobs", "logprob", "float64"), ("logprobs", "entropy", "bfloat16"),
    ("logprobs", "top_ids", "int64"), ("logprobs", "top_logprobs", "float64"),
    ("head", "hidden", "float16"), ("head", "W", "float32"), ("head", "targets", "int64"),
    ("head", "logprob", "float64"), ("head", "entropy", "float64")])
def test_tensors_of_another_type_are_refused(zo, op, name, wrong):
    """An int64 position would be read as two int32 ones, a double loss written as half of one."""
    torch = pytest.importorskip("torch")
    call = _calls(zo, torch)[op]
    with pytest.raises(zo.ZoError):
        call()                                   # the right types reach the library
    if name != "x":
        with pytest.raises(zo.ZoError):
            call(**{name: 16})                   # and so does a bare address
    with pytest.raises(TypeError, match=name if name != "x" else "float16"):
        call(**{name: torch.zeros(64, dtype=getattr(torch, wrong))})


def test_head_limits_are_those_of_the_header(zo):
    assert zo.zo_head_logprobs_workspace(2 ** 31 - 258, 8) > 0 and zo.zo_head_logprobs_workspace(1, 2 ** 31 - 514) > 0
    for rows, vocab in ((2 ** 31 - 257, 8), (1, 2 ** 31 - 513)):
        with pytest.raises(zo.ZoError):
            zo.zo_head_logprobs_workspace(rows, vocab)
