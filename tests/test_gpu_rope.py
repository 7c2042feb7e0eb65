"""zo_rope against the rotation in 64 bits.

Tolerance per output, for a pair (a, b): the reduced angle is rounded to fp32 (2^-26 of a turn,
9.4e-8 rad), sine and cosine are within one unit in the last place (2^-23 at most) and rounded
once more by the magnitude (2^-24), each output takes three fp32 roundings (2^-24 each): below
6e-7 magnitude (|a| + |b|), plus half a step of bf16 (2^-8 of the value) where that is the type.
The frequencies' own fp64 rounding moves an angle by at most 2^-51 of its value.
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


def reference(zo, x, positions, cfg, heads, hd):
    """(rotated fp64 rows, |a| + |b| of every feature's pair; 0 where only copied)."""
    rot = cfg["rot_dim"]
    f = torch.from_numpy(zo.zo_rope_frequencies(cfg)).cuda()
    t = positions.double()[:, None] * f
    y = x[:, : heads * hd].double().reshape(len(x), heads, hd).clone()
    mag = float(np.float32(cfg.get("magnitude", 1.0)))
    i = torch.arange(rot // 2, device="cuda")
    ia, ib = (2 * i, 2 * i + 1) if cfg.get("interleaved") else (i, i + rot // 2)
    a, b = y[..., ia].clone(), y[..., ib].clone()
    c, s = t.cos()[:, None, :] * mag, t.sin()[:, None, :] * mag
    size = torch.zeros_like(y)
    size[..., ia] = size[..., ib] = (a.abs() + b.abs()) * abs(mag)
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    return y.reshape(len(x), -1), size.reshape(len(x), -1), t.abs().max().item()


def check(zo, out, x, positions, cfg, heads, hd):
    ref, size, far = reference(zo, x, positions, cfg, heads, hd)
    tol = size * (6e-7 + far * 2.0 ** -50)
    if out.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * ref.abs()
    bad = (out.double() - ref).abs() > tol
    assert not bad.any(), (bad.sum().item(), (out.double() - ref).abs().max().item())


def cfg_of(rot, interleaved=False, **more):
    return dict(dict(theta=1.0e6, rot_dim=rot, interleaved=interleaved), **more)


BANDS = dict(scaling="bands", factor=4.0, orig_len=4096.0, band_low=1.0, band_high=32.0, magnitude=1.125)

SHAPES = [  # rows, heads, head_dim, rot_dim
    (1, 40, 128, 128), (1, 1, 2, 2), (7, 3, 64, 64), (300, 24, 128, 128), (257, 5, 64, 32), (33, 2, 80, 44),
    (19, 7, 96, 96), (64, 4, 256, 256), (1000, 1, 256, 130), (5, 300, 64, 16), (2, 9, 100, 100)]


@pytest.mark.parametrize("rows,heads,hd,rot", SHAPES)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rope_matches_the_rotation(zo, ctx, rows, heads, hd, rot, interleaved, dtype):
    g = torch.Generator(device="cuda").manual_seed(rows * 7 + heads + hd + rot)
    x = torch.randn(rows, heads * hd, generator=g, device="cuda").to(TYPES[dtype])
    pos = torch.randint(0, 5000, (rows,), generator=g, device="cuda", dtype=torch.int32)
    cfg = cfg_of(rot, interleaved)
    out = torch.full_like(x, 7.0)
    zo.zo_rope(ctx, x, out, pos, cfg, rows, heads * hd, heads * hd, heads, hd)
    check(zo, out, x, pos, cfg, heads, hd)
    # in place: the same bits
    y = x.clone()
    zo.zo_rope(ctx, y, y, pos, cfg, rows, heads * hd, heads * hd, heads, hd)
    assert torch.equal(y, out)
    # without positions: row r is position r
    zo.zo_rope(ctx, x, out, None, cfg, rows, heads * hd, heads * hd, heads, hd)
    check(zo, out, x, torch.arange(rows, device="cuda", dtype=torch.int32), cfg, heads, hd)
    assert zo.zo_sync(ctx) == 0


@pytest.mark.parametrize("scaling", [dict(scaling="linear", factor=8.0), BANDS, dict(magnitude=-0.5)])
@pytest.mark.parametrize("positions", ["far", "edge"])
def test_rope_scaled_and_far_positions(zo, ctx, scaling, positions):
    heads, hd = 3, 128
    if positions == "far":
        pos = torch.tensor([0, 1, 4095, 131071, 1000000, 99999999], dtype=torch.int32, device="cuda")
    else:
        pos = torch.tensor([-1, -4096, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32, device="cuda")
    x = torch.randn(len(pos), heads * hd, device="cuda")
    cfg = cfg_of(128, **scaling)
    out = torch.empty_like(x)
    zo.zo_rope(ctx, x, out, pos, cfg, len(pos), heads * hd, heads * hd, heads, hd)
    check(zo, out, x, pos, cfg, heads, hd)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("pad_in,pad_out,shift", [(64, 0, 0), (3, 5, 1), (8, 24, 8), (1, 0, 0)])
def test_rope_strides_and_untouched_memory(zo, ctx, dtype, pad_in, pad_out, shift):
    """Rows inside wider ones, from an address off 16 bytes: what lies around is left alone."""
    rows, heads, hd = 37, 5, 64
    w = heads * hd
    x = torch.randn(rows * (w + pad_in) + shift, device="cuda").to(TYPES[dtype])[shift:].view(rows, w + pad_in)
    flat = torch.full((rows * (w + pad_out) + shift + 4,), -3.0, device="cuda", dtype=TYPES[dtype])
    out = flat[shift: shift + rows * (w + pad_out)].view(rows, w + pad_out)
    pos = torch.arange(rows, device="cuda", dtype=torch.int32) * 11
    cfg = cfg_of(48)
    zo.zo_rope(ctx, x, out, pos, cfg, rows, w + pad_in, w + pad_out, heads, hd)
    check(zo, out[:, :w], x, pos, cfg, heads, hd)
    assert torch.all(out[:, w:] == -3.0) and torch.all(flat[:shift] == -3.0) and torch.all(flat[-4:] == -3.0)
    before = x.clone()
    zo.zo_rope(ctx, x, x, pos, cfg, rows, w + pad_in, w + pad_in, heads, hd)
    assert torch.equal(x[:, :w], out[:, :w]) and torch.equal(x[:, w:], before[:, w:])


def test_rope_query_and_key_heads_of_a_fused_projection_as_the_model_rotates(zo, ctx):
    """Non-finite features stay in their own pair."""
    x = torch.randn(4, 2 * 64, device="cuda")
    x[1, 3] = math.inf
    x[2, 70] = math.nan
    out = torch.empty_like(x)
    pos = torch.tensor([5, 6, 7, 8], dtype=torch.int32, device="cuda")
    zo.zo_rope(ctx, x, out, pos, cfg_of(64), 4, 128, 128, 2, 64)
    bad = ~torch.isfinite(out)
    expect = torch.zeros_like(bad)
    expect[1, 3] = expect[1, 35] = expect[2, 70] = expect[2, 102] = True
    assert torch.equal(bad, expect)


def test_rope_more_rows_than_a_grid_dimension(zo, ctx):
    """One row to a block and more of them than 65535 (heads of 256 that are not 16-byte aligned)."""
    rows, hd = 65535 + 700, 256
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(rows, hd + 1, generator=g, device="cuda")
    out = torch.zeros(rows, hd, device="cuda")
    cfg = dict(theta=1.0e4, rot_dim=hd)
    zo.zo_rope(ctx, x, out, None, cfg, rows, hd + 1, hd, 1, hd)
    part = list(range(40)) + list(range(65500, 65600)) + list(range(rows - 40, rows))
    want = torch.zeros(len(part), hd, device="cuda")
    zo.zo_rope(ctx, x[part].contiguous(), want, torch.tensor(part, dtype=torch.int32, device="cuda"), cfg, len(part),
               hd + 1, hd, 1, hd)
    assert torch.equal(out[part], want) and torch.all(out.abs().sum(1) > 0)


def test_rope_on_another_stream_and_replayed(zo):
    """A context on its own stream, its call captured once and replayed on changed inputs."""
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        c = zo.zo_create(torch.zeros(64, device="cuda"), stream=s)
        x = torch.randn(50, 4 * 64, device="cuda")
        pos = torch.arange(50, dtype=torch.int32, device="cuda")
        out = torch.zeros_like(x)
        cfg = cfg_of(64, True)
        zo.zo_rope(c, x, out, pos, cfg, 50, 256, 256, 4, 64)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        zo.zo_rope(c, x, out, pos, cfg, 50, 256, 256, 4, 64)
    for seed in range(3):
        with torch.cuda.stream(s):
            x.copy_(torch.randn(50, 256, device="cuda", generator=torch.Generator("cuda").manual_seed(seed)))
            pos.add_(17)
            g.replay()
        s.synchronize()
        check(zo, out, x, pos, cfg, 4, 64)
    del g
    c.close()


def test_rope_refusals(zo, ctx):
    x = torch.randn(8, 128, device="cuda")
    out = torch.full_like(x, 9.0)
    pos = torch.arange(8, dtype=torch.int32, device="cuda")

    def refused(**k):
        a = dict(x=x, out=out, pos=pos, cfg=cfg_of(64), rows=8, ldx=128, ldo=128, heads=2, hd=64, dtype=None)
        a.update(k)
        with pytest.raises(zo.ZoError) as e:
            zo.zo_rope(ctx, a["x"], a["out"], a["pos"], a["cfg"], a["rows"], a["ldx"], a["ldo"], a["heads"],
                       a["hd"], a["dtype"])
        assert e.value.status == zo.ZO_ERR_INVALID and str(e.value) != "ZO_ERR_INVALID: "

    refused(x=0, dtype=0)
    refused(out=0)
    refused(rows=0)
    refused(rows=1 << 31)
    refused(heads=0)
    refused(heads=65536, ldx=1 << 30, ldo=1 << 30)
    refused(ldx=127)
    refused(ldo=127)
    refused(hd=63)
    refused(hd=258, heads=1)
    refused(dtype=2)
    refused(cfg=cfg_of(65))
    refused(cfg=cfg_of(128))            # more than the head
    refused(cfg=cfg_of(64, theta=0.0))
    refused(x=x.data_ptr() + 2, dtype=0)
    refused(out=x, ldo=256)             # in place with another stride
    with pytest.raises(TypeError):
        zo.zo_rope(ctx, x.half(), out, pos, cfg_of(64), 8, 128, 128, 2, 64)
    torch.cuda.synchronize()
    assert torch.all(out == 9.0)
