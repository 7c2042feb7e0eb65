"""A forward pass that scores packed prompts with the operators together: norm, fused projection, rotary
positions in place, packed attention, output projection with the residual, norm, and the given tokens'
log probabilities from the head.  Each operator is checked on the input that the one before it wrote,
with its own bound:
  projections   K 2^-23 sum_k |a_k b_k| (fp32 sums of exact products) + 2^-8 |ref| where rounded to bf16,
                2^-24 (|x| + |ref|) more where added to the fp32 residual,
  rotation      6e-7 (|a| + |b|) + 2^-8 |ref|,
  attention     1.02 (A (2^-8 + 2^-20 + 2 e) + 2^-8 |ref|), A = sum_j w_j |v_j|, e the scores' error,
  scores        as in the tests of zo_head_logprobs,
and the scores of a prompt are those that it gets by itself, bit for bit."""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

D, H, HK, E, V = 256, 4, 2, 64, 3000
ROPE = dict(theta=1.0e4, rot_dim=E)
LENS = [5, 40, 1, 0, 33, 20]


def weights(seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def t(*shape, scale):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(torch.bfloat16)

    return dict(n1=1 + t(D, scale=0.1), qkv=t((H + 2 * HK) * E, D, scale=D ** -0.5), o=t(D, H * E, scale=(H * E) ** -0.5),
                n2=1 + t(D, scale=0.1), head=t(V, D, scale=0.2))


class Pass:
    """The buffers of one forward pass over up to `total` tokens."""

    def __init__(self, zo, ctx, w, total, n_seqs):
        self.zo, self.ctx, self.w, self.total = zo, ctx, w, total
        bf = dict(dtype=torch.bfloat16, device="cuda")
        self.x = torch.zeros(total, D, device="cuda")
        self.h, self.h2 = torch.zeros(total, D, **bf), torch.zeros(total, D, **bf)
        self.qkv, self.att = torch.zeros(total, (H + 2 * HK) * E, **bf), torch.zeros(total, H * E, **bf)
        self.before, self.x0 = torch.zeros_like(self.qkv), torch.zeros_like(self.x)
        self.positions, self.targets = (torch.zeros(total, dtype=torch.int32, device="cuda") for _ in range(2))
        self.cu = torch.zeros(n_seqs + 1, dtype=torch.int32, device="cuda")
        self.logprob, self.entropy = torch.zeros(total, device="cuda"), torch.zeros(total, device="cuda")
        self.space = torch.zeros(zo.zo_head_logprobs_workspace(total, V), dtype=torch.uint8, device="cuda")

    def fill(self, x, targets, lens):
        n = sum(lens)
        self.x.zero_()
        self.att.zero_()
        self.x[:n] = x
        self.targets.fill_(-1)
        self.targets[:n] = targets
        self.positions[:n] = torch.from_numpy(np.concatenate([np.arange(k) for k in lens]).astype(np.int32)).cuda()
        self.cu.copy_(torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32))

    def run(self):
        zo, c, w, n, ld = self.zo, self.ctx, self.w, self.total, (H + 2 * HK) * E
        self.x0.copy_(self.x)
        zo.zo_rmsnorm(c, self.x, w["n1"], self.h, n, D, 1e-6)
        zo.zo_gemm_bf16(c, self.h, w["qkv"], None, self.qkv, n, ld, D, ld, zo.ZO_EPI_BIAS_BF16)
        self.before.copy_(self.qkv)
        zo.zo_rope(c, self.qkv, self.qkv, self.positions, ROPE, n, ld, ld, H + HK, E)
        zo.zo_attention_packed(c, self.qkv, self.qkv[:, H * E:], self.qkv[:, (H + HK) * E:], self.att, self.cu,
                               self.cu.numel() - 1, n, ld, ld, ld, H * E, H, HK, E, E ** -0.5)
        zo.zo_gemm_bf16(c, self.att, w["o"], None, self.x, n, D, H * E, D, zo.ZO_EPI_RESID_F32)
        zo.zo_rmsnorm(c, self.x, w["n2"], self.h2, n, D, 1e-6)
        zo.zo_head_logprobs(c, self.h2, w["head"], n, V, D, D, D, self.targets, self.logprob, self.entropy, self.space)


def inputs(seed, n):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(n, D, generator=g, device="cuda"),
            torch.randint(0, V, (n,), generator=g, device="cuda", dtype=torch.int32))


@pytest.fixture
def stream():
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        yield s
    s.synchronize()


def test_each_operator_on_the_output_of_the_one_before(zo, stream):
    ctx = zo.zo_create(torch.zeros(64, dtype=torch.bfloat16, device="cuda"), stream=stream)
    n = sum(LENS)
    p = Pass(zo, ctx, weights(), n + 3, len(LENS))
    p.fill(*inputs(1, n), LENS)
    p.run()
    assert zo.zo_sync(ctx) == 0
    h, w = p.h.double(), p.w["qkv"].double()
    ref = h @ w.T
    assert torch.all((p.before.double() - ref).abs() <= D * 2.0 ** -23 * (h.abs() @ w.abs().T) + 2.0 ** -8 * ref.abs())
    # rotation
    t = p.positions.double()[:, None] * torch.from_numpy(zo.zo_rope_frequencies(ROPE)).cuda()
    qk = p.before[:, : (H + HK) * E].double().reshape(-1, H + HK, E)
    a, b = qk[..., : E // 2], qk[..., E // 2:]
    c, s = t.cos()[:, None], t.sin()[:, None]
    ref = torch.cat([a * c - b * s, b * c + a * s], -1).reshape(len(qk), -1)
    size = (a.abs() + b.abs()).repeat(1, 1, 2).reshape(len(qk), -1)
    assert torch.all((p.qkv[:, : (H + HK) * E].double() - ref).abs() <= 6e-7 * size + 2.0 ** -8 * ref.abs())
    assert torch.equal(p.qkv[:, (H + HK) * E:], p.before[:, (H + HK) * E:])
    # attention
    at = 0
    for k in LENS:
        rows = p.qkv[at: at + k].double()
        Q = rows[:, : H * E].reshape(k, H, E).transpose(0, 1)
        K = rows[:, H * E: (H + HK) * E].reshape(k, HK, E).transpose(0, 1).repeat_interleave(H // HK, 0)
        W = rows[:, (H + HK) * E:].reshape(k, HK, E).transpose(0, 1).repeat_interleave(H // HK, 0)
        mask = torch.ones(k, k, dtype=torch.bool, device="cuda").triu(1)
        score = (Q @ K.transpose(1, 2) * E ** -0.5)
        err = 2 * E * 2.0 ** -23 * (Q.abs() @ K.abs().transpose(1, 2) * E ** -0.5) + 2.0 ** -23 * score.abs()
        wgt = torch.softmax(score.masked_fill(mask, -math.inf), -1)
        if k:
            e = err.masked_fill(mask, 0).amax(-1)[..., None]
            ref, A = wgt @ W, wgt @ W.abs()
            got = p.att[at: at + k].double().reshape(k, H, E).transpose(0, 1)
            assert torch.all((got - ref).abs() <= 1.02 * (A * (2.0 ** -8 + 2.0 ** -20 + 2 * e) + 2.0 ** -8 * ref.abs()))
        at += k
    assert torch.all(p.att[n:] == 0)
    # output projection onto the residual
    A, W = p.att.double(), p.w["o"].double()
    ref = p.x0.double() + A @ W.T
    tol = H * E * 2.0 ** -23 * (A.abs() @ W.abs().T) + 2.0 ** -24 * (p.x0.double().abs() + ref.abs())
    assert torch.all((p.x.double() - ref).abs() <= tol)
    # scores
    x = p.h2.double() @ p.w["head"].double().T
    e = D * 2.0 ** -23 * (p.h2.double().abs() @ p.w["head"].double().abs().T).amax(1)
    lsm = torch.log_softmax(x, 1)
    want = torch.where(p.targets >= 0, lsm.gather(1, p.targets.long().clamp(min=0)[:, None])[:, 0], torch.zeros_like(e))
    E0 = (V / 16 + 24) * 2.0 ** -24 + 2.0 ** -21
    gap = x.amax(1) - x.gather(1, p.targets.long().clamp(min=0)[:, None])[:, 0]
    assert torch.all((p.logprob.double() - want).abs() <= 2 * e + E0 + 2.0 ** -25 * gap + 2.0 ** -24 * want.abs())
    assert torch.all(p.logprob[n:] == 0)
    ctx.close()


def test_a_prompt_scores_the_same_packed_and_alone(zo, stream):
    ctx = zo.zo_create(torch.zeros(64, dtype=torch.bfloat16, device="cuda"), stream=stream)
    n, w = sum(LENS), weights()
    x, t = inputs(2, n)
    p = Pass(zo, ctx, w, n, len(LENS))
    p.fill(x, t, LENS)
    p.run()
    at = 0
    for k in LENS:
        if k:
            one = Pass(zo, ctx, w, k, 1)
            one.fill(x[at: at + k], t[at: at + k], [k])
            one.run()
            assert torch.equal(one.logprob, p.logprob[at: at + k]) and torch.equal(one.entropy, p.entropy[at: at + k])
        at += k
    assert zo.zo_sync(ctx) == 0
    ctx.close()


def test_captured_passes_of_two_contexts_side_by_side(zo):
    """Each context has a stream, buffers and a graph of its own; replayed at the same time with prompts
    of other lengths in the same buffers, they give what the calls give one after another."""
    w, total = weights(), 120
    packs = [[100, 7, 13], [1, 1, 90], [0, 64, 0], [40, 40, 40]]
    streams = [torch.cuda.Stream() for _ in range(2)]
    ctxs, passes, graphs = [], [], []
    torch.cuda.synchronize()
    for s in streams:
        with torch.cuda.stream(s):
            c = zo.zo_create(torch.zeros(64, device="cuda"), stream=s)
            p = Pass(zo, c, w, total, 3)
            p.fill(*inputs(0, sum(packs[0])), packs[0])
            p.run()  # once before the capture, as any kernel's first launch sets it up
        s.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            p.run()
        ctxs.append(c)
        passes.append(p)
        graphs.append(g)
    with torch.cuda.stream(streams[0]):
        eager = Pass(zo, ctxs[0], w, total, 3)
    streams[0].synchronize()
    for i, lens in enumerate(packs):
        x, t = inputs(10 + i, sum(lens))
        torch.cuda.synchronize()
        for p, s in zip(passes, streams):
            with torch.cuda.stream(s):
                p.fill(x, t, lens)
        torch.cuda.synchronize()
        for _ in range(3):
            for p, s, g in zip(passes, streams, graphs):
                with torch.cuda.stream(s):
                    p.x[: len(x)] = x
                    p.x[len(x):] = 0
                    g.replay()
        torch.cuda.synchronize()
        with torch.cuda.stream(streams[0]):
            eager.fill(x, t, lens)
            eager.run()
        torch.cuda.synchronize()
        for p in passes:
            assert torch.equal(p.logprob, eager.logprob) and torch.equal(p.entropy, eager.entropy)
            assert torch.equal(p.att, eager.att)
    for c in ctxs:
        assert zo.zo_sync(c) == 0
    del graphs, g
    for c in ctxs:
        c.close()


def test_calls_in_a_row_see_what_the_ones_before_wrote(zo, stream):
    """Kernels may start before their predecessors have ended, and wait for them: long calls one right
    behind another give what they give with a synchronisation between."""
    ctx = zo.zo_create(torch.zeros(64, dtype=torch.bfloat16, device="cuda"), stream=stream)
    n, lens = 6000, [2500, 30, 1470, 2000]
    ld = (H + 2 * HK) * E
    g = torch.Generator(device="cuda").manual_seed(5)
    head = (torch.randn(20000, H * E, generator=g, device="cuda") * 0.1).to(torch.bfloat16)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    space = torch.empty(zo.zo_head_logprobs_workspace(n, 20000), dtype=torch.uint8, device="cuda")
    logits = torch.empty(n, 3000, device="cuda")

    def run(x, t, wait):
        qkv, att = torch.zeros(n, ld, dtype=torch.bfloat16, device="cuda"), torch.zeros(n, H * E, dtype=torch.bfloat16,
                                                                                      device="cuda")
        out = [torch.zeros(n, device="cuda") for _ in range(3)]
        steps = [lambda: zo.zo_rope(ctx, x, qkv, None, ROPE, n, ld, ld, ld // E, E),
                 lambda: zo.zo_attention_packed(ctx, qkv, qkv[:, H * E:], qkv[:, (H + HK) * E:], att, cu, len(lens), n, ld,
                                                ld, ld, H * E, H, HK, E, E ** -0.5),
                 lambda: zo.zo_head_logprobs(ctx, att, head, n, 20000, H * E, H * E, H * E, t, out[0], out[1], space),
                 lambda: zo.zo_rope(ctx, att, att, None, ROPE, n, H * E, H * E, H, E),
                 lambda: logits.zero_(),
                 lambda: zo.zo_gemm_bf16(ctx, att, head, None, logits, n, 3000, H * E, 3000, zo.ZO_EPI_RESID_F32),
                 lambda: zo.zo_logprobs(ctx, logits, n, 3000, 3000, None, None, out[2])]
        for s in steps:
            s()
            if wait:
                stream.synchronize()
        return [qkv, att] + out

    for _ in range(4):
        x = torch.randn(n, ld, generator=g, device="cuda").to(torch.bfloat16)
        t = torch.randint(0, 20000, (n,), generator=g, device="cuda", dtype=torch.int32)
        got, want = run(x, t, False), run(x, t, True)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert zo.zo_sync(ctx) == 0
    ctx.close()


def test_a_loss_pass_behind_an_operator_reads_what_it_wrote(zo, stream):
    """The quadratic's pass streams theta and D as soon as it may start."""
    rows, heads, e = 8192, 16, 64
    m = rows * heads * e
    theta = torch.randn(m, device="cuda")
    ctx = zo.zo_create(theta, stream=stream)
    x = torch.randn(rows, heads * e, device="cuda")
    d = torch.zeros(m, device="cuda")
    losses = torch.zeros(2, dtype=torch.float64, device="cuda")
    for i in range(3):
        for k, wait in enumerate((True, False)):
            d.zero_()
            stream.synchronize()
            zo.zo_rope(ctx, x, d, None, dict(theta=1.0e4, rot_dim=e, magnitude=1.0 + i), rows, heads * e, heads * e, heads, e)
            if wait:
                stream.synchronize()
            zo.zo_quad_loss(ctx, d, losses[k:])
        assert zo.zo_sync(ctx) == 0
        assert losses[0] != 0 and losses[0] == losses[1]
    ctx.close()


@pytest.mark.parametrize("op", ["rope", "attention short", "attention", "logprobs", "head"])
def test_a_launch_that_fails_does_not_fail_the_next_call(zo, stream, op):
    """A stream whose capture has been invalidated (on the host) takes no launch: the call says so, and the
    one after it, with the capture over, does what it does."""
    import ctypes
    cu = ctypes.CDLL("libcuda.so.1")
    n = 300
    bf = dict(dtype=torch.bfloat16, device="cuda")
    ctx = zo.zo_create(torch.zeros(64, **bf), stream=stream)
    x, out, f = torch.randn(n, 64, device="cuda").to(torch.bfloat16), torch.zeros(n, 64, **bf), torch.zeros(n, device="cuda")
    offsets = torch.tensor([0, n] if op == "attention" else [0, 20, n], dtype=torch.int32, device="cuda")
    targets, space = torch.zeros(n, dtype=torch.int32, device="cuda"), torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")

    def call():
        if op == "rope":
            zo.zo_rope(ctx, x, out, None, dict(theta=1.0e4, rot_dim=64), n, 64, 64, 1, 64)
        elif op.startswith("attention"):
            zo.zo_attention_packed(ctx, x, x, x, out, offsets, len(offsets) - 1, n, 64, 64, 64, 64, 1, 1, 64, 0.125)
        elif op == "logprobs":
            zo.zo_logprobs(ctx, x, n, 64, 64, targets, f, None)
        else:
            zo.zo_head_logprobs(ctx, x, x, n, n, 64, 64, 64, targets, f, None, space)

    call()
    assert zo.zo_sync(ctx) == 0
    handle, graph = ctypes.c_void_p(stream.cuda_stream), ctypes.c_void_p()
    assert cu.cuStreamBeginCapture_v2(handle, 2) == 0      # CU_STREAM_CAPTURE_MODE_RELAXED
    assert cu.cuStreamSynchronize(handle) != 0             # not allowed in a capture, which ends it
    with pytest.raises(zo.ZoError) as e:
        call()
    assert e.value.status == zo.ZO_ERR_CUDA
    assert cu.cuStreamEndCapture(handle, ctypes.byref(graph)) != 0
    h, w = torch.ones(8, 64, device="cuda"), torch.ones(64, **bf)
    zo.zo_rmsnorm(ctx, h, w, out, 8, 64, 0.0)
    assert zo.zo_sync(ctx) == 0 and torch.all(out[:8] == 1.0)
    ctx.close()
