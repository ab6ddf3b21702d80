"""The gated delta rule on the GPU against its plain 64-bit form, through the public entry points.

Tolerances, relative L2 per tensor.  Operands are cut into bf16 parts that hold all 24 bits of an
fp32 value and every sum is fp32, so fp32 results carry the roundings of a few hundred dependent
fp32 operations, 2^-24 each with random signs: 2e-5 leaves a factor of ten.  bf16 outputs are those
rounded once, at most 2^-9 of each value: 2.5e-3.  fp32 outputs of bf16 inputs are held to the fp32
bound, the inputs being exact in both.
"""
import pytest
import torch

import delta_ref as ref
from gpu_common import say
from mamba_ssd_chunked_amd import ssd

pytestmark = pytest.mark.gpu

TOL = {torch.float32: 2e-5, torch.bfloat16: 2.5e-3}
F32, BF16 = torch.float32, torch.bfloat16
GRADS = ("d_q", "d_k", "d_v", "d_g", "d_beta", "d_init")


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ssd.load_library()


def dev(w):
    return {n: t.cuda() if isinstance(t, torch.Tensor) else t for n, t in w.items()}


def run(w, valid_len=None, d_final=True, back=True):
    """Outputs of the forward and the gradient on inputs w (device), with poisoned workspaces."""
    q, k, v, g, beta, init = (w[n] for n in ("q", "k", "v", "g", "beta", "init"))
    ws = ssd.delta_workspace(q, k, v, False).fill_(0xff)
    y, final = ssd.delta_rule(q, k, v, g, beta, init=init, valid_len=valid_len, ws=ws)
    out = {"y": y, "final": final}
    if back:
        ws = ssd.delta_workspace(q, k, v, True).fill_(0xff)
        out |= ssd.delta_rule_bwd(w["dy"], q, k, v, g, beta, init=init, d_final=w["d_final"] if d_final else None,
                                  valid_len=valid_len, ws=ws)
    torch.cuda.synchronize()
    return out


def expect(w, valid_len=None, d_final=True):
    a = [w[n] for n in ("q", "k", "v", "g", "beta", "init")]
    y, final = ref.delta_rule(*a, valid_len)
    return {"y": y, "final": final} | ref.delta_rule_bwd(w["dy"], *a, w["d_final"] if d_final else None, valid_len)


def check(got, want, label, names=None):
    errs = {n: ref.rel(got[n], want[n]) for n in (names or want)}
    say(label, " ".join(f"{n}={e:.1e}" for n, e in errs.items()))
    for n, e in errs.items():
        assert e <= TOL[got[n].dtype], f"{label}: {n} off by {e:.2e}"


# (b, s, hk, h, p, r): one token, around a chunk, partial chunks, every p and r, shared keys
SHAPES = [(1, 1, 1, 1, 16, 16), (2, 2, 1, 2, 32, 16), (2, 15, 2, 2, 16, 64), (1, 63, 2, 2, 32, 64),
          (2, 64, 1, 3, 64, 128), (1, 65, 2, 4, 16, 32), (1, 129, 2, 2, 128, 16), (2, 200, 1, 4, 64, 64),
          (1, 257, 3, 3, 32, 128), (1, 96, 2, 2, 128, 128), (3, 70, 2, 2, 64, 32), (1, 300, 2, 6, 128, 32),
          (1, 190, 1, 1, 128, 64), (2, 127, 5, 5, 64, 16), (1, 333, 1, 2, 16, 128)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape", SHAPES)
def test_parity(shape, dtype):
    w = ref.delta_inputs(*shape, seed=11 + sum(shape), dtype=dtype)
    say("case", shape, dtype)
    check(run(dev(w)), expect(w), f"{shape} {dtype}")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("init,d_final", [(False, True), (True, False), (False, False)])
def test_without_states(init, d_final, dtype):
    w = ref.delta_inputs(2, 100, 1, 2, 32, 64, seed=21, dtype=dtype)
    if not init:
        w["init"] = None
    say("case init", init, "d_final", d_final, dtype)
    check(run(dev(w), d_final=d_final), expect(w, d_final=d_final), f"init={init} d_final={d_final}")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("r", [16, 128])
@pytest.mark.parametrize("heads,p", [(40, 64), (100, 64), (144, 64), (300, 32), (40, 128)])
def test_many_heads(heads, p, r, dtype):
    """Every split of value columns over workgroups and waves; three heads are compared."""
    w = ref.delta_inputs(1, 70, heads, heads, p, r, seed=31, dtype=dtype)
    say("case heads", heads, p, r, dtype)
    got = run(dev(w))
    pick = [0, heads // 2 + 1, heads - 1]
    cut = {n: t[:, pick] if n in ("init", "d_final") else t[:, :, pick] for n, t in w.items()}
    want = expect(cut)
    got = {n: t[:, pick] if n in ("final", "d_init") else t[:, :, pick] for n, t in got.items()}
    check(got, want, f"heads {heads} p {p} r {r}")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("b,s,h,p,r,lens", [
    (1, 2100, 1, 16, 16, None), (2, 2048, 1, 32, 32, (2048, 2047)), (1, 4160, 2, 128, 64, None),
    (1, 4096, 4, 64, 128, None), (1, 4096, 8, 64, 128, None), (1, 2560, 6, 64, 16, None), (1, 5800, 1, 16, 128, None),
    (5, 2600, 1, 64, 64, (2600, 0, 1, 640, 1300)), (4, 2600, 1, 16, 32, (577, 1152, 1153, 576))])
def test_long_sequences_of_few_heads(b, s, h, p, r, lens, dtype):
    """The chunks in segments side by side: every split, rows that end in, at and before any segment."""
    w = ref.delta_inputs(b, s, h, h, p, r, seed=35 + s, dtype=dtype)
    w["g"] *= 0.05  # the first segments are not forgotten by the last one
    pick = [0, h - 1] if h > 1 else [0]
    cut = {n: t[:, pick] if n in ("init", "d_final") else t[:, :, pick] for n, t in w.items()}
    y, final = ref.delta_rule(*(cut[n] for n in ("q", "k", "v", "g", "beta", "init")), lens)
    if lens:
        for i, n in enumerate(lens):
            for t in ("q", "k", "v", "beta"):
                w[t][i, n:] = float("nan")
    say("case long", b, s, h, p, r, dtype)
    got = run(dev(w), None if lens is None else list(lens), back=False)
    check({"y": got["y"][:, :, pick], "final": got["final"][:, pick]}, {"y": y, "final": final}, f"long {s} {h}")
    for i, n in enumerate(lens or []):
        assert not got["y"][i, n:].any()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("grp", [1, 3])
def test_ragged_rows(grp, dtype):
    """Rows of any length, an empty one and whole empty chunks: padding is never read (NaN there, and
    infinities in the gates), leaves the state, and gives zeros."""
    lens = (150, 0, 1, 64, 65, 200)
    w = ref.delta_inputs(6, 200, 2, 2 * grp, 32, 64, seed=41, dtype=dtype)
    want = expect(w, lens)
    for i, n in enumerate(lens):
        for t in ("q", "k", "v", "dy", "beta"):
            w[t][i, n:] = float("nan")
        w["g"][i, n:] = float("inf")
    say("case ragged", grp, dtype)
    got = run(dev(w), torch.tensor(lens))
    check(got, want, f"ragged {dtype}")
    for i, n in enumerate(lens):
        for t in ("y",) + GRADS[:5]:
            assert not got[t][i, n:].any(), t
    assert torch.equal(got["final"][1].cpu(), w["init"][1])
    assert torch.equal(got["d_init"][1].cpu(), w["d_final"][1])


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_slices_of_one_projection(dtype):
    """q, k and v read in place out of one projection's output, and with the token axis outermost."""
    b, s, hk, h, p, r = 2, 90, 2, 4, 32, 64
    w = dev(ref.delta_inputs(b, s, hk, h, p, r, seed=51, dtype=dtype))
    plain = run(w)
    f = torch.cat([w["q"].flatten(2), w["k"].flatten(2), w["v"].flatten(2)], -1)
    q, k, v = f.split([hk * r, hk * r, h * p], -1)
    say("case slices", dtype)
    got = run({**w, "q": q.unflatten(-1, (hk, r)), "k": k.unflatten(-1, (hk, r)), "v": v.unflatten(-1, (h, p))})
    for n in plain:
        assert torch.equal(got[n], plain[n]), n
    turn = {n: w[n].transpose(0, 1).contiguous().transpose(0, 1) for n in ("q", "k", "v")}
    for n, t in run({**w, **turn}).items():
        assert torch.equal(t, plain[n]), n


def test_one_key_head_read_by_expansion():
    """A key head expanded with stride 0 gives what its copies give."""
    w = dev(ref.delta_inputs(2, 70, 1, 3, 16, 32, seed=52))
    wide = {n: w[n].expand(-1, -1, 3, -1) for n in ("q", "k")}
    say("case expanded")
    got, want = run({**w, **wide}), run({**w, **{n: t.contiguous() for n, t in wide.items()}})
    for n in want:
        assert torch.equal(got[n], want[n]), n


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("kind", ["same_key", "overwrite", "forget", "no_decay", "no_write", "strong_decay"])
def test_hard_gates_and_keys(kind, dtype):
    """Keys that are all alike (the triangular system far from the identity), full overwrites, states
    that are forgotten at once (g = -inf), no decay at all, no writes, and decays that underflow."""
    w = ref.delta_inputs(1, 140, 1, 2, 32, 64, seed=61, dtype=dtype)
    if kind == "same_key":
        w["k"] = w["k"][:, :1].expand(-1, 140, -1, -1).contiguous()
        w["beta"].fill_(0.9)
        w["g"].mul_(0.01)
    elif kind == "overwrite":
        w["beta"].fill_(1.0)
    elif kind == "forget":
        w["g"][:, 5::17] = -float("inf")
        w["g"][:, 64] = -float("inf")
    elif kind == "no_decay":
        w["g"].zero_()
    elif kind == "no_write":
        w["beta"].zero_()
    else:
        w["g"].fill_(-80.0)
    say("case", kind, dtype)
    want, got = expect(w), run(dev(w))
    if kind == "forget":  # exp(-inf) kills every path through g
        assert not got["d_g"][:, 5::17].any() and not got["d_g"][:, 64].any()
    if kind == "strong_decay":  # e^-80 of a state: what is left of d_init and d_g is below fp32's sums
        for n in ("d_g", "d_init"):
            assert (got[n].double().cpu() - want[n]).abs().max() < 1e-30, n
            del want[n]
    check(got, want, kind)


def test_single_token_decay_gradient_is_zero_without_a_state():
    w = dev(ref.delta_inputs(2, 1, 2, 2, 32, 64, seed=71, init=False))
    say("case one token")
    assert not run(w)["d_g"].any()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_gradient_against_differences(dtype):
    """Directional differences of the GPU's own forward.  In fp32 with a step of 2^-7 along directions
    of unit scale: truncation of the third derivative, 2^-14 of it, and rounding of the loss, 1e-6 of
    it over the step: 2e-3 of the derivative's scale.  bf16: differences in the fp32 inputs only."""
    w = dev(ref.delta_inputs(2, 100, 2, 4, 16, 32, seed=81, dtype=dtype))
    got = run(w)
    gen = torch.Generator().manual_seed(82)

    def loss(a):
        o = run(a, back=False)
        return ((o["y"].double() * w["dy"].double()).sum() + (o["final"].double() * w["d_final"].double()).sum()).item()

    names = ("q", "k", "v", "g", "beta", "init") if dtype == F32 else ("init",)
    for n in names:
        d = torch.randn(w[n].shape, generator=gen).cuda()
        step = 2.0 ** -7 if dtype == F32 else 1.0  # linear in the initial state
        diff = (loss({**w, n: w[n] + step * d}) - loss({**w, n: w[n] - step * d})) / (2 * step)
        want = (got["d_" + n].double() * d.double()).sum().item()
        size = (got["d_" + n].double() ** 2).sum().sqrt().item()  # the derivative along a unit direction
        say("differences", n, diff, want, size)
        assert abs(diff - want) <= (2e-3 if dtype == F32 else 1e-2) * max(size, abs(want)), n


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_steps_follow_the_scan(dtype):
    """Prefill then decode: states in any slots of a pool, an idle row, and the outputs of one scan."""
    b, s, n, hk, h, p, r = 3, 90, 10, 2, 4, 64, 32
    w = ref.delta_inputs(b, s + n, hk, h, p, r, seed=91, dtype=dtype)
    want_y, want_final = ref.delta_rule(*(w[x] for x in ("q", "k", "v", "g", "beta", "init")))
    w = dev(w)
    cut = [w[x][:, :s] for x in ("q", "k", "v")] + [w[x][:, :s].contiguous() for x in ("g", "beta")]
    say("case steps", dtype)
    _, final = ssd.delta_rule(*cut, init=w["init"])
    pool = torch.full((7, h, p, r), 9.0, device="cuda")
    slots = torch.tensor([5, 0, 3, -1, 7], dtype=torch.int32, device="cuda")  # two idle rows: < 0, past the pool
    pool[slots[:b].long()] = final
    ys = []
    for t in range(s, s + n):
        tok = [torch.cat([w[x][:, t], w[x][:2, t] * float("nan")]) for x in ("q", "k", "v", "g", "beta")]
        ys.append(ssd.delta_step(*tok, state=pool, slots=slots))
    torch.cuda.synchronize()
    y = torch.stack(ys, 1)
    check({"y": y[:b], "final": pool[slots[:b].long()]}, {"y": want_y[:, s:], "final": want_final}, f"steps {dtype}")
    assert not y[b:].any()
    for idle in (1, 2, 4, 6):
        assert (pool[idle] == 9.0).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("p,r", [(p, r) for p in (16, 32, 64, 128) for r in (16, 32, 64, 128)])
def test_step_shapes(p, r, dtype):
    w = ref.delta_inputs(3, 1, 2, 6, p, r, seed=101 + p + r, dtype=dtype)
    y, final = ref.delta_rule(*(w[x] for x in ("q", "k", "v", "g", "beta", "init")))
    w = dev(w)
    state = w["init"].clone()
    got = ssd.delta_step(*(w[x][:, 0] for x in ("q", "k", "v", "g", "beta")), state=state)
    torch.cuda.synchronize()
    say("case step", p, r, dtype)
    check({"y": got, "final": state}, {"y": y[:, 0], "final": final}, f"step {p} {r}")


def test_empty_problems():
    w = dev(ref.delta_inputs(2, 5, 1, 2, 16, 32, seed=111))
    e = {n: t[:, :0] if n in ("q", "k", "v", "g", "beta", "dy") else t for n, t in w.items()}
    say("case empty")
    got = run(e)
    assert got["y"].shape == (2, 0, 2, 16) and torch.equal(got["final"], w["init"])
    assert torch.equal(got["d_init"], w["d_final"])
    got = run({n: t[:0] for n, t in w.items()})
    assert got["final"].shape == (0, 2, 16, 32)
    none = run({**e, "init": None, "d_final": None})
    assert not none["final"].any() and not none["d_init"].any()
    y = ssd.delta_step(*(w[x][:0, 0] for x in ("q", "k", "v", "g", "beta")), state=w["init"])
    assert y.shape == (0, 2, 16)


def test_bitwise_reproducible_and_on_another_stream():
    w = dev(ref.delta_inputs(2, 200, 2, 4, 64, 128, seed=121, dtype=BF16))
    lens = [200, 77]
    first = run(w, lens)
    say("case streams")
    for _ in range(3):
        for n, t in run(w, lens).items():
            assert torch.equal(t, first[n]), n
    st = torch.cuda.Stream()
    big = torch.randn(4096, 4096, device="cuda")
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        late = w["v"] * 1.0 + 0 * (big @ big)[0, 0].to(BF16)  # ready only once the stream gets there
    y, final = ssd.delta_rule(w["q"], w["k"], late, w["g"], w["beta"], init=w["init"], valid_len=lens, stream=st)
    g = ssd.delta_rule_bwd(w["dy"], w["q"], w["k"], late, w["g"], w["beta"], init=w["init"], d_final=w["d_final"],
                           valid_len=lens, stream=st.cuda_stream)
    st.synchronize()
    for n, t in {"y": y, "final": final, **g}.items():
        assert torch.equal(t, first[n]), n


def test_graph_replay():
    """Prefill, gradient and a decode step in one graph; each replay gives the eager results."""
    w = dev(ref.delta_inputs(2, 130, 2, 4, 32, 64, seed=131, dtype=BF16))
    a = [w[n] for n in ("q", "k", "v", "g", "beta")]
    lens = torch.tensor([130, 40])
    tok = [x[:, 7].contiguous() for x in a]
    io = lambda t: torch.empty_like(t)  # noqa: E731
    y, final, state, ys = io(a[2]), io(w["init"]), io(w["init"]), io(tok[2])
    grads = [io(t) for t in (*a, w["init"])]
    wf, wb = ssd.delta_workspace(*a[:3], False), ssd.delta_workspace(*a[:3], True)

    def steps():
        assert ssd.ssd_delta_fwd(*a, w["init"], lens, y, final, wf) == 0
        assert ssd.ssd_delta_bwd(w["dy"], w["d_final"], *a, w["init"], lens, *grads, wb) == 0
        state.copy_(final)
        assert ssd.ssd_delta_step(*tok, state, None, ys) == 0

    outs = [y, final, state, ys, *grads]
    say("case graph")
    steps()
    torch.cuda.synchronize()
    want = [t.clone() for t in outs]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        steps()
    for it in range(3):
        for t in outs:
            t.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for i, (t, x) in enumerate(zip(outs, want)):
            assert torch.equal(t, x), (it, i)
        steps()
        torch.cuda.synchronize()


def test_offsets_past_32_bits():
    """Batch rows of q, k and v and slots of the state pool more than 2^31 elements apart."""
    b, s, h, p, r = 2, 70, 2, 32, 64
    w = dev(ref.delta_inputs(b, s, h, h, p, r, seed=141, dtype=BF16))
    want = run(w)
    far = 2 ** 31 + 4096
    buf = torch.empty(far + 4 * s * h * r, dtype=BF16, device="cuda")
    views = {}
    for i, n in enumerate(("q", "k", "v")):
        sh = w[n].shape
        views[n] = buf.as_strided(sh, (far, sh[2] * sh[3], sh[3], 1), i * s * h * r)
        views[n].copy_(w[n])
    say("case far rows")
    for n, t in run({**w, **views}).items():
        assert torch.equal(t, want[n]), n
    del buf, views
    nslots = 2 ** 31 // (h * p * r) + 5
    pool = torch.empty(nslots, h, p, r, device="cuda")
    slots = torch.tensor([nslots - 1, 3], dtype=torch.int32, device="cuda")
    pool[slots.long()] = w["init"]
    state = w["init"].clone()
    tok = [w[x][:, 0].contiguous() for x in ("q", "k", "v", "g", "beta")]
    say("case far slots")
    y0, y1 = ssd.delta_step(*tok, state=state), ssd.delta_step(*tok, state=pool, slots=slots)
    torch.cuda.synchronize()
    assert torch.equal(y0, y1) and torch.equal(pool[slots.long()], state)


def test_binding_refusals_on_the_device():
    w = dev(ref.delta_inputs(2, 9, 1, 2, 32, 64, seed=151))
    a = [w[n] for n in ("q", "k", "v", "g", "beta")]
    say("case refusals")
    with pytest.raises(ssd.SsdError, match="valid_len"):
        ssd.delta_rule(*a, valid_len=[10, 1])
    with pytest.raises((ValueError, TypeError)):
        ssd.delta_rule(*a, valid_len=torch.tensor([9, 1], device="cuda"))
    with pytest.raises(ValueError):
        ssd.delta_rule(*a[:3], w["g"][:, :8], w["beta"])
    with pytest.raises(ValueError):
        ssd.delta_rule(*a, init=w["init"][:1])
    with pytest.raises(ValueError, match="last axis"):
        ssd.delta_rule(a[0], a[1], a[2].transpose(2, 3).contiguous().transpose(2, 3), *a[3:])
    with pytest.raises(ssd.SsdError, match="16 bytes"):
        ssd.delta_rule(torch.zeros(2, 9, 1, 66, device="cuda")[..., :64], *a[1:])
    with pytest.raises(ssd.SsdError, match="16"):
        odd = torch.zeros(w["v"].numel() + 1, device="cuda")[1:].view(w["v"].shape)
        ssd.delta_rule(a[0], a[1], odd, *a[3:])
    with pytest.raises(ssd.SsdError, match="workspace"):
        ssd.delta_rule(*a, ws=torch.empty(512, dtype=torch.uint8, device="cuda"))
    tok = [x[:, 0].contiguous() for x in a]
    with pytest.raises(ValueError, match="slots"):
        ssd.delta_step(*tok, state=w["init"], slots=torch.tensor([0, 1], device="cuda"))
    with pytest.raises(ValueError, match="state"):
        ssd.delta_step(*tok, state=w["init"][..., :32].contiguous())
    with pytest.raises(ssd.SsdError, match="slot"):
        ssd.delta_step(*tok, state=w["init"][:1])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("b,s,h,p,r", [(1, 2100, 1, 16, 16), (2, 2600, 2, 64, 64), (1, 4096, 8, 64, 128), (3, 1100, 1, 128, 128)])
def test_long_sequences_are_bitwise_reproducible(b, s, h, p, r, dtype):
    """Segments joined in a fixed order, whatever the workspace held before."""
    w = dev(ref.delta_inputs(b, s, h, h, p, r, seed=161, dtype=dtype))
    a = [w[n] for n in ("q", "k", "v", "g", "beta")]
    say("case long again", b, s, h, p, r, dtype)
    ws = ssd.delta_workspace(*a[:3], False)
    first = None
    for fill in (0xff, 0, 0x3f, 0xff, 0x7b):
        y, final = ssd.delta_rule(*a, init=w["init"], ws=ws.fill_(fill))
        torch.cuda.synchronize()
        first = first or (y, final)
        assert torch.isfinite(final).all()
        assert torch.equal(y, first[0]) and torch.equal(final, first[1])
