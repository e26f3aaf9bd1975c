"""Causal attention over packed prompts (packed_gqa_prefill) against its plain
64-bit form, at the lengths, groups and strides where it can go wrong."""
import pytest
import torch

import paged_gqa_decode_03_gb300 as pgd
from step_util import assert_attention, attention, packed_seen

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    yield
    assert pgd.pgd_check_device_error() == 0


def case(lens, Hq, Hkv, D, seed=0, gap=0):
    """gap: rows between the prompts that belong to none (NaN)."""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    T = sum(lens)
    qkv = torch.randn((T, Hq + 2 * Hkv, D), generator=g, device=DEV).half()
    cu = torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device=DEV)
    return dict(q=qkv[:, :Hq], k=qkv[:, Hq:Hq + Hkv], v=qkv[:, Hq + Hkv:], cu=cu, lens=lens,
                scale=D ** -0.5, D=D)


def run(c, dtype=torch.float16, extra=0, **kw):
    out = torch.full((c["q"].shape[0], c["q"].shape[1], c["D"]), 7.0, dtype=dtype, device=DEV)
    pgd.packed_gqa_prefill(out, c["q"], c["k"], c["v"], c["cu"], c["scale"],
                           max(c["lens"], default=0), **kw)
    torch.cuda.synchronize()
    return out


def check(out, c, what, prompts=None):
    at = 0
    for s, n in enumerate(c["lens"]):
        if n and (prompts is None or s in prompts):
            rows = slice(at, at + n)
            ref, A = attention(c["q"][rows], c["k"][rows], c["v"][rows], packed_seen(n), c["scale"])
            assert_attention(out[rows], ref, A, n, c["D"], float(c["v"][rows].abs().max()),
                             f"{what} prompt {s}", c["scale"])
        at += n


LENS = [1, 2, 31, 127, 128, 129, 0, 300, 513, 64]


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Hq,Hkv", [(32, 8), (16, 2), (4, 4), (24, 4), (5, 1), (32, 1), (130, 2)])
def test_shapes(D, Hq, Hkv):
    c = case(LENS, Hq, Hkv, D, seed=D + Hq)
    check(run(c), c, f"D{D} {Hq}/{Hkv}")
    assert pgd.pgd_check_device_error() == 0


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n", [1, 16, 33, 65, 255, 256, 257, 1000, 2049])
def test_one_prompt(D, n):
    c = case([n], 8, 2, D, seed=n)
    check(run(c, dtype=torch.float32), c, f"D{D} n {n}")


@pytest.mark.parametrize("D", [64, 128, 256])
def test_many_prompts(D):
    """Thousands of units, several turns per CTA."""
    g = torch.Generator()
    g.manual_seed(D)
    lens = torch.randint(0, 200, (300,), generator=g).tolist()
    c = case(lens, 16, 4, D, seed=3)
    check(run(c), c, f"D{D}", prompts=range(0, 300, 23))


def test_long_prompt():
    c = case([6001], 8, 2, 128, seed=5)
    check(run(c), c, "long")


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("scale", [-0.07, 0.0, 0.3])
def test_any_scale(D, scale):
    c = case([70, 5, 130, 300], 8, 2, D, seed=8)
    c["scale"] = scale * (128 / D) ** 0.5
    check(run(c), c, f"scale {scale}")


@pytest.mark.parametrize("D", [64, 128, 256])
def test_growing_scores_rescale(D):
    """Keys that grow along the prompt: the maximum moves in every stage."""
    c = case([700], 8, 2, D, seed=9)
    ramp = torch.linspace(0.2, 6.0, 700, device=DEV)[:, None, None]
    c["k"] = (c["q"][:, ::4] * ramp).half().contiguous()
    out = run(c, dtype=torch.float32)
    ref, A = attention(c["q"], c["k"], c["v"], packed_seen(700), c["scale"])
    # scores up to 6 D scale: the score's own rounding (D fp32 additions of
    # sums up to that) enters the weights with factor 2, as in step_util
    grow = 6.0 * D * c["scale"] * D * 2.0 ** -23
    lim = (2.0 ** -11 + 2 * (grow + 2.0 ** -13)) * A + 700 * 2.0 ** -25 * 5 + 1e-6
    assert (abs(out.cpu().double().numpy() - ref) <= lim).all()


@pytest.mark.parametrize("D", [64, 128, 256])
def test_rows_of_no_prompt_stay_and_do_not_leak(D):
    """Rows before, between and behind the prompts hold NaN and infinities."""
    c = case([50, 77, 200, 9, 30], 8, 2, D, seed=11)
    for t in (c["q"], c["k"], c["v"]):
        t[50:127] = float("nan")
        t[327:336] = float("inf")
    starts = [0, 127, 336]
    c2 = dict(c, cu=torch.tensor([0, 50], dtype=torch.int32, device=DEV))
    want = []
    for a, n in zip(starts, (50, 200, 30)):
        ref, A = attention(*(c[x][a:a + n] for x in "qkv"), packed_seen(n), c["scale"])
        want.append((a, n, ref, A))
    # cu_seqlens as pairs: every second "prompt" is one of the NaN stretches
    out = run(c)
    for a, n, ref, A in want:
        assert_attention(out[a:a + n], ref, A, n, D, 6.0, f"D{D} at {a}")
    # one prompt of a longer batch: the rest is not written
    out = torch.full_like(out, 7.0)
    pgd.packed_gqa_prefill(out, c["q"], c["k"], c["v"], c2["cu"], c["scale"], 50)
    torch.cuda.synchronize()
    assert_attention(out[:50], want[0][2], want[0][3], 50, D, 6.0, "first")
    assert (out[50:] == 7.0).all()


def test_strides_outputs_and_workspaces_agree():
    c = case([300, 41, 513], 24, 4, 128, seed=12)
    base = run(c)
    check(base, c, "base")
    flat = dict(c, **{x: c[x].contiguous() for x in "qkv"})
    assert torch.equal(run(flat), base)
    head_major = dict(c, **{x: c[x].transpose(0, 1).contiguous().transpose(0, 1) for x in "qkv"})
    assert torch.equal(run(head_major), base)
    assert torch.equal(run(c, dtype=torch.float32).half(), base)
    need = pgd.pgd_prefill_plan(3, 854, 24, 4, 128)
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    for _ in range(3):
        assert torch.equal(run(c, workspace=ws), base)
    with pytest.raises(pgd.PGDError):
        run(c, workspace=ws[: need - 1])


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
def test_output_on_a_16_byte_border(D, dtype):
    c = case([140, 33], 8, 2, D, seed=14)
    base = run(c, dtype=dtype)
    size = base.element_size()
    flat = torch.full((base.numel() + 32,), 7.0, dtype=dtype, device=DEV)
    out = flat[16 // size: 16 // size + base.numel()].view(base.shape)
    assert out.data_ptr() % 32 == 16
    pgd.packed_gqa_prefill(out, c["q"], c["k"], c["v"], c["cu"], c["scale"], 140)
    torch.cuda.synchronize()
    assert torch.equal(out, base)
    assert (flat[: 16 // size] == 7.0).all() and (flat[16 // size + base.numel():] == 7.0).all()


def test_flags():
    c = case([100, 60, 40], 8, 2, 128, seed=13)
    good = run(c)
    out = torch.full_like(good, 7.0)
    pgd.packed_gqa_prefill(out, c["q"], c["k"], c["v"], c["cu"], c["scale"], 99)   # above max_len
    torch.cuda.synchronize()
    assert pgd.pgd_check_device_error() == pgd.DEVERR_QUERY_LEN
    assert (out[:100] == 7.0).all() and torch.equal(out[100:], good[100:])
    cu = torch.tensor([0, 100, 90, 201], dtype=torch.int32, device=DEV)  # negative; past the rows
    out = torch.full_like(good, 7.0)
    pgd.packed_gqa_prefill(out, c["q"], c["k"], c["v"], cu, c["scale"], 200)
    torch.cuda.synchronize()
    assert pgd.pgd_check_device_error() == pgd.DEVERR_QUERY_LEN
    assert torch.equal(out[:100], good[:100]) and (out[100:] == 7.0).all()
    # nothing to do
    none = c["q"][:0]
    pgd.packed_gqa_prefill(out[:0], none, c["k"][:0], c["v"][:0], c["cu"][:1], c["scale"], 0)
    pgd.packed_gqa_prefill(out, c["q"], c["k"], c["v"], c["cu"][:1], c["scale"], 0)
    torch.cuda.synchronize()


def test_captured_and_replayed_beside_another_call():
    c, d = case([900, 40, 300], 16, 4, 128, seed=4), case([64, 700], 16, 4, 256, seed=5)
    base, other = run(c), run(d)
    out, out2 = torch.zeros_like(base), torch.zeros_like(other)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pgd.packed_gqa_prefill(out, c["q"], c["k"], c["v"], c["cu"], c["scale"], 900)
    side = torch.cuda.Stream()
    for _ in range(4):
        out.zero_()
        out2.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            pgd.packed_gqa_prefill(out2, d["q"], d["k"], d["v"], d["cu"], d["scale"], 700)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, base) and torch.equal(out2, other)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_every_length_beside_prompts_of_nan(D):
    """Prompts of 1 to 140 tokens, a prompt of NaN rows behind each: no weight of
    0 meets them, wherever in a stage the prompt ends."""
    lens = [n for k in range(1, 141) for n in (k, 3)]
    c = case(lens, 4, 2, D, seed=21)
    at = 0
    for s, n in enumerate(lens):
        if s % 2:
            for t in (c["q"], c["k"], c["v"]):
                t[at:at + n] = float("nan")
        at += n
    check(run(c), c, f"D{D}", prompts=set(range(0, len(lens), 2)))


def test_rows_past_32_bit_offsets():
    """q and out of more than 2^31 elements; groups of 128 heads."""
    n, D = 6, 256
    S = (2 ** 31 + 2 ** 24) // (128 * D * n)
    T = S * n
    q = torch.empty((T, 128, D), dtype=torch.float16, device=DEV).normal_()
    k, v = (torch.randn((T, 1, D), device=DEV).half() for _ in range(2))
    cu = torch.arange(S + 1, dtype=torch.int32, device=DEV) * n
    out = torch.full_like(q, 7.0)
    pgd.packed_gqa_prefill(out, q, k, v, cu, D ** -0.5, n)
    torch.cuda.synchronize()
    for s in (0, S // 2, S - 2, S - 1):
        rows = slice(s * n, s * n + n)
        ref, A = attention(q[rows], k[rows], v[rows], packed_seen(n), D ** -0.5)
        assert_attention(out[rows], ref, A, n, D, float(v[rows].abs().max()), f"prompt {s}")
