"""Gradient norms, clipping and the clipped sum of per-example gradients, against 64-bit forms."""

import math

import pytest
import torch

import synth
from train_ref import BF16, DEV, F32, rnd, within

pytestmark = pytest.mark.gpu

HALF = {torch.bfloat16: BF16, torch.float32: F32}
INF = float("inf")


def flat_list(sizes, dtype, seed=0, gap=0, scale=1.0):
    """(buffer, views of it): tensors one after the other, `gap` elements apart."""
    flat = rnd(sum(sizes) + gap * len(sizes), seed=seed, dtype=dtype, scale=scale)
    at, out = 0, []
    for n in sizes:
        out.append(flat[at:at + n])
        at += n + gap
    return flat, out


def norm64(ts, kind):
    if kind == INF:
        return max((float(t.double().abs().max()) for t in ts if t.numel()), default=0.0)
    return math.sqrt(sum(float(t.double().square().sum()) for t in ts))


LISTS = {
    "one": [1], "none": [], "empty": [0, 5, 0], "short": [1, 2, 3, 7, 8, 9, 15, 17, 31],
    "chunks": [8191, 8192, 8193, 16384, 24577], "many": [3 + i % 50 for i in range(2500)], "large": [3_000_001, 64],
    "adapters": [16 * 896, 16 * 4864] * 30,
}


@pytest.mark.parametrize("kind", [2.0, INF])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("name", LISTS)
def test_norm_and_clip(lib, name, dtype, kind):
    """Squares are summed in f32 over at most 64 chunks' worth a thread (32 elements of each chunk), the rest in f64."""
    flat, ts = flat_list(LISTS[name], dtype, gap=1)
    want = norm64(ts, kind)
    tol = 0.0 if kind == INF else 256 * F32 * want
    assert abs(float(lib.grad_norm(ts, norm_type=kind)) - want) <= tol
    for limit in (0.3 * want + 1e-3, 2 * want + 1.0):
        _, outs = flat_list(LISTS[name], dtype, seed=1, gap=1)
        k = min(1.0, limit / (want + 1e-6))
        got = lib.clip_grad_norm(ts, limit, norm_type=kind, out=outs)
        assert abs(float(got) - want) <= tol
        for o, t in zip(outs, ts):
            ref = t.double() * k
            within(o, ref, (HALF[dtype] + 300 * F32) * ref.abs() + 1e-44)
            if k == 1.0:
                assert torch.equal(o, t)
        # in place, on copies (aligned otherwise, so their squares join in another order): the bits of out
        inplace = [t.clone() for t in ts]
        copies = [torch.empty_like(t) for t in ts]
        got = lib.clip_grad_norm(inplace, limit, norm_type=kind, out=copies)
        assert abs(float(got) - want) <= tol
        assert torch.equal(lib.clip_grad_norm(inplace, limit, norm_type=kind), got)
        assert all(torch.equal(a, b) for a, b in zip(inplace, copies))
    assert lib.poll_status() == 0


def test_neighbours_are_left_alone(lib):
    """In place over views of one buffer, elements between them: they keep their bits."""
    flat, ts = flat_list([5, 8192, 3, 100], torch.bfloat16, gap=3)
    before = flat.clone()
    lib.clip_grad_norm(ts, 1e-3)
    at = 0
    for t in ts:
        assert torch.equal(flat[at + t.numel():at + t.numel() + 3], before[at + t.numel():at + t.numel() + 3])
        at += t.numel() + 3
    assert not torch.equal(flat, before)


def test_overlapping_outputs_are_refused(lib):
    """The norm of a list may see a tensor twice; nothing is written twice."""
    t = rnd(100, dtype=torch.float32)
    want = norm64([t, t], 2.0)
    assert abs(float(lib.grad_norm([t, t])) - want) <= 256 * F32 * want
    before = t.clone()
    for bad in ([t, t], [t, t[50:]], [t[:60], t[59:]]):
        with pytest.raises(ValueError, match="overlap"):
            lib.clip_grad_norm(bad, 1e-3)
    with pytest.raises(ValueError, match="overlap"):
        lib.clip_grad_norm([t, t], 1e-3, out=[before, before])
    g, o = rnd(2, 30), torch.zeros(30, device=DEV)
    with pytest.raises(ValueError, match="overlap"):
        lib.clip_examples([g, g], 1.0, out=[o, o])
    assert torch.equal(t, before)
    a, b = torch.empty_like(t), torch.empty_like(t)
    lib.clip_grad_norm([t, t], 1e-3, out=[a, b])
    assert torch.equal(a, b) and not torch.equal(a, t)


def test_types_and_alignments_mixed(lib):
    """bf16 and f32 in one list; an output at another distance from a 16-byte boundary than its input."""
    b, f = rnd(5000), rnd(5000, seed=1, dtype=torch.float32)
    ts = [b[3:4003], f[1:4002], b[4003:4004], f[4002:]]
    outs = [torch.zeros(4005, dtype=torch.bfloat16, device=DEV)[4:4004],
            torch.zeros(4005, dtype=torch.float32, device=DEV)[2:4003],
            torch.zeros(3, dtype=torch.bfloat16, device=DEV)[2:3], torch.zeros(998, dtype=torch.float32, device=DEV)]
    want = norm64(ts, 2.0)
    got = lib.clip_grad_norm(ts, 2.5, out=outs)
    assert abs(float(got) - want) <= 256 * F32 * want
    for o, t in zip(outs, ts):
        ref = t.double() * (2.5 / (want + 1e-6))
        within(o, ref, (HALF[t.dtype] + 300 * F32) * ref.abs())


@pytest.mark.parametrize("kind", [2.0, INF])
def test_norms_that_are_not_finite(lib, kind):
    t = rnd(20000, dtype=torch.float32)
    t[12345] = float("nan")
    a = t.clone()
    assert math.isnan(float(lib.clip_grad_norm([a], 1.0, norm_type=kind))) and bool(a.isnan().all())
    t[12345] = float("-inf")
    a = t.clone()
    assert float(lib.clip_grad_norm([a], 1.0, norm_type=kind)) == INF
    assert bool(a[12345].isnan()) and int((a == 0).sum()) == 19999
    out = torch.empty_like(t)
    lib.clip_grad_norm([t], INF, norm_type=kind, out=[out])
    assert torch.equal(out, t)
    z = torch.zeros(77, device=DEV)
    assert float(lib.clip_grad_norm([z], 1.0, norm_type=kind)) == 0.0 and not bool(z.any())


def test_the_largest_lists_keep_their_precision(lib):
    """100 million squares of one size and a few large ones."""
    t = torch.full((100_000_001,), 1e-3, dtype=torch.float32, device=DEV)
    t[5] = 30.0
    want = norm64([t], 2.0)
    assert abs(float(lib.grad_norm([t])) - want) <= 256 * F32 * want


def test_a_tensor_beyond_32_bit_offsets(lib):
    """2^31 + 5 elements, and an example's gradients of which the last start past 2^31."""
    t = torch.zeros((1 << 31) + 5, dtype=torch.bfloat16, device=DEV)
    t[-3:] = torch.tensor([3.0, -4.0, 12.0], device=DEV)
    assert float(lib.grad_norm([t])) == 13.0
    lib.clip_grad_norm([t], 6.5)
    within(t[-3:], torch.tensor([1.5, -2.0, 6.0], device=DEV).double(), 2 * BF16 * 6.0)
    del t
    g = torch.zeros(3, 1 << 30, dtype=torch.bfloat16, device=DEV)
    g[:, -1] = torch.tensor([1.0, 2.0, 4.0], device=DEV)
    (s,), sq = lib.clip_examples([g], 2.0)
    assert sq.tolist() == [1.0, 4.0, 16.0] and float(s[-1]) == 5.0 and not bool(s[:-1].any())


def test_lists_are_kept_and_replayed(lib):
    """A list built once serves later calls and a captured one, whose launch keeps its own copy."""
    _, ts = flat_list([4096, 4096, 30], torch.bfloat16)
    _, outs = flat_list([4096, 4096, 30], torch.bfloat16, seed=1)
    kept, out = lib.tensor_list(ts), lib.tensor_list(outs)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        lib.clip_grad_norm(kept, 1.0, out=out)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            norm = lib.clip_grad_norm(kept, 1.0, out=out)
    del kept, out
    for k in range(2):
        torch.cuda.synchronize()
        ts[0].copy_(rnd(4096, seed=30 + k))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in outs]
        want = [torch.empty_like(o) for o in outs]
        assert torch.equal(lib.clip_grad_norm(ts, 1.0, out=want), norm)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


# ------------------------------------------------------------------ per-example gradients

def examples64(ts, limit, scale, sq=None):
    sq = sum(t.double().flatten(1).square().sum(1) for t in ts) if sq is None else sq.double()
    c = torch.clamp(limit / sq.sqrt(), max=1.0)
    shape = lambda t: (-1,) + (1,) * (t.dim() - 1)  # noqa: E731
    return ([scale * (c.view(shape(t)) * t.double()).sum(0) for t in ts], sq,
            [abs(scale) * (c.view(shape(t)) * t.double().abs()).sum(0) for t in ts])


def check_examples(lib, ts, limit, scale=1.0, given=False):
    sums64, sq64, size = examples64(ts, limit, scale)
    n = ts[0].shape[0]
    sums, sq = lib.clip_examples(ts, limit, scale=scale, sq_norms=sq64.float() if given else None)
    within(sq, sq64, (256 * F32 if not given else F32) * sq64 + 1e-45, "sq_norms")
    for a, b, c in zip(sums, sums64, size):
        assert a.dtype == torch.float32
        within(a, b, (n + 300) * F32 * c + 1e-44, "sums")
    return sums, sq


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n", [1, 2, 7, 32, 255, 256, 257, 600])
def test_clipped_sum(lib, n, dtype):
    shapes = [(n, 16, 24), (n, 7), (n, 4104), (n, 1), (n, 3, 5), (n, 8), (n, 12)]
    size = torch.exp(rnd(n, 1, seed=9, dtype=torch.float32))
    ts = [(rnd(*s, seed=i, dtype=torch.float32) * size.view((n,) + (1,) * (len(s) - 1))).to(dtype) for i, s in enumerate(shapes)]
    for given in (False, True):
        check_examples(lib, ts, 60.0, 1.0 / n, given)
    check_examples(lib, ts, 1e9, -2.0)
    check_examples(lib, ts, INF)
    a, b = lib.clip_examples(ts, 60.0), lib.clip_examples(ts, 60.0)
    assert all(torch.equal(p, q) for p, q in zip(a[0], b[0])) and torch.equal(a[1], b[1])


def test_views_and_many_tensors(lib):
    """Per-example blocks at odd places, more tensors than one launch holds."""
    n = 3
    flat = rnd(n * 1100 * 40 + 1)
    ts = [flat[1 + 40 * n * i:1 + 40 * n * (i + 1)].view(n, 40) for i in range(1100)]
    check_examples(lib, ts, 50.0, 0.5)


def test_examples_at_the_edges(lib):
    """An example of zeros keeps its factor of one; one that is not finite makes NaN of what it is added to."""
    ts = [rnd(4, 100), rnd(4, 33, seed=1)]
    ts[0][1] = 0
    ts[1][1] = 0
    check_examples(lib, ts, 2.0)
    ts[0][2, 7] = float("nan")
    sums, sq = lib.clip_examples(ts, 2.0)
    assert bool(sq[2].isnan()) and all(bool(s.isnan().all()) for s in sums)
    ts[0][2, 7] = float("inf")
    sums, sq = lib.clip_examples(ts, 2.0)
    assert float(sq[2]) == INF and bool(sums[0][7].isnan()) and int(sums[0].isnan().sum()) == 1
    empty = [torch.empty(3, 0, dtype=torch.bfloat16, device=DEV), rnd(3, 9)]
    check_examples(lib, empty, 1.0)


def test_of_the_mlps_per_example_gradients(lib):
    """Two MLPs' per-example gradients as the backward gives them, their norms added up: one clipped sum,
    the same with the norms known and computed."""
    n, parts, sq = 4, [], 0
    for seed in (0, 1):
        cfg = synth.MLP_CONFIGS["tiny"].replace(M=128)
        t = {k: v.to(DEV) for k, v in synth.make_mlp_inputs(cfg, seed=seed).items()}
        lin = lambda m: (t["W_" + m], t["A_" + m], t["B_" + m])  # noqa: E731
        _, saved = lib.mlp_forward(t["x"], lin("gate"), lin("up"), lin("down"), cfg.s, cfg.act)
        g = lib.mlp_backward_per_example(t["x"], lin("gate"), lin("up"), lin("down"), cfg.s, cfg.act, saved, t["dy"], n)
        parts += [g[k] for k in ("dA_gate", "dB_gate", "dA_up", "dB_up", "dA_down", "dB_down")]
        sq = sq + g["sq_norms"]
    limit = 0.8 * float(sq.sqrt().median())
    sums64, sq64, size = examples64(parts, limit, 1.0 / n)
    within(sq, sq64, 4000 * F32 * sq64)              # the backward sums a thread's share in one f32 chain
    for known in (sq, None):
        got, norms = lib.clip_examples(parts, limit, sq_norms=known, scale=1.0 / n)
        for a, b, c in zip(got, sums64, size):
            within(a, b, 5000 * F32 * c + 1e-44)
    assert lib.poll_status() == 0
