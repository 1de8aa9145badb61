"""RMS norm with the residual's addition, in bf16 and e4m3, and its gradient, against 64-bit forms."""

import pytest
import torch

from train_ref import BF16, DEV, F32, check_norm, check_norm_grad, norm64, rnd, within

pytestmark = pytest.mark.gpu

# one dim for each width of row the kernels know and the sizes around them
DIMS = [8, 56, 64, 72, 128, 256, 264, 512, 896, 1024, 1032, 2048, 2056, 4096, 4104, 8192, 8200, 16384, 16392, 32768]


def rows(tokens, dim, seed=0):
    """Rows of unlike size."""
    size = torch.exp(2 * rnd(tokens, 1, seed=seed + 9, dtype=torch.float32))
    return (rnd(tokens, dim, seed=seed, dtype=torch.float32) * size).to(torch.bfloat16)


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("dim", DIMS)
def test_rows_of_every_width(lib, dim, fmt):
    for tokens, add, offset in ((1, True, 0.0), (7, False, 1.0), (33, True, 1.0)):
        x, w = rows(tokens, dim), rnd(dim, seed=2, scale=0.3)
        r = rows(tokens, dim, 5) if add else None
        y, s, rstd = lib.rms_norm(x, w, residual=r, offset=offset, format=fmt, training=True)
        check_norm(y, s, rstd, x, w, r, offset=offset)
    assert lib.poll_status() == 0


@pytest.mark.parametrize("dim", DIMS)
def test_gradient_of_every_width(lib, dim):
    for tokens, add, offset in ((1, True, 0.0), (7, False, 1.0), (130, True, 1.0)):
        s, dy, w = rows(tokens, dim), rnd(tokens, dim, seed=3), rnd(dim, seed=2, scale=0.3)
        ds = rnd(tokens, dim, seed=4) if add else None
        rstd = norm64(s, w, 1e-6, 0)[1].float()
        dx, dw = lib.rms_norm_backward(dy, s, w, rstd, offset=offset, ds=ds)
        check_norm_grad(dx, dw, dy, s, w, rstd, offset, ds)
        dx2, none = lib.rms_norm_backward(dy, s, w, rstd, offset=offset, ds=ds, dweight=False)
        assert none is None and torch.equal(dx, dx2)
    assert lib.poll_status() == 0


@pytest.mark.parametrize("tokens", [1, 15, 607, 608, 609, 5000])
def test_gradient_of_the_weight_over_many_rows(lib, tokens):
    """More rows than blocks: a block walks several."""
    for dim in (64, 896, 2056):
        s, dy, w = rows(tokens, dim), rnd(tokens, dim, seed=3), rnd(dim, seed=2)
        rstd = norm64(s, w, 1e-6, 0)[1].float()
        dx, dw = lib.rms_norm_backward(dy, s, w, rstd)
        check_norm_grad(dx, dw, dy, s, w, rstd)
        assert torch.equal(dw, lib.rms_norm_backward(dy, s, w, rstd)[1])


@pytest.mark.parametrize("heads,dim", [(1, 128), (3, 64), (14, 64), (32, 128), (5, 256), (4, 1040)])
def test_views(lib, heads, dim):
    """Heads inside a packed buffer, heads first, every second row; x, the residual and the gradients each
    with strides of their own."""
    t = 21
    packed = rnd(t, 3 * heads * dim)
    views = [packed[:, heads * dim:2 * heads * dim].unflatten(1, (heads, dim)),
             rnd(heads, t, dim, seed=1).transpose(0, 1), rnd(2 * t, heads, dim, seed=2)[::2]]
    w = rnd(dim, seed=3)
    for a, x in enumerate(views):
        r = views[(a + 1) % 3]
        out = torch.full((t, heads, 2 * dim), float("nan"), dtype=torch.bfloat16, device=DEV)
        y, s, rstd = lib.rms_norm(x, w, residual=r, training=True, sum_out=out[..., :dim])
        check_norm(y, s, rstd, x, w, r)
        assert bool(out[..., dim:].isnan().all())
        dx, dw = lib.rms_norm_backward(r, s, w, rstd, ds=views[(a + 2) % 3])
        check_norm_grad(dx, dw, r, s, w, rstd, ds=views[(a + 2) % 3])


def test_sum_in_place(lib):
    """The stream is updated where it is: sum_out the residual, or x; y over a dense x."""
    for dim in (128, 896, 4096):
        x, r, w = rows(40, dim), rows(40, dim, 5), rnd(dim, seed=2)
        want = lib.rms_norm(x, w, residual=r)
        for which in (0, 1):
            a, b = x.clone(), r.clone()
            y, s, _ = lib.rms_norm(a, w, residual=b, sum_out=(a, b)[which])
            assert torch.equal(y, want[0]) and torch.equal((a, b)[which], want[1])
        a = x.clone()
        y = lib.rms_norm(a, w, out=a)[0]
        assert y.data_ptr() == a.data_ptr() and torch.equal(a, lib.rms_norm(x, w)[0])
        rstd = lib.rms_norm(x, w, training=True)[2]
        dx = lib.rms_norm_backward(r, x, w, rstd, ds=want[0])[0]
        for which in (0, 1):
            dy, ds = r.clone(), want[0].clone()
            assert torch.equal(lib.rms_norm_backward(dy, x, w, rstd, ds=ds, dx=(dy, ds)[which])[0], dx)


def test_rows_of_zeros_and_extremes(lib):
    """A row of zeros: rstd is eps's alone, y 0, the scale the least one.  Large rows stay finite, tiny ones
    lose nothing but what eps takes."""
    dim = 896
    x = rows(6, dim)
    x[0] = 0
    x[1] = 3e18 * torch.sign(x[1].float()).to(torch.bfloat16)
    x[2] *= 1e-30
    w = rnd(dim, seed=2)
    for fmt in ("bf16", "fp8"):
        y, s, rstd = lib.rms_norm(x, w, format=fmt, training=True)
        check_norm(y, s, rstd, x, w)
    y, _, rstd = lib.rms_norm(x, w, eps=0.0, training=True)
    assert rstd[0] == float("inf") and bool(y[0].isnan().all())
    codes, scale = lib.rms_norm(x, w, format="fp8")[0]
    assert float(scale[0]) == 2.0 ** -126 and not bool(codes[0].float().any())


@pytest.mark.parametrize("dim", [64, 896, 4096])
def test_what_is_not_finite_stays_in_its_row(lib, dim):
    x = rows(9, dim)
    clean = x.clone()
    x[2, 5] = float("nan")
    x[4, dim - 1] = float("inf")
    x[8, 0] = float("-inf")
    w = rnd(dim, seed=2)
    good = [0, 1, 3, 5, 6, 7]
    y = lib.rms_norm(x, w)[0]
    assert torch.equal(y[good], lib.rms_norm(clean, w)[0][good])
    assert bool(y[2].isnan().all()) and bool(y[4, -1].isnan()) and bool(y[8, 0].isnan())
    (codes, scale), (c0, s0) = lib.rms_norm(x, w, format="fp8")[0], lib.rms_norm(clean, w, format="fp8")[0]
    assert torch.equal(codes[good].view(torch.uint8), c0[good].view(torch.uint8)) and torch.equal(scale[good], s0[good])
    for r in (2, 4, 8):
        assert bool(scale[r].isnan()) and not bool(codes[r].view(torch.uint8).any())


def test_one_row_and_no_rows(lib):
    w = rnd(128, seed=2)
    x = torch.empty(0, 128, dtype=torch.bfloat16, device=DEV)
    y, s, rstd = lib.rms_norm(x, w, training=True)
    assert y.shape == (0, 128) and rstd.shape == (0,)
    dx, dw = lib.rms_norm_backward(x, x, w, rstd)
    assert dx.shape == (0, 128) and not bool(dw.any())
    one = rnd(1, 128)
    check_norm(*lib.rms_norm(one, w, training=True), one, w)


def test_outputs_stay_inside_their_rows(lib):
    """Guard bands around every output."""
    dim, t = 1032, 5
    for fmt, dt in (("bf16", torch.bfloat16), ("fp8", torch.uint8)):
        buf = torch.full((t + 2, dim), 7, dtype=dt, device=DEV)
        out = buf[1:-1] if fmt == "bf16" else buf[1:-1].view(torch.float8_e4m3fn)
        x, w = rows(t, dim), rnd(dim, seed=2)
        lib.rms_norm(x, w, format=fmt, out=out)
        assert bool((buf[0] == 7).all()) and bool((buf[-1] == 7).all()) and not bool((buf[1:-1] == 7).all())


def test_rows_beyond_32_bit_offsets(lib):
    """2.4G elements: the last rows lie past 2^31 elements and 2^32 bytes."""
    t, dim = 600_000, 4096
    x, w = torch.empty(t, dim, dtype=torch.bfloat16, device=DEV), rnd(dim, seed=2)
    x.normal_(generator=torch.Generator(device=DEV).manual_seed(1))
    y, _, rstd = lib.rms_norm(x, w, training=True)
    codes, scale = lib.rms_norm(x, w, format="fp8")[0]
    last = slice(t - 50, t)
    check_norm(y[last], x[last], rstd[last], x[last], w)
    check_norm((codes[last], scale[last]), x[last], rstd[last], x[last], w)
    dx = lib.rms_norm_backward(y, x, w, rstd, dweight=False)[0]
    check_norm_grad(dx[last], None, y[last], x[last], w, rstd[last])


def test_in_a_graph_and_on_another_stream(lib):
    x, r, w, dy = rows(70, 896), rows(70, 896, 5), rnd(896, seed=2), rnd(70, 896, seed=6)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())

    def step():
        y, total, rstd = lib.rms_norm(x, w, residual=r, training=True)
        return y, total, rstd, *lib.rms_norm_backward(dy, total, w, rstd, ds=y)

    with torch.cuda.stream(s):
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            got = step()
    for k in range(2):
        torch.cuda.synchronize()
        x.copy_(rows(70, 896, 20 + k))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, step()):
            assert torch.equal(a, b)
    assert lib.poll_status() == 0


@pytest.mark.parametrize("offset", [0.0, 1.0])
@pytest.mark.parametrize("add", [True, False])
def test_autograd(lib, add, offset):
    """Gradients through loss.backward() are the library's; against differences of the 64-bit form too."""
    from rank_mlp_gb300.autograd import lora_rms_norm
    x, w = rnd(2, 5, 64).requires_grad_(), rnd(64, seed=2).requires_grad_()
    r = rnd(2, 5, 64, seed=3).requires_grad_() if add else None
    out = lora_rms_norm(x, w, r, offset=offset)
    y, s = out if add else (out, x)
    dy, ds = rnd(2, 5, 64, seed=4), rnd(2, 5, 64, seed=5)
    torch.autograd.backward([y, s] if add else [y], [dy, ds] if add else [dy])
    rstd = lib.rms_norm(x.detach().view(10, 64), w.detach(), residual=None if r is None else r.detach().view(10, 64),
                        training=True)[2]
    rows_of = s.detach().reshape(10, 64)
    dx, dw = lib.rms_norm_backward(dy.view(10, 64), rows_of, w.detach(), rstd, offset=offset,
                                   ds=ds.view(10, 64) if add else None)
    assert torch.equal(x.grad.view(10, 64), dx) and torch.equal(w.grad, dw)
    if add:
        assert torch.equal(r.grad, x.grad)
    # differences: <dy, y> + <ds, s> along a direction, from the 64-bit form
    d = rnd(10, 64, seed=8).double()
    f = lambda t: (norm64(rows_of.double() + t * d, w.detach(), 1e-6, offset)[0] * dy.view(10, 64).double()).sum()  # noqa: E731
    want = (f(1e-5) - f(-1e-5)) / 2e-5 + (float((ds.view(10, 64).double() * d).sum()) if add else 0.0)
    size = (dx.double().abs() * d.abs()).sum()
    assert abs(float((dx.double() * d).sum()) - float(want)) <= float(2 * BF16 * size) + 1e-6
    # a frozen weight, and an output that the loss leaves out
    x2, w2 = x.detach().requires_grad_(), w.detach()
    if add:
        y2, s2 = lora_rms_norm(x2, w2, r.detach(), offset=offset)
        s2.backward(ds)
        assert torch.equal(x2.grad, ds)
    else:
        lora_rms_norm(x2, w2, offset=offset).backward(dy)
        assert torch.equal(x2.grad, x.grad)
    heads = rnd(7, 4 * 64).requires_grad_()
    lora_rms_norm(heads.unflatten(1, (4, 64))[:, 1:3], w2).sum().backward()
    assert not bool(heads.grad[:, :64].any()) and bool(heads.grad[:, 64:192].any())
    assert lib.poll_status() == 0


def test_long_sums_keep_their_precision(lib):
    """rstd over the widest rows, all of one sign and size but a few."""
    x = torch.ones(3, 32768, dtype=torch.bfloat16, device=DEV)
    x[1, ::2] = 2 ** -8
    x[2, 17] = 256.0
    rstd = lib.rms_norm(x, torch.ones(32768, dtype=torch.bfloat16, device=DEV), training=True)[2]
    want = norm64(x, x[0], 1e-6, 0)[1]
    within(rstd, want, 64 * F32 * want)
