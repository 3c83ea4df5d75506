"""linear, grouped_linear and swiglu with their gradients against the formulas
in 64 bits.

Tolerances, with u the half step of the 16-bit type (eps / 2):
  - an output is rounded once: u |value|;
  - a sum of K products on the tensor cores adds at most one truncation of
    2^-23 of the running sum (at most S = sum |a| |b|) per 16 products, and
    one rounding of 2^-24 S per joined part (at most 16 of them) and for the
    bias and the residual: (K / 16 + 10) 2^-23 S;
  - the activations have slopes up to 1.13 and are computed to a few fp32
    ulps: 2^-20 of |z| + |act(z)|;
  - dz = dout act'(z) is rounded to the 16-bit type before the products: u S
    more where there is an activation, and act' is good to 2^-20.
"""
import math

import pytest
import torch

from sparse_moe_layer_gemm_b200 import binding as B

gpu = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16}
ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh"]


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def act64(z, name):
    if name == "relu":
        return torch.relu(z)  # slope 0 at 0 (clamp's is 1)
    if name == "silu":
        return z * torch.sigmoid(z)
    if name == "gelu":
        return z * torch.special.ndtr(z)
    if name == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    return z


def slope64(z, name):
    z = z.detach().clone().requires_grad_(True)
    act64(z, name).sum().backward()
    return z.grad


def normal(gen, dtype, *shape, std=1.0):
    return (torch.randn(*shape, generator=gen, dtype=torch.float32) * std).to(dtype).cuda()


def sum_bound(depth, s):
    return (depth / 16 + 10) * 2.0 ** -23 * s


def close(got, want, bound, what):
    got, want = got.double(), want.double()
    assert torch.isfinite(got).all(), what
    off = (got - want).abs()
    bad = off > bound
    assert not bad.any(), (what, int(bad.sum()), float((off - bound).max()),
                           [tuple(i.tolist()) for i in bad.nonzero()[:4]])


def check_rows(out, x, w, bias, residual, act, preact=None):
    """One group's forward against the formula."""
    u = half_step(out.dtype)
    x, w = x.double(), w.double()
    z, s = x @ w, x.abs() @ w.abs()
    if bias is not None:
        z, s = z + bias.double(), s + bias.double().abs()
    y = act64(z, act)
    want = y if residual is None else y + residual.double()
    err = sum_bound(x.shape[1], s)
    extra = 0.0 if residual is None else 2.0 ** -24 * (y.abs() + residual.double().abs())
    fn = 0.0 if act == "none" else 2.0 ** -20 * (z.abs() + y.abs())
    tiny = torch.finfo(out.dtype).tiny  # subnormal outputs: half the smallest step
    close(out, want, u * want.abs() * 1.01 + 1.2 * err + extra + fn + tiny * u * 2, "out")
    if preact is not None:
        close(preact, z, u * z.abs() * 1.01 + err + tiny * u * 2, "preact")


def check_grads(dx, dw, db, dout, x, w, preact, act):
    """One group's gradients against the formulas."""
    u = half_step(dout.dtype)
    tiny = torch.finfo(dout.dtype).tiny * u * 2
    dz = dout.double()
    dz_err = 0.0
    if act != "none":
        z = preact.double()
        dz = dz * slope64(z, act)
        dz_err = u + 2.0 ** -20
    slack = 2.0 ** -20 * dout.double().abs() if act != "none" else 0 * dout.double()
    slack = slack + (tiny if act != "none" else 0)
    if dx is not None:
        want, s = dz @ w.double().t(), dz.abs() @ w.double().abs().t()
        more = slack @ w.double().abs().t()
        close(dx, want, u * want.abs() * 1.01 + sum_bound(dz.shape[1], s) + dz_err * s + more + tiny,
              "dx")
    if dw is not None:
        want, s = x.double().t() @ dz, x.double().abs().t() @ dz.abs()
        more = x.double().abs().t() @ slack
        close(dw, want, u * want.abs() * 1.01 + sum_bound(max(1, dz.shape[0]), s) + dz_err * s
              + more + tiny, "dw")
    if db is not None:
        want, s = dz.sum(0), dz.abs().sum(0)
        # fp32 additions: at most one rounding of 2^-24 S per row
        close(db, want, u * want.abs() * 1.01 + (dz.shape[0] + 8) * 2.0 ** -24 * s + slack.sum(0)
              + tiny, "db")


def tiles_of(x, w, offsets=None, residual=None, act="none", dout=None):
    """The tiles that the product takes with a new output, and dx and dw if there
    is a dout, as tuples (pairs, rows, accumulators, split, slots, slot_steps)."""
    lib, (rows, k), n = B.load_library(), x.shape, w.shape[-1]
    G = 0 if offsets is None else w.shape[0]
    cfg = B.moe_linear_config_t(rows, k, n, G, B.MOE_BF16, B.ACTIVATIONS[act])
    ld = lambda c: c if rows > 1 else (c + 7) // 8 * 8
    off = None if offsets is None else offsets.data_ptr()
    wide = w.stride(0) if G > 1 else 0
    new, more = torch.empty(rows, n, dtype=x.dtype, device="cuda"), torch.empty_like(x)
    got = [B.moe_linear_tiles_t() for _ in range(3)]
    a = B.moe_linear_args_t(x.data_ptr(), ld(k), off, w.data_ptr(), n, wide, None,
                            None if residual is None else residual.data_ptr(), ld(n),
                            new.data_ptr(), ld(n), None, 0)
    assert lib.moe_linear_tiles(cfg, a, got[0]) == B.MOE_OK
    if dout is not None:
        dw = torch.empty_like(w)
        pre = None if act == "none" else new.data_ptr()
        g = B.moe_linear_grads_t(dout.data_ptr(), ld(n), x.data_ptr(), ld(k), off, w.data_ptr(), n,
                                 wide, pre, ld(n), more.data_ptr(), ld(k), dw.data_ptr(), None)
        assert lib.moe_linear_backward_tiles(cfg, g, got[1], got[2]) == B.MOE_OK
    return [tuple(getattr(t, f) for f, _ in t._fields_) for t in got]


# ----------------------------------------------------------------- linear
SHAPES = [(1, 64, 128), (1, 4096, 256), (2, 8, 8), (5, 1, 1), (16, 130, 264), (17, 64, 200),
          (33, 1000, 72), (64, 512, 1280), (77, 110, 77), (128, 256, 128), (129, 257, 129),
          (300, 640, 384), (1000, 72, 520), (2049, 320, 640)]


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("rows,k,n", SHAPES)
def test_linear_plain(rows, k, n, dtype):
    gen = torch.Generator().manual_seed(rows * 7 + k + n)
    x, w = normal(gen, DT[dtype], rows, k), normal(gen, DT[dtype], k, n, std=k ** -0.5)
    check_rows(B.linear(x, w), x, w, None, None, "none")


@gpu
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("rows,k,n", [(1, 256, 300), (40, 128, 77), (260, 200, 264)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_linear_epilogue(rows, k, n, act, dtype):
    gen = torch.Generator().manual_seed(rows + k + n)
    x, w = normal(gen, DT[dtype], rows, k, std=2.0), normal(gen, DT[dtype], k, n, std=k ** -0.5)
    bias, res = normal(gen, DT[dtype], n), normal(gen, DT[dtype], rows, n)
    pre = torch.empty(rows, n, dtype=x.dtype, device="cuda")
    out = B.linear(x, w, bias, residual=res, activation=act, preact=pre)
    check_rows(out, x, w, bias, res, act, pre)


@gpu
def test_linear_residual_in_place():
    gen = torch.Generator().manual_seed(1)
    x, w = normal(gen, torch.bfloat16, 70, 128), normal(gen, torch.bfloat16, 128, 200, std=0.1)
    res = normal(gen, torch.bfloat16, 70, 200)
    buf = res.clone()
    assert B.linear(x, w, residual=buf, out=buf) is buf
    check_rows(buf, x, w, None, res, "none")


@gpu
@pytest.mark.parametrize("rows", [3, 200])
def test_linear_strides_and_alignment(rows):
    """Slices of larger tensors: aligned strides, odd strides, odd bases; what
    lies around the outputs stays as it was."""
    gen = torch.Generator().manual_seed(rows)
    K, N = 96, 136
    for xs, ws, os_ in ((8, 8, 8), (1, 8, 4), (8, 3, 1), (5, 5, 5)):
        x = normal(gen, torch.bfloat16, rows, K + 2 * xs)[:, xs:xs + K]
        w = normal(gen, torch.bfloat16, K, N + 2 * ws, std=0.1)[:, ws:ws + N]
        wide = torch.full((rows + 2, N + 2 * os_), 7.0, dtype=torch.bfloat16, device="cuda")
        out = wide[1:1 + rows, os_:os_ + N]
        B.linear(x, w, out=out)
        check_rows(out, x, w, None, None, "none")
        edge = wide.clone()
        edge[1:1 + rows, os_:os_ + N] = 7.0
        assert (edge == 7.0).all()


@gpu
@pytest.mark.parametrize("act", ["none", "silu"])
@pytest.mark.parametrize("rows,k,n", SHAPES)
def test_linear_backward(rows, k, n, act):
    gen = torch.Generator().manual_seed(rows + 3 * k + n)
    dt = torch.bfloat16 if (rows + k) % 2 else torch.float16
    x, w = normal(gen, dt, rows, k), normal(gen, dt, k, n, std=k ** -0.5)
    dout = normal(gen, dt, rows, n)
    pre = normal(gen, dt, rows, n, std=2.0) if act != "none" else None
    dx, dw, db = B.linear_backward(dout, x, w, preact=pre, activation=act)
    check_grads(dx, dw, db, dout, x, w, pre, act)


@gpu
@pytest.mark.parametrize("act", ACTS)
def test_linear_backward_parts(act):
    """Each gradient alone equals the one computed with the others, bit for bit."""
    gen = torch.Generator().manual_seed(5)
    x, w = normal(gen, torch.bfloat16, 90, 72), normal(gen, torch.bfloat16, 72, 99)
    dout = normal(gen, torch.bfloat16, 90, 99)
    pre = normal(gen, torch.bfloat16, 90, 99, std=3.0) if act != "none" else None
    whole = B.linear_backward(dout, x, w, preact=pre, activation=act)
    check_grads(*whole, dout, x, w, pre, act)
    for i in range(3):
        need = dict(need_dx=i == 0, need_dw=i == 1, need_db=i == 2)
        part = B.linear_backward(dout, x if i == 1 else None, w, preact=pre, activation=act, **need)
        assert [p is None for p in part] == [j != i for j in range(3)]
        assert torch.equal(part[i], whole[i])


@gpu
def test_slopes_at_zero_and_far_out():
    """relu's slope at 0 is 0; far from 0 every slope is 0 or 1, without NaN."""
    z = torch.tensor([[0.0, -0.0, 300.0, -300.0, 6e4, -6e4, 1e30, -1e30]],
                     dtype=torch.bfloat16, device="cuda")
    one, eye = torch.ones_like(z), torch.eye(8, dtype=z.dtype, device="cuda")
    for act, at0 in (("relu", 0.0), ("silu", 0.5), ("gelu", 0.5), ("gelu_tanh", 0.5)):
        dx, _, db = B.linear_backward(one, None, eye, preact=z, activation=act, need_dw=False)
        want = [at0, at0, 1.0, 0.0, 1.0, 0.0, 1.0, 0.0]
        assert dx[0].tolist() == want and db.tolist() == want, act
        x = torch.zeros(1, 8, dtype=z.dtype, device="cuda")
        out = B.linear(x, eye, z[0].contiguous(), activation=act)
        keep = torch.where(z > 0, z, torch.zeros_like(z))
        assert torch.equal(out, keep), act


@gpu
@pytest.mark.parametrize("act,at", [("silu", 2.4), ("gelu", 1.414), ("gelu_tanh", 1.414)])
@pytest.mark.parametrize("rows,k,n", [(3, 40, 24), (130, 72, 99), (300, 2056, 264)])
def test_fp16_gradients_of_large_values(rows, k, n, act, at):
    """dz = dout act'(z) passes fp16's largest value (slopes reach 1.13) where dx,
    dw and db do not."""
    gen = torch.Generator().manual_seed(rows)
    dt = torch.float16
    dout = torch.full((rows, n), 65504.0, dtype=dt, device="cuda")
    dout[:, ::2] *= -1
    pre = torch.full((rows, n), at, dtype=dt, device="cuda")
    x, w = normal(gen, dt, rows, k, std=2.0 ** -10), normal(gen, dt, k, n, std=2.0 ** -10)
    assert float((dout.double() * slope64(pre.double(), act)).abs().max()) > 65504
    dx, dw, _ = B.linear_backward(dout, x, w, preact=pre, activation=act, need_db=False)
    check_grads(dx, dw, None, dout, x, w, pre, act)
    off = offsets_of([rows - 2, 0, 2])
    dx, dw, _ = B.grouped_linear_backward(dout, x, off, w.expand(3, k, n).contiguous(),
                                          preact=pre, activation=act, need_db=False)
    for g, (a, b) in enumerate(((0, rows - 2), (0, 0), (rows - 2, rows))):
        if a < b:
            check_grads(dx[a:b], dw[g], None, dout[a:b], x[a:b], w, pre[a:b], act)


@gpu
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_fp16_gradients_of_small_values(act):
    """Gradients around fp16's smallest: dz keeps steps of 2^-23, half of one off
    at most, whatever many rows of it add up to."""
    gen = torch.Generator().manual_seed(4)
    dt, rows, k, n = torch.float16, 500, 72, 136
    dout = normal(gen, dt, rows, n, std=3e-7)
    pre, x = normal(gen, dt, rows, n, std=2.0), normal(gen, dt, rows, k, std=30.0)
    w = normal(gen, dt, k, n, std=30.0)
    grads = B.linear_backward(dout, x, w, preact=pre, activation=act)
    check_grads(*grads, dout, x, w, pre, act)


@gpu
def test_offsets_past_32_bits():
    """Row strides that take the last rows more than 2^32 elements away."""
    gen = torch.Generator().manual_seed(9)
    rows, K, N, ld = 2100, 64, 72, (1 << 21) + 64
    big = torch.empty(rows, ld, dtype=torch.bfloat16, device="cuda")  # 8.8 GB
    x, res, dout = big[:, :K], big[:, 128:128 + N], big[:, 256:256 + N]
    out, dx = big[:, 512:512 + N], big[:, 1024:1024 + K]
    x.copy_(normal(gen, torch.bfloat16, rows, K))
    res.copy_(normal(gen, torch.bfloat16, rows, N))
    dout.copy_(normal(gen, torch.bfloat16, rows, N))
    w = normal(gen, torch.bfloat16, K, N, std=0.1)
    for lo, hi in ((0, rows), (rows - 3, rows)):  # CTA pairs or not, split or not
        B.linear(x[lo:hi], w, residual=res[lo:hi], activation="silu", out=out[lo:hi])
        check_rows(out[lo:hi], x[lo:hi], w, None, res[lo:hi], "silu")
        _, dw, db = B.linear_backward(dout[lo:hi], x[lo:hi], w, preact=res[lo:hi],
                                      activation="silu", dx=dx[lo:hi])
        check_grads(dx[lo:hi], dw, db, dout[lo:hi], x[lo:hi], w, res[lo:hi], "silu")
    h = big[:, 2048:2048 + N]
    B.swiglu(res, dout, out=h)
    assert torch.equal(h, B.swiglu(res.contiguous(), dout.contiguous()))


@gpu
def test_linear_backward_strides():
    gen = torch.Generator().manual_seed(6)
    for s in (8, 3):
        x = normal(gen, torch.bfloat16, 50, 64 + s)[:, s:]
        w = normal(gen, torch.bfloat16, 64, 80 + s)[:, s:]
        dout = normal(gen, torch.bfloat16, 50, 80 + s)[:, s:]
        pre = normal(gen, torch.bfloat16, 50, 80 + s)[:, s:]
        for act, p in (("none", None), ("gelu", pre)):
            dx, dw, db = B.linear_backward(dout, x, w, preact=p, activation=act)
            check_grads(dx, dw, db, dout, x, w, p, act)


@gpu
@pytest.mark.parametrize("act", ACTS)
def test_gradients_against_differences(act):
    """The gradients along random directions against central differences of
    the formula in 64 bits (their own error, about (1e-4)^2, is far below the
    bound of the 16-bit gradients)."""
    gen = torch.Generator().manual_seed(8)
    x, w = normal(gen, torch.float16, 20, 48), normal(gen, torch.float16, 48, 40, std=0.2)
    bias, dout = normal(gen, torch.float16, 40), normal(gen, torch.float16, 20, 40)
    pre = torch.empty(20, 40, dtype=torch.float16, device="cuda")
    B.linear(x, w, bias, activation=act, preact=pre)
    if act == "relu":  # differences across the kink say nothing
        dout = dout * (pre.abs() > 0.01)
    dx, dw, db = B.linear_backward(dout, x, w, preact=None if act == "none" else pre,
                                   activation=act)

    def loss(a, b, c):
        return (dout.double() * act64(a @ b + c, act)).sum()

    at = [t.double() for t in (x, w, bias)]
    for i, grad in enumerate((dx, dw, db)):
        v = torch.randn(at[i].shape, generator=gen, dtype=torch.float64).cuda()
        h = 1e-4
        up, dn = list(at), list(at)
        up[i], dn[i] = at[i] + h * v, at[i] - h * v
        want = (loss(*up) - loss(*dn)) / (2 * h)
        got = (grad.double() * v).sum()
        # each gradient element: u of itself, and u of dz and of z's rounding
        # (slopes change by at most 1.1 |dz/dz'| per unit of z) in its sums
        u = half_step(torch.float16)
        z = (at[0] @ at[1] + at[2]).abs()
        dzb = dout.double().abs() * (1.13 + 1.1 * z)
        s = (dzb @ at[1].abs().t(), at[0].abs().t() @ dzb, dzb.sum(0))[i]
        assert abs(float(got - want)) <= float((2 * u * s * v.abs()).sum()) + 1e-6


# large enough for CTA pairs: whole and ragged 256 x 256 tiles, odd depths
LARGE = [(2048, 512, 4096), (2500, 1000, 2312), (4111, 136, 1800), (1024, 4096, 2048),
         (1500, 3016, 2600)]


@gpu
@pytest.mark.parametrize("act", ["none", "silu"])
@pytest.mark.parametrize("rows,k,n", LARGE)
def test_linear_large(rows, k, n, act):
    gen = torch.Generator().manual_seed(rows + k)
    dt = torch.float16 if rows % 2 else torch.bfloat16
    x, w = normal(gen, dt, rows, k), normal(gen, dt, k, n, std=k ** -0.5)
    bias, res = normal(gen, dt, n), normal(gen, dt, rows, n)
    pre = torch.empty(rows, n, dtype=dt, device="cuda")
    out = B.linear(x, w, bias, residual=res, activation=act, preact=pre)
    check_rows(out, x, w, bias, res, act, pre)
    dout = normal(gen, dt, rows, n)
    grads = B.linear_backward(dout, x, w, preact=None if act == "none" else pre, activation=act)
    check_grads(*grads, dout, x, w, pre, act)


# tiles of two accumulators where nothing follows the product but a bias
TWO = [(2600, 2600, 2600), (4000, 4104, 1288), (2700, 2312, 2601), (1100, 4096, 4096),
       (2049, 1288, 5000)]


@gpu
@pytest.mark.parametrize("act", ["none", "silu"])
@pytest.mark.parametrize("rows,k,n", TWO)
def test_two_accumulators(rows, k, n, act):
    gen = torch.Generator().manual_seed(rows + n)
    dt = torch.float16 if rows % 4 else torch.bfloat16
    x, w = normal(gen, dt, rows, k), normal(gen, dt, k, n, std=k ** -0.5)
    bias, dout = normal(gen, dt, n), normal(gen, dt, rows, n)
    pre = normal(gen, dt, rows, n) if act != "none" else None
    assert 2 in [t[2] for t in tiles_of(x, w, act=act, dout=dout)]
    out = B.linear(x, w, bias)
    check_rows(out, x, w, bias, None, "none")
    grads = B.linear_backward(dout, x, w, preact=pre, activation=act)
    check_grads(*grads, dout, x, w, pre, act)
    again = B.linear_backward(dout, x, w, preact=pre, activation=act)
    assert torch.equal(out, B.linear(x, w, bias))
    assert all(torch.equal(a, b) for a, b in zip(grads, again))
    assert B.linear_device_error() == 0


@gpu
@pytest.mark.parametrize("rows,k,n", TWO + [(4096, 4096, 4096), (4096, 4096, 1280)])
def test_one_accumulator_below_an_epilogue(rows, k, n):
    """Tiles of two accumulators have no code for more than a bias."""
    x, w = (torch.empty(s, dtype=torch.bfloat16, device="cuda") for s in ((rows, k), (k, n)))
    assert tiles_of(x, w, residual=x.new_empty(rows, n))[0][2] == 1
    for act in ACTS[1:]:
        assert tiles_of(x, w, act=act)[0][2] == 1


@gpu
@pytest.mark.parametrize("sizes,k,n", [([5000, 300, 70], 2600, 2600), ([3000, 0, 1, 900], 4104, 2312),
                                       ([0, 2500, 131, 2469], 2600, 2600)])
def test_grouped_two_accumulators(sizes, k, n):
    """Tiles of two accumulators in ragged groups, shorter ones than a slot among
    them; the rows around the groups hold NaN."""
    gen = torch.Generator().manual_seed(n)
    G, first, behind = len(sizes), 7, 40
    rows = first + sum(sizes) + behind
    x, dout = normal(gen, torch.bfloat16, rows, k), normal(gen, torch.bfloat16, rows, n)
    w, bias = normal(gen, torch.bfloat16, G, k, n, std=k ** -0.5), normal(gen, torch.bfloat16, G, n)
    for t in (x, dout):
        t[:first] = math.nan
        t[rows - behind:] = math.inf
    off = offsets_of(sizes, first)
    assert 2 in [t[2] for t in tiles_of(x, w, off, dout=dout)]
    out = torch.full((rows, n), 3.0, dtype=x.dtype, device="cuda")
    dx = torch.full((rows, k), 3.0, dtype=x.dtype, device="cuda")
    B.grouped_linear(x, off, w, bias, out=out)
    _, dw, db = B.grouped_linear_backward(dout, x, off, w, dx=dx)
    for t in (out, dx):
        assert (t[:first] == 3).all() and (t[rows - behind:] == 3).all()
    o = off.tolist()
    for g in range(G):
        a, b = o[g], o[g + 1]
        if a == b:
            assert (dw[g] == 0).all() and (db[g] == 0).all()
            continue
        check_rows(out[a:b], x[a:b], w[g], bias[g], None, "none")
        check_grads(dx[a:b], dw[g], db[g], dout[a:b], x[a:b], w[g], None, "none")
    assert B.linear_device_error() == 0


# few tiles and a long contraction: clusters of CTAs or of CTA pairs share tiles
SHARED = [(7, 4096, 640), (16, 8192, 128), (40, 2056, 1111), (130, 4096, 512), (250, 4096, 4096),
          (384, 3000, 4096), (510, 4096, 1280), (700, 4104, 1288), (500, 4001, 515)]


@gpu
@pytest.mark.parametrize("act", ["none", "gelu"])
@pytest.mark.parametrize("rows,k,n", SHARED)
def test_linear_shared_tiles(rows, k, n, act):
    gen = torch.Generator().manual_seed(rows)
    dt = torch.float16 if rows % 2 else torch.bfloat16
    x, w = normal(gen, dt, rows, k), normal(gen, dt, k, n, std=k ** -0.5)
    bias, res = normal(gen, dt, n), normal(gen, dt, rows, n)
    pre = torch.empty(rows, n, dtype=dt, device="cuda")
    kw = dict(residual=res, activation=act)
    out = B.linear(x, w, bias, preact=pre, **kw)
    check_rows(out, x, w, bias, res, act, pre)
    plain = B.linear(x, w)
    check_rows(plain, x, w, None, None, "none")
    dout = normal(gen, dt, rows, n)
    bkw = dict(preact=None if act == "none" else pre, activation=act)
    grads = B.linear_backward(dout, x, w, **bkw)
    check_grads(*grads, dout, x, w, pre, act)
    for _ in range(3):  # the partials meet in one order
        assert torch.equal(out, B.linear(x, w, bias, **kw)) and torch.equal(plain, B.linear(x, w))
        assert all(torch.equal(a, b) for a, b in zip(grads, B.linear_backward(dout, x, w, **bkw)))
    inplace = res.clone()
    B.linear(x, w, bias, residual=inplace, activation=act, out=inplace)
    assert torch.equal(inplace, out)
    assert B.linear_device_error() == 0


@gpu
@pytest.mark.parametrize("sizes,k,n", [([100, 0, 37], 4096, 256), ([3, 1], 4096, 520),
                                       ([260, 130, 0, 9], 2048, 384), ([1, 0, 0], 8192, 72)])
def test_grouped_shared_tiles(sizes, k, n):
    """Shared tiles of ragged groups between rows that hold NaN."""
    gen = torch.Generator().manual_seed(k + n)
    G, first, behind = len(sizes), 3, 21
    rows = first + sum(sizes) + behind
    x, dout = normal(gen, torch.bfloat16, rows, k), normal(gen, torch.bfloat16, rows, n)
    w, bias = normal(gen, torch.bfloat16, G, k, n, std=k ** -0.5), normal(gen, torch.bfloat16, G, n)
    for t in (x, dout):
        t[:first] = math.nan
        t[rows - behind:] = math.inf
    off = offsets_of(sizes, first)
    out = torch.full((rows, n), 3.0, dtype=x.dtype, device="cuda")
    dx = torch.full((rows, k), 3.0, dtype=x.dtype, device="cuda")
    B.grouped_linear(x, off, w, bias, activation="silu", out=out)
    _, dw, db = B.grouped_linear_backward(dout, x, off, w, dx=dx)
    for t in (out, dx):
        assert (t[:first] == 3).all() and (t[rows - behind:] == 3).all()
    o = off.tolist()
    for g in range(G):
        a, b = o[g], o[g + 1]
        if a == b:
            assert (dw[g] == 0).all() and (db[g] == 0).all()
            continue
        check_rows(out[a:b], x[a:b], w[g], bias[g], None, "silu")
        check_grads(dx[a:b], dw[g], db[g], dout[a:b], x[a:b], w[g], None, "none")


@gpu
@pytest.mark.parametrize("act", ["none", "gelu"])
@pytest.mark.parametrize("sizes,k,n", [([8100, 0, 5, 77], 128, 128), ([8191, 1], 72, 64),
                                       ([0, 6000, 6000], 256, 256), ([20000, 0, 11000, 70], 250, 250),
                                       ([1, 8190], 128, 128)])
def test_grouped_shared_weight_gradients(sizes, k, n, act):
    """The weight gradients of long groups share their contraction in clusters:
    groups shorter than the parts, empty ones, rows of others behind the last
    slot; the rows around the groups hold NaN."""
    gen = torch.Generator().manual_seed(sum(sizes))
    G, first, behind = len(sizes), 9, 30
    rows = first + sum(sizes) + behind
    dt = torch.float16 if act == "none" else torch.bfloat16
    x, dout = normal(gen, dt, rows, k), normal(gen, dt, rows, n)
    w = normal(gen, dt, G, k, n, std=k ** -0.5)
    pre = normal(gen, dt, rows, n) if act != "none" else None
    for t in (x, dout):
        t[:first] = math.nan
        t[rows - behind:] = math.inf
    off = offsets_of(sizes, first)
    assert tiles_of(x, w, off, act=act, dout=dout)[2][3] > 1
    dx = torch.full((rows, k), 3.0, dtype=dt, device="cuda")
    kw = dict(preact=pre, activation=act)
    _, dw, db = B.grouped_linear_backward(dout, x, off, w, dx=dx, **kw)
    assert (dx[:first] == 3).all() and (dx[rows - behind:] == 3).all()
    o = off.tolist()
    for g in range(G):
        a, b = o[g], o[g + 1]
        if a == b:
            assert (dw[g] == 0).all() and (db[g] == 0).all()
            continue
        check_grads(dx[a:b], dw[g], db[g], dout[a:b], x[a:b], w[g],
                    None if pre is None else pre[a:b], act)
    for _ in range(3):
        again = B.grouped_linear_backward(dout, x, off, w, need_dx=False, **kw)
        assert torch.equal(dw, again[1]) and torch.equal(db, again[2])
    assert B.linear_device_error() == 0


# tiles of four pairs, forward and dx; dx on four and eight CTAs
MORE_SHARED = [(192, 8192, 3000), (190, 4096, 3000), (250, 8200, 2999), (192, 2816, 8192),
               (190, 2560, 16384), (128, 2000, 4096), (16, 1000, 8192)]


@gpu
@pytest.mark.parametrize("act", ["none", "gelu"])
@pytest.mark.parametrize("rows,k,n", MORE_SHARED)
def test_linear_more_shared_tiles(rows, k, n, act):
    test_linear_shared_tiles(rows, k, n, act)


@gpu
def test_shared_tile_sizes_cover_every_share():
    """What the sizes above are there for: products on clusters of 2, 4 and 8
    CTAs and of 2 and 4 pairs, dx among them."""
    seen = set()
    for rows, k, n in SHARED + MORE_SHARED:
        x, w = (torch.empty(s, dtype=torch.bfloat16, device="cuda") for s in ((rows, k), (k, n)))
        for what, t in zip(("forward", "dx", "dw"), tiles_of(x, w, dout=x.new_empty(rows, n))):
            seen.add((what, t[0], t[3]))
    shares = {s[1:] for s in seen}
    assert {(0, 2), (0, 4), (0, 8), (1, 2), (1, 4)} <= shares
    assert {("dx", 0, 4), ("dx", 0, 8), ("dx", 1, 2), ("dx", 1, 4)} <= seen, seen


@gpu
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("rows,k,n", [(32, 4096, 1280), (1, 4096, 1280), (24, 4096, 1024),
                                      (16, 8192, 128), (8000, 64, 72), (8192, 128, 128)])
def test_two_slots_at_least(rows, k, n, residual):
    """A pipeline loads a slot while its MMAs read another."""
    x, w = (torch.empty(s, dtype=torch.bfloat16, device="cuda") for s in ((rows, k), (k, n)))
    more = x.new_empty(rows, n)
    for t in tiles_of(x, w, residual=more if residual else None, dout=more):
        assert t[4] >= 2, t


@gpu
@pytest.mark.parametrize("rows,k,n", [(2100, 1000, 2307), (1500, 1001, 2600), (2048, 520, 2314)])
def test_linear_large_odd_rows(rows, k, n):
    """Pair tiles whose outputs, residual and pre-activation allow 2- and 4-byte
    accesses only, at strides of their own."""
    gen = torch.Generator().manual_seed(rows + n)
    dt = torch.bfloat16
    x, w = normal(gen, dt, rows, k), normal(gen, dt, k, n, std=k ** -0.5)
    bias, res = normal(gen, dt, n), normal(gen, dt, rows, n + 3)[:, 1:n + 1]
    out = torch.full((rows, n + 5), 7.0, dtype=dt, device="cuda")
    pre = torch.full((rows, n + 2), 7.0, dtype=dt, device="cuda")
    B.linear(x, w, bias, residual=res, activation="gelu", out=out[:, 2:n + 2], preact=pre[:, :n])
    check_rows(out[:, 2:n + 2], x, w, bias, res, "gelu", pre[:, :n])
    assert (out[:, :2] == 7).all() and (out[:, n + 2:] == 7).all() and (pre[:, n:] == 7).all()
    dout = normal(gen, dt, rows, n)
    grads = B.linear_backward(dout, x, w, preact=pre[:, :n], activation="gelu")
    check_grads(*grads, dout, x, w, pre[:, :n], "gelu")


@gpu
@pytest.mark.parametrize("rows,k,n", [(4096, 256, 2048), (1000, 64, 520), (300, 512, 1000)])
def test_linear_large_residual_in_place(rows, k, n):
    """The residual is read several chunks of rows ahead: in place it gives the
    same bits as apart from the output."""
    gen = torch.Generator().manual_seed(rows)
    x, w = normal(gen, torch.bfloat16, rows, k), normal(gen, torch.bfloat16, k, n, std=0.1)
    res = normal(gen, torch.bfloat16, rows, n)
    want = B.linear(x, w, residual=res, activation="silu")
    check_rows(want, x, w, None, res, "silu")
    B.linear(x, w, residual=res, activation="silu", out=res)
    assert torch.equal(res, want)


@gpu
@pytest.mark.parametrize("rows", [100, 5000])
def test_bias_gradient_alone(rows):
    """db without dx and dw: the same bits as with them."""
    gen = torch.Generator().manual_seed(rows)
    dout, pre = normal(gen, torch.bfloat16, rows, 328), normal(gen, torch.bfloat16, rows, 328)
    x, w = normal(gen, torch.bfloat16, rows, 72), normal(gen, torch.bfloat16, 72, 328)
    for act in ("none", "gelu"):
        kw = dict(preact=None if act == "none" else pre, activation=act)
        db = B.linear_backward(dout, x, w, **kw)[2]
        dx, dw, alone = B.linear_backward(dout, None, w, need_dx=False, need_dw=False, **kw)
        assert dx is None and dw is None and torch.equal(alone, db)
        check_grads(None, None, db, dout, x, w, pre, act)


@gpu
@pytest.mark.parametrize("act", ["none", "gelu_tanh"])
@pytest.mark.parametrize("sizes,cols", [([20000], 1024), ([20000], 1023),
                                        ([9000, 0, 10877, 1, 129], 1024),
                                        ([127, 16500, 128, 300], 1278)])
def test_bias_gradient_of_many_rows(sizes, cols, act):
    """Chunks of 128 rows: (rows / 128 + groups) x (columns / 256) >= 512."""
    gen = torch.Generator().manual_seed(cols)
    rows = sum(sizes) + 11
    assert (rows // 128 + len(sizes)) * -(-cols // 256) >= 512
    dout, x = normal(gen, torch.bfloat16, rows, cols), normal(gen, torch.bfloat16, rows, 24)
    w = normal(gen, torch.bfloat16, len(sizes), 24, cols)
    pre = normal(gen, torch.bfloat16, rows, cols) if act != "none" else None
    off = offsets_of(sizes, 4)
    dx, dw, db = B.grouped_linear_backward(dout, x, off, w, preact=pre, activation=act)
    o = off.tolist()
    for g in range(len(sizes)):
        a, b = o[g], o[g + 1]
        if a < b:
            check_grads(dx[a:b], dw[g], db[g], dout[a:b], x[a:b], w[g],
                        None if pre is None else pre[a:b], act)
        else:
            assert (db[g] == 0).all()


@gpu
def test_backward_calls_at_once():
    """Calls on two streams, their launches interleaved by two host threads,
    give the bits of calls one after another."""
    import threading
    gen = torch.Generator().manual_seed(21)
    sets = []
    for rows, k, n in ((700, 513, 771), (1500, 640, 1288)):
        x, w = normal(gen, torch.bfloat16, rows, k), normal(gen, torch.bfloat16, k, n, std=k ** -0.5)
        dout, pre = normal(gen, torch.bfloat16, rows, n), normal(gen, torch.bfloat16, rows, n)
        sets.append((dout, x, w, pre))
    run = lambda s: B.linear_backward(*s[:3], preact=s[3], activation="silu")
    want = [run(s) for s in sets]
    torch.cuda.synchronize()
    got = [[], []]

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(20):
                got[i].append(run(sets[i]))
        torch.cuda.synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for i in range(2):
        assert len(got[i]) == 20
        for g in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(g, want[i]))
    assert B.linear_device_error() == 0


# ----------------------------------------------------------------- grouped
def offsets_of(sizes, first=0):
    o = torch.tensor([first] + list(sizes), dtype=torch.int64).cumsum(0)
    return o.to(torch.int32).cuda()


GROUPS = [
    ([1], 64, 72), ([0, 0, 3, 0], 64, 128), ([5, 1, 0, 130, 16, 17], 72, 200),
    ([300, 0, 129, 128, 1], 128, 264), ([0, 0], 64, 64), ([2] * 40, 256, 160),
    ([700, 3, 0, 41], 130, 77), ([64, 64, 64], 320, 128),
]


@gpu
@pytest.mark.parametrize("sizes,k,n", GROUPS)
@pytest.mark.parametrize("act", ["none", "gelu"])
def test_grouped_linear(sizes, k, n, act):
    gen = torch.Generator().manual_seed(sum(sizes) + k)
    G, first, behind = len(sizes), 2, 5
    rows = first + sum(sizes) + behind
    x = normal(gen, torch.bfloat16, rows, k)
    w = normal(gen, torch.bfloat16, G, k, n, std=k ** -0.5)
    bias = normal(gen, torch.bfloat16, G, n)
    res = normal(gen, torch.bfloat16, rows, n)
    off = offsets_of(sizes, first)
    # rows of no group hold NaN and must neither be read into others nor written
    x[:first] = math.nan
    x[rows - behind:] = math.inf
    out = torch.full((rows, n), 3.0, dtype=torch.bfloat16, device="cuda")
    pre = out.clone()
    B.grouped_linear(x, off, w, bias, residual=res, activation=act, out=out, preact=pre)
    assert (out[:first] == 3).all() and (out[rows - behind:] == 3).all()
    assert (pre[:first] == 3).all() and (pre[rows - behind:] == 3).all()
    o = off.tolist()
    for g in range(G):
        a, b = o[g], o[g + 1]
        check_rows(out[a:b], x[a:b], w[g], bias[g], res[a:b], act, pre[a:b])


@gpu
@pytest.mark.parametrize("sizes,k,n", GROUPS)
@pytest.mark.parametrize("act", ["none", "silu"])
def test_grouped_linear_backward(sizes, k, n, act):
    gen = torch.Generator().manual_seed(sum(sizes) + n)
    G, first, behind = len(sizes), 3, 4
    rows = first + sum(sizes) + behind
    dt = torch.float16 if k % 3 else torch.bfloat16
    x, dout = normal(gen, dt, rows, k), normal(gen, dt, rows, n)
    w = normal(gen, dt, G, k, n, std=k ** -0.5)
    pre = normal(gen, dt, rows, n) if act != "none" else None
    for t in (x, dout) + (() if pre is None else (pre,)):
        t[:first] = math.nan
        t[rows - behind:] = math.inf
    off = offsets_of(sizes, first)
    dx = torch.full((rows, k), 3.0, dtype=dt, device="cuda")
    dw = torch.full((G, k, n), 5.0, dtype=dt, device="cuda")
    got = B.grouped_linear_backward(dout, x, off, w, preact=pre, activation=act, dx=dx, dw=dw)
    assert got[0] is dx and got[1] is dw
    db = got[2]
    assert (dx[:first] == 3).all() and (dx[rows - behind:] == 3).all()
    o = off.tolist()
    for g in range(G):
        a, b = o[g], o[g + 1]
        if a == b:
            assert (dw[g] == 0).all() and (db[g] == 0).all()
            continue
        check_grads(dx[a:b], dw[g], db[g], dout[a:b], x[a:b], w[g],
                    None if pre is None else pre[a:b], act)


@gpu
@pytest.mark.parametrize("sizes,k,n", [
    ([700, 1, 0, 513, 256, 255, 900], 512, 2304), ([3, 2000, 17, 1999], 1288, 1032),
    ([1100, 900, 30], 2600, 264),
])
def test_grouped_large(sizes, k, n):
    """Ragged groups on CTA pairs; the rows around the groups hold NaN."""
    gen = torch.Generator().manual_seed(k)
    G, first, behind = len(sizes), 5, 70
    rows = first + sum(sizes) + behind
    x, dout = normal(gen, torch.bfloat16, rows, k), normal(gen, torch.bfloat16, rows, n)
    w = normal(gen, torch.bfloat16, G, k, n, std=k ** -0.5)
    for t in (x, dout):
        t[:first] = math.nan
        t[rows - behind:] = math.inf
    off = offsets_of(sizes, first)
    out = torch.full((rows, n), 3.0, dtype=x.dtype, device="cuda")
    dx = torch.full((rows, k), 3.0, dtype=x.dtype, device="cuda")
    B.grouped_linear(x, off, w, out=out)
    _, dw, db = B.grouped_linear_backward(dout, x, off, w, dx=dx)
    for t in (out, dx):
        assert (t[:first] == 3).all() and (t[rows - behind:] == 3).all()
    o = off.tolist()
    for g in range(G):
        a, b = o[g], o[g + 1]
        if a == b:
            assert (dw[g] == 0).all() and (db[g] == 0).all()
            continue
        check_rows(out[a:b], x[a:b], w[g], None, None, "none")
        check_grads(dx[a:b], dw[g], db[g], dout[a:b], x[a:b], w[g], None, "none")


@gpu
def test_grouped_neighbours_do_not_leak():
    """A group of NaN and infinities changes nothing in the groups around it."""
    gen = torch.Generator().manual_seed(11)
    sizes = [70, 9, 30]
    x, dout = normal(gen, torch.bfloat16, 109, 64), normal(gen, torch.bfloat16, 109, 128)
    w, off = normal(gen, torch.bfloat16, 3, 64, 128), offsets_of(sizes)
    out = B.grouped_linear(x, off, w)
    dx, dw, db = B.grouped_linear_backward(dout, x, off, w)
    x2, dout2, w2 = x.clone(), dout.clone(), w.clone()
    x2[70:79], dout2[70:79], w2[1] = math.nan, math.inf, math.nan
    out2 = B.grouped_linear(x2, off, w2)
    dx2, dw2, db2 = B.grouped_linear_backward(dout2, x2, off, w2)
    keep = torch.ones(109, dtype=torch.bool)
    keep[70:79] = False
    assert torch.equal(out[keep], out2[keep]) and torch.equal(dx[keep], dx2[keep])
    for a, b in ((dw, dw2), (db, db2)):
        assert torch.equal(a[0], b[0]) and torch.equal(a[2], b[2])
        assert a.shape == b.shape
    assert torch.isnan(out2[70:79]).all() and torch.isnan(dw2[1]).any()


@gpu
def test_grouped_one_group_is_linear():
    gen = torch.Generator().manual_seed(12)
    x, w = normal(gen, torch.bfloat16, 150, 96), normal(gen, torch.bfloat16, 96, 136)
    assert torch.equal(B.grouped_linear(x, offsets_of([150]), w[None]), B.linear(x, w))


@gpu
def test_grouped_many_groups():
    gen = torch.Generator().manual_seed(13)
    sizes = [int(v) for v in torch.randint(0, 3, (1024,), generator=gen)]
    rows = sum(sizes)
    x, w = normal(gen, torch.bfloat16, rows, 16), normal(gen, torch.bfloat16, 1024, 16, 24)
    off = offsets_of(sizes)
    out = B.grouped_linear(x, off, w)
    group = torch.repeat_interleave(torch.arange(1024), torch.tensor(sizes)).cuda()
    want = torch.einsum("rk,rkn->rn", x.double(), w.double()[group])
    s = torch.einsum("rk,rkn->rn", x.double().abs(), w.double().abs()[group])
    close(out, want, half_step(x.dtype) * want.abs() * 1.01 + sum_bound(16, s), "out")


@gpu
def test_grouped_weights_with_strides():
    """gate and up as halves of one [G, K, 2N] tensor."""
    gen = torch.Generator().manual_seed(14)
    sizes = [33, 0, 12]
    x, both = normal(gen, torch.bfloat16, 45, 64), normal(gen, torch.bfloat16, 3, 64, 144)
    off = offsets_of(sizes)
    for w in (both[:, :, :72], both[:, :, 72:], both[:, :, 1:73]):
        assert torch.equal(B.grouped_linear(x, off, w), B.grouped_linear(x, off, w.contiguous()))


@gpu
def test_grouped_odd_weights_of_empty_groups():
    """Weights that the kernels cannot address are copied, but not those of
    groups without rows: theirs may hold anything."""
    gen = torch.Generator().manual_seed(22)
    sizes = [0, 0, 17, 0, 1, 0, 140, 0]
    k, n = 77, 131
    x, w = normal(gen, torch.bfloat16, 158, k), normal(gen, torch.bfloat16, 8, k, n, std=0.1)
    dout, off = normal(gen, torch.bfloat16, 158, n), offsets_of(sizes)
    for g, c in enumerate(sizes):
        if c == 0:
            w[g] = math.nan
    out = B.grouped_linear(x, off, w)
    dx, dw, db = B.grouped_linear_backward(dout, x, off, w)
    o = off.tolist()
    for g, c in enumerate(sizes):
        a, b = o[g], o[g + 1]
        if c == 0:
            assert (dw[g] == 0).all() and (db[g] == 0).all()
            continue
        check_rows(out[a:b], x[a:b], w[g], None, None, "none")
        check_grads(dx[a:b], dw[g], db[g], dout[a:b], x[a:b], w[g], None, "none")


@gpu
def test_bad_offsets_stay_inside():
    """Offsets that decrease or pass the ends are clamped: nothing outside the
    outputs is written and every group's gradient is finite."""
    gen = torch.Generator().manual_seed(15)
    x, w = normal(gen, torch.bfloat16, 60, 64), normal(gen, torch.bfloat16, 4, 64, 72)
    dout = normal(gen, torch.bfloat16, 60, 72)
    off = torch.tensor([-7, 50, 20, 90, 10], dtype=torch.int32, device="cuda")
    wide = torch.full((80, 72), 9.0, dtype=torch.bfloat16, device="cuda")
    B.grouped_linear(x, off, w, out=wide[10:70])
    assert (wide[:10] == 9).all() and (wide[70:] == 9).all()
    # clamped: [0, 50), [50, 50), [50, 60), [60, 60)
    check_rows(wide[10:60], x[:50], w[0], None, None, "none")
    check_rows(wide[60:70], x[50:], w[2], None, None, "none")
    dx, dw, db = B.grouped_linear_backward(dout, x, off, w)
    check_grads(dx[:50], dw[0], db[0], dout[:50], x[:50], w[0], None, "none")
    assert (dw[1] == 0).all() and (dw[3] == 0).all() and (db[1] == 0).all()


@gpu
def test_no_rows():
    dt = torch.bfloat16
    x, w = torch.empty(0, 16, dtype=dt, device="cuda"), torch.ones(2, 16, 24, dtype=dt, device="cuda")
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    assert B.grouped_linear(x, off, w).shape == (0, 24)
    dx, dw, db = B.grouped_linear_backward(torch.empty(0, 24, dtype=dt, device="cuda"), x, off, w)
    assert dx.shape == (0, 16) and (dw == 0).all() and (db == 0).all()
    assert B.linear(x, w[0]).shape == (0, 24)
    assert B.swiglu(x, x).shape == (0, 16)
    torch.cuda.synchronize()


@gpu
def test_long_contraction_of_small_outputs():
    """Few tiles, long sums: the split over a cluster."""
    gen = torch.Generator().manual_seed(16)
    x, w = normal(gen, torch.bfloat16, 3, 16384), normal(gen, torch.bfloat16, 16384, 100, std=0.01)
    check_rows(B.linear(x, w), x, w, None, None, "none")
    x, dout = normal(gen, torch.bfloat16, 8000, 64), normal(gen, torch.bfloat16, 8000, 72)
    _, dw, db = B.linear_backward(dout, x, torch.zeros(64, 72, dtype=x.dtype, device="cuda"),
                                  need_dx=False)
    check_grads(None, dw, db, dout, x, None, None, "none")


@gpu
def test_same_bits_every_time():
    gen = torch.Generator().manual_seed(17)
    sizes = [100, 0, 257, 3]
    x, w = normal(gen, torch.bfloat16, 360, 200), normal(gen, torch.bfloat16, 4, 200, 300)
    dout, off = normal(gen, torch.bfloat16, 360, 300), offsets_of(sizes)
    first = (B.grouped_linear(x, off, w),) + B.grouped_linear_backward(dout, x, off, w)
    for _ in range(3):
        again = (B.grouped_linear(x, off, w),) + B.grouped_linear_backward(dout, x, off, w)
        assert all(torch.equal(a, b) for a, b in zip(first, again))


@gpu
def test_graphs_and_streams():
    """Captured calls replay on new inputs, two graphs and an eager call keep
    their own workspaces, and a call on a given stream is ordered on it."""
    gen = torch.Generator().manual_seed(18)
    # misaligned weights: both directions need a workspace
    x, w = normal(gen, torch.bfloat16, 40, 64), normal(gen, torch.bfloat16, 64, 83)[:, 2:]
    dout, pre = normal(gen, torch.bfloat16, 40, 81), normal(gen, torch.bfloat16, 40, 81)
    x2 = normal(gen, torch.bfloat16, 40, 64)

    def step(a):
        return (B.linear(a, w, activation="silu"),) + \
            B.linear_backward(dout, a, w, preact=pre, activation="silu")

    want, want2 = step(x), step(x2)
    graphs, outs, statics = [], [], []
    for _ in range(2):
        static = x.clone()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step(static))
        graphs.append(g)
        statics.append(static)
    statics[1].copy_(x2)
    torch.cuda.synchronize()
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for g, s in zip(graphs, side):
            with torch.cuda.stream(s):
                g.replay()
        eager = step(x)
    torch.cuda.synchronize()
    for got, ref in ((outs[0], want), (outs[1], want2), (eager, want)):
        assert all(torch.equal(a, b) for a, b in zip(got, ref))
    s = torch.cuda.Stream()
    big = torch.empty(1 << 26, device="cuda")
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(20):
            big.fill_(1.0)
        late = x2.clone()
    got = B.linear(late, w, activation="silu", stream=s)  # waits for late: the same stream
    s.synchronize()
    assert torch.equal(got, want2[0])
    assert B.linear_device_error() == 0


# ----------------------------------------------------------------- swiglu
def swiglu64(gate, up, scale, limit):
    a = gate.clamp(max=limit) if limit > 0 else gate
    v = up.clamp(-limit, limit) if limit > 0 else up
    y = a * torch.sigmoid(a) * v
    return y if scale is None else y * scale[:, None]


SW_DT = {"f32": torch.float32, **DT}


@gpu
@pytest.mark.parametrize("dtype", list(SW_DT))
@pytest.mark.parametrize("rows,width", [(1, 1), (1, 1280), (3, 77), (50, 256), (33, 2600)])
@pytest.mark.parametrize("limit,scaled", [(0.0, False), (0.0, True), (1.5, True)])
def test_swiglu(rows, width, limit, scaled, dtype):
    gen = torch.Generator().manual_seed(rows + width)
    dt = SW_DT[dtype]
    u = half_step(dt)
    both = normal(gen, dt, rows, 2 * width, std=2.0)
    gate, up = both[:, :width], both[:, width:]
    scale = torch.rand(rows, generator=gen).cuda() if scaled else None
    dout = normal(gen, dt, rows, width)
    out = B.swiglu(gate, up, scale, limit=limit)
    dgate, dup, dscale = B.swiglu_backward(dout, gate, up, scale, limit=limit)
    g, v = (t.double().clone().requires_grad_(True) for t in (gate, up))
    s = None if scale is None else scale.double().clone().requires_grad_(True)
    want = swiglu64(g, v, s, limit)
    want.backward(dout.double())
    # a handful of fp32 roundings (2^-24 each, the sigmoid's 2^-21), one to the type
    rel = u * 1.01 + 2.0 ** -20
    sc = 1.0 if scale is None else scale.double()[:, None]
    tiny = torch.finfo(dt).tiny * u * 2
    close(out, want.detach(), rel * want.detach().abs() + tiny, "out")
    # dgate's bracket 1 + a (1 - sigmoid) can cancel: its error is that of its terms
    d, gd, ud = dout.double().abs(), g.detach(), v.detach()
    a = gd.clamp(max=limit) if limit > 0 else gd
    b = (ud.clamp(-limit, limit) if limit > 0 else ud).abs()
    p = torch.sigmoid(a)
    terms = d * sc * b * p * (1 + a.abs() * (1 - p))
    close(dgate, g.grad, u * g.grad.abs() * 1.01 + 2.0 ** -20 * terms + tiny, "dgate")
    close(dup, v.grad, rel * v.grad.abs() + tiny, "dup")
    if scaled:
        sums = (d * (a * p).abs() * b).sum(1)
        close(dscale, s.grad, (2.0 ** -20 + (width / 32 + 16) * 2.0 ** -24) * sums, "dscale")
    else:
        assert dscale is None


@gpu
@pytest.mark.parametrize("dtype", list(SW_DT))
@pytest.mark.parametrize("rows,width", [(1024, 256), (1500, 1280), (2051, 77), (4099, 8)])
@pytest.mark.parametrize("limit,scaled", [(0.0, True), (1.5, True), (1.5, False)])
def test_swiglu_many_rows(rows, width, limit, scaled, dtype):
    """A warp per row from 1024 rows on."""
    test_swiglu(rows, width, limit, scaled, dtype)


@gpu
@pytest.mark.parametrize("width", [72, 77])
def test_swiglu_many_rows_of_no_group_and_in_place(width):
    gen = torch.Generator().manual_seed(22)
    gate, up, dout = (normal(gen, torch.float16, 1300, width) for _ in range(3))
    scale, off = torch.rand(1300, generator=gen).cuda(), offsets_of([600, 0, 650], 20)
    want, grads = B.swiglu(gate, up, scale), B.swiglu_backward(dout, gate, up, scale)
    out, into = torch.full_like(gate, 3.0), [torch.full_like(gate, 3.0), torch.full_like(gate, 3.0),
                                             torch.full((1300,), 3.0, device="cuda")]
    B.swiglu(gate, up, scale, offsets=off, out=out)
    B.swiglu_backward(dout, gate, up, scale, offsets=off, dgate=into[0], dup=into[1], dscale=into[2])
    for t, ref in zip([out] + into, (want,) + grads):
        assert (t[:20] == 3).all() and (t[1270:] == 3).all() and torch.equal(t[20:1270], ref[20:1270])
    g2, u2, d2 = gate.clone(), up.clone(), dout.clone()
    ds = B.swiglu_backward(d2, g2, u2, scale, dgate=g2, dup=d2)[2]
    assert torch.equal(g2, grads[0]) and torch.equal(d2, grads[1]) and torch.equal(ds, grads[2])
    assert torch.equal(B.swiglu(gate, up, scale, out=gate), want)


@gpu
def test_swiglu_rows_of_no_group_and_in_place():
    gen = torch.Generator().manual_seed(21)
    gate, up = normal(gen, torch.bfloat16, 30, 64), normal(gen, torch.bfloat16, 30, 64)
    scale, dout = torch.rand(30, generator=gen).cuda(), normal(gen, torch.bfloat16, 30, 64)
    off = torch.tensor([4, 9, 25], dtype=torch.int32, device="cuda")
    want = B.swiglu(gate, up, scale)
    grads = B.swiglu_backward(dout, gate, up, scale)
    out = torch.full_like(gate, 3.0)
    B.swiglu(gate, up, scale, offsets=off, out=out)
    assert (out[:4] == 3).all() and (out[25:] == 3).all() and torch.equal(out[4:25], want[4:25])
    into = [torch.full_like(gate, 3.0), torch.full_like(gate, 3.0),
            torch.full((30,), 3.0, device="cuda")]
    B.swiglu_backward(dout, gate, up, scale, offsets=off, dgate=into[0], dup=into[1],
                      dscale=into[2])
    for t, ref in zip(into, grads):
        assert (t[:4] == 3).all() and (t[25:] == 3).all() and torch.equal(t[4:25], ref[4:25])
    g2, u2, d2 = gate.clone(), up.clone(), dout.clone()
    assert torch.equal(B.swiglu(g2, u2, scale, out=g2), want)
    g2 = gate.clone()
    B.swiglu_backward(d2, g2, u2, scale, dgate=g2, dup=u2)
    assert torch.equal(g2, grads[0]) and torch.equal(u2, grads[1])
    # into the halves of one tensor, as one product's output
    both = torch.cat([gate, up], 1)
    halves = torch.empty_like(both)
    B.swiglu_backward(dout, both[:, :64], both[:, 64:], scale, dgate=halves[:, :64],
                      dup=halves[:, 64:])
    assert torch.equal(halves, torch.cat(grads[:2], 1))


@gpu
def test_swiglu_clamp_edges_and_nan():
    """At the limit itself the gradient passes; NaN passes the clamp."""
    dt = torch.bfloat16
    gate = torch.tensor([[7.0, 7.0625, -9.0, math.nan, 1.0]], dtype=dt, device="cuda")
    up = torch.tensor([[7.0, 1.0, -7.0625, 1.0, math.nan]], dtype=dt, device="cuda")
    out = B.swiglu(gate, up, limit=7.0)
    assert torch.isnan(out[0]).tolist() == [False, False, False, True, True]
    dgate, dup, _ = B.swiglu_backward(torch.ones_like(gate), gate, up, limit=7.0)
    assert dgate[0, 0] != 0 and dgate[0, 1] == 0 and dgate[0, 2] != 0
    assert dup[0, 0] != 0 and dup[0, 1] != 0 and dup[0, 2] == 0


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_gelu_keeps_its_tail(dtype):
    """gelu's relative error below zero, where 1 + erf would cancel: one rounding
    to the type, and in fp32 2^-17: the polynomial 3.2e-7, the exponent 26 at most
    with two roundings of 2^-24 and its constant's 2^-25 (26 * 2.5 * 2^-24 ln 2 =
    2.7e-6), reciprocal, exponential and the polynomial's steps 2^-22 each."""
    dt = DT[dtype]
    z = -torch.linspace(2.0 ** -6, 6.0, 64 * 64).reshape(64, 64).to(dt).cuda()
    out = B.linear(z, torch.eye(64, dtype=dt, device="cuda"), activation="gelu")
    want = act64(z.double(), "gelu")
    u, tiny = half_step(dt), torch.finfo(dt).tiny
    close(out, want, (u * 1.01 + 2.0 ** -17) * want.abs() + tiny * u * 2, "gelu")


@gpu
def test_silu_far_below_zero():
    """Where 1 + exp(-z) passes 2^126 the reciprocal is no normal number, but silu
    is (-5e-37 at -88) and bf16 holds it."""
    dt = torch.bfloat16
    z = torch.tensor([[-80.0, -86.5, -87.0, -87.5, -88.0, -88.5, -1.0, 0.0]], dtype=dt, device="cuda")
    one, eye = torch.ones_like(z), torch.eye(8, dtype=dt, device="cuda")
    want = act64(z.double(), "silu")
    # the exponent's rounding, 2^-18 of 2^x at |x| < 128 and log2(e)'s as much again
    bound = (half_step(dt) + 2.0 ** -16) * want.abs()
    close(B.swiglu(z, one), want, bound, "swiglu")
    close(B.swiglu_backward(one, z, one)[1], want, bound, "dup")
    x = torch.zeros(1, 8, dtype=dt, device="cuda")
    close(B.linear(x, eye, z[0].contiguous(), activation="silu"), want, bound, "linear")
    slope = slope64(z.double(), "silu")
    bound = (half_step(dt) + 2.0 ** -16) * slope.abs()
    close(B.swiglu_backward(one, z, one)[0], slope, bound, "dgate")
    # (dz is rounded, times one in dx)
    dx, _, db = B.linear_backward(one, None, eye, preact=z, activation="silu", need_dw=False)
    close(dx, slope, bound, "dx")
    close(db[None], slope, bound, "db")


# ------------------------------------------------------------ a run of them together
@gpu
def test_expert_ffn_forward_matches_the_layer():
    """The layer's experts from its own routing and the stand-alone operators:
    gather, gate and up products, SwiGLU with the gate weights, down product,
    sum per token."""
    T, H, E, k, I, L = 96, 256, 12, 4, 128, 2.0
    gen = torch.Generator().manual_seed(30)
    x = normal(gen, torch.bfloat16, T, H)
    rw, rb = normal(gen, torch.float32, H, E, std=0.05), normal(gen, torch.float32, E, std=0.1)
    wg, wu = (normal(gen, torch.bfloat16, E, H, I, std=0.08) for _ in range(2))
    wd = normal(gen, torch.bfloat16, E, I, H, std=0.08)
    sg, su = (normal(gen, torch.bfloat16, H, I, std=0.08) for _ in range(2))
    sd = normal(gen, torch.bfloat16, I, H, std=0.08)
    layer = B.MoeLayer(B.make_config(H, E, k, I, swiglu_limit=L, swiglu_limit_shared=L))
    layer.load_weights(rw, rb, wg, wu, wd, sg, su, sd)
    want, rt = layer.forward(x, routing=True)
    off, perm = rt["offsets"], rt["perm"].long()
    rows = x[perm // k]
    h = B.swiglu(B.grouped_linear(rows, off, wg), B.grouped_linear(rows, off, wu),
                 rt["topk_w"].flatten()[perm], limit=L)
    y = B.grouped_linear(h, off, wd)
    shared = B.swiglu(B.linear(x, sg), B.linear(x, su), limit=L)
    out = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    out.index_add_(0, perm // k, y.double())
    out += B.linear(shared, sd).double()
    # gate, up, h and y each rounded to bf16 on either side: 2^-8 of values whose
    # errors are independent; ten of them stay under 10 * 2^-9 of the norm
    off_by = (out - want.double()).norm() / want.double().norm()
    assert float(off_by) < 10 * 2.0 ** -9
    layer.close()


@gpu
def test_expert_ffn_gradients():
    """A training step's gradients of routed experts (inputs, weights, gate
    weights) against autograd of the definition in 64 bits."""
    gen = torch.Generator().manual_seed(31)
    sizes, H, I, L = [40, 0, 7, 65], 96, 72, 3.0
    R, G = sum(sizes), len(sizes)
    off = offsets_of(sizes)
    dt = torch.float16
    x, s = normal(gen, dt, R, H), torch.rand(R, generator=gen).cuda() + 0.1
    w13, w2 = normal(gen, dt, G, H, 2 * I, std=0.15), normal(gen, dt, G, I, H, std=0.15)
    dout = normal(gen, dt, R, H)
    gu = B.grouped_linear(x, off, w13)
    h = B.swiglu(gu[:, :I], gu[:, I:], s, limit=L)
    y = B.grouped_linear(h, off, w2)
    dh, dw2, _ = B.grouped_linear_backward(dout, h, off, w2, need_db=False)
    dgu = torch.empty_like(gu)
    _, _, ds = B.swiglu_backward(dh, gu[:, :I], gu[:, I:], s, limit=L, dgate=dgu[:, :I],
                                 dup=dgu[:, I:])
    dx, dw13, _ = B.grouped_linear_backward(dgu, x, off, w13, need_db=False)
    xd, sd, ad, bd = (t.double().clone().requires_grad_(True) for t in (x, s, w13, w2))
    want, o = [], off.tolist()
    for g in range(G):
        z = xd[o[g]:o[g + 1]] @ ad[g]
        want.append(swiglu64(z[:, :I], z[:, I:], sd[o[g]:o[g + 1]], L) @ bd[g])
    want = torch.cat(want)
    want.backward(dout.double())
    # up to five roundings of 2^-11 in a chain, each relative to values of its own
    # size: independent errors, 5 * 2^-11 of the norm bounds their sum (and the few
    # clamped elements whose side a rounding changes are within the same share)
    for got, ref, name in ((y, want.detach(), "y"), (dx, xd.grad, "dx"), (ds, sd.grad, "dscale"),
                           (dw13, ad.grad, "dw13"), (dw2, bd.grad, "dw2")):
        off_by = float((got.double() - ref).norm() / ref.norm())
        assert off_by < 5 * 2.0 ** -11, (name, off_by)


# ----------------------------------------------------------------- refusals (no GPU)
@pytest.fixture(scope="module")
def lib():
    import os
    if not os.path.exists(B.LIB_PATH):
        from sparse_moe_layer_gemm_b200.build import build
        build()
    return B.load_library()


def _cfg(**kw):
    base = dict(rows=4, in_features=64, out_features=72, groups=0, dtype=B.MOE_BF16, activation=0)
    base.update(kw)
    return B.moe_linear_config_t(*base.values())


@pytest.mark.parametrize("kw,want", [
    (dict(), "MOE_OK"), (dict(rows=0), "MOE_OK"), (dict(dtype=3), "MOE_OK"),
    (dict(groups=1024), "MOE_OK"),
    (dict(rows=-1), "MOE_ERR_INVALID_ARG"), (dict(in_features=0), "MOE_ERR_INVALID_ARG"),
    (dict(out_features=0), "MOE_ERR_INVALID_ARG"), (dict(groups=-1), "MOE_ERR_INVALID_ARG"),
    (dict(activation=5), "MOE_ERR_INVALID_ARG"), (dict(activation=-1), "MOE_ERR_INVALID_ARG"),
    (dict(dtype=4), "MOE_ERR_INVALID_ARG"), (dict(dtype=0), "MOE_ERR_UNSUPPORTED"),
    (dict(dtype=2), "MOE_ERR_UNSUPPORTED"), (dict(groups=1025), "MOE_ERR_UNSUPPORTED"),
    (dict(rows=(1 << 24) + 1), "MOE_ERR_UNSUPPORTED"),
    (dict(in_features=65537), "MOE_ERR_UNSUPPORTED"),
])
def test_linear_config_check(lib, kw, want):
    import ctypes
    assert lib.moe_linear_config_check(ctypes.byref(_cfg(**kw))) == getattr(B, want)


# made-up device addresses: every call below is refused on the host
X, W, OUT, OFF, RES, PRE, BIAS = (0x10000000 * (i + 1) for i in range(7))


def _args(**kw):
    base = dict(x=X, ld_x=64, offsets=None, w=W, ld_w=72, group_stride_w=0, bias=None,
                residual=None, ld_residual=0, out=OUT, ld_out=72, preact=None, ld_preact=0)
    base.update(kw)
    return B.moe_linear_args_t(*base.values())


@pytest.mark.parametrize("cfg,kw", [
    ({}, dict(x=None)), ({}, dict(w=None)), ({}, dict(out=None)), ({}, dict(ld_x=63)),
    ({}, dict(ld_w=71)), ({}, dict(ld_out=71)), ({}, dict(x=X + 1)), ({}, dict(offsets=OFF)),
    ({}, dict(out=X)), ({}, dict(out=W + 16)), ({}, dict(ld_out=1 << 32)),
    ({}, dict(residual=RES, ld_residual=10)), ({}, dict(preact=PRE, ld_preact=10)),
    ({}, dict(out=X + 100, ld_x=256, ld_out=256)), ({}, dict(out=X + 256, ld_out=80)),
    ({}, dict(preact=OUT, ld_preact=72)), ({}, dict(residual=OUT + 16, ld_residual=72)),
    (dict(groups=2), dict()), (dict(groups=2), dict(offsets=OFF, group_stride_w=100)),
    (dict(groups=2), dict(offsets=OFF + 2, group_stride_w=64 * 72)),
])
def test_linear_refuses(lib, cfg, kw):
    import ctypes
    c, a, n = _cfg(**cfg), _args(**kw), ctypes.c_size_t()
    assert lib.moe_linear_workspace_size(ctypes.byref(c), ctypes.byref(a), ctypes.byref(n)) == \
        B.MOE_ERR_INVALID_ARG
    assert lib.moe_linear(ctypes.byref(c), ctypes.byref(a), None, 0, None) == B.MOE_ERR_INVALID_ARG


def test_slices_of_one_tensor_are_apart(lib):
    """Columns of the same rows do not overlap, whatever their extents."""
    import ctypes
    n = ctypes.c_size_t()
    for kw in (dict(ld_x=256, out=X + 2 * 128, ld_out=256),          # x | out in rows of 256
               dict(x=X + 2 * 160, ld_x=256, out=X + 2 * 16, ld_out=256),
               dict(w=X + 2 * 64, ld_w=256, ld_x=256, out=X + 2 * 176, ld_out=256,
                    residual=X + 2 * 256 * 64, ld_residual=256)):
        c, a = _cfg(), _args(**kw)
        assert lib.moe_linear_workspace_size(ctypes.byref(c), ctypes.byref(a), ctypes.byref(n)) \
            == B.MOE_OK, kw
    c = _cfg(rows=1)
    for at, want in ((128, B.MOE_OK), (126, B.MOE_ERR_INVALID_ARG)):  # one row of 64, then out
        a = _args(out=X + at)
        assert lib.moe_linear_workspace_size(ctypes.byref(c), ctypes.byref(a), ctypes.byref(n)) \
            == want


def test_tiles_refuse_what_the_calls_refuse(lib):
    c, t = _cfg(), B.moe_linear_tiles_t()
    assert lib.moe_linear_tiles(c, _args(), None) == B.MOE_ERR_INVALID_ARG
    assert lib.moe_linear_tiles(c, _args(ld_x=63), t) == B.MOE_ERR_INVALID_ARG
    assert lib.moe_linear_backward_tiles(c, _grads(), t, None) == B.MOE_ERR_INVALID_ARG
    assert lib.moe_linear_backward_tiles(c, _grads(dout=None), t, t) == B.MOE_ERR_INVALID_ARG
    t.rows = 7
    assert lib.moe_linear_tiles(_cfg(rows=0), _args(), t) == B.MOE_OK and t.rows == 0


def test_linear_workspace(lib):
    """Aligned operands need none; a misaligned one needs its copy, and a call
    without it is refused."""
    import ctypes
    n = ctypes.c_size_t()

    def size(c, a):
        assert lib.moe_linear_workspace_size(ctypes.byref(c), ctypes.byref(a),
                                             ctypes.byref(n)) == B.MOE_OK
        return n.value

    assert size(_cfg(), _args()) == 0
    assert size(_cfg(rows=0), _args(x=None)) == 0
    assert size(_cfg(), _args(x=X + 2)) >= 4 * 64 * 2
    assert size(_cfg(), _args(ld_w=73)) >= 64 * 72 * 2
    c, a = _cfg(), _args(ld_w=73)
    assert lib.moe_linear(ctypes.byref(c), ctypes.byref(a), None, 0, None) == B.MOE_ERR_WORKSPACE
    assert lib.moe_linear(ctypes.byref(c), ctypes.byref(a), ctypes.c_void_p(0x90000001), 1 << 20,
                          None) == B.MOE_ERR_WORKSPACE


def _grads(**kw):
    base = dict(dout=OUT, ld_dout=72, x=X, ld_x=64, offsets=None, w=W, ld_w=72, group_stride_w=0,
                preact=None, ld_preact=0, dx=RES, ld_dx=64, dw=PRE, dbias=BIAS)
    base.update(kw)
    return B.moe_linear_grads_t(*base.values())


@pytest.mark.parametrize("cfg,kw", [
    ({}, dict(dout=None)), ({}, dict(x=None)), ({}, dict(w=None)), ({}, dict(ld_dout=71)),
    ({}, dict(ld_dx=63)), ({}, dict(preact=OFF, ld_preact=72)), (dict(activation=2), dict()),
    ({}, dict(dx=OUT)), ({}, dict(dw=X)), ({}, dict(dbias=PRE)), ({}, dict(dx=X)),
    (dict(groups=3), dict()), ({}, dict(offsets=OFF)),
])
def test_linear_backward_refuses(lib, cfg, kw):
    import ctypes
    c, a, n = _cfg(**cfg), _grads(**kw), ctypes.c_size_t()
    assert lib.moe_linear_backward_workspace_size(ctypes.byref(c), ctypes.byref(a),
                                                  ctypes.byref(n)) == B.MOE_ERR_INVALID_ARG
    assert lib.moe_linear_backward(ctypes.byref(c), ctypes.byref(a), None, 0, None) == \
        B.MOE_ERR_INVALID_ARG


def test_linear_backward_workspace(lib):
    import ctypes
    n = ctypes.c_size_t()

    def size(c, a):
        assert lib.moe_linear_backward_workspace_size(ctypes.byref(c), ctypes.byref(a),
                                                      ctypes.byref(n)) == B.MOE_OK
        return n.value

    assert size(_cfg(), _grads(dbias=None)) == 0
    assert size(_cfg(), _grads(x=None, dw=None, dbias=None)) == 0
    assert size(_cfg(), _grads(w=None, dx=None, dbias=None)) == 0
    with_dz = size(_cfg(activation=2), _grads(preact=OFF, ld_preact=72, dbias=None))
    assert with_dz >= 4 * 72 * 2
    # no dz where only the bias gradient is wanted
    assert size(_cfg(activation=2), _grads(preact=OFF, ld_preact=72, w=None, dx=None, x=None,
                                           dw=None)) == 0
    # the column sums of many rows meet in the workspace
    c, a = _cfg(rows=200), _grads()
    assert size(c, a) >= 200 // 32 * 72 * 4
    assert lib.moe_linear_backward(ctypes.byref(c), ctypes.byref(a), None, 0, None) == \
        B.MOE_ERR_WORKSPACE


def test_swiglu_refuses(lib):
    import ctypes

    def fwd(cfg=(4, 64, 0, 1, 0.0), gate=X, ldg=64, up=W, ldu=64, scale=None, off=None, out=OUT,
            ldo=64):
        c = B.moe_swiglu_config_t(*cfg)
        return lib.moe_swiglu(ctypes.byref(c), gate, ldg, up, ldu, scale, off, out, ldo, None)

    bad = B.MOE_ERR_INVALID_ARG
    assert lib.moe_swiglu(None, X, 64, W, 64, None, None, OUT, 64, None) == bad
    assert fwd(cfg=(0, 64, 0, 1, 0.0), gate=None) == B.MOE_OK
    for kw in (dict(cfg=(-1, 64, 0, 1, 0.0)), dict(cfg=(4, 0, 0, 1, 0.0)),
               dict(cfg=(4, 64, 0, 4, 0.0)), dict(cfg=(4, 64, 0, 1, -1.0)),
               dict(cfg=(4, 64, 0, 1, math.nan)), dict(cfg=(4, 64, 2, 1, 0.0)), dict(off=OFF),
               dict(gate=None), dict(up=None), dict(out=None), dict(ldg=63), dict(ldo=10),
               dict(gate=X + 1), dict(out=X + 16), dict(scale=OUT)):
        assert fwd(**kw) == bad, kw
    for cfg in ((4, 64, 0, 2, 0.0), ((1 << 24) + 1, 64, 0, 1, 0.0), (4, 65537, 0, 1, 0.0)):
        assert fwd(cfg=cfg) == B.MOE_ERR_UNSUPPORTED

    def bwd(dgate=RES, dup=PRE, dscale=None, dout=OUT, ldd=64):
        c = B.moe_swiglu_config_t(4, 64, 0, 1, 0.0)
        return lib.moe_swiglu_backward(ctypes.byref(c), dout, ldd, X, 64, W, 64, None, None,
                                       dgate, 64, dup, 64, dscale, None)

    for kw in (dict(dgate=None), dict(dup=None), dict(dup=RES), dict(dgate=X + 32),
               dict(dout=None), dict(ldd=3), dict(dscale=X), dict(dscale=RES), dict(dscale=BIAS + 2)):
        assert bwd(**kw) == bad, kw


def test_tensors_are_recorded_on_a_given_stream(monkeypatch):
    """Fakes in place of the device: what a call on another stream uses is
    recorded on it, after the call; on the current stream nothing is."""
    import contextlib
    done = []

    class Stream:
        device = "cuda:0"

    class Tensor:
        device = "cuda:0"

        def __init__(self, name):
            self.name = name

        def record_stream(self, s):
            done.append((self.name, s))

    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "device", lambda d: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d: Stream())
    s = Stream()
    with B._Elsewhere(Tensor("x"), s, Tensor("w"), None, Tensor("out")):
        done.append("call")
    assert done == ["call", ("x", s), ("w", s), ("out", s)]
    done.clear()
    with B._Elsewhere(Tensor("x"), None, Tensor("w")):
        pass
    assert done == []


@gpu
@pytest.mark.parametrize("call", ["linear", "grouped_backward", "swiglu", "swiglu_backward"])
def test_dropped_tensors_of_a_call_on_another_stream(call):
    """Tensors dropped right after a call on another stream keep their memory
    until that call is done."""
    gen = torch.Generator().manual_seed(40)
    rows, k = 4096, 512
    a, b = normal(gen, torch.bfloat16, rows, k), normal(gen, torch.bfloat16, rows, k)
    c, w = normal(gen, torch.bfloat16, rows, k), normal(gen, torch.bfloat16, k, k, std=0.05)
    off = offsets_of([rows])

    def run(a, b, c, w, off, **kw):
        if call == "linear":
            return (B.linear(a, w, residual=b, **kw),)
        if call == "grouped_backward":
            return B.grouped_linear_backward(a, b, off, w[None], preact=c, activation="silu", **kw)
        if call == "swiglu":
            return (B.swiglu(a, b, **kw),)
        return B.swiglu_backward(a, b, c, **kw)[:2]

    want = run(a, b, c, w, off)
    s, busy = torch.cuda.Stream(), torch.empty(1 << 28, device="cuda")
    copies = [t.clone() for t in (a, b, c, w, off)]
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(20):  # some milliseconds, so that the call has not begun below
            busy.fill_(1.0)
    got = run(*copies, stream=s)
    del copies
    # memory that may be the dropped tensors', overwritten on the current stream
    spoilt = [torch.full((rows, k), math.nan, dtype=a.dtype, device="cuda") for _ in range(8)]
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    del spoilt


@pytest.mark.parametrize("status,word,want", [
    (0, 0, 0), ("MOE_ERR_DEVICE_TIMEOUT", 3, 3), ("MOE_ERR_CUDA", 0, None),
    ("MOE_ERR_UNSUPPORTED", 0, None)])
def test_device_error_that_could_not_be_read(monkeypatch, status, word, want):
    """A status word that could not be read is an error, not 0."""
    import contextlib
    code = status if status == 0 else getattr(B, status)

    class Library:
        @staticmethod
        def moe_linear_get_device_error(p):
            p._obj.value = word
            return code

    monkeypatch.setattr(B, "load_library", lambda: Library)
    monkeypatch.setattr(B, "status_string", str)
    monkeypatch.setattr(torch.cuda, "device", lambda d: contextlib.nullcontext())
    if want is None:
        with pytest.raises(B.MoeError):
            B.linear_device_error()
    else:
        assert B.linear_device_error() == want


def test_python_refusals_on_the_host():
    x, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(64, 72, dtype=torch.bfloat16)
    for call in (lambda: B.linear(x, w),                               # not on a GPU
                 lambda: B.linear(x, w, activation="tanh"),
                 lambda: B.linear(x.float(), w),
                 lambda: B.linear(x, w.t()),
                 lambda: B.linear(x.t().contiguous().t(), w),          # columns, not rows
                 lambda: B.linear(x[0], w),
                 lambda: B.linear(x, w, bias=torch.zeros(71, dtype=torch.bfloat16)),
                 lambda: B.linear(x, w, residual=torch.zeros(4, 71, dtype=torch.bfloat16)),
                 lambda: B.grouped_linear(x, None, w[None]),
                 lambda: B.grouped_linear(x, torch.zeros(2, dtype=torch.int64), w[None]),
                 lambda: B.grouped_linear(x, torch.zeros(3, dtype=torch.int32), w[None]),
                 lambda: B.grouped_linear(x, torch.zeros(1, dtype=torch.int32), w[None][:0]),
                 lambda: B.linear(x.expand(2, 4, 64)[:, 0], w[:, :1].expand(64, 72)),
                 lambda: B.linear_backward(torch.zeros(4, 72, dtype=torch.bfloat16), None, w),
                 lambda: B.linear_backward(torch.zeros(4, 72, dtype=torch.bfloat16), x, w,
                                           activation="relu"),
                 lambda: B.swiglu(x, x[:3]),
                 lambda: B.swiglu(x.double(), x.double()),
                 lambda: B.swiglu(x, x, torch.zeros(4)[:3]),
                 lambda: B.swiglu(x, x, offsets=torch.zeros(1, dtype=torch.int32)),
                 lambda: B.swiglu_backward(x, x, x, dscale=torch.zeros(4))):
        with pytest.raises(ValueError):
            call()
